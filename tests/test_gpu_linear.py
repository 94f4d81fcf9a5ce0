"""moe_linear and moe_grouped_linear on the GPU against 64-bit references whose bounds count the
operators' roundings (tests/linear_cases.py)."""
import math
import os
import random
import subprocess
import sys
import threading

import pytest
import torch

from mixture_experts_layer_05_gb300 import binding, configs, inputs
from tests.linear_cases import ACTS, BF16, Linear

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _status(ws):
    return binding.moe_get_device_status(ws)


# ------------------------------------------------------------------------------ dense
@pytest.mark.parametrize("T", [1, 2, 7, 8, 15, 16, 17, 31, 33, 48, 63, 64, 65, 96, 127, 128, 129, 160,
                               200, 255, 256, 257, 300, 384, 511, 520, 777, 1025])
@pytest.mark.parametrize("K,N", [(8, 1), (64, 128), (72, 130), (520, 257), (1024, 640)])
def test_linear(cuda_lib, T, K, N):
    c = Linear(T, K, N)
    c.check(c.call(binding))


@pytest.mark.parametrize("T,K,N", [(1, 4096, 6144), (3, 7168, 2048), (16, 14336, 4096), (5, 2048, 28672),
                                   (130, 4096, 4096), (640, 2048, 8200), (2100, 1032, 5000)])
def test_linear_wide(cuda_lib, T, K, N):
    c = Linear(T, K, N, residual=True)
    c.check(c.call(binding))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("bias,residual,weighted", [(False, False, False), (True, False, False),
                                                    (False, True, False), (False, False, True),
                                                    (True, True, True)])
@pytest.mark.parametrize("T", [1, 21, 140, 530])
@pytest.mark.parametrize("fp8", [False, True])
def test_linear_epilogues(cuda_lib, act, bias, residual, weighted, T, fp8):
    for K, N in ((256, 256), (384, 768)):
        c = Linear(T, K, N, act=act, bias=bias, residual=residual, weighted=weighted, fp8=fp8)
        c.check(c.call(binding))


@pytest.mark.parametrize("N", [32, 64, 96, 160, 288, 544, 1056])
@pytest.mark.parametrize("T", [1, 40, 300, 700])
def test_linear_gated_widths(cuda_lib, N, T):
    c = Linear(T, 200, N, act="silu_mul", bias=True)
    c.check(c.call(binding))


@pytest.mark.parametrize("T", [1, 2, 9, 16, 17, 33, 64, 65, 100, 128, 130, 250, 257, 511, 600, 1030])
@pytest.mark.parametrize("K,N", [(128, 1), (256, 127), (640, 129), (1152, 300), (2048, 1024)])
def test_linear_fp8(cuda_lib, T, K, N):
    c = Linear(T, K, N, fp8=True)
    c.check(c.call(binding))


@pytest.mark.parametrize("T,K,N,act", [(1, 7168, 6144, "none"), (16, 7168, 4096, "silu_mul"),
                                       (300, 7168, 2048, "none"), (2050, 2048, 7168, "none"),
                                       (700, 4096, 4096, "silu_mul")])
def test_linear_fp8_wide(cuda_lib, T, K, N, act):
    c = Linear(T, K, N, act=act, fp8=True, residual=True)
    c.check(c.call(binding))


# sizes that the cut of few rows answers with clusters of up to 8 CTAs, tiles of 8 to 128 weight rows and
# one or two rounds of units (a few go to the kernels for many rows); clusters of the other numbers of CTAs,
# and those that walk several rounds, are tests/linear_cuts.py's
CUTS = [(1, 512, 256), (1, 512, 24576), (48, 4096, 4096), (1, 4096, 2048), (24, 4096, 2048),
        (64, 4096, 2048), (64, 2048, 2048), (24, 8192, 1024), (48, 2048, 256), (64, 2048, 1024),
        (80, 512, 12288), (80, 512, 24576), (80, 4096, 4096), (64, 8192, 24576), (1, 8192, 4096),
        (80, 2048, 2048), (1, 8192, 2048), (80, 2048, 1024), (80, 4096, 1024), (96, 4160, 1000)]


@pytest.mark.parametrize("T,K,N", CUTS)
@pytest.mark.parametrize("act", ["none", "silu_mul"])
@pytest.mark.parametrize("fp8", [False, True])
def test_linear_cuts_of_few_rows(cuda_lib, T, K, N, act, fp8):
    if fp8 and K % 128 or act == "silu_mul" and N % 256:
        pytest.skip("sizes of the other form")
    c = Linear(T, K, N, act=act, fp8=fp8, bias=True, residual=True)
    c.check(c.call(binding))


@pytest.mark.parametrize("T", [96, 97, 192, 256, 257])
@pytest.mark.parametrize("K,N", [(512, 1024), (2048, 9000)])
@pytest.mark.parametrize("fp8", [False, True])
def test_linear_between_few_and_many_rows(cuda_lib, T, K, N, fp8):
    c = Linear(T, K, N, act="silu", fp8=fp8, residual=True)
    c.check(c.call(binding))


def test_linear_large_values_of_activations(cuda_lib):
    """Where exp overflows or vanishes the activations take their limits."""
    K = 64
    x = torch.zeros(8, K, dtype=torch.bfloat16, device=DEV)
    x[:, 0] = torch.tensor([-3e38, -1e4, -200.0, -88.0, 88.0, 200.0, 1e4, 3e38], device=DEV)
    w = torch.zeros(64, K, dtype=torch.bfloat16, device=DEV)
    w[:, 0] = 1
    z = x[:, 0].double()
    for act in ("relu", "silu", "gelu", "gelu_tanh"):
        y = binding.moe_linear(x, w, activation=act).double()
        want = z.clamp_min(0)
        assert torch.isfinite(y).all()
        # silu(-88) = -88 e^-88, below 1e-36
        assert ((y - want[:, None]).abs() <= BF16 * want.abs()[:, None] + 1e-36).all(), act
    y = binding.moe_linear(x, w, activation="silu_mul").double()
    want = z.clamp_min(0) * z
    ok = want < 1e38                               # the others overflow bf16 as they should
    assert ((y - want[:, None]).abs()[ok] <= 2 * BF16 * want.abs()[ok, None] + 1e-33).all()
    assert (y[-1] == math.inf).all()


# ------------------------------------------------------------------------------ rows, strides
@pytest.mark.parametrize("T", [5, 150, 600])
@pytest.mark.parametrize("fp8", [False, True])
def test_linear_strided_rows(cuda_lib, T, fp8):
    c = Linear(T, 256, 200, fp8=fp8, residual=True)
    want = c.call(binding)
    kind = torch.uint8 if fp8 else torch.bfloat16
    bad = 0x7F if fp8 else math.nan                # NaN beside the columns
    big = torch.full((T, 512), bad, dtype=kind, device=DEV)
    big[:, 128:384] = c.x.view(kind)
    res = torch.full((T, 333), math.nan, dtype=torch.bfloat16, device=DEV)
    res[:, 7:207] = c.residual
    out = torch.full((T, 301), 9.0, dtype=torch.bfloat16, device=DEV)
    x = big[:, 128:384]
    got = c.call(binding, x=x.view(c.x.dtype) if fp8 else x, residual=res[:, 7:207],
                 out=out[:, 3:203])
    assert torch.equal(got, want) and got.data_ptr() == out[:, 3:].data_ptr()
    assert (out[:, :3] == 9).all() and (out[:, 203:] == 9).all()
    both = c.residual.clone()                      # in place of the residual
    assert c.call(binding, residual=both, out=both) is both and torch.equal(both, want)


def test_linear_takes_bytes_as_codes(cuda_lib):
    c = Linear(9, 128, 100, fp8=True)
    want = c.call(binding)
    got = binding.moe_linear(c.x.view(torch.uint8), c.weight.view(torch.uint8), x_scale=c.x_scale,
                             weight_scale=c.weight_scale)
    assert torch.equal(want, got)


@pytest.mark.parametrize("T", [3, 40, 200, 600])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("act", ["none", "silu_mul"])
def test_linear_non_finite_values_stay_in_their_row_and_column(cuda_lib, T, fp8, act):
    c = Linear(T, 384, 256, act=act, fp8=fp8)
    want = c.call(binding)
    r, n = T // 2, 37
    if fp8:
        c.x.view(torch.uint8)[r, 5] = 0x7F
        c.weight.view(torch.uint8)[n, 200] = 0xFF
    else:
        c.x[r, 5], c.weight[n, 200] = math.nan, math.inf
    got = c.call(binding)
    assert got[r].isnan().all() and not torch.isfinite(got[:, n]).any()
    keep = torch.ones_like(want, dtype=torch.bool)
    keep[r], keep[:, n] = False, False
    assert torch.equal(got[keep], want[keep])


def test_linear_empty_and_refused(cuda_lib):
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.zeros(48, 64, dtype=torch.bfloat16, device=DEV)
    assert binding.moe_linear(x, w).shape == (0, 48)
    off = torch.zeros(2, dtype=torch.int32, device=DEV)
    assert binding.moe_grouped_linear(x, w[None], off).shape == (0, 48)
    with pytest.raises(binding.GbmoeError):        # 48 rows do not split into gates and ups of 16
        binding.moe_linear(torch.zeros(1, 64, dtype=torch.bfloat16, device=DEV), w,
                           activation="silu_mul")
    with pytest.raises(binding.GbmoeError):
        binding.moe_linear(torch.zeros(1, 12, dtype=torch.bfloat16, device=DEV),
                           torch.zeros(4, 12, dtype=torch.bfloat16, device=DEV))


# ------------------------------------------------------------------------------ grouped
SIZES = [[1], [5, 0, 3], [0, 0, 1], [16, 16], [17, 1, 0, 15, 40], [0, 130, 2], [300, 0, 0, 7],
         [64, 65, 63, 1, 128, 129, 127], [1, 600, 1], [257, 256, 255], [0, 1000, 0, 33, 500]]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("act", ["none", "silu_mul", "gelu"])
def test_grouped(cuda_lib, sizes, fp8, act):
    for K, N in ((128, 256), (640, 512), (384, 130)):
        if act == "silu_mul" and N % 256:
            continue
        c = Linear(0, K, N, sizes=sizes, act=act, fp8=fp8, bias=True, weighted=True)
        ws = binding.alloc_workspace(256)
        c.check(c.call(binding, workspace=ws))
        assert _status(ws) == binding.OK


@pytest.mark.parametrize("seed", range(12))
def test_grouped_drawn(cuda_lib, seed):
    rng = random.Random(seed)
    G = rng.choice([2, 8, 30, 64, 200])
    sizes = [rng.choice([0, 0, 1, 2, rng.randint(1, 40), rng.randint(1, 300)]) for _ in range(G)]
    fp8 = seed % 2 == 1
    c = Linear(0, 128 * rng.randint(1, 5), 256 * rng.randint(1, 3), sizes=sizes or [1], fp8=fp8,
               act=rng.choice(ACTS), bias=rng.random() < 0.5, weighted=rng.random() < 0.5,
               residual=rng.random() < 0.5, lead=rng.choice([0, 3]), tail=rng.choice([0, 9]))
    if c.T:
        c.check(c.call(binding))


# (either several CTAs to a tile or several rounds; both at once: tests/linear_cuts.py)
@pytest.mark.parametrize("sizes", [[4], [1, 2], [0, 9, 8, 7], [100, 3, 0, 1]])
@pytest.mark.parametrize("K,N", [(4096, 512), (8192, 2048), (512, 8192), (2048, 96 * 128)])
@pytest.mark.parametrize("act", ["none", "silu_mul"])
@pytest.mark.parametrize("fp8", [False, True])
def test_grouped_few_groups(cuda_lib, sizes, K, N, act, fp8):
    """Long sums for few rows: several CTAs to a tile, in several rounds where the tiles are small."""
    c = Linear(0, K, N, sizes=sizes, act=act, fp8=fp8, weighted=True, residual=True)
    c.check(c.call(binding))


@pytest.mark.parametrize("mean", [8, 9, 32, 33])
@pytest.mark.parametrize("fp8", [False, True])
def test_grouped_between_few_and_many_rows(cuda_lib, mean, fp8):
    rng = random.Random(mean)
    sizes = [rng.randint(0, 2 * mean) for _ in range(11)]
    sizes.append(max(0, 12 * mean - sum(sizes)))
    c = Linear(0, 640, 768, sizes=sizes, act="silu_mul", fp8=fp8, bias=True)
    c.check(c.call(binding))


def test_grouped_most_groups(cuda_lib):
    rng = random.Random(1)
    sizes = [rng.choice([0, 1, 1, 3]) for _ in range(1024)]
    c = Linear(0, 64, 48, sizes=sizes)
    c.check(c.call(binding))
    one = [0] * 1023 + [70]
    c = Linear(0, 64, 48, sizes=one)
    c.check(c.call(binding))


@pytest.mark.parametrize("sizes", [[3, 0, 5], [100, 200], [600, 0, 300]])
@pytest.mark.parametrize("fp8", [False, True])
def test_grouped_leaves_other_rows(cuda_lib, sizes, fp8):
    """Rows before the first run and behind the last are neither written nor do they matter, and a
    run does not see its neighbours'."""
    c = Linear(0, 256, 256, sizes=sizes, fp8=fp8, lead=11, tail=20)
    end = 11 + sum(sizes)
    kind, bad = (torch.uint8, 0x7F) if fp8 else (torch.bfloat16, math.nan)
    clean = c.call(binding)
    x = c.x.clone()
    x.view(kind)[:11], x.view(kind)[end:] = bad, bad
    out = torch.full((c.T, 256), 7.0, dtype=torch.bfloat16, device=DEV)
    got = c.call(binding, x=x, out=out)
    assert (got[:11] == 7).all() and (got[end:] == 7).all()
    assert torch.equal(got[11:end], clean[11:end])
    runs = c.runs()
    g, a, b = runs[0]
    x.view(kind)[a:b] = bad                        # the first run's rows and weight
    c.weight.view(kind)[g] = bad
    got = c.call(binding, x=x, out=out)
    assert got[a:b].isnan().all() and torch.equal(got[b:end], clean[b:end])


@pytest.mark.parametrize("rows", [6, 300])
def test_grouped_bad_offsets_are_reported(cuda_lib, rows):
    """A run that goes back or leaves the rows has none; the others are computed, and nothing else
    is touched."""
    c = Linear(0, 64, 128, sizes=[rows, rows, rows])
    want = c.call(binding)
    ws = binding.alloc_workspace(256)
    R = rows
    for off, good in (([0, R, 3 * R + 1, 3 * R], [(0, R)]), ([-4, R, 2 * R, 3 * R], [(R, 2 * R), (2 * R, 3 * R)]),
                      ([0, R, 2 * R, R], [(0, R), (R, 2 * R)]),
                      ([0, R, 2 * R, 2 ** 31 - 1], [(0, R), (R, 2 * R)]),
                      ([-2 ** 31, -5, R, 2 * R], [])):
        out = torch.full((c.T, 128), 7.0, dtype=torch.bfloat16, device=DEV)
        got = c.call(binding, out=out, workspace=ws,
                     offsets=torch.tensor(off, dtype=torch.int32, device=DEV))
        assert _status(ws) == binding.ERR_DEVICE_CHECK, off
        assert _status(ws) == binding.OK
        named = torch.zeros(c.T, dtype=torch.bool, device=DEV)
        for a, b in good:
            assert torch.equal(got[a:b], want[a:b]), off
        for g in range(3):                         # runs that are inside the rows are written
            if 0 <= off[g] <= off[g + 1] <= c.T:
                named[off[g]:off[g + 1]] = True
        assert (got[~named] == 7).all(), off


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows", [5, 300, 20000])
def test_grouped_offsets_that_go_back_and_come_again(cuda_lib, rows, fp8):
    """All rows belong to the first run, and to every second one behind it: reported, each row has some
    run's values, and rows behind the runs are left alone."""
    G = 40
    w = torch.ones(G, 128, 128, dtype=torch.bfloat16, device=DEV)
    x = torch.ones(rows + 3, 128, dtype=torch.bfloat16, device=DEV)
    kw = {}
    if fp8:
        w, x = w.to(torch.float8_e4m3fn), x.to(torch.float8_e4m3fn)
        kw = dict(x_scale=torch.ones(1, rows + 3, device=DEV), weight_scale=torch.ones(G, 1, 1, device=DEV))
    off = torch.tensor([0, rows] * (G // 2) + [0], dtype=torch.int32, device=DEV)
    out = torch.full((rows + 3, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = binding.alloc_workspace(256)
    binding.moe_grouped_linear(x, w, off, out=out, workspace=ws, **kw)
    assert _status(ws) == binding.ERR_DEVICE_CHECK
    assert (out[:rows] == 128).all() and (out[rows:] == 7).all()


def test_grouped_offsets_whose_units_would_pass_32_bits(cuda_lib):
    """512 runs of all 4096 rows: 2^17 blocks of 16 rows by 2^14 tiles."""
    T, G, K, N = 4096, 1024, 8, 2 ** 21 - 2
    w = torch.ones(G, N, K, dtype=torch.bfloat16, device=DEV)
    x = torch.ones(T, K, dtype=torch.bfloat16, device=DEV)
    off = torch.tensor([0, T] * (G // 2) + [0], dtype=torch.int32, device=DEV)
    out = torch.full((T, N), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = binding.alloc_workspace(256)
    binding.moe_grouped_linear(x, w, off, out=out, workspace=ws)
    assert _status(ws) == binding.ERR_DEVICE_CHECK
    assert (out[::97] == K).all() and (out[:, -1] == K).all() and (out[:, ::4099] == K).all()


def test_past_32_bits(cuda_lib):
    """Weights, outputs and rows whose offsets pass 2^31 elements."""
    N, K, G = 8192, 4160, 64
    w = torch.empty(G, N, K, dtype=torch.bfloat16, device=DEV).normal_(std=K ** -0.5)
    assert w.numel() > 2 ** 31
    c = Linear(0, 8, 8, sizes=[0] * (G - 2) + [3, 20])
    c.K, c.N, c.cols, c.weight = K, N, N, w
    c.x = torch.randn(c.T, K, device=DEV).to(torch.bfloat16)
    c.check(c.call(binding))
    del w, c.weight
    T, K = 270000, 64
    x, w = (torch.randn(n, K, device=DEV).to(torch.bfloat16) for n in (T, N))
    out = binding.moe_linear(x, w)
    assert out.numel() > 2 ** 31
    c = Linear(8, K, N)
    c.T, c.x, c.weight = T, x, w
    for a in (0, 131000, 262100, T - 300):
        y, off = c.reference(a, a + 300, 0)
        assert ((out[a:a + 300].double() - y).abs() <= off).all()


# ------------------------------------------------------------------------------ use
@pytest.mark.parametrize("fp8", [False, True])
def test_calls_repeat_bit_for_bit(cuda_lib, fp8):
    for T, K, N in ((1, 7168, 4096), (60, 4096, 1024), (700, 2048, 2048)):
        c = Linear(T, K, N, fp8=fp8)
        first = c.call(binding)
        for _ in range(5):
            assert torch.equal(c.call(binding), first)


def test_rows_do_not_depend_on_their_batch_of_groups(cuda_lib):
    """A run's rows come out the same whatever the other runs of the call hold."""
    c = Linear(0, 512, 384, sizes=[20, 0, 33, 4])
    whole = c.call(binding)
    other = c.x.clone()
    other[:20] *= -3
    assert torch.equal(c.call(binding, x=other)[20:], whole[20:])


@pytest.mark.parametrize("rows", [8, 500])
@pytest.mark.parametrize("fp8", [False, True])
def test_other_streams(cuda_lib, rows, fp8):
    c = Linear(0, 1024, 512, sizes=[rows, 3, rows], fp8=fp8)
    want = c.call(binding)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [[c.call(binding, stream=s) for _ in range(4)] for s in streams]
    with torch.cuda.stream(streams[0]):
        outs.append([c.call(binding)])
    torch.cuda.synchronize()
    for o in outs:
        for t in o:
            assert torch.equal(t, want)


@pytest.mark.parametrize("rows", [4, 400])
@pytest.mark.parametrize("fp8", [False, True])
def test_captured_calls_follow_their_offsets(cuda_lib, rows, fp8):
    c = Linear(0, 512, 512, sizes=[rows, rows, 0, rows], fp8=fp8, act="silu_mul")
    c.call(binding)
    s = torch.cuda.Stream()
    graphs, outs = [], []
    for _ in range(2):                             # two graphs over the same operands
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs.append(c.call(binding))
        graphs.append(graph)
    for sizes in ([rows, rows, 0, rows], [0, 3 * rows, 0, 0], [1, 0, 3 * rows - 1, 0]):
        c.offsets.copy_(torch.tensor([0] + sizes).cumsum(0))
        c.sizes = sizes
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for o in outs:
            c.check(o)


FIRST_IN_CAPTURE = """
import sys
sys.path.insert(0, {root!r})
import torch
from mixture_experts_layer_05_gb300 import binding
from tests.linear_cases import Linear
cases = [Linear(T, 512, 1024, act=act, fp8=fp8) for T in (3, 600) for act in ("none", "silu_mul")
         for fp8 in (False, True)] + [Linear(48, 4096, 4096)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    outs = [c.call(binding) for c in cases]
graph.replay()
torch.cuda.synchronize()
for c, o in zip(cases, outs):
    c.check(o)
print("captured")
"""


def test_first_calls_of_a_process_in_a_capture(cuda_lib):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_IN_CAPTURE.format(root=root)], capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_calls_from_several_threads(cuda_lib):
    cases = [Linear(T, 1024, 768, fp8=T % 2 == 1) for T in (1, 2, 40, 41, 300, 301)]
    want = [c.call(binding) for c in cases]
    torch.cuda.synchronize()
    got = [None] * len(cases)

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got[i] = cases[i].call(binding)
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for g, w in zip(got, want):
        assert torch.equal(g, w)


def test_binding_refuses(cuda_lib):
    c = Linear(6, 256, 64)
    for kw in (dict(bias=c.x[0, :63]), dict(residual=c.x), dict(out=c.x), dict(row_weight=c.x[:, 0]),
               dict(activation="tanh"), dict(x_scale=torch.zeros(2, 6, device=DEV)),
               dict(workspace=torch.zeros(8, device=DEV))):
        with pytest.raises(ValueError):
            c.call(binding, **kw)


# ------------------------------------------------------------------------------ together
@pytest.mark.parametrize("T", [1, 12, 300])
@pytest.mark.parametrize("quant", [None, "fp8"])
def test_pieces_give_the_layer(cuda_lib, T, quant):
    """Routing, the rows sorted by expert, gate and up with the activation, the way down times the
    routing weights, and the sum per token: FusedMoE's output from the pieces."""
    w = configs.shrink(configs.DSV3, num_experts=16, top_k=4, num_expert_group=4, topk_group=2,
                       hidden_size=512, intermediate_size=256, shared_intermediate_size=0)
    x, logits = (t.to(DEV) for t in inputs.make_tokens(w, T))
    cfg = binding.config_from_workload(w, weight_quant=quant)
    if quant:
        q = {k: None if v is None else v.to(DEV) for k, v in inputs.make_fp8_weights(w, 0).items()}
        w13, w2, bias = q["w13_q"], q["w2_q"], q["bias"]
        layer = binding.FusedMoE(cfg, w13, w2, bias, max_tokens=T, w13_scale=q["w13_s"],
                                 w2_scale=q["w2_s"])
    else:
        q = {k: None if v is None else v.to(DEV) for k, v in inputs.make_weights(w, 0).items()}
        w13, w2, bias = q["w13"], q["w2"], q["bias"]
        layer = binding.FusedMoE(cfg, w13, w2, bias, max_tokens=T)
    want = layer(x, logits).float()
    weights = torch.empty(T, w.top_k, device=DEV)
    ids = torch.empty(T, w.top_k, dtype=torch.int32, device=DEV)
    binding.moe_topk(cfg, logits, bias, weights, ids)
    order = ids.flatten().argsort(stable=True)
    counts = torch.bincount(ids.flatten().long(), minlength=w.num_experts)
    off = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).to(torch.int32)
    rows = (x[order // w.top_k]).contiguous()
    up = dict(activation="silu_mul")
    down = dict(row_weight=weights.flatten()[order].contiguous())
    if quant:
        rows, xs = binding.moe_quant_fp8_per_token_group(rows)
        up.update(x_scale=xs, weight_scale=q["w13_s"])
    act = binding.moe_grouped_linear(rows, w13, off, **up)
    if quant:
        act, xs = binding.moe_quant_fp8_per_token_group(act)
        down.update(x_scale=xs, weight_scale=q["w2_s"])
    o = binding.moe_grouped_linear(act, w2, off, **down)
    y = torch.zeros(T, w.hidden_size, device=DEV).index_add_(0, order // w.top_k, o.float())
    # the layer keeps its slots in fp32 and rounds once; here each of top_k rows is rounded, then
    # the layer's own output; the act is rounded once on both sides, to bf16 (a sum in another
    # order may round the other way: a whole step of each of `intermediate` terms, as a random
    # walk), and with e4m3 the act's bf16 rounding can move its code by one step, 2^-3
    size = torch.zeros_like(y).index_add_(0, order // w.top_k, o.float().abs())
    step = 2 * BF16 + (2.0 ** -3 if quant else 0)
    spread = (y ** 2).mean().sqrt()
    off_by = BF16 * (size + want.abs()) + step * spread
    assert ((y - want).abs() <= off_by).all()
