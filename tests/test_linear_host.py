"""moe_linear and moe_grouped_linear on the host: what the C ABI and the binding refuse."""
import ctypes

import pytest
import torch

from mixture_experts_layer_05_gb300 import binding
from mixture_experts_layer_05_gb300 import build as build_mod

P = ctypes.c_void_p
OK, BAD, UNSUP = binding.OK, binding.ERR_INVALID_ARG, binding.ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return binding.load()


def _call(lib, T=4, K=256, N=512, G=None, offsets=256, **kw):
    d = dict(x=256, x_stride=max(K, 0), x_scale=None, weight=256, weight_scale=None, bias=None,
             activation=0, weight_quant=0, residual=None, residual_stride=0, row_weight=None, out=256,
             out_stride=max(N, 0), workspace=None)
    d.update(kw)
    a = ctypes.byref(binding.LinearArgs(**d))
    if G is None:
        return lib.moe_linear(T, K, N, a, None)
    return lib.moe_grouped_linear(T, G, K, N, P(offsets or None), a, None)


FP8 = dict(weight_quant=1, x_scale=256, weight_scale=256)


@pytest.mark.parametrize("G", [None, 3])
def test_refusals(lib, G):
    assert _call(lib, T=0, G=G) == OK                                  # empty batch
    assert _call(lib, T=0, G=G, x=None, weight=None, out=None) == OK
    for kw in (dict(T=-1), dict(T=(1 << 22) + 1), dict(K=0), dict(K=-8), dict(N=0), dict(x=None),
               dict(weight=None), dict(out=None), dict(activation=-1), dict(activation=6),
               dict(weight_quant=3), dict(weight_quant=-1), dict(x_scale=256),
               dict(weight_scale=256), dict(weight_quant=1), dict(weight_quant=1, x_scale=256),
               dict(weight_quant=1, weight_scale=256), dict(x_stride=248), dict(x_stride=260),
               dict(out_stride=511), dict(residual=256, residual_stride=511), dict(x=264),
               dict(weight=264), dict(bias=257), dict(residual=257, residual_stride=512),
               dict(row_weight=258), dict(out=257), dict(workspace=128),
               dict(FP8, x_scale=258), dict(FP8, weight_scale=258), dict(FP8, x_stride=264)):
        assert _call(lib, G=G, **kw) == BAD, kw
    for kw in (dict(K=100), dict(K=4), dict(FP8, K=136), dict(FP8, K=64), dict(activation=5, N=528),
               dict(activation=5, N=33), dict(FP8, activation=5, N=128), dict(FP8, activation=5, N=384),
               dict(weight_quant=2), dict(T=1 << 22, N=1 << 23), dict(K=(1 << 24) + 8),
               dict(x_stride=1 << 39)):
        assert _call(lib, G=G, **kw) == UNSUP, kw


def test_grouped_refusals(lib):
    assert lib.moe_linear(4, 256, 512, None, None) == BAD
    assert lib.moe_grouped_linear(4, 3, 256, 512, P(256), None, None) == BAD
    assert _call(lib, G=0) == BAD and _call(lib, G=-1) == BAD
    assert _call(lib, G=3, offsets=0) == BAD and _call(lib, G=3, offsets=258) == BAD
    assert _call(lib, G=1025) == UNSUP
    assert _call(lib, G=1024, N=1 << 21) == UNSUP


def test_refuses_weights_whose_last_tile_passes_32_bits(lib):
    """A tile ends up to 255 rows behind the last, and rows and columns are counted in 32 bits."""
    for N in ((1 << 31) - 1, (1 << 31) - 256, (1 << 31) - 1024):
        assert _call(lib, T=1, K=8, N=N) == UNSUP, N
    assert _call(lib, T=1, K=8, N=(1 << 28) - 128, G=8) == UNSUP


def test_binding_refuses_host_tensors(lib):
    x, w = torch.zeros(2, 256, dtype=torch.bfloat16), torch.zeros(64, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        binding.moe_linear(x, w)
    with pytest.raises(ValueError):
        binding.moe_grouped_linear(x, w[None], torch.tensor([0, 2], dtype=torch.int32))
    with pytest.raises(ValueError):
        binding.moe_grouped_linear(x, w[None], None)
    for act in ("swish", 1, ""):
        with pytest.raises(ValueError):
            binding.moe_linear(x, w, activation=act)


def test_binding_checks_shapes_and_devices(lib):
    """On fake tensors: what a call of other shapes, types or devices is told."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        def t(*shape, dtype=torch.bfloat16, device="cuda:0"):
            return torch.empty(*shape, dtype=dtype, device=device)

        f8, f32, i32 = torch.float8_e4m3fn, torch.float32, torch.int32
        x, w = t(6, 256), t(64, 256)
        q, wq = t(6, 256, dtype=f8), t(130, 256, dtype=f8)
        s = dict(x_scale=t(2, 6, dtype=f32), weight_scale=t(2, 2, dtype=f32))
        for args, kw in (((x, t(64, 128)), {}), ((x, w.float()), {}), ((x.float(), w), {}),
                         ((x, t(3, 64, 256)), {}), ((x, t(256, 64).t()), {}), ((t(256, 6).t(), w), {}),
                         ((x, w), dict(bias=t(63))), ((x, w), dict(bias=t(64, dtype=f32))),
                         ((x, w), dict(residual=t(6, 63))), ((x, w), dict(residual=t(5, 64))),
                         ((x, w), dict(residual=t(64, 6).t())), ((x, w), dict(row_weight=t(6))),
                         ((x, w), dict(row_weight=t(5, dtype=f32))), ((x, w), dict(out=t(6, 63))),
                         ((x, w), dict(out=t(6, 64, dtype=f32))), ((x, w), dict(workspace=t(100))),
                         ((x, w), dict(workspace=t(256, device="cpu"))),
                         ((x, w), dict(activation="silu_mul", residual=t(6, 64))),
                         ((x, w), s), ((q, wq), {}), ((q, wq), dict(x_scale=s["x_scale"])),
                         ((q, wq), dict(weight_scale=s["weight_scale"])),
                         ((q, wq), dict(s, x_scale=t(6, 2, dtype=f32))),
                         ((q, wq), dict(s, weight_scale=t(1, 2, dtype=f32))),
                         ((q, w), s), ((x, t(64, 256, device="cuda:1")), {}),
                         ((x, w), dict(bias=t(64, device="cuda:1"))),
                         ((x, w), dict(residual=t(6, 64, device="cuda:1"))),
                         ((x, w), dict(out=t(6, 64, device="cuda:1")))):
            with pytest.raises(ValueError):
                binding.moe_linear(*args, **kw)
        off, g = t(4, dtype=i32), t(3, 64, 256)
        for args, kw in (((x, w, off), {}), ((x, g, t(3, dtype=i32)), {}),
                         ((x, g, t(4, dtype=torch.int64)), {}),
                         ((x, g, t(4, dtype=i32, device="cuda:1")), {}),
                         ((x, g, off), dict(bias=t(64))), ((x, g, off), dict(bias=t(3, 63)))):
            with pytest.raises(ValueError):
                binding.moe_grouped_linear(*args, **kw)
        with pytest.raises(ValueError):            # rows past 32 bits
            binding.moe_linear(t(1 << 31, 8), t(8, 8))
