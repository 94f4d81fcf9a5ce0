"""moe_linear and moe_grouped_linear where a value, an alignment or a cut is at its edge."""
import math

import pytest
import torch

from mixture_experts_layer_05_gb300 import binding
from tests.linear_cases import BF16, FP32, Linear
from tests.linear_cuts import CLUSTERS, GATED_FP8, ROUNDS

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("T", [8, 128, 640])
@pytest.mark.parametrize("fp8", [False, True])
def test_gelu_keeps_its_left_tail(cuda_lib, T, fp8):
    """z (1 + erf(z / sqrt 2)) / 2 down to -12, where 1 + erf is 1e-32 and its fp32 sum would be 0."""
    K, N = 128, 256
    z = torch.linspace(-12, 1, T, device=DEV).to(torch.bfloat16)
    x, w = torch.zeros(T, K, device=DEV), torch.zeros(N, K, device=DEV)
    x[:, 5] = 1 if fp8 else z.float()
    w[:, 5] = 1
    if fp8:
        y = binding.moe_linear(x.to(torch.float8_e4m3fn), w.to(torch.float8_e4m3fn), activation="gelu",
                               x_scale=z.float()[None].contiguous(),
                               weight_scale=torch.ones(2, 1, device=DEV))
    else:
        y = binding.moe_linear(x.to(torch.bfloat16), w.to(torch.bfloat16), activation="gelu")
    z = z.double()                                 # exact in every step up to the activation
    want = 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    # q = exp(-z^2 / 2) t P(t), in units of FP32: the fit 3; t 6 (quotient 4, constant, sum), which moves
    # t P(t) by 2.7 of it at most; P's 8 steps and coefficients 2 + 1 of its terms' magnitudes, 1.9 P; three
    # products; the exponential of x = z^2 / 2 off by 2 + 1.16 x steps of 2, and by x of its argument
    x = 0.5 * z * z
    q = 0.5 * torch.special.erfc(z.abs() / math.sqrt(2))
    off = FP32 * (3 + 2.7 * 6 + 1.9 * 8 * 3 + 3 + 2 * (2 + 1.16 * x) + x) * z.abs() * q + FP32 * want.abs()
    off = off + BF16 * (want.abs() + off)
    assert ((y.double() - want[:, None]).abs() <= off[:, None]).all()


def test_gelu_of_infinities(cuda_lib):
    """As the formula has it: inf stays, -inf times 0 and NaN are NaN."""
    w = torch.zeros(64, 64, dtype=torch.bfloat16, device=DEV)
    w[:, 0] = 1
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV)
    x[:, 0] = torch.tensor([math.inf, -math.inf, math.nan, 3e38], device=DEV)
    y = binding.moe_linear(x, w, activation="gelu")
    assert (y[0] == math.inf).all() and y[1:3].isnan().all() and (y[3] == x[3, 0]).all()


@pytest.mark.parametrize("rows,K,N,act,fp8,ctas,rounds", CLUSTERS + ROUNDS)
def test_clusters_and_their_rounds(cuda_lib, rows, K, N, act, fp8, ctas, rounds):
    """Every number of CTAs that cut K, and clusters that walk several units: the room of the partial sums is
    used again only once all have taken theirs."""
    T, sizes = (rows, None) if isinstance(rows, int) else (0, list(rows))
    ws = binding.alloc_workspace(256)
    c = Linear(T, K, N, sizes=sizes, act=act, fp8=fp8, bias=True, residual=True, weighted=True)
    y = c.call(binding, workspace=ws)
    c.check(y)
    for _ in range(3):
        assert torch.equal(c.call(binding, workspace=ws), y)
    assert binding.moe_get_device_status(ws) == binding.OK


@pytest.mark.parametrize("rows,K,N", GATED_FP8)
@pytest.mark.parametrize("off_out,off_residual,off_bias", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 3, 1)])
def test_gated_e4m3_of_many_rows_off_16_bytes(cuda_lib, rows, K, N, off_out, off_residual, off_bias):
    """out, residual or bias (elements) off the alignment that 16-byte accesses need, or of such a row stride."""
    T, sizes = (rows, None) if isinstance(rows, int) else (0, list(rows))
    c = Linear(T, K, N, sizes=sizes, act="silu_mul", fp8=True, bias=True, residual=True, weighted=True)

    def moved(t, by):
        """The same values `by` elements into other memory; rows of a 2-D one odd strides apart."""
        if not by:
            return t
        if t is c.bias:
            flat = torch.empty(t.numel() + by, dtype=t.dtype, device=DEV)[by:]
            return flat.copy_(t.flatten()).view(t.shape)
        wide = torch.full((t.shape[0], t.shape[1] + 2 * by + 1), 9.0, dtype=t.dtype, device=DEV)
        wide[:, by:by + t.shape[1]] = t
        return wide[:, by:by + t.shape[1]]

    out = moved(torch.full((c.T, c.cols), 7.0, dtype=torch.bfloat16, device=DEV), off_out)
    got = c.call(binding, out=out, residual=moved(c.residual, off_residual), bias=moved(c.bias, off_bias))
    assert got is out
    c.check(got)
    if off_out:                                    # what lies between the rows is left alone
        base = torch.as_strided(out, (c.T, out.stride(0)), (out.stride(0), 1), 0)
        assert (base[:, :off_out] == 9).all() and (base[:, off_out + c.cols:] == 9).all()
