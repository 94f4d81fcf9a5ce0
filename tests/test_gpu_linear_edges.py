"""moe_linear and moe_grouped_linear where a value, an alignment or a cut is at its edge."""
import math

import pytest
import torch

from mixture_experts_layer_05_gb300 import binding
from tests.linear_cases import BF16, FP32, Linear

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
