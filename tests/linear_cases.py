"""Inputs, 64-bit references and bounds of the dense and grouped product tests."""
import math

import torch

BF16, FP32 = 2.0 ** -8, 2.0 ** -24                 # half a step, relative
BLOCK = 128
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh", "silu_mul")


class Linear:
    """Random operands of one call: sizes None is the dense product, else rows per group (before
    them `lead` rows and behind them `tail` rows of no group)."""

    def __init__(self, T, K, N, sizes=None, act="none", fp8=False, bias=False, residual=False,
                 weighted=False, lead=0, tail=0, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed + 1000003 * T + 1009 * K + N)

        def randn(*shape, std=1.0):
            return torch.randn(*shape, generator=g, device=device) * std

        self.act, self.fp8, self.N, self.K = act, fp8, N, K
        self.sizes, self.lead = sizes, lead
        self.G = 1 if sizes is None else len(sizes)
        if sizes is not None:
            T = lead + sum(sizes) + tail
        self.T = T
        self.cols = N // 2 if act == "silu_mul" else N
        w = randn(self.G, N, K, std=K ** -0.5)
        x = randn(T, K)
        self.x_scale = self.weight_scale = None
        if fp8:
            nb = -(-N // BLOCK)
            self.x_scale = torch.rand(K // BLOCK, T, generator=g, device=device) * 0.05 + 0.01
            self.weight_scale = torch.rand(self.G, nb, K // BLOCK, generator=g, device=device) + 0.5
            self.x = (x * 40).to(torch.float8_e4m3fn)
            self.weight = w.to(torch.float8_e4m3fn)
        else:
            self.x, self.weight = x.to(torch.bfloat16), w.to(torch.bfloat16)
        self.bias = randn(self.G, N, std=0.5).to(torch.bfloat16) if bias else None
        self.residual = randn(T, self.cols, std=2.0).to(torch.bfloat16) if residual else None
        self.row_weight = torch.rand(T, generator=g, device=device) if weighted else None
        if sizes is None:
            self.offsets = None
            self.weight = self.weight[0]
            if fp8:
                self.weight_scale = self.weight_scale[0]
            if bias:
                self.bias = self.bias[0]
        else:
            self.offsets = (lead + torch.tensor([0] + list(sizes)).cumsum(0)).to(torch.int32).to(device)

    def call(self, binding, **kw):
        args = dict(bias=self.bias, activation=self.act, residual=self.residual,
                    row_weight=self.row_weight, x_scale=self.x_scale,
                    weight_scale=self.weight_scale)
        args.update(kw)
        x = args.pop("x", self.x)
        if self.offsets is None:
            return binding.moe_linear(x, self.weight, **args)
        return binding.moe_grouped_linear(x, self.weight, args.pop("offsets", self.offsets), **args)

    def runs(self):
        """(group, first row, end) of the runs that have rows."""
        if self.sizes is None:
            return [(0, 0, self.T)]
        at, out = self.lead, []
        for g, n in enumerate(self.sizes):
            if n:
                out.append((g, at, at + n))
            at += n
        return out

    def reference(self, a, b, g):
        """The output rows [a, b) of group g in 64 bits, and how far a kernel may be off.

        A sum's K products enter fp32 in at most K / 16 steps of the matrix unit, within each of
        which 16 products are aligned and added, then at most 8 cut pieces are joined (e4m3:
        every block of 128 is scaled first, K / 128 more steps of one product and one addition);
        a step that drops bits is off by 2 FP32 of the sum of magnitudes at most.
        """
        x, w = self.x[a:b].double(), (self.weight if self.sizes is None else self.weight[g]).double()
        if self.fp8:
            xs = self.x_scale[:, a:b].t().double().repeat_interleave(BLOCK, 1)
            ws = (self.weight_scale if self.sizes is None else self.weight_scale[g]).double()
            x = x * xs
            w = w * ws.repeat_interleave(BLOCK, 0)[:self.N].repeat_interleave(BLOCK, 1)
        z, size = x @ w.t(), x.abs() @ w.abs().t()
        steps = self.K / 16 + 16 + 8 + (3 * self.K / BLOCK if self.fp8 else 0)
        off = 2 * FP32 * steps * size
        if self.bias is not None:
            bias = (self.bias if self.sizes is None else self.bias[g]).double()
            z = z + bias
            off = off + FP32 * z.abs()
        # values: the exponential is off by (2 + 1.2 |z|) steps of 2 FP32, the sum, the quotient and
        # the product by a few more; erf and tanh by 4 of 1, and the polynomial in front of tanh
        # by a few of its value, which moves tanh by less than 1 / |value| of it. Slopes: the
        # activations' derivatives lie within [-0.13, 1.13]
        fine = 2 * FP32 * (8 + 1.2 * z.abs()) * z.abs()
        if self.act == "silu_mul":
            h = self.cols
            gate, up = z[:, :h], z[:, h:]
            s = gate * torch.sigmoid(gate)
            y = s * up
            off = (1.13 * off[:, :h] + fine[:, :h]) * (up.abs() + off[:, h:]) + s.abs() * off[:, h:]
        elif self.act == "none":
            y = z
        else:
            if self.act == "relu":
                y = z.clamp_min(0)
            elif self.act == "silu":
                y = z * torch.sigmoid(z)
            elif self.act == "gelu":
                y = 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
            else:
                y = z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
            off = 1.13 * off + fine
        off = off + 2 * FP32 * y.abs()
        if self.row_weight is not None:
            rw = self.row_weight[a:b, None].double()
            y, off = y * rw, (off + 2 * FP32 * y.abs()) * rw.abs()
        if self.residual is not None:
            y = y + self.residual[a:b].double()
            off = off + FP32 * y.abs()
        return y, off + BF16 * (y.abs() + off)

    def check(self, out):
        assert out.shape == (self.T, self.cols) and out.dtype == torch.bfloat16
        for g, a, b in self.runs():
            for i in range(a, b, 2048):
                j = min(i + 2048, b)
                y, off = self.reference(i, j, g)
                bad = ~((out[i:j].double() - y).abs() <= off)
                assert not bad.any(), (g, i, int(bad.sum()), bad.nonzero()[:4].tolist(),
                                       out[i:j][bad][:4].tolist(), y[bad][:4].tolist())
