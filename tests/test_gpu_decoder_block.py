"""The decoder block of examples/decoder_block.py: tokens served one by one or in chunks over the
cache get the attention that the whole prompt gets, and the block runs through to its output."""
import os
import sys

import pytest
import torch

from mixture_experts_layer_05_gb300 import binding
from tests.block_cases import BF16

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
import decoder_block as db  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_served_tokens_match_the_whole_prompt(cuda_lib, cache):
    s = db.Sizes(hidden=512, q_heads=8, kv_heads=2, head_dim=64, page=16, pages=256, experts=8,
                 top_k=2, intermediate=256, max_position=512, cache=cache)
    lens = [150, 37]
    g = torch.Generator(device="cuda").manual_seed(2)
    x = [torch.randn(n, s.hidden, generator=g, device="cuda").to(torch.bfloat16) for n in lens]
    whole = db.DecoderBlock(s, max_tokens=256)
    batch = db.Sequences(s, 2).extend(lens)
    want, _ = whole.attend(torch.cat(x), None, batch)
    want = list(want.split(lens))
    out, res = whole(torch.cat(x), None, batch)
    assert torch.isfinite(out).all() and torch.isfinite(res).all()
    served = db.DecoderBlock(s, max_tokens=256)
    seqs = db.Sequences(s, 2)
    done = [0, 0]
    for new in ([100, 5], [1, 1], [1, 1], [40, 1], [1, 29], [7, 0]):
        rows = torch.cat([x[i][done[i]:done[i] + n] for i, n in enumerate(new)])
        batch = seqs.extend(new)
        got, _ = served.attend(rows, None, batch)
        y, _ = served(rows, None, batch)           # writes the same cache rows again
        assert torch.isfinite(y).all()
        for i, part in enumerate(got.split(new)):
            ref = want[i][done[i]:done[i] + new[i]].float()
            done[i] += new[i]
            # the rows differ by the rounding of the weights to 16 bits and of the outputs, on
            # either side, and by the dense projection's sums (another shape of the product):
            # q and v up to a rounding apart, so scores by |q||k| / sqrt(d) roundings; in the
            # 8-bit cache that rounding can move a value to the next code, 1/8 of it
            size = want[i].float().abs().max()
            step = 6 * BF16 + (2.0 ** -3 if cache == "fp8" else 0.0)
            assert ((part.float() - ref).abs() <= 2 * BF16 * ref.abs() + step * size).all()
    assert done == lens
    assert served.status() == (binding.OK, binding.OK)


def test_example_runs(cuda_lib, capsys):
    db.main(["--prompts", "70", "3", "--steps", "2", "--cache", "fp8"])
    assert "one token each" in capsys.readouterr().out


def test_status_covers_the_projections(cuda_lib, monkeypatch):
    """What a projection reports (a wait that ran out, say) is what the block reports, once."""
    s = db.Sizes(hidden=512, q_heads=8, kv_heads=2, head_dim=64, page=16, pages=16, experts=8, top_k=2,
                 intermediate=256, max_position=64)
    block = db.DecoderBlock(s, max_tokens=8)
    batch = db.Sequences(s, 1).extend([3])
    x = torch.randn(3, s.hidden, device="cuda").to(torch.bfloat16)
    run, given = binding.moe_linear, []
    monkeypatch.setattr(binding, "moe_linear", lambda *a, workspace=None, **kw: (
        given.append(workspace), run(*a, workspace=workspace, **kw))[1])
    block(x, None, batch)
    assert block.status() == (binding.OK, binding.OK)
    assert len(given) == 2
    for workspace in given:
        workspace[:4].view(torch.int32).fill_(binding.ERR_DEVICE_CHECK)
        assert block.status() == (binding.ERR_DEVICE_CHECK, binding.OK)
        assert block.status() == (binding.OK, binding.OK)
