"""The target-layer operators together: an attention block over a paged cache
feeding the verify step (examples/verify_round.py) against a plain form."""
import math
import os
import sys

import pytest
import torch

import speculative_decoding_verification_22_gb300 as sv

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
import verify_round as vr  # noqa: E402

pytestmark = pytest.mark.gpu


def plain_hidden(block, tokens):
    """Final hidden states of whole contexts [B, n] in 64 bits, unquantised."""
    x = block.embed[tokens.long()].double()
    B, n, d = x.shape
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * block.norm1.double()
    qkv = y @ block.w_qkv.double().t()
    hq, hkv, D = block.hq, block.hkv, block.D
    q = qkv[..., :hq * D].view(B, n, hq, D)
    k = qkv[..., hq * D:(hq + hkv) * D].view(B, n, hkv, D)
    v = qkv[..., (hq + hkv) * D:].view(B, n, hkv, D)
    angle = torch.arange(n, device=x.device).double()[:, None] * block.freqs * 2 * math.pi
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]

    def turn(t):
        a, b = t.chunk(2, -1)
        return torch.cat((a * cos - b * sin, a * sin + b * cos), -1) * block.magnitude
    q, k = turn(q), turn(k)
    k, v = k.repeat_interleave(hq // hkv, 2), v.repeat_interleave(hq // hkv, 2)
    s = torch.einsum("bihd,bjhd->bhij", q, k) / math.sqrt(D)
    s = s.masked_fill(torch.ones(n, n, device=x.device).triu(1).bool(), -math.inf)
    o = torch.einsum("bhij,bjhd->bihd", s.softmax(-1), v).reshape(B, n, hq * D)
    h = x + o @ block.w_out.double().t()
    return h * torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-6) * block.norm2.double()


def test_block_in_pieces_matches_the_whole_context():
    """A prompt chunk, then rounds of 5, 1 and 3 tokens."""
    block = vr.Block()
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    tokens = torch.randint(0, block.V, (block.B, 209), generator=g, device="cuda",
                           dtype=torch.int32)
    start = torch.zeros(block.B, dtype=torch.int32, device="cuda")
    got = []
    for n in (200, 5, 1, 3):
        got.append(block.hidden(tokens[:, start[0]:start[0] + n], start))
        start = start + n
    want = plain_hidden(block, tokens)
    err = (torch.cat(got, 1).double() - want).norm(dim=-1) / want.norm(dim=-1)
    # weights and rows in E4M3: at most 2^-4 a value each, with random signs;
    # the residual's norm is the larger part of the output's
    assert err.max().item() < 2 ** -4, err.max().item()
    assert block.ops.status() == sv.SV_OK


def test_rounds_emit_the_target_argmax_and_roll_back():
    """Greedy rounds with prompt-lookup drafts: every emitted token is the plain
    target's argmax where that one is clear."""
    block = vr.Block(seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    prompt = torch.randint(0, block.V, (block.B, 40), generator=g, device="cuda",
                           dtype=torch.int32)
    prompt[:, 20:] = prompt[:, :20]
    ctx, length, accepted = vr.generate(block, prompt, 12)
    assert block.ops.status() == sv.SV_OK and block.verify.status() == sv.SV_OK
    assert torch.equal(length, 40 + 12 + accepted.sum(0).int())
    n = int(length.min())
    logits = plain_hidden(block, ctx[:, :n]) @ block.head.double().t()
    top = logits.topk(2, -1)
    clear = (top.values[..., 0] - top.values[..., 1]) > 0.5
    want, got = top.indices[:, 39:n - 1, 0], ctx[:, 40:n].long()
    use = clear[:, 39:n - 1]
    assert use.float().mean() > 0.2
    assert torch.equal(want[use], got[use])
