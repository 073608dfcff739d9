"""A whole layer over a paged cache feeding the verify step: the attention block, the
gated feed-forward block with a norm after each, and the log probabilities of what was
emitted (examples/verify_round.py with a feed-forward block) against a plain form."""
import math
import os
import subprocess
import sys

import pytest
import torch

import speculative_decoding_verification_22_gb300 as sv
from layer_common import log_probs_error, log_probs_ref
from target_common import within

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
import verify_round as vr  # noqa: E402

pytestmark = pytest.mark.gpu


def unit(v, w):
    return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + 1e-6) * w.double()


def plain_layer(block, tokens):
    """Final hidden states of whole contexts [B, n] in 64 bits, unquantised."""
    x = block.embed[tokens.long()].double()
    B, n, _ = x.shape
    hq, hkv, D = block.hq, block.hkv, block.D
    qkv = unit(x, block.norm1) @ block.w_qkv.double().t()
    q, k, v = (t.unflatten(-1, (-1, D)) for t in qkv.split([hq * D, hkv * D, hkv * D], -1))
    angle = torch.arange(n, device=x.device).double()[:, None] * block.freqs * 2 * math.pi
    turn = torch.polar(torch.full_like(angle, block.magnitude), angle)[:, None]

    def rotate(t):
        z = torch.complex(*(p.contiguous() for p in t.chunk(2, -1))) * turn
        return torch.cat((z.real, z.imag), -1)
    q, k = rotate(q), rotate(k).repeat_interleave(hq // hkv, 2)
    s = torch.einsum("bihd,bjhd->bhij", q, k) / math.sqrt(D)
    s = s.masked_fill(torch.ones(n, n, device=x.device).triu(1).bool(), -math.inf)
    o = torch.einsum("bhij,bjhd->bihd", s.softmax(-1), v.repeat_interleave(hq // hkv, 2))
    h = x + unit(o.flatten(2) @ block.w_out.double().t(), block.post1)
    y = unit(h, block.norm2)
    g, u = y @ block.w_gate.double().t(), y @ block.w_up.double().t()
    z = (g * torch.sigmoid(g) * u) @ block.w_down.double().t()
    return unit(h + unit(z, block.post2), block.norm3)


def test_the_layer_in_pieces_matches_the_whole_context():
    """A prompt chunk (many rows), then rounds of 5, 1 and 3 tokens (few)."""
    block = vr.Block(ffn=1408)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    tokens = torch.randint(0, block.V, (block.B, 209), generator=g, device="cuda",
                           dtype=torch.int32)
    start = torch.zeros(block.B, dtype=torch.int32, device="cuda")
    got = []
    for n in (200, 5, 1, 3):
        got.append(block.hidden(tokens[:, start[0]:start[0] + n], start))
        start = start + n
    want = plain_layer(block, tokens)
    err = (torch.cat(got, 1).double() - want).norm(dim=-1) / want.norm(dim=-1)
    # What E4M3 does to the QKV projection passes through the layer, by rms: its weights
    # and rows are off by up to 2^-4 a value, 2^-4 / sqrt 3 = 0.036, so q, k and v by
    # 0.036 sqrt 2 = 0.051.  A score (q, k of unit variance, scaled) is then off by
    # 0.051 sqrt 2 = 0.072 and so is each weight, the attention's output with v's own
    # errors by sqrt(0.072^2 + 0.051^2) = 0.088.  Normed, it is as long as x: the state is
    # off by 0.088 in sqrt 2, that is 0.062, each factor of silu(g) u by that, their
    # product by up to 0.124, and x + a + z by sqrt(0.088^2 + 0.124^2) in sqrt 3, that is
    # 0.088: 2^-3 leaves rows of 512 room for four tenths more.  (bf16's 2^-8 are far
    # below; the next test takes the part behind the attention by itself.)
    assert err.max().item() < 2 ** -3, err.max().item()
    assert block.ops.status() == sv.SV_OK


@pytest.mark.parametrize("rows", [1, 20, 300])
def test_the_layer_behind_the_attention(rows):
    """From the attention's output on, against 64 bits.  Each of the six roundings to
    bf16 is off by 2^-8 at most, 2^-8 / sqrt 3 by rms; the two norms make each branch as
    long as the state, so none grows: the gated product doubles what reaches it (two
    roundings before, each in two factors), and the final rounding is one more.  By rms
    sqrt(1 + 1 + 4 + 4 + 1 + 1 + 1) 2^-8 / sqrt 3 = 0.0081 of the state."""
    block = vr.Block(ffn=1408, seed=rows)
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    o = torch.randn(rows, block.hq * block.D, generator=g, device="cuda").bfloat16()
    x = torch.randn(rows, block.d, generator=g, device="cuda").bfloat16()
    got = block.feed_forward(o, x)
    h = x.double() + unit(o.double() @ block.w_out.double().t(), block.post1)
    y = unit(h, block.norm2)
    a, u = y @ block.w_gate.double().t(), y @ block.w_up.double().t()
    z = (a * torch.sigmoid(a) * u) @ block.w_down.double().t()
    want = unit(h + unit(z, block.post2), block.norm3)
    err = (got.double() - want).norm(dim=-1) / want.norm(dim=-1)
    assert err.max().item() < 0.0081, err.max().item()
    assert block.ops.status() == sv.SV_OK


def test_rounds_with_their_log_probabilities():
    """Greedy rounds: each emitted token is the first alternative of its row, and the
    scores are those of the verify step's logits."""
    block = vr.Block(seed=3, ffn=704)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    prompt = torch.randint(0, block.V, (block.B, 40), generator=g, device="cuda",
                           dtype=torch.int32)
    prompt[:, 20:] = prompt[:, :20]
    ctx, length, accepted, scores = vr.generate(block, prompt, 10, top=3)
    assert block.ops.status() == sv.SV_OK and block.verify.status() == sv.SV_OK
    assert torch.equal(length, 40 + 10 + accepted.sum(0).int()) and len(scores) == 10
    at = torch.full((block.B,), 40, device="cuda")
    for n_acc, (lp, entropy, ids, top_lp) in zip(accepted, scores):
        for b in range(block.B):
            n = int(n_acc[b]) + 1
            assert torch.equal(ids[b, :n, 0], ctx[b, at[b]:at[b] + n])
            assert torch.equal(lp[b, :n], top_lp[b, :n, 0])
            assert (lp[b, n:] == 0).all() and (entropy[b] > 0).all()
            at[b] += n
    # the last round's, against its logits
    logits = block.verify.logits()
    V, R = block.V, logits.shape[0]
    lp, _, ids, top_lp = scores[-1]
    want = log_probs_ref(logits, ids[..., :1].reshape(R, 1), 3, 1.0)
    assert torch.equal(ids.view(R, 3), want[2])
    within(top_lp.view(R, 3), want[3], log_probs_error(want[3], V))


def test_without_a_feed_forward_block_the_example_is_as_it_was():
    """The same weights whether or not the block has one behind them."""
    plain, wide = vr.Block(seed=5), vr.Block(seed=5, ffn=64)
    for name in ("embed", "norm1", "norm2", "w_qkv", "w_out", "head"):
        assert torch.equal(getattr(plain, name), getattr(wide, name)), name
    assert not hasattr(plain, "w_gate")


def test_the_example_runs_from_the_command_line():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "verify_round.py"),
                        "--rounds", "3", "--batch", "2", "--ffn", "256", "--top", "4"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "status (0, 0)" in r.stdout and "log probability" in r.stdout
