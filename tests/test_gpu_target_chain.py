"""The target-layer operators handing on to the other forms of the verify step:
the norm's E4M3 rows to the FP8 LM head, and a tree of drafts through its mask and
the attention to the tree walk."""
import os
import sys

import numpy as np
import pytest
import torch

import oracle
import spec_inputs as si
import speculative_decoding_verification_22_gb300 as sv
from gpu_common import FLAG_GREEDY, compare_tokens
from test_gpu_target_round import plain_hidden

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
import verify_round as vr  # noqa: E402

pytestmark = pytest.mark.gpu


class LastNorm:
    """The block's operators; keeps what the final norm was given."""

    def __init__(self, ops):
        self.ops = ops

    def __getattr__(self, name):
        return getattr(self.ops, name)

    def rms_norm(self, x, weight, residual):
        self.given = x, weight, residual
        return self.ops.rms_norm(x, weight, residual=residual)


def prompt_of(block, n, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    tokens = torch.randint(0, block.V, (block.B, n), generator=g, device="cuda",
                           dtype=torch.int32)
    start = torch.zeros(block.B, dtype=torch.int32, device="cuda")
    block.hidden(tokens[:, :-1], start)  # all but the newest are cached
    return tokens, start + n - 1


def plain_choice(block, tokens):
    """The plain target's next token of contexts [B, n] (E4M3 nowhere)."""
    return (plain_hidden(block, tokens)[:, -1] @ block.head.double().t()).argmax(-1).int()


def test_rows_of_the_norm_in_e4m3_feed_the_fp8_head():
    """The final norm with a scale a row, its values and scales verified as they
    are: logits and tokens of the oracle on the same numbers. Drafts follow the
    plain target for two tokens."""
    block = vr.Block(seed=5)
    B, K, d = block.B, block.K, block.d
    tokens, start = prompt_of(block, 50, 6)
    ctx = tokens
    for _ in range(2):
        ctx = torch.cat((ctx, plain_choice(block, ctx)[:, None]), 1)
    draft = torch.zeros(B, K, dtype=torch.int32, device="cuda")
    draft[:, :2] = ctx[:, -2:]
    block.ops = LastNorm(block.ops)
    block.hidden(torch.cat((tokens[:, -1:], draft), 1), start)
    x, weight, residual = block.ops.given
    h8, scale, _ = block.ops.rms_norm_fp8(x, weight, residual=residual, group=0)
    h8, scale = h8.view(torch.uint8).view(B, K + 1, d), scale.view(B, K + 1)
    W8, ws = si.quantize_rows_e4m3(block.head)
    uniforms = torch.zeros(B, K + 1, device="cuda")
    eng = sv.SpecVerify(block.V, d, B, K, "fp8")
    out, n = eng.run_fp8(h8, scale, W8, ws, draft, None, uniforms, 0.0)
    assert eng.status() == sv.SV_OK and block.ops.status() == sv.SV_OK
    ref = oracle.verify_fp8(si.to_oracle(h8), si.to_oracle(scale), si.to_oracle(W8),
                            si.to_oracle(ws), si.to_oracle(draft), None, si.to_oracle(uniforms),
                            0.0, want_logits=True)
    assert np.abs(eng.logits().cpu().numpy() - ref["logits"]).max() <= 2e-2
    got = {"tokens": out.cpu().numpy(), "n_accepted": n.cpu().numpy()}
    bad, flagged = compare_tokens(got, ref, 0.0)
    assert bad == 0 and flagged == 0
    assert (got["n_accepted"] > 0).any()
    # and the plain target's choice where that one is clear
    top = (plain_hidden(block, tokens)[:, -1] @ block.head.double().t()).topk(2, -1)
    clear = (top.values[:, 0] - top.values[:, 1]) > 0.5
    assert clear.any() and torch.equal(out[clear, 0].long(), top.indices[clear, 0])
    eng.close()


def test_a_tree_goes_from_drafts_through_the_attention_to_the_walk():
    """Nodes at their depths' positions, each seeing the context and its ancestors:
    hidden states near the plain target's on every node's own path, and the walk
    of the oracle on them."""
    N = 6
    block = vr.Block(seed=8, K=N)
    B, d, hq, hkv, D = block.B, block.d, block.hq, block.hkv, block.D
    tokens, start = prompt_of(block, 45, 9)
    rng = np.random.default_rng(10)
    parents = np.array([[rng.integers(-1, j) if j else -1 for j in range(N)] for _ in range(B)],
                       np.int32)
    paths = [[tokens[b] for _ in range(N + 1)] for b in range(B)]  # row 0 the root
    nodes = np.zeros((B, N), np.int32)
    depth = np.zeros((B, N + 1), np.int64)
    for b in range(B):
        for j in range(N):
            above = parents[b, j] + 1
            follow = plain_choice(block, paths[b][above][None])[0]
            nodes[b, j] = int(follow) if j < 2 or rng.random() < 0.5 else rng.integers(block.V)
            paths[b][j + 1] = torch.cat((paths[b][above], tokens.new_tensor([nodes[b, j]])))
            depth[b, j + 1] = depth[b, above] + 1
    par, tree = torch.from_numpy(parents).cuda(), torch.from_numpy(nodes).cuda()

    ops = block.ops
    x = block.embed[torch.cat((tokens[:, -1:], tree), 1).reshape(-1).long()]
    a8, scale = ops.rms_norm_fp8(x, block.norm1)
    qkv = ops.matmul_fp8(a8, scale, block.w8, block.ws)
    q, k, v = (t.view(-1, t.shape[1] // D, D) for t in
               qkv.split([hq * D, hkv * D, hkv * D], 1))
    at = start.long()[:, None] + torch.from_numpy(depth).cuda()
    slots = block.slots(start.long()[:, None] + torch.arange(N + 1, device="cuda"))
    q = ops.rope_append(q, k, v, at.view(-1).contiguous(), slots, block.freqs, block.k_cache,
                        block.v_cache, magnitude=block.magnitude)
    q_start = torch.arange(B + 1, device="cuda", dtype=torch.int32) * (N + 1)
    o = ops.attention(q, block.k_cache, block.v_cache, block.table, q_start,
                      (start + N + 1).int(), tree_mask=ops.tree_mask(par))
    o = o.view(-1, hq * D) @ block.w_out.t()
    h = ops.rms_norm(o, block.norm2, residual=x)[0].view(B, N + 1, d)
    out, path, n = block.verify.run_tree_greedy(h, block.head, tree, par)
    assert ops.status() == sv.SV_OK and block.verify.status() == sv.SV_OK

    want = torch.stack([torch.stack([plain_hidden(block, p[None])[0, -1] for p in rows])
                        for rows in paths])
    err = (h.double() - want).norm(dim=-1) / want.norm(dim=-1)
    # weights and rows in E4M3, at most 2^-4 a value each (see the rounds' tests)
    assert err.max().item() < 2 ** -4, err.max().item()
    ref = oracle.tree_greedy(si.to_oracle(h), si.to_oracle(block.head), nodes, parents)
    assert (ref["gap"] > FLAG_GREEDY).all()
    assert np.array_equal(out.cpu().numpy(), ref["tokens"])
    assert np.array_equal(path.cpu().numpy(), ref["nodes"])
    assert np.array_equal(n.cpu().numpy(), ref["n"]) and (ref["n"] > 0).any()
