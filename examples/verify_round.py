"""Speculative decoding rounds through one attention block of a target with
random weights: the target-layer operators feed the verify step.

A round takes each sequence's last token and up to K drafted ones:

    embeddings -> residual RMS norm (E4M3, scales of 128) -> 8-bit QKV product
    -> rotary positions, K and V into the pages -> attention over the pages
    -> output projection (bf16) -> residual norm -> spec_verify_run

With a feed-forward block (--ffn) the layer goes on behind the attention, with a
norm after each of its blocks:

    -> output projection -> norm after, residual, norm before -> gated projections
    -> down projection -> norm after, residual, final norm -> spec_verify_run

and with --top each round says how likely its tokens were and what else was, from
the verify step's logits.  The cache is rolled back by its length alone: what the
accepted tokens do not cover is overwritten by the next round.  Drafts come from
prompt lookup.

    python examples/verify_round.py [--rounds 16] [--batch 4] [--drafts 4]
                                    [--ffn 1408] [--top 5]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_22_gb300 as sv  # noqa: E402

E4M3_MAX = 448.0


def quantise_weight(w):
    """E4M3 values and one scale per block of 128 x 128."""
    n, k = w.shape
    p = torch.nn.functional.pad(w.float(), (0, -k % 128, 0, -n % 128))
    b = p.view(p.shape[0] // 128, 128, p.shape[1] // 128, 128)
    s = b.abs().amax(dim=(1, 3)).clamp_min(1e-30) / E4M3_MAX
    q = (b / s[:, None, :, None]).view(p.shape)[:n, :k]
    return q.to(torch.float8_e4m3fn).contiguous(), s.contiguous()


class Block:
    """The weights and the paged cache of one attention block, and with ``ffn`` > 0
    of the gated feed-forward block behind it."""

    def __init__(self, V=1000, d=512, hq=8, hkv=2, D=64, B=4, K=4, page=16, max_len=1024,
                 seed=0, device="cuda", ffn=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def randn(*shape, std=1.0):
            return torch.randn(*shape, generator=g, device=device) * std
        self.V, self.d, self.hq, self.hkv, self.D, self.B, self.K = V, d, hq, hkv, D, B, K
        self.page = page
        self.embed = randn(V, d).bfloat16()
        self.norm1 = (1 + 0.1 * randn(d)).bfloat16()
        self.norm2 = (1 + 0.1 * randn(d)).bfloat16()
        self.w_qkv = randn((hq + 2 * hkv) * D, d, std=d ** -0.5)
        self.w8, self.ws = quantise_weight(self.w_qkv)
        self.w_out = randn(d, hq * D, std=(hq * D) ** -0.5).bfloat16()
        self.head = randn(V, d, std=d ** -0.5).bfloat16()
        pages = -(-max_len // page)
        self.k_cache = torch.empty(B * pages, page, hkv, D, dtype=torch.bfloat16, device=device)
        self.v_cache = torch.empty_like(self.k_cache)
        self.table = torch.randperm(B * pages, generator=g, device=device).int().view(B, pages)
        self.ffn = ffn
        if ffn:
            self.w_gate, self.w_up = randn(2, ffn, d, std=d ** -0.5).bfloat16()
            self.w_down = randn(d, ffn, std=ffn ** -0.5).bfloat16()
            self.post1, self.post2, self.norm3 = (1 + 0.1 * randn(3, d)).bfloat16()
        freqs, self.magnitude = sv.spec_target_rope_freqs(D, 500000.0, "banded", 8.0, 8192)
        self.freqs = freqs.to(device)
        self.ops = sv.TargetOps(device)
        self.verify = sv.SpecVerify(V, d, B, K, "bf16", device=device)

    def slots(self, positions):
        """Cache slots of positions [B, n]."""
        page = self.table.gather(1, (positions // self.page)).long()
        return (page * self.page + positions % self.page).view(-1).contiguous()

    def hidden(self, tokens, start):
        """Final hidden states [B, n, d] of the tokens [B, n] that follow the
        `start` [B] cached ones; their keys and values are cached."""
        B, n = tokens.shape
        x = self.embed[tokens.reshape(-1).long()]
        positions = start.long()[:, None] + torch.arange(n, device=x.device)
        a8, scale = self.ops.rms_norm_fp8(x, self.norm1)
        qkv = self.ops.matmul_fp8(a8, scale, self.w8, self.ws)
        hq, hkv, D = self.hq, self.hkv, self.D
        q = qkv[:, :hq * D].view(-1, hq, D)
        k = qkv[:, hq * D:(hq + hkv) * D].view(-1, hkv, D)
        v = qkv[:, (hq + hkv) * D:].view(-1, hkv, D)
        q = self.ops.rope_append(q, k, v, positions.view(-1), self.slots(positions), self.freqs,
                                 self.k_cache, self.v_cache, magnitude=self.magnitude)
        q_start = torch.arange(B + 1, device=x.device, dtype=torch.int32) * n
        o = self.ops.attention(q, self.k_cache, self.v_cache, self.table, q_start,
                               (start + n).int())
        if self.ffn:
            return self.feed_forward(o.view(-1, hq * D), x).view(B, n, self.d)
        o = self.ops.linear(o.view(-1, hq * D), self.w_out)
        return self.ops.rms_norm(o, self.norm2, residual=x)[0].view(B, n, self.d)

    def feed_forward(self, o, x):
        """The layer from the attention's output on, x its residual."""
        y, h = self.ops.block_norm(self.ops.linear(o, self.w_out), x, self.norm2,
                                   post_weight=self.post1)
        y = self.ops.gated_linear(y, self.w_gate, self.w_up, activation="silu")
        return self.ops.block_norm(self.ops.linear(y, self.w_down), h, self.norm3,
                                   post_weight=self.post2)[0]

    def round(self, last, draft, start, temperature=0.0, uniforms=None):
        """One verified round: `last` [B] the newest token of each sequence (not
        yet cached), `draft` int32 [B, K] (-1 ends it).  Returns the emitted
        tokens [B, K+1] and the accepted counts [B]."""
        tokens = torch.cat((last[:, None], draft.clamp_min(0)), 1)
        h = self.hidden(tokens, start)
        if uniforms is None:
            uniforms = torch.zeros(self.B, self.K + 1, device=h.device)
        return self.verify.run(h, self.head, draft, None, uniforms, temperature)


def generate(block, prompt, rounds, top=0):
    """Greedy decoding from prompt [B, n] with prompt-lookup drafts; returns the
    contexts, their lengths and the accepted count of each round, and with ``top`` > 0
    each round's log probabilities (SpecVerify.log_probs)."""
    B, n = prompt.shape
    ctx = torch.zeros(B, n + rounds * (block.K + 1) + 1, dtype=torch.int32, device=prompt.device)
    ctx[:, :n] = prompt
    length = torch.full((B,), n, dtype=torch.int32, device=prompt.device)
    block.hidden(prompt[:, :-1], torch.zeros_like(length))  # the prompt as one chunk
    accepted, scores = [], []
    col = torch.arange(block.K + 1, device=prompt.device)
    for _ in range(rounds):
        draft, _ = sv.spec_ngram_draft(ctx, length, block.K, 1, 3)
        last = ctx.gather(1, (length - 1).long()[:, None])[:, 0]
        out, n_acc = block.round(last, draft, length - 1)
        if top:
            scores.append(block.verify.log_probs(out, top))
        at = length.long()[:, None] + col
        live = col[None] <= n_acc[:, None]
        ctx.scatter_(1, torch.where(live, at, ctx.shape[1] - 1), torch.where(live, out, 0))
        length += n_acc + 1
        accepted.append(n_acc.clone())
    done = ctx, length, torch.stack(accepted)
    return (*done, scores) if top else done


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--rounds", type=int, default=16)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--drafts", type=int, default=4)
    ap.add_argument("--ffn", type=int, default=0, help="width of a gated feed-forward block")
    ap.add_argument("--top", type=int, default=0, help="alternatives to each emitted token")
    a = ap.parse_args()
    block = Block(B=a.batch, K=a.drafts, ffn=a.ffn)
    prompt = torch.randint(0, block.V, (a.batch, 48), device="cuda", dtype=torch.int32)
    prompt[:, 24:] = prompt[:, :24]  # something to look up
    ctx, length, accepted, *scores = generate(block, prompt, a.rounds, a.top)
    codes = block.ops.status(), block.verify.status()
    print(f"{a.rounds} rounds, {a.batch} sequences: lengths {length.tolist()}, "
          f"accepted {accepted.sum(0).tolist()} of the drafts, status {codes}")
    if a.top:
        total = sum(s[0].sum(1) for s in scores[0])
        print(f"log probability of the new tokens: {[round(t, 2) for t in total.tolist()]}; "
              f"sequence 0's first token was chosen over {scores[0][0][2][0, 0].tolist()}")


if __name__ == "__main__":
    main()
