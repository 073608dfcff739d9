"""Speculative decoding rounds through one attention block of a target with
random weights: the target-layer operators feed the verify step.

A round takes each sequence's last token and up to K drafted ones:

    embeddings -> residual RMS norm (E4M3, scales of 128) -> 8-bit QKV product
    -> rotary positions, K and V into the pages -> attention over the pages
    -> output projection (bf16) -> residual norm -> spec_verify_run

and the cache is rolled back by its length alone: what the accepted tokens do
not cover is overwritten by the next round.  Drafts come from prompt lookup.

    python examples/verify_round.py [--rounds 16] [--batch 4] [--drafts 4]
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
    """The weights and the paged cache of one attention block."""

    def __init__(self, V=1000, d=512, hq=8, hkv=2, D=64, B=4, K=4, page=16, max_len=1024,
                 seed=0, device="cuda"):
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
        o = o.view(-1, hq * D) @ self.w_out.t()
        return self.ops.rms_norm(o, self.norm2, residual=x)[0].view(B, n, self.d)

    def round(self, last, draft, start, temperature=0.0, uniforms=None):
        """One verified round: `last` [B] the newest token of each sequence (not
        yet cached), `draft` int32 [B, K] (-1 ends it).  Returns the emitted
        tokens [B, K+1] and the accepted counts [B]."""
        tokens = torch.cat((last[:, None], draft.clamp_min(0)), 1)
        h = self.hidden(tokens, start)
        if uniforms is None:
            uniforms = torch.zeros(self.B, self.K + 1, device=h.device)
        return self.verify.run(h, self.head, draft, None, uniforms, temperature)


def generate(block, prompt, rounds):
    """Greedy decoding from prompt [B, n] with prompt-lookup drafts; returns the
    contexts, their lengths and the accepted count of each round."""
    B, n = prompt.shape
    ctx = torch.zeros(B, n + rounds * (block.K + 1) + 1, dtype=torch.int32, device=prompt.device)
    ctx[:, :n] = prompt
    length = torch.full((B,), n, dtype=torch.int32, device=prompt.device)
    block.hidden(prompt[:, :-1], torch.zeros_like(length))  # the prompt as one chunk
    accepted = []
    col = torch.arange(block.K + 1, device=prompt.device)
    for _ in range(rounds):
        draft, _ = sv.spec_ngram_draft(ctx, length, block.K, 1, 3)
        last = ctx.gather(1, (length - 1).long()[:, None])[:, 0]
        out, n_acc = block.round(last, draft, length - 1)
        at = length.long()[:, None] + col
        live = col[None] <= n_acc[:, None]
        ctx.scatter_(1, torch.where(live, at, ctx.shape[1] - 1), torch.where(live, out, 0))
        length += n_acc + 1
        accepted.append(n_acc.clone())
    return ctx, length, torch.stack(accepted)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--rounds", type=int, default=16)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--drafts", type=int, default=4)
    a = ap.parse_args()
    block = Block(B=a.batch, K=a.drafts)
    prompt = torch.randint(0, block.V, (a.batch, 48), device="cuda", dtype=torch.int32)
    prompt[:, 24:] = prompt[:, :24]  # something to look up
    ctx, length, accepted = generate(block, prompt, a.rounds)
    codes = block.ops.status(), block.verify.status()
    print(f"{a.rounds} rounds, {a.batch} sequences: lengths {length.tolist()}, "
          f"accepted {accepted.sum(0).tolist()} of the drafts, status {codes}")


if __name__ == "__main__":
    main()
