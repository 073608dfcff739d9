"""Plain 64-bit implementations of the target-layer operators, and the inputs
and tolerances of their tests.

Half a step of a type t is eps(t) / 2 of the value (bf16 2^-8, fp16 2^-11,
fp32 2^-24, E4M3 2^-4); the tolerances below count such roundings.
"""
import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# half of the smallest step near zero
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def randn(g, shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device=g.device) * scale).to(dtype)


def within(got, ref, bound):
    """got finite exactly where ref is, and within the bound there."""
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), "NaN in other places"
    fine = torch.isfinite(ref)
    assert torch.equal(got[~fine & ~torch.isnan(ref)], ref[~fine & ~torch.isnan(ref)])
    if fine.any():
        over = ((got - ref).abs() - bound)[fine].max().item()
        assert over <= 0, f"over the bound by {over:.3g}"


# ---- norm -------------------------------------------------------------------

def norm_ref(x, w, eps, residual=None):
    h = x.double() + (0 if residual is None else residual.double())
    return h * torch.rsqrt((h * h).mean(1, keepdim=True) + eps) * w.double(), h


# A thread adds up to 128 squares one after another (d <= 2^16 in the tests),
# five shuffles and 32 warps follow: < 256 roundings of positive terms, halved
# by the root, and a few more of the other steps.
NORM_REL = 130 * 2.0 ** -24


# ---- 8-bit product ------------------------------------------------------------

def quant_blocks(x, rows):
    """E4M3 values and fp32 scales of blocks [rows, 128] of x."""
    R, K = x.shape
    y = torch.nn.functional.pad(x, (0, -K % 128, 0, -R % rows))
    b = y.view(y.shape[0] // rows, rows, y.shape[1] // 128, 128)
    s = b.abs().amax(dim=(1, 3)).clamp_min(1e-30) / 448.0
    q = (b / s[:, None, :, None]).clamp(-448, 448).view(y.shape)[:R, :K]
    return q.to(torch.float8_e4m3fn).contiguous(), s.float().contiguous()


def matmul_ref(a, sa, w, sw):
    """The product and the same sum of magnitudes."""
    K, N = a.shape[1], w.shape[0]
    x = a.double() * sa.double().repeat_interleave(128, 1)[:, :K]
    y = w.double() * sw.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return x @ y.t(), x.abs() @ y.abs().t()


def matmul_bound(ref, mags, K, dtype):
    """Up to 128 products are summed by the tensor cores, whose additions may
    cut instead of round (2^-23 each); then the blocks are scaled (two
    roundings) and summed in fp32 (half a step each)."""
    blocks = -(-K // 128)
    return (mags * (128 * 2.0 ** -23 + (blocks + 8) * 2.0 ** -24)
            + ref.abs() * HALF_STEP[dtype] * 1.01 + TINY[dtype])


# ---- rotary -------------------------------------------------------------------

def rope_ref(x, positions, freqs, interleaved, magnitude):
    """Rotated x, and |a| + |b| of each element's pair (0 where copied)."""
    rot = 2 * freqs.numel()
    y, mag = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    turns = positions.double()[:, None] * freqs
    angle = ((turns - turns.floor()) * (2 * math.pi))[:, None]
    i = torch.arange(rot // 2, device=x.device)
    i, j = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    a, b = x.double()[..., i], x.double()[..., j]
    y[..., i] = magnitude * (a * angle.cos() - b * angle.sin())
    y[..., j] = magnitude * (a * angle.sin() + b * angle.cos())
    mag[..., i] = mag[..., j] = a.abs() + b.abs()
    return y, mag * magnitude


def rope_bound(ref, mag, dtype):
    """cos and sin: the fraction of a turn is rounded to fp32 (2^-25 of up to
    half a turn, 2 pi times that in radians), two units of the functions, the
    magnitude, the products: below 2^-20 of |a| + |b|."""
    return mag * 2.0 ** -20 + ref.abs() * HALF_STEP[dtype] * 1.01 + TINY[dtype]


# ---- attention ------------------------------------------------------------------

def build_cache(g, lens, page, hkv, D, dtype, spare=3, fill=float("nan"), heads_first=False):
    """Shuffled pages holding K and V of sequences of the given lengths; what
    no sequence uses is `fill`.  Returns caches, table and the plain K, V."""
    per = max(1, max(-(-n // page) for n in lens))
    pages = len(lens) * per + spare
    order = torch.randperm(pages, generator=g, device=g.device)
    table = order[:len(lens) * per].to(torch.int32).view(len(lens), per).contiguous()
    shape = (pages, hkv, page, D) if heads_first else (pages, page, hkv, D)
    kc = torch.full(shape, fill, dtype=dtype, device=g.device)
    vc = torch.full(shape, fill, dtype=dtype, device=g.device)
    if heads_first:
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    ks, vs = [], []
    for b, n in enumerate(lens):
        k, v = randn(g, (n, hkv, D), dtype), randn(g, (n, hkv, D), dtype)
        at = torch.arange(n, device=g.device)
        pg = table[b].long()[at // page]
        kc[pg, at % page] = k
        vc[pg, at % page] = v
        ks.append(k)
        vs.append(v)
    return kc, vc, table, ks, vs


def attention_ref(q, ks, vs, news, scale, window=0, see=None):
    """o, sum_j p_j |v_j|, lse and the largest sum |q||k| of a seen score;
    `see`: [n, n] of each sequence for a tree.  What is masked is left out."""
    T, Hq, D = q.shape
    o = torch.zeros((T, Hq, D), dtype=torch.float64, device=q.device)
    mag = torch.zeros_like(o)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=q.device)
    big = 0.0
    t0 = 0
    for b, n in enumerate(news):
        kv, hkv = ks[b].shape[0], ks[b].shape[1]
        G = Hq // hkv
        ctx = kv - n
        if n and kv:
            j = torch.arange(kv, device=q.device)[None]
            at = torch.arange(n, device=q.device)[:, None] + ctx
            mask = j <= at
            if window:
                mask = mask & (j > at - window)
            if see is not None:
                mask = torch.ones((n, kv), dtype=torch.bool, device=q.device)
                if ctx >= 0:
                    mask[:, ctx:] = see[b]
                else:
                    mask[:] = see[b][:, -ctx:]
            for h in range(Hq):
                k, v = ks[b][:, h // G].double(), vs[b][:, h // G].double()
                qh = q[t0:t0 + n, h].double()
                # rows one by one where something is not finite, so that only
                # what a row sees enters its sums
                plain = bool(torch.isfinite(k).all() and torch.isfinite(v).all())
                rows = [slice(0, n)] if plain else [slice(i, i + 1) for i in range(n)]
                for r in rows:
                    m = mask[r]
                    keep = slice(None) if plain else m[0]
                    kk, vv, mm = k[keep], v[keep], m[:, keep]
                    if not plain and kk.shape[0] == 0:
                        continue
                    x = (qh[r] @ kk.t() * scale).masked_fill(~mm, -math.inf)
                    top = x.amax(1, keepdim=True)
                    some = top != -math.inf
                    p = torch.exp(x - torch.where(some, top, 0.0))
                    l = p.sum(1, keepdim=True)
                    p = p / torch.where(some, l, 1.0)
                    rr = slice(t0 + r.start, t0 + r.stop)
                    o[rr, h] = p @ vv
                    mag[rr, h] = p @ vv.abs()
                    lse[rr, h] = torch.where(some, top + l.log(), -math.inf)[:, 0]
                    s = (qh[r].abs() @ kk.abs().t())[mm]
                    s = s[torch.isfinite(s)]
                    if s.numel():
                        big = max(big, s.max().item() * abs(scale))
        t0 += n
    return o, mag, lse, big


def score_error(big, D):
    """A score's sum of D products by the tensor cores (cut additions, 2^-23
    each) and its scaling, and the exponential's own error."""
    return (D + 4) * 2.0 ** -23 * big + 2.0 ** -20


def attention_bound(o, mag, big, D, dtype):
    """Each weight is off by its score's error (twice: its own and the sum's)
    and one rounding to the 16-bit type before its product; the output by one
    more."""
    w = 2 * score_error(big, D) + HALF_STEP[dtype] + 2.0 ** -14
    return mag * w + o.abs() * HALF_STEP[dtype] * 1.01 + TINY[dtype]
