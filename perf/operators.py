"""The operators of a target layer's verification pass, as they are measured:
RMS norm with the residual (plain or 8-bit output), the 8-bit block-scaled
product, rotary positions with the append to the paged cache, and attention of
new tokens over the pages.

`run` computes a pass in its plain form (elementary torch operations in 32
bits), or, where `own` is true, through the framework's entry points.  `exact`
gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEV = "cuda"

_handle = None


def _ops():
    """The framework's handle: one for the process, as a serving program keeps it."""
    global _handle
    if _handle is None:
        from speculative_decoding_verification_22_gb300 import TargetOps
        _handle = TargetOps()
    return _handle


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # the residual norm of one verification round: 5 positions of one sequence
        dict(name="norm round", op="norm", rows=5, d=4096, dtype="bf16", residual=True, out="same"),
        # a batch of 64 sequences with 5 drafts, feeding the 8-bit product
        dict(name="norm batch e4m3", op="norm", rows=384, d=8192, dtype="bf16", residual=True,
             out="e4m3_block"),
        # the tokens of a prompt batch, 8-bit rows for the 8-bit LM head
        dict(name="norm prompt e4m3 rows", op="norm", rows=16384, d=4096, dtype="bf16",
             residual=True, out="e4m3_row"),
        # QKV projection of one round (32 + 8 + 8 heads of 128)
        dict(name="product round", op="matmul", M=5, N=6144, K=4096, dtype="bf16"),
        # a projection of a batch of rounds: ragged row count, wide K
        dict(name="product batch", op="matmul", M=205, N=8192, K=8192, dtype="bf16"),
        # a projection of a prompt chunk
        dict(name="product prompt", op="matmul", M=4096, N=14336, K=4096, dtype="bf16"),
        # rotary positions and cache append of a batch of rounds
        dict(name="rope batch", op="rope", tokens=40, hq=32, hkv=8, D=128, rot=128,
             interleaved=False, scaling="banded", page=16, far=131072, dtype="bf16"),
        # a prompt chunk, part of the head, interleaved pairs
        dict(name="rope prompt", op="rope", tokens=8192, hq=32, hkv=8, D=128, rot=64,
             interleaved=True, scaling="yarn", page=64, far=131072, dtype="fp16"),
        # one round of one sequence: 5 positions over a short cache
        dict(name="attention round", op="attn", B=1, n=5, kv=1000, hq=32, hkv=8, D=128, page=16,
             kind="causal", window=0, dtype="bf16"),
        # single tokens of a ragged batch over long caches
        dict(name="attention decode", op="attn", B=64, n=1, kv=8192, hq=32, hkv=8, D=128, page=16,
             kind="causal", window=0, dtype="bf16"),
        # a tree of 64 drafts and its root for each of 8 sequences
        dict(name="attention tree", op="attn", B=8, n=65, kv=4097, hq=32, hkv=8, D=128, page=64,
             kind="tree", window=0, dtype="bf16"),
        # a chunk of a long prompt over what is cached of it
        dict(name="attention chunk", op="attn", B=1, n=4096, kv=16384, hq=32, hkv=8, D=128,
             page=64, kind="causal", window=0, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "matmul", "rope", "attn"))
    if op == "norm":
        rows = _log(rng, 1, 16384)
        top = min(16384, 16384 * 4096 // rows)
        d = _log(rng, min(64, top), top)
        if rng.random() < 0.75:
            d = max(8, d // 8 * 8)
        return dict(op=op, rows=rows, d=d, dtype=rng.choice(("bf16", "fp16", "fp32")),
                    residual=rng.random() < 0.7, out=rng.choice(("same", "e4m3_block", "e4m3_row")))
    if op == "matmul":
        M = _log(rng, 1, 4096)
        N = _log(rng, 64, 16384)
        K = max(16, _log(rng, 64, 16384) // 16 * 16)
        if M * N * K > 4096 * 14336 * 4096:
            M = max(1, 4096 * 14336 * 4096 // (N * K))
        return dict(op=op, M=M, N=N, K=K, dtype=rng.choice(("bf16", "bf16", "fp16", "fp32")))
    hq, hkv = rng.choice(((32, 8), (64, 8), (16, 16), (8, 1), (24, 8), (12, 4), (28, 4)))
    D = rng.choice((64, 80, 96, 128, 128))
    page = rng.choice((8, 16, 32, 64, 128))
    dtype = rng.choice(("bf16", "bf16", "fp16"))
    if op == "rope":
        return dict(op=op, tokens=min(_log(rng, 1, 8192), 8192 * 48 // (hq + 2 * hkv)), hq=hq,
                    hkv=hkv, D=D, rot=rng.choice((D, D, D // 2)), interleaved=rng.random() < 0.5,
                    scaling=rng.choice(("plain", "linear", "ntk", "banded", "yarn")), page=page,
                    far=_log(rng, 1024, 1 << 20), dtype=dtype)
    kind = rng.choice(("causal", "causal", "tree"))
    n = _log(rng, 1, 65) if kind == "tree" or rng.random() < 0.6 else _log(rng, 65, 4096)
    B = _log(rng, 1, 64) if n <= 65 else _log(rng, 1, 4)
    kv = n + _log(rng, 1, 16384)
    kv = min(kv, max(n, 64 * 8192 * 8 // (B * hkv)))
    while B * n * kv * hq * D > 4096 * 16384 * 32 * 128 // 2 and n > 1:
        n //= 2
    window = _log(rng, 16, 4096) if kind == "causal" and rng.random() < 0.25 else 0
    return dict(op=op, B=B, n=n, kv=max(kv, n), hq=hq, hkv=hkv, D=D, page=page, kind=kind,
                window=window, dtype=dtype)


# --------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)


def _quant(x, block_rows):
    """E4M3 values and scales of blocks [block_rows, 128] of x (a caller's quantised weights or
    rows)."""
    R, K = x.shape
    pr, pk = -R % block_rows, -K % BLOCK
    y = torch.nn.functional.pad(x, (0, pk, 0, pr))
    b = y.view((R + pr) // block_rows, block_rows, (K + pk) // BLOCK, BLOCK)
    s = b.abs().amax(dim=(1, 3)).clamp_min(1e-30) / E4M3_MAX
    q = (b / s[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).view(R + pr, K + pk)[:R, :K]
    return q.to(torch.float8_e4m3fn).contiguous(), s.contiguous()


def _freqs(case):
    """Turns per position of each rotated pair (64 bits) and the magnitude of the rotation."""
    rot, base, factor, orig = case["rot"], 500000.0, 8.0, 8192.0
    i = torch.arange(rot // 2, dtype=torch.float64)
    m = 1.0
    if case["scaling"] == "ntk":
        base *= factor ** (rot / max(rot - 2, 1))
    f = base ** (-2.0 * i / rot) / (2.0 * math.pi)
    if case["scaling"] == "linear":
        f = f / factor
    elif case["scaling"] == "banded":
        # wavelengths over orig are stretched, those under orig / 4 kept, linear between
        t = ((orig * f - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        f = (1.0 - t) * f / factor + t * f
    elif case["scaling"] == "yarn":
        def at(turns):
            return rot * math.log(orig / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
        t = ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        f = t * f / factor + (1.0 - t) * f
        m = 0.1 * math.log(factor) + 1.0
    return f.to(DEV), m


def _tree(g, B, n):
    """Random draft trees of n - 1 nodes and their root: who sees whom, and the same as bits."""
    see = torch.zeros((B, n, n), dtype=torch.bool, device=DEV)
    see[:, 0, 0] = True
    at = torch.arange(B, device=DEV)
    for j in range(1, n):
        parent = (torch.rand(B, generator=g, device=DEV) * j).long().clamp(max=j - 1)
        see[:, j] = see[at, parent]
        see[:, j, j] = True
    words = (n + 31) // 32
    bits = torch.nn.functional.pad(see, (0, words * 32 - n)).view(B * n, words, 32).long()
    bits = (bits << torch.arange(32, device=DEV)).sum(-1)
    return see, torch.where(bits >= 2 ** 31, bits - 2 ** 32, bits).to(torch.int32).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    op = case["op"]
    dt = TYPES[case["dtype"]]
    if op == "norm":
        rows, d = case["rows"], case["d"]
        s["x"] = _randn(g, (rows, d), dt)
        s["res"] = _randn(g, (rows, d), dt, 3.0) if case["residual"] else None
        s["w"] = (1.0 + 0.1 * torch.randn(d, generator=g, device=DEV)).to(dt)
    elif op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        s["a"], s["as"] = _quant(_randn(g, (M, K)), 1)
        s["w"], s["ws"] = _quant(_randn(g, (N, K), scale=0.02), BLOCK)
    elif op == "rope":
        T, hq, hkv, D, page = (case[k] for k in ("tokens", "hq", "hkv", "D", "page"))
        # q, k, v are slices of one fused projection
        qkv = _randn(g, (T, (hq + 2 * hkv) * D), dt)
        s["q"] = qkv[:, :hq * D].view(T, hq, D)
        s["k"] = qkv[:, hq * D:(hq + hkv) * D].view(T, hkv, D)
        s["v"] = qkv[:, (hq + hkv) * D:].view(T, hkv, D)
        s["freqs"], s["m"] = _freqs(case)
        pages = (T + page - 1) // page + 1
        first = int(torch.randint(0, max(1, case["far"]), (1,), generator=g, device=DEV))
        s["pos"] = first + torch.arange(T, device=DEV, dtype=torch.int64)
        slots = torch.randperm(pages, generator=g, device=DEV)[:, None] * page + \
            torch.arange(page, device=DEV)
        s["slots"] = slots.reshape(-1)[:T].contiguous()
        s["kc"] = _randn(g, (pages, page, hkv, D), dt)
        s["vc"] = _randn(g, (pages, page, hkv, D), dt)
    else:
        B, n, kv, hq, hkv, D, page = (case[k] for k in ("B", "n", "kv", "hq", "hkv", "D", "page"))
        # sequences of different age: from a quarter of the longest to the longest
        ctx = kv - n
        lens = (ctx * (0.25 + 0.75 * torch.rand(B, generator=g, device=DEV))).long()
        lens[0] = ctx
        s["kv_len"] = (lens + n).to(torch.int32)
        s["q_start"] = torch.arange(B + 1, device=DEV, dtype=torch.int32) * n
        per = (kv + page - 1) // page
        s["table"] = torch.randperm(B * per, generator=g, device=DEV).to(torch.int32).view(B, per)
        s["kc"] = torch.empty((B * per, page, hkv, D), dtype=dt, device=DEV)
        s["vc"] = torch.empty((B * per, page, hkv, D), dtype=dt, device=DEV)
        s["kc"].normal_(generator=g)
        s["vc"].normal_(generator=g)
        s["q"] = _randn(g, (B * n, hq, D), dt)
        s["scale"] = 1.0 / math.sqrt(D)
        s["see"], s["bits"] = _tree(g, B, n) if case["kind"] == "tree" else (None, None)
    return s


# --------------------------------------------------------------------------- plain forms

def _plain_norm(s):
    c = s["case"]
    h = s["x"].float()
    if s["res"] is not None:
        h = h + s["res"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-6) * s["w"].float()
    res = [h.to(s["x"].dtype)] if s["res"] is not None else []
    if c["out"] == "same":
        return [y.to(s["x"].dtype)] + res
    rows, d = y.shape
    group = BLOCK if c["out"] == "e4m3_block" else d
    y = torch.nn.functional.pad(y, (0, -d % group)).view(rows, -1, group)
    scale = y.abs().amax(-1).clamp_min(1e-30) / E4M3_MAX
    q = (y / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).view(rows, -1)[:, :d]
    return [q.to(torch.float8_e4m3fn), scale if c["out"] == "e4m3_block" else scale[:, 0]] + res


def _plain_matmul(s):
    M, K = s["a"].shape
    N = s["w"].shape[0]
    a = s["a"].float() * s["as"].repeat_interleave(BLOCK, 1)[:, :K]
    ws = s["ws"].repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]
    return (a @ (s["w"].float() * ws).t()).to(TYPES[s["case"]["dtype"]])


def _rotate(x, cos, sin, rot, interleaved):
    a, rest = x[..., :rot].float(), x[..., rot:]
    if interleaved:
        u, v = a[..., 0::2], a[..., 1::2]
    else:
        u, v = a[..., :rot // 2], a[..., rot // 2:]
    u, v = u * cos - v * sin, u * sin + v * cos
    y = torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)
    return torch.cat((y.to(x.dtype), rest), -1)


def _plain_rope(s):
    c = s["case"]
    turns = s["pos"].double()[:, None] * s["freqs"]
    angle = (turns - turns.floor()) * (2.0 * math.pi)
    cos = (angle.cos() * s["m"]).float()[:, None]
    sin = (angle.sin() * s["m"]).float()[:, None]
    q = _rotate(s["q"], cos, sin, c["rot"], c["interleaved"])
    k = _rotate(s["k"], cos, sin, c["rot"], c["interleaved"])
    s["kc"].view(-1, c["hkv"], c["D"])[s["slots"]] = k
    s["vc"].view(-1, c["hkv"], c["D"])[s["slots"]] = s["v"]
    return [q, s["kc"], s["vc"]]


def _plain_attn(s):
    c = s["case"]
    B, n, hq, hkv, D, page = (c[k] for k in ("B", "n", "hq", "hkv", "D", "page"))
    G = hq // hkv
    table = s["table"].long()
    L = table.shape[1] * page
    k = s["kc"][table].view(B, L, hkv, D).permute(0, 2, 3, 1).float()
    q = s["q"].view(B, n, hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, hkv, G * n, D).float()
    x = torch.matmul(q, k).view(B, hkv, G, n, L) * s["scale"]
    del k
    j = torch.arange(L, device=x.device)
    pos = (s["kv_len"].long() - n)[:, None] + torch.arange(n, device=x.device)
    if c["kind"] == "tree":
        at = j[None] - (s["kv_len"].long() - n)[:, None]           # index among the new tokens
        seen = s["see"].gather(2, at.clamp(0, n - 1)[:, None].expand(B, n, L))
        mask = (at < 0)[:, None] | (seen & (at < n)[:, None])
    else:
        mask = j <= pos[..., None]
        if c["window"]:
            mask = mask & (j > pos[..., None] - c["window"])
    x = x.masked_fill_(~mask[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp_(x.sub_(torch.where(top > -math.inf, top, torch.zeros_like(top))))
    total = p.sum(-1, keepdim=True)
    v = s["vc"][table].view(B, L, hkv, D).permute(0, 2, 1, 3).float()
    o = torch.matmul(p.view(B, hkv, G * n, L), v).view(B, hkv, G, n, D)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    return o.permute(0, 3, 1, 2, 4).reshape(B * n, hq, D).to(s["q"].dtype)


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"norm": _plain_norm, "matmul": _plain_matmul, "rope": _plain_rope,
                "attn": _plain_attn}[c["op"]](s)
    ops = _ops()
    if c["op"] == "norm":
        if c["out"] == "same":
            y = ops.rms_norm(s["x"], s["w"], 1e-6, residual=s["res"])
        else:
            y = ops.rms_norm_fp8(s["x"], s["w"], 1e-6, residual=s["res"],
                                 group=BLOCK if c["out"] == "e4m3_block" else 0)
        return y
    if c["op"] == "matmul":
        return ops.matmul_fp8(s["a"], s["as"], s["w"], s["ws"], out_dtype=TYPES[c["dtype"]])
    if c["op"] == "rope":
        q = ops.rope_append(s["q"], s["k"], s["v"], s["pos"], s["slots"], s["freqs"], s["kc"],
                            s["vc"], interleaved=c["interleaved"], magnitude=s["m"])
        return [q, s["kc"], s["vc"]]
    return ops.attention(s["q"], s["kc"], s["vc"], s["table"], s["q_start"], s["kv_len"],
                         scale=s["scale"], window=c["window"], tree_mask=s["bits"])


# --------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    e = 4 if case["dtype"] == "fp32" else 2
    if op == "norm":
        rows, d = case["rows"], case["d"]
        b = rows * d * e + d * e + (2 * rows * d * e if case["residual"] else 0)
        if case["out"] == "same":
            b += rows * d * e
        else:
            b += rows * d + 4 * rows * (-(-d // BLOCK) if case["out"] == "e4m3_block" else 1)
        return {"bytes": b, "flops": 5 * rows * d}
    if op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        kb = -(-K // BLOCK)
        return {"bytes": M * K + N * K + 4 * M * kb + 4 * -(-N // BLOCK) * kb + e * M * N,
                "flops": 2 * M * N * K}
    if op == "rope":
        T, w = case["tokens"], (case["hq"] + 2 * case["hkv"]) * case["D"]
        return {"bytes": 2 * T * w * e + 16 * T,
                "flops": 3 * T * (case["hq"] + case["hkv"]) * case["rot"]}
    B, n, kv, hq, hkv, D = (case[k] for k in ("B", "n", "kv", "hq", "hkv", "D"))
    # the first sequence is the longest, the others average five eighths of its context
    keys = kv + (B - 1) * (n + 0.625 * (kv - n))
    seen = kv - n / 2 + (B - 1) * (n / 2 + 0.625 * (kv - n))
    if case["window"]:
        seen = min(seen, B * case["window"])
        keys = min(keys, B * (case["window"] + n))
    return {"bytes": int(2 * keys * hkv * D * e + 2 * B * n * hq * D * e),
            "flops": int(4 * n * seen * hq * D)}


# --------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        x = s["x"].double()
        h = x if s["res"] is None else x + s["res"].double()
        ms = torch.linalg.vecdot(h, h)[:, None] / h.shape[1]
        y = h / torch.sqrt(ms + 1e-6) * s["w"].double()
        tail = [] if s["res"] is None else [h]
        if case["out"] == "same":
            return [y] + tail
        scale = []
        parts = y.split(BLOCK, 1) if case["out"] == "e4m3_block" else [y]
        q = torch.empty_like(y)
        at = 0
        for part in parts:
            sc = part.abs().max(1).values.clamp(min=1e-30) / 448.0
            q[:, at:at + part.shape[1]] = part / sc[:, None]
            at += part.shape[1]
            scale.append(sc)
        scale = torch.stack(scale, 1) if case["out"] == "e4m3_block" else scale[0]
        return [q, scale] + tail
    if op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        out = torch.zeros((M, N), dtype=torch.float64, device=DEV)
        ws = s["ws"].double()
        nb = torch.arange(N, device=DEV) // BLOCK
        for kb in range((K + BLOCK - 1) // BLOCK):
            sl = slice(kb * BLOCK, min(K, (kb + 1) * BLOCK))
            w = s["w"][:, sl].double() * ws[:, kb][nb][:, None]
            out.addmm_(s["a"][:, sl].double() * s["as"][:, kb].double()[:, None], w.t())
        return out
    if op == "rope":
        rot, D = case["rot"], case["D"]
        turns = torch.outer(s["pos"].double(), s["freqs"].double())
        z = torch.polar(torch.full_like(turns, s["m"]), (turns % 1.0) * (2.0 * math.pi))[:, None]

        def turn(x):
            y = x.double()
            half = rot // 2
            a = torch.arange(half, device=DEV)
            i, j = (2 * a, 2 * a + 1) if case["interleaved"] else (a, a + half)
            w = torch.complex(y[..., i], y[..., j]) * z
            y[..., i], y[..., j] = w.real, w.imag
            return y
        kc, vc = s["kc"].double(), s["vc"].double()
        page = case["page"]
        kc[s["slots"] // page, s["slots"] % page] = turn(s["k"])
        vc[s["slots"] // page, s["slots"] % page] = s["v"].double()
        return [turn(s["q"]), kc, vc]
    B, n, hq, hkv, D, page = (case[k] for k in ("B", "n", "hq", "hkv", "D", "page"))
    G = hq // hkv
    out = torch.zeros((B * n, hq, D), dtype=torch.float64, device=DEV)
    for b in range(B):
        kv = int(s["kv_len"][b])
        at = torch.arange(kv, device=DEV)
        pg, off = s["table"][b].long()[at // page], at % page
        i = torch.arange(n, device=DEV)[:, None] + (kv - n)
        mask = at[None] <= i
        if case["window"]:
            mask = mask & (i - at[None] < case["window"])
        if case["kind"] == "tree":
            mask = torch.ones((n, kv), dtype=torch.bool, device=DEV)
            mask[:, kv - n:] = s["see"][b]
        for h in range(hkv):
            k, v = s["kc"][pg, off, h].double(), s["vc"][pg, off, h].double()
            q = s["q"][b * n:(b + 1) * n, h * G:(h + 1) * G].double()
            x = torch.einsum("igd,jd->gij", q, k) * s["scale"]
            p = torch.softmax(x.masked_fill(~mask, -math.inf), -1)
            out[b * n:(b + 1) * n, h * G:(h + 1) * G] = torch.einsum("gij,jd->igd", p, v)
    return out
