"""The operators of the second half of a target layer, and of what a service says
of its answers, as they are measured: the 16-bit product with bias, activation and
residual, the gated projections of a feed-forward block, the norms around a block
with its gate and scale, and the log probabilities of logit rows.

`run` computes a pass in its plain form (elementary torch operations in 32 bits),
or, where `own` is true, through the framework's entry points.  `exact` gives the
same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
EPS = 1e-6
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
        # the output projection of one verification round, onto the residual
        dict(name="linear round", op="linear", M=5, N=4096, K=4096, dtype="bf16", bias=False,
             act="none", residual=True),
        # the down projection of eight sequences' rounds, onto the residual
        dict(name="linear rounds", op="linear", M=40, N=4096, K=14336, dtype="bf16", bias=False,
             act="none", residual=True),
        # the first half of a plain feed-forward block for a ragged batch of rounds
        dict(name="linear batch", op="linear", M=205, N=8190, K=8192, dtype="fp16", bias=True,
             act="gelu", residual=False),
        # the down projection of a prompt chunk, onto the residual
        dict(name="linear prompt", op="linear", M=4096, N=4096, K=14336, dtype="bf16", bias=False,
             act="none", residual=True),
        # the gated projections of one round
        dict(name="gated round", op="gated", M=5, F=14336, K=4096, dtype="bf16", bias=False,
             act="silu"),
        # the same of a ragged batch of rounds, wide layer
        dict(name="gated batch", op="gated", M=205, F=28672, K=8192, dtype="bf16", bias=False,
             act="silu"),
        # the same of a prompt chunk
        dict(name="gated prompt", op="gated", M=4096, F=14336, K=4096, dtype="bf16", bias=False,
             act="silu"),
        # between two blocks of one round: norm after, residual, norm before
        dict(name="block norm round", op="norm", rows=5, d=4096, dtype="bf16", post=True,
             gate="none", out="same"),
        # the tokens of a prompt batch with a gate a column, feeding the 8-bit product
        dict(name="block norm prompt", op="norm", rows=16384, d=4096, dtype="bf16", post=True,
             gate="column", out="e4m3_block"),
        # the emitted tokens of one round with five alternatives
        dict(name="log probs round", op="logp", R=5, V=128256, n=1, top=5, dtype="fp32",
             temperature=1.0),
        # a batch of 64 rounds with twenty alternatives, sampled at 0.7
        dict(name="log probs batch", op="logp", R=320, V=128256, n=1, top=20, dtype="fp32",
             temperature=0.7),
        # a prompt's tokens scored from 16-bit logits of an odd vocabulary
        dict(name="log probs prompt", op="logp", R=4095, V=128003, n=1, top=5, dtype="bf16",
             temperature=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "gated", "norm", "logp"))
    if op in ("linear", "gated"):
        M = _log(rng, 1, 4096)
        N = _log(rng, 64, 16384)
        K = max(64, _log(rng, 64, 16384) // 8 * 8)
        if rng.random() < 0.7:
            N = max(64, N // 8 * 8)
        most = 4096 * 4096 * 14336 // (2 if op == "gated" else 1)
        if M * N * K > most:
            M = max(1, most // (N * K))
        case = dict(op=op, M=M, K=K, dtype=rng.choice(("bf16", "bf16", "fp16")),
                    bias=rng.random() < 0.4,
                    act=rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu")))
        if op == "gated":
            return dict(case, F=N, act=rng.choice(("silu", "silu", "gelu", "gelu_tanh")))
        return dict(case, N=N, residual=rng.random() < 0.6)
    if op == "norm":
        rows = _log(rng, 1, 16384)
        top = min(16384, 16384 * 4096 // rows)
        d = _log(rng, min(64, top), top)
        if rng.random() < 0.75:
            d = max(8, d // 8 * 8)
        return dict(op=op, rows=rows, d=d, dtype=rng.choice(("bf16", "fp16", "fp32")),
                    post=rng.random() < 0.8, gate=rng.choice(("none", "column", "row", "full")),
                    out=rng.choice(("same", "e4m3_block", "e4m3_row")))
    V = _log(rng, 1000, 131072)
    R = min(_log(rng, 1, 16384), 4095 * 128003 // V)
    dtype = rng.choice(("bf16", "fp16", "fp32"))
    if dtype == "fp32":
        R = max(1, R // 2)
    return dict(op=op, R=R, V=V, n=rng.choice((1, 1, 2, 5)), top=rng.choice((0, 1, 5, 20)),
                dtype=dtype, temperature=rng.choice((1.0, 1.0, 0.7)))


# --------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype=torch.float32, scale=1.0):
    x = torch.empty(shape, dtype=dtype, device=DEV)
    return x.normal_(0.0, scale, generator=g)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    op = case["op"]
    dt = TYPES[case["dtype"]]
    if op in ("linear", "gated"):
        M, K = case["M"], case["K"]
        N = case["N"] if op == "linear" else case["F"]
        s["x"] = _randn(g, (M, K), dt)
        names = [("w", "b")] if op == "linear" else [("wg", "bg"), ("wu", "bu")]
        for w, b in names:
            s[w] = _randn(g, (N, K), dt, K ** -0.5)
            s[b] = _randn(g, (N,), dt, 0.5) if case["bias"] else None
        if op == "linear":
            s["res"] = _randn(g, (M, N), dt, 3.0) if case["residual"] else None
    elif op == "norm":
        rows, d = case["rows"], case["d"]
        s["x"] = _randn(g, (rows, d), dt)
        s["res"] = _randn(g, (rows, d), dt, 3.0)
        s["w"] = (1.0 + 0.1 * _randn(g, (d,))).to(dt)
        s["post"] = (1.0 + 0.1 * _randn(g, (d,))).to(dt) if case["post"] else None
        shape = {"none": None, "column": (d,), "row": (rows, 1), "full": (rows, d)}[case["gate"]]
        s["gate"] = None if shape is None else _randn(g, shape, dt, 0.5)
        s["scale"] = 0.7
    else:
        R, V, n = case["R"], case["V"], case["n"]
        # logits of a peaked distribution: a few tokens stand out in each row
        s["x"] = _randn(g, (R, V), dt, 2.0)
        few = torch.randint(0, V, (R, 1), generator=g, device=DEV)
        few = (few + V // 8 * torch.arange(8, device=DEV)) % V
        lift = (6.0 + 6.0 * torch.rand((R, 8), generator=g, device=DEV)).to(dt)
        s["x"].scatter_(1, few, lift)
        # the given tokens: mostly likely ones; -1 where a round emitted fewer
        t = few[:, :n].clone()
        u = torch.rand((R, n), generator=g, device=DEV)
        any_ = torch.randint(0, V, (R, n), generator=g, device=DEV)
        t = torch.where(u < 0.2, any_, t)
        s["t"] = torch.where(u > 0.95, -1, t).to(torch.int32)
    return s


# --------------------------------------------------------------------------- plain forms

def _act(x, name):
    if name == "relu":
        return x.clamp_min(0.0)
    if name == "gelu":
        return 0.5 * x * (1.0 + torch.erf(x * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))
    if name == "silu":
        return x / (1.0 + torch.exp(-x))
    return x


def _project(x, w, b):
    y = x @ w.float().t()
    return y if b is None else y + b.float()


def _plain_linear(s):
    y = _act(_project(s["x"].float(), s["w"], s["b"]), s["case"]["act"])
    if s["res"] is not None:
        y = y + s["res"].float()
    return y.to(s["x"].dtype)


def _plain_gated(s):
    x = s["x"].float()
    g = _act(_project(x, s["wg"], s["bg"]), s["case"]["act"])
    return (g * _project(x, s["wu"], s["bu"])).to(s["x"].dtype)


def _plain_norm(s):
    c = s["case"]
    dt = s["x"].dtype
    y = s["x"].float()
    if s["post"] is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * s["post"].float()
    y = y * s["scale"]
    if s["gate"] is not None:
        y = y * s["gate"].float()
    h = s["res"].float() + y
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["w"].float()
    if c["out"] == "same":
        return [y.to(dt), h.to(dt)]
    rows, d = y.shape
    group = BLOCK if c["out"] == "e4m3_block" else d
    y = torch.nn.functional.pad(y, (0, -d % group)).view(rows, -1, group)
    scale = y.abs().amax(-1).clamp_min(1e-30) / E4M3_MAX
    q = (y / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).view(rows, -1)[:, :d]
    return [q.to(torch.float8_e4m3fn), scale if c["out"] == "e4m3_block" else scale[:, 0],
            h.to(dt)]


def _plain_logp(s):
    c = s["case"]
    outs = []
    for x, t in zip(s["x"].split(512), s["t"].split(512)):
        x = x.float()
        z = x / c["temperature"]
        z = z - z.amax(-1, keepdim=True)
        e = torch.exp(z)
        total = e.sum(-1, keepdim=True)
        z = z - torch.log(total)
        t = t.long()
        lp = z.gather(1, t.clamp_min(0)).masked_fill(t < 0, 0.0)
        part = [lp, -(e * z).sum(-1) / total[:, 0]]
        if c["top"]:
            ids = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :c["top"]]
            part += [ids.to(torch.int32), z.gather(1, ids)]
        outs.append(part)
    return [torch.cat(p) for p in zip(*outs)]


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        return {"linear": _plain_linear, "gated": _plain_gated, "norm": _plain_norm,
                "logp": _plain_logp}[op](s)
    ops = _ops()
    if op == "linear":
        return ops.linear(s["x"], s["w"], bias=s["b"], activation=c["act"], residual=s["res"])
    if op == "gated":
        return ops.gated_linear(s["x"], s["wg"], s["wu"], bias_gate=s["bg"], bias_up=s["bu"],
                                activation=c["act"])
    if op == "norm":
        if c["out"] == "same":
            return ops.block_norm(s["x"], s["res"], s["w"], post_weight=s["post"], gate=s["gate"],
                                  branch_scale=s["scale"], eps=EPS)
        return ops.block_norm_fp8(s["x"], s["res"], s["w"], post_weight=s["post"],
                                  gate=s["gate"], branch_scale=s["scale"], eps=EPS,
                                  group=BLOCK if c["out"] == "e4m3_block" else 0)
    return ops.log_probs(s["x"], s["t"], top=c["top"], temperature=c["temperature"])


# --------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    e = 4 if case["dtype"] == "fp32" else 2
    if op in ("linear", "gated"):
        M, K = case["M"], case["K"]
        N, w = (case["N"], 1) if op == "linear" else (case["F"], 2)
        b = e * (M * K + w * N * K + M * N)
        if case["bias"]:
            b += e * w * N
        if op == "linear" and case["residual"]:
            b += e * M * N
        return {"bytes": b, "flops": 2 * w * M * N * K}
    if op == "norm":
        rows, d = case["rows"], case["d"]
        b = 3 * rows * d * e + d * e * (2 if case["post"] else 1)
        b += {"none": 0, "column": d * e, "row": rows * e, "full": rows * d * e}[case["gate"]]
        if case["out"] == "same":
            b += rows * d * e
        else:
            b += rows * d + 4 * rows * (-(-d // BLOCK) if case["out"] == "e4m3_block" else 1)
        return {"bytes": b, "flops": 10 * rows * d}
    R, V = case["R"], case["V"]
    return {"bytes": R * V * e + R * (8 * case["n"] + 4 + 8 * case["top"]), "flops": 6 * R * V}


# --------------------------------------------------------------------------- 64 bits

def _act64(x, name):
    if name == "none":
        return x
    if name == "relu":
        return torch.where(x > 0, x, torch.zeros_like(x))
    if name == "gelu":
        return x * torch.special.ndtr(x)
    if name == "gelu_tanh":
        # (1 + tanh u) / 2 = sigmoid(2 u)
        return x * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3))
    return x * torch.sigmoid(x)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("linear", "gated"):
        x = s["x"].double()

        def affine(w, b):
            parts = [torch.mm(x, p.double().t()) for p in w.split(8192)]
            y = torch.cat(parts, 1)
            return y if b is None else y.add_(b.double())
        if op == "gated":
            return _act64(affine(s["wg"], s["bg"]), case["act"]) * affine(s["wu"], s["bu"])
        y = _act64(affine(s["w"], s["b"]), case["act"])
        return y if s["res"] is None else y + s["res"].double()
    if op == "norm":
        def unit(v):
            return v / torch.sqrt(torch.linalg.vecdot(v, v)[:, None] / v.shape[1] + EPS)
        y = s["x"].double()
        if s["post"] is not None:
            y = unit(y) * s["post"].double()
        g = 1.0 if s["gate"] is None else s["gate"].double()
        h = torch.addcmul(s["res"].double(), y, torch.as_tensor(g * s["scale"], device=DEV,
                                                                dtype=torch.float64))
        y = unit(h) * s["w"].double()
        if case["out"] == "same":
            return [y, h]
        parts = y.split(BLOCK, 1) if case["out"] == "e4m3_block" else [y]
        scales = [p.abs().max(1).values.clamp(min=1e-30) / 448.0 for p in parts]
        q = torch.cat([p / sc[:, None] for p, sc in zip(parts, scales)], 1)
        return [q, torch.stack(scales, 1) if case["out"] == "e4m3_block" else scales[0], h]
    lps, ents, ids, tops = [], [], [], []
    for r in range(0, case["R"], 256):
        x = s["x"][r:r + 256].double()
        lse = torch.logsumexp(x / case["temperature"], 1)
        logp = x / case["temperature"] - lse[:, None]
        t = s["t"][r:r + 256].long()
        at = torch.arange(t.shape[0], device=DEV)[:, None].expand_as(t)
        lps.append(torch.where(t < 0, 0.0, logp[at, t.clamp(min=0)]))
        ents.append(-torch.linalg.vecdot(torch.exp(logp), logp))
        if case["top"]:
            # one after another: the largest, of equal ones the first
            left, col = x.clone(), torch.arange(x.shape[1], device=DEV)
            got = []
            for _ in range(case["top"]):
                best = left.max(1, keepdim=True).values
                i = torch.where(left == best, col, x.shape[1]).min(1, keepdim=True).values
                got.append(i)
                left.scatter_(1, i, -math.inf)
            got = torch.cat(got, 1)
            ids.append(got.to(torch.int32))
            tops.append(logp.gather(1, got))
    out = [torch.cat(lps), torch.cat(ents)]
    return out + [torch.cat(ids), torch.cat(tops)] if case["top"] else out
