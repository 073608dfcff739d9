"""Plain 64-bit implementations of the operators of a layer's second half and
of the log probabilities, with the bounds of their tests.

Half a step of a type t is eps(t) / 2 of the value (bf16 2^-8, fp16 2^-11,
fp32 2^-24, E4M3 2^-4); the bounds below count such roundings.
"""
import math

import torch

from target_common import HALF_STEP, TINY

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def act_ref(v, name):
    """The activation in 64 bits and the relative error of its fp32 form."""
    if name == "relu":
        return v.clamp_min(0), torch.zeros_like(v)
    if name == "gelu":
        # erfc is good to a few units, and its argument's rounding (2^-23 with the
        # product's) grows by d ln erfc / d ln z, which is at most 2 z^2 + 2 = v^2 + 2
        return v * 0.5 * torch.special.erfc(-v * math.sqrt(0.5)), (v * v + 16) * 2.0 ** -23
    if name == "gelu_tanh":
        u = 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
        return v * torch.sigmoid(u), (6 * u.abs() + 16) * 2.0 ** -23
    if name == "silu":
        return v * torch.sigmoid(v), torch.full_like(v, 16 * 2.0 ** -23)
    return v, torch.zeros_like(v)


def project(x, w, b):
    """x w^T + b and the bound of its fp32 form: K products summed with errors of at
    most 2^-23 of the magnitudes each (the tensor cores' additions may cut), the
    bias one more rounding."""
    y = x.double() @ w.double().t()
    err = (x.double().abs() @ w.double().abs().t()) * (x.shape[1] + 8) * 2.0 ** -23
    if b is not None:
        y = y + b.double()
    return y, err + y.abs() * 2.0 ** -23


def rounded(ref, err, dtype):
    """The bound after one rounding to dtype (exponentials below 2^-126 may be
    zero: 2^-110 covers what they multiply)."""
    return err + (ref.abs() + err) * HALF_STEP[dtype] * 1.01 + TINY[dtype] + 2.0 ** -110


def linear_ref(x, w, bias=None, act="none", residual=None, out_dtype=None):
    y, err = project(x, w, bias)
    a, rel = act_ref(y, act)
    err = 1.13 * err + a.abs() * rel  # no activation is steeper than 1.13
    if residual is not None:
        a = a + residual.double()
    return a, rounded(a, err + a.abs() * 2.0 ** -24, out_dtype or x.dtype)


def gated_ref(x, wg, wu, bg=None, bu=None, act="silu", out_dtype=None):
    g, eg = project(x, wg, bg)
    u, eu = project(x, wu, bu)
    a, rel = act_ref(g, act)
    eg = 1.13 * eg + a.abs() * rel
    y = a * u
    err = eg * u.abs() + a.abs() * eu + eg * eu
    return y, rounded(y, err + y.abs() * 2.0 ** -23, out_dtype or x.dtype)


# A sum of d <= 2^16 squares: a thread adds up to 128 one after another, five
# shuffles and up to 32 warps follow; halved by the root, and a few other steps.
SUM_REL = 130 * 2.0 ** -24


def block_norm_ref(x, residual, weight, post=None, gate=None, scale=1.0, eps=1e-6):
    """out, h and the bounds of both before they are rounded."""
    scale = torch.tensor(scale, dtype=torch.float32).double().item()  # as it is passed
    eps = torch.tensor(eps, dtype=torch.float32).double().item()
    y = x.double()
    if post is not None:
        y = y * torch.rsqrt((y * y).mean(1, keepdim=True) + eps) * post.double()
    y = y * scale
    if gate is not None:
        y = y * gate.double()
    h = residual.double() + y
    dh = y.abs() * (SUM_REL + 8 * 2.0 ** -24) + h.abs() * 2.0 ** -24
    inv = torch.rsqrt((h * h).mean(1, keepdim=True) + eps)
    out = h * inv * weight.double()
    # the root moves by at most |dh| / |h| of the whole row
    move = dh.norm(dim=1, keepdim=True) / h.norm(dim=1, keepdim=True).clamp_min(1e-300)
    dout = inv * weight.double().abs() * (dh + h.abs() * (move.clamp_max(1.0) + SUM_REL
                                                          + 8 * 2.0 ** -24))
    return out, h, dout, dh


def log_probs_ref(logits, tokens, top, temperature):
    """log probabilities of the tokens, entropy, top ids and their log
    probabilities; rows without a finite maximum are NaN and -1."""
    T = torch.tensor(temperature, dtype=torch.float32).double().item()
    x = logits.double()
    m = x.amax(1, keepdim=True)  # a NaN stays
    fine = torch.isfinite(m)[:, 0]
    z = (x - torch.where(fine[:, None], m, 0.0)) / T
    z[~fine] = math.nan
    s = z.exp().sum(1, keepdim=True)
    lp = z - s.log()
    p = lp.exp()
    ent = -torch.where(p == 0, 0.0, p * lp).sum(1)
    out = [torch.zeros(tokens.shape, dtype=torch.float64, device=x.device), ent]
    t = tokens.long()
    V = x.shape[1]
    got = lp.gather(1, t.clamp(0, V - 1))
    out[0] = torch.where(t == -1, 0.0, torch.where((t < 0) | (t >= V), math.nan, got))
    if top:
        ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :top]
        out += [torch.where(fine[:, None], ids, -1).int(), lp.gather(1, ids)]
    return out


def log_probs_error(ref, V):
    """A logit's distance d from the maximum is rounded three times (2^-24 of d, at
    most |ref| + log V, each); a thread adds at most V / 256 exponentials one after
    another, and 64 roundings cover joins, the exponential and the logarithm."""
    return (ref.abs() + math.log(V)) * 2.0 ** -22 + (V / 256 + 64) * 2.0 ** -24
