"""The target-layer operators on the GPU where roles, masks, types and streams
meet: cases beside those of test_gpu_target_ops.py."""
import math

import pytest
import torch

import speculative_decoding_verification_22_gb300 as sv
from target_common import (attention_bound, attention_ref, build_cache, gen, randn, score_error,
                           within)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    o = sv.TargetOps()
    yield o
    torch.cuda.synchronize()
    o.close()


def int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def starts(news):
    return int32([sum(news[:i]) for i in range(len(news) + 1)])


# ---- attention: blocks of many rows and of few in turn on one SM -------------------

@pytest.mark.parametrize("D,page", [(128, 16), (128, 64), (64, 8)])
def test_attention_wide_and_narrow_items_in_turn(ops, D, page):
    """Long runs of items of 256 rows, whose V one warp brings, between items of
    few rows, whose V another brings: the two stay within one round of the ring."""
    g = gen(D + page)
    news, lens, hq, hkv = [], [], 8, 2
    for i in range(24):
        news += [300, 3, 1]
        lens += [1500 + 64 * i, 700 + i, 90 + i]
    kc, vc, table, ks, vs = build_cache(g, lens, page, hkv, D, torch.bfloat16, fill=0.0)
    q = randn(g, (sum(news), hq, D), torch.bfloat16)
    qs, kl = starts(news), int32(lens)
    want = ops.attention(q, kc, vc, table, qs, kl)
    o, mag, _, big = attention_ref(q, ks, vs, news, 1 / math.sqrt(D))
    within(want, o, attention_bound(o, mag, big, D, torch.bfloat16))
    outs = [ops.attention(q, kc, vc, table, qs, kl) for _ in range(40)]
    assert ops.status() == sv.SV_OK
    for out in outs:
        assert torch.equal(out, want)


# ---- attention: parts of a row that are not finite ----------------------------------

@pytest.mark.parametrize("n,kv", [(64, 20000), (5, 6000), (150, 3000)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_attention_cut_rows_with_some_columns_not_finite(ops, dtype, n, kv):
    """NaN and infinities behind the mask in single columns of V, in items that are
    cut over many SMs: a row's other columns and its lse come out the same bit for
    bit however the warps that join the parts are timed."""
    g = gen(n)
    kc, vc, table, ks, vs = build_cache(g, [kv], 16, 1, 128, dtype)
    for back, col, bad in ((1, 3, math.nan), (2, 77, math.inf), (3, 126, -math.inf)):
        at = kv - back
        vs[0][at, 0, col] = bad
        vc[int(table[0, at // 16]), at % 16, 0, col] = bad
    q = randn(g, (n, 4, 128), dtype)
    qs, kl = starts([n]), int32([kv])

    def call():
        lse = torch.empty(n, 4, device="cuda")
        return ops.attention(q, kc, vc, table, qs, kl, lse=lse), lse
    out, lse = call()
    o, mag, l, big = attention_ref(q, ks, vs, [n], 128 ** -0.5)
    within(out, o, attention_bound(o, torch.nan_to_num(mag, posinf=0.0), big, 128, dtype))
    within(lse, l, score_error(big, 128) + 2.0 ** -20 * l.abs())
    for _ in range(50):
        again = call()
        assert torch.equal(out.view(torch.int16), again[0].view(torch.int16))
        assert torch.equal(lse.view(torch.int32), again[1].view(torch.int32))
    assert ops.status() == sv.SV_OK
