"""The target-layer operators on the GPU where roles, masks, types and streams
meet: cases beside those of test_gpu_target_ops.py."""
import math
from fractions import Fraction

import pytest
import torch

import speculative_decoding_verification_22_gb300 as sv
from target_common import (DTYPES, attention_bound, attention_ref, build_cache, gen, randn,
                           score_error, within)

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


# ---- attention: pages that are not there ----------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("page", [8, 16, 32])
@pytest.mark.parametrize("news,lens,window", [
    ([1], [1000], 37), ([3, 300], [700, 2000], 100),  # few rows; blocks of many
    ([5], [30000], 20001), ([90], [4000], 130)])      # a cut item; one wide item
def test_attention_window_over_freed_pages(ops, dtype, page, news, lens, window):
    """Pages that lie wholly below the window may be gone from the table; the
    last one that is seen may not."""
    g = gen(page + window)
    dt = DTYPES[dtype]
    kc, vc, table, ks, vs = build_cache(g, lens, page, 2, 128, dt)
    q = randn(g, (sum(news), 8, 128), dt)
    seen = [max(0, kv - n + 1 - window) // page for n, kv in zip(news, lens)]
    for b, first in enumerate(seen):
        table[b, :first] = -1
    out = ops.attention(q, kc, vc, table, starts(news), int32(lens), window=window)
    assert ops.status() == sv.SV_OK
    o, mag, _, big = attention_ref(q, ks, vs, news, 128 ** -0.5, window)
    within(out, o, attention_bound(o, mag, big, 128, dt))
    table[-1, seen[-1]] = -1
    ops.attention(q, kc, vc, table, starts(news), int32(lens), window=window)
    assert ops.status() == sv.SV_ERR_CACHE


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_tree_over_pages_that_no_node_sees(ops, dtype):
    """A tree padded to 40 nodes of which 17 are live: the others' pages may be
    missing, those of live nodes may not."""
    dt = DTYPES[dtype]
    g = gen(3)
    n, live, kv, page = 40, 17, 140, 8
    see = torch.zeros(n, n, dtype=torch.bool, device="cuda")
    see[:live, :live] = torch.ones(live, live, device="cuda").tril().bool()
    bits = torch.nn.functional.pad(see, (0, 24)).view(n, 2, 32).long()
    bits = (bits << torch.arange(32, device="cuda")).sum(-1)
    mask = torch.where(bits >= 2 ** 31, bits - 2 ** 32, bits).int().contiguous()
    kc, vc, table, ks, vs = build_cache(g, [kv], page, 2, 64, dt)
    q = randn(g, (n, 4, 64), dt)
    end = kv - n + live
    table[0, -(-end // page):] = -1
    out = ops.attention(q, kc, vc, table, starts([n]), int32([kv]), tree_mask=mask)
    assert ops.status() == sv.SV_OK
    o, mag, _, big = attention_ref(q, ks, vs, [n], 0.125, see=[see])
    within(out, o, attention_bound(o, mag, big, 64, dt))
    table[0, (end - 1) // page] = -1
    ops.attention(q, kc, vc, table, starts([n]), int32([kv]), tree_mask=mask)
    assert ops.status() == sv.SV_ERR_CACHE


def test_attention_windows_of_any_size(ops):
    """A window beyond 32 bits is one of all keys, and a negative one is refused."""
    g = gen(4)
    kc, vc, table, _, _ = build_cache(g, [400], 16, 2, 64, torch.bfloat16)
    q = randn(g, (9, 4, 64), torch.bfloat16)
    args = q, kc, vc, table, starts([9]), int32([400])
    want = ops.attention(*args)
    for window in (2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 62 + 7):
        assert torch.equal(ops.attention(*args, window=window), want)
    for window in (-1, -2 ** 32, 5 - 2 ** 32, -2 ** 62):
        with pytest.raises(sv.SpecVerifyError):
            ops.attention(*args, window=window)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_largest_window_with_more_tokens_than_keys(ops, dtype):
    g = gen(5)
    dt = DTYPES[dtype]
    news, lens, window = [40, 300], [7, 200], 2 ** 31 - 1
    kc, vc, table, ks, vs = build_cache(g, lens, 16, 2, 64, dt)
    q = randn(g, (340, 4, 64), dt)
    out = ops.attention(q, kc, vc, table, starts(news), int32(lens), window=window)
    o, mag, _, big = attention_ref(q, ks, vs, news, 0.125, window)
    within(out, o, attention_bound(o, mag, big, 64, dt))
    assert ops.status() == sv.SV_OK


# ---- attention: many small weights under a large one ---------------------------------

@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("n", [1, 40])  # few rows, a block of many
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_attention_small_weights_of_a_long_cache_count(ops, dtype, n, first):
    """One key 17 nats above 131072 equal ones, whose weights of e^-17 make half a
    percent of the sum. As many sequences as keep each on one SM, over the same
    pages. In fp16 a weight is rounded to half a step or, below the normal range,
    by 2^-25 at most, which stands for 2^-32 of the largest."""
    g = gen(6)
    dt = DTYPES[dtype]
    B, D, page, kv = 160, 64, 64, 131073
    kc, vc, table, ks, vs = build_cache(g, [kv], page, 1, D, dt, fill=0.0)
    top = 0 if first else kv - n - 1  # before the new tokens: every row sees it
    at = int(table[0, top // page]), top % page
    for t in (kc, ks[0]):
        t.zero_()
    for t in (vc, vs[0]):
        t.fill_(1.0)
    kc[at] = ks[0][top] = 2.125  # 64 * 2.125 / 8 = 17
    vc[at] = vs[0][top] = 0.0
    q = torch.ones(B * n, 4, D, dtype=dt, device="cuda")
    lse = torch.empty(B * n, 4, device="cuda")
    out = ops.attention(q, kc, vc, table.expand(B, -1).contiguous(), starts([n] * B),
                        int32([kv] * B), lse=lse)
    o, mag, l, big = attention_ref(q[:n], ks, vs, [n], 0.125)
    bound = attention_bound(o, mag, big, D, dt) + (kv * 2.0 ** -32 if dtype == "fp16" else 0.0)
    within(out, o.repeat(B, 1, 1), bound.repeat(B, 1, 1))
    l = l.repeat(B, 1)
    within(lse, l, score_error(big, D) + 2.0 ** -20 * l.abs())
    assert ops.status() == sv.SV_OK


# ---- rotary: far positions ------------------------------------------------------------

@pytest.mark.parametrize("far", [2 ** 21, 2 ** 28, 2 ** 34, 2 ** 40, 2 ** 46, 2 ** 52])
def test_rope_far_positions(ops, far):
    """Fractions of a turn against exact products. They are rounded to fp32 (2^-25
    of a turn, 2 pi times that in radians, below 2^-22), then cos and sin have two
    units of half a step each and the products one: together below 2^-20."""
    T, D = 64, 64
    freqs, _ = sv.spec_target_rope_freqs(D, 10000.0)
    pos = far + torch.randint(0, far, (T,), generator=gen(7), device="cuda")
    pos[::2] *= -1
    x = torch.zeros(T, 1, D, device="cuda")
    x[..., :D // 2] = 1.0
    c = torch.zeros(1, 1, 1, D, device="cuda")
    none = torch.full((T,), -1, device="cuda")
    y = ops.rope_append(x, x, x, pos, none, freqs.cuda(), c, c.clone())
    turns = [[float(p * Fraction(f) % 1) for f in freqs.tolist()] for p in pos.tolist()]
    angle = torch.tensor(turns, dtype=torch.float64, device="cuda")[:, None] * (2 * math.pi)
    want = torch.cat((angle.cos(), angle.sin()), -1)
    within(y, want, torch.full_like(want, 2.0 ** -20))
    assert ops.status() == sv.SV_OK


# ---- refusals -------------------------------------------------------------------------

def test_norm_into_eight_bits_that_are_not_e4m3_is_refused(ops):
    x, w = torch.ones(4, 128, device="cuda"), torch.ones(128, device="cuda")
    for dtype in (torch.float8_e5m2, torch.int8, torch.bool):
        with pytest.raises(ValueError, match="e4m3"):
            ops.rms_norm_fp8(x, w, out=torch.zeros(4, 128, device="cuda").to(dtype))
    want = ops.rms_norm_fp8(x, w)[0]
    out = torch.empty(4, 128, dtype=torch.uint8, device="cuda")
    assert torch.equal(ops.rms_norm_fp8(x, w, out=out)[0], want.view(torch.uint8))


def test_norm_groups_beyond_32_bits_are_refused(ops):
    x, w = torch.ones(4, 256, device="cuda"), torch.ones(256, device="cuda")
    for group in (2 ** 32, 2 ** 32 + 128, 128 - 2 ** 32):
        with pytest.raises(sv.SpecVerifyError):
            ops.rms_norm_fp8(x, w, group=group)


def test_tree_masks_without_words_are_refused(ops):
    """As the C entry point does; it is not a call without a mask."""
    g = gen(8)
    kc, vc, table, _, _ = build_cache(g, [40], 16, 1, 64, torch.bfloat16)
    q = randn(g, (4, 2, 64), torch.bfloat16)
    none = torch.empty(4, 0, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="word"):
        ops.attention(q, kc, vc, table, starts([4]), int32([40]), tree_mask=none)


def test_tensors_of_another_device_are_refused(ops):
    """A handle that says it belongs to the next device refuses this one's tensors
    before anything is launched, whichever argument they are."""
    other = sv.TargetOps.__new__(sv.TargetOps)
    other.__dict__.update(ops.__dict__)
    other._index = ops._index + 1
    x, w = torch.ones(4, 128, device="cuda"), torch.ones(128, device="cuda")
    q, c = x.view(4, 1, 128), x.view(1, 4, 1, 128)
    e, s = x.to(torch.float8_e4m3fn), torch.ones(4, 1, device="cuda")
    pos, f = torch.arange(4, device="cuda"), torch.zeros(64, dtype=torch.float64, device="cuda")
    try:
        for call in (lambda: other.rms_norm(x, w), lambda: other.rms_norm_fp8(x, w),
                     lambda: other.matmul_fp8(e, s, e, s[:1]),
                     lambda: other.rope_append(q, q, q, pos, pos, f, c, c.clone()),
                     lambda: other.attention(q, c, c, int32([[0]]), int32([0, 4]), int32([4])),
                     lambda: other.tree_mask(int32([[-1, 0]]))):
            with pytest.raises(ValueError, match="GPU of the handle"):
                call()
    finally:
        other.h = other._raw = None  # the handle is the fixture's
    assert ops.status() == sv.SV_OK


# ---- streams --------------------------------------------------------------------------

def stream_of(t):
    """The stream whose pool a tensor's memory belongs to."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's memory")


def test_outputs_come_from_the_given_stream(ops):
    """New outputs are of the memory of the stream that the call goes to, so that
    nothing enqueued elsewhere may still use it."""
    x, w = torch.ones(4, 128, device="cuda"), torch.ones(128, device="cuda")
    parents = int32([[-1, 0, 0, 2]])
    want = ops.tree_mask(parents)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        for call in (lambda s: ops.rms_norm(x, w, stream=s)[0],
                     lambda s: ops.tree_mask(parents, stream=s)):
            assert stream_of(call(stream)) == side.cuda_stream
            assert stream_of(call(None)) == torch.cuda.current_stream().cuda_stream
        got = ops.tree_mask(parents, stream=stream)
        side.synchronize()
        assert torch.equal(got, want)
    assert torch.equal(ops.tree_mask(parents, stream=0), want)
    assert ops.status() == sv.SV_OK
