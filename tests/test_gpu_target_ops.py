"""The target-layer operators on the GPU against plain 64-bit implementations."""
import math

import pytest
import torch

import speculative_decoding_verification_22_gb300 as sv
from target_common import (DTYPES, HALF_STEP, NORM_REL, TINY, attention_bound, attention_ref,
                           build_cache, gen, matmul_bound, matmul_ref, norm_ref, quant_blocks,
                           randn, rope_bound, rope_ref, score_error, within)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    o = sv.TargetOps()
    yield o
    torch.cuda.synchronize()
    o.close()


# ---- norm ---------------------------------------------------------------------

@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,d", [(1, 1), (1, 8), (3, 7), (5, 4096), (2, 128), (130, 136),
                                    (7, 1000), (4, 8200), (3, 16384), (2, 20000), (1, 40000),
                                    (2, 4095), (300, 256)])
def test_norm(ops, dtype, rows, d):
    dt = DTYPES[dtype]
    g = gen(rows * 1000 + d)
    x, r = randn(g, (rows, d), dt), randn(g, (rows, d), dt, 3.0)
    w = randn(g, (d,), dt, 0.3) + 1
    for res in (None, r):
        ref, h = norm_ref(x, w, 1e-6, res)
        out = ops.rms_norm(x, w, 1e-6, residual=res)
        within(out[0], ref, ref.abs() * (HALF_STEP[dt] * 1.01 + NORM_REL) + TINY[dt])
        assert len(out) == (1 if res is None else 2)
        if res is not None:
            within(out[1], h, h.abs() * HALF_STEP[dt] * 1.01 + TINY[dt])
    assert ops.status() == sv.SV_OK


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("group", [128, 0])
@pytest.mark.parametrize("rows,d", [(1, 1), (3, 7), (5, 4096), (130, 136), (4, 8200), (2, 20000),
                                    (6, 129), (3, 1001), (1, 40000), (33, 128)])
def test_norm_e4m3(ops, dtype, group, rows, d):
    dt = DTYPES[dtype]
    g = gen(rows * 77 + d)
    x, r = randn(g, (rows, d), dt), randn(g, (rows, d), dt, 3.0)
    x[0] = 0
    r[0] = 0  # a row of zeros
    w = randn(g, (d,), dt, 0.3) + 1
    q, s, ro = ops.rms_norm_fp8(x, w, 1e-6, residual=r, group=group)
    y, h = norm_ref(x, w, 1e-6, r)
    within(ro, h, h.abs() * HALF_STEP[dt] * 1.01 + TINY[dt])
    width = group or d
    yp = torch.nn.functional.pad(y, (0, -d % width)).view(rows, -1, width)
    want = yp.abs().amax(-1).clamp_min(1e-30) / 448.0
    got = s.view(rows, -1)
    within(got, want, want * (NORM_REL + 2.0 ** -22))
    step = y / got.double().repeat_interleave(width, 1)[:, :d]
    # half a step of E4M3: 2^-4 of the value, 2^-10 below the normal range
    within(q, step, torch.maximum(step.abs() * 2.0 ** -4, torch.full_like(step, 2.0 ** -10))
           + step.abs() * (NORM_REL + 2.0 ** -22))
    assert not q[0].float().any()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,d", [(3, 127), (4, 129), (200, 2047), (2, 4097), (3, 8191),
                                    (2, 8193), (2, 16383), (2, 16385)])
def test_norm_odd_widths(ops, dtype, rows, d):
    test_norm(ops, dtype, rows, d)
    for group in (128, 0):
        test_norm_e4m3(ops, dtype, group, rows, d)


def test_norm_strides_in_place_and_unaligned(ops):
    g = gen(5)
    big = randn(g, (9, 3 * 512 + 8), torch.bfloat16)
    w = randn(g, (512,), torch.bfloat16)
    for off in (0, 8, 3):  # 3: rows not on 16 bytes
        x, r = big[:, off:off + 512], big[:, 520 + off:520 + off + 512]
        ref, h = norm_ref(x, w, 1e-5, r)
        bound = ref.abs() * (2.0 ** -8 * 1.01 + NORM_REL) + TINY[torch.bfloat16]
        keep = big.clone()
        out, ro = ops.rms_norm(x, w, 1e-5, residual=r)
        within(out, ref, bound)
        assert torch.equal(big, keep)
        out, ro = ops.rms_norm(x, w, 1e-5, residual=r, out=x, residual_out=r)
        assert out.data_ptr() == x.data_ptr()
        within(x, ref, bound)
        within(r, h, h.abs() * 2.0 ** -8 * 1.01)
        big.copy_(keep)


def test_norm_not_finite_and_extremes(ops):
    x = torch.ones(4, 256, device="cuda")
    x[0, 3] = float("nan")
    x[1, 200] = float("inf")
    x[2] = 1e18   # the sum of squares stays in fp32
    x[3] = 1e-30  # squares below fp32: eps decides
    w = torch.ones(256, device="cuda")
    y = ops.rms_norm(x, w, 1e-6)[0]
    assert torch.isnan(y[0]).all() and torch.isnan(y[1, 200]) and (y[1, :200] == 0).all()
    assert torch.allclose(y[2], torch.ones_like(y[2]), rtol=1e-5)
    assert torch.allclose(y[3], x[3] * 1e3, rtol=1e-5, atol=0)
    for group in (128, 0):
        q, s = ops.rms_norm_fp8(x, w, 1e-6, group=group)
        deq = q.float() * s.view(4, -1).repeat_interleave(group or 256, 1)
        assert torch.isnan(deq[0]).all() and not torch.isfinite(deq[1]).all()
        assert torch.allclose(deq[2], torch.ones_like(deq[2]), rtol=2 ** -4)


def test_norm_of_no_rows(ops):
    x = torch.empty(0, 64, device="cuda")
    assert ops.rms_norm(x, torch.ones(64, device="cuda"))[0].shape == (0, 64)


# ---- 8-bit product --------------------------------------------------------------

SHAPES = [(1, 1, 16), (1, 128, 128), (5, 130, 144), (5, 6144, 4096), (16, 257, 128),
          (17, 1000, 1040), (33, 384, 512), (64, 512, 8192), (65, 200, 272), (100, 96, 4096),
          (128, 128, 128), (129, 640, 400), (205, 1024, 2048), (256, 257, 1024),
          (300, 2049, 528), (512, 2048, 4096), (1000, 700, 1200), (2048, 1536, 640)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_matmul_fp8(ops, M, N, K):
    g = gen(M + N + K)
    a, sa = quant_blocks(randn(g, (M, K)) * torch.logspace(-2, 2, M, device="cuda")[:, None], 1)
    w, sw = quant_blocks(randn(g, (N, K), scale=0.02), 128)
    ref, mags = matmul_ref(a, sa, w, sw)
    for dt in DTYPES.values():
        out = ops.matmul_fp8(a, sa, w, sw, out_dtype=dt)
        within(out, ref, matmul_bound(ref, mags, K, dt))
    again = ops.matmul_fp8(a, sa, w, sw, out_dtype=dt)
    assert torch.equal(out, again)
    assert ops.status() == sv.SV_OK


def test_matmul_fp8_scales_differ_by_block(ops):
    """Every scale counts once, at its own place: powers of two as scales and
    small whole numbers as values give exact sums."""
    M, N, K = 70, 390, 656
    g = gen(3)
    a = torch.randint(-4, 5, (M, K), generator=g, device="cuda").float()
    w = torch.randint(-4, 5, (N, K), generator=g, device="cuda").float()
    sa = 2.0 ** torch.randint(-2, 3, (M, 6), generator=g, device="cuda").float()
    sw = 2.0 ** torch.randint(-2, 3, (4, 6), generator=g, device="cuda").float()
    ref, _ = matmul_ref(a, sa, w, sw)
    out = ops.matmul_fp8(a.to(torch.float8_e4m3fn), sa, w.to(torch.float8_e4m3fn), sw,
                         out_dtype=torch.float32)
    assert torch.equal(out.double(), ref)


def test_matmul_fp8_strided_output_and_what_lies_beside_it(ops):
    g = gen(4)
    a, sa = quant_blocks(randn(g, (130, 256)), 1)
    w, sw = quant_blocks(randn(g, (200, 256)), 128)
    ref, mags = matmul_ref(a, sa, w, sw)
    for dt, off in ((torch.bfloat16, 0), (torch.bfloat16, 3), (torch.float32, 5),
                    (torch.float16, 8)):
        big = torch.full((130, 240), 7.0, dtype=dt, device="cuda")
        out = big[:, off:off + 200]
        ops.matmul_fp8(a, sa, w, sw, out=out)
        within(out, ref, matmul_bound(ref, mags, 256, dt))
        assert (big[:, :off] == 7).all() and (big[:, off + 200:] == 7).all()


def test_matmul_fp8_not_finite(ops):
    """A NaN or infinite scale reaches its own row or columns only."""
    g = gen(6)
    for M in (6, 200):
        a, sa = quant_blocks(randn(g, (M, 512)), 1)
        w, sw = quant_blocks(randn(g, (300, 512)), 128)
        sa[2, 1] = float("nan")
        sw[1, 3] = float("inf")
        out = ops.matmul_fp8(a, sa, w, sw, out_dtype=torch.float32)
        assert torch.isnan(out[2]).all()
        keep = torch.ones(M, dtype=torch.bool, device="cuda")
        keep[2] = False
        assert not torch.isfinite(out[keep][:, 128:256]).any()
        assert torch.isfinite(out[keep][:, :128]).all()
        assert torch.isfinite(out[keep][:, 256:]).all()


# ---- rotary ---------------------------------------------------------------------

@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot,hq,hkv,page,T", [
    (128, 128, 32, 8, 16, 5), (128, 64, 4, 4, 64, 37), (64, 64, 7, 1, 8, 130), (96, 48, 6, 2, 1, 9),
    (80, 80, 3, 3, 5, 11), (17, 10, 2, 1, 3, 4), (256, 256, 2, 2, 16, 3), (64, 2, 2, 1, 16, 1),
    (128, 0, 2, 2, 16, 3)])
def test_rope_append(ops, dtype, interleaved, D, rot, hq, hkv, page, T):
    dt = DTYPES[dtype]
    g = gen(D + rot + T)
    qkv = randn(g, (T, (hq + 2 * hkv) * D), dt)
    q = qkv[:, :hq * D].view(T, hq, D)
    k = qkv[:, hq * D:(hq + hkv) * D].view(T, hkv, D)
    v = qkv[:, (hq + hkv) * D:].view(T, hkv, D)
    freqs, m = (sv.spec_target_rope_freqs(rot, 500000.0, "yarn", 8.0, 8192) if rot
                else (torch.empty(0, dtype=torch.float64), 1.0))
    freqs = freqs.cuda()
    pos = torch.randint(0, 1 << 21, (T,), generator=g, device="cuda")
    pos[0] = 0
    pages = T // page + 2
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T].contiguous()
    if T > 3:
        slots[2] = -1
    kc = randn(g, (pages, page, hkv, D), dt)
    vc = randn(g, (pages, page, hkv, D), dt)
    kw, vw = kc.double().view(-1, hkv, D), vc.double().view(-1, hkv, D)
    km = torch.zeros_like(kw)
    qr, qm = rope_ref(q, pos, freqs, interleaved, m)
    kr, kmag = rope_ref(k, pos, freqs, interleaved, m)
    live = slots >= 0
    kw[slots[live]], vw[slots[live]], km[slots[live]] = kr[live], v.double()[live], kmag[live]
    qo = ops.rope_append(q, k, v, pos, slots, freqs, kc, vc, interleaved, m)
    within(qo, qr, rope_bound(qr, qm, dt))
    within(kc.view(-1, hkv, D), kw, rope_bound(kw, km, dt))
    assert torch.equal(vc.double().view(-1, hkv, D), vw)
    assert torch.equal(qo[..., rot:], q[..., rot:])
    # in place
    ops.rope_append(q, k, v, pos, slots, freqs, kc, vc, interleaved, m, q_out=q)
    assert torch.equal(q, qo)
    assert ops.status() == sv.SV_OK


def test_rope_append_heads_first_cache_and_bad_slots(ops):
    g = gen(8)
    T, hkv, D = 6, 2, 64
    q, k, v = (randn(g, (T, hkv, D), torch.bfloat16) for _ in range(3))
    kc = torch.zeros(4, hkv, 16, D, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    vc = torch.zeros_like(kc)
    freqs = sv.spec_target_rope_freqs(64)[0].cuda()
    pos = torch.arange(T, device="cuda")
    slots = torch.tensor([0, 17, 63, 64, -2, 1 << 40], device="cuda")
    ops.rope_append(q, k, v, pos, slots, freqs, kc, vc)
    assert ops.status() == sv.SV_ERR_CACHE
    assert ops.status() == sv.SV_OK
    assert torch.equal(vc[0, 0], v[0]) and torch.equal(vc[1, 1], v[1])
    assert torch.equal(vc[3, 15], v[2])
    assert int((vc != 0).any(-1).any(-1).sum()) == 3


def test_rope_turns_back(ops):
    """Rotating by p and then by -p gives the input; angles of p and p + a whole
    period of a pair agree."""
    g = gen(9)
    T, D = 50, 64
    x = randn(g, (T, 1, D))
    c = torch.zeros(1, 1, 1, D, device="cuda")
    none = torch.full((T,), -1, device="cuda")
    freqs = sv.spec_target_rope_freqs(D, 10000.0)[0].cuda()
    pos = torch.randint(0, 1 << 30, (T,), generator=g, device="cuda")
    y = ops.rope_append(x, x, x, pos, none, freqs, c, c.clone())
    z = ops.rope_append(y, x, x, -pos, none, freqs, c, c.clone())
    assert (z - x).abs().max() < 2.0 ** -18 * 8
    eighth = torch.full((D // 2,), 0.125, dtype=torch.float64, device="cuda")
    a = ops.rope_append(x, x, x, pos, none, eighth, c, c.clone())
    b = ops.rope_append(x, x, x, pos + 8 * (1 << 28), none, eighth, c, c.clone())
    assert torch.equal(a, b)


# ---- attention --------------------------------------------------------------------

def check_attention(ops, g, dtype, hq, hkv, D, page, news, lens, window=0, see=None, scale=None,
                    heads_first=False, fused=False, fill=float("nan"), spoil=None):
    dt = DTYPES[dtype]
    kc, vc, table, ks, vs = build_cache(g, lens, page, hkv, D, dt, fill=fill,
                                        heads_first=heads_first)
    if spoil:
        spoil(kc, vc, table, ks, vs)
    T = sum(news)
    q = randn(g, (T, hq + 2, D), dt)[:, 1:hq + 1] if fused else randn(g, (T, hq, D), dt)
    q_start = torch.tensor([0] + [sum(news[:i + 1]) for i in range(len(news))], dtype=torch.int32,
                           device="cuda")
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    mask = None
    if see is not None:
        words = max(1, -(-max(news) // 32))
        rows = []
        for s in see:
            n = s.shape[0]
            bits = torch.nn.functional.pad(s, (0, words * 32 - n)).view(n, words, 32).long()
            bits = (bits << torch.arange(32, device="cuda")).sum(-1)
            rows.append(torch.where(bits >= 2 ** 31, bits - 2 ** 32, bits).int())
        mask = torch.cat(rows).contiguous()
    lse = torch.empty(T, hq, device="cuda")
    out = ops.attention(q, kc, vc, table, q_start, kv_len, scale=scale, window=window,
                        tree_mask=mask, lse=lse)
    sc = 1 / math.sqrt(D) if scale is None else scale
    o, mag, l, big = attention_ref(q, ks, vs, news, sc, window, see)
    within(out, o, attention_bound(o, torch.nan_to_num(mag, posinf=0.0), big, D, dt))
    within(lse, l, score_error(big, D) + 2.0 ** -20 * l.abs().nan_to_num(posinf=0.0))
    assert ops.status() == sv.SV_OK
    again = ops.attention(q, kc, vc, table, q_start, kv_len, scale=scale, window=window,
                          tree_mask=mask)
    assert torch.equal(torch.nan_to_num(out), torch.nan_to_num(again))
    return out


RAGGED = [([1], [1]), ([1, 1, 1], [2, 128, 129]), ([5], [5]), ([5, 5], [1000, 127]),
          ([0, 3, 1], [10, 257, 64]), ([1, 7, 2], [0, 3, 400]),  # rows that see nothing
          ([65, 17], [65, 700]), ([130, 1, 300], [300, 513, 1024]), ([257], [2049])]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("case", range(len(RAGGED)))
@pytest.mark.parametrize("hq,hkv,D,page", [(8, 2, 128, 16), (4, 4, 64, 64), (6, 1, 80, 8),
                                           (7, 1, 128, 128), (5, 1, 96, 256), (2, 2, 48, 3)])
def test_attention_ragged(ops, dtype, case, hq, hkv, D, page):
    news, lens = RAGGED[case]
    check_attention(ops, gen(case * 7 + D), dtype, hq, hkv, D, page, news, lens)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("hq,hkv,D,page", [(32, 8, 128, 16), (16, 1, 128, 32), (12, 4, 64, 16),
                                           (1, 1, 8, 8), (3, 1, 256, 16), (2, 1, 13, 16),
                                           (40, 1, 128, 64), (200, 1, 64, 16)])
def test_attention_head_layouts(ops, dtype, hq, hkv, D, page):
    check_attention(ops, gen(hq + D), dtype, hq, hkv, D, page, [4, 1, 9], [333, 1200, 9])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("window", [1, 2, 100, 128, 129, 5000])
def test_attention_window(ops, dtype, window):
    check_attention(ops, gen(window), dtype, 8, 2, 128, 16, [1, 5, 300, 2], [4000, 600, 777, 2],
                    window=window)


def tree_of(g, n):
    see = torch.zeros((n, n), dtype=torch.bool, device="cuda")
    parents = []
    for i in range(n):
        if i:
            p = int(torch.randint(0, i, (1,), generator=g, device="cuda"))
            see[i] = see[p]
            parents.append(p - 1)
        see[i, i] = True
    return see, parents


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n,kv", [(2, 2), (33, 400), (65, 65), (65, 1025), (40, 127)])
def test_attention_tree(ops, dtype, n, kv):
    g = gen(n * kv)
    trees = [tree_of(g, n) for _ in range(3)]
    parents = torch.tensor([t[1] for t in trees], dtype=torch.int32, device="cuda")
    out = check_attention(ops, g, dtype, 8, 2, 128, 16, [n] * 3, [kv, kv + 100, kv + 1],
                          see=[t[0] for t in trees])
    assert out.shape[0] == 3 * n
    # the mask made from the parents is the same
    words = ops.tree_mask(parents)
    want = torch.cat([t[0] for t in trees])
    got = ((words[:, :, None] >> torch.arange(32, device="cuda")) & 1).flatten(1)[:, :n].bool()
    assert torch.equal(got, want)
    assert ops.status() == sv.SV_OK


def test_attention_tree_rows_that_see_nothing(ops):
    g = gen(2)
    see = torch.zeros((5, 5), dtype=torch.bool, device="cuda")
    see[1, 3] = True
    see[4] = True
    out = check_attention(ops, g, "bf16", 4, 2, 64, 16, [5], [5], see=[see])
    assert not out[0].any() and not out[2].any() and out[1].any()


def test_tree_mask_of_a_bad_parent(ops):
    p = torch.tensor([[-1, 0, 5, 2]], dtype=torch.int32, device="cuda")
    m = ops.tree_mask(p)
    assert ops.status() == sv.SV_ERR_TOKEN
    assert m[:, 0].tolist()[:3] == [1, 3, 7]


@pytest.mark.parametrize("heads_first,fused", [(True, False), (False, True), (True, True)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_strides(ops, dtype, heads_first, fused):
    check_attention(ops, gen(1), dtype, 8, 4, 64, 32, [3, 140], [200, 350],
                    heads_first=heads_first, fused=fused)


@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("page", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("hkv", [1, 3])
def test_attention_heads_of_128(ops, heads_first, page, hkv):
    """Rows of two 128-byte halves, in both orders of the cache; one and many
    rows, ends inside a page and on its edge."""
    check_attention(ops, gen(page), "bf16", 2 * hkv, hkv, 128, page, [1, 5, 150, 2],
                    [page, 517, 150, 2 * page + 1], heads_first=heads_first)


@pytest.mark.parametrize("n", [6, 200])
def test_attention_heads_of_128_masked_values_do_not_count(ops, n):
    def spoil(kc, vc, table, ks, vs):
        kv = vs[0].shape[0]
        at = kv - 2
        pg, off = int(table[0, at // 16]), at % 16
        vs[0][at, 0, 3] = vc[pg, off, 0, 3] = float("inf")
        vs[0][at, 1, 100] = vc[pg, off, 1, 100] = float("nan")
        at = kv - 1
        pg, off = int(table[0, at // 16]), at % 16
        ks[0][at, 1, 70] = float("nan")
        kc[pg, off, 1, 70] = float("nan")
    check_attention(ops, gen(n), "fp16", 4, 2, 128, 16, [n, 3], [n + 300, 70], spoil=spoil)


@pytest.mark.parametrize("page", [8, 16, 32])
def test_attention_cache_orders_agree(ops, page):
    """K and V of different orders give what equal orders give."""
    g = gen(page)
    news, lens, hkv = [5, 140], [700, 333], 2
    kc, vc, table, _, _ = build_cache(g, lens, page, hkv, 128, torch.bfloat16)
    q = randn(g, (sum(news), 3 * hkv, 128), torch.bfloat16)
    qs = torch.tensor([0, 5, 145], dtype=torch.int32, device="cuda")
    kl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    turn = lambda c: c.transpose(1, 2).contiguous().transpose(1, 2)
    want = ops.attention(q, kc, vc, table, qs, kl)
    for k, v in ((kc, turn(vc)), (turn(kc), vc), (turn(kc), turn(vc))):
        assert torch.equal(ops.attention(q, k, v, table, qs, kl), want)
    assert torch.isfinite(want).all() and ops.status() == sv.SV_OK


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n", [6, 200])
def test_attention_masked_values_do_not_count(ops, dtype, n):
    """NaN and infinities in the keys and values that some rows do not see."""
    g = gen(n)

    def spoil(kc, vc, table, ks, vs):
        kv = vs[0].shape[0]
        for at, bad in ((kv - 2, float("nan")), (kv - 4, float("inf"))):
            pg, off = int(table[0, at // 16]), at % 16
            vs[0][at, 0, 3] = vc[pg, off, 0, 3] = bad
        at = kv - 1
        pg, off = int(table[0, at // 16]), at % 16
        ks[0][at, 1] = float("nan")
        kc[pg, off, 1] = float("nan")
    check_attention(ops, g, dtype, 8, 2, 64, 16, [n, 3], [n + 300, 70], spoil=spoil)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_attention_large_scores(ops, dtype):
    """One key takes all the weight, then another; negative and zero scales."""
    for scale in (40.0, -3.0, 0.0):
        check_attention(ops, gen(11), dtype, 4, 1, 64, 16, [9, 1], [900, 333], scale=scale)


def test_attention_bad_sequences(ops):
    g = gen(12)
    kc, vc, table, ks, vs = build_cache(g, [100, 50, 40], 16, 2, 64, torch.bfloat16, fill=1.0)
    q = randn(g, (6, 4, 64), torch.bfloat16)
    qs = torch.tensor([0, 2, 4, 6], dtype=torch.int32, device="cuda")
    good = torch.tensor([100, 50, 40], dtype=torch.int32, device="cuda")
    want = ops.attention(q, kc, vc, table, qs, good)
    lens = torch.tensor([100, 1 << 20, -1], dtype=torch.int32, device="cuda")
    out = ops.attention(q, kc, vc, table, qs, lens)
    assert ops.status() == sv.SV_ERR_CACHE
    assert torch.equal(out[:2], want[:2]) and not out[2:].any()
    bad = table.clone()
    bad[1, 0] = 1 << 30
    bad[2, 1] = -7
    out = ops.attention(q, kc, vc, bad, qs, good)
    assert ops.status() == sv.SV_ERR_CACHE
    assert torch.equal(out[:2], want[:2]) and torch.isfinite(out).all()
    out = torch.full_like(q, 9.0)
    ops.attention(q, kc, vc, table, torch.tensor([0, 2, 99, 6], dtype=torch.int32, device="cuda"),
                  good, out=out)
    assert ops.status() == sv.SV_ERR_CACHE
    assert torch.equal(out[:2], want[:2]) and (out[2:] == 9).all()


def test_attention_output_strides(ops):
    g = gen(13)
    kc, vc, table, ks, vs = build_cache(g, [70, 200], 16, 2, 64, torch.bfloat16)
    q = randn(g, (12, 4, 64), torch.bfloat16)
    qs = torch.tensor([0, 5, 12], dtype=torch.int32, device="cuda")
    kl = torch.tensor([70, 200], dtype=torch.int32, device="cuda")
    want = ops.attention(q, kc, vc, table, qs, kl)
    big = torch.full((12, 6, 72), 5.0, dtype=torch.bfloat16, device="cuda")
    for off in (0, 3):
        big.fill_(5.0)
        out = big[:, 1:5, off:off + 64]
        ops.attention(q, kc, vc, table, qs, kl, out=out)
        assert torch.equal(out, want)
        assert int((big != 5.0).sum()) <= want.numel()


@pytest.mark.parametrize("B", [33, 64, 400, 1000])
def test_attention_many_sequences(ops, B):
    """More sequences than a warp and than a block counts at once, some empty."""
    g = gen(B)
    news = torch.randint(0, 4, (B,), generator=g, device="cuda").tolist()
    lens = torch.randint(0, 300, (B,), generator=g, device="cuda").tolist()
    news[0], news[-1], lens[B // 2] = 0, 2, 0
    check_attention(ops, g, "bf16", 4, 2, 64, 16, news, lens)


@pytest.mark.parametrize("hq,hkv,news,lens", [
    (4, 1, [3, 1], [30000, 500]),        # one cache head: parts on every SM
    (4, 1, [2100], [2500]),              # more items of a sequence than lanes
    (2, 2, [1300, 40, 7], [1300, 9000, 64]),
])
def test_attention_long(ops, hq, hkv, news, lens):
    check_attention(ops, gen(len(news)), "bf16", hq, hkv, 64, 32, news, lens)


def test_attention_odd_alignments(ops):
    """Queries and caches off 16 bytes, and strides that are no multiple of them."""
    g = gen(14)
    for name in ("q", "cache", "both"):
        kc, vc, table, ks, vs = build_cache(g, [200, 90], 16, 2, 64, torch.bfloat16, fill=0.0)
        q = randn(g, (6, 4, 64), torch.bfloat16)
        want_q = q
        if name != "cache":
            q = torch.nn.functional.pad(q, (1, 2))[..., 1:65]
        if name != "q":
            kc = torch.nn.functional.pad(kc, (3, 0))[..., 3:]
            vc = torch.nn.functional.pad(vc, (1, 0))[..., 1:]
        qs = torch.tensor([0, 4, 6], dtype=torch.int32, device="cuda")
        kl = torch.tensor([200, 90], dtype=torch.int32, device="cuda")
        out = ops.attention(q, kc, vc, table, qs, kl)
        o, mag, _, big = attention_ref(want_q, ks, vs, [4, 2], 0.125)
        within(out, o, attention_bound(o, mag, big, 64, torch.bfloat16))


def test_attention_query_not_finite(ops):
    """A NaN query spoils its own row only."""
    g = gen(15)
    kc, vc, table, ks, vs = build_cache(g, [300], 16, 1, 64, torch.bfloat16)
    q = randn(g, (9, 4, 64), torch.bfloat16)
    qs = torch.tensor([0, 9], dtype=torch.int32, device="cuda")
    kl = torch.tensor([300], dtype=torch.int32, device="cuda")
    want = ops.attention(q, kc, vc, table, qs, kl)
    q[4, 2, 5] = float("nan")
    out = ops.attention(q, kc, vc, table, qs, kl)
    assert torch.isnan(out[4, 2]).all()
    out[4, 2] = want[4, 2]
    assert torch.equal(out, want)


# ---- refusals through Python, waits that run out ---------------------------------------

def test_refusals_through_python(ops):
    x = torch.ones(4, 72, device="cuda").to(torch.float8_e4m3fn)
    s = torch.ones(4, 1, device="cuda")
    with pytest.raises(sv.SpecVerifyError) as e:
        ops.matmul_fp8(x, s, x, torch.ones(1, 1, device="cuda"))  # K no multiple of 16
    assert e.value.code == sv.SV_ERR_SHAPE
    h = torch.ones(4, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    with pytest.raises(sv.SpecVerifyError) as e:
        ops.rms_norm(h, w, eps=-1.0)
    assert e.value.code == sv.SV_ERR_ARG
    with pytest.raises(sv.SpecVerifyError) as e:
        ops.rms_norm_fp8(h, w, group=64)
    assert e.value.code == sv.SV_ERR_ARG
    for bad in (h.cpu(), h.double(), h[0], "x"):
        with pytest.raises(ValueError):
            ops.rms_norm(bad, w)
    with pytest.raises(ValueError):
        ops.matmul_fp8(x, s, x, torch.ones(1, 1, device="cuda"), out_dtype=torch.float64)
    c = torch.zeros(2, 16, 1, 64, device="cuda")
    q = torch.zeros(2, 3, 64, device="cuda")
    i = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    two = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    one = torch.tensor([2], dtype=torch.int32, device="cuda")
    with pytest.raises(sv.SpecVerifyError):
        ops.attention(q, c, c, i, two, one, window=-1)
    with pytest.raises(ValueError):
        ops.attention(q, c, c, i.long(), two, one)
    with pytest.raises(ValueError):
        ops.attention(q, c, c.half(), i, two, one)
    assert ops.attention(q, c, c, i, two, one).shape == q.shape
    closed = sv.TargetOps()
    closed.close()
    with pytest.raises(sv.SpecVerifyError) as e:
        closed.rms_norm(h, w)
    assert e.value.code == sv.SV_ERR_ARG


def test_a_given_stream(ops):
    g = gen(16)
    x, w = randn(g, (33, 512), torch.bfloat16), randn(g, (512,), torch.bfloat16)
    want = ops.rms_norm(x, w)[0]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        got = ops.rms_norm(x, w, stream=stream)[0]
        side.synchronize()
        assert torch.equal(got, want)
    assert torch.cuda.current_stream() != side


def test_a_wait_limit_of_nothing():
    """With a limit of nothing a wait that is not soon satisfied gives up: the
    call ends, either with its result or with a status that says so, and the
    next call is right."""
    ops = sv.TargetOps()
    g = gen(17)
    a, sa = quant_blocks(randn(g, (40, 2048)), 1)
    w, sw = quant_blocks(randn(g, (512, 2048)), 128)
    kc, vc, table, ks, vs = build_cache(g, [900], 16, 2, 64, torch.bfloat16, fill=0.0)
    q = randn(g, (5, 4, 64), torch.bfloat16)
    qs = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    kl = torch.tensor([900], dtype=torch.int32, device="cuda")
    calls = (lambda: ops.matmul_fp8(a, sa, w, sw), lambda: ops.attention(q, kc, vc, table, qs, kl))
    for call in calls:
        want = call()
        assert ops.status() == sv.SV_OK
        ops.set_wait_limit(0)
        for _ in range(20):
            got = call()
            code = ops.status()
            assert code == sv.SV_ERR_TIMEOUT or (code == sv.SV_OK and torch.equal(got, want))
        ops.set_wait_limit(10 ** 9)
        assert torch.equal(call(), want)
        assert ops.status() == sv.SV_OK


# ---- streams, graphs, use together ---------------------------------------------------

def test_other_streams_and_graphs(ops):
    g = gen(21)
    a, sa = quant_blocks(randn(g, (20, 512)), 1)
    w, sw = quant_blocks(randn(g, (384, 512)), 128)
    kc, vc, table, ks, vs = build_cache(g, [300, 77], 16, 2, 64, torch.bfloat16)
    q = randn(g, (7, 4, 64), torch.bfloat16)
    qs = torch.tensor([0, 4, 7], dtype=torch.int32, device="cuda")
    kl = torch.tensor([300, 77], dtype=torch.int32, device="cuda")
    x = randn(g, (20, 512), torch.bfloat16)
    nw = randn(g, (512,), torch.bfloat16)

    def calls():
        return [ops.matmul_fp8(a, sa, w, sw), ops.attention(q, kc, vc, table, qs, kl),
                *ops.rms_norm_fp8(x, nw, 1e-6)]
    want = [t.clone() for t in calls()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = calls()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = calls()
    for _ in range(3):
        for t in held:
            t.view(torch.uint8).zero_()
        graph.replay()
    torch.cuda.synchronize()
    for u, v, z in zip(want, got, held):
        assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))
        assert torch.equal(u.view(torch.uint8), z.view(torch.uint8))
    # a graph whose cache lengths change between replays
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = ops.attention(q, kc, vc, table, qs, kl)
    kl.copy_(torch.tensor([150, 60], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held, ops.attention(q, kc, vc, table, qs, kl))
