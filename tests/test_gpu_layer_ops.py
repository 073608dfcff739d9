"""The operators of a layer's second half and the log probabilities against
plain 64-bit implementations."""
import math

import pytest
import torch

import speculative_decoding_verification_22_gb300 as sv
from layer_common import (ACTS, block_norm_ref, gated_ref, linear_ref, log_probs_error,
                          log_probs_ref, rounded)
from target_common import DTYPES, HALF_STEP, TINY, gen, randn, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    o = sv.TargetOps()
    yield o
    o.close()


# ---- linear and gated linear ----------------------------------------------------

# (M, N, K): single tokens, a round, both sides of every change of form, ragged
# rows, columns and K, one column, many rows
SIZES = [(1, 64, 64), (1, 1, 8), (5, 4096, 512), (5, 192, 4096), (8, 1000, 136), (16, 250, 1032),
         (17, 129, 72), (33, 640, 2048), (64, 257, 520), (65, 384, 256), (96, 8, 128),
         (128, 130, 192), (129, 513, 328), (200, 1024, 1000), (256, 256, 64), (257, 255, 72),
         (300, 72, 4104), (513, 1030, 264), (1000, 520, 512), (2049, 264, 128), (800, 1408, 512),
         (1500, 1120, 192), (260, 4000, 320)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_linear_of_whole_numbers_is_exact(ops, M, N, K, dtype):
    """Products and sums of small whole numbers are exact in fp32 whatever their
    order, so every element counts."""
    g = gen(M + 3 * N + 7 * K)
    dt = DTYPES[dtype]

    def whole(*shape):
        return torch.randint(-2, 3, shape, generator=g, device="cuda").to(dt)
    x, w, b = whole(M, K), whole(N, K), whole(N)
    res = whole(M, N).float()
    got = ops.linear(x, w, bias=b, activation="relu", residual=res, out_dtype=torch.float32)
    want = (x.double() @ w.double().t() + b.double()).clamp_min(0) + res.double()
    assert torch.equal(got.double(), want)
    assert torch.equal(ops.linear(x, w), (x.double() @ w.double().t()).to(dt))
    assert ops.status() == sv.SV_OK


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_gated_linear_of_whole_numbers_is_exact(ops, M, N, K, dtype):
    g = gen(M + 5 * N + 11 * K)
    dt = DTYPES[dtype]

    def whole(*shape):
        return torch.randint(-1, 2, shape, generator=g, device="cuda").to(dt)
    x, wg, wu, bg, bu = whole(M, K), whole(N, K), whole(N, K), whole(N), whole(N)
    got = ops.gated_linear(x, wg, wu, bg, bu, activation="relu", out_dtype=torch.float32)
    a = (x.double() @ wg.double().t() + bg.double()).clamp_min(0)
    u = x.double() @ wu.double().t() + bu.double()
    assert torch.equal(got.double(), (a * u).float().double())
    got = ops.gated_linear(x, wg, wu, activation="none")
    a, u = x.double() @ wg.double().t(), x.double() @ wu.double().t()
    assert torch.equal(got, (a * u).float().to(dt))
    assert ops.status() == sv.SV_OK


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [3, 70, 300])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"),
                                       ("fp16", "bf16"), ("fp32", "fp32"), ("fp32", "fp16")])
def test_linear_epilogue(ops, act, M, dtype, out):
    g = gen(M + len(act))
    N, K = 200, 320
    dt, od = DTYPES[dtype], DTYPES[out]
    x, w = randn(g, (M, K), dt), randn(g, (N, K), dt, 3 * K ** -0.5)
    b, res = randn(g, (N,), dt, 4.0), randn(g, (M, N), od, 2.0)
    for bias, r in ((None, None), (b, None), (None, res), (b, res)):
        ref, bound = linear_ref(x, w, bias, act, r, od)
        within(ops.linear(x, w, bias, act, r, od), ref, bound)
    wu = randn(g, (N, K), dt, K ** -0.5)
    for bg, bu in ((None, None), (b, None), (None, b), (b, b)):
        ref, bound = gated_ref(x, w, wu, bg, bu, act, od)
        within(ops.gated_linear(x, w, wu, bg, bu, act, od), ref, bound)
    assert ops.status() == sv.SV_OK


@pytest.mark.parametrize("M", [2, 40, 200])
@pytest.mark.parametrize("act", ACTS)
def test_activations_far_from_zero_and_beyond(ops, M, act):
    """Through an identity: values of every size, both signs, zeros, infinities and
    NaN; what the limit forms give is compared with the 64-bit formulas."""
    v = torch.tensor([0.0, -0.0, 1e-6, -1e-6, 0.3, -0.3, 1.0, -1.0, 3.0, -3.0, 6.0, -6.0, 9.0, -9.0,
                      12.0, -12.0, 20.0, -20.0, 87.5, -87.5, 300.0, -300.0, 6e4, -6e4, 3e8, -3e8,
                      math.inf, math.nan, 0.5, -0.5, 2.0, -2.0], device="cuda")
    K = v.numel()
    eye = torch.eye(K, device="cuda").bfloat16()
    zero = torch.zeros(M, K, device="cuda").bfloat16()
    got = ops.linear(zero, eye, v.bfloat16(), act, out_dtype=torch.float32)
    ref, bound = linear_ref(zero, eye, v.bfloat16(), act, None, torch.float32)
    ref[:, v == math.inf] = math.inf
    within(got, ref, bound)


@pytest.mark.parametrize("M", [1, 5, 90, 140, 400])
@pytest.mark.parametrize("kind", ["slices", "odd k", "odd rows", "odd start", "odd out", "fused"])
def test_products_of_other_layouts(ops, M, kind):
    """Rows of wider tensors, strides and starts that no 16-byte load can take."""
    g = gen(M + len(kind))
    N, K = 136, 192
    if kind == "odd k":
        K = 187
    big_x, big_w = randn(g, (M, K + 64), torch.bfloat16), randn(g, (2 * N, K + 64),
                                                                torch.bfloat16, K ** -0.5)
    x, w, wu = big_x[:, :K], big_w[:N, :K], big_w[N:, :K]
    out = torch.full((M, N + 16), 7.0, dtype=torch.bfloat16, device="cuda")[:, 8:N + 8]
    if kind == "odd rows":
        x = randn(g, (M, K + 3), torch.bfloat16)[:, :K]
    if kind == "odd start":
        w, wu = big_w[:N, 1:K + 1], big_w[N:, 3:K + 3]
    if kind == "odd out":
        out = torch.full((M, N + 5), 7.0, dtype=torch.bfloat16, device="cuda")[:, 1:N + 1]
    if kind == "fused":
        x, fused = big_x[:, :K].contiguous(), randn(g, (2 * N, K), torch.bfloat16, K ** -0.5)
        w, wu = fused[:N], fused[N:]
    wide = out._base if out._base is not None else out
    bias = randn(g, (N,), torch.bfloat16)
    back = ops.linear(x, w, bias, "silu", out=out)
    assert back.data_ptr() == out.data_ptr()
    within(out, *linear_ref(x, w, bias, "silu"))
    res = out.clone()
    ops.linear(x, w, residual=out, out=out)  # in place
    within(out, *linear_ref(x, w, residual=res))
    ops.gated_linear(x, w, wu, out=out)
    within(out, *gated_ref(x, w, wu))
    left = torch.ones(wide.shape, dtype=torch.bool, device="cuda")
    left.as_strided(out.shape, out.stride(), out.storage_offset()).fill_(False)
    assert (wide[left] == 7).all()  # nothing beside the output was touched
    assert ops.status() == sv.SV_OK


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 5, 3), (7, 9, 5), (3, 130, 1), (40, 33, 7),
                                   (150, 70, 9), (260, 300, 3)])
@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_products_of_the_smallest_depths(ops, M, N, K, aligned, dtype):
    """K below a 16-byte load, in rows that are aligned and in dense ones; whole
    numbers, so exact."""
    g = gen(M + N + K)
    dt, width = DTYPES[dtype], 16 if aligned else K

    def whole(rows):
        t = torch.full((rows, width), math.nan, dtype=dt, device="cuda")  # nothing beside is read
        t[:, :K] = torch.randint(-3, 4, (rows, K), generator=g, device="cuda").to(dt)
        return t[:, :K]
    x, w, u = whole(M), whole(N), whole(N)
    want = x.double() @ w.double().t()
    assert torch.equal(ops.linear(x, w, out_dtype=torch.float32).double(), want)
    assert torch.equal(ops.gated_linear(x, w, u, activation="none", out_dtype=torch.float32)
                       .double(), want * (x.double() @ u.double().t()))


@pytest.mark.parametrize("M", [1, 3, 8, 9, 31, 32, 33, 100])
@pytest.mark.parametrize("N,K", [(1, 40), (17, 1), (255, 1000), (600, 333)])
def test_products_in_fp32(ops, M, N, K):
    g = gen(M + N)
    x, w = randn(g, (M, K)), randn(g, (N, K), scale=K ** -0.5)
    u, b, r = randn(g, (N, K), scale=K ** -0.5), randn(g, (N,)), randn(g, (M, N))
    within(ops.linear(x, w, b, "gelu_tanh", r), *linear_ref(x, w, b, "gelu_tanh", r))
    within(ops.gated_linear(x, w, u, b, b), *gated_ref(x, w, u, b, b))


@pytest.mark.parametrize("M", [4, 100, 260])
def test_not_finite_inputs_stay_in_their_rows_and_columns(ops, M):
    g = gen(M)
    N, K = 140, 136
    x, w = randn(g, (M, K), torch.bfloat16), randn(g, (N, K), torch.bfloat16)
    want = ops.linear(x, w)
    x[1, 5], w[7, 3] = math.nan, math.inf
    got = ops.linear(x, w)
    assert torch.isnan(got[1]).all()
    rows = torch.arange(M, device="cuda") != 1
    assert not torch.isfinite(got[rows][:, 7]).any()
    cols = torch.arange(N, device="cuda") != 7
    assert torch.equal(got[rows][:, cols], want[rows][:, cols])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_no_rows(ops, dtype):
    x = torch.empty(0, 64, dtype=DTYPES[dtype], device="cuda")
    w = torch.ones(24, 64, dtype=DTYPES[dtype], device="cuda")
    assert ops.linear(x, w).shape == (0, 24)
    assert ops.gated_linear(x, w, w).shape == (0, 24)
    out, h = ops.block_norm(x, x, w[0])
    assert out.shape == h.shape == (0, 64)
    assert ops.log_probs(x, top=2)[2].shape == (0, 2)


# ---- block norm ------------------------------------------------------------------

def gate_of(g, kind, rows, d, dt):
    shape = {"none": None, "column": (d,), "one row": (1, d), "row": (rows, 1), "full": (rows, d),
             "one": (1, 1)}[kind]
    return None if shape is None else randn(g, shape, dt)


@pytest.mark.parametrize("rows,d", [(1, 1), (1, 8), (3, 100), (5, 4096), (2, 4100), (7, 129),
                                    (300, 512), (4, 8192), (2, 8200), (3, 16384), (160, 1000),
                                    (2, 12290), (2, 40000)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("gate", ["none", "column", "row", "full"])
def test_block_norm(ops, rows, d, dtype, gate):
    g = gen(rows * 31 + d)
    dt = DTYPES[dtype]
    x, res = randn(g, (rows, d), dt), randn(g, (rows, d), dt, 3.0)
    w, post = randn(g, (d,), dt), randn(g, (d,), dt)
    gt = gate_of(g, gate, rows, d, dt)
    for p in (None, post):
        want, h, dout, dh = block_norm_ref(x, res, w, p, gt, 0.7, 1e-5)
        out, ho = ops.block_norm(x, res, w, p, gt, 0.7, 1e-5)
        within(out, want, rounded(want, dout, dt))
        within(ho, h, rounded(h, dh, dt))
    assert ops.status() == sv.SV_OK


@pytest.mark.parametrize("rows,d", [(1, 1), (6, 512), (5, 130), (200, 1024)])
@pytest.mark.parametrize("gate", ["one row", "one"])
def test_block_norm_gates_for_all_rows(ops, rows, d, gate):
    g = gen(rows + d)
    x, res, w = (randn(g, s, torch.bfloat16) for s in ((rows, d), (rows, d), (d,)))
    gt = gate_of(g, gate, rows, d, torch.bfloat16)
    want, h, dout, dh = block_norm_ref(x, res, w, None, gt, -1.5)
    out, ho = ops.block_norm(x, res, w, None, gt, -1.5)
    within(out, want, rounded(want, dout, torch.bfloat16))
    within(ho, h, rounded(h, dh, torch.bfloat16))


@pytest.mark.parametrize("rows,d", [(1, 128), (4, 200), (5, 4096), (33, 8192), (3, 4090), (2, 20000)])
@pytest.mark.parametrize("group", [128, 0])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_block_norm_in_eight_bits(ops, rows, d, group, dtype):
    """The scale is that of the row's or block's maximum, and each value within half
    a step of E4M3 (2^-4, or 2^-10 where it is subnormal) of what it stands for."""
    g = gen(rows + d)
    dt = DTYPES[dtype]
    x, res = randn(g, (rows, d), dt), randn(g, (rows, d), dt, 3.0)
    w, post, gt = randn(g, (d,), dt), randn(g, (d,), dt), randn(g, (rows, d), dt)
    want, h, dout, dh = block_norm_ref(x, res, w, post, gt, 1.0, 1e-6)
    out8, scale, ho = ops.block_norm_fp8(x, res, w, post, gt, group=group)
    width = group or d
    pad = torch.nn.functional.pad(want, (0, -d % width)).view(rows, -1, width)
    most = pad.abs().amax(-1)
    err = torch.nn.functional.pad(dout, (0, -d % width)).view(rows, -1, width).amax(-1)
    s = scale.double().view(rows, -1)
    assert ((s - most / 448).abs() <= err / 448 + most / 448 * 2.0 ** -22).all()
    each = s.repeat_interleave(width, 1)[:, :d]
    got = out8.double() * each
    bound = dout + want.abs() * (2.0 ** -4 + 2.0 ** -20) + each * 2.0 ** -10 * 1.01
    assert ((got - want).abs() <= bound).all()
    within(ho, h, rounded(h, dh, dt))


@pytest.mark.parametrize("d", [256, 250])
@pytest.mark.parametrize("kind", ["in place", "x in place", "strides", "odd starts"])
def test_block_norm_layouts(ops, d, kind):
    g = gen(d + len(kind))
    rows, dt = 37, torch.bfloat16
    x, res = randn(g, (rows, d + 8), dt)[:, :d], randn(g, (rows, d + 16), dt)[:, :d]
    if kind == "odd starts":
        x, res = randn(g, (rows, d + 7), dt)[:, 1:d + 1], randn(g, (rows, d + 5), dt)[:, 3:d + 3]
    w, post = randn(g, (d,), dt), randn(g, (d,), dt)
    gt = randn(g, (rows, d + 24), dt)[:, :d]
    want, h, dout, dh = block_norm_ref(x, res, w, post, gt)
    out, ro = None, None
    if kind == "in place":
        ro = res
    if kind == "x in place":
        out, ro = x, res
    if kind == "strides":
        out = torch.zeros(rows, d + 40, dtype=dt, device="cuda")[:, :d]
        ro = torch.zeros(rows, d + 32, dtype=dt, device="cuda")[:, :d]
    got, ho = ops.block_norm(x, res, w, post, gt, out=out, residual_out=ro)
    within(got, want, rounded(want, dout, dt))
    within(ho, h, rounded(h, dh, dt))


@pytest.mark.parametrize("d", [64, 4096, 4099])
def test_block_norm_of_zeros_and_of_what_is_not_finite(ops, d):
    x = torch.zeros(3, d, device="cuda")
    res, w = torch.zeros(3, d, device="cuda"), torch.ones(d, device="cuda")
    x[1, 3], res[2, 1] = math.nan, math.inf
    out, h = ops.block_norm(x, res, w, w)
    assert (out[0] == 0).all() and (h[0] == 0).all()
    assert torch.isnan(out[1]).all() and torch.isnan(h[1]).all()
    assert h[2, 1] == math.inf and torch.isnan(out[2, 1]) and (h[2, 2:] == 0).all()
    out8, scale, _ = ops.block_norm_fp8(x, res, w, w, group=0)
    assert (out8[0].float() == 0).all() and scale[0] > 0 and torch.isnan(scale[1:]).all()


def test_block_norm_equals_the_residual_norm_without_its_extras(ops):
    """post_weight, gate and scale left out: the same formula as rms_norm."""
    g = gen(5)
    x, res, w = (randn(g, s, torch.bfloat16) for s in ((9, 512), (9, 512), (512,)))
    out, h = ops.block_norm(x, res, w)
    out2, h2 = ops.rms_norm(x, w, residual=res)
    assert torch.equal(h, h2)
    # sums in another order: the norms may differ by their roundings
    assert ((out - out2).double().abs() <= out2.double().abs() * 2.0 ** -7).all()


# ---- log probabilities --------------------------------------------------------------

def check_log_probs(ops, x, t, top, T):
    V = x.shape[1]
    want = log_probs_ref(x, t, top, T)
    got = ops.log_probs(x, t, top, T)
    assert len(got) == (4 if top else 2)
    within(got[0], want[0], log_probs_error(want[0], V))
    ent = want[1].abs() * (V / 256 + 64) * 2.0 ** -22 + (V / 256 + 64) * 2.0 ** -24
    within(got[1], want[1], ent)
    if top:
        assert torch.equal(got[2], want[2])
        within(got[3], want[3], log_probs_error(want[3], V))
    return got


def logit_rows(g, R, V, dt, spread=3.0):
    x = randn(g, (R, V), torch.float32, spread)
    x[:, :: max(1, V // 5)] += 8.0
    return x.to(dt)


@pytest.mark.parametrize("R,V", [(1, 1), (1, 7), (3, 64), (2, 1000), (5, 32003), (5, 128256),
                                 (1, 131072), (40, 5000), (160, 1001), (700, 515), (3000, 40),
                                 (310, 20001)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("top", [0, 1, 5, 64])
def test_log_probs(ops, R, V, dtype, top):
    g = gen(R + V)
    x = logit_rows(g, R, V, DTYPES[dtype])
    t = torch.randint(-1, V, (R, 3), generator=g, device="cuda", dtype=torch.int32)
    check_log_probs(ops, x, t, min(top, V), 1.0 if top != 5 else 0.7)
    assert ops.status() == sv.SV_OK


@pytest.mark.parametrize("R", [1, 4, 600])
@pytest.mark.parametrize("V", [33, 4096, 50001])
@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "two values", "last", "masked",
                                  "one left", "far", "lowest", "late"])
def test_log_probs_of_hard_rows(ops, R, V, kind):
    """Orders and ties that make every element a candidate, masks of -inf and of the
    type's lowest value, rows with one token left."""
    g = gen(V + R)
    dt = torch.bfloat16 if kind in ("two values", "lowest") else torch.float32
    x = torch.arange(V, device="cuda").float()[None].repeat(R, 1) / V * 20
    if kind == "equal":
        x = torch.full_like(x, -3.0)
    elif kind == "falling":
        x = -x
    elif kind == "two values":
        x = torch.randint(0, 2, (R, V), generator=g, device="cuda").float()
    elif kind == "last":
        x = torch.zeros_like(x)
        x[:, -1] = 1.0
    elif kind == "masked":
        x = torch.where(torch.rand(R, V, generator=g, device="cuda") < 0.95, -math.inf, x)
        x[:, 7] = 1.0
    elif kind == "one left":
        x = torch.full_like(x, -math.inf)
        x[:, V // 2] = -5.0
    elif kind == "far":
        x = torch.where(torch.arange(V, device="cuda") % 7 == 0, x + 1000, x - 1000)
    elif kind == "lowest":
        x = torch.where(torch.rand(R, V, generator=g, device="cuda") < 0.5,
                        torch.finfo(dt).min, x)
        x[:, 7] = 1.0
    elif kind == "late":
        x = randn(g, (R, V))
        x[:, V - V // 4:] += 30
    t = torch.randint(0, V, (R, 2), generator=g, device="cuda", dtype=torch.int32)
    check_log_probs(ops, x.to(dt).contiguous(), t, 20, 1.0)


@pytest.mark.parametrize("R,V", [(3, 70), (2, 1000), (5, 128256), (300, 20003)])
@pytest.mark.parametrize("keep", [1, 9, 64, 65])
@pytest.mark.parametrize("where", ["anywhere", "first", "last"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("mask", [-math.inf, -30000.0])
def test_log_probs_of_rows_with_few_tokens_left(ops, R, V, keep, where, dtype, mask):
    """As many tokens allowed as alternatives, one more, fewer: the first of those that
    are not fill up.  Of the allowed ones two are equal and one is the lowest value, which may be below
    the mask's."""
    g = gen(V + keep)
    order = torch.rand(R, V, generator=g, device="cuda").argsort(1).argsort(1)
    if where != "anywhere":
        order = torch.arange(V, device="cuda")[None].repeat(R, 1)
        order = order if where == "first" else V - 1 - order
    x = randn(g, (R, V), torch.float32, 3.0).to(DTYPES[dtype])
    x[order == 1] = 1.0
    x[order == 2] = 1.0
    x[order == 3] = torch.finfo(x.dtype).min
    x[order >= keep] = mask
    t = torch.randint(0, V, (R, 2), generator=g, device="cuda", dtype=torch.int32)
    for top in (1, 8, 64):
        check_log_probs(ops, x, t, top, 1.0)


@pytest.mark.parametrize("V", [50, 70001])
def test_log_probs_of_rows_without_a_finite_maximum(ops, V):
    g = gen(V)
    x = randn(g, (6, V))
    x[1, 9], x[2, V - 1], x[3], x[4, 0] = math.nan, math.inf, -math.inf, -math.inf
    t = torch.full((6, 1), 3, dtype=torch.int32, device="cuda")
    got = check_log_probs(ops, x, t, 4, 1.0)
    for r in (1, 2, 3):
        assert torch.isnan(got[0][r]).all() and torch.isnan(got[1][r])
        assert (got[2][r] == -1).all() and torch.isnan(got[3][r]).all()


def test_log_probs_of_tokens_outside_the_vocabulary(ops):
    x = randn(gen(1), (3, 100))
    t = torch.tensor([[5, -1], [100, 2], [-2, 99]], dtype=torch.int32, device="cuda")
    got = check_log_probs(ops, x, t, 0, 1.0)
    assert got[0][0, 1] == 0 and torch.isnan(got[0][1, 0]) and torch.isnan(got[0][2, 0])
    assert ops.status() == sv.SV_ERR_TOKEN and ops.status() == sv.SV_OK


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("off", [0, 1, 3])
def test_log_probs_layouts(ops, dtype, off):
    g = gen(off)
    x = logit_rows(g, 9, 5000, DTYPES[dtype])[:, off:4700 + off]
    t = torch.randint(0, 4700, (9, 1), generator=g, device="cuda", dtype=torch.int32)
    got = check_log_probs(ops, x, t, 10, 1.0)
    outs = [torch.empty_like(o) for o in got]
    back = ops.log_probs(x, t, 10, 1.0, out=outs)
    assert all(torch.equal(a, b) and b.data_ptr() == c.data_ptr()
               for a, b, c in zip(got, outs, back))
    assert torch.equal(ops.log_probs(x)[1], got[1])  # no tokens, no alternatives


# ---- streams, graphs, repetition -------------------------------------------------------

def every_operator(ops, s, stream=None):
    outs = [ops.linear(s["x"], s["w"], s["b"], "gelu", s["r"], stream=stream),
            ops.gated_linear(s["x"], s["w"], s["w2"], stream=stream)]
    outs += ops.block_norm(s["r"], s["r2"], s["b"], s["b"], s["g"], 0.5, stream=stream)
    outs += ops.block_norm_fp8(s["r"], s["r2"], s["b"], s["b"], s["g"], 0.5, stream=stream)
    outs += ops.log_probs(s["l"], s["t"], 7, 0.8, stream=stream)
    return outs


def some_inputs(M, seed):
    g = gen(seed)
    N, K, V = 520, 328, 9001
    return dict(x=randn(g, (M, K), torch.bfloat16), w=randn(g, (N, K), torch.bfloat16, 0.05),
                w2=randn(g, (N, K), torch.bfloat16, 0.05), b=randn(g, (N,), torch.bfloat16),
                r=randn(g, (M, N), torch.bfloat16), r2=randn(g, (M, N), torch.bfloat16),
                g=randn(g, (M, 1), torch.bfloat16), l=randn(g, (M, V), torch.float32, 3.0),
                t=torch.randint(0, V, (M, 2), generator=g, device="cuda", dtype=torch.int32))


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("M", [1, 6, 130, 700])
def test_repeated_calls_are_the_same_bit_for_bit(ops, M):
    s = some_inputs(M, M)
    first = every_operator(ops, s)
    for _ in range(5):
        assert same(first, every_operator(ops, s))


@pytest.mark.parametrize("M", [6, 300])
def test_two_streams_on_one_handle_and_a_given_stream(ops, M):
    """The operators use no scratch, so calls on one handle may overlap."""
    one, two = some_inputs(M, 1), some_inputs(M, 2)
    want = every_operator(ops, one), every_operator(ops, two)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        got.append((every_operator(ops, one, a), every_operator(ops, two, b.cuda_stream)))
    torch.cuda.synchronize()
    for x, y in got:
        assert same(x, want[0]) and same(y, want[1])
    assert ops.status() == sv.SV_OK


@pytest.mark.parametrize("M", [6, 300])
def test_captured_and_replayed_with_other_inputs(ops, M):
    s, other = some_inputs(M, 3), some_inputs(M, 4)
    every_operator(ops, s)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = every_operator(ops, s)
        graphs.append((graph, outs))
    want = every_operator(ops, other)
    for k in s:
        s[k].copy_(other[k])
    for graph, _ in graphs:
        graph.replay()
    torch.cuda.synchronize()
    for _, outs in graphs:
        assert same(outs, want)


@pytest.mark.parametrize("M", [4, 200])
def test_the_block_of_a_layer(ops, M):
    """As a layer runs them: gated projections, the down projection onto the
    residual, the norm of the next block, its logits and what is said of them."""
    g = gen(M)
    d, F, V, bf = 256, 704, 1000, torch.bfloat16
    x, res = randn(g, (M, d), bf), randn(g, (M, d), bf)
    wg, wu = randn(g, (F, d), bf, d ** -0.5), randn(g, (F, d), bf, d ** -0.5)
    wd, head, n1 = randn(g, (d, F), bf, F ** -0.5), randn(g, (V, d), bf, d ** -0.5), randn(g, (d,), bf)
    h = ops.gated_linear(x, wg, wu)
    within(h, *gated_ref(x, wg, wu))
    y = ops.linear(h, wd, residual=res)
    within(y, *linear_ref(h, wd, residual=res))
    y2 = ops.linear(h, wd)
    out, r2 = ops.block_norm(y2, res, n1, n1, branch_scale=0.5)
    want, hh, dout, dh = block_norm_ref(y2, res, n1, n1, None, 0.5)
    within(out, want, rounded(want, dout, bf))
    logits = ops.linear(out, head, out_dtype=torch.float32)
    t = torch.randint(0, V, (M, 1), generator=g, device="cuda", dtype=torch.int32)
    check_log_probs(ops, logits, t, 5, 1.0)
    a8, scale, _ = ops.block_norm_fp8(y2, res, n1, n1, branch_scale=0.5)
    w8 = torch.ones(128, d, device="cuda").to(torch.float8_e4m3fn)
    got = ops.matmul_fp8(a8, scale, w8, torch.ones(1, 2, device="cuda"), torch.float32)
    # d values of half a step of E4M3 each
    total = want.sum(1, keepdim=True)
    assert ((got.double() - total).abs() <= want.abs().sum(1, keepdim=True) * 2.0 ** -3).all()
    assert ops.status() == sv.SV_OK


@pytest.mark.parametrize("M,N,K", [(5, 1024, 4096), (40, 300, 2048), (120, 2048, 512),
                                   (200, 512, 4096), (300, 3000, 1024), (700, 1030, 512)])
def test_a_wait_limit_of_nothing(M, N, K):
    """With a limit of nothing a wait that is not soon satisfied gives up: the call
    ends, either with its result or with a status that says so, and the next call is
    right."""
    ops = sv.TargetOps()
    g = gen(M)
    x, w = randn(g, (M, K), torch.bfloat16), randn(g, (N, K), torch.bfloat16)
    for call in (lambda: ops.linear(x, w), lambda: ops.gated_linear(x, w, w)):
        want = call()
        assert ops.status() == sv.SV_OK
        ops.set_wait_limit(0)
        for _ in range(10):
            got = call()
            code = ops.status()
            assert code == sv.SV_ERR_TIMEOUT or (code == sv.SV_OK and torch.equal(got, want))
        ops.set_wait_limit(10 ** 9)
        assert torch.equal(call(), want)
        assert ops.status() == sv.SV_OK
    ops.close()


def some_rows(n):
    return torch.tensor([0, 1, n // 2, n - 2, n - 1], device="cuda")


def test_products_past_32_bits_of_elements(ops):
    """An output of more than 2^31 elements, and rows 2^31 elements apart."""
    g = gen(1)
    M, N, K = 140001, 16384, 64

    def whole(*shape):
        return torch.randint(-2, 3, shape, generator=g, device="cuda").bfloat16()
    x, w, r = whole(M, K), whole(N, K), some_rows(M)
    out = ops.linear(x, w)
    want = x[r].double() @ w.double().t()
    assert torch.equal(out[r], want.bfloat16())
    ops.gated_linear(x, w, w, activation="none", out=out)
    assert torch.equal(out[r], (want * want).float().bfloat16())
    del out
    far = torch.zeros(2, (1 << 31) + 64, dtype=torch.bfloat16, device="cuda")[:, :64]
    ops.linear(x[:2], w[:64], out=far)
    assert torch.equal(far, (x[:2].double() @ w[:64].double().t()).bfloat16())


def test_rows_past_32_bits_of_elements(ops):
    g = gen(2)
    R, V, bf = 17001, 128257, torch.bfloat16
    x = torch.empty(R, V, dtype=bf, device="cuda").normal_(0, 3, generator=g)
    t = torch.randint(0, V, (R, 1), generator=g, device="cuda", dtype=torch.int32)
    r = some_rows(R)
    got, want = ops.log_probs(x, t, 5), log_probs_ref(x[r], t[r], 5, 1.0)
    within(got[0][r], want[0], log_probs_error(want[0], V))
    assert torch.equal(got[2][r], want[2])
    del x
    far = torch.empty(2, (1 << 31) + 64, dtype=bf, device="cuda")[:, :64]
    far.normal_(generator=g)
    near, w = randn(g, (2, 64), bf), randn(g, (64,), bf)
    want, h, dout, dh = block_norm_ref(far, near, w, w)
    out, ho = ops.block_norm(far, near, w, w)
    within(out, want, rounded(want, dout, bf))
    within(ho, h, rounded(h, dh, bf))


def test_refused_before_anything_is_launched(ops):
    x, w = torch.ones(4, 64, device="cuda").bfloat16(), torch.ones(8, 64, device="cuda").bfloat16()
    r = torch.ones(4, 8, device="cuda").bfloat16()
    for bad in (lambda: ops.linear(x, w, residual=r.half()), lambda: ops.linear(x, w, bias=w[0]),
                lambda: ops.linear(x, w, out=r.t()), lambda: ops.linear(x, w.cpu()),
                lambda: ops.linear(x, w, residual=r, out_dtype=torch.float32),
                lambda: ops.block_norm(x, x, w[0], gate=torch.ones(3, 1, device="cuda").bfloat16()),
                lambda: ops.block_norm(x, x, w[0], gate=w[0].float()),
                lambda: ops.block_norm_fp8(x, x, w[0], group=64),
                lambda: ops.log_probs(x, top=65), lambda: ops.log_probs(r, top=9),
                lambda: ops.log_probs(x, torch.ones(4, 1, device="cuda")),
                lambda: ops.log_probs(x, out=[r])):
        with pytest.raises(ValueError):
            bad()
    for refused in (lambda: ops.linear(x[:1].expand(4, 64), w),
                    lambda: ops.log_probs(x, temperature=0.0),
                    lambda: ops.block_norm(x, x, w[0], eps=-1.0)):
        with pytest.raises(sv.SpecVerifyError):
            refused()
    assert ops.status() == sv.SV_OK
