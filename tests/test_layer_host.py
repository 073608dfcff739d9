"""CPU checks of the layer's second half: refusals before CUDA is touched."""
import ctypes

import pytest
import torch

import speculative_decoding_verification_22_gb300 as sv
from speculative_decoding_verification_22_gb300 import target

GOOD = 1 << 12  # aligned fake address: the checks never dereference
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_22_gb300 import build as b
    b.build()
    return sv.load_library()


def test_null_handles_and_structures_are_refused(lib):
    for name in ("linear", "gated_linear", "block_norm", "log_probs"):
        f = getattr(lib, f"spec_layer_{name}")
        assert f(None, GOOD, None) == sv.SV_ERR_ARG, name
        assert f(GOOD, None, None) == sv.SV_ERR_ARG, name


LINEAR = dict(x=GOOD, w=GOOD, bias=0, res=0, out=GOOD, xs=64, ws=64, rs=0, os=96, M=3, N=96, K=64,
              dtype=0, out_dtype=0, act=0, pad=0)


@pytest.mark.parametrize("change,want", [
    (dict(x=0), sv.SV_ERR_ARG), (dict(w=0), sv.SV_ERR_ARG), (dict(out=0), sv.SV_ERR_ARG),
    (dict(dtype=2), sv.SV_ERR_ARG), (dict(out_dtype=2), sv.SV_ERR_ARG),
    (dict(dtype=-1), sv.SV_ERR_ARG), (dict(act=5), sv.SV_ERR_ARG), (dict(act=-1), sv.SV_ERR_ARG),
    (dict(M=-1), sv.SV_ERR_SHAPE), (dict(N=0), sv.SV_ERR_SHAPE), (dict(K=0), sv.SV_ERR_SHAPE),
    (dict(M=(1 << 24) + 1), sv.SV_ERR_SHAPE), (dict(N=(1 << 24) + 1), sv.SV_ERR_SHAPE),
    (dict(K=(1 << 24) + 1), sv.SV_ERR_SHAPE), (dict(xs=63), sv.SV_ERR_SHAPE),
    (dict(ws=63), sv.SV_ERR_SHAPE), (dict(os=95), sv.SV_ERR_SHAPE),
    (dict(os=(1 << 36) + 1), sv.SV_ERR_SHAPE), (dict(res=GOOD, rs=95), sv.SV_ERR_SHAPE),
    (dict(x=GOOD + 1), sv.SV_ERR_ALIGN), (dict(bias=GOOD + 1), sv.SV_ERR_ALIGN),
    (dict(out=GOOD + 2, out_dtype=1), sv.SV_ERR_ALIGN),
    (dict(res=GOOD + 2, rs=96, out_dtype=1), sv.SV_ERR_ALIGN),
    (dict(M=0, x=0, w=0, out=0), sv.SV_OK),
])
def test_linear_refusals(lib, change, want):
    assert lib.spec_layer_linear(GOOD, target._LINEAR.pack(*(LINEAR | change).values()),
                                 None) == want


GATED = dict(x=GOOD, wg=GOOD, wu=GOOD, bg=0, bu=0, out=GOOD, xs=64, gs=64, us=64, os=96, M=3, N=96,
             K=64, dtype=0, out_dtype=0, act=4, pad=0)


@pytest.mark.parametrize("change,want", [
    (dict(x=0), sv.SV_ERR_ARG), (dict(wg=0), sv.SV_ERR_ARG), (dict(wu=0), sv.SV_ERR_ARG),
    (dict(out=0), sv.SV_ERR_ARG), (dict(dtype=2), sv.SV_ERR_ARG), (dict(act=5), sv.SV_ERR_ARG),
    (dict(M=-1), sv.SV_ERR_SHAPE), (dict(K=0), sv.SV_ERR_SHAPE), (dict(gs=63), sv.SV_ERR_SHAPE),
    (dict(us=63), sv.SV_ERR_SHAPE), (dict(os=95), sv.SV_ERR_SHAPE),
    (dict(wu=GOOD + 1), sv.SV_ERR_ALIGN), (dict(bu=GOOD + 1), sv.SV_ERR_ALIGN),
    (dict(M=0, x=0), sv.SV_OK),
])
def test_gated_linear_refusals(lib, change, want):
    assert lib.spec_layer_gated_linear(GOOD, target._GATED.pack(*(GATED | change).values()),
                                       None) == want


NORM = dict(x=GOOD, res=GOOD, post=0, gate=0, w=GOOD, out=GOOD, scale=0, ro=0, xs=64, rs=64, os=64,
            ros=64, gr=0, gc=1, rows=2, d=64, dtype=0, group=-1, eps=1e-6, s=1.0)


@pytest.mark.parametrize("change,want", [
    (dict(x=0), sv.SV_ERR_ARG), (dict(res=0), sv.SV_ERR_ARG), (dict(w=0), sv.SV_ERR_ARG),
    (dict(out=0), sv.SV_ERR_ARG), (dict(dtype=2), sv.SV_ERR_ARG), (dict(group=64), sv.SV_ERR_ARG),
    (dict(group=128), sv.SV_ERR_ARG),  # no scales
    (dict(eps=-1.0), sv.SV_ERR_ARG), (dict(eps=NAN), sv.SV_ERR_ARG), (dict(s=NAN), sv.SV_ERR_ARG),
    (dict(s=INF), sv.SV_ERR_ARG), (dict(rows=-1), sv.SV_ERR_ARG),
    (dict(gate=GOOD, gc=2), sv.SV_ERR_ARG), (dict(gate=GOOD, gr=-1), sv.SV_ERR_ARG),
    (dict(d=0), sv.SV_ERR_SHAPE), (dict(d=(1 << 20) + 1), sv.SV_ERR_SHAPE),
    (dict(xs=63), sv.SV_ERR_SHAPE), (dict(rs=63), sv.SV_ERR_SHAPE), (dict(os=63), sv.SV_ERR_SHAPE),
    (dict(ro=GOOD, ros=63), sv.SV_ERR_SHAPE), (dict(x=GOOD + 1), sv.SV_ERR_ALIGN),
    (dict(out=GOOD + 1), sv.SV_ERR_ALIGN), (dict(post=GOOD + 1), sv.SV_ERR_ALIGN),
    (dict(gate=GOOD + 1), sv.SV_ERR_ALIGN), (dict(group=0, scale=GOOD + 2), sv.SV_ERR_ALIGN),
    (dict(rows=0, x=0), sv.SV_OK),
])
def test_block_norm_refusals(lib, change, want):
    assert lib.spec_layer_block_norm(GOOD, target._BLOCK_NORM.pack(*(NORM | change).values()),
                                     None) == want


LOGP = dict(x=GOOD, t=GOOD, lp=GOOD, ent=GOOD, ids=GOOD, top_lp=GOOD, stride=100, rows=2, V=100,
            dtype=0, n=1, top=5, T=1.0)


@pytest.mark.parametrize("change,want", [
    (dict(x=0), sv.SV_ERR_ARG), (dict(t=0), sv.SV_ERR_ARG), (dict(lp=0), sv.SV_ERR_ARG),
    (dict(ids=0), sv.SV_ERR_ARG), (dict(top_lp=0), sv.SV_ERR_ARG), (dict(dtype=2), sv.SV_ERR_ARG),
    (dict(T=0.0), sv.SV_ERR_ARG), (dict(T=-1.0), sv.SV_ERR_ARG), (dict(T=NAN), sv.SV_ERR_ARG),
    (dict(T=INF), sv.SV_ERR_ARG), (dict(T=1e-40), sv.SV_ERR_ARG), (dict(n=-1), sv.SV_ERR_ARG),
    (dict(V=0), sv.SV_ERR_SHAPE), (dict(V=(1 << 24) + 1), sv.SV_ERR_SHAPE),
    (dict(top=65), sv.SV_ERR_SHAPE), (dict(top=-1), sv.SV_ERR_SHAPE),
    (dict(V=4, top=5), sv.SV_ERR_SHAPE), (dict(n=(1 << 16) + 1), sv.SV_ERR_SHAPE),
    (dict(rows=-1), sv.SV_ERR_SHAPE), (dict(rows=(1 << 24) + 1), sv.SV_ERR_SHAPE),
    (dict(stride=99), sv.SV_ERR_SHAPE), (dict(x=GOOD + 1), sv.SV_ERR_ALIGN),
    (dict(x=GOOD + 2, dtype=1), sv.SV_ERR_ALIGN), (dict(t=GOOD + 2), sv.SV_ERR_ALIGN),
    (dict(ent=GOOD + 2), sv.SV_ERR_ALIGN), (dict(rows=0, x=0), sv.SV_OK),
])
def test_log_probs_refusals(lib, change, want):
    assert lib.spec_layer_log_probs(GOOD, target._LOG_PROBS.pack(*(LOGP | change).values()),
                                    None) == want


def test_every_entry_point_is_bound(lib):
    names = [n for n in sv.EXPORTS if n.startswith("spec_layer_")]
    assert len(names) == 4
    for n in names:
        assert getattr(lib, n).argtypes is not None and getattr(lib, n).restype is ctypes.c_int


def test_the_binding_refuses_wrong_tensors():
    """Types, shapes and the device, before anything is called."""
    ops = sv.TargetOps.__new__(sv.TargetOps)  # no GPU, no handle
    ops.h, ops._lib = None, None
    x, w = torch.zeros(4, 64).bfloat16(), torch.zeros(96, 64).bfloat16()
    for bad in (lambda: ops.linear(x, w.half()), lambda: ops.linear(x, w[:, :32]),
                lambda: ops.linear(x.int(), w), lambda: ops.linear(x[0], w),
                lambda: ops.linear(x, w, activation="tanh"),
                lambda: ops.linear(x, w, out_dtype=torch.int32),
                lambda: ops.gated_linear(x, w, w[:95]), lambda: ops.gated_linear(x, w, w.half()),
                lambda: ops.log_probs(x[0]), lambda: ops.log_probs(x.int()),
                lambda: ops.block_norm(x[0], x, w[0])):
        with pytest.raises(ValueError):
            bad()
    for far in (lambda: ops.linear(x, w), lambda: ops.gated_linear(x, w, w),
                lambda: ops.log_probs(x), lambda: ops.block_norm(x, x, w[0])):
        with pytest.raises(ValueError, match="on the GPU"):
            far()


def test_verify_log_probs_refusals(lib):
    f = lib.spec_verify_log_probs
    assert f(None, GOOD, 1.0, 0, GOOD, GOOD, None, None) == sv.SV_ERR_ARG
    eng = sv.SpecVerify.__new__(sv.SpecVerify)  # no GPU, no handle
    eng.B, eng.K, eng.V, eng.h = 2, 3, 40, None
    for kw in (dict(tokens=torch.zeros(2, 3, dtype=torch.int32)),
               dict(tokens=torch.zeros(2, 4, dtype=torch.int64)),
               dict(tokens=torch.zeros(2, 4, dtype=torch.int32)),  # not on the GPU
               dict(top=65), dict(top=41), dict(top=-1)):
        with pytest.raises(ValueError):
            eng.log_probs(**kw)
