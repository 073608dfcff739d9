"""CPU checks of the target-layer operators: refusals before CUDA is touched,
and the rotary frequencies against their formulas."""
import ctypes
import math
import subprocess
import sys

import pytest
import torch

import speculative_decoding_verification_22_gb300 as sv
from speculative_decoding_verification_22_gb300 import target

GOOD = 1 << 12  # aligned fake address: the checks never dereference


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_22_gb300 import build as b
    b.build()
    return sv.load_library()


def test_null_handles_are_refused(lib):
    assert lib.spec_target_create(None) == sv.SV_ERR_ARG
    assert lib.spec_target_status(None, None) == sv.SV_ERR_ARG
    assert lib.spec_target_set_wait_limit(None, 1) == sv.SV_ERR_ARG
    assert lib.spec_target_rope_append(None, None, None) == sv.SV_ERR_ARG
    assert lib.spec_target_attention(GOOD, None, None) == sv.SV_ERR_ARG
    assert lib.spec_target_tree_mask(None, GOOD, 1, 1, GOOD, None) == sv.SV_ERR_ARG
    lib.spec_target_destroy(None)


@pytest.mark.parametrize("change,want", [
    (dict(h=None), sv.SV_ERR_ARG), (dict(x=None), sv.SV_ERR_ARG), (dict(w=None), sv.SV_ERR_ARG),
    (dict(out=None), sv.SV_ERR_ARG), (dict(dtype=2), sv.SV_ERR_ARG),
    (dict(eps=-1.0), sv.SV_ERR_ARG), (dict(eps=float("nan")), sv.SV_ERR_ARG),
    (dict(eps=float("inf")), sv.SV_ERR_ARG), (dict(rows=-1), sv.SV_ERR_ARG),
    (dict(d=0), sv.SV_ERR_SHAPE), (dict(d=(1 << 20) + 1), sv.SV_ERR_SHAPE),
    (dict(xs=63), sv.SV_ERR_SHAPE), (dict(res=GOOD, rs=63), sv.SV_ERR_SHAPE),
    (dict(ro=GOOD, ros=63), sv.SV_ERR_SHAPE), (dict(x=GOOD + 1), sv.SV_ERR_ALIGN),
    (dict(ro=GOOD + 1, ros=64), sv.SV_ERR_ALIGN),
])
def test_norm_refusals(lib, change, want):
    a = dict(h=GOOD, x=GOOD, xs=64, res=None, rs=0, w=GOOD, eps=1e-6, rows=2, d=64, dtype=0,
             out=GOOD, os=64, ro=None, ros=0) | change
    head = (a["h"], a["x"], a["xs"], a["res"], a["rs"], a["w"], a["eps"], a["rows"], a["d"],
            a["dtype"])
    assert lib.spec_target_rms_norm(*head, a["out"], a["os"], a["ro"], a["ros"], None) == want
    assert lib.spec_target_rms_norm_fp8(*head, 128, a["out"], GOOD, a["ro"], a["ros"],
                                        None) == want


def test_norm_fp8_refuses_another_group_and_a_missing_scale(lib):
    head = (GOOD, GOOD, 64, None, 0, GOOD, 1e-6, 2, 64, 0)
    assert lib.spec_target_rms_norm_fp8(*head, 64, GOOD, GOOD, None, 0, None) == sv.SV_ERR_ARG
    assert lib.spec_target_rms_norm_fp8(*head, 128, GOOD, None, None, 0, None) == sv.SV_ERR_ARG
    assert lib.spec_target_rms_norm_fp8(*head, 0, GOOD, GOOD + 2, None, 0,
                                        None) == sv.SV_ERR_ALIGN


@pytest.mark.parametrize("i,value,want", [
    (0, None, sv.SV_ERR_ARG), (1, None, sv.SV_ERR_ARG), (2, None, sv.SV_ERR_ARG),
    (3, None, sv.SV_ERR_ARG), (4, None, sv.SV_ERR_ARG), (9, None, sv.SV_ERR_ARG),
    (8, 2, sv.SV_ERR_ARG), (8, 9, sv.SV_ERR_ARG), (5, -1, sv.SV_ERR_SHAPE),
    (6, 0, sv.SV_ERR_SHAPE), (7, 0, sv.SV_ERR_SHAPE), (7, 136, sv.SV_ERR_SHAPE),
    (5, 1 << 25, sv.SV_ERR_SHAPE), (10, 127, sv.SV_ERR_SHAPE), (1, GOOD + 8, sv.SV_ERR_ALIGN),
    (3, GOOD + 8, sv.SV_ERR_ALIGN), (2, GOOD + 2, sv.SV_ERR_ALIGN), (9, GOOD + 1, sv.SV_ERR_ALIGN),
])
def test_matmul_refusals(lib, i, value, want):
    args = [GOOD, GOOD, GOOD, GOOD, GOOD, 4, 128, 256, 0, GOOD, 128, None]
    args[i] = value
    assert lib.spec_target_matmul_fp8(*args) == want


ROPE = dict(q=GOOD, k=GOOD, v=GOOD, qt=64, qh=64, kt=64, kh=64, vt=64, vh=64, pos=GOOD,
            slots=GOOD, freqs=GOOD, qo=GOOD, qot=64, qoh=64, kc=GOOD, vc=GOOD, a=1024, b=64, c=64,
            d=1024, e=64, f=64, pages=4, page=16, T=3, Hq=2, Hkv=1, D=64, rot=64, inter=0,
            dtype=0, mag=1.0, pad=0)


@pytest.mark.parametrize("change,want", [
    (dict(q=0), sv.SV_ERR_ARG), (dict(pos=0), sv.SV_ERR_ARG), (dict(slots=0), sv.SV_ERR_ARG),
    (dict(freqs=0), sv.SV_ERR_ARG), (dict(vc=0), sv.SV_ERR_ARG), (dict(dtype=2), sv.SV_ERR_ARG),
    (dict(mag=float("nan")), sv.SV_ERR_ARG), (dict(T=-1), sv.SV_ERR_SHAPE),
    (dict(D=257), sv.SV_ERR_SHAPE), (dict(rot=63), sv.SV_ERR_SHAPE),
    (dict(rot=66), sv.SV_ERR_SHAPE), (dict(page=0), sv.SV_ERR_SHAPE),
    (dict(pages=0), sv.SV_ERR_SHAPE), (dict(Hkv=0), sv.SV_ERR_SHAPE),
    (dict(k=GOOD + 1), sv.SV_ERR_ALIGN), (dict(slots=GOOD + 4), sv.SV_ERR_ALIGN),
])
def test_rope_refusals(lib, change, want):
    arg = target._ROPE.pack(*(ROPE | change).values())
    assert lib.spec_target_rope_append(GOOD, arg, None) == want


ATTN = dict(q=GOOD, k=GOOD, v=GOOD, table=GOOD, qs=GOOD, kl=GOOD, tree=0, out=GOOD, lse=0, qt=128,
            qh=64, ot=128, oh=64, a=1024, b=64, c=64, d=1024, e=64, f=64, ts=8, pages=9, T=3, B=2,
            Hq=2, Hkv=1, D=64, page=16, mp=8, words=0, window=0, dtype=0, scale=0.125, pad=0)


@pytest.mark.parametrize("change,want", [
    (dict(q=0), sv.SV_ERR_ARG), (dict(k=0), sv.SV_ERR_ARG), (dict(table=0), sv.SV_ERR_ARG),
    (dict(qs=0), sv.SV_ERR_ARG), (dict(kl=0), sv.SV_ERR_ARG), (dict(out=0), sv.SV_ERR_ARG),
    (dict(dtype=2), sv.SV_ERR_ARG), (dict(scale=float("inf")), sv.SV_ERR_ARG),
    (dict(window=-1), sv.SV_ERR_ARG), (dict(tree=GOOD, words=1, window=4), sv.SV_ERR_ARG),
    (dict(tree=GOOD, words=0), sv.SV_ERR_ARG), (dict(Hq=3, Hkv=2), sv.SV_ERR_ARG),
    (dict(T=-1), sv.SV_ERR_SHAPE), (dict(B=0), sv.SV_ERR_SHAPE), (dict(B=4097), sv.SV_ERR_SHAPE),
    (dict(D=0), sv.SV_ERR_SHAPE), (dict(D=257), sv.SV_ERR_SHAPE), (dict(page=0), sv.SV_ERR_SHAPE),
    (dict(mp=0), sv.SV_ERR_SHAPE), (dict(pages=0), sv.SV_ERR_SHAPE),
    (dict(mp=1 << 27, page=16), sv.SV_ERR_SHAPE), (dict(T=1 << 24, Hq=128), sv.SV_ERR_SHAPE),
    (dict(q=GOOD + 1), sv.SV_ERR_ALIGN), (dict(kl=GOOD + 2), sv.SV_ERR_ALIGN),
    (dict(lse=GOOD + 2), sv.SV_ERR_ALIGN),
])
def test_attention_refusals(lib, change, want):
    arg = target._ATTN.pack(*(ATTN | change).values())
    assert lib.spec_target_attention(GOOD, arg, None) == want


def test_tree_mask_refusals(lib):
    f = lib.spec_target_tree_mask
    assert f(GOOD, None, 1, 4, GOOD, None) == sv.SV_ERR_ARG
    assert f(GOOD, GOOD, 0, 4, GOOD, None) == sv.SV_ERR_ARG
    assert f(GOOD, GOOD, 1, 0, GOOD, None) == sv.SV_ERR_ARG
    assert f(GOOD, GOOD, 1, 65, GOOD, None) == sv.SV_ERR_ARG
    assert f(GOOD, GOOD + 2, 1, 4, GOOD, None) == sv.SV_ERR_ALIGN


def test_calls_without_rows_do_nothing(lib):
    assert lib.spec_target_rms_norm(GOOD, None, 64, None, 0, None, 1e-6, 0, 64, 0, None, 64, None,
                                    0, None) == sv.SV_OK
    assert lib.spec_target_matmul_fp8(GOOD, None, None, None, None, 0, 128, 128, 0, None, 128,
                                      None) == sv.SV_OK
    assert lib.spec_target_rope_append(GOOD, target._ROPE.pack(*(ROPE | dict(T=0)).values()),
                                       None) == sv.SV_OK
    assert lib.spec_target_attention(GOOD, target._ATTN.pack(*(ATTN | dict(T=0)).values()),
                                     None) == sv.SV_OK


def test_argument_structures_have_the_headers_sizes():
    assert target._ROPE.size == 232 and target._ATTN.size == 216


# ---- frequencies ---------------------------------------------------------------

def plain(rot, base):
    return [base ** (-2 * i / rot) / (2 * math.pi) for i in range(rot // 2)]


@pytest.mark.parametrize("rot", [2, 64, 96, 128, 256])
def test_plain_linear_and_ntk_frequencies(lib, rot):
    f0 = plain(rot, 10000.0)
    for kind, want in (("plain", f0), ("linear", [f / 4 for f in f0]),
                       ("ntk", plain(rot, 10000.0 * 4 ** (rot / (rot - 2))) if rot > 2 else f0)):
        f, m = sv.spec_target_rope_freqs(rot, 10000.0, kind, 4.0)
        assert m == 1.0
        assert f.tolist() == pytest.approx(want, rel=1e-14)
    # the slowest pair of ntk turns factor times slower
    if rot > 2:
        assert f[-1].item() == pytest.approx(f0[-1] / 4, rel=1e-12)


def test_banded_frequencies(lib):
    f0 = plain(128, 500000.0)
    f, m = sv.spec_target_rope_freqs(128, 500000.0, "banded", 8.0, 8192, low=1.0, high=4.0)
    assert m == 1.0
    kinds = set()
    for a, b in zip(f0, f.tolist()):
        wave = 1.0 / a
        if wave > 8192:
            kinds.add("slow")
            assert b == pytest.approx(a / 8, rel=1e-14)
        elif wave < 2048:
            kinds.add("fast")
            assert b == pytest.approx(a, rel=1e-14)
        else:
            kinds.add("between")
            s = (8192 / wave - 1.0) / 3.0
            assert b == pytest.approx((1 - s) * a / 8 + s * a, rel=1e-13)
    assert kinds == {"slow", "fast", "between"}


def test_yarn_frequencies(lib):
    f0 = plain(128, 10000.0)
    f, m = sv.spec_target_rope_freqs(128, 10000.0, "yarn", 4.0, 4096)
    assert m == pytest.approx(0.1 * math.log(4.0) + 1.0)
    ratio = [b / a for a, b in zip(f0, f.tolist())]
    # pairs that turn more than 32 times over the original length are kept,
    # those that turn less than once are stretched
    for a, r in zip(f0, ratio):
        if a * 4096 > 40:
            assert r == pytest.approx(1.0)
        if a * 4096 < 0.8:
            assert r == pytest.approx(0.25)
    assert all(x >= y - 1e-12 for x, y in zip(ratio, ratio[1:]))


@pytest.mark.parametrize("change,want", [
    (dict(rot_dim=63), sv.SV_ERR_SHAPE), (dict(rot_dim=0), sv.SV_ERR_SHAPE),
    (dict(rot_dim=258), sv.SV_ERR_SHAPE), (dict(base=1.0), sv.SV_ERR_ARG),
    (dict(scaling="linear", factor=0.5), sv.SV_ERR_ARG),
    (dict(scaling="banded", low=4.0, high=4.0), sv.SV_ERR_ARG),
    (dict(scaling="yarn", beta_fast=1.0, beta_slow=1.0), sv.SV_ERR_ARG),
    (dict(scaling="yarn", original_len=0), sv.SV_ERR_ARG),
])
def test_frequency_refusals(lib, change, want):
    with pytest.raises(sv.SpecVerifyError) as e:
        sv.spec_target_rope_freqs(**(dict(rot_dim=64) | change))
    assert e.value.code == want


def test_python_checks_come_before_the_call():
    ops = sv.TargetOps.__new__(sv.TargetOps)  # no GPU, no handle
    ops.h, ops._lib = None, None
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ops.rms_norm(x, w[:32])
    with pytest.raises(ValueError):
        ops.rms_norm(x, w.float())
    with pytest.raises(ValueError):
        ops.rms_norm(x.double(), w.double())
    with pytest.raises(ValueError):
        ops.rms_norm(x, w)                      # not on the GPU
    with pytest.raises(ValueError):
        ops.rms_norm(x.t().contiguous().t(), w)   # rows not dense
    a = torch.zeros(4, 256, dtype=torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        ops.matmul_fp8(a, torch.ones(4, 1), a, torch.ones(1, 2))
    with pytest.raises(ValueError):
        ops.attention(x.view(4, 1, 64), x.view(1, 4, 1, 64), x.view(1, 4, 1, 64).half(),
                      torch.zeros(1, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                      torch.zeros(1, dtype=torch.int32))
    q = x.view(4, 1, 64)
    pos = torch.arange(4)
    with pytest.raises(ValueError):
        ops.rope_append(q, q, q, pos.int(), pos, torch.zeros(32, dtype=torch.float64),
                        q.view(1, 4, 1, 64), q.view(1, 4, 1, 64))


def test_every_entry_point_is_bound(lib):
    names = [n for n in sv.EXPORTS if n.startswith("spec_target_")]
    assert len(names) == 11
    for n in names:
        f = getattr(lib, n)
        assert f.argtypes is not None, n
        assert f.restype in (ctypes.c_int, None), n


@pytest.mark.parametrize("dtype", [torch.float8_e5m2, torch.int8, torch.bool])
def test_eight_bits_that_are_not_e4m3_are_refused(dtype):
    ops = sv.TargetOps.__new__(sv.TargetOps)  # no GPU, no handle
    ops.h, ops._lib = None, None
    good, bad = (torch.zeros(128, 128).to(t) for t in (torch.float8_e4m3fn, dtype))
    s, one = torch.ones(128, 1), torch.ones(1, 1)
    for a, w in ((good, bad), (bad, good)):
        with pytest.raises(ValueError, match="must be float8_e4m3fn"):
            ops.matmul_fp8(a, s, w, one)
    for a in (good, good.view(torch.uint8)):  # these come to the check of the device
        with pytest.raises(ValueError, match="on the GPU"):
            ops.matmul_fp8(a, s, good, one)


# ---- build -----------------------------------------------------------------------

@pytest.fixture
def fake_build(monkeypatch, tmp_path):
    """The build with commands that only make their outputs; those whose compiler
    is in `broken` fail."""
    from speculative_decoding_verification_22_gb300 import build as b
    for name, path in (("BUILD", "objects"), ("LIB", "lib.so"), ("BIND", "bind.so")):
        monkeypatch.setattr(b, name, str(tmp_path / path))
    broken, ran = set(), []

    def run(cmd, **_):
        ran.append(cmd[0])
        if cmd[0] not in broken:
            open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, int(cmd[0] in broken), "", "")
    monkeypatch.setattr(b.subprocess, "run", run)
    return b, broken, ran, tmp_path


def test_the_library_is_built_where_the_binding_cannot_be(fake_build):
    b, broken, ran, path = fake_build
    broken.add("g++")
    with pytest.raises(RuntimeError, match="g\\+\\+"):
        b.build(force=True)
    assert (path / "lib.so").exists() and not (path / "bind.so").exists()
    broken.clear()
    assert b.build() == str(path / "lib.so") and (path / "bind.so").exists()


def test_a_broken_library_is_an_error_and_links_nothing(fake_build):
    b, broken, ran, path = fake_build
    broken.add(b._nvcc())
    with pytest.raises(RuntimeError, match="nvcc"):
        b.build(force=True)
    assert not (path / "lib.so").exists() and not (path / "bind.so").exists()


@pytest.mark.parametrize("torch_is", ["missing", "without CUDA"])
def test_without_a_torch_to_bind_to_the_library_alone_is_built(fake_build, monkeypatch, torch_is):
    b, broken, ran, path = fake_build
    if torch_is == "missing":
        monkeypatch.setitem(sys.modules, "torch", None)
    else:
        monkeypatch.setattr(torch.version, "cuda", None)
    assert b.build(force=True) == str(path / "lib.so")
    assert (path / "lib.so").exists() and "g++" not in ran
