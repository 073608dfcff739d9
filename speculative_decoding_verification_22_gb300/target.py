"""Python binding of the target-layer operators (``include/spec_target.h``).

``TargetOps`` owns one handle; its methods take torch tensors on the GPU,
check shapes and types (``ValueError``), and enqueue the C entry point of the
same name on the current CUDA stream (or ``stream``).  Argument marshalling
only: every step runs in the CUDA kernels.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import SV_BF16, SV_ERR_ARG, SV_FP32, SpecVerifyError, _check, load_library

SV_FP16 = 3
SV_SCALE_BLOCK = 128
SV_MAX_HEAD_DIM = 256
ROPE_SCALINGS = ("plain", "linear", "ntk", "banded", "yarn")

_CODES = {torch.bfloat16: SV_BF16, torch.float32: SV_FP32, torch.float16: SV_FP16}

# field order of sv_rope_append_t and sv_attention_t
_ROPE = struct.Struct("@3P6q3P1P2q2P6q1q8i1f1i")
_ATTN = struct.Struct("@8P1P4q6q1q1q10i1f1i")


class sv_rope_t(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("scaling", ctypes.c_int32)] + [
        (n, ctypes.c_double) for n in ("base", "factor", "original_len", "low", "high",
                                       "beta_fast", "beta_slow")]


# The checks below are written out in each method and keep to few attribute
# reads: a call on a few tokens costs the GPU 2 to 10 us, so the host's share
# is what such a caller waits for.
def _need(ok, message):
    if not ok:
        raise ValueError(message)


def _row_stride(t, what):
    """Row stride of a 2-D tensor whose rows are dense."""
    rows, inner = t.stride()
    if inner != 1 and t.shape[1] != 1:
        raise ValueError(f"{what}: rows must be dense")
    return rows


def spec_target_rope_freqs(rot_dim, base=10000.0, scaling="plain", factor=1.0,
                           original_len=8192, low=1.0, high=4.0, beta_fast=32.0,
                           beta_slow=1.0):
    """Turns per position of each rotated pair (float64, on the host) and the
    magnitude of the rotation, for a scaling of ``ROPE_SCALINGS``."""
    _need(scaling in ROPE_SCALINGS, f"unknown scaling {scaling!r}")
    cfg = sv_rope_t(int(rot_dim), ROPE_SCALINGS.index(scaling), float(base), float(factor),
                    float(original_len), float(low), float(high), float(beta_fast),
                    float(beta_slow))
    out = torch.empty(max(int(rot_dim) // 2, 1), dtype=torch.float64)
    m = ctypes.c_double()
    _check(load_library().spec_target_rope_freqs(ctypes.byref(cfg), out.data_ptr(),
                                                 ctypes.byref(m)), "spec_target_rope_freqs")
    return out, m.value


class TargetOps:
    """One handle of the target-layer operators.  Calls on one handle that may
    overlap on the GPU (different streams) race on its scratch: use a handle
    for each stream.  Calls go to the current stream of the handle's device,
    or to ``stream``."""

    def __init__(self, device=None):
        self.h = None
        self.device = torch.device("cuda" if device is None else device)
        self._lib = lib = load_library()
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            self._index = torch.cuda.current_device()
            _check(lib.spec_target_create(ctypes.byref(h)), "spec_target_create")
        self.h = h
        self._raw = h.value

    def _stream(self, stream):
        if stream is None:
            return torch._C._cuda_getCurrentRawStream(self._index)
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)

    def status(self, stream=None) -> int:
        """Waits for the stream; the first device-side error since the last call."""
        return int(self._lib.spec_target_status(self._handle(), self._stream(stream)))

    def set_wait_limit(self, limit_ns: int) -> None:
        _check(self._lib.spec_target_set_wait_limit(self._handle(), int(limit_ns)),
               "spec_target_set_wait_limit")

    def close(self):
        if getattr(self, "h", None):
            self._lib.spec_target_destroy(self.h)
            self.h = self._raw = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _handle(self):
        if not self.h:
            raise SpecVerifyError(SV_ERR_ARG, "closed handle")
        return self._raw

    # ---- norm ---------------------------------------------------------------
    def rms_norm(self, x, weight, eps=1e-6, residual=None, out=None, residual_out=None,
                 stream=None):
        """h = x + residual; out = h / sqrt(mean(h^2) + eps) * weight.  Returns
        [out], or [out, residual_out] (= h) with a residual."""
        return self._norm(x, weight, eps, residual, None, out, None, residual_out, stream)

    def rms_norm_fp8(self, x, weight, eps=1e-6, residual=None, group=SV_SCALE_BLOCK, out=None,
                     scale=None, residual_out=None, stream=None):
        """The norm in E4M3: group 128, scales [rows, ceil(d/128)] for
        ``matmul_fp8``; group 0, scales [rows] for ``spec_verify_run_fp8``.
        Returns [out8, scale], and residual_out with a residual."""
        return self._norm(x, weight, eps, residual, int(group), out, scale, residual_out, stream)

    def _norm(self, x, weight, eps, residual, group, out, scale, residual_out, stream):
        shape, dt = x.shape, x.dtype
        code = _CODES.get(dt)
        if code is None:
            raise ValueError(f"rms_norm: bfloat16, float16 or float32 expected, got {dt}")
        if len(shape) != 2 or weight.shape != shape[1:]:
            raise ValueError("rms_norm: x [rows, d] and weight [d]")
        if weight.dtype != dt or not weight.is_contiguous():
            raise ValueError("rms_norm: weight must be dense and of x's type")
        if not (x.is_cuda and weight.is_cuda):
            raise ValueError("rms_norm: tensors must be on the GPU")
        rows, d = shape
        xs, res, rs, ro, ros = _row_stride(x, "x"), None, 0, None, 0
        if residual is not None:
            if residual.shape != shape or residual.dtype != dt or not residual.is_cuda:
                raise ValueError("rms_norm: residual must have x's shape and type")
            res, rs = residual.data_ptr(), _row_stride(residual, "residual")
            if residual_out is None:
                residual_out = torch.empty(shape, dtype=dt, device=x.device)
                ro, ros = residual_out.data_ptr(), d
        if residual_out is not None and ro is None:
            if residual_out.shape != shape or residual_out.dtype != dt or not residual_out.is_cuda:
                raise ValueError("rms_norm: residual_out must have x's shape and type")
            ro, ros = residual_out.data_ptr(), _row_stride(residual_out, "residual_out")
        if group is None:
            if out is None:
                out, os = torch.empty(shape, dtype=dt, device=x.device), d
            elif out.shape != shape or out.dtype != dt or not out.is_cuda:
                raise ValueError("rms_norm: out must have x's shape and type")
            else:
                os = _row_stride(out, "out")
            code = self._lib.spec_target_rms_norm(
                self._handle(), x.data_ptr(), xs, res, rs, weight.data_ptr(), eps, rows, d, code,
                out.data_ptr(), os, ro, ros, self._stream(stream))
            got = [out]
        else:
            want = (rows, -(-d // SV_SCALE_BLOCK)) if group else (rows,)
            if out is None:
                out = torch.empty(shape, dtype=torch.float8_e4m3fn, device=x.device)
            elif (out.shape != shape or out.element_size() != 1 or not out.is_contiguous()
                  or not out.is_cuda):
                raise ValueError("rms_norm_fp8: out must be dense bytes of x's shape")
            if scale is None:
                scale = torch.empty(want, dtype=torch.float32, device=x.device)
            elif (scale.shape != want or scale.dtype != torch.float32
                  or not scale.is_contiguous() or not scale.is_cuda):
                raise ValueError(f"rms_norm_fp8: scale must be float32 {want}")
            code = self._lib.spec_target_rms_norm_fp8(
                self._handle(), x.data_ptr(), xs, res, rs, weight.data_ptr(), eps, rows, d, code,
                group, out.data_ptr(), scale.data_ptr(), ro, ros, self._stream(stream))
            got = [out, scale]
        if code:
            raise SpecVerifyError(code, "spec_target_rms_norm")
        if residual_out is not None:
            got.append(residual_out)
        return got

    # ---- 8-bit product --------------------------------------------------------
    def matmul_fp8(self, a8, a_scale, w8, w_scale, out_dtype=torch.bfloat16, out=None,
                   stream=None):
        """a8 [M, K] and w8 [N, K] in E4M3 with scales [M, ceil(K/128)] and
        [ceil(N/128), ceil(K/128)]: the [M, N] product a8 w8^T."""
        M, K = a8.shape
        N, Kw = w8.shape
        kb = -(-K // SV_SCALE_BLOCK)
        if Kw != K:
            raise ValueError("matmul_fp8: a8 [M, K] and w8 [N, K]")
        if a8.element_size() != 1 or w8.element_size() != 1:
            raise ValueError("matmul_fp8: a8 and w8 hold E4M3 bytes")
        f32 = torch.float32
        if (a_scale.shape != (M, kb) or w_scale.shape != (-(-N // SV_SCALE_BLOCK), kb)
                or a_scale.dtype != f32 or w_scale.dtype != f32):
            raise ValueError("matmul_fp8: float32 scales [M, ceil(K/128)] and "
                             "[ceil(N/128), ceil(K/128)]")
        if not (a8.is_contiguous() and w8.is_contiguous() and a_scale.is_contiguous()
                and w_scale.is_contiguous()):
            raise ValueError("tensors must be contiguous")
        if not (a8.is_cuda and w8.is_cuda and a_scale.is_cuda and w_scale.is_cuda):
            raise ValueError("matmul_fp8: tensors must be on the GPU")
        if out is None:
            out, os = torch.empty((M, N), dtype=out_dtype, device=a8.device), N
        elif out.shape != (M, N) or not out.is_cuda:
            raise ValueError("matmul_fp8: out must be [M, N] on the GPU")
        else:
            os = _row_stride(out, "out")
        code = _CODES.get(out.dtype)
        if code is None:
            raise ValueError("matmul_fp8: out must be bfloat16, float16 or float32")
        code = self._lib.spec_target_matmul_fp8(
            self._handle(), a8.data_ptr(), a_scale.data_ptr(), w8.data_ptr(), w_scale.data_ptr(),
            M, N, K, code, out.data_ptr(), os, self._stream(stream))
        if code:
            raise SpecVerifyError(code, "spec_target_matmul_fp8")
        return out

    # ---- rotary positions and append --------------------------------------------
    def rope_append(self, q, k, v, positions, slots, freqs, k_cache, v_cache, interleaved=False,
                    magnitude=1.0, q_out=None, stream=None):
        """Rotates q [T, Hq, D] and k [T, Hkv, D] by their int64 positions and
        writes k and v to their int64 slots (page * page_size + offset; -1:
        none) of the caches [pages, page_size, Hkv, D].  ``freqs``: float64
        [rot_dim/2] on the GPU.  Returns the rotated q."""
        T, Hq, D = q.shape
        ks, cs, dt = k.shape, k_cache.shape, q.dtype
        pages, page_size = cs[0], cs[1]
        Hkv = ks[1]
        if ks != (T, Hkv, D) or v.shape != ks:
            raise ValueError("rope_append: q [T, Hq, D], k and v [T, Hkv, D]")
        if cs != (pages, page_size, Hkv, D) or v_cache.shape != cs:
            raise ValueError("rope_append: caches must be [pages, page_size, Hkv, D]")
        code = _CODES.get(dt)
        if (code is None or k.dtype != dt or v.dtype != dt or k_cache.dtype != dt
                or v_cache.dtype != dt):
            raise ValueError("rope_append: q, k, v and the caches must have one type of "
                             "bfloat16, float16, float32")
        i64 = torch.int64
        if (positions.dtype != i64 or slots.dtype != i64 or positions.numel() != T
                or slots.numel() != T or not positions.is_contiguous()
                or not slots.is_contiguous()):
            raise ValueError("rope_append: positions and slots are int64 [T]")
        if freqs.dtype != torch.float64 or not freqs.is_contiguous():
            raise ValueError("rope_append: freqs is float64 [rot_dim/2]")
        if not (q.is_cuda and k.is_cuda and v.is_cuda and positions.is_cuda and slots.is_cuda
                and freqs.is_cuda and k_cache.is_cuda and v_cache.is_cuda):
            raise ValueError("rope_append: tensors must be on the GPU")
        if q_out is None:
            q_out, qos = torch.empty((T, Hq, D), dtype=dt, device=q.device), (Hq * D, D, 1)
        elif q_out.shape != q.shape or q_out.dtype != dt or not q_out.is_cuda:
            raise ValueError("rope_append: q_out must have q's shape and type")
        else:
            qos = q_out.stride()
        q0, q1, q2 = q.stride()
        k0, k1, k2 = k.stride()
        v0, v1, v2 = v.stride()
        a0, a1, a2, a3 = k_cache.stride()
        b0, b1, b2, b3 = v_cache.stride()
        if D != 1 and not (q2 == k2 == v2 == a3 == b3 == qos[2] == 1):
            raise ValueError("rope_append: heads must be dense")
        code = self._lib.spec_target_rope_append(self._handle(), _ROPE.pack(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), q0, q1, k0, k1, v0, v1,
            positions.data_ptr(), slots.data_ptr(), freqs.data_ptr(), q_out.data_ptr(), qos[0],
            qos[1], k_cache.data_ptr(), v_cache.data_ptr(), a0, a1, a2, b0, b1, b2, pages,
            page_size, T, Hq, Hkv, D, 2 * freqs.numel(), 1 if interleaved else 0, code,
            magnitude, 0), self._stream(stream))
        if code:
            raise SpecVerifyError(code, "spec_target_rope_append")
        return q_out

    # ---- attention ----------------------------------------------------------------
    def attention(self, q, k_cache, v_cache, page_table, q_start, kv_len, scale=None, window=0,
                  tree_mask=None, out=None, lse=None, stream=None):
        """Attention of the new tokens q [T, Hq, D] over their sequences' pages:
        int32 page_table [B, max_pages], q_start [B+1], kv_len [B] (the new
        tokens are the last of the cached ones), optionally a window or a tree
        mask (int32 [T, words]).  ``lse``: float32 [T, Hq] to be filled.
        Returns out [T, Hq, D]."""
        T, Hq, D = q.shape
        pages, page_size, Hkv, Dk = cs = k_cache.shape
        B, max_pages = page_table.shape
        dt, i32 = q.dtype, torch.int32
        if Dk != D or v_cache.shape != cs:
            raise ValueError("attention: caches must be [pages, page_size, Hkv, D]")
        code = _CODES.get(dt)
        if code is None or k_cache.dtype != dt or v_cache.dtype != dt:
            raise ValueError("attention: q and the caches must have one type of bfloat16, "
                             "float16, float32")
        if (page_table.dtype != i32 or q_start.dtype != i32 or kv_len.dtype != i32
                or q_start.numel() != B + 1 or kv_len.numel() != B
                or not q_start.is_contiguous() or not kv_len.is_contiguous()):
            raise ValueError("attention: int32 page_table [B, max_pages], q_start [B+1], "
                             "kv_len [B]")
        if not (q.is_cuda and k_cache.is_cuda and v_cache.is_cuda and page_table.is_cuda
                and q_start.is_cuda and kv_len.is_cuda):
            raise ValueError("attention: tensors must be on the GPU")
        words = tree = lse_at = 0
        if tree_mask is not None:
            if (tree_mask.dim() != 2 or tree_mask.shape[0] != T or tree_mask.dtype != i32
                    or not tree_mask.is_contiguous() or not tree_mask.is_cuda):
                raise ValueError("attention: tree_mask must be int32 [T, words]")
            words, tree = tree_mask.shape[1], tree_mask.data_ptr()
        if out is None:
            out, os = torch.empty((T, Hq, D), dtype=dt, device=q.device), (Hq * D, D, 1)
        elif out.shape != q.shape or out.dtype != dt or not out.is_cuda:
            raise ValueError("attention: out must have q's shape and type")
        else:
            os = out.stride()
        if lse is not None:
            if (lse.shape != (T, Hq) or lse.dtype != torch.float32 or not lse.is_contiguous()
                    or not lse.is_cuda):
                raise ValueError("attention: lse must be float32 [T, Hq]")
            lse_at = lse.data_ptr()
        q0, q1, q2 = q.stride()
        a0, a1, a2, a3 = k_cache.stride()
        b0, b1, b2, b3 = v_cache.stride()
        if D != 1 and not (q2 == a3 == b3 == os[2] == 1):
            raise ValueError("attention: heads must be dense")
        if scale is None:
            scale = 1.0 / math.sqrt(D)
        code = self._lib.spec_target_attention(self._handle(), _ATTN.pack(
            q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(),
            q_start.data_ptr(), kv_len.data_ptr(), tree, out.data_ptr(), lse_at, q0, q1, os[0],
            os[1], a0, a1, a2, b0, b1, b2, _row_stride(page_table, "page_table"), pages, T, B,
            Hq, Hkv, D, page_size, max_pages, words, window, code, scale, 0),
            self._stream(stream))
        if code:
            raise SpecVerifyError(code, "spec_target_attention")
        return out

    def tree_mask(self, tree_parents, out=None, stream=None):
        """The attention's mask for draft trees: int32 parents [B, N] as
        ``spec_verify_tree_greedy`` takes them; returns int32
        [B * (N + 1), ceil((N + 1) / 32)], row 0 of a sequence its root."""
        B, N = tree_parents.shape
        _need(tree_parents.dtype == torch.int32 and tree_parents.is_contiguous()
              and tree_parents.is_cuda, "tree_mask: parents must be int32 [B, N] on the GPU")
        shape = (B * (N + 1), (N + 32) // 32)
        if out is None:
            out = torch.empty(shape, dtype=torch.int32, device=tree_parents.device)
        else:
            _need(tuple(out.shape) == shape and out.dtype == torch.int32
                  and out.is_contiguous() and out.is_cuda,
                  f"tree_mask: out must be int32 {shape}")
        _check(self._lib.spec_target_tree_mask(self._handle(), tree_parents.data_ptr(), B, N,
                                               out.data_ptr(), self._stream(stream)),
               "spec_target_tree_mask")
        return out
