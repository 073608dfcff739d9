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

from . import (SV_BF16, SV_ERR_ARG, SV_FP32, SpecVerifyError, _check, _stream_handle,
               load_library)

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


def _dtype_code(t, what):
    code = _CODES.get(t.dtype)
    if code is None:
        raise ValueError(f"{what}: bfloat16, float16 or float32 expected, got {t.dtype}")
    return code


def _need(ok, message):
    if not ok:
        raise ValueError(message)


def _on_gpu(what, *tensors):
    for t in tensors:
        if t is not None and not t.is_cuda:
            raise ValueError(f"{what}: tensors must be on the GPU")


def _row_stride(t, what):
    """Row stride of a 2-D tensor whose rows are dense."""
    if t.stride(1) != 1 and t.shape[1] != 1:
        raise ValueError(f"{what}: rows must be dense")
    return t.stride(0)


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
    for each stream."""

    def __init__(self, device=None):
        self.h = None
        self.device = torch.device("cuda" if device is None else device)
        self._lib = load_library()
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            _check(self._lib.spec_target_create(ctypes.byref(h)), "spec_target_create")
        self.h = h

    def status(self, stream=None) -> int:
        """Waits for the stream; the first device-side error since the last call."""
        return int(self._lib.spec_target_status(self._handle(), _stream_handle(stream)))

    def set_wait_limit(self, limit_ns: int) -> None:
        _check(self._lib.spec_target_set_wait_limit(self._handle(), int(limit_ns)),
               "spec_target_set_wait_limit")

    def close(self):
        if getattr(self, "h", None):
            self._lib.spec_target_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _handle(self):
        if not self.h:
            raise SpecVerifyError(SV_ERR_ARG, "closed handle")
        return self.h

    # ---- norm ---------------------------------------------------------------
    def _norm_args(self, x, weight, residual, residual_out):
        _need(x.dim() == 2 and weight.dim() == 1 and weight.shape[0] == x.shape[1],
              "rms_norm: x [rows, d] and weight [d]")
        _need(weight.dtype == x.dtype and weight.is_contiguous(),
              "rms_norm: weight must be dense and of x's type")
        xs, rs, ros = _row_stride(x, "x"), 0, 0
        if residual is not None:
            _need(residual.shape == x.shape and residual.dtype == x.dtype,
                  "rms_norm: residual must have x's shape and type")
            rs = _row_stride(residual, "residual")
            if residual_out is None:
                residual_out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        if residual_out is not None:
            _need(residual_out.shape == x.shape and residual_out.dtype == x.dtype,
                  "rms_norm: residual_out must have x's shape and type")
            ros = _row_stride(residual_out, "residual_out")
        return xs, rs, residual_out, ros

    def rms_norm(self, x, weight, eps=1e-6, residual=None, out=None, residual_out=None,
                 stream=None):
        """h = x + residual; out = h / sqrt(mean(h^2) + eps) * weight.  Returns
        [out], or [out, residual_out] (= h) with a residual."""
        code = _dtype_code(x, "rms_norm")
        xs, rs, residual_out, ros = self._norm_args(x, weight, residual, residual_out)
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        else:
            _need(out.shape == x.shape and out.dtype == x.dtype,
                  "rms_norm: out must have x's shape and type")
        rows, d = x.shape
        _on_gpu("rms_norm", x, weight, residual, out, residual_out)
        _check(self._lib.spec_target_rms_norm(
            self._handle(), x.data_ptr(), xs,
            None if residual is None else residual.data_ptr(), rs, weight.data_ptr(), eps, rows,
            d, code, out.data_ptr(), _row_stride(out, "out"),
            None if residual_out is None else residual_out.data_ptr(), ros,
            _stream_handle(stream)), "spec_target_rms_norm")
        return [out] if residual_out is None else [out, residual_out]

    def rms_norm_fp8(self, x, weight, eps=1e-6, residual=None, group=SV_SCALE_BLOCK, out=None,
                     scale=None, residual_out=None, stream=None):
        """The norm in E4M3: group 128, scales [rows, ceil(d/128)] for
        ``matmul_fp8``; group 0, scales [rows] for ``spec_verify_run_fp8``.
        Returns [out8, scale], and residual_out with a residual."""
        code = _dtype_code(x, "rms_norm_fp8")
        xs, rs, residual_out, ros = self._norm_args(x, weight, residual, residual_out)
        rows, d = x.shape
        want = (rows, -(-d // SV_SCALE_BLOCK)) if group else (rows,)
        if out is None:
            out = torch.empty((rows, d), dtype=torch.float8_e4m3fn, device=x.device)
        else:
            _need(out.shape == x.shape and out.element_size() == 1 and out.is_contiguous(),
                  "rms_norm_fp8: out must be dense bytes of x's shape")
        if scale is None:
            scale = torch.empty(want, dtype=torch.float32, device=x.device)
        else:
            _need(tuple(scale.shape) == want and scale.dtype == torch.float32
                  and scale.is_contiguous(), f"rms_norm_fp8: scale must be float32 {want}")
        _on_gpu("rms_norm_fp8", x, weight, residual, out, scale, residual_out)
        _check(self._lib.spec_target_rms_norm_fp8(
            self._handle(), x.data_ptr(), xs,
            None if residual is None else residual.data_ptr(), rs, weight.data_ptr(), eps, rows,
            d, code, group, out.data_ptr(), scale.data_ptr(),
            None if residual_out is None else residual_out.data_ptr(), ros,
            _stream_handle(stream)), "spec_target_rms_norm_fp8")
        return [out, scale] if residual_out is None else [out, scale, residual_out]

    # ---- 8-bit product --------------------------------------------------------
    def matmul_fp8(self, a8, a_scale, w8, w_scale, out_dtype=torch.bfloat16, out=None,
                   stream=None):
        """a8 [M, K] and w8 [N, K] in E4M3 with scales [M, ceil(K/128)] and
        [ceil(N/128), ceil(K/128)]: the [M, N] product a8 w8^T."""
        M, K = a8.shape
        N = w8.shape[0]
        kb = -(-K // SV_SCALE_BLOCK)
        _need(w8.dim() == 2 and w8.shape[1] == K, "matmul_fp8: a8 [M, K] and w8 [N, K]")
        _need(a8.element_size() == 1 and w8.element_size() == 1,
              "matmul_fp8: a8 and w8 hold E4M3 bytes")
        _need(tuple(a_scale.shape) == (M, kb)
              and tuple(w_scale.shape) == (-(-N // SV_SCALE_BLOCK), kb)
              and a_scale.dtype == torch.float32 and w_scale.dtype == torch.float32,
              "matmul_fp8: float32 scales [M, ceil(K/128)] and [ceil(N/128), ceil(K/128)]")
        _need(a8.is_contiguous() and w8.is_contiguous() and a_scale.is_contiguous()
              and w_scale.is_contiguous(), "tensors must be contiguous")
        if out is None:
            out = torch.empty((M, N), dtype=out_dtype, device=a8.device)
        else:
            _need(tuple(out.shape) == (M, N), "matmul_fp8: out must be [M, N]")
        _on_gpu("matmul_fp8", a8, a_scale, w8, w_scale, out)
        _check(self._lib.spec_target_matmul_fp8(
            self._handle(), a8.data_ptr(), a_scale.data_ptr(), w8.data_ptr(),
            w_scale.data_ptr(), M, N, K, _dtype_code(out, "matmul_fp8"), out.data_ptr(),
            _row_stride(out, "out"), _stream_handle(stream)), "spec_target_matmul_fp8")
        return out

    # ---- rotary positions and append --------------------------------------------
    def rope_append(self, q, k, v, positions, slots, freqs, k_cache, v_cache, interleaved=False,
                    magnitude=1.0, q_out=None, stream=None):
        """Rotates q [T, Hq, D] and k [T, Hkv, D] by their int64 positions and
        writes k and v to their int64 slots (page * page_size + offset; -1:
        none) of the caches [pages, page_size, Hkv, D].  ``freqs``: float64
        [rot_dim/2] on the GPU.  Returns the rotated q."""
        T, Hq, D = q.shape
        Hkv = k.shape[1]
        pages, page_size = k_cache.shape[0], k_cache.shape[1]
        _need(tuple(k.shape) == (T, Hkv, D) and v.shape == k.shape,
              "rope_append: q [T, Hq, D], k and v [T, Hkv, D]")
        _need(tuple(k_cache.shape) == (pages, page_size, Hkv, D)
              and v_cache.shape == k_cache.shape,
              "rope_append: caches must be [pages, page_size, Hkv, D]")
        dt = q.dtype
        _need(k.dtype == dt and v.dtype == dt and k_cache.dtype == dt and v_cache.dtype == dt,
              "rope_append: q, k, v and the caches must have one type")
        _need(positions.dtype == torch.int64 and slots.dtype == torch.int64
              and positions.numel() == T and slots.numel() == T and positions.is_contiguous()
              and slots.is_contiguous(), "rope_append: positions and slots are int64 [T]")
        _need(freqs.dtype == torch.float64 and freqs.is_contiguous(),
              "rope_append: freqs is float64 [rot_dim/2]")
        if q_out is None:
            q_out = torch.empty((T, Hq, D), dtype=dt, device=q.device)
        else:
            _need(q_out.shape == q.shape and q_out.dtype == dt,
                  "rope_append: q_out must have q's shape and type")
        s = (q.stride(), k.stride(), v.stride(), q_out.stride(), k_cache.stride(),
             v_cache.stride())
        _need(D == 1 or all(x[-1] == 1 for x in s), "rope_append: heads must be dense")
        _on_gpu("rope_append", q, k, v, positions, slots, freqs, k_cache, v_cache, q_out)
        arg = _ROPE.pack(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), s[0][0], s[0][1], s[1][0], s[1][1],
            s[2][0], s[2][1], positions.data_ptr(), slots.data_ptr(), freqs.data_ptr(),
            q_out.data_ptr(), s[3][0], s[3][1], k_cache.data_ptr(), v_cache.data_ptr(),
            s[4][0], s[4][1], s[4][2], s[5][0], s[5][1], s[5][2], pages, page_size, T, Hq, Hkv,
            D, 2 * freqs.numel(), 1 if interleaved else 0, _dtype_code(q, "rope_append"),
            magnitude, 0)
        _check(self._lib.spec_target_rope_append(self._handle(), arg, _stream_handle(stream)),
               "spec_target_rope_append")
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
        pages, page_size, Hkv, Dk = k_cache.shape
        B, max_pages = page_table.shape
        dt = q.dtype
        _need(Dk == D and v_cache.shape == k_cache.shape,
              "attention: caches must be [pages, page_size, Hkv, D]")
        _need(k_cache.dtype == dt and v_cache.dtype == dt,
              "attention: q and the caches must have one type")
        _need(page_table.dtype == torch.int32 and q_start.dtype == torch.int32
              and kv_len.dtype == torch.int32 and q_start.numel() == B + 1
              and kv_len.numel() == B and q_start.is_contiguous() and kv_len.is_contiguous(),
              "attention: int32 page_table [B, max_pages], q_start [B+1], kv_len [B]")
        words, tree = 0, None
        if tree_mask is not None:
            _need(tree_mask.dim() == 2 and tree_mask.shape[0] == T
                  and tree_mask.dtype == torch.int32 and tree_mask.is_contiguous(),
                  "attention: tree_mask must be int32 [T, words]")
            words, tree = tree_mask.shape[1], tree_mask.data_ptr()
        if out is None:
            out = torch.empty((T, Hq, D), dtype=dt, device=q.device)
        else:
            _need(out.shape == q.shape and out.dtype == dt,
                  "attention: out must have q's shape and type")
        if lse is not None:
            _need(tuple(lse.shape) == (T, Hq) and lse.dtype == torch.float32
                  and lse.is_contiguous(), "attention: lse must be float32 [T, Hq]")
        s = (q.stride(), out.stride(), k_cache.stride(), v_cache.stride())
        _need(D == 1 or all(x[-1] == 1 for x in s), "attention: heads must be dense")
        if scale is None:
            scale = 1.0 / math.sqrt(D)
        _on_gpu("attention", q, k_cache, v_cache, page_table, q_start, kv_len, tree_mask, out,
                lse)
        arg = _ATTN.pack(
            q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(),
            q_start.data_ptr(), kv_len.data_ptr(), tree or 0, out.data_ptr(),
            0 if lse is None else lse.data_ptr(), s[0][0], s[0][1], s[1][0], s[1][1], s[2][0],
            s[2][1], s[2][2], s[3][0], s[3][1], s[3][2], _row_stride(page_table, "page_table"),
            pages, T, B, Hq, Hkv, D, page_size, max_pages, words, window,
            _dtype_code(q, "attention"), scale, 0)
        _check(self._lib.spec_target_attention(self._handle(), arg, _stream_handle(stream)),
               "spec_target_attention")
        return out

    def tree_mask(self, tree_parents, out=None, stream=None):
        """The attention's mask for draft trees: int32 parents [B, N] as
        ``spec_verify_tree_greedy`` takes them; returns int32
        [B * (N + 1), ceil((N + 1) / 32)], row 0 of a sequence its root."""
        B, N = tree_parents.shape
        _need(tree_parents.dtype == torch.int32 and tree_parents.is_contiguous(),
              "tree_mask: parents must be int32 [B, N]")
        shape = (B * (N + 1), (N + 32) // 32)
        if out is None:
            out = torch.empty(shape, dtype=torch.int32, device=tree_parents.device)
        else:
            _need(tuple(out.shape) == shape and out.dtype == torch.int32
                  and out.is_contiguous(), f"tree_mask: out must be int32 {shape}")
        _on_gpu("tree_mask", tree_parents, out)
        _check(self._lib.spec_target_tree_mask(self._handle(), tree_parents.data_ptr(), B, N,
                                               out.data_ptr(), _stream_handle(stream)),
               "spec_target_tree_mask")
        return out
