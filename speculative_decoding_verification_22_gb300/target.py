"""Python binding of the target-layer operators (``include/spec_target.h``).

``TargetOps`` owns one handle; its methods take torch tensors on the GPU,
check shapes and types (``ValueError``), and enqueue the C entry point of the
same name on the current CUDA stream (or ``stream``).  Argument marshalling
only, compiled (``csrc/sv_bind.cpp``) for the calls of a decode step: every
step of the operators runs in the CUDA kernels.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import SV_BF16, SV_ERR_ARG, SV_FP32, SpecVerifyError, _check, load_library

SV_FP16 = 3
SV_SCALE_BLOCK = 128
SV_MAX_HEAD_DIM = 256
ROPE_SCALINGS = ("plain", "linear", "ntk", "banded", "yarn")

_CODES = {torch.bfloat16: SV_BF16, torch.float32: SV_FP32, torch.float16: SV_FP16}

# sv_rope_append_t and sv_attention_t, for callers that fill them from Python
_ROPE = struct.Struct("@3P6q3P1P2q2P6q1q8i1f1i")
_ATTN = struct.Struct("@8P1P4q6q1q1q10i1f1i")


class sv_rope_t(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("scaling", ctypes.c_int32)] + [
        (n, ctypes.c_double) for n in ("base", "factor", "original_len", "low", "high",
                                       "beta_fast", "beta_slow")]


def _need(ok, message):
    if not ok:
        raise ValueError(message)


def _binding():
    """The compiled argument marshalling (raises if it was not built)."""
    try:
        from . import _target_bind
    except ImportError as e:
        raise RuntimeError("the target-layer binding is missing: build it with "
                           "__graft_entry__.build() (or python -m "
                           f"speculative_decoding_verification_22_gb300.build): {e}") from e
    _target_bind.set_error(SpecVerifyError)  # raised with (code, what)
    return _target_bind


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
        self.h = self._raw = None
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

    def _torch_stream(self, stream):
        """The given stream as torch's (None, which changes nothing, for none)."""
        if stream is None or isinstance(stream, torch.cuda.Stream):
            return stream
        raw = self._stream(stream)
        if raw == 0:
            return torch.cuda.default_stream(self._index)
        return torch.cuda.ExternalStream(raw, device=self._index)

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

    def _has(self, t):
        return t.is_cuda and t.get_device() == self._index

    def rms_norm(self, x, weight, eps=1e-6, residual=None, out=None, residual_out=None,
                 stream=None):
        """h = x + residual; out = h / sqrt(mean(h^2) + eps) * weight.  Returns
        [out], or [out, residual_out] (= h) with a residual."""
        return _bound.norm(self, x, weight, eps, residual, None, out, None, residual_out, stream)

    def rms_norm_fp8(self, x, weight, eps=1e-6, residual=None, group=SV_SCALE_BLOCK, out=None,
                     scale=None, residual_out=None, stream=None):
        """The norm in E4M3: group 128, scales [rows, ceil(d/128)] for
        ``matmul_fp8``; group 0, scales [rows] for ``spec_verify_run_fp8``.
        Returns [out8, scale], and residual_out with a residual."""
        return _bound.norm(self, x, weight, eps, residual, group, out, scale, residual_out,
                           stream)

    def matmul_fp8(self, a8, a_scale, w8, w_scale, out_dtype=torch.bfloat16, out=None,
                   stream=None):
        """a8 [M, K] and w8 [N, K] in E4M3 (float8_e4m3fn, or its bytes as uint8)
        with scales [M, ceil(K/128)] and [ceil(N/128), ceil(K/128)]: the [M, N]
        product a8 w8^T."""
        code = _CODES.get(out_dtype)
        if code is None:
            raise ValueError("matmul_fp8: out must be bfloat16, float16 or float32")
        return _bound.matmul(self, a8, a_scale, w8, w_scale, code, out, stream)

    def rope_append(self, q, k, v, positions, slots, freqs, k_cache, v_cache, interleaved=False,
                    magnitude=1.0, q_out=None, stream=None):
        """Rotates q [T, Hq, D] and k [T, Hkv, D] by their int64 positions and
        writes k and v to their int64 slots (page * page_size + offset; -1:
        none) of the caches [pages, page_size, Hkv, D].  ``freqs``: float64
        [rot_dim/2] on the GPU.  Returns the rotated q."""
        return _bound.rope(self, q, k, v, positions, slots, freqs, k_cache, v_cache, interleaved,
                           magnitude, q_out, stream)

    def attention(self, q, k_cache, v_cache, page_table, q_start, kv_len, scale=None, window=0,
                  tree_mask=None, out=None, lse=None, stream=None):
        """Attention of the new tokens q [T, Hq, D] over their sequences' pages:
        int32 page_table [B, max_pages], q_start [B+1], kv_len [B] (the new
        tokens are the last of the cached ones), optionally a window or a tree
        mask (int32 [T, words]).  ``lse``: float32 [T, Hq] to be filled.
        ``scale`` is 1 / sqrt(D) if not given.  Returns out [T, Hq, D]."""
        return _bound.attention(self, q, k_cache, v_cache, page_table, q_start, kv_len, scale,
                                window, tree_mask, out, lse, stream)

    def tree_mask(self, tree_parents, out=None, stream=None):
        """The attention's mask for draft trees: int32 parents [B, N] as
        ``spec_verify_tree_greedy`` takes them; returns int32
        [B * (N + 1), ceil((N + 1) / 32)], row 0 of a sequence its root."""
        B, N = tree_parents.shape
        _need(tree_parents.dtype == torch.int32 and tree_parents.is_contiguous()
              and self._has(tree_parents),
              "tree_mask: parents must be int32 [B, N] on the GPU of the handle")
        shape = (B * (N + 1), (N + 32) // 32)
        if out is None:
            # from the call's own stream, whose order its memory is reused in
            with torch.cuda.stream(self._torch_stream(stream)):
                out = torch.empty(shape, dtype=torch.int32, device=tree_parents.device)
        else:
            _need(tuple(out.shape) == shape and out.dtype == torch.int32
                  and out.is_contiguous() and self._has(out),
                  f"tree_mask: out must be int32 {shape} on the GPU of the handle")
        _check(self._lib.spec_target_tree_mask(self._handle(), tree_parents.data_ptr(), B, N,
                                               out.data_ptr(), self._stream(stream)),
               "spec_target_tree_mask")
        return out


class _Bound:
    """Loads the compiled binding at its first use."""

    def __getattr__(self, name):
        global _bound
        _bound = _binding()
        return getattr(_bound, name)


_bound = _Bound()
