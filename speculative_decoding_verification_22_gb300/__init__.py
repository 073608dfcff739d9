"""Python binding of the GB300 verify-and-sample library (libspec_verify.so).

Argument marshalling only: every step of the verify path runs in the CUDA
kernels behind the C ABI of ``include/spec_verify.h``; the functions here
carry the same names as the C entry points, take torch tensors (device
memory) and pass their pointers and the current CUDA stream through.
There is no fallback: if the library has not been built, importing the
entry points raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libspec_verify.so")

SV_OK = 0
SV_ERR_ARG = -1
SV_ERR_ALIGN = -2
SV_ERR_SHAPE = -3
SV_ERR_CUDA = -4
SV_ERR_ARCH = -5
SV_ERR_TIMEOUT = -6
SV_ERR_TOKEN = -7
SV_ERR_NONFINITE = -8
SV_ERR_CACHE = -9
SV_BF16 = 0
SV_FP32 = 1
SV_FP8 = 2
SV_MAX_K = 64
SV_MAX_B = 4096
SV_MAX_ROWS_BF16 = 384
SV_NGRAM_MAX = 16

# every symbol of include/spec_verify.h, include/spec_target.h and include/spec_layer.h
EXPORTS = ("spec_verify_create", "spec_verify_run", "spec_verify_run_host",
           "spec_verify_status", "spec_verify_set_stream",
           "spec_verify_debug_logits", "spec_verify_debug_lse",
           "spec_verify_set_wait_limit", "spec_verify_timing",
           "spec_verify_timing_read", "spec_verify_launches_per_run",
           "spec_verify_strerror", "spec_verify_destroy",
           "spec_verify_run_noalloc", "spec_ngram_draft", "spec_verify_run_truncated",
           "spec_verify_tree_greedy", "spec_verify_run_fp8", "spec_verify_plan",
           "spec_verify_debug_stall", "spec_verify_submit_host", "spec_verify_wait_host",
           "spec_verify_log_probs", "spec_verify_stream",
           "spec_target_create", "spec_target_destroy", "spec_target_status",
           "spec_target_set_wait_limit", "spec_target_rms_norm", "spec_target_rms_norm_fp8",
           "spec_target_matmul_fp8", "spec_target_rope_freqs", "spec_target_rope_append",
           "spec_target_attention", "spec_target_tree_mask", "spec_layer_linear",
           "spec_layer_gated_linear", "spec_layer_block_norm", "spec_layer_log_probs")


class sv_plan_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "npad", "drain_cols", "half", "kblock_elems", "kblocks", "chunks", "stages",
        "stage_bytes", "smem_bytes", "grid", "tmem_cols", "tmem_buffers", "tmem_slots")]


class SpecVerifyError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {spec_verify_strerror(code)} ({code})")
        self.code = code


class sv_config_t(ctypes.Structure):
    _fields_ = [("V", ctypes.c_int64), ("d", ctypes.c_int64),
                ("B", ctypes.c_int32), ("K", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("stream", ctypes.c_void_p)]


_lib = None


def load_library():
    """Loads the in-tree CUDA library (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                "(or python -m speculative_decoding_verification_22_gb300.build)")
        lib = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, f32 = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                             ctypes.c_float)
        lib.spec_verify_create.argtypes = [ctypes.POINTER(sv_config_t),
                                           ctypes.POINTER(vp)]
        lib.spec_verify_run.argtypes = [vp, vp, vp, vp, vp, vp, f32, vp, vp]
        lib.spec_verify_run_host.argtypes = [vp, vp, vp, vp, vp, vp, f32, vp, vp]
        lib.spec_verify_status.argtypes = [vp]
        lib.spec_verify_set_stream.argtypes = [vp, vp]
        lib.spec_verify_stream.argtypes = [vp]
        lib.spec_verify_stream.restype = vp
        lib.spec_verify_debug_logits.argtypes = [vp, vp]
        lib.spec_verify_debug_lse.argtypes = [vp, vp]
        lib.spec_verify_set_wait_limit.argtypes = [vp, ctypes.c_uint64]
        lib.spec_verify_debug_stall.argtypes = [vp, ctypes.c_int]
        lib.spec_verify_submit_host.argtypes = [vp, ctypes.c_int, vp, vp, vp, vp, vp, f32, vp,
                                                vp]
        lib.spec_verify_wait_host.argtypes = [vp, ctypes.c_int]
        lib.spec_verify_log_probs.argtypes = [vp, vp, f32, ctypes.c_int32, vp, vp, vp, vp]
        lib.spec_verify_timing.argtypes = [vp, ctypes.c_int]
        lib.spec_verify_timing_read.argtypes = [vp, ctypes.POINTER(ctypes.c_double),
                                                ctypes.POINTER(i64)]
        lib.spec_verify_launches_per_run.argtypes = [vp, f32]
        lib.spec_verify_strerror.argtypes = [ctypes.c_int]
        lib.spec_verify_strerror.restype = ctypes.c_char_p
        lib.spec_verify_destroy.argtypes = [vp]
        lib.spec_verify_destroy.restype = None
        lib.spec_verify_run_noalloc.argtypes = [ctypes.POINTER(sv_config_t), vp, vp, vp, vp,
                                                vp, f32, vp, vp]
        i32 = ctypes.c_int32
        lib.spec_verify_run_truncated.argtypes = [vp, vp, vp, vp, vp, vp, f32, i32, f32, i32,
                                                  f32, vp, vp]
        lib.spec_verify_tree_greedy.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp]
        lib.spec_verify_run_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, f32, vp, vp]
        lib.spec_ngram_draft.argtypes = [vp, ctypes.c_int64, vp, i32, i32, i32, i32, vp, vp,
                                         vp]
        lib.spec_verify_plan.argtypes = [ctypes.POINTER(sv_config_t), i32, i32,
                                         ctypes.POINTER(sv_plan_t)]
        lib.spec_target_create.argtypes = [ctypes.POINTER(vp)]
        lib.spec_target_destroy.argtypes = [vp]
        lib.spec_target_destroy.restype = None
        lib.spec_target_status.argtypes = [vp, vp]
        lib.spec_target_set_wait_limit.argtypes = [vp, ctypes.c_uint64]
        lib.spec_target_rms_norm.argtypes = [vp, vp, i64, vp, i64, vp, f32, i64, i64, i32, vp,
                                             i64, vp, i64, vp]
        lib.spec_target_rms_norm_fp8.argtypes = [vp, vp, i64, vp, i64, vp, f32, i64, i64, i32,
                                                 i32, vp, vp, vp, i64, vp]
        lib.spec_target_matmul_fp8.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, vp, i64,
                                               vp]
        lib.spec_target_rope_freqs.argtypes = [vp, vp, vp]
        lib.spec_target_rope_append.argtypes = [vp, vp, vp]
        lib.spec_target_attention.argtypes = [vp, vp, vp]
        lib.spec_target_tree_mask.argtypes = [vp, vp, i32, i32, vp, vp]
        for name in ("linear", "gated_linear", "block_norm", "log_probs"):
            getattr(lib, f"spec_layer_{name}").argtypes = [vp, vp, vp]
        for name in EXPORTS:
            if name not in ("spec_verify_strerror", "spec_verify_destroy", "spec_verify_stream",
                            "spec_target_destroy"):
                getattr(lib, name).restype = ctypes.c_int
        _lib = lib
    return _lib


def _check(code: int, what: str):
    if code != SV_OK:
        raise SpecVerifyError(code, what)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _stream_handle(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def spec_verify_strerror(code: int) -> str:
    return load_library().spec_verify_strerror(int(code)).decode()


def spec_verify_plan(V: int, d: int, B: int, K: int, dtype="bf16", num_sms: int = 152,
                     smem_optin: int = 232448) -> dict:
    """The contraction's launch plan for a shape (host arithmetic, no GPU):
    accumulation mode, pipeline stages, shared and tensor memory layout."""
    code = {"bf16": SV_BF16, "fp8": SV_FP8}.get(dtype, dtype)
    cfg = sv_config_t(V, d, B, K, code, None)
    out = sv_plan_t()
    _check(load_library().spec_verify_plan(ctypes.byref(cfg), num_sms, smem_optin,
                                           ctypes.byref(out)), "spec_verify_plan")
    return {n: getattr(out, n) for n, _ in sv_plan_t._fields_}


def spec_verify_create(V: int, d: int, B: int, K: int, dtype="bf16", stream=None):
    """Creates a handle; ``dtype`` is "bf16"/"fp32" (or SV_BF16/SV_FP32)."""
    code = {"bf16": SV_BF16, "fp32": SV_FP32, "fp8": SV_FP8}.get(dtype, dtype)
    cfg = sv_config_t(int(V), int(d), int(B), int(K), int(code),
                      _stream_handle(stream))
    h = ctypes.c_void_p()
    _check(load_library().spec_verify_create(ctypes.byref(cfg), ctypes.byref(h)),
           "spec_verify_create")
    return h


def spec_verify_run(h, hidden, W_lm, draft_tokens, q_logits, uniforms,
                    temperature: float, out_tokens, out_n_accepted) -> None:
    _check(load_library().spec_verify_run(
        h, _ptr(hidden), _ptr(W_lm), _ptr(draft_tokens), _ptr(q_logits),
        _ptr(uniforms), float(temperature), _ptr(out_tokens),
        _ptr(out_n_accepted)), "spec_verify_run")


def spec_verify_run_host(h, hidden, W_lm, draft_tokens, q_logits, uniforms,
                         temperature: float, out_tokens, out_n_accepted) -> None:
    """Host-buffer variant: hidden/draft/q/uniforms/outputs are host
    (preferably pinned) tensors, W_lm a device tensor; returns after the
    outputs have been copied back."""
    _check(load_library().spec_verify_run_host(
        h, _ptr(hidden), _ptr(W_lm), _ptr(draft_tokens), _ptr(q_logits),
        _ptr(uniforms), float(temperature), _ptr(out_tokens),
        _ptr(out_n_accepted)), "spec_verify_run_host")


def spec_verify_submit_host(h, slot: int, hidden, W_lm, draft_tokens, q_logits, uniforms,
                            temperature: float, out_tokens, out_n_accepted) -> None:
    """Double-buffered host round: enqueue it in slot 0 or 1 (pinned host
    tensors for inputs and outputs, W_lm on the device) and return."""
    _check(load_library().spec_verify_submit_host(
        h, int(slot), _ptr(hidden), _ptr(W_lm), _ptr(draft_tokens), _ptr(q_logits),
        _ptr(uniforms), float(temperature), _ptr(out_tokens), _ptr(out_n_accepted)),
        "spec_verify_submit_host")


def spec_verify_wait_host(h, slot: int) -> int:
    """Waits for the round in `slot`; returns its status code."""
    return int(load_library().spec_verify_wait_host(h, int(slot)))


def spec_verify_status(h) -> int:
    return int(load_library().spec_verify_status(h))


def spec_verify_set_stream(h, stream=None) -> None:
    _check(load_library().spec_verify_set_stream(h, _stream_handle(stream)),
           "spec_verify_set_stream")


def spec_verify_stream(h) -> int:
    """The number of the stream that calls are enqueued on (0: the legacy default one)."""
    return load_library().spec_verify_stream(h) or 0


def spec_verify_debug_logits(h, dst) -> None:
    _check(load_library().spec_verify_debug_logits(h, _ptr(dst)),
           "spec_verify_debug_logits")


def spec_verify_log_probs(h, tokens, temperature: float, top: int, log_probs, entropy,
                          top_ids, top_log_probs) -> None:
    """Log probabilities, entropies and most likely tokens from the last run's logits."""
    _check(load_library().spec_verify_log_probs(
        h, _ptr(tokens), float(temperature), int(top), _ptr(log_probs), _ptr(entropy),
        _ptr(top_ids), _ptr(top_log_probs)), "spec_verify_log_probs")


def spec_verify_debug_lse(h, dst) -> None:
    _check(load_library().spec_verify_debug_lse(h, _ptr(dst)),
           "spec_verify_debug_lse")


def spec_verify_set_wait_limit(h, limit_ns: int) -> None:
    _check(load_library().spec_verify_set_wait_limit(h, int(limit_ns)),
           "spec_verify_set_wait_limit")


def spec_verify_debug_stall(h, enable: bool) -> None:
    """Tests only: every run first waits for a flag nothing sets (bounded by
    the wait limit), so it reports SV_ERR_TIMEOUT and withdraws sequence 0."""
    _check(load_library().spec_verify_debug_stall(h, int(bool(enable))),
           "spec_verify_debug_stall")


def spec_verify_timing(h, enable: bool) -> None:
    _check(load_library().spec_verify_timing(h, int(bool(enable))),
           "spec_verify_timing")


def spec_verify_timing_read(h):
    ms = ctypes.c_double()
    n = ctypes.c_int64()
    _check(load_library().spec_verify_timing_read(h, ctypes.byref(ms), ctypes.byref(n)),
           "spec_verify_timing_read")
    return ms.value, n.value


def spec_verify_launches_per_run(h, temperature: float) -> int:
    n = load_library().spec_verify_launches_per_run(h, float(temperature))
    if n < 0:
        raise SpecVerifyError(n, "spec_verify_launches_per_run")
    return n


def spec_verify_run_noalloc(V, d, B, K, dtype, hidden, W_lm, draft_tokens, q_logits,
                            uniforms, temperature: float, out_tokens, out_n_accepted,
                            stream=None) -> None:
    """The step without a handle or any allocation (scratch in a fixed
    device array inside the library); for callers that cannot allocate
    device memory at call time.  Calls that overlap on the GPU race."""
    code = {"bf16": SV_BF16, "fp32": SV_FP32, "fp8": SV_FP8}.get(dtype, dtype)
    cfg = sv_config_t(int(V), int(d), int(B), int(K), int(code), _stream_handle(stream))
    _check(load_library().spec_verify_run_noalloc(
        ctypes.byref(cfg), _ptr(hidden), _ptr(W_lm), _ptr(draft_tokens), _ptr(q_logits),
        _ptr(uniforms), float(temperature), _ptr(out_tokens), _ptr(out_n_accepted)),
        "spec_verify_run_noalloc")


def spec_verify_run_truncated(h, hidden, W_lm, draft_tokens, q_logits, uniforms,
                              temperature: float, target_top_k: int, target_top_p: float,
                              draft_top_k: int, draft_top_p: float, out_tokens,
                              out_n_accepted) -> None:
    """The step with truncated sampling (top-k, then top-p; per side)."""
    _check(load_library().spec_verify_run_truncated(
        h, _ptr(hidden), _ptr(W_lm), _ptr(draft_tokens), _ptr(q_logits), _ptr(uniforms),
        float(temperature), int(target_top_k), float(target_top_p), int(draft_top_k),
        float(draft_top_p), _ptr(out_tokens), _ptr(out_n_accepted)),
        "spec_verify_run_truncated")


def spec_verify_run_fp8(h, hidden8, hidden_scale, W8, w_scale, draft_tokens, q_logits,
                        uniforms, temperature: float, out_tokens, out_n_accepted) -> None:
    """The step with an FP8 E4M3 LM head (handle dtype "fp8")."""
    _check(load_library().spec_verify_run_fp8(
        h, _ptr(hidden8), _ptr(hidden_scale), _ptr(W8), _ptr(w_scale), _ptr(draft_tokens),
        _ptr(q_logits), _ptr(uniforms), float(temperature), _ptr(out_tokens),
        _ptr(out_n_accepted)), "spec_verify_run_fp8")


def spec_verify_tree_greedy(h, hidden, W_lm, tree_tokens, tree_parents, out_tokens,
                            out_nodes, out_n) -> None:
    """Greedy tree verification: the longest path whose tokens are the
    target's argmax choices (N = the handle's K nodes)."""
    _check(load_library().spec_verify_tree_greedy(
        h, _ptr(hidden), _ptr(W_lm), _ptr(tree_tokens), _ptr(tree_parents), _ptr(out_tokens),
        _ptr(out_nodes), _ptr(out_n)), "spec_verify_tree_greedy")


def spec_ngram_draft(tokens, lengths, K: int, n_min: int = 2, n_max: int = 5,
                     out_draft=None, out_len=None, stream=None):
    """Prompt-lookup drafts for B contexts (tokens [B, L] int32 on the GPU,
    lengths [B] int32): the up to K tokens that followed the latest earlier
    occurrence of the longest recurring suffix of n_max..n_min tokens.
    Returns (draft [B, K] with -1 after the proposal, length [B]); the
    draft feeds spec_verify_run with q_logits=None."""
    B, L = tokens.shape
    if out_draft is None:
        out_draft = torch.empty((B, K), dtype=torch.int32, device=tokens.device)
    if out_len is None:
        out_len = torch.empty((B,), dtype=torch.int32, device=tokens.device)
    _check(load_library().spec_ngram_draft(
        _ptr(tokens), int(L), _ptr(lengths), int(B), int(K), int(n_min), int(n_max),
        _ptr(out_draft), _ptr(out_len), _stream_handle(stream)), "spec_ngram_draft")
    return out_draft, out_len


def spec_verify_destroy(h) -> None:
    if h:
        load_library().spec_verify_destroy(h)


class SpecVerify:
    """Owns one handle; ``run`` writes tokens [B, K+1] and n_accepted [B].  Everything is
    enqueued on the handle's stream, whose memory the outputs made here are: used on
    another stream, they have to be kept until that use has ended, or recorded there."""

    def __init__(self, V, d, B, K, dtype="bf16", device=None, stream=None):
        self.V, self.d, self.B, self.K, self.dtype = V, d, B, K, dtype
        self.device = torch.device("cuda" if device is None else device)
        with torch.cuda.device(self.device):
            self.device = torch.device("cuda", torch.cuda.current_device())
            self.h = spec_verify_create(V, d, B, K, dtype, stream)

    def _own_stream(self):
        """The handle's stream made the current one (nothing to do where it is), so that
        what is allocated meanwhile is that stream's memory."""
        raw = spec_verify_stream(self.h)
        if (torch.cuda.current_device() == self.device.index
                and torch.cuda.current_stream().cuda_stream == raw):
            return contextlib.nullcontext()
        return torch.cuda.stream(torch.cuda.ExternalStream(raw, self.device) if raw > 1
                                 else torch.cuda.default_stream(self.device))

    def _outputs(self, out_tokens, out_n_accepted, nodes=False):
        """A run's outputs, those that are not given made under the handle's stream."""
        missing = [s for s, t in (((self.B, self.K + 1), out_tokens),
                                  ((self.B,), out_n_accepted)) if t is None]
        if nodes:
            missing.append((self.B, max(self.K, 1)))
        if not missing:
            return out_tokens, out_n_accepted
        with self._own_stream():
            made = [torch.empty(s, dtype=torch.int32, device=self.device) for s in missing]
        given = (made.pop(0) if out_tokens is None else out_tokens,
                 made.pop(0) if out_n_accepted is None else out_n_accepted)
        return (*given, *made)

    def run(self, hidden, W_lm, draft_tokens, q_logits, uniforms, temperature,
            out_tokens=None, out_n_accepted=None):
        out_tokens, out_n_accepted = self._outputs(out_tokens, out_n_accepted)
        spec_verify_run(self.h, hidden, W_lm, draft_tokens, q_logits, uniforms,
                        temperature, out_tokens, out_n_accepted)
        return out_tokens, out_n_accepted

    def run_truncated(self, hidden, W_lm, draft_tokens, q_logits, uniforms, temperature,
                      target_top_k=0, target_top_p=1.0, draft_top_k=0, draft_top_p=1.0,
                      out_tokens=None, out_n_accepted=None):
        out_tokens, out_n_accepted = self._outputs(out_tokens, out_n_accepted)
        spec_verify_run_truncated(self.h, hidden, W_lm, draft_tokens, q_logits, uniforms,
                                  temperature, target_top_k, target_top_p, draft_top_k,
                                  draft_top_p, out_tokens, out_n_accepted)
        return out_tokens, out_n_accepted

    def run_fp8(self, hidden8, hidden_scale, W8, w_scale, draft_tokens, q_logits, uniforms,
                temperature, out_tokens=None, out_n_accepted=None):
        out_tokens, out_n_accepted = self._outputs(out_tokens, out_n_accepted)
        spec_verify_run_fp8(self.h, hidden8, hidden_scale, W8, w_scale, draft_tokens, q_logits,
                            uniforms, temperature, out_tokens, out_n_accepted)
        return out_tokens, out_n_accepted

    def run_tree_greedy(self, hidden, W_lm, tree_tokens, tree_parents):
        """Returns (tokens [B, N+1], nodes [B, N], n [B])."""
        out_t, out_n, out_nodes = self._outputs(None, None, True)
        spec_verify_tree_greedy(self.h, hidden, W_lm, tree_tokens, tree_parents, out_t,
                                out_nodes, out_n)
        return out_t, out_nodes[:, :self.K], out_n

    def log_probs(self, tokens=None, top=0, temperature=1.0, out=None):
        """What the last run's logits say of its answers: log probabilities
        [B, K+1] of ``tokens`` (int32 [B, K+1], as ``run`` returns them; -1 gets 0;
        None in their place without tokens), the rows' entropies [B, K+1], and with
        ``top`` > 0 the most likely ids int32 [B, K+1, top] and their log
        probabilities.  ``out``: the same tensors to be filled.  Enqueued on the
        handle's stream, whose memory the outputs made here are."""
        shape = (self.B, self.K + 1)

        def check(t, what, want, dtype):
            if (not torch.is_tensor(t) or tuple(t.shape) != want or t.dtype != dtype
                    or t.device.type != "cuda" or t.device != self.device):
                raise ValueError(f"log_probs: {what} must be {dtype} {want} on the handle's GPU")
        if tokens is not None:
            check(tokens, "tokens", shape, torch.int32)
        if not 0 <= top <= min(64, self.V):
            raise ValueError("log_probs: top must be from 0 to 64 and at most V")
        kinds = [(shape, torch.float32), (shape, torch.float32)]
        if top:
            kinds += [(shape + (top,), torch.int32), (shape + (top,), torch.float32)]
        if out is not None:
            out = list(out)
            if len(out) != len(kinds) or (out[0] is None) != (tokens is None):
                raise ValueError("log_probs: out must hold two tensors, or four with top (the "
                                 "first None without tokens)")
            for i, (want, dtype) in enumerate(kinds):
                if i or tokens is not None:
                    check(out[i], "out", want, dtype)
        with self._own_stream():
            if out is None:
                out = [torch.empty(want, dtype=dtype, device=self.device)
                       if i or tokens is not None else None
                       for i, (want, dtype) in enumerate(kinds)]
            spec_verify_log_probs(self.h, tokens, temperature, top, out[0], out[1],
                                  *(out[2:] or (None, None)))
        return out

    def status(self) -> int:
        return spec_verify_status(self.h)

    def logits(self):
        out = torch.empty((self.B * (self.K + 1), self.V), dtype=torch.float32,
                          device=self.device)
        spec_verify_debug_logits(self.h, out)
        return out

    def lse(self):
        out = torch.empty((self.B * (self.K + 1) + self.B * self.K,), dtype=torch.float64,
                          device=self.device)
        spec_verify_debug_lse(self.h, out)
        return out

    def close(self):
        if getattr(self, "h", None):
            spec_verify_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


from .target import (ACTIVATIONS, ROPE_SCALINGS, SV_FP16, SV_MAX_HEAD_DIM,  # noqa: E402
                     SV_MAX_TOP, SV_SCALE_BLOCK, TargetOps, spec_target_rope_freqs)
