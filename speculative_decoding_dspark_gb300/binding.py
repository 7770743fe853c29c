"""Python binding of libdspark.so: the C ABI in include/dspark.h, one function per
entry point with the same name.

Argument marshalling only -- shapes are read from the tensors, pointers and the
current CUDA stream are passed through, and a negative status raises
DSparkError.  Every step of the cycle runs in the library's CUDA kernels; there
is no CPU or PyTorch fallback: if the shared library is missing the import of
this module fails.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# DSPARK_LIBRARY may name another build of the library (the DSPARK_DEBUG one)
LIB_PATH = os.environ.get("DSPARK_LIBRARY") or os.path.join(_HERE, "libdspark.so")

DSPARK_OK = 0
DSPARK_ERR_INVALID_ARG = -1
DSPARK_ERR_UNSUPPORTED = -2
DSPARK_ERR_CAPACITY = -3
DSPARK_ERR_CUDA = -4
DSPARK_ERR_TIMEOUT = -5
DSPARK_ERR_DEVICE_INPUT = -6
DSPARK_ERR_WORKSPACE = -7
DSPARK_ERR_BOUNDS = -8

DSPARK_F32, DSPARK_BF16 = 0, 1
DSPARK_OP_DRAFT, DSPARK_OP_VERIFY, DSPARK_OP_SELECT, DSPARK_OP_VERIFY_MARKOV, DSPARK_OP_CALIBRATE = 0, 1, 2, 3, 4
DSPARK_OP_DRAFT_FUSED = 5
DSPARK_OP_MARKOV_GRAD = 6
DSPARK_DISTILL_REST = 1
DSPARK_GRAD_ACCUMULATE = 1
DSPARK_TOP_MAX = 128
DSPARK_ROWS_MAX_V = 1 << 22
DSPARK_FUSED_MAX_D = 16384
DSPARK_HEADS_MAX_D = 256
DSPARK_ROPE_INTERLEAVED = 1
DSPARK_ATTN_FULL_BLOCK = 1
DSPARK_DRAFT_FORCE_SIMT = 1
DSPARK_VERIFY_HOST_TARGET = 1
DSPARK_SELECT_FIXED, DSPARK_SELECT_HISTORY, DSPARK_SELECT_CURRENT, DSPARK_SELECT_FIRST_STOP = 0, 1, 2, 3
DSPARK_SELECT_CONF_CUTOFF, DSPARK_SELECT_SURVIVAL_CUTOFF = 4, 5
DSPARK_INJECT_VERIFY_BARRIER, DSPARK_INJECT_DRAFT_BARRIER, DSPARK_INJECT_ATTENTION_QUERIES = 1, 2, 4
DSPARK_INJECT_MARKOV_OPERANDS = 8

EXPORTED = ["dspark_status_string", "dspark_version", "dspark_workspace_size", "dspark_philox4x32_10",
            "dspark_markov_draft_uses_tensor_cores", "dspark_markov_draft", "dspark_verify",
            "dspark_select_prefix", "dspark_commit_lengths", "dspark_verify_static_scratch",
            "dspark_verify_markov", "dspark_set_wait_limit_ns", "dspark_set_fault_injection",
            "dspark_plan_cycles", "dspark_fit_temperatures", "dspark_kv_reserve", "dspark_kv_commit",
            "dspark_markov_draft_fused", "dspark_qk_norm_rope", "dspark_kv_append",
            "dspark_attention_workspace_size", "dspark_verify_attention", "dspark_prefix_attention",
            "dspark_token_logprobs", "dspark_distill_loss", "dspark_markov_grad"]


class DSparkError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} failed: {status} ({_status_string(status)})")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() "
                          "(or python -m speculative_decoding_dspark_gb300.build)")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, u32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint32, ctypes.c_float, ctypes.c_size_t
    L.dspark_status_string.argtypes = [i32]
    L.dspark_status_string.restype = ctypes.c_char_p
    L.dspark_version.restype = i32
    L.dspark_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32, ctypes.c_uint]
    L.dspark_workspace_size.restype = sz
    L.dspark_markov_draft_uses_tensor_cores.argtypes = [i32, i32, i32, i32, i32, ctypes.c_uint]
    L.dspark_markov_draft_uses_tensor_cores.restype = i32
    L.dspark_markov_draft.argtypes = [vp, i32, vp, vp, i32, vp, vp, u32, f32, i32, i32, i32, i32,
                                      vp, vp, vp, vp, ctypes.c_uint, vp, sz, vp, vp]
    L.dspark_markov_draft.restype = i32
    L.dspark_markov_draft_fused.argtypes = [vp, vp, i32, vp, vp, vp, vp, u32, f32, i32, i32, i32, i32,
                                            vp, vp, vp, vp, vp, sz, vp, vp]
    L.dspark_markov_draft_fused.restype = i32
    L.dspark_verify.argtypes = [vp, vp, vp, vp, vp, vp, vp, u32, f32, i32, i32, i32, i32,
                                vp, vp, vp, vp, sz, vp, vp]
    L.dspark_verify.restype = i32
    L.dspark_select_prefix.argtypes = [vp, vp, vp, vp, i32, i32, i32, f32, i32, i32, vp, vp, vp, vp,
                                       vp, sz, vp, vp]
    L.dspark_select_prefix.restype = i32
    L.dspark_plan_cycles.argtypes = [vp, vp, vp, vp, i32, i32, i32, f32, i32, i32, i32, i32, vp, vp, vp,
                                     vp, vp]
    L.dspark_plan_cycles.restype = i32
    L.dspark_verify_markov.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, u32, f32, i32, i32,
                                       i32, i32, vp, vp, vp, vp, sz, vp, vp]
    L.dspark_verify_markov.restype = i32
    L.dspark_verify_static_scratch.argtypes = [vp, vp, vp, vp, vp, vp, vp, u32, f32, i32, i32, i32,
                                               i32, vp, vp, vp, vp, vp]
    L.dspark_verify_static_scratch.restype = i32
    L.dspark_philox4x32_10.argtypes = [vp, vp, i32, vp, vp]
    L.dspark_philox4x32_10.restype = i32
    L.dspark_commit_lengths.argtypes = [vp, vp, i32, i32, vp, vp, vp, vp, vp, vp]
    L.dspark_commit_lengths.restype = i32
    L.dspark_fit_temperatures.argtypes = [vp, vp, i32, i32, vp, vp, vp, vp, sz, vp, vp]
    L.dspark_fit_temperatures.restype = i32
    L.dspark_kv_reserve.argtypes = [vp, vp, i32, i32, vp, i32, vp, vp, i32, vp, vp, vp]
    L.dspark_kv_reserve.restype = i32
    L.dspark_kv_commit.argtypes = [vp, vp, vp, i32, i32, vp, i32, vp, vp, i32, vp, vp]
    L.dspark_kv_commit.restype = i32
    i64, u = ctypes.c_int64, ctypes.c_uint
    L.dspark_qk_norm_rope.argtypes = [vp, i64, vp, i64, i32, vp, vp, f32, vp, vp, i32, i32, i32, i32, i32, vp, i64,
                                      vp, i64, i32, u, vp, vp]
    L.dspark_qk_norm_rope.restype = i32
    L.dspark_kv_append.argtypes = [vp, i64, vp, i64, vp, i64, i32, vp, vp, f32, vp, i32, vp, vp, vp] + [i32] * 8 + \
        [vp, vp, vp, i32, u, vp, vp]
    L.dspark_kv_append.restype = i32
    L.dspark_attention_workspace_size.argtypes = [i32] * 6
    L.dspark_attention_workspace_size.restype = sz
    L.dspark_verify_attention.argtypes = [vp] * 6 + [f32] + [i32] * 8 + [vp, vp, u, vp, sz, vp, vp]
    L.dspark_verify_attention.restype = i32
    L.dspark_prefix_attention.argtypes = [vp] * 8 + [i32, f32] + [i32] * 8 + [vp, vp, u, vp, sz, vp, vp]
    L.dspark_prefix_attention.restype = i32
    L.dspark_token_logprobs.argtypes = [vp, i64, i32, vp, vp, i32, i32, f32, i32, i32, i32] + [vp] * 7
    L.dspark_token_logprobs.restype = i32
    L.dspark_distill_loss.argtypes = [vp, i64, i32, vp, vp, i32, vp, f32, i32, i32, vp, vp, i64, i32, u, vp, vp]
    L.dspark_distill_loss.restype = i32
    L.dspark_markov_grad.argtypes = [vp, i64, vp, vp, vp, i32, i32, i32, vp, vp, vp, u, vp, sz, vp, vp]
    L.dspark_markov_grad.restype = i32
    L.dspark_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
    L.dspark_set_wait_limit_ns.restype = ctypes.c_uint64
    L.dspark_set_fault_injection.argtypes = [ctypes.c_uint]
    L.dspark_set_fault_injection.restype = ctypes.c_uint
    return L


_L = _load()


def library() -> ctypes.CDLL:
    return _L


def _status_string(status: int) -> str:
    return _L.dspark_status_string(int(status)).decode()


def dspark_status_string(status: int) -> str:
    return _status_string(status)


def dspark_version() -> int:
    return _L.dspark_version()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())  # of torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_DTYPE_CODES = {torch.float32: DSPARK_F32, torch.bfloat16: DSPARK_BF16}


def _dtype_code(t):
    code = _DTYPE_CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"expected float32 or bfloat16, got {t.dtype}")
    return code


def _check(t, name, dtype=None, shape=None, allow_none=False, allow_pinned=False):
    if (t is not None and t.is_cuda and (dtype is None or t.dtype is dtype) and (shape is None or t.shape == shape)
            and t.is_contiguous()):
        return
    if t is None:
        if allow_none:
            return
        raise ValueError(f"{name} is required")
    if not t.is_cuda and not (allow_pinned and t.is_pinned()):
        raise ValueError(f"{name} must be a CUDA tensor" + (" or pinned host memory" if allow_pinned else ""))
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _raise(fn, st):
    if st != DSPARK_OK:
        raise DSparkError(fn, st)


def dspark_workspace_size(op, R, gamma, V, rank=0, max_rows=0, w_dtype=DSPARK_BF16, flags=0) -> int:
    return int(_L.dspark_workspace_size(op, R, gamma, V, rank, max_rows, w_dtype, flags))


def dspark_markov_draft_uses_tensor_cores(u_dtype, w_dtype, R, V, rank, flags=0) -> bool:
    return bool(_L.dspark_markov_draft_uses_tensor_cores(u_dtype, w_dtype, R, V, rank, flags))


def dspark_set_wait_limit_ns(limit_ns: int) -> int:
    """Limit of the grid-wide device waits for later calls (0: the 2 s default);
    returns the previous limit."""
    return int(_L.dspark_set_wait_limit_ns(int(limit_ns)))


def dspark_set_fault_injection(mask: int) -> int:
    """Test hook: make the named grid-wide waits run out (see dspark.h); returns
    the previous mask."""
    return int(_L.dspark_set_fault_injection(int(mask)))


def workspace(nbytes: int, device=None) -> torch.Tensor:
    """A caller-owned workspace buffer (torch allocations are 256-byte aligned)."""
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device or "cuda")


def dspark_markov_draft(U, W1, W2, anchor, seeds, cycle, temperature, draft_tokens, q_lse=None,
                        q_tok=None, q_logits=None, ws=None, dev_status=None, flags=0, stream=None):
    R, gamma, V = U.shape
    rank = W1.shape[1]
    _check(U, "U", shape=(R, gamma, V))
    _check(W1, "W1", dtype=W2.dtype, shape=(V, rank))
    _check(W2, "W2", shape=(V, rank))
    _check(anchor, "anchor", torch.int32, (R,))
    _check(seeds, "seeds", torch.int64, (R,), allow_none=True)
    _check(draft_tokens, "draft_tokens", torch.int32, (R, gamma))
    _check(q_lse, "q_lse", torch.float32, (R, gamma), allow_none=True)
    _check(q_tok, "q_tok", torch.float32, (R, gamma), allow_none=True)
    _check(q_logits, "q_logits", torch.float32, (R, gamma, V), allow_none=True)
    _check(ws, "ws", torch.uint8)
    _check(dev_status, "dev_status", torch.int32, allow_none=True)
    st = _L.dspark_markov_draft(_ptr(U), _dtype_code(U), _ptr(W1), _ptr(W2), _dtype_code(W2),
                                _ptr(anchor), _ptr(seeds), int(cycle), float(temperature), R,
                                gamma, V, rank, _ptr(draft_tokens), _ptr(q_lse), _ptr(q_tok),
                                _ptr(q_logits), int(flags), _ptr(ws), ws.numel(),
                                _ptr(dev_status), _stream(stream))
    _raise("dspark_markov_draft", st)


def dspark_markov_draft_fused(h, W_lm, W1, W2, anchor, seeds, cycle, temperature, draft_tokens, q_lse=None,
                              q_tok=None, q_logits=None, ws=None, dev_status=None, stream=None):
    R, gamma, d = h.shape
    V = W_lm.shape[0]
    rank = W1.shape[1]
    _check(h, "h", torch.bfloat16, (R, gamma, d))
    _check(W_lm, "W_lm", torch.bfloat16, (V, d))
    _check(W1, "W1", torch.bfloat16, (V, rank))
    _check(W2, "W2", torch.bfloat16, (V, rank))
    _check(anchor, "anchor", torch.int32, (R,))
    _check(seeds, "seeds", torch.int64, (R,), allow_none=True)
    _check(draft_tokens, "draft_tokens", torch.int32, (R, gamma))
    _check(q_lse, "q_lse", torch.float32, (R, gamma), allow_none=True)
    _check(q_tok, "q_tok", torch.float32, (R, gamma), allow_none=True)
    _check(q_logits, "q_logits", torch.float32, (R, gamma, V), allow_none=True)
    _check(ws, "ws", torch.uint8)
    _check(dev_status, "dev_status", torch.int32, allow_none=True)
    st = _L.dspark_markov_draft_fused(_ptr(h), _ptr(W_lm), d, _ptr(W1), _ptr(W2), _ptr(anchor), _ptr(seeds),
                                      int(cycle), float(temperature), R, gamma, V, rank, _ptr(draft_tokens),
                                      _ptr(q_lse), _ptr(q_tok), _ptr(q_logits), _ptr(ws), ws.numel(),
                                      _ptr(dev_status), _stream(stream))
    _raise("dspark_markov_draft_fused", st)


def dspark_verify(target_logits, cu_seqlens, draft_tokens, q_logits, q_lse, q_tok, seeds, cycle,
                  temperature, max_rows, n_accepted, out_tokens, p_tok=None, ws=None,
                  dev_status=None, stream=None):
    R, gamma = draft_tokens.shape
    V = target_logits.shape[1]
    _check(target_logits, "target_logits", torch.float32)
    _check(cu_seqlens, "cu_seqlens", torch.int32, (R + 1,))
    _check(draft_tokens, "draft_tokens", torch.int32)
    _check(q_logits, "q_logits", torch.float32, (R, gamma, V), allow_none=True)
    _check(q_lse, "q_lse", torch.float32, (R, gamma), allow_none=True)
    _check(q_tok, "q_tok", torch.float32, (R, gamma), allow_none=True)
    _check(seeds, "seeds", torch.int64, (R,), allow_none=True)
    _check(n_accepted, "n_accepted", torch.int32, (R,))
    _check(out_tokens, "out_tokens", torch.int32, (R, gamma + 1))
    _check(p_tok, "p_tok", torch.float32, (R, gamma), allow_none=True)
    _check(ws, "ws", torch.uint8)
    _check(dev_status, "dev_status", torch.int32, allow_none=True)
    if target_logits.shape[0] < max_rows:
        raise ValueError("target_logits has fewer rows than max_rows")
    st = _L.dspark_verify(_ptr(target_logits), _ptr(cu_seqlens), _ptr(draft_tokens), _ptr(q_logits),
                          _ptr(q_lse), _ptr(q_tok), _ptr(seeds), int(cycle), float(temperature), R,
                          gamma, V, int(max_rows), _ptr(n_accepted), _ptr(out_tokens), _ptr(p_tok),
                          _ptr(ws), ws.numel(), _ptr(dev_status), _stream(stream))
    _raise("dspark_verify", st)


def dspark_verify_markov(target_logits, cu_seqlens, draft_tokens, U, W1, W2, anchor, q_lse, q_tok, seeds,
                         cycle, temperature, max_rows, n_accepted, out_tokens, p_tok=None, ws=None,
                         dev_status=None, stream=None):
    R, gamma = draft_tokens.shape
    V = target_logits.shape[1]
    rank = W1.shape[1]
    _check(target_logits, "target_logits", torch.float32, allow_pinned=True)
    _check(cu_seqlens, "cu_seqlens", torch.int32, (R + 1,))
    _check(draft_tokens, "draft_tokens", torch.int32)
    _check(U, "U", torch.bfloat16, (R, gamma, V))
    _check(W1, "W1", torch.bfloat16, (V, rank))
    _check(W2, "W2", torch.bfloat16, (V, rank))
    _check(anchor, "anchor", torch.int32, (R,))
    _check(q_lse, "q_lse", torch.float32, (R, gamma), allow_none=True)
    _check(q_tok, "q_tok", torch.float32, (R, gamma), allow_none=True)
    _check(seeds, "seeds", torch.int64, (R,), allow_none=True)
    _check(n_accepted, "n_accepted", torch.int32, (R,))
    _check(out_tokens, "out_tokens", torch.int32, (R, gamma + 1))
    _check(p_tok, "p_tok", torch.float32, (R, gamma), allow_none=True)
    _check(ws, "ws", torch.uint8)
    _check(dev_status, "dev_status", torch.int32, allow_none=True)
    if target_logits.shape[0] < max_rows:
        raise ValueError("target_logits has fewer rows than max_rows")
    st = _L.dspark_verify_markov(_ptr(target_logits), _ptr(cu_seqlens), _ptr(draft_tokens), _ptr(U), _ptr(W1),
                                 _ptr(W2), _ptr(anchor), rank, _ptr(q_lse), _ptr(q_tok), _ptr(seeds),
                                 int(cycle), float(temperature), R, gamma, V, int(max_rows),
                                 _ptr(n_accepted), _ptr(out_tokens), _ptr(p_tok), _ptr(ws), ws.numel(),
                                 _ptr(dev_status), _stream(stream))
    _raise("dspark_verify_markov", st)


def dspark_verify_static_scratch(target_logits, cu_seqlens, draft_tokens, q_logits, q_lse, q_tok,
                                 seeds, cycle, temperature, max_rows, n_accepted, out_tokens,
                                 p_tok=None, dev_status=None, stream=None):
    """dspark_verify without a workspace argument, for callers that are not
    allowed to allocate device memory (for example a plugin inside a serving
    engine whose device memory all belongs to the engine's pool).  The scratch
    is a fixed 4 MiB array inside the library, shared by every call on a
    device: calls must not overlap on the GPU, the first call on a device
    (which looks the array up) should happen before any stream capture, and
    the entry point must not be used after a cudaDeviceReset."""
    R, gamma = draft_tokens.shape
    V = target_logits.shape[1]
    _check(target_logits, "target_logits", torch.float32)
    _check(cu_seqlens, "cu_seqlens", torch.int32, (R + 1,))
    _check(draft_tokens, "draft_tokens", torch.int32)
    _check(q_logits, "q_logits", torch.float32, (R, gamma, V), allow_none=True)
    _check(q_lse, "q_lse", torch.float32, (R, gamma), allow_none=True)
    _check(q_tok, "q_tok", torch.float32, (R, gamma), allow_none=True)
    _check(seeds, "seeds", torch.int64, (R,), allow_none=True)
    _check(n_accepted, "n_accepted", torch.int32, (R,))
    _check(out_tokens, "out_tokens", torch.int32, (R, gamma + 1))
    _check(p_tok, "p_tok", torch.float32, (R, gamma), allow_none=True)
    _check(dev_status, "dev_status", torch.int32, allow_none=True)
    if target_logits.shape[0] < max_rows:
        raise ValueError("target_logits has fewer rows than max_rows")
    st = _L.dspark_verify_static_scratch(_ptr(target_logits), _ptr(cu_seqlens), _ptr(draft_tokens),
                                         _ptr(q_logits), _ptr(q_lse), _ptr(q_tok), _ptr(seeds),
                                         int(cycle), float(temperature), R, gamma, V, int(max_rows),
                                         _ptr(n_accepted), _ptr(out_tokens), _ptr(p_tok),
                                         _ptr(dev_status), _stream(stream))
    _raise("dspark_verify_static_scratch", st)


def dspark_select_prefix(c, c_hist, capture_sizes, sps, K_cap, mode, a, l, cu_seqlens, K_used,
                         ws=None, dev_status=None, stream=None, conf_min=0.0):
    R, gamma = c.shape
    _check(c, "c", torch.float32)
    _check(c_hist, "c_hist", torch.float32, (R, gamma), allow_none=True)
    _check(capture_sizes, "capture_sizes", torch.int32, allow_none=True)
    _check(sps, "sps", torch.float32, allow_none=True)
    _check(a, "a", torch.float32, (R, gamma))
    _check(l, "l", torch.int32, (R,))
    _check(cu_seqlens, "cu_seqlens", torch.int32, (R + 1,))
    _check(K_used, "K_used", torch.int32, (1,))
    _check(dev_status, "dev_status", torch.int32, allow_none=True)
    n_steps = 0 if capture_sizes is None else capture_sizes.numel()
    if sps is not None and sps.numel() != n_steps:
        raise ValueError("sps and capture_sizes differ in length")
    st = _L.dspark_select_prefix(_ptr(c), _ptr(c_hist), _ptr(capture_sizes), _ptr(sps), n_steps,
                                 int(K_cap), int(mode), float(conf_min), R, gamma, _ptr(a), _ptr(l),
                                 _ptr(cu_seqlens), _ptr(K_used), _ptr(ws),
                                 0 if ws is None else ws.numel(), _ptr(dev_status), _stream(stream))
    _raise("dspark_select_prefix", st)


def dspark_plan_cycles(c_seq, n_full, capture_sizes, sps, K_cap, mode, l_seq, K_seq, stats, conf_min=0.0,
                       lag=2, dev_status=None, stream=None):
    T, R, gamma = c_seq.shape
    _check(c_seq, "c_seq", torch.float32)
    _check(n_full, "n_full", torch.int32, (T, R), allow_none=True)
    _check(capture_sizes, "capture_sizes", torch.int32)
    _check(sps, "sps", torch.float32, (capture_sizes.numel(),))
    _check(l_seq, "l_seq", torch.int32, (T, R))
    _check(K_seq, "K_seq", torch.int32, (T,))
    _check(stats, "stats", torch.float64, (T, 4))
    _check(dev_status, "dev_status", torch.int32, allow_none=True)
    st = _L.dspark_plan_cycles(_ptr(c_seq), _ptr(n_full), _ptr(capture_sizes), _ptr(sps), capture_sizes.numel(),
                               int(K_cap), int(mode), float(conf_min), int(lag), T, R, gamma, _ptr(l_seq),
                               _ptr(K_seq), _ptr(stats), _ptr(dev_status), _stream(stream))
    _raise("dspark_plan_cycles", st)


def dspark_fit_temperatures(z, accepted, tau, nll=None, count=None, ws=None, dev_status=None, stream=None):
    N, gamma = z.shape
    _check(z, "z", torch.float32)
    _check(accepted, "accepted", torch.uint8, (N, gamma))
    _check(tau, "tau", torch.float32, (gamma,))
    _check(nll, "nll", torch.float64, (gamma,), allow_none=True)
    _check(count, "count", torch.int32, (gamma,), allow_none=True)
    _check(ws, "ws", torch.uint8)
    _check(dev_status, "dev_status", torch.int32, allow_none=True)
    st = _L.dspark_fit_temperatures(_ptr(z), _ptr(accepted), N, gamma, _ptr(tau), _ptr(nll), _ptr(count),
                                    _ptr(ws), ws.numel(), _ptr(dev_status), _stream(stream))
    _raise("dspark_fit_temperatures", st)


def dspark_kv_reserve(kv_len, l, page_size, block_table, free_pages, free_top, reserved=None, dev_status=None,
                      stream=None):
    R, max_blocks = block_table.shape
    _check(kv_len, "kv_len", torch.int32, (R,))
    _check(l, "l", torch.int32, (R,))
    _check(block_table, "block_table", torch.int32)
    _check(free_pages, "free_pages", torch.int32)
    _check(free_top, "free_top", torch.int32, (1,))
    _check(reserved, "reserved", torch.int32, (R,), allow_none=True)
    _check(dev_status, "dev_status", torch.int32, allow_none=True)
    _raise("dspark_kv_reserve",
           _L.dspark_kv_reserve(_ptr(kv_len), _ptr(l), R, int(page_size), _ptr(block_table), max_blocks,
                                _ptr(free_pages), _ptr(free_top), free_pages.numel(), _ptr(reserved),
                                _ptr(dev_status), _stream(stream)))


def dspark_kv_commit(kv_len, l, n_accepted, page_size, block_table, free_pages, free_top, dev_status=None,
                     stream=None):
    R, max_blocks = block_table.shape
    _check(kv_len, "kv_len", torch.int32, (R,))
    _check(l, "l", torch.int32, (R,))
    _check(n_accepted, "n_accepted", torch.int32, (R,))
    _check(block_table, "block_table", torch.int32)
    _check(free_pages, "free_pages", torch.int32)
    _check(free_top, "free_top", torch.int32, (1,))
    _check(dev_status, "dev_status", torch.int32, allow_none=True)
    _raise("dspark_kv_commit",
           _L.dspark_kv_commit(_ptr(kv_len), _ptr(l), _ptr(n_accepted), R, int(page_size), _ptr(block_table),
                               max_blocks, _ptr(free_pages), _ptr(free_top), free_pages.numel(), _ptr(dev_status),
                               _stream(stream)))


def _rows(t, name, dtype=None, shape=None):
    """A [rows, heads, head_dim] tensor whose rows may lie apart; the elements between rows."""
    if (t is not None and t.is_cuda and len(size := t.shape) == 3 and (shape is None or size == shape)
            and (dtype is None or t.dtype is dtype)):
        s0, s1, s2 = t.stride()
        if s2 == 1 and s1 == size[2]:
            return s0 if size[0] > 1 else size[1] * s1
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 3 or (shape is not None and tuple(t.shape) != tuple(shape)):
        raise ValueError(f"{name} must have shape {shape or '[rows, heads, head_dim]'}, got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    rows, heads, d = t.shape
    if (d > 1 and t.stride(2) != 1) or (heads > 1 and t.stride(1) != d):
        raise ValueError(f"{name} must have contiguous rows")
    return t.stride(0) if rows > 1 else heads * d


def dspark_qk_norm_rope(q, k, q_weight, k_weight, eps, positions, inv_freq, q_out, k_out, interleaved=False,
                        dev_status=None, stream=None):
    rows, hq, d = q.shape
    hkv = k.shape[1]
    q_stride = _rows(q, "q")
    k_stride = _rows(k, "k", q.dtype, (rows, hkv, d))
    qo_stride = _rows(q_out, "q_out", shape=(rows, hq, d))
    ko_stride = _rows(k_out, "k_out", q_out.dtype, (rows, hkv, d))
    _check(q_weight, "q_weight", q.dtype, (d,), allow_none=True)
    _check(k_weight, "k_weight", q.dtype, (d,), allow_none=True)
    _check(inv_freq, "inv_freq", torch.float32, allow_none=True)
    _check(positions, "positions", torch.int32, (rows,), allow_none=inv_freq is None)
    _check(dev_status, "dev_status", torch.int32, allow_none=True)
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    st = _L.dspark_qk_norm_rope(_ptr(q), q_stride, _ptr(k), k_stride, _dtype_code(q), _ptr(q_weight), _ptr(k_weight),
                                float(eps), _ptr(positions), _ptr(inv_freq), rot, rows, hq, hkv, d, _ptr(q_out),
                                qo_stride, _ptr(k_out), ko_stride, _dtype_code(q_out),
                                DSPARK_ROPE_INTERLEAVED if interleaved else 0, _ptr(dev_status), _stream(stream))
    _raise("dspark_qk_norm_rope", st)


def dspark_kv_append(q, k, v, q_weight, k_weight, eps, inv_freq, cu_seqlens, kv_len, block_table, k_cache, v_cache,
                     q_out, interleaved=False, dev_status=None, stream=None):
    rows, hkv, d = k.shape
    R, max_blocks = block_table.shape
    pages, page_size = k_cache.shape[0], k_cache.shape[2]
    k_stride = _rows(k, "k")
    v_stride = _rows(v, "v", k.dtype, (rows, hkv, d))
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    hq = 0 if q is None else q.shape[1]
    q_stride = 0 if q is None else _rows(q, "q", k.dtype, (rows, hq, d))
    _check(q_out, "q_out", k_cache.dtype, (rows, hq, d), allow_none=True)
    _check(q_weight, "q_weight", k.dtype, (d,), allow_none=True)
    _check(k_weight, "k_weight", k.dtype, (d,), allow_none=True)
    _check(inv_freq, "inv_freq", torch.float32, allow_none=True)
    _check(cu_seqlens, "cu_seqlens", torch.int32, (R + 1,))
    _check(kv_len, "kv_len", torch.int32, (R,))
    _check(block_table, "block_table", torch.int32)
    _check(k_cache, "k_cache", shape=(pages, hkv, page_size, d))
    _check(v_cache, "v_cache", k_cache.dtype, (pages, hkv, page_size, d))
    _check(dev_status, "dev_status", torch.int32, allow_none=True)
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    st = _L.dspark_kv_append(_ptr(q), q_stride, _ptr(k), k_stride, _ptr(v), v_stride, _dtype_code(k), _ptr(q_weight),
                             _ptr(k_weight), float(eps), _ptr(inv_freq), rot, _ptr(cu_seqlens), _ptr(kv_len),
                             _ptr(block_table), R, rows, hq, hkv, d, page_size, max_blocks, pages, _ptr(k_cache),
                             _ptr(v_cache), _ptr(q_out), _dtype_code(k_cache),
                             DSPARK_ROPE_INTERLEAVED if interleaved else 0, _ptr(dev_status), _stream(stream))
    _raise("dspark_kv_append", st)


def dspark_attention_workspace_size(R, n_groups, max_rows, n_q_heads, n_kv_heads, head_dim) -> int:
    return int(_L.dspark_attention_workspace_size(R, n_groups, max_rows, n_q_heads, n_kv_heads, head_dim))


def _attention_args(q, k_cache, v_cache, block_table, kv_len, cu_seqlens, out, lse, ws, dev_status):
    rows, hq, d = q.shape
    R, max_blocks = block_table.shape
    pages, hkv, page_size, _ = k_cache.shape
    _check(q, "q", torch.bfloat16)
    _check(k_cache, "k_cache", torch.bfloat16, (pages, hkv, page_size, d))
    _check(v_cache, "v_cache", torch.bfloat16, (pages, hkv, page_size, d))
    _check(block_table, "block_table", torch.int32)
    _check(kv_len, "kv_len", torch.int32, (R,))
    _check(cu_seqlens, "cu_seqlens", torch.int32, (R + 1,))
    _check(out, "out", torch.bfloat16, (rows, hq, d))
    _check(lse, "lse", torch.float32, (rows, hq), allow_none=True)
    _check(ws, "ws", torch.uint8)
    _check(dev_status, "dev_status", torch.int32, allow_none=True)
    return (R, rows, hq, hkv, d, page_size, max_blocks, pages)


def dspark_verify_attention(q, k_cache, v_cache, block_table, kv_len, cu_seqlens, scale, out, lse=None,
                            full_block=False, ws=None, dev_status=None, stream=None):
    sizes = _attention_args(q, k_cache, v_cache, block_table, kv_len, cu_seqlens, out, lse, ws, dev_status)
    st = _L.dspark_verify_attention(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(kv_len),
                                    _ptr(cu_seqlens), float(scale), *sizes, _ptr(out), _ptr(lse),
                                    DSPARK_ATTN_FULL_BLOCK if full_block else 0, _ptr(ws), ws.numel(),
                                    _ptr(dev_status), _stream(stream))
    _raise("dspark_verify_attention", st)


def dspark_prefix_attention(q, k_cache, v_cache, block_table, kv_len, cu_seqlens, group_start, shared_len, scale, out,
                            lse=None, full_block=False, ws=None, dev_status=None, stream=None):
    sizes = _attention_args(q, k_cache, v_cache, block_table, kv_len, cu_seqlens, out, lse, ws, dev_status)
    n_groups = shared_len.numel()
    _check(group_start, "group_start", torch.int32, (n_groups + 1,))
    _check(shared_len, "shared_len", torch.int32)
    st = _L.dspark_prefix_attention(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(kv_len),
                                    _ptr(cu_seqlens), _ptr(group_start), _ptr(shared_len), n_groups, float(scale),
                                    *sizes, _ptr(out), _ptr(lse), DSPARK_ATTN_FULL_BLOCK if full_block else 0,
                                    _ptr(ws), ws.numel(), _ptr(dev_status), _stream(stream))
    _raise("dspark_prefix_attention", st)


def _arg(t, name, dtype, shape=None, optional=False):
    """The address of a tensor that _check accepts."""
    if t is None and optional:
        return None
    if not (t is not None and t.is_cuda and t.dtype is dtype and (shape is None or t.shape == shape) and t.is_contiguous()):
        _check(t, name, dtype, shape)
    return t.data_ptr()


def _vocab_rows(t, name, dtype=None, shape=None):
    """A [rows, V] tensor whose rows may lie apart: rows, V, and the elements from row to row."""
    if (t is not None and t.is_cuda and len(size := t.shape) == 2 and (shape is None or size == shape)
            and (dtype is None or t.dtype is dtype)):
        (rows, V), (s0, s1) = size, t.stride()
        if s1 == 1:
            return rows, V, s0 if rows > 1 else V
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 2 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must have shape {shape or '[rows, V]'}, got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    rows, V = t.shape
    if V > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    return rows, V, t.stride(0) if rows > 1 else V


def dspark_token_logprobs(logits, tokens, temperature, logprob, lse=None, entropy=None, top_ids=None,
                          top_logprobs=None, cu_seqlens=None, dev_status=None, stream=None):
    rows, V, stride = _vocab_rows(logits, "logits")
    i32, f32 = torch.int32, torch.float32
    R = width = top_k = 0
    cu = None
    if cu_seqlens is not None:
        if tokens is None or tokens.dim() != 2:
            raise ValueError("tokens must have shape [R, width] beside cu_seqlens")
        R, width = tokens.shape
        cu = _arg(cu_seqlens, "cu_seqlens", i32, (R + 1,))
    tok = _arg(tokens, "tokens", i32, None if cu else (rows,), True)
    row = (rows,)
    if (top_ids is None) != (top_logprobs is None):
        raise ValueError("top_ids and top_logprobs go together")
    listed = None
    if top_ids is not None:
        listed = top_ids.shape
        if len(listed) != 2 or listed[0] != rows:
            raise ValueError("top_ids must have shape [rows, top_k]")
        top_k = listed[1]
    st = _L.dspark_token_logprobs(logits.data_ptr(), stride, _dtype_code(logits), tok, cu, R, width, float(temperature), rows,
                                  V, top_k, _arg(logprob, "logprob", f32, row, tok is None), _arg(lse, "lse", f32, row, True),
                                  _arg(entropy, "entropy", f32, row, True),
                                  _arg(top_ids, "top_ids", i32, None, True),
                                  _arg(top_logprobs, "top_logprobs", f32, listed, True),
                                  _arg(dev_status, "dev_status", i32, None, True), _stream(stream))
    if st:
        _raise("dspark_token_logprobs", st)


def dspark_distill_loss(student, teacher_ids, teacher_logprobs, temperature, loss, grad=None, row_weight=None,
                        rest=False, dev_status=None, stream=None):
    rows, V, stride = _vocab_rows(student, "student")
    i32, f32 = torch.int32, torch.float32
    if teacher_ids is None or len(listed := teacher_ids.shape) != 2 or listed[0] != rows:
        raise ValueError("teacher_ids must have shape [rows, top_k]")
    grad_ptr, grad_stride, grad_code = None, 0, 0
    if grad is not None:
        _, _, grad_stride = _vocab_rows(grad, "grad", None, (rows, V))
        grad_ptr, grad_code = grad.data_ptr(), _dtype_code(grad)
    st = _L.dspark_distill_loss(student.data_ptr(), stride, _dtype_code(student), _arg(teacher_ids, "teacher_ids", i32),
                                _arg(teacher_logprobs, "teacher_logprobs", f32, listed), listed[1],
                                _arg(row_weight, "row_weight", f32, (rows,), True), float(temperature), rows, V,
                                _arg(loss, "loss", f32, (rows,)), grad_ptr, grad_stride, grad_code,
                                DSPARK_DISTILL_REST if rest else 0, _arg(dev_status, "dev_status", i32, None, True),
                                _stream(stream))
    if st:
        _raise("dspark_distill_loss", st)


def dspark_markov_grad(grad, prev, W1, W2, grad_prev, dW1=None, dW2=None, accumulate=False, ws=None, dev_status=None,
                       stream=None):
    bf16, f32 = torch.bfloat16, torch.float32
    rows, V, stride = _vocab_rows(grad, "grad", bf16)
    rank = W1.shape[1]
    factor = (V, rank)
    st = _L.dspark_markov_grad(grad.data_ptr(), stride, _arg(prev, "prev", torch.int32, (rows,)), _arg(W1, "W1", bf16, factor),
                               _arg(W2, "W2", bf16, factor), rows, V, rank, _arg(grad_prev, "grad_prev", f32, (rows, rank)),
                               _arg(dW1, "dW1", f32, factor, True), _arg(dW2, "dW2", f32, factor, True),
                               DSPARK_GRAD_ACCUMULATE if accumulate else 0, _arg(ws, "ws", torch.uint8), ws.numel(),
                               _arg(dev_status, "dev_status", torch.int32, None, True), _stream(stream))
    if st:
        _raise("dspark_markov_grad", st)


def dspark_philox4x32_10(ctr, keys, out, stream=None):
    n = keys.shape[0]
    _check(ctr, "ctr", torch.int32, (n, 4))
    _check(keys, "keys", torch.int64, (n,))
    _check(out, "out", torch.int32, (n, 4))
    _raise("dspark_philox4x32_10",
           _L.dspark_philox4x32_10(_ptr(ctr), _ptr(keys), n, _ptr(out), _stream(stream)))


def dspark_commit_lengths(n_accepted, l, gamma, commit_len, cu_commit, discard, total=None,
                          dev_status=None, stream=None):
    R = n_accepted.shape[0]
    _check(n_accepted, "n_accepted", torch.int32, (R,))
    _check(l, "l", torch.int32, (R,), allow_none=True)
    _check(commit_len, "commit_len", torch.int32, (R,))
    _check(cu_commit, "cu_commit", torch.int32, (R + 1,))
    _check(discard, "discard", torch.int32, (R,))
    _check(total, "total", torch.int32, (1,), allow_none=True)
    _check(dev_status, "dev_status", torch.int32, allow_none=True)
    st = _L.dspark_commit_lengths(_ptr(n_accepted), _ptr(l), R, int(gamma), _ptr(commit_len),
                                  _ptr(cu_commit), _ptr(discard), _ptr(total), _ptr(dev_status),
                                  _stream(stream))
    _raise("dspark_commit_lengths", st)
