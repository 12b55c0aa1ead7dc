"""Python binding of libllm (include/llm.h): argument marshalling only.

Every computation runs in the CUDA library; this module converts Python/numpy/torch
arguments to the C ABI and raises on error statuses.  If libllm.so is missing the
import of the library fails loudly: there is no CPU path.
"""
import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libllm.so")

LLM_OK, LLM_ERR_CONFIG, LLM_ERR_WEIGHTS_SIZE, LLM_ERR_OOM, LLM_ERR_POS_RANGE = 0, 1, 2, 3, 4
LLM_ERR_TOKEN_RANGE, LLM_ERR_BATCH, LLM_ERR_ARG, LLM_ERR_CUDA, LLM_ERR_DEVICE_TIMEOUT = 5, 6, 7, 8, 9
LLM_DTYPE_F32, LLM_DTYPE_BF16 = 0, 1
LLM_CACHE_MODEL, LLM_CACHE_E4M3 = 0, 1

# every extern "C" symbol include/llm.h declares
EXPORTS = ("llm_weight_count", "llm_create", "llm_destroy", "llm_reset", "llm_prefill", "llm_decode",
           "llm_sample", "llm_step", "llm_prefill_dev", "llm_decode_dev", "llm_sample_dev",
           "llm_step_dev", "llm_synchronize", "llm_stream", "llm_logits_buffer", "llm_filled",
           "llm_last_error", "llm_status_string", "llm_kv_import", "llm_kv_export",
           "llm_debug_trace", "llm_profile_kernel", "llm_sample_noalloc",
           "llm_step_kernels", "llm_decode_rows", "llm_decode_rows_dev", "llm_step_rows",
           "llm_step_rows_dev", "llm_generate", "llm_generate_dev", "llm_decode_paged",
           "llm_decode_paged_dev", "llm_step_paged", "llm_step_paged_dev", "llm_check_wait_timeout",
           "llm_prefill_packed", "llm_qcache_write", "llm_qcache_read", "llm_qcache_workspace",
           "llm_qcache_attend", "llm_verify", "llm_verify_step", "llm_qcache_shared_workspace",
           "llm_qcache_attend_shared", "llm_pages_workspace", "llm_pages_update", "llm_pages_compact",
           "llm_qcache_copy_pages", "llm_copy_pages", "llm_sample_rows")


class LlmConfig(ctypes.Structure):
    _fields_ = [("kv_heads", ctypes.c_int32), ("group", ctypes.c_int32), ("half", ctypes.c_int32),
                ("ffn", ctypes.c_int32), ("layers", ctypes.c_int32), ("vocab", ctypes.c_int32),
                ("eps", ctypes.c_float), ("theta", ctypes.c_float), ("tied", ctypes.c_int32),
                ("rope_llama3", ctypes.c_int32), ("rope_factor", ctypes.c_float),
                ("rope_low_freq", ctypes.c_float), ("rope_high_freq", ctypes.c_float),
                ("rope_orig_max_pos", ctypes.c_float), ("max_batch", ctypes.c_int32),
                ("max_seq", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("debug_trace", ctypes.c_int32), ("tc_min_batch", ctypes.c_int32),
                ("max_tokens", ctypes.c_int32), ("step_kernel", ctypes.c_int32),
                ("cache_type", ctypes.c_int32)]


class LlmQcache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("rows", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("max_seq", ctypes.c_int32), ("head", ctypes.c_int32)]


class LlmPages(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("length", ctypes.c_void_p), ("rows", ctypes.c_int32),
                ("pages_per_row", ctypes.c_int32), ("pages", ctypes.c_int32)]


class LlmError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"{msg} (status {status})")
        self.status = status


# argument and result types of every entry point (ctypes)
_i32, _i64, _u64, _f32, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_float, ctypes.c_void_p
_pcfg = ctypes.POINTER(LlmConfig)
_pqc = ctypes.POINTER(LlmQcache)
_ppg = ctypes.POINTER(LlmPages)
SIGNATURES = {
    "llm_weight_count": ([_pcfg], _u64),
    "llm_create": ([_pcfg, _vp, _u64, _i32, _vp, ctypes.POINTER(_vp)], _i32),
    "llm_destroy": ([_vp], _i32),
    "llm_reset": ([_vp], _i32),
    "llm_prefill": ([_vp, _vp, _i32, _i32, _i32, _vp], _i32),
    "llm_decode": ([_vp, _vp, _i32, _i32, _vp], _i32),
    "llm_sample": ([_vp, _vp, _i32, _f32, _i32, _f32, _vp, _vp], _i32),
    "llm_step": ([_vp, _vp, _i32, _i32, _f32, _i32, _f32, _vp, _vp, _vp], _i32),
    "llm_prefill_dev": ([_vp, _vp, _i32, _i32, _i32, _vp], _i32),
    "llm_decode_dev": ([_vp, _vp, _i32, _i32, _vp], _i32),
    "llm_sample_dev": ([_vp, _vp, _i32, _f32, _i32, _f32, _vp, _vp], _i32),
    "llm_step_dev": ([_vp, _vp, _i32, _i32, _f32, _i32, _f32, _vp, _vp, _vp], _i32),
    "llm_decode_rows": ([_vp, _vp, _i32, _vp, _vp], _i32),
    "llm_decode_rows_dev": ([_vp, _vp, _i32, _vp, _vp], _i32),
    "llm_step_rows": ([_vp, _vp, _i32, _vp, _f32, _i32, _f32, _vp, _vp, _vp], _i32),
    "llm_step_rows_dev": ([_vp, _vp, _i32, _vp, _f32, _i32, _f32, _vp, _vp, _vp], _i32),
    "llm_generate": ([_vp, _vp, _i32, _i32, _i32, _f32, _i32, _f32, _vp, _vp], _i32),
    "llm_generate_dev": ([_vp, _vp, _i32, _i32, _i32, _f32, _i32, _f32, _vp, _vp], _i32),
    "llm_decode_paged": ([_vp, _vp, _i32, _vp, _vp, _i32, _vp], _i32),
    "llm_decode_paged_dev": ([_vp, _vp, _i32, _vp, _vp, _i32, _vp], _i32),
    "llm_step_paged": ([_vp, _vp, _i32, _vp, _vp, _i32, _f32, _i32, _f32, _vp, _vp, _vp], _i32),
    "llm_step_paged_dev": ([_vp, _vp, _i32, _vp, _vp, _i32, _f32, _i32, _f32, _vp, _vp, _vp], _i32),
    "llm_prefill_packed": ([_vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _vp], _i32),
    "llm_synchronize": ([_vp], _i32),
    "llm_stream": ([_vp], _vp),
    "llm_logits_buffer": ([_vp], _vp),
    "llm_filled": ([_vp, _i32], _i32),
    "llm_last_error": ([_vp], ctypes.c_char_p),
    "llm_status_string": ([_i32], ctypes.c_char_p),
    "llm_kv_import": ([_vp, _i32, _i32, _i32, _i32, _vp, _vp], _i32),
    "llm_kv_export": ([_vp, _i32, _i32, _i32, _i32, _vp, _vp], _i32),
    "llm_debug_trace": ([_vp, _i32, ctypes.c_char_p, _vp], _i32),
    "llm_profile_kernel": ([_vp, _i32, _i32, _i32, _i32, ctypes.POINTER(_f32)], _i32),
    "llm_sample_noalloc": ([_vp, _i32, _i32, _f32, _i32, _f32, _vp, _vp, _vp], _i32),
    "llm_step_kernels": ([_vp, _i32, _f32, _i32, ctypes.POINTER(_i32)], _i32),
    "llm_check_wait_timeout": ([_vp, _i64], _i32),
    "llm_qcache_write": ([_pqc, _vp, _vp, _i32, _i64, _i32, _i32, _vp, _vp, _vp, _i32, _vp, _vp], _i32),
    "llm_qcache_read": ([_pqc, _i32, _i32, _vp, _vp, _vp, _i32, _vp, _vp, _i32, _i64, _vp, _vp], _i32),
    "llm_qcache_workspace": ([_pqc, _i32, _i32, _i32, ctypes.POINTER(_u64)], _i32),
    "llm_qcache_attend": ([_pqc, _vp, _i32, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _i32, _f32, _vp, _i64, _vp, _u64,
                           _vp, _vp], _i32),
    "llm_verify_step": ([_vp, _vp, _i32, _i32, _vp, _f32, _vp, _vp, _vp, _vp, _vp], _i32),
    "llm_verify": ([_vp, _vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp], _i32),
    "llm_qcache_shared_workspace": ([_pqc, _i32, _i32, _i32, _i32, ctypes.POINTER(_u64)], _i32),
    "llm_qcache_attend_shared": ([_pqc, _vp, _i32, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _i32, _vp, _vp, _i32, _f32, _vp,
                                  _i64, _vp, _u64, _vp, _vp], _i32),
    "llm_pages_workspace": ([_ppg, ctypes.POINTER(_u64)], _i32),
    "llm_pages_update": ([_ppg, _ppg, _vp, _vp, _vp, _vp, _vp, _u64, _vp, _vp], _i32),
    "llm_pages_compact": ([_ppg, _ppg, _vp, _vp, _vp, _u64, _vp, _vp], _i32),
    "llm_qcache_copy_pages": ([_vp, _i32, _vp, _i32, _vp, _vp, _vp], _i32),
    "llm_copy_pages": ([_vp, _vp, _i32], _i32),
    "llm_sample_rows": ([_vp, _i64, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp], _i32),
    }

_lib = None


def lib():
    """The loaded libllm.so (ctypes).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m llama_architecture_kv_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def config(shape, max_batch, max_seq, debug_trace=False, tc_min_batch=0, max_tokens=0,
           step_kernel=0, cache_type=LLM_CACHE_MODEL) -> LlmConfig:
    """An llm_config from a shape description (fields kv, g, half, ffn, layers, vocab, eps,
    theta, tied, llama3, factor, low_freq, high_freq, orig_max, bf16)."""
    return LlmConfig(shape.kv, shape.g, shape.half, shape.ffn, shape.layers, shape.vocab,
                     shape.eps, shape.theta, int(shape.tied), int(shape.llama3), shape.factor,
                     shape.low_freq, shape.high_freq, shape.orig_max, max_batch, max_seq,
                     LLM_DTYPE_BF16 if shape.bf16 else LLM_DTYPE_F32, int(debug_trace),
                     int(tc_min_batch), int(max_tokens), int(step_kernel), int(cache_type))


def _ptr(a):
    if a is None:
        return None
    if isinstance(a, int):
        return a
    if isinstance(a, np.ndarray):
        assert a.flags.c_contiguous
        return a.ctypes.data
    if hasattr(a, "data_ptr"):  # torch tensor
        assert a.is_contiguous()
        return a.data_ptr()
    raise TypeError(type(a))


def _check(h, status):
    if status != LLM_OK:
        msg = lib().llm_last_error(h) if h else None
        name = lib().llm_status_string(status).decode()
        raise LlmError(status, f"{name}: {msg.decode() if msg else ''}")


# ---- the C functions under their own names -------------------------------------------------

def llm_weight_count(cfg: LlmConfig) -> int:
    return int(lib().llm_weight_count(ctypes.byref(cfg)))


def llm_create(cfg: LlmConfig, weights, weights_on_device=False, stream=None):
    nbytes = weights.nbytes if isinstance(weights, np.ndarray) else weights.numel() * weights.element_size()
    h = ctypes.c_void_p()
    st = lib().llm_create(ctypes.byref(cfg), _ptr(weights), nbytes, int(weights_on_device),
                          stream, ctypes.byref(h))
    if st != LLM_OK:
        why = lib().llm_last_error(None)
        raise LlmError(st, f"llm_create: {lib().llm_status_string(st).decode()}: "
                           f"{why.decode() if why else ''}")
    return h.value


def llm_destroy(h):
    _check(None, lib().llm_destroy(h))


def llm_reset(h):
    _check(h, lib().llm_reset(h))


def llm_prefill(h, tokens, B, S, pos, logits=None):
    _check(h, lib().llm_prefill(h, _ptr(tokens), B, S, pos, _ptr(logits)))


def llm_decode(h, tokens, B, pos, logits):
    _check(h, lib().llm_decode(h, _ptr(tokens), B, pos, _ptr(logits)))


def llm_sample(h, logits, B, temp, k, p, u, ids):
    _check(h, lib().llm_sample(h, _ptr(logits), B, temp, k, p, _ptr(u), _ptr(ids)))


def llm_step(h, tokens, B, pos, temp, k, p, u, ids, logits=None):
    _check(h, lib().llm_step(h, _ptr(tokens), B, pos, temp, k, p, _ptr(u), _ptr(ids), _ptr(logits)))


def llm_prefill_dev(h, tokens, B, S, pos, logits=None):
    _check(h, lib().llm_prefill_dev(h, _ptr(tokens), B, S, pos, _ptr(logits)))


def llm_decode_dev(h, tokens, B, pos, logits):
    _check(h, lib().llm_decode_dev(h, _ptr(tokens), B, pos, _ptr(logits)))


def llm_sample_dev(h, logits, B, temp, k, p, u, ids):
    _check(h, lib().llm_sample_dev(h, _ptr(logits), B, temp, k, p, _ptr(u), _ptr(ids)))


def llm_step_dev(h, tokens, B, pos, temp, k, p, u, ids, logits=None):
    _check(h, lib().llm_step_dev(h, _ptr(tokens), B, pos, temp, k, p, _ptr(u), _ptr(ids), _ptr(logits)))


def llm_decode_rows(h, tokens, B, positions, logits):
    _check(h, lib().llm_decode_rows(h, _ptr(tokens), B, _ptr(positions), _ptr(logits)))


def llm_decode_rows_dev(h, tokens, B, positions, logits):
    _check(h, lib().llm_decode_rows_dev(h, _ptr(tokens), B, _ptr(positions), _ptr(logits)))


def llm_step_rows(h, tokens, B, positions, temp, k, p, u, ids, logits=None):
    _check(h, lib().llm_step_rows(h, _ptr(tokens), B, _ptr(positions), temp, k, p, _ptr(u), _ptr(ids),
                                  _ptr(logits)))


def llm_step_rows_dev(h, tokens, B, positions, temp, k, p, u, ids, logits=None):
    _check(h, lib().llm_step_rows_dev(h, _ptr(tokens), B, _ptr(positions), temp, k, p, _ptr(u), _ptr(ids),
                                      _ptr(logits)))


def llm_generate(h, tokens, B, pos, n_steps, temp, k, p, u, ids):
    _check(h, lib().llm_generate(h, _ptr(tokens), B, pos, n_steps, temp, k, p, _ptr(u), _ptr(ids)))


def llm_generate_dev(h, tokens, B, pos, n_steps, temp, k, p, u, ids):
    _check(h, lib().llm_generate_dev(h, _ptr(tokens), B, pos, n_steps, temp, k, p, _ptr(u), _ptr(ids)))


def llm_decode_paged(h, tokens, B, positions, table, pages_per_row, logits):
    _check(h, lib().llm_decode_paged(h, _ptr(tokens), B, _ptr(positions), _ptr(table), pages_per_row,
                                     _ptr(logits)))


def llm_decode_paged_dev(h, tokens, B, positions, table, pages_per_row, logits):
    _check(h, lib().llm_decode_paged_dev(h, _ptr(tokens), B, _ptr(positions), _ptr(table), pages_per_row,
                                         _ptr(logits)))


def llm_step_paged(h, tokens, B, positions, table, pages_per_row, temp, k, p, u, ids, logits=None):
    _check(h, lib().llm_step_paged(h, _ptr(tokens), B, _ptr(positions), _ptr(table), pages_per_row, temp, k, p,
                                   _ptr(u), _ptr(ids), _ptr(logits)))


def llm_step_paged_dev(h, tokens, B, positions, table, pages_per_row, temp, k, p, u, ids, logits=None):
    _check(h, lib().llm_step_paged_dev(h, _ptr(tokens), B, _ptr(positions), _ptr(table), pages_per_row, temp, k,
                                       p, _ptr(u), _ptr(ids), _ptr(logits)))


def llm_prefill_packed(h, tokens, rows, positions, segments, P, last, nlast, logits):
    _check(h, lib().llm_prefill_packed(h, _ptr(tokens), _ptr(rows), _ptr(positions), _ptr(segments), P,
                                       _ptr(last), nlast, _ptr(logits)))


def llm_verify_step(h, tokens, B, S, positions, temp, q, u, p, ids, accepted):
    _check(h, lib().llm_verify_step(h, _ptr(tokens), B, S, _ptr(positions), temp, _ptr(q), _ptr(u), _ptr(p),
                                    _ptr(ids), _ptr(accepted)))


def llm_copy_pages(h, moves, m):
    _check(h, lib().llm_copy_pages(h, _ptr(moves), m))


def llm_synchronize(h):
    _check(h, lib().llm_synchronize(h))


def llm_stream(h) -> int:
    return lib().llm_stream(h) or 0


def llm_logits_buffer(h) -> int:
    return lib().llm_logits_buffer(h)


def llm_filled(h, b) -> int:
    return int(lib().llm_filled(h, b))


def llm_kv_import(h, layer, row, pos0, k, v):
    n = k.shape[1]
    _check(h, lib().llm_kv_import(h, layer, row, pos0, n, _ptr(k), _ptr(v)))


def llm_kv_export(h, layer, row, pos0, k, v):
    n = k.shape[1]
    _check(h, lib().llm_kv_export(h, layer, row, pos0, n, _ptr(k), _ptr(v)))


def llm_debug_trace(h, layer, name, dst):
    _check(h, lib().llm_debug_trace(h, layer, name.encode(), _ptr(dst)))


KERNELS = {"qkv": 0, "attention": 1, "o_proj": 2, "gate_up": 3, "down": 4, "lm_head": 5, "sampler": 6}


def llm_profile_kernel(h, which, B, pos, reps) -> float:
    ms = ctypes.c_float()
    _check(h, lib().llm_profile_kernel(h, which, B, pos, reps, ctypes.byref(ms)))
    return float(ms.value)


def llm_step_kernels(h, B, temp, k=1 << 30) -> int:
    n = ctypes.c_int32()
    _check(h, lib().llm_step_kernels(h, B, temp, k, ctypes.byref(n)))
    return int(n.value)


def llm_check_wait_timeout(h, limit_cycles):
    _check(h, lib().llm_check_wait_timeout(h, limit_cycles))


SAMPLE_NOALLOC_MAX_ELEMS = 262144


def llm_sample_noalloc(logits, B, V, temp, k, p, u, ids, stream=None):
    """Sampling on device buffers with no handle and no allocation (see include/llm.h): for
    callers that cannot allocate device memory.  B * (V rounded up to 32) <= 262144."""
    st = lib().llm_sample_noalloc(_ptr(logits), B, V, temp, k, p, _ptr(u), _ptr(ids), stream)
    if st != LLM_OK:
        raise LlmError(st, f"llm_sample_noalloc: {lib().llm_status_string(st).decode()}")


# ---- operators on torch CUDA tensors, without a handle (include/llm.h) --------------------
# Shapes, types, contiguity and the device are checked here; the library checks the rest.  A call on
# small tensors is bound by this host code, so the checks read plain attributes and build no text.

_torch = None


def _need_torch():
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _refused(name, st):
    why = lib().llm_last_error(None)
    raise LlmError(st, f"{name}: {lib().llm_status_string(st).decode()}: {why.decode() if why else ''}")


def _bad(what):
    raise LlmError(LLM_ERR_ARG, what)


def _int32(t, name, dev, n):
    """The address of a contiguous int32 tensor of n elements on CUDA device dev (None: 0)."""
    if t is None:
        return None
    if t.dtype is not _torch.int32 or t.get_device() != dev or t.numel() != n or not t.is_contiguous():
        _bad(f"{name} must be a contiguous int32 tensor of {n} elements on cuda:{dev}")
    return t.data_ptr()


def _rows(t, name, dev, B, S, width):
    """Token rows [B, S, heads, head] (or [B, S, heads * head]): the address and the distance between
    tokens in elements; rows of a wider tensor may be given as a slice."""
    shape, st = t.shape, t.stride()
    if t.get_device() != dev or len(shape) not in (3, 4) or shape[0] != B or shape[1] != S or t.numel() != B * S * width:
        _bad(f"{name} must hold {B} x {S} rows of {width} elements on cuda:{dev}, not {tuple(shape)}")
    # (the stride of a dimension of size 1 carries no meaning)
    step = st[1] if S > 1 else st[0] if B > 1 else width
    if st[-1] != 1 or (len(shape) == 4 and shape[2] > 1 and st[2] != shape[3]) or (B > 1 and S > 1 and st[0] != S * step):
        _bad(f"{name}: the elements of a row must be contiguous and the rows evenly spaced")
    return t.data_ptr(), step


def _stream(stream, dev):
    return _torch.cuda.current_stream(dev).cuda_stream if stream is None else stream


class QCache:
    """An 8-bit key/value cache over torch tensors: codes k, v [rows, kv_heads, max_seq, head]
    (uint8 or float8_e4m3fn) and scales [rows, kv_heads, max_seq // 16] (float32), all zeroed before
    their first use.  The tensors stay the caller's; calls are ordered on `stream` (a cudaStream_t,
    None: torch's current stream) and return without waiting.  `pos`, `length`, `count` [B] and
    `table` [B, pages] are int32 CUDA tensors, `status` one int32; rows of tokens are f32 or bf16."""

    def __init__(self, k, v, k_scale, v_scale):
        torch = _need_torch()
        if k.dim() != 4 or not k.is_cuda:
            _bad("k must be codes [rows, kv_heads, max_seq, head] in CUDA memory")
        rows, kv, cap, hd = k.shape
        for t, name in ((k, "k"), (v, "v")):
            if t.dtype not in (torch.uint8, torch.float8_e4m3fn) or not t.is_contiguous() or t.device != k.device or t.shape != k.shape:
                _bad(f"{name} must be contiguous codes [rows, kv_heads, max_seq, head] (uint8 or float8_e4m3fn)")
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if tuple(t.shape) != (rows, kv, cap // 16) or t.dtype != torch.float32 or not t.is_contiguous() or t.device != k.device:
                _bad(f"{name} must be contiguous float32 [rows, kv_heads, max_seq // 16] beside the codes")
        self.tensors = (k, v, k_scale, v_scale)  # kept alive with the addresses below
        self.device, self.kv, self.hd = k.device, kv, hd
        self._dev, self._scale = k.get_device(), hd ** -0.5
        self.c = LlmQcache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), rows, kv, cap, hd)
        self._c, self._lib = ctypes.byref(self.c), lib()
        self._f32, self._bf16 = torch.float32, torch.bfloat16

    @classmethod
    def empty(cls, rows, kv_heads, max_seq, head, device="cuda"):
        """A zeroed cache in new tensors."""
        torch = _need_torch()
        code = lambda: torch.zeros(rows, kv_heads, max_seq, head, dtype=torch.uint8, device=device)  # noqa: E731
        scale = lambda: torch.zeros(rows, kv_heads, max_seq // 16, device=device)  # noqa: E731
        return cls(code(), code(), scale(), scale())

    def _dtype(self, a, b):
        t = a.dtype
        if b.dtype is not t or (t is not self._f32 and t is not self._bf16):
            _bad("rows must be f32 or bf16, all of one type")
        return LLM_DTYPE_F32 if t is self._f32 else LLM_DTYPE_BF16

    def _call_rows(self, B, first, name, count, table, status):
        """Addresses of positions (or lengths), counts, pages and the status word, and the pages per row."""
        dev = self._dev
        if _torch.cuda.current_device() != dev:
            _bad(f"the cache lies on cuda:{dev} and another CUDA device is current")
        if first is None:
            _bad(f"{name} is missing")
        pages = 0
        if table is not None:
            if table.dim() != 2 or table.shape[0] != B:
                _bad(f"table must be [{B}, pages]")
            pages = table.shape[1]
        return (_int32(first, name, dev, B), None if count is None else _int32(count, "count", dev, B),
                None if table is None else _int32(table, "table", dev, B * pages), pages,
                None if status is None else _int32(status, "status", dev, 1))

    def write(self, k, v, pos, count=None, table=None, status=None, stream=None):
        """Keys and values [B, S, kv_heads, head] at positions pos[b] + i of row b (llm_qcache_write)."""
        B, S = k.shape[:2]
        first, count, table, pages, status = self._call_rows(B, pos, "pos", count, table, status)
        width = self.kv * self.hd
        kp, step = _rows(k, "k", self._dev, B, S, width)
        vp, vstep = _rows(v, "v", self._dev, B, S, width)
        if step != vstep:
            _bad("k and v must have the same row stride")
        st = self._lib.llm_qcache_write(self._c, kp, vp, self._dtype(k, v), step, B, S, first, count, table, pages, status,
                                        _stream(stream, self._dev))
        if st != LLM_OK:
            _refused("llm_qcache_write", st)

    def read(self, pos, k, v, count=None, table=None, status=None, stream=None):
        """Positions pos[b] + i of row b into k and v [B, S, kv_heads, head] (llm_qcache_read)."""
        B, S = k.shape[:2]
        first, count, table, pages, status = self._call_rows(B, pos, "pos", count, table, status)
        width = self.kv * self.hd
        kp, step = _rows(k, "k", self._dev, B, S, width)
        vp, vstep = _rows(v, "v", self._dev, B, S, width)
        if step != vstep:
            _bad("k and v must have the same row stride")
        st = self._lib.llm_qcache_read(self._c, B, S, first, count, table, pages, kp, vp, self._dtype(k, v), step, status,
                                       _stream(stream, self._dev))
        if st != LLM_OK:
            _refused("llm_qcache_read", st)

    def workspace(self, group, B, S):
        """A zeroed workspace for attend() with this group, rows and tokens per row."""
        if _torch.cuda.current_device() != self._dev:
            _bad(f"the cache lies on cuda:{self._dev} and another CUDA device is current")
        n = ctypes.c_uint64()
        st = self._lib.llm_qcache_workspace(self._c, group, B, S, ctypes.byref(n))
        if st != LLM_OK:
            _refused("llm_qcache_workspace", st)
        return _torch.zeros(max(16, n.value), dtype=_torch.uint8, device=self.device)

    def attend(self, q, length, out, workspace, count=None, table=None, scale=None, status=None, stream=None):
        """Attention of q [B, S, heads, head] over the first length[b] positions of row b, the tokens
        themselves being the last of them, into out (llm_qcache_attend); scale defaults to
        head ** -0.5."""
        B, S = q.shape[:2]
        per = self.kv * self.hd
        n = q.numel()
        group = n // (B * S * per) if B * S else 0
        if n != B * S * group * per:
            _bad("q must hold a whole number of heads per key/value head")
        first, count, table, pages, status = self._call_rows(B, length, "length", count, table, status)
        qp, qstep = _rows(q, "q", self._dev, B, S, group * per)
        op, ostep = _rows(out, "out", self._dev, B, S, group * per)
        if workspace.get_device() != self._dev or not workspace.is_contiguous():
            _bad("workspace must be contiguous CUDA memory beside the cache")
        st = self._lib.llm_qcache_attend(self._c, qp, self._dtype(q, out), qstep, group, B, S, first, count, table, pages,
                                         self._scale if scale is None else scale, op, ostep, workspace.data_ptr(),
                                         workspace.numel() * workspace.element_size(), status,
                                         _stream(stream, self._dev))
        if st != LLM_OK:
            _refused("llm_qcache_attend", st)


    def workspace_shared(self, group, B, S, groups):
        """A workspace for attend_shared() with this group, rows, tokens per row and groups of rows."""
        if _torch.cuda.current_device() != self._dev:
            _bad(f"the cache lies on cuda:{self._dev} and another CUDA device is current")
        n = ctypes.c_uint64()
        st = self._lib.llm_qcache_shared_workspace(self._c, group, B, S, groups, ctypes.byref(n))
        if st != LLM_OK:
            _refused("llm_qcache_shared_workspace", st)
        return _torch.empty(max(16, n.value), dtype=_torch.uint8, device=self.device)

    def attend_shared(self, q, length, groups, shared, out, workspace, count=None, table=None, scale=None, status=None,
                      stream=None):
        """attend() for rows that share places: rows groups[i] .. groups[i + 1] - 1 take their positions below
        shared[i] from the places of the group's first row, which are read once for many of them where that pays by B, S, the
        number of groups and the table's width (llm_qcache_attend_shared; with as many groups as rows it is not).  groups [G + 1] and shared [G] are int32 CUDA tensors."""
        B, S = q.shape[:2]
        per = self.kv * self.hd
        n = q.numel()
        group = n // (B * S * per) if B * S else 0
        if n != B * S * group * per:
            _bad("q must hold a whole number of heads per key/value head")
        first, count, table, pages, status = self._call_rows(B, length, "length", count, table, status)
        if shared is None or groups is None:
            _bad("groups and shared are missing")
        G = shared.numel()
        dev = self._dev
        bound, part = _int32(groups, "groups", dev, G + 1), _int32(shared, "shared", dev, G)
        qp, qstep = _rows(q, "q", dev, B, S, group * per)
        op, ostep = _rows(out, "out", dev, B, S, group * per)
        if workspace.get_device() != dev or not workspace.is_contiguous():
            _bad("workspace must be contiguous CUDA memory beside the cache")
        st = self._lib.llm_qcache_attend_shared(self._c, qp, self._dtype(q, out), qstep, group, B, S, first, count, table, pages,
                                                bound, part, G, self._scale if scale is None else scale, op, ostep,
                                                workspace.data_ptr(), workspace.numel() * workspace.element_size(), status,
                                                _stream(stream, dev))
        if st != LLM_OK:
            _refused("llm_qcache_attend_shared", st)


class QCacheLayers:
    """The 8-bit caches of a model's layers, all of one shape (QCache), whose pages are copied together."""

    def __init__(self, caches):
        caches = list(caches)
        if not caches:
            _bad("at least one cache is needed")
        if any(c._dev != caches[0]._dev for c in caches):
            _bad("the caches must lie on one device")
        self.caches = caches
        self._dev, self._lib = caches[0]._dev, lib()
        self._array = (LlmQcache * len(caches))(*[c.c for c in caches])

    def copy(self, moves, counts=None, status=None, stream=None):
        """Copy pages moves[i][0] to moves[i][1] in every layer (llm_qcache_copy_pages): moves [m, 2] and counts (the
        first of its elements: how many of them there are) int32 CUDA tensors, as Pages.update and compact write them."""
        dev = self._dev
        if _torch.cuda.current_device() != dev:
            _bad(f"the caches lie on cuda:{dev} and another CUDA device is current")
        m = moves.shape[0] if moves.dim() == 2 else -1
        if m == 0:
            return
        st = self._lib.llm_qcache_copy_pages(self._array, len(self.caches), _int32(moves, "moves", dev, 2 * m), m,
                                             None if counts is None else _int32(counts, "counts", dev, 2),
                                             None if status is None else _int32(status, "status", dev, 1), _stream(stream, dev))
        if st != LLM_OK:
            _refused("llm_qcache_copy_pages", st)


class Pages:
    """A page table [rows, pages_per_row] and lengths [rows] (int32 CUDA tensors) over a pool of `pages`
    pages of 64 positions (llm_pages).  update and compact write what becomes of it into another Pages of
    the same shape; calls are ordered on `stream` (None: torch's current stream) and return without waiting."""

    def __init__(self, table, length, pages):
        torch = _need_torch()
        for t, name in ((table, "table"), (length, "length")):
            if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
                _bad(f"{name} must be a contiguous int32 tensor in CUDA memory")
        if table.dim() != 2 or tuple(length.shape) != (table.shape[0],) or length.device != table.device:
            _bad("table must be [rows, pages_per_row] and length [rows] beside it")
        self.table, self.length, self.pages = table, length, int(pages)
        self._dev = table.get_device()
        self.c = LlmPages(table.data_ptr(), length.data_ptr(), table.shape[0], table.shape[1], self.pages)
        self._c, self._lib = ctypes.byref(self.c), lib()

    @classmethod
    def empty(cls, rows, pages_per_row, pages, device="cuda"):
        """Rows that hold nothing."""
        torch = _need_torch()
        return cls(torch.full((rows, pages_per_row), -1, dtype=torch.int32, device=device),
                   torch.zeros(rows, dtype=torch.int32, device=device), pages)

    def workspace(self):
        """A workspace for update() and compact()."""
        n = ctypes.c_uint64()
        st = self._lib.llm_pages_workspace(self._c, ctypes.byref(n))
        if st != LLM_OK:
            _refused("llm_pages_workspace", st)
        return _torch.empty(n.value // 4, dtype=_torch.int32, device=self.table.device)

    def _call(self, out, moves, m, counts, workspace, status):
        dev = self._dev
        if _torch.cuda.current_device() != dev:
            _bad(f"the table lies on cuda:{dev} and another CUDA device is current")
        if out._dev != dev or workspace.get_device() != dev or not workspace.is_contiguous():
            _bad("out and workspace must lie beside the table, the workspace contiguous")
        if moves is None or counts is None:
            _bad("moves and counts are missing")
        return (_int32(moves, "moves", dev, 2 * m), _int32(counts, "counts", dev, 2), workspace.data_ptr(),
                workspace.numel() * workspace.element_size(), None if status is None else _int32(status, "status", dev, 1))

    def update(self, out, moves, counts, workspace, parent=None, length=None, status=None, stream=None):
        """Row r of out becomes the first length[r] positions of row parent[r] of this table (parent -1: empty;
        None: every row its own; length None: the parent's), with pages for positions it does not hold yet.
        moves [rows, 2] receives the pages to copy (QCacheLayers.copy), counts [2] their number and the
        pages in use (llm_pages_update)."""
        moves, counts, ws, n, status = self._call(out, moves, self.c.rows, counts, workspace, status)
        st = self._lib.llm_pages_update(self._c, out._c, None if parent is None else _int32(parent, "parent", self._dev, self.c.rows),
                                        None if length is None else _int32(length, "length", self._dev, self.c.rows), moves, counts,
                                        ws, n, status, _stream(stream, self._dev))
        if st != LLM_OK:
            _refused("llm_pages_update", st)

    def compact(self, out, moves, counts, workspace, status=None, stream=None):
        """The pages in use as numbers 0 .. used - 1 in out; moves [max(1, pages // 2), 2] and counts as
        for update (llm_pages_compact)."""
        moves, counts, ws, n, status = self._call(out, moves, max(1, self.pages // 2), counts, workspace, status)
        st = self._lib.llm_pages_compact(self._c, out._c, moves, counts, ws, n, status, _stream(stream, self._dev))
        if st != LLM_OK:
            _refused("llm_pages_compact", st)


def _f32s(t, name, dev, n):
    if t.dtype is not _torch.float32 or t.get_device() != dev or t.numel() != n or not t.is_contiguous():
        _bad(f"{name} must be a contiguous float32 tensor of {n} elements on cuda:{dev}")
    return t.data_ptr()


def llm_verify(p, q, drafts, u, ids, accepted, count=None, stream=None):
    """Verification of drafts [B, S] against the target's probabilities p [B, S + 1, V], the draft
    model's q [B, S, V] (None: deterministic drafts) and draws u [B, S + 1], into ids [B, S + 1] and
    accepted [B] (see include/llm.h); CUDA tensors, f32 and int32; ordered on `stream` (None: torch's
    current stream)."""
    torch = _torch or _need_torch()
    if drafts.dim() != 2 or p.dim() != 3:
        _bad("drafts must be [B, S] and p [B, S + 1, V]")
    B, S = drafts.shape
    V, dev = p.shape[2], p.get_device()
    if dev < 0 or torch.cuda.current_device() != dev:
        _bad("p must lie on the current CUDA device")
    if p.shape[0] != B or p.shape[1] != S + 1 or (q is not None and tuple(q.shape) != (B, S, V)):
        _bad("p must be [B, S + 1, V] and q [B, S, V]")
    if ids is None or accepted is None or drafts is None:
        _bad("ids and accepted are missing")
    st = lib().llm_verify(_f32s(p, "p", dev, B * (S + 1) * V), None if q is None else _f32s(q, "q", dev, B * S * V),
                          _int32(drafts, "drafts", dev, B * S), None if count is None else _int32(count, "count", dev, B),
                          B, S, V, _f32s(u, "u", dev, B * (S + 1)), _int32(ids, "ids", dev, B * (S + 1)),
                          _int32(accepted, "accepted", dev, B), _stream(stream, dev))
    if st != LLM_OK:
        _refused("llm_verify", st)


def llm_sample_rows(logits, temp, u, ids, k=None, p=None, min_p=None, status=None, stream=None):
    """One token per row of logits [B, V] (rows may be a slice of wider ones), drawn with the row's own temp, k,
    p, min_p and u [B] into ids [B] (see include/llm.h); CUDA tensors, f32 and int32 (k, ids, status); temp None: 1,
    k None: V, p None: 1, min_p None: 0; ordered on `stream` (None: torch's current stream)."""
    torch = _torch or _need_torch()
    if logits.dim() != 2 or logits.dtype is not torch.float32:
        _bad("logits must be float32 [B, V]")
    B, V = logits.shape
    dev = logits.get_device()
    if dev < 0 or torch.cuda.current_device() != dev:
        _bad("logits must lie on the current CUDA device")
    step, one = logits.stride()
    if V > 1 and one != 1:
        _bad("the logits of a row must be contiguous")
    if u is None or ids is None:
        _bad("u and ids are missing")
    st = lib().llm_sample_rows(logits.data_ptr(), step if B > 1 else max(step, V), B, V, None if temp is None else _f32s(temp, "temp", dev, B),
                               None if k is None else _int32(k, "k", dev, B), None if p is None else _f32s(p, "p", dev, B),
                               None if min_p is None else _f32s(min_p, "min_p", dev, B), _f32s(u, "u", dev, B),
                               _int32(ids, "ids", dev, B), None if status is None else _int32(status, "status", dev, 1),
                               _stream(stream, dev))
    if st != LLM_OK:
        _refused("llm_sample_rows", st)


# ---- a small convenience wrapper --------------------------------------------------------

class Model:
    """One handle: host-memory entry points with numpy arrays."""

    def __init__(self, shape, weights, max_batch, max_seq, stream=None, debug_trace=False,
                 weights_on_device=False, tc_min_batch=0, max_tokens=0, step_kernel=0, cache_type=LLM_CACHE_MODEL):
        self.shape = shape
        self.cfg = config(shape, max_batch, max_seq, debug_trace, tc_min_batch, max_tokens, step_kernel, cache_type)
        self.h = llm_create(self.cfg, weights, weights_on_device, stream)
        self.V = shape.vocab
        self.cache_dtype = np.uint16 if shape.bf16 else np.float32

    def close(self):
        if self.h:
            llm_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def prefill(self, tokens, pos=0, logits=True):
        tokens = np.ascontiguousarray(tokens, np.int32)
        B, S = tokens.shape
        out = np.empty((B, self.V), np.float32) if logits else None
        llm_prefill(self.h, tokens, B, S, pos, out)
        return out

    def decode(self, tokens, pos):
        tokens = np.ascontiguousarray(tokens, np.int32).reshape(-1)
        out = np.empty((tokens.size, self.V), np.float32)
        llm_decode(self.h, tokens, tokens.size, pos, out)
        return out

    def decode_rows(self, tokens, positions):
        """One token per row, row b at its own position positions[b]."""
        tokens = np.ascontiguousarray(tokens, np.int32).reshape(-1)
        positions = np.ascontiguousarray(positions, np.int32).reshape(-1)
        assert positions.size == tokens.size
        out = np.empty((tokens.size, self.V), np.float32)
        llm_decode_rows(self.h, tokens, tokens.size, positions, out)
        return out

    def step_rows(self, tokens, positions, temp=0.0, k=1, p=1.0, u=None, logits=False):
        tokens = np.ascontiguousarray(tokens, np.int32).reshape(-1)
        positions = np.ascontiguousarray(positions, np.int32).reshape(-1)
        assert positions.size == tokens.size
        B = tokens.size
        ids = np.empty(B, np.int32)
        out = np.empty((B, self.V), np.float32) if logits else None
        u = None if u is None else np.ascontiguousarray(u, np.float32)
        llm_step_rows(self.h, tokens, B, positions, temp, k, p, u, ids, out)
        return (ids, out) if logits else ids

    def generate(self, tokens, pos, n_steps, temp=0.0, k=1, p=1.0, u=None):
        """n_steps chained decode + draw steps inside CUDA graphs; ids [n_steps][B]."""
        tokens = np.ascontiguousarray(tokens, np.int32).reshape(-1)
        B = tokens.size
        ids = np.empty((n_steps, B), np.int32)
        u = None if u is None else np.ascontiguousarray(u, np.float32).reshape(n_steps, B)
        llm_generate(self.h, tokens, B, pos, n_steps, temp, k, p, u, ids)
        return ids

    def decode_paged(self, tokens, positions, table):
        """One token per row at its own position, the cache read and written through the row's
        pages: table [B][pages_per_row] of pool pages (64 positions each)."""
        tokens = np.ascontiguousarray(tokens, np.int32).reshape(-1)
        positions = np.ascontiguousarray(positions, np.int32).reshape(-1)
        table = np.ascontiguousarray(table, np.int32)
        assert positions.size == tokens.size and table.shape[0] == tokens.size
        out = np.empty((tokens.size, self.V), np.float32)
        llm_decode_paged(self.h, tokens, tokens.size, positions, table, table.shape[1], out)
        return out

    def step_paged(self, tokens, positions, table, temp=0.0, k=1, p=1.0, u=None, logits=False):
        tokens = np.ascontiguousarray(tokens, np.int32).reshape(-1)
        positions = np.ascontiguousarray(positions, np.int32).reshape(-1)
        table = np.ascontiguousarray(table, np.int32)
        B = tokens.size
        ids = np.empty(B, np.int32)
        out = np.empty((B, self.V), np.float32) if logits else None
        u = None if u is None else np.ascontiguousarray(u, np.float32)
        llm_step_paged(self.h, tokens, B, positions, table, table.shape[1], temp, k, p, u, ids, out)
        return (ids, out) if logits else ids

    def prefill_packed(self, tokens, rows, positions, segments, last, logits=True):
        """Prompts packed end to end; logits [len(last)][V] after the tokens last names."""
        arrs = [np.ascontiguousarray(a, np.int32).reshape(-1) for a in (tokens, rows, positions, segments, last)]
        tokens, rows, positions, segments, last = arrs
        P = tokens.size
        assert rows.size == P and positions.size == P and segments.size == P
        out = np.empty((last.size, self.V), np.float32) if logits else None
        llm_prefill_packed(self.h, tokens, rows, positions, segments, P, last, last.size, out)
        return out

    def verify_step(self, tokens, positions, u, temp=0.0, q=None):
        """The last token and S drafts of each row (tokens [B][S + 1]) at positions[b] .. + S in one pass,
        verified against the model: the row's next tokens ids [B][S + 1] (the kept drafts, one drawn
        token, then -1), the drafts kept [B], and the probabilities p [B][S + 1][V].  q [B][S][V]: the
        draft model's probabilities (None: deterministic drafts); u [B][S + 1] draws."""
        import torch
        tokens = np.ascontiguousarray(tokens, np.int32)
        B, S = tokens.shape[0], tokens.shape[1] - 1
        positions = np.ascontiguousarray(positions, np.int32).reshape(-1)
        u = np.ascontiguousarray(u, np.float32)
        assert positions.size == B and u.shape == (B, S + 1) and (q is None or q.shape == (B, S, self.V))
        dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda()  # noqa: E731
        ud, qd, p = dev(u), dev(q), torch.empty(B, S + 1, self.V, device="cuda")
        ids, acc = torch.empty(B, S + 1, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()  # (the copies ran on torch's stream)
        llm_verify_step(self.h, tokens, B, S, positions, temp, qd, ud, p, ids, acc)
        self.synchronize()
        return ids.cpu().numpy(), acc.cpu().numpy(), p.cpu().numpy()

    def copy_pages(self, moves):
        """Copy pages moves[i][0] to moves[i][1] of the paged steps' pool, in every layer."""
        moves = np.ascontiguousarray(moves, np.int32).reshape(-1, 2)
        if len(moves):
            llm_copy_pages(self.h, moves, len(moves))

    def sample(self, logits, temp, k, p, u):
        logits = np.ascontiguousarray(logits, np.float32)
        B = logits.shape[0]
        ids = np.empty(B, np.int32)
        u = None if u is None else np.ascontiguousarray(u, np.float32)
        llm_sample(self.h, logits, B, temp, k, p, u, ids)
        return ids

    def step(self, tokens, pos, temp=0.0, k=1, p=1.0, u=None, logits=False):
        tokens = np.ascontiguousarray(tokens, np.int32).reshape(-1)
        B = tokens.size
        ids = np.empty(B, np.int32)
        out = np.empty((B, self.V), np.float32) if logits else None
        u = None if u is None else np.ascontiguousarray(u, np.float32)
        llm_step(self.h, tokens, B, pos, temp, k, p, u, ids, out)
        return (ids, out) if logits else ids

    def kv_import(self, layer, row, pos0, k, v):
        llm_kv_import(self.h, layer, row, pos0, np.ascontiguousarray(k, self.cache_dtype),
                      np.ascontiguousarray(v, self.cache_dtype))

    def kv_export(self, layer, row, pos0, n):
        k = np.empty((self.shape.kv, n, self.shape.hd), self.cache_dtype)
        v = np.empty_like(k)
        llm_kv_export(self.h, layer, row, pos0, k, v)
        return k, v

    def trace(self, layer, name):
        """One intermediate of the last traced step: [max_batch][width] (include/llm.h lists the
        names)."""
        w = {"swiglu": self.shape.ffn, "k": self.shape.kvw, "v": self.shape.kvw,
             "kr": self.shape.kvw}.get(name, self.shape.d)
        out = np.empty((self.cfg.max_batch, w), np.float32)
        llm_debug_trace(self.h, layer, name, out)
        return out

    def synchronize(self):
        llm_synchronize(self.h)

    def filled(self, b=0):
        return llm_filled(self.h, b)
