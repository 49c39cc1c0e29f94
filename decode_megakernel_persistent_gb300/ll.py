"""Thin ctypes binding of libll.so (the C ABI in include/ll.h).

Every function here has the name of the C entry point it calls and does only
argument marshalling: torch tensors supply device pointers and the stream, and
every step of the decode runs in the library's CUDA kernels. There is no
fallback: if libll.so is missing or fails to load, the first call raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

LL_OK = 0
LL_ERR_ARG = -1
LL_ERR_SHAPE = -2
LL_ERR_CUDA = -3
LL_ERR_DEP_TIMEOUT = -4
LL_ERR_OOM = -5
LL_ERR_DEVICE = -6
LL_ERR_NUMERIC = -7

LL_BACKEND_MEGAKERNEL = 0
LL_BACKEND_CHAIN = 1

LL_Q_NUM_SMS = 0
LL_Q_ATTN_SPLITS = 1
LL_Q_PAGE_BYTES = 2
LL_Q_NUM_PAGES = 3
LL_Q_SCRATCH_BYTES = 4
LL_Q_MAX_INSTRS = 5
LL_Q_LAUNCHES_PER_STEP = 6
LL_Q_SMEM_BYTES = 7
LL_Q_TRACE_BYTES = 8
LL_Q_MV_TC = 9
LL_Q_BATCH_CC = 12
LL_Q_BATCH = 10
LL_Q_KV_BITS = 13
LL_MAX_BATCH = 8

LL_BF16 = 0
LL_F32 = 1
LL_E4M3 = 2

LL_ROPE_PLAIN = 0
LL_ROPE_LINEAR = 1
LL_ROPE_BANDS = 2
LL_ROPE_RAMP = 3

LL_STATIC_SCRATCH_BYTES = 4194304
LL_STATIC_MAX_LAYERS = 256

LL_FAULT_NONE = 0
LL_FAULT_DROP_SIGNAL = 1

OP_QKV, OP_ATTN, OP_OPROJ, OP_GATEUP, OP_DOWN = range(5)

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libll.so")

EXPORTS = ("ll_init", "ll_init_error", "ll_decode_step", "ll_decode_step_async", "ll_decode_steps", "ll_synchronize",
           "ll_set_trace", "ll_set_timeout_ns", "ll_query", "ll_debug_inject", "ll_plan", "ll_last_error",
           "ll_free", "ll_decode_step_static", "ll_init_batch", "ll_decode_steps_batch", "ll_handle_plan",
           "ll_prefill", "ll_kvq_write", "ll_kvq_read", "ll_kvq_attention", "ll_init_kvq",
           "ll_qmat_write", "ll_qmat_read", "ll_qmat_mul", "ll_rmsnorm", "ll_rope_plan", "ll_rope", "ll_verify")


class LLError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"libll error {code}: {msg}")
        self.code = code


class ll_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "n_layers", "hidden", "n_q_heads", "n_kv_heads", "head_dim", "inter", "vocab", "max_seq",
        "tied", "backend")] + [("rms_eps", ctypes.c_float), ("rope_theta", ctypes.c_float)]


_P16 = ctypes.c_void_p
_PP16 = ctypes.POINTER(ctypes.c_void_p)
LAYER_KEYS = ("attn_norm", "wq", "wk", "wv", "wo", "mlp_norm", "wg", "wu", "wd")


class ll_weights(ctypes.Structure):
    _fields_ = [("embed", _P16), ("lm_head", _P16), ("final_norm", _P16)] + [
        (k, _PP16) for k in LAYER_KEYS]


class ll_kvq_cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_codes", "v_codes", "k_params", "v_params")] + [
        ("seq_rows", ctypes.c_int64)] + [(n, ctypes.c_int32) for n in (
            "n_seq", "n_kv_heads", "head_dim", "max_seq", "bits")]


class ll_kvq_rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p)] + [(n, ctypes.c_int64) for n in ("seq", "token", "head")]


class ll_qmat(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("params", ctypes.c_void_p)] + [(n, ctypes.c_int32) for n in ("rows", "cols", "group")]


class ll_rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride", ctypes.c_int64), ("type", ctypes.c_int32), ("group", ctypes.c_int32),
                ("scale", ctypes.c_void_p)]


class ll_rope_table(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("head_dim", "rot_dims", "interleaved")] + [
        ("size", ctypes.c_float), ("turns", ctypes.c_uint64 * 128)]


_matrix_rows_bytes = struct.Struct("@PqiiP").pack  # an ll_rows
_rows_bytes = struct.Struct("@Pqqq").pack  # an ll_kvq_rows, a fifth of the time that the ctypes object takes


_lib = None


def lib() -> ctypes.CDLL:
    """Open libll.so (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                           "(there is no CPU fallback)")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, u64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint64
    L.ll_init.argtypes = [ctypes.POINTER(ll_config), ctypes.POINTER(ll_weights), vp, vp, vp,
                          ctypes.POINTER(vp)]
    L.ll_init.restype = ctypes.c_int
    L.ll_init_error.argtypes = []
    L.ll_init_error.restype = ctypes.c_char_p
    L.ll_decode_step.argtypes = [vp, i32, i32, vp, ctypes.POINTER(i32)]
    L.ll_decode_step.restype = ctypes.c_int
    L.ll_decode_step_async.argtypes = [vp, vp, i32, vp, vp]
    L.ll_decode_step_async.restype = ctypes.c_int
    L.ll_decode_steps.argtypes = [vp, vp, i32, i32, vp, vp]
    L.ll_decode_steps.restype = ctypes.c_int
    L.ll_synchronize.argtypes = [vp]
    L.ll_synchronize.restype = ctypes.c_int
    L.ll_set_trace.argtypes = [vp, vp, ctypes.c_size_t]
    L.ll_set_trace.restype = ctypes.c_int
    L.ll_set_timeout_ns.argtypes = [vp, u64]
    L.ll_set_timeout_ns.restype = ctypes.c_int
    L.ll_query.argtypes = [vp, ctypes.c_int, ctypes.POINTER(ctypes.c_int64)]
    L.ll_query.restype = ctypes.c_int
    L.ll_debug_inject.argtypes = [vp, ctypes.c_int, ctypes.c_int, ctypes.c_int]
    L.ll_debug_inject.restype = ctypes.c_int
    L.ll_plan.argtypes = [ctypes.POINTER(ll_config), i32, vp, ctypes.c_size_t, ctypes.POINTER(i32)]
    L.ll_plan.restype = ctypes.c_int
    L.ll_last_error.argtypes = [vp]
    L.ll_last_error.restype = ctypes.c_char_p
    L.ll_free.argtypes = [vp]
    L.ll_free.restype = None
    L.ll_decode_step_static.argtypes = [ctypes.POINTER(ll_config), ctypes.POINTER(ll_weights), vp, vp, i32, i32,
                                        vp, ctypes.POINTER(i32), vp, ctypes.c_char_p, ctypes.c_size_t]
    L.ll_decode_step_static.restype = ctypes.c_int
    L.ll_init_batch.argtypes = [ctypes.POINTER(ll_config), ctypes.POINTER(ll_weights), ctypes.POINTER(vp),
                                ctypes.POINTER(vp), i32, vp, ctypes.POINTER(vp)]
    L.ll_init_batch.restype = ctypes.c_int
    L.ll_decode_steps_batch.argtypes = [vp, vp, ctypes.POINTER(i32), i32, vp, vp]
    L.ll_decode_steps_batch.restype = ctypes.c_int
    L.ll_handle_plan.argtypes = [vp, vp, ctypes.c_size_t, ctypes.POINTER(i32)]
    L.ll_handle_plan.restype = ctypes.c_int
    L.ll_prefill.argtypes = [vp, vp, i32, i32, vp, vp]
    L.ll_prefill.restype = ctypes.c_int
    # (rows: an ll_kvq_rows by reference, or its bytes)
    cachep, rowsp, err = ctypes.POINTER(ll_kvq_cache), vp, [ctypes.c_char_p, ctypes.c_size_t]
    L.ll_kvq_write.argtypes = [cachep, rowsp, rowsp, i32, i32, vp, vp, vp] + err
    L.ll_kvq_write.restype = ctypes.c_int
    L.ll_kvq_read.argtypes = [cachep, rowsp, rowsp, i32, vp, vp, vp] + err
    L.ll_kvq_read.restype = ctypes.c_int
    L.ll_kvq_attention.argtypes = [cachep, rowsp, i32, i32, vp, vp, i32, ctypes.c_float, rowsp, vp] + err
    L.ll_kvq_attention.restype = ctypes.c_int
    L.ll_init_kvq.argtypes = [ctypes.POINTER(ll_config), ctypes.POINTER(ll_weights), cachep, vp, ctypes.POINTER(vp)]
    L.ll_init_kvq.restype = ctypes.c_int
    L.ll_qmat_write.argtypes = [ctypes.POINTER(ll_qmat), vp, i32, ctypes.c_int64, vp] + err
    L.ll_qmat_write.restype = ctypes.c_int
    L.ll_qmat_read.argtypes = [ctypes.POINTER(ll_qmat), vp, i32, ctypes.c_int64, vp] + err
    L.ll_qmat_read.restype = ctypes.c_int
    L.ll_qmat_mul.argtypes = [ctypes.POINTER(ll_qmat), vp, i32, vp, vp, vp] + err
    L.ll_qmat_mul.restype = ctypes.c_int
    L.ll_rmsnorm.argtypes = [vp, vp, vp, vp, ctypes.c_float, i32, i32, vp, vp] + err
    L.ll_rmsnorm.restype = ctypes.c_int
    L.ll_rope_plan.argtypes = [ctypes.POINTER(ll_rope_table), i32, i32, i32, ctypes.c_double, i32] + 4 * [ctypes.c_double] + err
    L.ll_rope_plan.restype = ctypes.c_int
    L.ll_rope.argtypes = [ctypes.POINTER(ll_rope_table), vp, vp, i32, vp, vp, i32, i32, i32, i32, vp, vp, i32, vp] + err
    L.ll_rope.restype = ctypes.c_int
    i64 = ctypes.c_int64
    L.ll_verify.argtypes = [vp, i32, i64, i64, vp, vp, vp, i64, i64, vp, vp, i32, i32, i32, vp, vp, vp] + err
    L.ll_verify.restype = ctypes.c_int
    _lib = L
    return L


def _ptr(t) -> int:
    return 0 if t is None else int(t.data_ptr())


def _check(h, rc: int):
    if rc != LL_OK:
        raise LLError(rc, lib().ll_last_error(h).decode())


def make_config(shape, max_seq: int, backend: int = LL_BACKEND_MEGAKERNEL) -> ll_config:
    """ll_config from a shape description with the attributes of synth.ModelShape."""
    c = ll_config()
    for n in ("n_layers", "hidden", "n_q_heads", "n_kv_heads", "head_dim", "inter", "vocab"):
        setattr(c, n, int(getattr(shape, n)))
    c.max_seq = int(max_seq)
    c.tied = int(bool(shape.tied))
    c.backend = int(backend)
    c.rms_eps = float(shape.rms_eps)
    c.rope_theta = float(shape.rope_theta)
    return c


def _weights_struct(weights: dict):
    """ll_weights for a dict of CUDA bf16 tensors, plus the host arrays it points into."""
    w = ll_weights()
    w.embed = _ptr(weights["embed"])
    w.final_norm = _ptr(weights["final_norm"])
    w.lm_head = _ptr(weights.get("lm_head"))
    keep = []
    for k in LAYER_KEYS:
        arr = (ctypes.c_void_p * max(1, len(weights[k])))(*[_ptr(t) for t in weights[k]])
        keep.append(arr)
        setattr(w, k, ctypes.cast(arr, _PP16))
    return w, keep


def ll_init(cfg: ll_config, weights: dict, k_cache, v_cache, stream=None):
    """Create a handle. ``weights`` maps names to CUDA bf16 tensors (per-layer names
    to lists); ``stream`` is a torch.cuda.Stream or None for torch's current stream."""
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    w, keep = _weights_struct(weights)
    h = ctypes.c_void_p()
    rc = lib().ll_init(ctypes.byref(cfg), ctypes.byref(w), _ptr(k_cache), _ptr(v_cache),
                       ctypes.c_void_p(stream.cuda_stream), ctypes.byref(h))
    if rc != LL_OK:
        raise LLError(rc, lib().ll_init_error().decode())
    return h


def ll_decode_step(h, token: int, pos: int, logits=None) -> int:
    """Synchronous step; returns the greedy next token."""
    nxt = ctypes.c_int32(-1)
    _check(h, lib().ll_decode_step(h, int(token), int(pos), _ptr(logits), ctypes.byref(nxt)))
    return int(nxt.value)


def ll_decode_steps(h, token_dev, pos: int, n_steps: int, logits, tokens_dev) -> None:
    _check(h, lib().ll_decode_steps(h, _ptr(token_dev), int(pos), int(n_steps), _ptr(logits), _ptr(tokens_dev)))


def ll_decode_step_async(h, token_dev, pos: int, logits, next_token_dev) -> None:
    _check(h, lib().ll_decode_step_async(h, _ptr(token_dev), int(pos), _ptr(logits),
                                         _ptr(next_token_dev)))


def ll_synchronize(h) -> None:
    _check(h, lib().ll_synchronize(h))


def ll_set_trace(h, trace_dev=None) -> None:
    """Enable (a CUDA uint64/int64 tensor of LL_Q_TRACE_BYTES bytes) or disable (None) tracing."""
    nbytes = 0 if trace_dev is None else trace_dev.numel() * trace_dev.element_size()
    _check(h, lib().ll_set_trace(h, _ptr(trace_dev), nbytes))


def ll_set_timeout_ns(h, ns: int) -> None:
    _check(h, lib().ll_set_timeout_ns(h, int(ns)))


def ll_query(h, what: int) -> int:
    v = ctypes.c_int64()
    _check(h, lib().ll_query(h, int(what), ctypes.byref(v)))
    return int(v.value)


def ll_debug_inject(h, kind: int, layer: int = 0, op: int = 0) -> None:
    _check(h, lib().ll_debug_inject(h, int(kind), int(layer), int(op)))


def ll_plan(cfg: ll_config, nsm: int):
    """The schedule for `nsm` SMs as an int32 numpy array [nsm, max_instr, 7] (host only)."""
    import numpy as np
    mx = ctypes.c_int32()
    rc = lib().ll_plan(ctypes.byref(cfg), int(nsm), None, 0, ctypes.byref(mx))
    if rc != LL_OK:
        raise LLError(rc, "ll_plan rejected the configuration")
    out = np.zeros((int(nsm), mx.value, 7), dtype=np.int32)
    rc = lib().ll_plan(ctypes.byref(cfg), int(nsm), out.ctypes.data, out.size, ctypes.byref(mx))
    if rc != LL_OK:
        raise LLError(rc, "ll_plan failed")
    return out


def ll_prefill(h, tokens_dev, n: int, pos0: int, logits, next_token_dev) -> None:
    _check(h, lib().ll_prefill(h, _ptr(tokens_dev), int(n), int(pos0), _ptr(logits), _ptr(next_token_dev)))


def ll_handle_plan(h):
    """The handle's own schedule as an int32 numpy array [nsm, max_instr, 7]."""
    import numpy as np
    mx = ctypes.c_int32()
    _check(h, lib().ll_handle_plan(h, None, 0, ctypes.byref(mx)))
    nsm = ll_query(h, LL_Q_NUM_SMS)
    out = np.zeros((nsm, mx.value, 7), dtype=np.int32)
    _check(h, lib().ll_handle_plan(h, out.ctypes.data, out.size, ctypes.byref(mx)))
    return out


def ll_decode_step_static(cfg: ll_config, weights: dict, k_cache, v_cache, token: int, pos: int,
                          logits=None, stream=None) -> int:
    """One decode step without a handle and without device allocation; returns the
    greedy next token. ``stream`` is a torch.cuda.Stream or None for torch's current one."""
    import torch
    check_static_args(cfg, weights, k_cache, v_cache, logits)
    if stream is None:
        stream = torch.cuda.current_stream()
    w, keep = _weights_struct(weights)
    nxt = ctypes.c_int32(-1)
    err = ctypes.create_string_buffer(256)
    rc = lib().ll_decode_step_static(ctypes.byref(cfg), ctypes.byref(w), _ptr(k_cache), _ptr(v_cache), int(token),
                                     int(pos), _ptr(logits), ctypes.byref(nxt), ctypes.c_void_p(stream.cuda_stream),
                                     err, len(err))
    del keep
    if rc != LL_OK:
        raise LLError(rc, err.value.decode())
    return int(nxt.value)


def ll_init_batch(cfg: ll_config, weights: dict, k_caches, v_caches, stream=None):
    """A batched handle: one (k, v) cache pair per sequence (lists of CUDA bf16 tensors)."""
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    w, keep = _weights_struct(weights)
    n = len(k_caches)
    kp = (ctypes.c_void_p * max(1, n))(*[_ptr(t) for t in k_caches])
    vp_ = (ctypes.c_void_p * max(1, len(v_caches)))(*[_ptr(t) for t in v_caches])
    h = ctypes.c_void_p()
    rc = lib().ll_init_batch(ctypes.byref(cfg), ctypes.byref(w), kp, vp_, int(n), ctypes.c_void_p(stream.cuda_stream),
                             ctypes.byref(h))
    if rc != LL_OK:
        raise LLError(rc, lib().ll_init_error().decode())
    return h


def ll_decode_steps_batch(h, tokens_in_dev, positions, n_steps: int, logits, tokens_dev) -> None:
    pos = (ctypes.c_int32 * max(1, len(positions)))(*[int(x) for x in positions])
    _check(h, lib().ll_decode_steps_batch(h, _ptr(tokens_in_dev), pos, int(n_steps), _ptr(logits), _ptr(tokens_dev)))


def ll_init_kvq(cfg: ll_config, weights: dict, cache: "KVQCache", stream=None):
    """A handle whose KV cache is packed: ``cache`` has the model's layers as its sequences."""
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    w, keep = _weights_struct(weights)
    h = ctypes.c_void_p()
    rc = lib().ll_init_kvq(ctypes.byref(cfg), ctypes.byref(w), cache.ref, ctypes.c_void_p(stream.cuda_stream),
                           ctypes.byref(h))
    if rc != LL_OK:
        raise LLError(rc, lib().ll_init_error().decode())
    return h


class _KVQThread(threading.local):
    """A thread's buffer for the reason of a refusal."""

    def __init__(self):
        self.err = ctypes.create_string_buffer(256)


_kvq_thread = _KVQThread()


def _kvq_call(fn, cache: "KVQCache", *args) -> None:
    """One packed-cache call on torch's current stream of the cache's device. (A call's GPU
    work takes a few microseconds, so its checks here are kept to as few lookups as
    they need.)"""
    index, torch_c = cache.index, cache.torch_c
    if index != torch_c._cuda_getDevice():
        import torch
        with torch.cuda.device(index):
            return _kvq_call(fn, cache, *args)
    err = _kvq_thread.err
    rc = fn(cache.ref, *args, torch_c._cuda_getCurrentRawStream(index), err, 256)
    if rc != LL_OK:
        raise LLError(rc, err.value.decode())


def ll_kvq_write(cache: "KVQCache", k, v, lens, n_toks=None) -> None:
    """Quantise k and v [n_seq, n_tok, n_kv_heads, head_dim] (bf16 or fp32, any strides
    but the last) into ``cache`` as the last tokens of sequences ``lens`` long."""
    dtype = getattr(k, "dtype", None)
    if dtype not in cache.in_types:
        raise LLError(LL_ERR_ARG, f"k must be bfloat16 or float32, not {dtype}")
    kr, n_tok = cache._rows(k, "k", dtype, cache.n_kv_heads)
    vr, _ = cache._rows(v, "v", dtype, cache.n_kv_heads, n_tok)
    _kvq_call(cache.lib.ll_kvq_write, cache, kr, vr, cache.in_types[dtype], n_tok,
              cache._lens(lens, "lens"), cache._lens(n_toks, "n_toks") if n_toks is not None else None)


def ll_kvq_read(cache: "KVQCache", k_out, v_out, lens, n_toks=None) -> None:
    """The last tokens' rows of ``cache`` read back into k_out and v_out
    [n_seq, n_tok, n_kv_heads, head_dim] (bf16)."""
    kr, n_tok = cache._rows(k_out, "k_out", cache.bf16, cache.n_kv_heads, None, True)
    vr, _ = cache._rows(v_out, "v_out", cache.bf16, cache.n_kv_heads, n_tok, True)
    if kr == vr:
        raise LLError(LL_ERR_ARG, "k_out and v_out are the same rows")
    _kvq_call(cache.lib.ll_kvq_read, cache, kr, vr, n_tok, cache._lens(lens, "lens"),
              cache._lens(n_toks, "n_toks") if n_toks is not None else None)


def ll_kvq_attention(cache: "KVQCache", q, lens, n_toks=None, out=None, scale=None, max_len: int = 0):
    """Causal attention of the last tokens' queries q [n_seq, n_tok, n_q_heads, head_dim]
    (bf16) over ``cache``; out like q (made if None: rows of padded tokens then hold zeros)."""
    if getattr(q, "ndim", 0) != 4:
        raise LLError(LL_ERR_ARG, "q must be [n_seq, n_tok, n_q_heads, head_dim]")
    heads = q.shape[2]
    qr, n_tok = cache._rows(q, "q", cache.bf16, heads)
    if scale is None:
        scale = 0.0
    elif not ctypes.c_float(scale).value > 0:  # (as the call gets it: a smaller one would be 0, the default)
        raise LLError(LL_ERR_ARG, f"scale must be positive in fp32, not {scale}")
    lp, np_ = cache._lens(lens, "lens"), cache._lens(n_toks, "n_toks") if n_toks is not None else None
    if out is None:
        import torch
        out = (torch.zeros if np_ else torch.empty)(q.shape, dtype=q.dtype, device=q.device)
    o, _ = cache._rows(out, "out", cache.bf16, heads, n_tok, True)
    _kvq_call(cache.lib.ll_kvq_attention, cache, qr, heads, n_tok, lp, np_, max_len, scale, o)
    return out


_codes = {}  # torch's dtypes by the library's


class _Types:
    """torch's dtypes, and what every call looks up, found once."""

    @classmethod
    def get(cls) -> dict:
        if not _codes:
            import torch
            cls.bf16, cls.f32, cls.e4m3, cls.int32 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int32
            cls.torch, cls.lib = torch, lib()
            cls.device, cls.stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
            _codes.update({torch.bfloat16: LL_BF16, torch.float32: LL_F32, torch.float8_e4m3fn: LL_E4M3})
        return _codes


def _device_call(fn, index: int, *args) -> None:
    """One call without a handle on torch's current stream of device `index`."""
    types = _Types
    if index != types.device():
        with types.torch.cuda.device(index):
            return _device_call(fn, index, *args)
    err = _kvq_thread.err
    rc = fn(*args, types.stream(index), err, 256)
    if rc:
        raise LLError(rc, err.value.decode())


def _matrix_rows(t, name: str, shape, index: int, scale: int = 0, group: int = 0) -> bytes:
    """t (of this shape [n, width], on device `index`) as an ll_rows' bytes. (The library checks types and
    strides, which it sees. A small call's GPU work takes two microseconds, so what is right is passed by as few lookups
    as show it; the rest finds the reason.)"""
    try:
        if t.get_device() == index and t.shape == shape:
            stride, last = t.stride()
            if last == 1 or shape[1] <= 1:
                return _matrix_rows_bytes(t.data_ptr(), stride, _codes[t.dtype], group, scale)
    except (AttributeError, KeyError):
        pass
    if not getattr(t, "is_cuda", False) or t.get_device() != index:
        raise LLError(LL_ERR_ARG, f"{name} must be a CUDA tensor" + (f" on cuda:{index}" if index >= 0 else ""))
    if t.dtype not in _codes:
        raise LLError(LL_ERR_ARG, f"{name} must not be {t.dtype}")
    if t.shape != shape:
        raise LLError(LL_ERR_ARG, f"{name} is {tuple(t.shape)}, the call needs {list(shape)}")
    raise LLError(LL_ERR_ARG, f"{name}'s last dim must be contiguous")


def _array(t, name: str, dtype, shape, index: int) -> int:
    """The address of a contiguous tensor of this type and shape on device `index`."""
    try:
        if t.get_device() == index and t.dtype == dtype and t.shape == shape and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    raise LLError(LL_ERR_ARG, f"{name} must be a contiguous {dtype} tensor {list(shape)} on cuda" + (f":{index}" if index >= 0 else ""))


def _scales(scale, name: str, n: int, width: int, index: int):
    """The group (0: the row) that the scales [n, groups] of e4m3 rows stand for."""
    if not getattr(scale, "is_cuda", False) or scale.get_device() != index or scale.dtype != _Types.f32 or scale.dim() != 2 or not scale.is_contiguous():
        raise LLError(LL_ERR_ARG, f"{name} must be a contiguous float32 tensor [{n}, groups] on cuda:{index}")
    tiles = (width + 127) // 128
    if scale.shape not in ((n, 1), (n, tiles)):
        raise LLError(LL_ERR_ARG, f"{name} is {tuple(scale.shape)}, the call needs [{n}, 1] or [{n}, {tiles}]")
    return 128 if scale.shape[1] == tiles and tiles > 1 else 0


def ll_qmat_write(m: "Q4Matrix", w) -> None:
    """Quantise w [rows, cols] (bf16 or fp32) into the matrix."""
    _matrix_rows(w, "w", (m.rows, m.cols), m.index)
    _kvq_call(m.lib.ll_qmat_write, m, w.data_ptr(), _codes[w.dtype], w.stride(0))


def ll_qmat_read(m: "Q4Matrix", out=None, dtype=None):
    """The matrix's values [rows, cols], each rounded once to bf16 (or fp32)."""
    if out is None:
        out = _Types.torch.empty(m.rows, m.cols, dtype=dtype or _Types.bf16, device=m.device)
    _matrix_rows(out, "out", (m.rows, m.cols), m.index)
    _kvq_call(m.lib.ll_qmat_read, m, out.data_ptr(), _codes[out.dtype], out.stride(0))
    return out


def ll_qmat_mul(m: "Q4Matrix", x, scale=None, add=None, out=None, out_dtype=None):
    """x [n, cols] times the matrix's transpose (+ add [n, rows]): [n, rows]. x is bf16, fp32, or
    float8_e4m3fn with ``scale`` (fp32 [n, 1] or [n, ceil(cols / 128)]); out like add, or of
    ``out_dtype`` (bf16 if None). out may be add."""
    index = m.index
    if getattr(x, "ndim", 0) != 2:
        raise LLError(LL_ERR_ARG, "x must be [n, cols]")
    n, cols = x.shape
    if x.dtype == _Types.e4m3:
        if scale is None:
            raise LLError(LL_ERR_ARG, "x in float8_e4m3fn needs its scales")
        group = _scales(scale, "scale", n, m.cols, index)
        xr = _matrix_rows(x, "x", (n, m.cols), index, scale.data_ptr(), group)
    elif scale is not None:
        raise LLError(LL_ERR_ARG, f"x in {x.dtype} has no scales")
    else:
        xr = _matrix_rows(x, "x", (n, m.cols), index)
    shape = (n, m.rows)
    if out is None:
        out = _Types.torch.empty(shape, dtype=out_dtype or (add.dtype if add is not None else _Types.bf16), device=m.device)
    yr = _matrix_rows(out, "out", shape, index)
    ar = None if add is None else _matrix_rows(add, "add", shape, index)
    if out.dtype == _Types.e4m3:
        raise LLError(LL_ERR_ARG, "out must be bfloat16 or float32")
    _kvq_call(m.lib.ll_qmat_mul, m, xr, n, ar, yr)
    return out


def ll_rmsnorm(x, gain, eps: float = 1e-5, residual=None, residual_out=None, out=None, out_dtype=None, group: int = 0, scale=None):
    """RMS norm of the rows of x [n, width], with the residual's addition in front if there is
    one (residual_out: where the sum goes, residual itself if None). Returns out (of x's type, or
    ``out_dtype``); for float8_e4m3fn (out, scale), a scale for each row (group 0) or 128 columns."""
    if not getattr(x, "is_cuda", False) or x.ndim != 2:
        raise LLError(LL_ERR_ARG, "x must be a CUDA tensor [n, width]")
    types = _Types
    if not _codes:
        types.get()
    shape, index = x.shape, x.get_device()
    n, width = shape
    xr = _matrix_rows(x, "x", shape, index)
    if out is None:
        out = types.torch.empty(shape, dtype=out_dtype or x.dtype, device=x.device)
    e4m3 = getattr(out, "dtype", None) == types.e4m3
    at = 0
    if group not in (0, 128) or (group and not e4m3):
        raise LLError(LL_ERR_ARG, "group is 0, or 128 for float8_e4m3fn")
    if e4m3:
        groups = (n, (width + 127) // 128 if group else 1)
        if scale is None:
            scale = types.torch.empty(groups, dtype=types.f32, device=x.device)
        at = _array(scale, "scale", types.f32, groups, index)
    elif scale is not None:
        raise LLError(LL_ERR_ARG, f"out in {out.dtype} has no scales")
    outr = _matrix_rows(out, "out", shape, index, at, group)
    gp = _array(gain, "gain", types.bf16, (width,), index)
    rr = ro = None
    if residual is not None:
        rr = _matrix_rows(residual, "residual", shape, index)
        ro = rr if residual_out is None else _matrix_rows(residual_out, "residual_out", shape, index)
    elif residual_out is not None:
        raise LLError(LL_ERR_ARG, "residual_out needs a residual")
    _device_call(types.lib.ll_rmsnorm, index, xr, rr, ro, gp, eps, n, width, outr)
    return (out, scale) if e4m3 else out


def ll_verify(logits, drafts, u, probs=None, n_drafts=None, temperature=None, tokens=None, accepted=None):
    """Verify drafts int32 [n_seq, n_draft] against logits [n_seq, n_draft + 1, vocab] (bf16 or fp32)
    with the random numbers u [n_seq, n_draft + 1] (include/ll.h: ll_verify); n_draft may be 0.
    probs [n_seq, n_draft, vocab]: the drafts' own distribution, or None; n_drafts int32 [n_seq] and
    temperature fp32 [n_seq], or None. Returns tokens int32 [n_seq, n_draft + 1] (accepted drafts, the new
    token, then -1) and accepted int32 [n_seq]."""
    if not getattr(logits, "is_cuda", False) or logits.ndim != 3:
        raise LLError(LL_ERR_ARG, "logits must be a CUDA tensor [n_seq, n_draft + 1, vocab]")
    types = _Types
    if not _codes:
        types.get()
    index = logits.get_device()
    S, rows, V = logits.shape
    D = rows - 1
    code = _codes.get(logits.dtype)
    f32, int32 = types.f32, types.int32
    ls, lr, last = logits.stride()
    if code not in (LL_BF16, LL_F32) or (last != 1 and V > 1):
        raise LLError(LL_ERR_ARG, "logits must be bfloat16 or float32, contiguous in the last dim")
    if tokens is None:
        tokens = types.torch.empty((S, rows), dtype=int32, device=logits.device)
    if accepted is None:
        accepted = types.torch.empty((S,), dtype=int32, device=logits.device)
    dp = _array(drafts, "drafts", int32, (S, D), index) if D or drafts is not None else None
    up = _array(u, "u", f32, (S, rows), index)
    tp, ap = _array(tokens, "tokens", int32, (S, rows), index), _array(accepted, "accepted", int32, (S,), index)
    np_ = _array(n_drafts, "n_drafts", int32, (S,), index) if n_drafts is not None else None
    temp = _array(temperature, "temperature", f32, (S,), index) if temperature is not None else None
    pp, ps, pr = None, 0, 0
    if probs is not None:
        if not getattr(probs, "is_cuda", False) or probs.get_device() != index or probs.dtype != f32 or probs.shape != (S, D, V) or (V > 1 and probs.stride(2) != 1):
            raise LLError(LL_ERR_ARG, f"probs must be a float32 tensor {[S, D, V]} on cuda:{index}, contiguous in the last dim")
        pp, ps, pr = probs.data_ptr(), probs.stride(0), probs.stride(1)
    _device_call(types.lib.ll_verify, index, logits.data_ptr(), code, ls, lr, dp, np_, pp, ps, pr, up, temp, S, D, V, tp, ap)
    return tokens, accepted


def ll_last_error(h) -> str:
    return lib().ll_last_error(h).decode()


def ll_free(h) -> None:
    if h:
        lib().ll_free(h)


def _need(t, name: str, dtype, min_numel: int, device, optional: bool = True) -> None:
    """The library takes raw device pointers and cannot see a buffer's size, so
    the buffers a step writes or reads are checked here: a CUDA tensor of the
    right dtype on the decoder's device, contiguous, with room for min_numel
    elements (raises LLError(LL_ERR_ARG) before anything is launched)."""
    if t is None:
        if optional:
            return
        raise LLError(LL_ERR_ARG, f"{name} is required")
    if not getattr(t, "is_cuda", False):
        raise LLError(LL_ERR_ARG, f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise LLError(LL_ERR_ARG, f"{name} must be {dtype}, not {t.dtype}")
    if device is not None and t.device != device:
        raise LLError(LL_ERR_ARG, f"{name} is on {t.device}, the decoder on {device}")
    if not t.is_contiguous():
        raise LLError(LL_ERR_ARG, f"{name} must be contiguous")
    if t.numel() < min_numel:
        raise LLError(LL_ERR_ARG, f"{name} holds {t.numel()} elements, the call needs {min_numel}")


def check_weights(shape, weights: dict) -> None:
    """The weights a handle will read, against the shape: every tensor a contiguous
    CUDA bf16 tensor on the embedding's device with exactly the elements of its
    matrix or vector, per-layer lists n_layers long (raises LLError(LL_ERR_ARG)
    naming the first misfit)."""
    import torch
    H, V, I, L = int(shape.hidden), int(shape.vocab), int(shape.inter), int(shape.n_layers)
    q, kv = int(shape.n_q_heads) * int(shape.head_dim), int(shape.n_kv_heads) * int(shape.head_dim)
    dev = getattr(weights.get("embed"), "device", None)

    def exact(t, name, n):
        _need(t, name, torch.bfloat16, n, dev, optional=False)
        if t.numel() != n:
            raise LLError(LL_ERR_ARG, f"{name} holds {t.numel()} elements, the shape has {n}")

    exact(weights.get("embed"), "embed", V * H)
    exact(weights.get("final_norm"), "final_norm", H)
    if not shape.tied:
        exact(weights.get("lm_head"), "lm_head", V * H)
    per_layer = {"attn_norm": H, "wq": q * H, "wk": kv * H, "wv": kv * H, "wo": H * q,
                 "mlp_norm": H, "wg": I * H, "wu": I * H, "wd": H * I}
    for key, n in per_layer.items():
        ts = weights.get(key)
        if ts is None or len(ts) != L:
            raise LLError(LL_ERR_ARG, f"{key} must list one tensor per layer ({L})")
        for i, t in enumerate(ts):
            exact(t, f"{key}[{i}]", n)


def check_model(shape, weights: dict, k_cache, v_cache, max_seq: int) -> None:
    """check_weights, and the caches ll_init will read: contiguous CUDA bf16 tensors
    on the embedding's device with room for [n_layers][n_kv_heads][max_seq][head_dim]
    (raises LLError(LL_ERR_ARG))."""
    import torch
    check_weights(shape, weights)
    dev = getattr(weights.get("embed"), "device", None)
    cache = int(shape.n_layers) * int(shape.n_kv_heads) * int(shape.head_dim) * int(max_seq)
    _need(k_cache, "k_cache", torch.bfloat16, cache, dev, optional=False)
    _need(v_cache, "v_cache", torch.bfloat16, cache, dev, optional=False)


def check_static_args(cfg: ll_config, weights: dict, k_cache, v_cache, logits) -> None:
    """What ll_decode_step_static will read and write, against cfg: one tensor per
    layer in every per-layer list (the C side walks n_layers entries of each),
    every weight of its exact size, caches with room for
    [n_layers][n_kv_heads][max_seq][head_dim], logits (if given) with room for
    vocab floats, all on one device, and that device torch's current one, which
    the library sets up from cudaGetDevice (raises LLError(LL_ERR_ARG))."""
    import types

    import torch
    L = int(cfg.n_layers)
    for key in LAYER_KEYS:
        ts = weights.get(key)
        if ts is None or len(ts) != L:
            raise LLError(LL_ERR_ARG, f"{key} must list one tensor per layer ({L})")
    shape = types.SimpleNamespace(**{n: int(getattr(cfg, n)) for n in (
        "n_layers", "hidden", "n_q_heads", "n_kv_heads", "head_dim", "inter", "vocab")}, tied=bool(cfg.tied))
    check_model(shape, weights, k_cache, v_cache, int(cfg.max_seq))
    dev = weights["embed"].device
    _need(logits, "logits", torch.float32, int(cfg.vocab), dev)
    cur = torch.device("cuda", torch.cuda.current_device())
    if dev != cur:
        raise LLError(LL_ERR_ARG, f"the tensors are on {dev}, torch's current device is {cur}")


class Decoder:
    """Owns a handle plus references to the tensors it points into. The model's
    tensors are checked at construction (check_model) and the buffers of every
    step before its library call (_need)."""

    def __init__(self, shape, weights: dict, k_cache, v_cache, max_seq: int,
                 backend: int = LL_BACKEND_MEGAKERNEL, stream=None):
        import torch
        self.handle = None
        check_model(shape, weights, k_cache, v_cache, max_seq)
        self.shape = shape
        self.weights = weights
        self.k_cache, self.v_cache = k_cache, v_cache
        self.stream = stream if stream is not None else torch.cuda.current_stream()
        self.cfg = make_config(shape, max_seq, backend)
        self.device = getattr(weights["embed"], "device", None)
        self.handle = ll_init(self.cfg, weights, k_cache, v_cache, self.stream)

    def _bufs(self, token_dev, logits, n_logits: int, out, n_out: int, out_required: bool = False) -> None:
        import torch
        V = int(self.shape.vocab)
        if token_dev is not None:
            _need(token_dev, "token_dev", torch.int32, 1, self.device, optional=False)
        _need(logits, "logits", torch.float32, n_logits * V, self.device)
        _need(out, "next-token buffer", torch.int32, n_out, self.device, optional=not out_required)

    def step(self, token: int, pos: int, logits=None) -> int:
        self._bufs(None, logits, 1, None, 0)
        return ll_decode_step(self.handle, token, pos, logits)

    def step_async(self, token_dev, pos: int, logits, next_token_dev) -> None:
        self._bufs(token_dev, logits, 1, next_token_dev, 1)
        ll_decode_step_async(self.handle, token_dev, pos, logits, next_token_dev)

    def steps(self, token_dev, pos: int, n_steps: int, logits, tokens_dev) -> None:
        n = max(int(n_steps), 0)
        self._bufs(token_dev, logits, n, tokens_dev, n, out_required=True)
        ll_decode_steps(self.handle, token_dev, pos, n_steps, logits, tokens_dev)

    def prefill(self, tokens_dev, pos0: int, logits, next_token_dev) -> None:
        """All of tokens_dev (int32 [n]) at positions pos0..pos0+n-1 in one pass;
        the last position's logits ([vocab] fp32, or None) and greedy token."""
        import torch
        n = int(tokens_dev.numel()) if tokens_dev is not None else 0
        _need(tokens_dev, "tokens_dev", torch.int32, max(n, 1), self.device, optional=False)
        _need(logits, "logits", torch.float32, int(self.shape.vocab), self.device)
        _need(next_token_dev, "next_token_dev", torch.int32, 1, self.device, optional=False)
        ll_prefill(self.handle, tokens_dev, n, pos0, logits, next_token_dev)

    def synchronize(self) -> None:
        ll_synchronize(self.handle)

    def query(self, what: int) -> int:
        return ll_query(self.handle, what)

    def close(self) -> None:
        if self.handle:
            ll_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class BatchDecoder(Decoder):
    """A batched handle (ll_init_batch) plus references to the tensors it points
    into: n sequences, one (k, v) cache pair each, share every pass over the
    weights. The model's tensors and every cache are checked at construction, the
    buffers of every launch before its library call."""

    def __init__(self, shape, weights: dict, k_caches, v_caches, max_seq: int, stream=None):
        import torch
        self.handle = None
        n = len(k_caches)
        if n not in (1, 2, 4, 8) or len(v_caches) != n:
            raise LLError(LL_ERR_ARG, "the batch must be 1, 2, 4 or 8 sequences, one (k, v) cache pair each")
        for k, v in zip(k_caches, v_caches):
            check_model(shape, weights, k, v, max_seq)
        self.n = n
        self.shape = shape
        self.weights = weights
        self.k_caches, self.v_caches = list(k_caches), list(v_caches)
        self.stream = stream if stream is not None else torch.cuda.current_stream()
        self.cfg = make_config(shape, max_seq, LL_BACKEND_MEGAKERNEL)
        self.device = getattr(weights["embed"], "device", None)
        self.handle = ll_init_batch(self.cfg, weights, self.k_caches, self.v_caches, self.stream)

    def steps_batch(self, tokens_in_dev, positions, n_steps: int, logits, tokens_dev) -> None:
        """n_steps greedy steps of every sequence in one launch: tokens_in_dev [n]
        int32, positions a host list of n first positions, logits [n_steps][n][vocab]
        fp32 or None, tokens_dev [n_steps][n] int32."""
        import torch
        if len(positions) != self.n:
            raise LLError(LL_ERR_ARG, f"{self.n} positions needed, got {len(positions)}")
        steps = max(int(n_steps), 0)
        _need(tokens_in_dev, "tokens_in_dev", torch.int32, self.n, self.device, optional=False)
        _need(logits, "logits", torch.float32, steps * self.n * int(self.shape.vocab), self.device)
        _need(tokens_dev, "tokens_dev", torch.int32, steps * self.n, self.device, optional=False)
        ll_decode_steps_batch(self.handle, tokens_in_dev, positions, n_steps, logits, tokens_dev)


class KVQDecoder(Decoder):
    """A decoder whose KV cache is packed (ll_init_kvq): ``cache`` is a KVQCache with the
    model's layers as its sequences, holding max_seq positions. Steps and prefill as
    Decoder's, one kernel per operation."""

    def __init__(self, shape, weights: dict, cache: "KVQCache", stream=None):
        import torch
        self.handle = None
        check_weights(shape, weights)
        want = (int(shape.n_layers), int(shape.n_kv_heads), int(shape.head_dim))
        if (cache.n_seq, cache.n_kv_heads, cache.head_dim) != want:
            raise LLError(LL_ERR_ARG, f"the cache is {(cache.n_seq, cache.n_kv_heads, cache.head_dim)} "
                                      f"(sequences as layers, KV heads, dims), the model {want}")
        if cache.device != weights["embed"].device:
            raise LLError(LL_ERR_ARG, f"the cache is on {cache.device}, the weights on {weights['embed'].device}")
        self.shape = shape
        self.weights = weights
        self.cache = cache
        self.stream = stream if stream is not None else torch.cuda.current_stream()
        self.cfg = make_config(shape, cache.max_seq, LL_BACKEND_CHAIN)
        self.device = weights["embed"].device
        self.handle = ll_init_kvq(self.cfg, weights, cache, self.stream)


class KVQCache:
    """A packed KV cache (the format in include/ll.h) over the caller's tensors:
    codes uint8 [n_seq, n_kv_heads, max_seq, head_dim * bits / 8] and parameters
    float16 [n_seq, n_kv_heads, max_seq, head_dim / 32, 2] of K and of V, contiguous
    within a sequence. Its calls are ll_kvq_write, ll_kvq_read and
    ll_kvq_attention; ``lens`` (int32 [n_seq], on the device) counts each sequence's positions with
    the call's own tokens as the last, ``n_toks`` (alike, or None for all) how many
    of the call's tokens each sequence has."""

    def __init__(self, k_codes, k_params, v_codes, v_params, bits: int):
        import torch
        if bits not in (4, 8):
            raise LLError(LL_ERR_SHAPE, f"bits must be 4 or 8, not {bits}")
        dev = getattr(k_codes, "device", None)
        for t, name, dtype, dims in ((k_codes, "k_codes", torch.uint8, 4), (v_codes, "v_codes", torch.uint8, 4),
                                     (k_params, "k_params", torch.float16, 5), (v_params, "v_params", torch.float16, 5)):
            if not getattr(t, "is_cuda", False):
                raise LLError(LL_ERR_ARG, f"{name} must be a CUDA tensor")
            if t.dtype != dtype or t.dim() != dims or t.device != dev:
                raise LLError(LL_ERR_ARG, f"{name} must be {dtype} of {dims} dims on {dev}")
        S, KV, M, row = k_codes.shape
        hd = row * 8 // bits
        if hd not in (64, 128) or row * 8 != hd * bits:
            raise LLError(LL_ERR_SHAPE, f"a row of {row} bytes in {bits} bits is {row * 8 / bits:g} dims: 64 or 128 are held")
        if min(S, KV, M) < 1:
            raise LLError(LL_ERR_SHAPE, "every size must be positive")
        rows = {KV * M}
        for t, name, shape in ((k_codes, "k_codes", (S, KV, M, row)), (v_codes, "v_codes", (S, KV, M, row)),
                               (k_params, "k_params", (S, KV, M, hd // 32, 2)), (v_params, "v_params", (S, KV, M, hd // 32, 2))):
            if tuple(t.shape) != shape or not t[0].is_contiguous():
                raise LLError(LL_ERR_ARG, f"{name} must be {shape}, contiguous within a sequence, not {tuple(t.shape)}")
        if S > 1:  # rows from one sequence to the next
            rows = {t.stride(0) / t[0, 0, 0].numel() for t in (k_codes, v_codes, k_params, v_params)}
            if len(rows) > 1 or min(rows) < KV * M or min(rows) % 1:
                raise LLError(LL_ERR_ARG, "the four arrays must be the same number of whole rows, at least "
                                          "n_kv_heads * max_seq, apart from sequence to sequence")
        self.k_codes, self.k_params, self.v_codes, self.v_params = k_codes, k_params, v_codes, v_params
        self.n_seq, self.n_kv_heads, self.max_seq, self.head_dim, self.bits = S, KV, M, hd, bits
        self.device = dev
        self.struct = ll_kvq_cache(_ptr(k_codes), _ptr(v_codes), _ptr(k_params), _ptr(v_params), int(rows.pop()), S, KV, hd, M,
                                   bits)
        self.ref = ctypes.byref(self.struct)
        # what every call looks up
        self.lib, self.index, self.torch_c = lib(), dev.index, torch._C
        self.bf16, self.int32 = torch.bfloat16, torch.int32
        self.in_types = {torch.bfloat16: LL_BF16, torch.float32: LL_F32}

    @classmethod
    def empty(cls, n_seq: int, n_kv_heads: int, max_seq: int, head_dim: int, bits: int, device="cuda"):
        """A cache of new tensors (all zeros)."""
        import torch
        if bits not in (4, 8) or head_dim not in (64, 128):
            raise LLError(LL_ERR_SHAPE, f"bits must be 4 or 8 and head_dim 64 or 128, not {bits} and {head_dim}")
        lead = (n_seq, n_kv_heads, max_seq)
        codes = [torch.zeros(*lead, head_dim * bits // 8, dtype=torch.uint8, device=device) for _ in range(2)]
        params = [torch.zeros(*lead, head_dim // 32, 2, dtype=torch.float16, device=device) for _ in range(2)]
        return cls(codes[0], params[0], codes[1], params[1], bits)

    def _rows(self, t, name: str, dtype, heads: int, n_tok=None, written: bool = False):
        """t as an ll_kvq_rows' bytes, and its tokens."""
        if getattr(t, "device", None) != self.device:
            raise LLError(LL_ERR_ARG, f"{name} must be a CUDA tensor on {self.device}, the cache's device")
        if t.dtype != dtype:
            raise LLError(LL_ERR_ARG, f"{name} must be {dtype}, not {t.dtype}")
        shape = t.shape
        tokens = n_tok if n_tok is not None else shape[1] if len(shape) == 4 else 0
        if shape != (self.n_seq, tokens, heads, self.head_dim):
            raise LLError(LL_ERR_ARG, f"{name} is {tuple(shape)}, the call needs "
                                      f"[{self.n_seq}, {tokens or 'n_tok'}, {heads}, {self.head_dim}]")
        seq, token, head, last = t.stride()
        if last != 1:
            raise LLError(LL_ERR_ARG, f"{name}'s last dim must be contiguous")
        if written and not t.is_contiguous():  # no two rows of an output may share memory
            reach = self.head_dim
            for stride, size in sorted(((seq, self.n_seq), (token, tokens), (head, heads))):
                if size > 1:
                    if stride < reach:
                        raise LLError(LL_ERR_ARG, f"{name} is written and its rows overlap")
                    reach += stride * (size - 1)
        return _rows_bytes(t.data_ptr(), seq, token, head), tokens

    def _lens(self, t, name: str) -> int:
        if getattr(t, "device", None) != self.device or t.dtype != self.int32 or t.shape != (self.n_seq,) or not t.is_contiguous():
            raise LLError(LL_ERR_ARG, f"{name} must be a contiguous int32 tensor [{self.n_seq}] on {self.device}")
        return t.data_ptr()

    def write(self, k, v, lens, n_toks=None) -> None:
        ll_kvq_write(self, k, v, lens, n_toks)

    def read(self, k_out, v_out, lens, n_toks=None) -> None:
        ll_kvq_read(self, k_out, v_out, lens, n_toks)

    def attention(self, q, lens, n_toks=None, out=None, scale=None, max_len: int = 0):
        return ll_kvq_attention(self, q, lens, n_toks, out, scale, max_len)


class Q4Matrix:
    """A matrix [rows, cols] in 4 bits (the format in include/ll.h) over the caller's tensors: codes uint8
    [ceil(rows / 16), ceil(cols / 128), 1024] and parameters float16 [ceil(rows / 16), ceil(cols / 128),
    128 / group, 16, 2], contiguous, with groups of 32, 64 or 128 columns. Its calls are ll_qmat_write,
    ll_qmat_read and ll_qmat_mul."""

    def __init__(self, codes, params, rows: int, cols: int):
        import torch
        dev = getattr(codes, "device", None)
        for t, name, dtype, dims in ((codes, "codes", torch.uint8, 3), (params, "params", torch.float16, 5)):
            if not getattr(t, "is_cuda", False):
                raise LLError(LL_ERR_ARG, f"{name} must be a CUDA tensor")
            if t.dtype != dtype or t.dim() != dims or t.device != dev or not t.is_contiguous():
                raise LLError(LL_ERR_ARG, f"{name} must be contiguous {dtype} of {dims} dims on {dev}")
        if rows < 1 or cols < 1:
            raise LLError(LL_ERR_SHAPE, "every size must be positive")
        per = params.shape[2]
        if per not in (1, 2, 4):
            raise LLError(LL_ERR_SHAPE, f"{per} groups to 128 columns: groups are 32, 64 or 128 wide")
        tiles = ((rows + 15) // 16, (cols + 127) // 128)
        for t, name, shape in ((codes, "codes", (*tiles, 1024)), (params, "params", (*tiles, per, 16, 2))):
            if tuple(t.shape) != shape:
                raise LLError(LL_ERR_ARG, f"{name} must be {shape} for a matrix of {rows} by {cols}, not {tuple(t.shape)}")
        self.codes, self.params = codes, params
        self.rows, self.cols, self.group = rows, cols, 128 // per
        self.device = dev
        self.struct = ll_qmat(_ptr(codes), _ptr(params), rows, cols, self.group)
        self.ref = ctypes.byref(self.struct)
        self.lib, self.index, self.torch_c = lib(), dev.index, torch._C  # what every call looks up
        _Types.get()

    @classmethod
    def empty(cls, rows: int, cols: int, group: int = 128, device="cuda"):
        """A matrix of new tensors (all zeros)."""
        import torch
        if group not in (32, 64, 128) or rows < 1 or cols < 1:
            raise LLError(LL_ERR_SHAPE, "every size must be positive, and group 32, 64 or 128")
        tiles = ((rows + 15) // 16, (cols + 127) // 128)
        return cls(torch.zeros(*tiles, 1024, dtype=torch.uint8, device=device),
                   torch.zeros(*tiles, 128 // group, 16, 2, dtype=torch.float16, device=device), rows, cols)

    @classmethod
    def quantised(cls, w, group: int = 128):
        """The matrix w [rows, cols] (bf16 or fp32, on the GPU) in 4 bits."""
        m = cls.empty(w.shape[0], w.shape[1], group, w.device)
        m.write(w)
        return m

    def write(self, w) -> None:
        ll_qmat_write(self, w)

    def read(self, out=None, dtype=None):
        return ll_qmat_read(self, out, dtype)

    def matvec(self, x, scale=None, add=None, out=None, out_dtype=None):
        return ll_qmat_mul(self, x, scale, add, out, out_dtype)


class Rope:
    """Rotary positions of head_dim-wide heads (include/ll.h: ll_rope): ``rot_dims`` of them (all if None),
    halves or interleaved pairs, frequencies from ``theta``. scaling: None, or a dict of "kind" and its values:
    "linear" (factor), "bands" (factor, low, high, length), "ramp" (factor, fast, slow, length; fast and slow
    the turns over the original length that bound the ramp). apply's lens and n_toks are as KVQCache's."""

    def __init__(self, head_dim: int, theta: float = 500000.0, rot_dims=None, interleaved: bool = False, scaling=None):
        s = dict(scaling or {"kind": "plain"})
        kind = s.pop("kind", None)
        keys = {"plain": (), "linear": ("factor",), "bands": ("factor", "low", "high", "length"), "ramp": ("factor", "fast", "slow", "length")}
        if kind not in keys or set(s) != set(keys[kind]):
            raise LLError(LL_ERR_ARG, f"scaling {scaling} is not one of " + ", ".join(f"{k} {v}" for k, v in keys.items()))
        if kind == "ramp":
            s["low"], s["high"] = s.pop("slow"), s.pop("fast")
        self.table = ll_rope_table()
        self.ref = ctypes.byref(self.table)
        self.lib, self.head_dim = lib(), head_dim
        self.codes = {t: code for t, code in _Types.get().items() if code != LL_E4M3}
        err = ctypes.create_string_buffer(256)
        rc = self.lib.ll_rope_plan(self.ref, head_dim, head_dim if rot_dims is None else rot_dims, int(interleaved), theta,
                                   list(keys).index(kind), s.get("factor", 1.0), s.get("low", 0.0), s.get("high", 0.0),
                                   s.get("length", 0.0), err, 256)
        if rc != LL_OK:
            raise LLError(rc, err.value.decode())

    def _rows(self, t, name: str, shape, dtype, index: int, written: bool) -> bytes:
        try:
            if t.get_device() == index and t.dtype == dtype and t.shape == shape:
                seq, token, head, last = t.stride()
                if last == 1 and (not written or t.is_contiguous()):
                    return _rows_bytes(t.data_ptr(), seq, token, head)
        except AttributeError:
            pass
        if not getattr(t, "is_cuda", False) or t.get_device() != index or t.dtype != dtype:
            raise LLError(LL_ERR_ARG, f"{name} must be {dtype} on cuda:{index}, as q")
        if t.shape != shape:
            raise LLError(LL_ERR_ARG, f"{name} is {tuple(t.shape)}, the call needs {list(shape)}")
        if last != 1:
            raise LLError(LL_ERR_ARG, f"{name}'s last dim must be contiguous")
        reach = self.head_dim  # (no two rows of an output may share memory)
        for stride, size in sorted(((seq, shape[0]), (token, shape[1]), (head, shape[2]))):
            if size > 1:
                if stride < reach:
                    raise LLError(LL_ERR_ARG, f"{name} is written and its rows overlap")
                reach += stride * (size - 1)
        return _rows_bytes(t.data_ptr(), seq, token, head)

    def apply(self, q, k, lens, n_toks=None, q_out=None, k_out=None, inverse: bool = False):
        """Turn the last tokens' q [n_seq, n_tok, n_q_heads, head_dim] and k [n_seq, n_tok, n_k_heads, head_dim]
        (or None), bf16 or fp32, into q_out and k_out (in place where None). Rows of padded
        tokens keep what they hold."""
        if not getattr(q, "is_cuda", False) or q.ndim != 4:
            raise LLError(LL_ERR_ARG, "q must be a CUDA tensor [n_seq, n_tok, n_q_heads, head_dim]")
        dtype, index, shape = q.dtype, q.get_device(), q.shape
        code = self.codes.get(dtype)
        if code is None:
            raise LLError(LL_ERR_ARG, f"q must be bfloat16 or float32, not {dtype}")
        S, n_tok, heads, width = shape
        if width != self.head_dim:
            raise LLError(LL_ERR_ARG, f"q's heads are {width} wide, not {self.head_dim}")
        qr = self._rows(q, "q", shape, dtype, index, q_out is None)
        qor = qr if q_out is None else self._rows(q_out, "q_out", shape, dtype, index, True)
        kr = kor = None
        k_heads = 0
        if k is not None:
            k_heads = k.shape[2] if getattr(k, "ndim", 0) == 4 else 0
            shape = (S, n_tok, k_heads, width)
            kr = self._rows(k, "k", shape, dtype, index, k_out is None)
            kor = kr if k_out is None else self._rows(k_out, "k_out", shape, dtype, index, True)
        elif k_out is not None:
            raise LLError(LL_ERR_ARG, "k_out needs a k")
        int32 = _Types.int32
        lp = _array(lens, "lens", int32, (S,), index)
        np_ = None if n_toks is None else _array(n_toks, "n_toks", int32, (S,), index)
        _device_call(self.lib.ll_rope, index, self.ref, qr, qor, heads, kr, kor, k_heads, code, S, n_tok, lp, np_, 1 if inverse else 0)
        return q if q_out is None else q_out, (k if k_out is None else k_out)
