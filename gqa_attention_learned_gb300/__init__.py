"""Python binding of libsinkattn (GQA attention with learned per-head sinks).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI declared in ``include/sinkattn.h``.  PyTorch supplies
device memory and the current stream.  There is no fallback: if the shared
library is missing or fails to load, every call raises.
"""

import contextlib
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsinkattn.so")

OK, INVALID_ARGUMENT, UNSUPPORTED, WORKSPACE_TOO_SMALL, CUDA_ERROR = range(5)

_c_int, _c_float, _c_size, _vp = ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_void_p

# name -> (restype, argtypes), in the order of include/sinkattn.h
SIGNATURES = {
    "sinkattn_status_string": (ctypes.c_char_p, [_c_int]),
    "sinkattn_version": (_c_int, []),
    "sinkattn_last_error": (ctypes.c_char_p, []),
    "sinkattn_set_programmatic_launch": (_c_int, [_c_int]),
    "sinkattn_decode_plan": (_c_int, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int,
                                      ctypes.POINTER(_c_int), ctypes.POINTER(_c_size)]),
    "sinkattn_decode_workspace_bytes": (_c_size, [_c_int, _c_int, _c_int, _c_int]),
    "sinkattn_decode": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _vp, _vp, _c_float, _vp, _vp,
                                 _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int,
                                 _vp, _c_size, _vp]),
    "sinkattn_decode_ex": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _vp, _vp, _c_float, _vp, _vp,
                                    _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int,
                                    _c_int, _vp, _c_size, _c_int, _vp]),
    "sinkattn_verify_plan": (_c_int, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int,
                                      _c_int, ctypes.POINTER(_c_int), ctypes.POINTER(_c_size)]),
    "sinkattn_verify": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _vp, _vp, _vp, _c_float, _vp, _vp,
                                 _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int,
                                 _c_int, _vp, _c_size, _vp]),
    "sinkattn_verify_ex": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _vp, _vp, _vp, _c_float, _vp,
                                    _vp, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int,
                                    _c_int, _c_int, _vp, _c_size, _c_int, _vp]),
    "sinkattn_prefill": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _vp, _c_float, _vp,
                                  _vp, _c_int, _c_int, _c_int, _vp]),
    "sinkattn_prefill_paged": (_c_int, [_vp, _vp, _c_int, _c_int, _c_int, _vp, _vp, _vp, _c_int,
                                        _vp, _c_int, _c_int, _vp, _c_float, _vp, _vp, _c_int,
                                        _c_int, _c_int, _c_int, _vp]),
    "sinkattn_yarn_table": (_c_int, [_c_int, ctypes.c_double, ctypes.c_double, ctypes.c_double,
                                     ctypes.c_double, ctypes.c_double,
                                     ctypes.POINTER(_c_float), ctypes.POINTER(_c_float)]),
    "sinkattn_qkv_prologue": (_c_int, [_vp, _vp, _vp, _vp, ctypes.POINTER(_c_float), _c_float,
                                       _c_int, _vp, _vp, _vp, _c_int, _c_int, _c_int, _c_int,
                                       _c_int, _c_int, _vp]),
    "sinkattn_decode_static_scratch": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _vp, _vp, _c_float,
                                                _vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int,
                                                _c_int, _c_int, _c_int, _vp]),
    "sinkattn_decode_window_plan": (_c_int, [_c_int] * 9 + [ctypes.POINTER(_c_int),
                                                            ctypes.POINTER(_c_size)]),
    "sinkattn_decode_window": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _vp, _vp, _c_float, _c_int,
                                        _c_int, _vp, _vp] + [_c_int] * 8 +
                               [_vp, _c_size, _c_int, _vp]),
    "sinkattn_prefill_window": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _c_int, _c_int, _vp, _c_float,
                                         _c_int, _c_int, _vp, _vp, _c_int, _c_int, _c_int, _vp]),
    "sinkattn_prefill_paged_window": (_c_int, [_vp, _vp, _c_int, _c_int, _c_int, _vp, _vp, _vp,
                                               _c_int, _vp, _c_int, _c_int, _vp, _c_float, _c_int,
                                               _c_int, _vp, _vp, _c_int, _c_int, _c_int, _c_int,
                                               _vp]),
    "sinkattn_decode_mass": (_c_int, [_vp, _vp, _vp, _c_int, _vp, _vp, _c_float, _vp] +
                             [_c_int] * 8 + [_vp]),
    "sinkattn_prefill_mass": (_c_int, [_vp, _vp, _c_int, _c_int, _c_int, _vp, _vp, _c_int, _vp,
                                       _c_int, _c_int, _vp, _c_float, _vp] + [_c_int] * 5 + [_vp]),
    "sinkattn_evict": (_c_int, [_vp, _vp, _vp, _c_int, _vp, _vp, _c_int, _c_int, _c_int, _c_int,
                                _vp, _c_int, _vp, _c_int, _vp, _vp] + [_c_int] * 6 + [_vp]),
}

STATIC_SCRATCH_BYTES = 16 << 20
LAUNCH_DEFAULT, LAUNCH_PLAIN, LAUNCH_PROGRAMMATIC = 0, 1, 2
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
MAX_VERIFY_TOKENS = 64

_lib = None


class SinkAttnError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        detail = ""
        if status == CUDA_ERROR:
            detail = ": " + load().sinkattn_last_error().decode()
        super().__init__(f"{fn} failed: {status_string(status)} ({status}){detail}")


def load():
    """Load libsinkattn.so (built by ``build.build()``); raises if absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libsinkattn.so not built ({LIB_PATH}); run "
                               "`python -m gqa_attention_learned_gb300.build`")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _lib = lib
    return _lib


def status_string(status):
    return load().sinkattn_status_string(int(status)).decode()


def set_programmatic_launch(enable):
    """Process-wide DEFAULT launch mode of the decode and verification
    kernels (decode, decode_static_scratch, verify called without
    `programmatic=`); returns the previous setting.  In programmatic mode,
    kv_lens and page_table of a call must not be written by the kernel
    launched just before it on the stream."""
    return bool(load().sinkattn_set_programmatic_launch(1 if enable else 0))


def _launch_flags(programmatic):
    """None: the process-wide default; True / False: this call's own mode."""
    if programmatic is None:
        return LAUNCH_DEFAULT
    return LAUNCH_PROGRAMMATIC if programmatic else LAUNCH_PLAIN


def _check(fn, status):
    if status != OK:
        raise SinkAttnError(fn, status)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _on(dev):
    """Makes `dev` the current device for a call (no-op when it already is)."""
    if dev.index is None or dev.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(dev)


_plans = {}
_PLANS_KEPT = 4096


def _plan(fn, *args):
    """fn(*args) for the current device, memoised: plans depend only on
    host-side sizes and the device's SM count (at most _PLANS_KEPT kept)."""
    key = (fn.__name__, torch.cuda.current_device()) + args
    hit = _plans.get(key)
    if hit is None:
        if len(_plans) >= _PLANS_KEPT:
            _plans.clear()
        hit = _plans[key] = fn(*args)
    return hit


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _want(t, name, dtype, dims=None, device=None):
    if (isinstance(t, torch.Tensor) and t.dtype == dtype and (dims is None or t.dim() == dims)
            and t.is_cuda and (device is None or t.device == device) and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if dims is not None and t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dims, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")


def decode_plan(batch, num_qo_heads, num_kv_heads, max_kv_len, num_splits=0, num_sms=0,
                head_dim=64, page_size=16):
    """(split count, workspace bytes) that `decode` will use (host only).  A
    workspace must be zero-filled before its first use (torch.zeros)."""
    s = _c_int(num_splits)
    w = _c_size(0)
    _check("sinkattn_decode_plan",
           load().sinkattn_decode_plan(batch, num_qo_heads, num_kv_heads, head_dim, page_size,
                                       max_kv_len, num_sms, ctypes.byref(s), ctypes.byref(w)))
    return s.value, w.value


def decode_workspace_bytes(batch, num_qo_heads, num_splits, head_dim=64):
    """Upper bound on decode's workspace for an explicit split count, valid
    for any KV head count (host only; 0 for one split)."""
    return int(load().sinkattn_decode_workspace_bytes(batch, num_qo_heads, head_dim, num_splits))


def decode(q, k_cache, v_cache, page_table, kv_lens, sinks, scale, max_kv_len, *, out=None,
           lse=None, num_splits=0, workspace=None, stream=None, want_lse=True, programmatic=None):
    """Paged decode.  q [B, Hq, 64] bf16; caches [pages, Hkv, 16, 64] bf16;
    page_table [B, max_pages] int32; kv_lens [B] int32; sinks [Hq] fp32.
    programmatic: None = the process-wide default launch mode, True / False =
    this call's own.  Returns (out [B, Hq, 64] bf16, lse [B, Hq] fp32 or None)."""
    dev = q.device
    _want(q, "q", torch.bfloat16, 3)
    _want(k_cache, "k_cache", torch.bfloat16, 4, dev)
    _want(v_cache, "v_cache", torch.bfloat16, 4, dev)
    _want(page_table, "page_table", torch.int32, 2, dev)
    _want(kv_lens, "kv_lens", torch.int32, 1, dev)
    _want(sinks, "sinks", torch.float32, 1, dev)
    batch, hq, d = q.shape
    num_pages, hkv, page, d2 = k_cache.shape
    if v_cache.shape != k_cache.shape or d2 != d:
        raise ValueError("k_cache/v_cache shapes disagree with q")
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty(batch, hq, dtype=torch.float32, device=dev)
    with _on(dev):
        splits, ws_bytes = _plan(decode_plan, batch, hq, hkv, int(max_kv_len), int(num_splits),
                                 0, d, page) if batch else (1, 0)
        if workspace is None and ws_bytes:
            # zero-filled once; decode leaves it ready for the next call
            workspace = torch.zeros(ws_bytes, dtype=torch.uint8, device=dev)
        ws_len = 0 if workspace is None else workspace.numel() * workspace.element_size()
        _check("sinkattn_decode_ex", load().sinkattn_decode_ex(
            _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table), page_table.shape[1],
            _ptr(kv_lens), _ptr(sinks), float(scale), _ptr(out), _ptr(lse), batch, hq, hkv, d,
            page, num_pages, int(max_kv_len), int(num_splits), _ptr(workspace), ws_len,
            _launch_flags(programmatic), _stream(stream)))
    return out, lse


def verify_plan(batch, q_len, num_qo_heads, num_kv_heads, max_kv_len, num_splits=0, num_sms=0,
                head_dim=64, page_size=16):
    """(split count, workspace bytes) that `verify` will use (host only)."""
    s = _c_int(num_splits)
    w = _c_size(0)
    _check("sinkattn_verify_plan",
           load().sinkattn_verify_plan(batch, q_len, num_qo_heads, num_kv_heads, head_dim,
                                       page_size, max_kv_len, num_sms, ctypes.byref(s),
                                       ctypes.byref(w)))
    return s.value, w.value


def verify(q, k_cache, v_cache, page_table, kv_lens, sinks, scale, max_kv_len, *, tree_mask=None,
           out=None, lse=None, num_splits=0, workspace=None, stream=None, want_lse=True,
           programmatic=None):
    """Verification of the q_len newest tokens of every request (speculative
    decoding).  q [B, q_len, Hq, 64] bf16; the tokens are the last q_len keys
    of each request's paged KV.  tree_mask: None (causal) or int64
    [B, q_len] holding the uint64 bit masks (bit u of row i: token i sees
    draft token u).  programmatic: as for decode.  Returns
    (out [B, q_len, Hq, 64], lse [B, q_len, Hq])."""
    dev = q.device
    _want(q, "q", torch.bfloat16, 4)
    _want(k_cache, "k_cache", torch.bfloat16, 4, dev)
    _want(v_cache, "v_cache", torch.bfloat16, 4, dev)
    _want(page_table, "page_table", torch.int32, 2, dev)
    _want(kv_lens, "kv_lens", torch.int32, 1, dev)
    _want(sinks, "sinks", torch.float32, 1, dev)
    batch, q_len, hq, d = q.shape
    if tree_mask is not None:
        _want(tree_mask, "tree_mask", torch.int64, 2, dev)
        if tuple(tree_mask.shape) != (batch, q_len):
            raise ValueError("tree_mask must be [batch, q_len]")
    num_pages, hkv, page, _ = k_cache.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty(batch, q_len, hq, dtype=torch.float32, device=dev)
    with _on(dev):
        splits, ws_bytes = _plan(verify_plan, batch, q_len, hq, hkv, int(max_kv_len),
                                 int(num_splits), 0, d, page) if batch else (1, 0)
        if workspace is None and ws_bytes:
            workspace = torch.zeros(ws_bytes, dtype=torch.uint8, device=dev)
        ws_len = 0 if workspace is None else workspace.numel() * workspace.element_size()
        _check("sinkattn_verify_ex", load().sinkattn_verify_ex(
            _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table), page_table.shape[1],
            _ptr(kv_lens), _ptr(tree_mask), _ptr(sinks), float(scale), _ptr(out), _ptr(lse), batch,
            q_len, hq, hkv, d, page, num_pages, int(max_kv_len), int(num_splits), _ptr(workspace),
            ws_len, _launch_flags(programmatic), _stream(stream)))
    return out, lse


def prefill(q, k, v, cu_seqlens, sinks, scale, max_seqlen, *, out=None, lse=None, stream=None,
            want_lse=True):
    """Ragged causal prefill.  q [T, Hq, 64], k/v [T, Hkv, 64] bf16;
    cu_seqlens [n+1] int32.  Returns (out [T, Hq, 64], lse [T, Hq] or None)."""
    dev = q.device
    _want(q, "q", torch.bfloat16, 3)
    _want(k, "k", torch.bfloat16, 3, dev)
    _want(v, "v", torch.bfloat16, 3, dev)
    _want(cu_seqlens, "cu_seqlens", torch.int32, 1, dev)
    _want(sinks, "sinks", torch.float32, 1, dev)
    total, hq, d = q.shape
    hkv = k.shape[1]
    if k.shape != v.shape or k.shape[0] != total or k.shape[2] != d:
        raise ValueError("q/k/v shapes disagree")
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty(total, hq, dtype=torch.float32, device=dev)
    with _on(dev):
        _check("sinkattn_prefill", load().sinkattn_prefill(
            _ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), cu_seqlens.numel() - 1, total,
            int(max_seqlen), _ptr(sinks), float(scale), _ptr(out), _ptr(lse), hq, hkv, d,
            _stream(stream)))
    return out, lse


def prefill_paged(q, cu_seqlens_q, k_cache, v_cache, page_table, kv_lens, sinks, scale,
                  max_q_len, max_kv_len, *, out=None, lse=None, stream=None, want_lse=True):
    """Chunked prefill against a paged KV prefix (bottom-right causal)."""
    dev = q.device
    _want(q, "q", torch.bfloat16, 3)
    _want(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1, dev)
    _want(k_cache, "k_cache", torch.bfloat16, 4, dev)
    _want(v_cache, "v_cache", torch.bfloat16, 4, dev)
    _want(page_table, "page_table", torch.int32, 2, dev)
    _want(kv_lens, "kv_lens", torch.int32, 1, dev)
    _want(sinks, "sinks", torch.float32, 1, dev)
    total, hq, d = q.shape
    num_pages, hkv, page, _ = k_cache.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty(total, hq, dtype=torch.float32, device=dev)
    with _on(dev):
        _check("sinkattn_prefill_paged", load().sinkattn_prefill_paged(
            _ptr(q), _ptr(cu_seqlens_q), cu_seqlens_q.numel() - 1, total, int(max_q_len),
            _ptr(k_cache), _ptr(v_cache), _ptr(page_table), page_table.shape[1], _ptr(kv_lens),
            num_pages, int(max_kv_len), _ptr(sinks), float(scale), _ptr(out), _ptr(lse), hq, hkv,
            d, page, _stream(stream)))
    return out, lse


def decode_static_scratch(q, k_cache, v_cache, page_table, kv_lens, sinks, scale, max_kv_len, *,
                          out=None, lse=None, num_splits=0, stream=None, want_lse=True):
    """Decode for callers that cannot allocate device memory: the split
    scratch is the library's own fixed 16 MiB device array instead of a
    caller-provided workspace.  Raises SinkAttnError (WORKSPACE_TOO_SMALL)
    when the sizes need more scratch than that.  Calls that overlap on the GPU
    share the array and race; order them on one stream."""
    dev = q.device
    _want(q, "q", torch.bfloat16, 3)
    _want(k_cache, "k_cache", torch.bfloat16, 4, dev)
    _want(v_cache, "v_cache", torch.bfloat16, 4, dev)
    _want(page_table, "page_table", torch.int32, 2, dev)
    _want(kv_lens, "kv_lens", torch.int32, 1, dev)
    _want(sinks, "sinks", torch.float32, 1, dev)
    batch, hq, d = q.shape
    num_pages, hkv, page, _ = k_cache.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None and want_lse:
        lse = torch.empty(batch, hq, dtype=torch.float32, device=dev)
    with _on(dev):
        _check("sinkattn_decode_static_scratch", load().sinkattn_decode_static_scratch(
            _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table), page_table.shape[1],
            _ptr(kv_lens), _ptr(sinks), float(scale), _ptr(out), _ptr(lse), batch, hq, hkv, d,
            page, num_pages, int(max_kv_len), int(num_splits), _stream(stream)))
    return out, lse


def yarn_table(head_dim=64, base=150000.0, factor=32.0, original_context=4096, beta_fast=32.0,
               beta_slow=1.0):
    """(inv_freq list of head_dim/2 floats, mscale): YaRN-scaled rotary
    frequencies and magnitude factor (host only)."""
    freq = (_c_float * (head_dim // 2))()
    ms = _c_float(0)
    _check("sinkattn_yarn_table",
           load().sinkattn_yarn_table(head_dim, float(base), float(factor), float(original_context),
                                      float(beta_fast), float(beta_slow), freq, ctypes.byref(ms)))
    return list(freq), ms.value


def qkv_prologue(qkv, bias, positions, slot_mapping, inv_freq, mscale, k_cache, v_cache,
                 num_qo_heads, num_kv_heads, *, rope_style=ROPE_HALF, q_out=None, stream=None):
    """QKV bias + rotary encoding of q and k + k/v written into the paged
    cache, one launch.  qkv [T, (Hq + 2 Hkv) * 64] bf16; bias same width or
    None; positions, slot_mapping [T] int32 (slot = page * 16 + offset, < 0:
    no write); inv_freq: sequence of 32 floats (host).  Returns q_out
    [T, Hq, 64] bf16; k_cache / v_cache are written in place."""
    dev = qkv.device
    _want(qkv, "qkv", torch.bfloat16, 2)
    if bias is not None:
        _want(bias, "bias", torch.bfloat16, 1, dev)
    _want(positions, "positions", torch.int32, 1, dev)
    _want(slot_mapping, "slot_mapping", torch.int32, 1, dev)
    _want(k_cache, "k_cache", torch.bfloat16, 4, dev)
    _want(v_cache, "v_cache", torch.bfloat16, 4, dev)
    tokens = qkv.shape[0]
    num_pages, hkv, page, d = k_cache.shape
    if hkv != num_kv_heads or qkv.shape[1] != (num_qo_heads + 2 * num_kv_heads) * d:
        raise ValueError("qkv width / cache heads disagree with the head counts")
    freq = (_c_float * (d // 2))(*[float(x) for x in inv_freq])
    if q_out is None:
        q_out = torch.empty(tokens, num_qo_heads, d, dtype=torch.bfloat16, device=dev)
    with _on(dev):
        _check("sinkattn_qkv_prologue", load().sinkattn_qkv_prologue(
            _ptr(qkv), _ptr(bias), _ptr(positions), _ptr(slot_mapping), freq, float(mscale),
            int(rope_style), _ptr(q_out), _ptr(k_cache), _ptr(v_cache), tokens, num_qo_heads,
            num_kv_heads, d, page, num_pages, _stream(stream)))
    return q_out


# ------------------------------------------------- bounding a long context
_INT_MAX = 2**31 - 1


_AS_IS = contextlib.nullcontext()


def _at(dev, stream):
    """Makes `dev` the current device and `stream` (if given) its current
    stream, so that what a call allocates or clears is ordered on the stream
    that it launches on (no-op when both already are)."""
    if stream is None and dev.index == torch._C._cuda_getDevice():
        return _AS_IS
    stack = contextlib.ExitStack()
    stack.enter_context(_on(dev))
    if stream is not None:
        stack.enter_context(torch.cuda.stream(stream))
    return stack


def _raw_stream(dev):
    """Handle of the device's current stream."""
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _size(v, name, least=0):
    """v as an int that fits the C ABI's (larger bounds mean no bound)."""
    if type(v) is int and least <= v <= _INT_MAX:
        return v
    v = int(v)
    if v < least:
        raise ValueError(f"{name} must be at least {least}, got {v}")
    return min(v, _INT_MAX)


def _shape(t, name, shape):
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


_Tensor, _BF16, _F32, _I32 = torch.Tensor, torch.bfloat16, torch.float32, torch.int32


def _is(t, dtype, dims, dev):
    """What `_want` asks for, as one quick test: the small calls spend more
    time on the host than on the GPU."""
    return (type(t) is _Tensor and t.dtype is dtype and t.dim() == dims and t.device == dev
            and t.is_contiguous())


def _paged_args(dev, batch, page_table, kv_lens, k_cache, v_cache=None):
    if not (_is(k_cache, _BF16, 4, dev) and _is(page_table, _I32, 2, dev)
            and _is(kv_lens, _I32, 1, dev) and (v_cache is None or _is(v_cache, _BF16, 4, dev))
            and dev.type == "cuda"):
        _want(k_cache, "k_cache", _BF16, 4, dev)
        _want(page_table, "page_table", _I32, 2, dev)
        _want(kv_lens, "kv_lens", _I32, 1, dev)
        if v_cache is not None:
            _want(v_cache, "v_cache", _BF16, 4, dev)
    if v_cache is not None and v_cache.shape != k_cache.shape:
        raise ValueError(f"v_cache must be {list(k_cache.shape)}, got {list(v_cache.shape)}")
    if page_table.shape[0] != batch or kv_lens.shape[0] != batch:
        raise ValueError(f"page_table and kv_lens must have {batch} rows, got "
                         f"{page_table.shape[0]} and {kv_lens.shape[0]}")


def _rows_out(q, out, lse, want_lse):
    """The bf16 result and the fp32 lse of the rows of q, checked or new."""
    if out is None:
        out = torch.empty_like(q)
    else:
        _want(out, "out", torch.bfloat16, q.dim(), q.device)
        _shape(out, "out", q.shape)
    if lse is not None:
        _want(lse, "lse", torch.float32, q.dim() - 1, q.device)
        _shape(lse, "lse", q.shape[:-1])
    elif want_lse:
        lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device)
    return out, lse


def decode_window_plan(batch, num_qo_heads, num_kv_heads, max_kv_len, window, first_tokens=0,
                       num_splits=0, num_sms=0, head_dim=64, page_size=16):
    """(split count, workspace bytes) that `decode_window` will use (host only)."""
    s = _c_int(num_splits)
    w = _c_size(0)
    _check("sinkattn_decode_window_plan",
           load().sinkattn_decode_window_plan(batch, num_qo_heads, num_kv_heads, head_dim,
                                              page_size, max_kv_len, window, first_tokens, num_sms,
                                              ctypes.byref(s), ctypes.byref(w)))
    return s.value, w.value


def decode_window(q, k_cache, v_cache, page_table, kv_lens, sinks, scale, max_kv_len, window,
                  first_tokens=0, *, out=None, lse=None, num_splits=0, workspace=None, stream=None,
                  want_lse=True, programmatic=None):
    """`decode` with a sliding window: the token sees its request's `window`
    newest keys (its own included) and the `first_tokens` oldest.  Pages
    without a visible key are not looked up (their page_table entries may hold
    anything).  Returns (out [B, Hq, 64] bf16, lse [B, Hq] fp32 or None)."""
    # the smallest calls last a few microseconds on the GPU: the checks are kept
    # to what an argument can get wrong, and the plan is made by the library
    # alone when the caller brings the workspace
    dev = q.device
    if not _is(q, _BF16, 3, dev):
        _want(q, "q", _BF16, 3)
    batch, hq, d = q.shape
    _paged_args(dev, batch, page_table, kv_lens, k_cache, v_cache)
    if not _is(sinks, _F32, 1, dev):
        _want(sinks, "sinks", _F32, 1, dev)
    num_pages, hkv, page, d2 = k_cache.shape
    if d2 != d or sinks.shape[0] != hq:
        raise ValueError("k_cache, sinks and q disagree in head_dim or heads")
    window, first = _size(window, "window", 1), _size(first_tokens, "first_tokens")
    max_kv_len, num_splits = _size(max_kv_len, "max_kv_len"), _size(num_splits, "num_splits")
    with _at(dev, stream):
        if out is None and lse is None and want_lse:
            out = torch.empty_like(q)
            lse = torch.empty((batch, hq), dtype=torch.float32, device=dev)
        else:
            out, lse = _rows_out(q, out, lse, want_lse)
        if workspace is None:
            ws_ptr = ws_len = None
            if batch:
                _, ws_len = _plan(decode_window_plan, batch, hq, hkv, max_kv_len, window, first,
                                  num_splits, 0, d, page)
            if ws_len:
                # zero-filled once; the call leaves it ready for the next one
                workspace = torch.zeros(ws_len, dtype=torch.uint8, device=dev)
                ws_ptr = workspace.data_ptr()
        else:
            if workspace.device != dev or not workspace.is_contiguous():
                raise ValueError(f"workspace must be contiguous and on {dev}")
            ws_ptr, ws_len = workspace.data_ptr(), workspace.nbytes
        status = load().sinkattn_decode_window(
            q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(),
            page_table.shape[1], kv_lens.data_ptr(), sinks.data_ptr(), float(scale), window, first,
            out.data_ptr(), None if lse is None else lse.data_ptr(), batch, hq, hkv, d, page,
            num_pages, max_kv_len, num_splits, ws_ptr, ws_len or 0,
            0 if programmatic is None else _launch_flags(programmatic), _raw_stream(dev))
        if status:
            _check("sinkattn_decode_window", status)
    return out, lse


def prefill_window(q, k, v, cu_seqlens, sinks, scale, max_seqlen, window, first_tokens=0, *,
                   out=None, lse=None, stream=None, want_lse=True):
    """`prefill` with a sliding window: token i of a sequence sees tokens
    i - window + 1 .. i and the sequence's `first_tokens` first ones (up to
    itself).  Returns (out [T, Hq, 64], lse [T, Hq] or None)."""
    dev = q.device
    if not (_is(q, _BF16, 3, dev) and _is(k, _BF16, 3, dev) and _is(v, _BF16, 3, dev)
            and _is(cu_seqlens, _I32, 1, dev) and _is(sinks, _F32, 1, dev) and dev.type == "cuda"):
        _want(q, "q", _BF16, 3)
        _want(k, "k", _BF16, 3, dev)
        _want(v, "v", _BF16, 3, dev)
        _want(cu_seqlens, "cu_seqlens", _I32, 1, dev)
        _want(sinks, "sinks", _F32, 1, dev)
    total, hq, d = q.shape
    hkv = k.shape[1]
    num_seqs = cu_seqlens.shape[0] - 1
    _shape(k, "k", (total, hkv, d))
    _shape(v, "v", k.shape)
    _shape(sinks, "sinks", (hq,))
    if num_seqs < 0:
        raise ValueError("cu_seqlens must hold num_seqs + 1 entries")
    window, first = _size(window, "window", 1), _size(first_tokens, "first_tokens")
    max_seqlen = _size(max_seqlen, "max_seqlen")
    with _at(dev, stream):
        out, lse = _rows_out(q, out, lse, want_lse)
        status = load().sinkattn_prefill_window(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_seqlens.data_ptr(), num_seqs, total,
            max_seqlen, sinks.data_ptr(), float(scale), window, first, out.data_ptr(), _ptr(lse),
            hq, hkv, d, _raw_stream(dev))
        if status:
            _check("sinkattn_prefill_window", status)
    return out, lse


def prefill_paged_window(q, cu_seqlens_q, k_cache, v_cache, page_table, kv_lens, sinks, scale,
                         max_q_len, max_kv_len, window, first_tokens=0, *, out=None, lse=None,
                         stream=None, want_lse=True):
    """`prefill_paged` with a sliding window (see `prefill_window`; positions
    count from the request's first cached key)."""
    dev = q.device
    if not (_is(q, _BF16, 3, dev) and _is(cu_seqlens_q, _I32, 1, dev) and _is(sinks, _F32, 1, dev)):
        _want(q, "q", _BF16, 3)
        _want(cu_seqlens_q, "cu_seqlens_q", _I32, 1, dev)
        _want(sinks, "sinks", _F32, 1, dev)
    total, hq, d = q.shape
    num_seqs = cu_seqlens_q.shape[0] - 1
    _paged_args(dev, num_seqs, page_table, kv_lens, k_cache, v_cache)
    _shape(sinks, "sinks", (hq,))
    num_pages, hkv, page, d2 = k_cache.shape
    if d2 != d:
        raise ValueError("k_cache and q disagree in head_dim")
    window, first = _size(window, "window", 1), _size(first_tokens, "first_tokens")
    max_q_len, max_kv_len = _size(max_q_len, "max_q_len"), _size(max_kv_len, "max_kv_len")
    with _at(dev, stream):
        out, lse = _rows_out(q, out, lse, want_lse)
        status = load().sinkattn_prefill_paged_window(
            q.data_ptr(), cu_seqlens_q.data_ptr(), num_seqs, total, max_q_len, k_cache.data_ptr(),
            v_cache.data_ptr(), page_table.data_ptr(), page_table.shape[1], kv_lens.data_ptr(),
            num_pages, max_kv_len, sinks.data_ptr(), float(scale), window, first, out.data_ptr(),
            _ptr(lse), hq, hkv, d, page, _raw_stream(dev))
        if status:
            _check("sinkattn_prefill_paged_window", status)
    return out, lse


def _mass_args(q, k_cache, page_table, kv_lens, lse, mass, batch):
    dev = q.device
    if not (_is(q, _BF16, 3, dev) and _is(lse, _F32, 2, dev) and _is(mass, _F32, 3, dev)):
        _want(q, "q", _BF16, 3)
        _want(lse, "lse", _F32, 2, dev)
        _want(mass, "mass", _F32, 3, dev)
    _paged_args(dev, batch, page_table, kv_lens, k_cache)
    if lse.shape != q.shape[:2]:
        _shape(lse, "lse", q.shape[:2])
    if mass.shape[0] != batch or mass.shape[1] != k_cache.shape[1]:
        raise ValueError(f"mass must be [{batch}, {k_cache.shape[1]}, ...], got {list(mass.shape)}")
    if k_cache.shape[3] != q.shape[2]:
        raise ValueError("k_cache and q disagree in head_dim")


def decode_mass(q, k_cache, page_table, kv_lens, lse, scale, max_kv_len, mass, *, stream=None):
    """Adds the attention weight that one new token per request gives to each
    cached key: mass[b, g, j] += sum over the heads h of KV head g of
    exp(scale * q_bh . k_gj - lse_bh), lse from `decode` on the same inputs.
    mass [B, Hkv, at least max_kv_len] fp32, updated in place and returned."""
    _mass_args(q, k_cache, page_table, kv_lens, lse, mass, q.shape[0])
    batch, hq, d = q.shape
    num_pages, hkv, page, _ = k_cache.shape
    with _at(q.device, stream):
        _check("sinkattn_decode_mass", load().sinkattn_decode_mass(
            _ptr(q), _ptr(k_cache), _ptr(page_table), page_table.shape[1], _ptr(kv_lens),
            _ptr(lse), float(scale), _ptr(mass), mass.shape[2], batch, hq, hkv, d, page, num_pages,
            _size(max_kv_len, "max_kv_len"), _raw_stream(q.device)))
    return mass


def prefill_mass(q, cu_seqlens_q, k_cache, page_table, kv_lens, lse, scale, max_q_len, max_kv_len,
                 mass, *, stream=None):
    """`decode_mass` for ragged rows: the queries of `prefill_paged` (or the
    last few of each prompt, so that only those vote), each row counting the
    keys up to its own position."""
    _want(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1, q.device)
    batch = cu_seqlens_q.numel() - 1
    _mass_args(q, k_cache, page_table, kv_lens, lse, mass, batch)
    total, hq, d = q.shape
    num_pages, hkv, page, _ = k_cache.shape
    with _at(q.device, stream):
        _check("sinkattn_prefill_mass", load().sinkattn_prefill_mass(
            _ptr(q), _ptr(cu_seqlens_q), batch, total, _size(max_q_len, "max_q_len"),
            _ptr(k_cache), _ptr(page_table), page_table.shape[1], _ptr(kv_lens), num_pages,
            _size(max_kv_len, "max_kv_len"), _ptr(lse), float(scale), _ptr(mass), mass.shape[2],
            hq, hkv, d, page, _raw_stream(q.device)))
    return mass


def evict(k_cache, v_cache, page_table, kv_lens, mass, budget, max_kv_len, *, first_tokens=0,
          recent=0, dst_page_table=None, dst_mass=None, new_kv_lens=None, kept=None, stream=None):
    """Cuts each request to `budget` keys: every KV head keeps its first
    `first_tokens`, its last `recent` and the heaviest others by `mass` (ties:
    the lower index), in order, moved to the request's first slots -- in place,
    or to the pages of dst_page_table [B, pages] and to dst_mass
    [B, Hkv, budget or more].  Returns (new_kv_lens [B] int32,
    kept [B, Hkv, budget] int32: former indices, -1 past the new length);
    a request that cannot be moved (lengths or pages out of range) is left
    alone with new length -1."""
    dev = k_cache.device
    batch = kv_lens.shape[0]
    _paged_args(dev, batch, page_table, kv_lens, k_cache, v_cache)
    num_pages, hkv, page, d = k_cache.shape
    for name, m in (("mass", mass), ("dst_mass", dst_mass)):
        if m is None and name == "dst_mass":
            continue
        if not _is(m, _F32, 3, dev):
            _want(m, name, _F32, 3, dev)
        if m.shape[0] != batch or m.shape[1] != hkv:
            raise ValueError(f"{name} must be [{batch}, {hkv}, ...], got {list(m.shape)}")
    if dst_page_table is not None:
        if not _is(dst_page_table, _I32, 2, dev):
            _want(dst_page_table, "dst_page_table", _I32, 2, dev)
        if dst_page_table.shape[0] != batch:
            raise ValueError(f"dst_page_table must have {batch} rows")
    budget = _size(budget, "budget", 1)
    first, recent = _size(first_tokens, "first_tokens"), _size(recent, "recent")
    with _at(dev, stream):
        if new_kv_lens is None:
            new_kv_lens = torch.empty(batch, dtype=torch.int32, device=dev)
        else:
            _want(new_kv_lens, "new_kv_lens", torch.int32, 1, dev)
            _shape(new_kv_lens, "new_kv_lens", (batch,))
        if kept is None:
            kept = torch.empty(batch, hkv, budget, dtype=torch.int32, device=dev)
        else:
            _want(kept, "kept", torch.int32, 3, dev)
            _shape(kept, "kept", (batch, hkv, budget))
        _check("sinkattn_evict", load().sinkattn_evict(
            _ptr(k_cache), _ptr(v_cache), _ptr(page_table), page_table.shape[1], _ptr(kv_lens),
            _ptr(mass), mass.shape[2], budget, first, recent, _ptr(dst_page_table),
            0 if dst_page_table is None else dst_page_table.shape[1], _ptr(dst_mass),
            0 if dst_mass is None else dst_mass.shape[2], _ptr(new_kv_lens), _ptr(kept), batch,
            hkv, d, page, num_pages, _size(max_kv_len, "max_kv_len"), _raw_stream(dev)))
    return new_kv_lens, kept
