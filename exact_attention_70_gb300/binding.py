"""ctypes binding of libattn.so: argument marshalling only.

Every step of the computation runs in the library's CUDA kernels; this module checks tensor
dtypes and shapes, allocates outputs and workspace with torch when the caller does not pass
them, and forwards raw device pointers and the current CUDA stream.  If the library has not
been built the first call raises ``AttnError`` -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

from . import build as _build

_lock = threading.Lock()
_lib = None

STATUS = {0: "ok", -1: "invalid argument", -2: "unsupported configuration",
          -3: "workspace missing or too small", -4: "CUDA call failed",
          -5: "a kernel wait exceeded its time limit", -6: "a device-side index was out of range"}


class AttnError(RuntimeError):
    def __init__(self, code, where):
        super().__init__(f"{where}: {STATUS.get(code, code)} ({code})")
        self.code = code


def lib_path() -> str:
    return _build.LIB


def load():
    """Load libattn.so (built by ``__graft_entry__.build()`` / ``exact_attention_70_gb300.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = _build.LIB
            if not os.path.exists(path):
                raise AttnError(-4, f"libattn.so not built (expected at {path})")
            lib = ctypes.CDLL(path)
            P, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
            lib.attn_fwd.restype = i32
            lib.attn_fwd.argtypes = [P, P, P, P, P, P, P, i32, i32, i32, i32, i32, i32, i32, i32,
                                     f32, i32, i32, i32, P, sz, P]
            lib.attn_fwd_workspace_bytes.restype = sz
            lib.attn_fwd_workspace_bytes.argtypes = [i32, i32, i32, i32]
            lib.attn_decode_kvcache.restype = i32
            lib.attn_decode_kvcache.argtypes = [P, P, P, P, P, i32, i32, P, P, i32, i32, i32, i32,
                                                i32, i32, f32, P, sz, P]
            lib.attn_decode_workspace_bytes.restype = sz
            lib.attn_decode_workspace_bytes.argtypes = [i32, i32, i32, i32]
            lib.attn_decode_num_splits.restype = i32
            lib.attn_decode_num_splits.argtypes = [i32, i32, i32, i32, i32, i32]
            lib.attn_get_device_status.restype = i32
            lib.attn_get_device_status.argtypes = [P]
            lib.attn_selftest_wait_timeout.restype = i32
            lib.attn_selftest_wait_timeout.argtypes = [P]
            lib.attn_selftest_softcap.restype = i32
            lib.attn_selftest_softcap.argtypes = [P, P, i32, f32, f32, P]
            lib.attn_fwd_kvcache.restype = i32
            lib.attn_fwd_kvcache.argtypes = [P, P, P, P, P, P, P, P, P, P, i32, i32, i32, P, P,
                                             i32, i32, i32, i32, i32, i32, i32, i32, i32,
                                             ctypes.c_float, i32, i32, i32, P, sz, P]
            lib.attn_quantize_fp8.restype = i32
            lib.attn_quantize_fp8.argtypes = [P] * 4 + [i32] * 8 + [P] * 8
            lib.attn_fwd_fp8.restype = i32
            lib.attn_fwd_fp8.argtypes = [P] * 10 + [i32] * 9 + [f32, i32, i32, i32, P]
            lib.attn_fwd_mods.restype = i32
            lib.attn_fwd_mods.argtypes = [P, P, P, P, P, P, P] + [i32] * 8 + [f32, i32, i32, i32,
                                                                            f32, P, P, sz, P]
            lib.attn_bwd.restype = i32
            lib.attn_bwd.argtypes = [P] * 11 + [i32] * 8 + [f32, i32, i32, i32, P, sz, P]
            lib.attn_bwd_workspace_bytes.restype = sz
            lib.attn_bwd_workspace_bytes.argtypes = [i32, i32]
            lib.attn_fwd_kvcache_workspace_bytes.restype = sz
            lib.attn_fwd_kvcache_workspace_bytes.argtypes = [i32] * 7
            lib.attn_kvcache_append_fp8.restype = i32
            lib.attn_kvcache_append_fp8.argtypes = [P] * 11 + [i32] * 10 + [P]
            lib.attn_kvcache_read_fp8.restype = i32
            lib.attn_kvcache_read_fp8.argtypes = [P] * 8 + [i32] * 7 + [P]
            lib.attn_decode_kvcache_fp8.restype = i32
            lib.attn_decode_kvcache_fp8.argtypes = [P] * 7 + [i32, P, P] + [i32] * 6 + [
                f32, P, sz, P]
            lib.attn_decode_kvcache_fp8_workspace_bytes.restype = sz
            lib.attn_decode_kvcache_fp8_workspace_bytes.argtypes = [i32] * 6
            lib.attn_fwd_kvcache_fp8.restype = i32
            lib.attn_fwd_kvcache_fp8.argtypes = [P] * 12 + [i32] * 3 + [P, P] + [i32] * 10 + [
                f32, i32, i32, i32, P, sz, P]
            lib.attn_fwd_kvcache_fp8_workspace_bytes.restype = sz
            lib.attn_fwd_kvcache_fp8_workspace_bytes.argtypes = [i32] * 10
            i64 = ctypes.c_int64
            how = [P, P, i32, f32, P, P, i32, i32, i32, P, i32, P, i32]  # weights .. sections_interleaved
            lib.attn_kvcache_plan.restype = i32
            lib.attn_kvcache_plan.argtypes = [P] * 10 + [i32] * 6 + [P, sz, P]
            lib.attn_kvcache_plan_workspace_bytes.restype = sz
            lib.attn_kvcache_plan_workspace_bytes.argtypes = [i32, i32]
            lib.attn_qk_norm_rope.restype = i32
            lib.attn_qk_norm_rope.argtypes = [P, P, i64, i64] + how + [P, P] + [i32] * 4 + [P]
            lib.attn_qk_norm_rope_bwd.restype = i32
            lib.attn_qk_norm_rope_bwd.argtypes = [P] * 4 + [i64, i64] + how + [
                P, P, i64, i64, P, P] + [i32] * 4 + [P, sz, P]
            lib.attn_qk_norm_rope_bwd_workspace_bytes.restype = sz
            lib.attn_qk_norm_rope_bwd_workspace_bytes.argtypes = [i32]
            lib.attn_kvcache_append_norm_rope.restype = i32
            lib.attn_kvcache_append_norm_rope.argtypes = [P] * 3 + [i64] * 3 + how + [
                P, P, P, P] + [i32] * 6 + [P]
            lib.attn_decode_kvcache_shared.restype = i32
            lib.attn_decode_kvcache_shared.argtypes = [P] * 8 + [i32, P, P] + [i32] * 9 + [
                f32, P, sz, P]
            lib.attn_decode_kvcache_shared_workspace_bytes.restype = sz
            lib.attn_decode_kvcache_shared_workspace_bytes.argtypes = [i32] * 6
            lib.attn_status_string.restype = ctypes.c_char_p
            lib.attn_status_string.argtypes = [i32]
            lib.attn_kv_block_range.restype = i32
            lib.attn_kv_block_range.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32,
                                                ctypes.POINTER(i32), ctypes.POINTER(i32)]
            lib.attn_kv_block_masked.restype = i32
            lib.attn_kv_block_masked.argtypes = [i32] * 9
            _lib = lib
    return _lib


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(t, name, dtype, ndim):
    if (type(t) is torch.Tensor and t.dtype is dtype and t.dim() == ndim and t.is_cuda
            and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def attn_bwd_workspace_bytes(total_q, nheads_q) -> int:
    return int(load().attn_bwd_workspace_bytes(int(total_q), int(nheads_q)))


def attn_fwd_workspace_bytes(batch, max_seqlen_q, nheads_q, nheads_kv) -> int:
    return int(load().attn_fwd_workspace_bytes(batch, max_seqlen_q, nheads_q, nheads_kv))


def attn_decode_workspace_bytes(batch, nheads_q, head_dim, num_splits) -> int:
    return int(load().attn_decode_workspace_bytes(batch, nheads_q, head_dim, num_splits))


def attn_decode_num_splits(batch, nheads_q, nheads_kv, max_pages_per_seq, page_size, num_sms):
    return int(load().attn_decode_num_splits(batch, nheads_q, nheads_kv, max_pages_per_seq,
                                             page_size, num_sms))


def attn_kv_block_range(i_min, i_max, seqlen_q, seqlen_k, block_n, causal, wl, wr):
    lo, hi = ctypes.c_int(), ctypes.c_int()
    rc = load().attn_kv_block_range(i_min, i_max, seqlen_q, seqlen_k, block_n, int(causal), wl,
                                    wr, ctypes.byref(lo), ctypes.byref(hi))
    if rc != 0:
        raise AttnError(-1, "attn_kv_block_range")
    return lo.value, hi.value


def attn_kv_block_masked(j, i_min, i_max, seqlen_q, seqlen_k, block_n, causal, wl, wr) -> bool:
    return bool(load().attn_kv_block_masked(j, i_min, i_max, seqlen_q, seqlen_k, block_n,
                                            int(causal), wl, wr))


def attn_get_device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status code."""
    return int(load().attn_get_device_status(_stream(stream)))


def attn_selftest_wait_timeout(stream=None) -> int:
    """Launch the bounded-wait self-test kernel (its wait runs out after 20 ms)."""
    return int(load().attn_selftest_wait_timeout(_stream(stream)))


def attn_selftest_softcap(scores, softmax_scale: float, softcap: float, stream=None):
    """softcap * tanh(softmax_scale * scores / softcap) as the modifier kernel computes it
    (scores: contiguous device fp32, even length)."""
    _check(scores, "scores", torch.float32, 1)
    out = torch.empty_like(scores)
    rc = load().attn_selftest_softcap(_ptr(scores), _ptr(out), scores.numel(),
                                      float(softmax_scale), float(softcap), _stream(stream))
    if rc != 0:
        raise AttnError(rc, "attn_selftest_softcap")
    return out


def _workspace(nbytes, device, workspace):
    if nbytes == 0:
        return None
    if workspace is not None:
        if workspace.numel() * workspace.element_size() < nbytes:
            raise AttnError(-3, "workspace")
        return workspace
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def attn_fwd(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k,
             softmax_scale=None, causal=False, window_left=-1, window_right=-1,
             out=None, lse=None, workspace=None, stream=None):
    """Varlen prefill.  q [total_q, Hq, d], k/v [total_k, Hkv, d] bf16; cu_seqlens int32.

    Returns (out [total_q, Hq, d] bf16, lse [Hq, total_q] fp32).
    """
    lib = load()
    _check(q, "q", torch.bfloat16, 3)
    _check(k, "k", torch.bfloat16, 3)
    _check(v, "v", torch.bfloat16, 3)
    _check(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    _check(cu_seqlens_k, "cu_seqlens_k", torch.int32, 1)
    total_q, Hq, d = q.shape
    total_k, Hkv, dk = k.shape
    if v.shape != k.shape or dk != d:
        raise ValueError("k and v must both be [total_k, Hkv, d] with q's d")
    batch = cu_seqlens_q.numel() - 1
    if cu_seqlens_k.numel() != batch + 1:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must have the same length")
    scale = d ** -0.5 if softmax_scale is None else float(softmax_scale)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((Hq, total_q), dtype=torch.float32, device=q.device)
    _check(out, "out", torch.bfloat16, 3)
    _check(lse, "lse", torch.float32, 2)
    nbytes = int(lib.attn_fwd_workspace_bytes(max(batch, 0), int(max_seqlen_q), Hq, Hkv))
    ws = _workspace(nbytes, q.device, workspace)
    rc = lib.attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(cu_seqlens_q),
                      _ptr(cu_seqlens_k), batch, total_q, total_k, int(max_seqlen_q),
                      int(max_seqlen_k), Hq, Hkv, d, scale, int(bool(causal)), int(window_left),
                      int(window_right), _ptr(ws), nbytes, _stream(stream))
    if rc != 0:
        raise AttnError(rc, "attn_fwd")
    return out, lse


def attn_fwd_mods(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k,
                  softmax_scale=None, causal=False, window_left=-1, window_right=-1,
                  softcap=0.0, alibi_slopes=None, out=None, lse=None, workspace=None,
                  stream=None):
    """attn_fwd with softcap (0 = off) and ALiBi slopes (fp32 [Hq] CUDA tensor or None)."""
    lib = load()
    _check(q, "q", torch.bfloat16, 3)
    _check(k, "k", torch.bfloat16, 3)
    _check(v, "v", torch.bfloat16, 3)
    if alibi_slopes is not None:
        _check(alibi_slopes, "alibi_slopes", torch.float32, 1)
    total_q, Hq, d = q.shape
    total_k, Hkv, _ = k.shape
    batch = cu_seqlens_q.numel() - 1
    scale = d ** -0.5 if softmax_scale is None else float(softmax_scale)
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty((Hq, total_q), dtype=torch.float32, device=q.device) if lse is None else lse
    nbytes = int(lib.attn_fwd_workspace_bytes(max(batch, 0), int(max_seqlen_q), Hq, Hkv))
    ws = _workspace(nbytes, q.device, workspace)
    rc = lib.attn_fwd_mods(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(cu_seqlens_q),
                           _ptr(cu_seqlens_k), batch, total_q, total_k, int(max_seqlen_q),
                           int(max_seqlen_k), Hq, Hkv, d, scale, int(bool(causal)),
                           int(window_left), int(window_right), float(softcap),
                           _ptr(alibi_slopes), _ptr(ws), nbytes, _stream(stream))
    if rc != 0:
        raise AttnError(rc, "attn_fwd_mods")
    return out, lse


def attn_quantize_fp8(q, k, v, cu_seqlens_k, max_seqlen_k, signs=None, key_blocks=None,
                      stream=None):
    """bf16 q, k, v (d = 128) -> (q8, q_scale, k8, k_scale, v8t, v_scale) for attn_fwd_fp8.
    signs: fp32 [128] CUDA tensor of +-1 (rotate Q and K) or None.  key_blocks defaults to
    ceil(total_k / 128) + batch."""
    lib = load()
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n, torch.bfloat16, 3)
    if signs is not None:
        _check(signs, "signs", torch.float32, 1)
    total_q, Hq, d = q.shape
    total_k, Hkv, _ = k.shape
    batch = cu_seqlens_k.numel() - 1
    kb = (total_k + 127) // 128 + batch if key_blocks is None else int(key_blocks)
    dev = q.device
    q8 = torch.empty((total_q, Hq, d), dtype=torch.uint8, device=dev)
    qs = torch.empty((Hq, max(1, (total_q + 127) // 128)), dtype=torch.float32, device=dev)
    k8 = torch.empty((total_k, Hkv, d), dtype=torch.uint8, device=dev)
    ks = torch.empty((Hkv, kb), dtype=torch.float32, device=dev)
    v8t = torch.empty((Hkv, d, 128 * kb), dtype=torch.uint8, device=dev)
    vs = torch.empty((max(batch, 1), Hkv), dtype=torch.float32, device=dev)
    rc = lib.attn_quantize_fp8(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens_k), batch, total_q,
                               total_k, int(max_seqlen_k), Hq, Hkv, d, kb, _ptr(signs), _ptr(q8),
                               _ptr(qs), _ptr(k8), _ptr(ks), _ptr(v8t), _ptr(vs), _stream(stream))
    if rc != 0:
        raise AttnError(rc, "attn_quantize_fp8")
    return q8, qs, k8, ks, v8t, vs


def attn_fwd_fp8(q8, k8, v8t, q_scale, k_scale, v_scale, cu_seqlens_q, cu_seqlens_k,
                 max_seqlen_q, max_seqlen_k, softmax_scale=None, causal=False, window_left=-1,
                 window_right=-1, out=None, lse=None, stream=None):
    """FP8 (e4m3) forward.  q8 [total_q, Hq, 128], k8 [total_k, Hkv, 128] and v8t [Hkv, 128,
    128 * key_blocks] are uint8 e4m3 codes; q_scale [Hq, ceil(total_q/128)], k_scale [Hkv,
    key_blocks], v_scale [batch, Hkv] fp32.  Returns (out bf16, lse fp32) as attn_fwd."""
    lib = load()
    _check(q8, "q8", torch.uint8, 3)
    _check(k8, "k8", torch.uint8, 3)
    _check(v8t, "v8t", torch.uint8, 3)
    _check(q_scale, "q_scale", torch.float32, 2)
    _check(k_scale, "k_scale", torch.float32, 2)
    _check(v_scale, "v_scale", torch.float32, 2)
    total_q, Hq, d = q8.shape
    total_k, Hkv, _ = k8.shape
    key_blocks = k_scale.shape[1]
    if v8t.shape != (Hkv, d, 128 * key_blocks):
        raise ValueError("v8t must be [Hkv, d, 128 * key_blocks]")
    batch = cu_seqlens_q.numel() - 1
    scale = d ** -0.5 if softmax_scale is None else float(softmax_scale)
    out = torch.empty((total_q, Hq, d), dtype=torch.bfloat16, device=q8.device) if out is None else out
    lse = torch.empty((Hq, total_q), dtype=torch.float32, device=q8.device) if lse is None else lse
    rc = lib.attn_fwd_fp8(_ptr(q8), _ptr(k8), _ptr(v8t), _ptr(q_scale), _ptr(k_scale),
                          _ptr(v_scale), _ptr(out), _ptr(lse), _ptr(cu_seqlens_q),
                          _ptr(cu_seqlens_k), batch, total_q, total_k, int(max_seqlen_q),
                          int(max_seqlen_k), Hq, Hkv, d, key_blocks, scale, int(bool(causal)),
                          int(window_left), int(window_right), _stream(stream))
    if rc != 0:
        raise AttnError(rc, "attn_fwd_fp8")
    return out, lse


def attn_bwd(q, k, v, out, dout, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k,
             softmax_scale=None, causal=False, window_left=-1, window_right=-1, dq=None,
             dk=None, dv=None, workspace=None, stream=None):
    """Gradients of sum(out * dout) for attn_fwd.  Returns (dq, dk, dv), bf16."""
    lib = load()
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (out, "out"), (dout, "dout")):
        _check(t, n, torch.bfloat16, 3)
    _check(lse, "lse", torch.float32, 2)
    _check(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    _check(cu_seqlens_k, "cu_seqlens_k", torch.int32, 1)
    total_q, Hq, d = q.shape
    total_k, Hkv, _ = k.shape
    batch = cu_seqlens_q.numel() - 1
    scale = d ** -0.5 if softmax_scale is None else float(softmax_scale)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    nbytes = int(lib.attn_bwd_workspace_bytes(total_q, Hq))
    ws = _workspace(nbytes, q.device, workspace)
    rc = lib.attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse), _ptr(dq),
                      _ptr(dk), _ptr(dv), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), batch, total_q,
                      total_k, int(max_seqlen_q), int(max_seqlen_k), Hq, Hkv, d, scale,
                      int(bool(causal)), int(window_left), int(window_right), _ptr(ws), nbytes,
                      _stream(stream))
    if rc != 0:
        raise AttnError(rc, "attn_bwd")
    return dq, dk, dv


def attn_fwd_kvcache(q, k_new, v_new, k_cache, v_cache, cache_seqlens, block_table,
                     cu_seqlens_q, max_seqlen_q, softmax_scale=None, causal=True,
                     window_left=-1, window_right=-1, rotary_cos=None, rotary_sin=None,
                     rotary_interleaved=False, out=None, lse=None, workspace=None, stream=None):
    """Chunked prefill against a paged cache; the new k, v (rotated k) are written into it.

    q [total_q, Hq, d], k_new / v_new [total_q, Hkv, d] bf16; caches
    [num_pages, page_size, Hkv, d] bf16 (updated in place); cache_seqlens [batch],
    block_table [batch, max_pages], cu_seqlens_q [batch + 1] int32; rotary_cos / rotary_sin
    fp32 [rows, rotary_dim / 2] or None.  Returns (out [total_q, Hq, d], lse [Hq, total_q]).
    """
    lib = load()
    _check(q, "q", torch.bfloat16, 3)
    _check(k_new, "k_new", torch.bfloat16, 3)
    _check(v_new, "v_new", torch.bfloat16, 3)
    _check(k_cache, "k_cache", torch.bfloat16, 4)
    _check(v_cache, "v_cache", torch.bfloat16, 4)
    _check(cache_seqlens, "cache_seqlens", torch.int32, 1)
    _check(block_table, "block_table", torch.int32, 2)
    _check(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    total_q, Hq, d = q.shape
    num_pages, page_size, Hkv, dk = k_cache.shape
    if v_cache.shape != k_cache.shape or dk != d or k_new.shape != (total_q, Hkv, d) or \
            v_new.shape != k_new.shape:
        raise ValueError("inconsistent q / k_new / v_new / cache shapes")
    batch = cu_seqlens_q.numel() - 1
    if cache_seqlens.numel() != batch or block_table.shape[0] != batch:
        raise ValueError("cache_seqlens and block_table must have one row per sequence")
    if rotary_cos is not None:
        _check(rotary_cos, "rotary_cos", torch.float32, 2)
        _check(rotary_sin, "rotary_sin", torch.float32, 2)
        rot_rows, rot_dim = rotary_cos.shape[0], 2 * rotary_cos.shape[1]
    else:
        rot_rows = rot_dim = 0
    scale = d ** -0.5 if softmax_scale is None else float(softmax_scale)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((Hq, total_q), dtype=torch.float32, device=q.device)
    nbytes = int(lib.attn_fwd_kvcache_workspace_bytes(max(batch, 0), total_q, int(max_seqlen_q),
                                                      Hq, Hkv, d, rot_dim))
    ws = _workspace(nbytes, q.device, workspace)
    rc = lib.attn_fwd_kvcache(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                              _ptr(cache_seqlens), _ptr(block_table), _ptr(cu_seqlens_q),
                              _ptr(rotary_cos), _ptr(rotary_sin), rot_dim, rot_rows,
                              int(bool(rotary_interleaved)), _ptr(out), _ptr(lse), batch, total_q,
                              int(max_seqlen_q), Hq, Hkv, d, page_size, block_table.shape[1],
                              num_pages, scale, int(bool(causal)), int(window_left),
                              int(window_right), _ptr(ws), nbytes, _stream(stream))
    if rc != 0:
        raise AttnError(rc, "attn_fwd_kvcache")
    return out, lse


def _decode_shapes(q, k_cache, v_cache, cache_seqlens, block_table):
    """Checks shared by both decode entry points: dtypes, ranks, and one table row and one
    length per sequence (a short table or length vector would be read past its end)."""
    _check(q, "q", torch.bfloat16, 3)
    _check(k_cache, "k_cache", torch.bfloat16, 4)
    _check(v_cache, "v_cache", torch.bfloat16, 4)
    _check(cache_seqlens, "cache_seqlens", torch.int32, 1)
    _check(block_table, "block_table", torch.int32, 2)
    batch, Hq, d = q.shape
    num_pages, page_size, Hkv, dk = k_cache.shape
    if v_cache.shape != k_cache.shape or dk != d:
        raise ValueError("k_cache and v_cache must both be [num_pages, page_size, Hkv, d]")
    if cache_seqlens.numel() != batch or block_table.shape[0] != batch:
        raise ValueError("cache_seqlens and block_table must have one row per sequence")
    return batch, Hq, Hkv, d, num_pages, page_size


def _decode_outputs(q, out, lse):
    batch, Hq, _ = q.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((batch, Hq), dtype=torch.float32, device=q.device)
    _check(out, "out", torch.bfloat16, 3)
    _check(lse, "lse", torch.float32, 2)
    if tuple(out.shape) != tuple(q.shape) or tuple(lse.shape) != (batch, Hq):
        raise ValueError("out must be [batch, Hq, d] and lse [batch, Hq]")
    return out, lse


def attn_decode_kvcache(q, k_cache, v_cache, cache_seqlens, block_table, softmax_scale=None,
                        num_splits=0, out=None, lse=None, workspace=None, stream=None):
    """Decode over a paged cache.  q [batch, Hq, d]; caches [num_pages, page_size, Hkv, d].

    Returns (out [batch, Hq, d] bf16, lse [batch, Hq] fp32).
    """
    lib = load()
    batch, Hq, Hkv, d, num_pages, page_size = _decode_shapes(q, k_cache, v_cache, cache_seqlens,
                                                             block_table)
    scale = d ** -0.5 if softmax_scale is None else float(softmax_scale)
    out, lse = _decode_outputs(q, out, lse)
    nbytes = int(lib.attn_decode_workspace_bytes(batch, Hq, d, int(num_splits)))
    ws = _workspace(nbytes, q.device, workspace)
    rc = lib.attn_decode_kvcache(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(cache_seqlens),
                                 _ptr(block_table), page_size, int(num_splits), _ptr(out),
                                 _ptr(lse), batch, Hq, Hkv, d, block_table.shape[1], num_pages,
                                 scale, _ptr(ws), nbytes, _stream(stream))
    if rc != 0:
        raise AttnError(rc, "attn_decode_kvcache")
    return out, lse


def attn_decode_kvcache_noalloc(q, k_cache, v_cache, cache_seqlens, block_table,
                                softmax_scale=None, num_splits=0, out=None, lse=None,
                                stream=None):
    """Decode over a paged cache without any workspace from the caller.

    For callers that cannot allocate device memory: the split partials live in a 32 MiB
    scratch array owned by the library (see attn_decode_kvcache_noalloc in include/attn.h).
    Calls on one device share that array, so calls whose kernels overlap on the GPU race.
    The outputs are allocated here only when `out` / `lse` are not given.
    """
    lib = load()
    fn = lib.attn_decode_kvcache_noalloc
    if fn.argtypes is None:
        P, i32, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        fn.restype = i32
        fn.argtypes = [P, P, P, P, P, i32, i32, P, P, i32, i32, i32, i32, i32, i32, f32, P]
    batch, Hq, Hkv, d, num_pages, page_size = _decode_shapes(q, k_cache, v_cache, cache_seqlens,
                                                             block_table)
    scale = d ** -0.5 if softmax_scale is None else float(softmax_scale)
    out, lse = _decode_outputs(q, out, lse)
    rc = fn(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(cache_seqlens), _ptr(block_table),
            page_size, int(num_splits), _ptr(out), _ptr(lse), batch, Hq, Hkv, d,
            block_table.shape[1], num_pages, scale, _stream(stream))
    if rc != 0:
        raise AttnError(rc, "attn_decode_kvcache_noalloc")
    return out, lse


# ---- 8-bit paged KV cache ------------------------------------------------------------------


# The current stream's handle without building a Stream object (a few microseconds a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


def _on(index, stream, body, *args):
    """body(stream handle, *args) with device `index` current and what it allocates belonging to
    `stream` (default: the device's current stream)."""
    if stream is None:
        if torch.cuda.current_device() == index:
            return body(_raw_stream(index), *args)
        with torch.cuda.device(index):
            return body(_raw_stream(index), *args)
    if stream.device.index != index:
        raise ValueError("the stream must belong to the tensors' device")
    with torch.cuda.device(index), torch.cuda.stream(stream):
        return body(stream.cuda_stream, *args)


_U8, _I32, _BF16, _F32 = torch.uint8, torch.int32, torch.bfloat16, torch.float32

# Each call below asks all it wants to know of its tensors in one expression: a function call per
# tensor was a third of a small call's time on the host.  What the expression does not accept goes
# to _refuse.
_WRONG = (AttributeError, TypeError, ValueError)  # of a None, another type, another number of dims


def _refuse(shapes, *args):
    """Raise for the first of args, (tensor, name, dtype, dims), that is not a contiguous tensor of
    its kind on the first one's CUDA device, or else for their sizes."""
    for t, name, dtype, ndim in args:
        _check(t, name, dtype, ndim)
        if t.get_device() != args[0][0].get_device():
            raise ValueError("all tensors must be on one CUDA device")
    raise ValueError(shapes)


def _kv8_sizes(k_cache, v_cache, k_scale, v_scale, block_table):
    """(num_pages, page_size, Hkv, d, batch, max_pages, device index) of an 8-bit cache."""
    try:
        shape = k_cache.shape
        num_pages, page_size, Hkv, d = shape
        scales = (num_pages, Hkv, page_size)
        batch, max_pages = block_table.shape
        index = k_cache.get_device()
        if (index >= 0 and k_cache.dtype is _U8 and v_cache.dtype is _U8 and k_scale.dtype is _U8
                and v_scale.dtype is _U8 and block_table.dtype is _I32 and v_cache.shape == shape
                and k_scale.shape == scales and v_scale.shape == scales
                and k_cache.is_contiguous() and v_cache.is_contiguous()
                and k_scale.is_contiguous() and v_scale.is_contiguous()
                and block_table.is_contiguous()
                and v_cache.get_device() == k_scale.get_device() == v_scale.get_device()
                == block_table.get_device() == index):
            return num_pages, page_size, Hkv, d, batch, max_pages, index
    except _WRONG:
        pass
    _refuse("k_cache and v_cache must be [num_pages, page_size, Hkv, d], k_scale and v_scale "
            "[num_pages, Hkv, page_size], block_table [batch, max_pages]",
            (k_cache, "k_cache", _U8, 4), (v_cache, "v_cache", _U8, 4),
            (k_scale, "k_scale", _U8, 3), (v_scale, "v_scale", _U8, 3),
            (block_table, "block_table", _I32, 2))


def _rotary(rotary_cos, rotary_sin, index):
    """(cos address, sin address, rotary_dim, rows)."""
    if rotary_cos is None and rotary_sin is None:
        return None, None, 0, 0
    try:
        shape = rotary_cos.shape
        rows, half = shape
        if (rotary_cos.dtype is _F32 and rotary_sin.dtype is _F32 and rotary_sin.shape == shape
                and rotary_cos.is_contiguous() and rotary_sin.is_contiguous()
                and rotary_cos.get_device() == rotary_sin.get_device() == index):
            return rotary_cos.data_ptr(), rotary_sin.data_ptr(), 2 * half, rows
    except _WRONG:
        pass
    _refuse("rotary_cos and rotary_sin must both be [rows, rotary_dim / 2] on the cache's device",
            (rotary_cos, "rotary_cos", _F32, 2), (rotary_sin, "rotary_sin", _F32, 2))


def _new_tokens(k_new, v_new, cache_seqlens, cu_seqlens_q, batch, Hkv, d, index):
    """The addresses of the new tokens' keys and values and of the lengths, and the tokens."""
    try:
        shape = k_new.shape
        total_q, heads, dim = shape
        if (heads == Hkv and dim == d and v_new.shape == shape and cache_seqlens.shape == (batch,)
                and cu_seqlens_q.shape == (batch + 1,) and k_new.dtype is _BF16
                and v_new.dtype is _BF16 and cache_seqlens.dtype is _I32
                and cu_seqlens_q.dtype is _I32 and k_new.is_contiguous() and v_new.is_contiguous()
                and cache_seqlens.is_contiguous() and cu_seqlens_q.is_contiguous()
                and k_new.get_device() == v_new.get_device() == cache_seqlens.get_device()
                == cu_seqlens_q.get_device() == index):
            return (k_new.data_ptr(), v_new.data_ptr(), cache_seqlens.data_ptr(),
                    cu_seqlens_q.data_ptr(), total_q)
    except _WRONG:
        pass
    _refuse("k_new and v_new must be [total_q, Hkv, d] with the cache's Hkv and d, cache_seqlens "
            "[batch] and cu_seqlens_q [batch + 1] with block_table's batch, on the cache's device",
            (k_new, "k_new", _BF16, 3), (v_new, "v_new", _BF16, 3),
            (cache_seqlens, "cache_seqlens", _I32, 1), (cu_seqlens_q, "cu_seqlens_q", _I32, 1))


def _output(t, name, dtype, shape, index):
    """Checks an output that the caller passes."""
    _check(t, name, dtype, len(shape))
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on the cache's device")


def _kv8_workspace(nbytes, device, workspace):
    if workspace is not None and not (workspace.is_contiguous() and workspace.device == device):
        # (the elements of one that is not contiguous may share memory)
        raise ValueError("workspace must be contiguous and on the cache's device")
    return _workspace(nbytes, device, workspace)


def _int32(value, name):
    """A size or bound that the library takes as a C int (ctypes would drop what is above it)."""
    n = int(value)
    if not -2 ** 31 <= n < 2 ** 31:
        raise ValueError(f"{name} must fit 32 bits")
    return n


def attn_kvcache_append_fp8(k_new, v_new, k_cache, v_cache, k_scale, v_scale, cache_seqlens,
                            block_table, cu_seqlens_q, rotary_cos=None, rotary_sin=None,
                            rotary_interleaved=False, stream=None):
    """Write new tokens' keys (rotated) and values into the 8-bit paged cache, in place.

    k_new / v_new [total_q, Hkv, d] bf16; caches uint8 e4m3 codes [num_pages, page_size, Hkv, d]
    with scale bytes uint8 [num_pages, Hkv, page_size]; token i of sequence b goes to position
    cache_seqlens[b] + i.  rotary_cos / rotary_sin fp32 [rows, rotary_dim / 2] or None.
    """
    lib = load()
    num_pages, page_size, Hkv, d, batch, max_pages, index = _kv8_sizes(
        k_cache, v_cache, k_scale, v_scale, block_table)
    kn, vn, sl, cu, total_q = _new_tokens(k_new, v_new, cache_seqlens, cu_seqlens_q, batch, Hkv, d,
                                          index)
    cos, sin, rot_dim, rot_rows = _rotary(rotary_cos, rotary_sin, index)

    def body(s):
        return lib.attn_kvcache_append_fp8(
            kn, vn, k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
            sl, block_table.data_ptr(), cu, cos, sin, rot_dim, rot_rows,
            1 if rotary_interleaved else 0, batch, total_q, Hkv, d, page_size, max_pages,
            num_pages, s)

    rc = _on(index, stream, body)
    if rc != 0:
        raise AttnError(rc, "attn_kvcache_append_fp8")


def attn_kvcache_read_fp8(k_cache, v_cache, k_scale, v_scale, block_table, cu_seqlens_k, total_k,
                          k=None, v=None, stream=None):
    """Read the first cu_seqlens_k[b + 1] - cu_seqlens_k[b] tokens of every sequence of the 8-bit
    cache back.  Returns (k, v), bf16 [total_k, Hkv, d], packed as attn_fwd takes them."""
    lib = load()
    num_pages, page_size, Hkv, d, batch, max_pages, index = _kv8_sizes(
        k_cache, v_cache, k_scale, v_scale, block_table)
    try:
        ok = (cu_seqlens_k.shape == (batch + 1,) and cu_seqlens_k.dtype is _I32
              and cu_seqlens_k.is_contiguous() and cu_seqlens_k.get_device() == index)
    except _WRONG:
        ok = False
    if not ok:
        _refuse("cu_seqlens_k must be [batch + 1] with block_table's batch, on the cache's device",
                (cu_seqlens_k, "cu_seqlens_k", _I32, 1))
    shape = (_int32(total_k, "total_k"), Hkv, d)
    if k is not None:
        _output(k, "k", _BF16, shape, index)
    if v is not None:
        _output(v, "v", _BF16, shape, index)

    def body(s):
        device = k_cache.device
        ko = torch.empty(shape, dtype=_BF16, device=device) if k is None else k
        vo = torch.empty(shape, dtype=_BF16, device=device) if v is None else v
        rc = lib.attn_kvcache_read_fp8(
            k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
            block_table.data_ptr(), cu_seqlens_k.data_ptr(), ko.data_ptr(), vo.data_ptr(), batch,
            shape[0], Hkv, d, page_size, max_pages, num_pages, s)
        if rc != 0:
            raise AttnError(rc, "attn_kvcache_read_fp8")
        return ko, vo

    return _on(index, stream, body)


def attn_decode_kvcache_fp8_workspace_bytes(batch, nheads_q, nheads_kv, head_dim, page_size,
                                            max_pages_per_seq) -> int:
    return int(load().attn_decode_kvcache_fp8_workspace_bytes(
        batch, nheads_q, nheads_kv, head_dim, page_size, max_pages_per_seq))


def attn_decode_kvcache_fp8(q, k_cache, v_cache, k_scale, v_scale, cache_seqlens, block_table,
                            softmax_scale=None, out=None, lse=None, workspace=None, stream=None):
    """Decode over the 8-bit paged cache.  q [batch, Hq, d] bf16, one token per sequence.

    Returns (out [batch, Hq, d] bf16, lse [batch, Hq] fp32).
    """
    lib = load()
    num_pages, page_size, Hkv, d, batch, max_pages, index = _kv8_sizes(
        k_cache, v_cache, k_scale, v_scale, block_table)
    try:
        rows, Hq, dim = q.shape
        ok = (rows == batch and dim == d and cache_seqlens.shape == (batch,) and q.dtype is _BF16
              and cache_seqlens.dtype is _I32 and q.is_contiguous()
              and cache_seqlens.is_contiguous()
              and q.get_device() == cache_seqlens.get_device() == index)
    except _WRONG:
        ok = False
    if not ok:
        _refuse("q must be [batch, Hq, d] with the cache's d and block_table's batch, cache_seqlens "
                "[batch], on the cache's device",
                (q, "q", _BF16, 3), (cache_seqlens, "cache_seqlens", _I32, 1))
    if out is not None:
        _output(out, "out", _BF16, (batch, Hq, d), index)
    if lse is not None:
        _output(lse, "lse", _F32, (batch, Hq), index)
    scale = d ** -0.5 if softmax_scale is None else float(softmax_scale)
    nbytes = lib.attn_decode_kvcache_fp8_workspace_bytes(batch, Hq, Hkv, d, page_size, max_pages)

    def body(s):
        device = q.device
        o = torch.empty_like(q) if out is None else out
        l = torch.empty((batch, Hq), dtype=_F32, device=device) if lse is None else lse
        ws = _kv8_workspace(nbytes, device, workspace)
        rc = lib.attn_decode_kvcache_fp8(
            q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
            v_scale.data_ptr(), cache_seqlens.data_ptr(), block_table.data_ptr(), page_size,
            o.data_ptr(), l.data_ptr(), batch, Hq, Hkv, d, max_pages, num_pages, scale, _ptr(ws),
            nbytes, s)
        if rc != 0:
            raise AttnError(rc, "attn_decode_kvcache_fp8")
        return o, l

    return _on(index, stream, body)


def attn_fwd_kvcache_fp8_workspace_bytes(batch, total_q, max_seqlen_q, max_total_k, nheads_q,
                                         nheads_kv, head_dim, page_size, max_pages_per_seq,
                                         rotary_dim=0) -> int:
    return int(load().attn_fwd_kvcache_fp8_workspace_bytes(
        batch, total_q, max_seqlen_q, max_total_k, nheads_q, nheads_kv, head_dim, page_size,
        max_pages_per_seq, rotary_dim))


def attn_fwd_kvcache_fp8(q, k_new, v_new, k_cache, v_cache, k_scale, v_scale, cache_seqlens,
                         block_table, cu_seqlens_q, max_seqlen_q, max_total_k=None,
                         softmax_scale=None, causal=True, window_left=-1, window_right=-1,
                         rotary_cos=None, rotary_sin=None, rotary_interleaved=False, out=None,
                         lse=None, workspace=None, stream=None):
    """A chunk of new tokens against the 8-bit paged cache; the new k, v are written into it.

    q [total_q, Hq, d], k_new / v_new [total_q, Hkv, d] bf16; the cache as for
    attn_kvcache_append_fp8.  Returns (out [total_q, Hq, d], lse [Hq, total_q]).

    max_total_k bounds sum_b (cache_seqlens[b] + new tokens of b) and sizes the workspace of calls
    with a long chunk: about 4 Hkv d bytes a key.  The default is what block_table can hold, so
    give the bound where the table is wider than the sequences are long (64 rows of 131072
    tokens, 8 kv heads, d 128: 32 GiB).
    """
    lib = load()
    num_pages, page_size, Hkv, d, batch, max_pages, index = _kv8_sizes(
        k_cache, v_cache, k_scale, v_scale, block_table)
    kn, vn, sl, cu, total_q = _new_tokens(k_new, v_new, cache_seqlens, cu_seqlens_q, batch, Hkv, d,
                                          index)
    try:
        rows, Hq, dim = q.shape
        ok = (rows == total_q and dim == d and q.dtype is _BF16 and q.is_contiguous()
              and q.get_device() == index)
    except _WRONG:
        ok = False
    if not ok:
        _refuse("q must be [total_q, Hq, d] with k_new's tokens and d, on the cache's device",
                (q, "q", _BF16, 3))
    cos, sin, rot_dim, rot_rows = _rotary(rotary_cos, rotary_sin, index)
    if out is not None:
        _output(out, "out", _BF16, (total_q, Hq, d), index)
    if lse is not None:
        _output(lse, "lse", _F32, (Hq, total_q), index)
    max_q = _int32(max_seqlen_q, "max_seqlen_q")
    total_k = (min(batch * max_pages * page_size, 2 ** 31 - 1) if max_total_k is None
               else _int32(max_total_k, "max_total_k"))
    left, right = _int32(window_left, "window_left"), _int32(window_right, "window_right")
    scale = d ** -0.5 if softmax_scale is None else float(softmax_scale)
    nbytes = lib.attn_fwd_kvcache_fp8_workspace_bytes(batch, total_q, max_q, total_k, Hq, Hkv, d,
                                                      page_size, max_pages, rot_dim)

    def body(s):
        device = q.device
        o = torch.empty_like(q) if out is None else out
        l = torch.empty((Hq, total_q), dtype=_F32, device=device) if lse is None else lse
        ws = _kv8_workspace(nbytes, device, workspace)
        rc = lib.attn_fwd_kvcache_fp8(
            q.data_ptr(), kn, vn, k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
            v_scale.data_ptr(), sl, block_table.data_ptr(), cu, cos, sin, rot_dim, rot_rows,
            1 if rotary_interleaved else 0, o.data_ptr(), l.data_ptr(), batch, total_q, max_q,
            total_k, Hq, Hkv, d, page_size, max_pages, num_pages, scale, 1 if causal else 0,
            left, right, _ptr(ws), nbytes, s)
        if rc != 0:
            raise AttnError(rc, "attn_fwd_kvcache_fp8")
        return o, l

    return _on(index, stream, body)


# ---- a step around paged attention -----------------------------------------------------------


def _step_tensor(t, name, dtype, shape, index):
    """Checks an input: a dense tensor of this dtype and shape (None: any size) on the call's device."""
    try:
        if (t.dtype is dtype and t.get_device() == index and t.is_contiguous()
                and (t.shape == shape or (len(t.shape) == len(shape) and all(
                    want is None or want == got for want, got in zip(shape, t.shape))))):
            return t.data_ptr()
    except _WRONG:
        pass
    _check(t, name, dtype, len(shape))
    if t.get_device() != index:
        raise ValueError(f"{name} must be on the device of the call's other tensors")
    raise ValueError(f"{name} must be {['any' if n is None else n for n in shape]}, got "
                     f"{list(t.shape)}")


def _device_index(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def attn_kvcache_plan_workspace_bytes(batch, total_q) -> int:
    return int(load().attn_kvcache_plan_workspace_bytes(batch, total_q))


_PLAN_OUTPUTS = ("cu_seqlens_q", "seqlens_after", "positions", "slot_map", "free_left")


def attn_kvcache_plan(cache_seqlens, new_lens, block_table, free_pages, free_count, page_size,
                      num_pages, total_q, cu_seqlens_q=None, seqlens_after=None, positions=None,
                      slot_map=None, free_left=None, workspace=None, stream=None):
    """Pages, positions and cache slots of a step's new tokens, from the lengths of its requests.

    cache_seqlens, new_lens [batch]; block_table [batch, max_pages], updated in place; free_pages
    [n], of which the first free_count[0] are free and are taken from the end; all int32.  total_q,
    at least sum(new_lens), sizes the outputs (behind the last token: position 0, slot -1).
    Returns (cu_seqlens_q [batch + 1], seqlens_after [batch], positions [total_q],
    slot_map [total_q], free_left [1]), int32; free_left may be free_count and seqlens_after
    cache_seqlens.
    """
    lib = load()
    total, ps, pages = _int32(total_q, "total_q"), _int32(page_size, "page_size"), _int32(num_pages, "num_pages")
    try:
        batch, max_pages = block_table.shape
        index = block_table.get_device()
        ok = (index >= 0 and cache_seqlens.shape == new_lens.shape == (batch,) and free_count.shape == (1,)
              and cache_seqlens.dtype is _I32 and new_lens.dtype is _I32 and block_table.dtype is _I32
              and free_pages.dtype is _I32 and free_count.dtype is _I32 and len(free_pages.shape) == 1
              and cache_seqlens.is_contiguous() and new_lens.is_contiguous()
              and block_table.is_contiguous() and free_pages.is_contiguous()
              and cache_seqlens.get_device() == new_lens.get_device() == free_pages.get_device()
              == free_count.get_device() == index)
    except _WRONG:
        ok = False
    if not ok:
        _refuse("cache_seqlens and new_lens must be [batch] with block_table's batch, free_count [1]",
                (block_table, "block_table", _I32, 2), (cache_seqlens, "cache_seqlens", _I32, 1),
                (new_lens, "new_lens", _I32, 1), (free_pages, "free_pages", _I32, 1),
                (free_count, "free_count", _I32, 1))
    if total < 0:
        raise AttnError(-1, "attn_kvcache_plan")
    given = (cu_seqlens_q, seqlens_after, positions, slot_map, free_left)
    sizes = (batch + 1, batch, total, total, 1)
    for t, name, size in zip(given, _PLAN_OUTPUTS, sizes):
        if t is not None:
            _step_tensor(t, name, _I32, (size,), index)
    nbytes = lib.attn_kvcache_plan_workspace_bytes(batch, total)

    def body(s):
        device = block_table.device
        outs = [torch.empty(size, dtype=_I32, device=device) if t is None else t
                for t, size in zip(given, sizes)]
        ws = _kv8_workspace(nbytes, device, workspace)
        cu, after, pos, slots, left = outs
        rc = lib.attn_kvcache_plan(
            cache_seqlens.data_ptr(), new_lens.data_ptr(), block_table.data_ptr(),
            free_pages.data_ptr(), free_count.data_ptr(), left.data_ptr(), cu.data_ptr(),
            after.data_ptr(), pos.data_ptr(), slots.data_ptr(), batch, total, ps, max_pages,
            free_pages.shape[0], pages, _ptr(ws), nbytes, s)
        if rc != 0:
            raise AttnError(rc, "attn_kvcache_plan")
        return tuple(outs)

    return _on(index, stream, body)


def _apart(t, heads, d):
    """Elements between the tokens of [tokens, heads, d] whose tokens are dense but may lie apart, as the
    parts of a projection's rows do (None: they are not dense)."""
    st, sh, sd = t.stride()
    if sd != 1 or (sh != d and heads != 1):
        return None
    return st if t.shape[0] > 1 else heads * d


def _refuse_rows(index, *args):
    """Raise for the first of args, (tensor, name, shape or None), that is not bf16 [tokens, heads, d]
    with dense tokens on this device."""
    for t, name, shape in args:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.device.type != "cuda" or t.get_device() != index:
            raise ValueError(f"{name} must be a CUDA tensor on the device of the call's other tensors")
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
        if t.dim() != 3 or (shape is not None and t.shape != shape):
            raise ValueError(f"{name} must be {'[tokens, heads, d]' if shape is None else list(shape)}, "
                             f"got {list(t.shape)}")
        if _apart(t, t.shape[1], t.shape[2]) is None:
            raise ValueError(f"the heads and components of a token of {name} must be dense")


def _norm_rope(q, k, q_weight, k_weight, eps, rotary_cos, rotary_sin, positions, rotary_interleaved,
               sections, sections_interleaved):
    """(device index, q's sizes and key heads, the strides of q and k, the arguments from q_weight to
    sections_interleaved as the library takes them)."""
    index = _device_index(q, "q") if not isinstance(q, torch.Tensor) else q.get_device()
    try:
        total, Hq, d = q.shape
        tokens, Hkv, dk = k.shape
        ok = (index >= 0 and tokens == total and dk == d and q.dtype is _BF16 and k.dtype is _BF16
              and k.get_device() == index)
        qs, ks = _apart(q, Hq, d), _apart(k, Hkv, d)
    except _WRONG:
        ok = False
    if not ok or qs is None or ks is None:
        _device_index(q, "q")
        _refuse_rows(index, (q, "q", None), (k, "k", None))
        raise ValueError("q and k must have the same tokens and components")
    w32 = 0
    qw = kw = None
    if q_weight is not None or k_weight is not None:
        try:
            dtype = (k_weight if q_weight is None else q_weight).dtype
            ok = dtype is _BF16 or dtype is _F32
            w32 = 1 if dtype is _F32 else 0
            if q_weight is not None:
                qw = q_weight.data_ptr()
                ok = (ok and q_weight.shape == (d,) and q_weight.is_contiguous()
                      and q_weight.get_device() == index)
            if k_weight is not None:
                kw = k_weight.data_ptr()
                ok = (ok and k_weight.shape == (d,) and k_weight.dtype is dtype
                      and k_weight.is_contiguous() and k_weight.get_device() == index)
        except _WRONG:
            ok = False
        if not ok:
            given = [(w, n) for w, n in ((q_weight, "q_weight"), (k_weight, "k_weight")) if w is not None]
            dtype = getattr(given[0][0], "dtype", None)
            if dtype not in (_F32, _BF16):
                raise TypeError("q_weight and k_weight must be torch.float32 or torch.bfloat16")
            for w, n in given:
                _step_tensor(w, n, dtype, (d,), index)
    cos, sin, rot_dim, rot_rows = _rotary(rotary_cos, rotary_sin, index)
    pos, axes, parts = None, 1, None
    if rot_dim:
        try:
            shape = positions.shape
            dims = len(shape)
            if (0 < dims < 3 and shape[-1] == total and positions.dtype is _I32
                    and positions.get_device() == index and positions.is_contiguous()):
                pos = positions.data_ptr()
                axes = shape[0] if dims == 2 else 1
        except _WRONG:
            pass
        if pos is None:
            if positions is None:
                raise ValueError("a rotation needs positions")
            _refuse("positions must be [T] or [axes, T], on the device of the call's other tensors",
                    (rotary_cos, "rotary_cos", _F32, 2),
                    (positions, "positions", _I32,
                     2 if isinstance(positions, torch.Tensor) and positions.dim() == 2 else 1))
        if sections is not None:
            if len(sections) != axes:
                raise ValueError("sections must have one entry per axis of positions")
            parts = (ctypes.c_int32 * axes)(*[_int32(n, "sections") for n in sections])
    return index, total, Hq, Hkv, d, qs, ks, (
        qw, kw, w32, float(eps), cos, sin, rot_dim, rot_rows, 1 if rotary_interleaved else 0, pos, axes,
        parts, 1 if sections_interleaved else 0)


def attn_qk_norm_rope(q, k, q_weight=None, k_weight=None, eps=1e-6, rotary_cos=None, rotary_sin=None,
                      positions=None, rotary_interleaved=False, sections=None,
                      sections_interleaved=False, q_out=None, k_out=None, stream=None):
    """RMS norm of every query and key per head, then the rotation, in one pass.

    q [T, Hq, d], k [T, Hkv, d] bf16, tokens dense but perhaps apart (parts of one projection's
    rows); weights [d] fp32 or bf16, None: no norm; rotary_cos / rotary_sin fp32
    [rows, rotary_dim / 2] or None; positions int32 [T] or, with several axes, [axes, T], and
    sections the planes of each axis (sections_interleaved: the axes take planes in turn).
    Returns (q_out, k_out), dense; q_out may be q and k_out k where those are dense.
    """
    lib = load()
    index, total, Hq, Hkv, d, qs, ks, how = _norm_rope(
        q, k, q_weight, k_weight, eps, rotary_cos, rotary_sin, positions, rotary_interleaved, sections,
        sections_interleaved)
    if q_out is not None:
        _step_tensor(q_out, "q_out", _BF16, q.shape, index)
    if k_out is not None:
        _step_tensor(k_out, "k_out", _BF16, k.shape, index)

    def body(s):
        device = q.device
        qo = torch.empty((total, Hq, d), dtype=_BF16, device=device) if q_out is None else q_out
        ko = torch.empty((total, Hkv, d), dtype=_BF16, device=device) if k_out is None else k_out
        rc = lib.attn_qk_norm_rope(q.data_ptr(), k.data_ptr(), qs, ks, *how, qo.data_ptr(), ko.data_ptr(),
                                   total, Hq, Hkv, d, s)
        if rc != 0:
            raise AttnError(rc, "attn_qk_norm_rope")
        return qo, ko

    return _on(index, stream, body)


def attn_qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight=None, k_weight=None, eps=1e-6,
                          rotary_cos=None, rotary_sin=None, positions=None,
                          rotary_interleaved=False, sections=None, sections_interleaved=False,
                          dq=None, dk=None, workspace=None, stream=None):
    """Backward pass of attn_qk_norm_rope: dq_out [T, Hq, d] and dk_out [T, Hkv, d] are the gradients
    of its outputs, the other arguments its own.

    Returns (dq, dk, dq_weight, dk_weight): bf16 like q and k, fp32 [d] (None without a weight).  dq
    and dk may be given, with tokens apart (parts of a projection's gradient).
    """
    lib = load()
    index, total, Hq, Hkv, d, qs, ks, how = _norm_rope(
        q, k, q_weight, k_weight, eps, rotary_cos, rotary_sin, positions, rotary_interleaved, sections,
        sections_interleaved)
    q_shape, k_shape = (total, Hq, d), (total, Hkv, d)
    dqs, dks = Hq * d, Hkv * d
    try:
        ok = (dq_out.shape == q_shape and dk_out.shape == k_shape and dq_out.dtype is _BF16
              and dk_out.dtype is _BF16 and dq_out.is_contiguous() and dk_out.is_contiguous()
              and dq_out.get_device() == dk_out.get_device() == index)
        if dq is not None:
            dqs = _apart(dq, Hq, d)
            ok = (ok and dq.shape == q_shape and dq.dtype is _BF16 and dq.get_device() == index
                  and dqs is not None)
        if dk is not None:
            dks = _apart(dk, Hkv, d)
            ok = (ok and dk.shape == k_shape and dk.dtype is _BF16 and dk.get_device() == index
                  and dks is not None)
    except _WRONG:
        ok = False
    if not ok:
        _step_tensor(dq_out, "dq_out", _BF16, q_shape, index)
        _step_tensor(dk_out, "dk_out", _BF16, k_shape, index)
        _refuse_rows(index, *[(t, n, torch.Size(shape)) for t, n, shape in (
            (dq, "dq", q_shape), (dk, "dk", k_shape)) if t is not None])
    nbytes = (lib.attn_qk_norm_rope_bwd_workspace_bytes(d)
              if q_weight is not None or k_weight is not None else 0)

    def body(s):
        device = q.device
        dqo = torch.empty(q_shape, dtype=_BF16, device=device) if dq is None else dq
        dko = torch.empty(k_shape, dtype=_BF16, device=device) if dk is None else dk
        dqw = None if q_weight is None else torch.empty(d, dtype=_F32, device=device)
        dkw = None if k_weight is None else torch.empty(d, dtype=_F32, device=device)
        ws = _kv8_workspace(nbytes, device, workspace)
        rc = lib.attn_qk_norm_rope_bwd(
            dq_out.data_ptr(), dk_out.data_ptr(), q.data_ptr(), k.data_ptr(), qs, ks, *how,
            dqo.data_ptr(), dko.data_ptr(), dqs, dks, _ptr(dqw), _ptr(dkw), total, Hq, Hkv, d, _ptr(ws),
            nbytes, s)
        if rc != 0:
            raise AttnError(rc, "attn_qk_norm_rope_bwd")
        return dqo, dko, dqw, dkw

    return _on(index, stream, body)


def attn_kvcache_append_norm_rope(q, k, v, k_cache, v_cache, slot_map, q_weight=None, k_weight=None,
                                  eps=1e-6, rotary_cos=None, rotary_sin=None, positions=None,
                                  rotary_interleaved=False, sections=None,
                                  sections_interleaved=False, q_out=None, stream=None):
    """attn_qk_norm_rope for serving: the keys and the values [T, Hkv, d] go to slot_map[t] (int32;
    negative: nowhere) of the bf16 paged cache [num_pages, page_size, Hkv, d], in place.

    Returns q_out [T, Hq, d].
    """
    lib = load()
    index, total, Hq, Hkv, d, qs, ks, how = _norm_rope(
        q, k, q_weight, k_weight, eps, rotary_cos, rotary_sin, positions, rotary_interleaved, sections,
        sections_interleaved)
    try:
        cache = k_cache.shape
        num_pages, page_size, heads, dim = cache
        vs = _apart(v, Hkv, d)
        ok = (heads == Hkv and dim == d and v_cache.shape == cache and v.shape == k.shape
              and vs is not None and slot_map.shape == (total,) and v.dtype is _BF16
              and k_cache.dtype is _BF16 and v_cache.dtype is _BF16 and slot_map.dtype is _I32
              and k_cache.is_contiguous() and v_cache.is_contiguous() and slot_map.is_contiguous()
              and v.get_device() == k_cache.get_device() == v_cache.get_device()
              == slot_map.get_device() == index)
    except _WRONG:
        ok = False
    if not ok:
        _refuse_rows(index, (v, "v", k.shape))
        _step_tensor(k_cache, "k_cache", _BF16, (None, None, Hkv, d), index)
        _step_tensor(v_cache, "v_cache", _BF16, k_cache.shape, index)
        _step_tensor(slot_map, "slot_map", _I32, (total,), index)
    if q_out is not None:
        _step_tensor(q_out, "q_out", _BF16, q.shape, index)

    def body(s):
        qo = torch.empty((total, Hq, d), dtype=_BF16, device=q.device) if q_out is None else q_out
        rc = lib.attn_kvcache_append_norm_rope(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), qs, ks, vs, *how, qo.data_ptr(),
            k_cache.data_ptr(), v_cache.data_ptr(), slot_map.data_ptr(), total, Hq, Hkv, d, page_size,
            num_pages, s)
        if rc != 0:
            raise AttnError(rc, "attn_kvcache_append_norm_rope")
        return qo

    return _on(index, stream, body)


def attn_decode_kvcache_shared_workspace_bytes(batch, num_groups, total_q, nheads_q, nheads_kv,
                                               head_dim) -> int:
    return int(load().attn_decode_kvcache_shared_workspace_bytes(batch, num_groups, total_q, nheads_q,
                                                                 nheads_kv, head_dim))


def attn_decode_kvcache_shared(q, k_cache, v_cache, cache_seqlens, block_table, group_starts=None,
                               prefix_lens=None, cu_seqlens_q=None, max_seqlen_q=1,
                               softmax_scale=None, out=None, lse=None, workspace=None, stream=None):
    """Decode over the bf16 paged cache where groups of sequences share prefixes, each read once.

    q [total_q, Hq, d]: one token per sequence or, with cu_seqlens_q [batch + 1], up to max_seqlen_q
    of them, the last of the sequence's cache_seqlens[b] keys.  Sequences group_starts[i] ..
    group_starts[i + 1] - 1 begin with the same prefix_lens[i] keys (both None: none share).
    Returns (out like q, lse fp32 [batch, Hq], or [Hq, total_q] with cu_seqlens_q).
    """
    lib = load()
    groups, starts, prefix, cu = 0, None, None, None
    try:
        total_q, Hq, d = q.shape
        cache = k_cache.shape
        num_pages, page_size, Hkv, dk = cache
        batch, max_pages = block_table.shape
        index = q.get_device()
        ok = (index >= 0 and dk == d and v_cache.shape == cache and cache_seqlens.shape == (batch,)
              and q.dtype is _BF16 and k_cache.dtype is _BF16 and v_cache.dtype is _BF16
              and cache_seqlens.dtype is _I32 and block_table.dtype is _I32 and q.is_contiguous()
              and k_cache.is_contiguous() and v_cache.is_contiguous()
              and cache_seqlens.is_contiguous() and block_table.is_contiguous()
              and k_cache.get_device() == v_cache.get_device() == cache_seqlens.get_device()
              == block_table.get_device() == index)
        if ok and prefix_lens is not None:
            groups, = prefix_lens.shape
            ok = (group_starts.shape == (groups + 1,) and group_starts.dtype is _I32
                  and prefix_lens.dtype is _I32 and group_starts.is_contiguous()
                  and prefix_lens.is_contiguous()
                  and group_starts.get_device() == prefix_lens.get_device() == index)
            starts, prefix = group_starts.data_ptr(), prefix_lens.data_ptr()
        elif group_starts is not None:
            ok = False
        if ok and cu_seqlens_q is not None:
            ok = (cu_seqlens_q.shape == (batch + 1,) and cu_seqlens_q.dtype is _I32
                  and cu_seqlens_q.is_contiguous() and cu_seqlens_q.get_device() == index)
            cu = cu_seqlens_q.data_ptr()
        elif total_q != batch:
            ok = False
    except _WRONG:
        ok = False
    if not ok:
        more = [(t, n, _I32, 1) for t, n in ((group_starts, "group_starts"), (prefix_lens, "prefix_lens"),
                                             (cu_seqlens_q, "cu_seqlens_q")) if t is not None]
        _refuse("q must be [total_q, Hq, d] (one token per sequence, or cu_seqlens_q [batch + 1]), k_cache "
                "and v_cache [num_pages, page_size, Hkv, d], cache_seqlens [batch], block_table "
                "[batch, max_pages], group_starts [groups + 1] and prefix_lens [groups], both or none",
                (q, "q", _BF16, 3), (k_cache, "k_cache", _BF16, 4), (v_cache, "v_cache", _BF16, 4),
                (cache_seqlens, "cache_seqlens", _I32, 1), (block_table, "block_table", _I32, 2), *more)
    max_q = 1 if cu is None else _int32(max_seqlen_q, "max_seqlen_q")
    shape = (batch, Hq) if cu is None else (Hq, total_q)
    if out is not None:
        _output(out, "out", _BF16, (total_q, Hq, d), index)
    if lse is not None:
        _output(lse, "lse", _F32, shape, index)
    scale = d ** -0.5 if softmax_scale is None else float(softmax_scale)
    nbytes = lib.attn_decode_kvcache_shared_workspace_bytes(batch, groups, total_q, Hq, Hkv, d)

    def body(s):
        device = q.device
        o = torch.empty_like(q) if out is None else out
        l = torch.empty(shape, dtype=_F32, device=device) if lse is None else lse
        ws = _kv8_workspace(nbytes, device, workspace)
        rc = lib.attn_decode_kvcache_shared(
            q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), cache_seqlens.data_ptr(),
            block_table.data_ptr(), starts, prefix, cu, page_size, o.data_ptr(), l.data_ptr(), batch,
            groups, total_q, max_q, Hq, Hkv, d, max_pages, num_pages, scale, _ptr(ws), nbytes, s)
        if rc != 0:
            raise AttnError(rc, "attn_decode_kvcache_shared")
        return o, l

    return _on(index, stream, body)
