"""Exact IO-aware attention on GB300 (sm_103a): a thin ctypes binding over libfa.so.

Every entry point has the name and argument order of the C function declared
in ``include/fa.h``; this module only turns torch tensors into device pointers
and sizes, passes the current CUDA stream and raises ``FaError`` on a non-zero
status.  All arithmetic happens in the library's CUDA kernels.  PyTorch serves
as the allocator and stream provider only.

There is no fallback: if ``libfa.so`` has not been built, or no GPU is present,
the calls raise.
"""
import ctypes
import math
import os

__all__ = [
    "FaError", "FA_F32", "FA_BF16", "FA_E4M3", "lib", "fa_fwd", "fa_fwd_fp8", "fa_fwd_gqa",
    "fa_fwd_fp8_per_head", "fa_fwd_fp8_per_block", "fa_bwd",
    "fa_bwd_workspace_size", "fa_bwd_noalloc", "fa_last_device_error", "fa_set_wait_timeout_ns",
    "fa_selftest_wait_timeout", "fa_status_string", "attention_forward", "attention_backward",
    "fa_qk_norm_rope", "fa_qk_norm_rope_bwd", "fa_qk_norm_rope_bwd_workspace_size",
    "fa_fwd_window", "fa_bwd_window", "fa_bwd_window_workspace_size", "fa_kv4_append", "fa_kv4_read", "fa_decode_kv4", "fa_decode_kv4_workspace_size",
    "rope_frequencies", "kv4_cache",
]

FA_F32, FA_BF16, FA_E4M3 = 0, 1, 2
FA_OK = 0
FA_ERR_DEVICE_TIMEOUT = 4
FA_ERR_DEVICE_INDEX = 5

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libfa.so")
_LIB = None


class FaError(RuntimeError):
    def __init__(self, status, what=""):
        self.status = int(status)
        super().__init__(f"{what}: {fa_status_string(self.status)} ({self.status})")


def lib():
    """Load libfa.so (built by ``__graft_entry__.build()``); raises if absent."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it first "
                               "(python -c 'import __graft_entry__ as g; g.build()')")
        L = ctypes.CDLL(LIB_PATH)
        vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        L.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, i, vp]
        L.fa_fwd.restype = i
        L.fa_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, f, f, f, i, i, i, i, f, i, vp]
        L.fa_fwd_fp8.restype = i
        L.fa_fwd_gqa.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp]
        L.fa_fwd_gqa.restype = i
        L.fa_fwd_fp8_per_head.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
        L.fa_fwd_fp8_per_head.restype = i
        L.fa_fwd_fp8_per_block.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
        L.fa_fwd_fp8_per_block.restype = i
        ll = ctypes.c_longlong
        L.fa_fwd_kv_shard.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, i, ll, ll, i, vp]
        L.fa_fwd_kv_shard.restype = i
        L.fa_lse_merge.argtypes = [vp, vp, i, vp, vp, i, i, i, i, i, vp]
        L.fa_lse_merge.restype = i
        L.fa_bwd_workspace_size.argtypes = [i, i, i, i]
        L.fa_bwd_workspace_size.restype = sz
        L.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, i, i, i, i, f, i, i, vp]
        L.fa_bwd_gqa.restype = i
        L.fa_bwd_gqa.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, i, i, i, i, i, f, i, i,
                                 vp]
        L.fa_bwd.restype = i
        L.fa_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, i, vp]
        L.fa_bwd_noalloc.restype = i
        L.fa_qk_norm_rope.argtypes = [vp] * 8 + [i] * 7 + [f, i, vp]
        L.fa_qk_norm_rope.restype = i
        L.fa_qk_norm_rope_bwd.argtypes = [vp] * 12 + [sz] + [i] * 7 + [f, i, vp]
        L.fa_qk_norm_rope_bwd.restype = i
        L.fa_qk_norm_rope_bwd_workspace_size.argtypes = [i] * 5
        L.fa_qk_norm_rope_bwd_workspace_size.restype = sz
        L.fa_fwd_window.argtypes = [vp] * 5 + [i] * 5 + [f, i, i, i, vp]
        L.fa_fwd_window.restype = i
        L.fa_bwd_window.argtypes = [vp] * 10 + [sz] + [i] * 5 + [f, i, i, i, vp]
        L.fa_bwd_window.restype = i
        L.fa_bwd_window_workspace_size.argtypes = [i] * 7
        L.fa_bwd_window_workspace_size.restype = sz
        L.fa_kv4_append.argtypes = [vp] * 9 + [i] * 7 + [vp]
        L.fa_kv4_append.restype = i
        L.fa_kv4_read.argtypes = [vp] * 8 + [i] * 7 + [vp]
        L.fa_kv4_read.restype = i
        L.fa_decode_kv4.argtypes = [vp] * 10 + [sz] + [i] * 8 + [f, i, i, vp]
        L.fa_decode_kv4.restype = i
        L.fa_decode_kv4_workspace_size.argtypes = [i] * 5
        L.fa_decode_kv4_workspace_size.restype = sz
        L.fa_last_device_error.argtypes = [vp]
        L.fa_last_device_error.restype = i
        L.fa_set_wait_timeout_ns.argtypes = [ctypes.c_uint64]
        L.fa_set_wait_timeout_ns.restype = None
        L.fa_selftest_wait_timeout.argtypes = [vp]
        L.fa_selftest_wait_timeout.restype = i
        L.fa_status_string.argtypes = [i]
        L.fa_status_string.restype = ctypes.c_char_p
        _LIB = L
    return _LIB


def fa_status_string(status):
    try:
        return lib().fa_status_string(int(status)).decode()
    except RuntimeError:
        return f"status {status}"


def _stream(stream):
    import torch
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _shape(q):
    if q.dim() != 4 or not q.is_contiguous():
        raise ValueError("tensors must be contiguous [B, H, N, d]")
    return tuple(int(x) for x in q.shape)


def _check(status, what):
    if status != FA_OK:
        raise FaError(status, what)


def fa_fwd(q, k, v, o, lse, scale, causal, dtype, stream=None):
    """O (and lse, may be None) <- attention(q, k, v); tensors [B, H, N, d] on the GPU."""
    B, H, N, d = _shape(q)
    _check(lib().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d, float(scale),
                        int(bool(causal)), int(dtype), _stream(stream)), "fa_fwd")


def fa_fwd_fp8(q8, k8, v8, o, lse, q_descale, k_descale, v_descale, scale, causal, stream=None):
    """FP8 forward: q8/k8/v8 uint8 E4M3 codes [B, H, N, d]; o bfloat16."""
    B, H, N, d = _shape(q8)
    _check(lib().fa_fwd_fp8(_ptr(q8), _ptr(k8), _ptr(v8), _ptr(o), _ptr(lse), float(q_descale),
                            float(k_descale), float(v_descale), B, H, N, d, float(scale),
                            int(bool(causal)), _stream(stream)), "fa_fwd_fp8")


def fa_fwd_gqa(q, k, v, o, lse, scale, causal, dtype, stream=None):
    """Grouped-query forward: q, o [B, H, N, d]; k, v [B, H_kv, N, d] with H % H_kv == 0."""
    B, H, N, d = _shape(q)
    H_kv = _shape(k)[1]
    _check(lib().fa_fwd_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, H_kv, N, d,
                            float(scale), int(bool(causal)), int(dtype), _stream(stream)),
           "fa_fwd_gqa")


def fa_fwd_fp8_per_head(q8, k8, v8, o, lse, q_descale, k_descale, v_descale, scale, causal,
                        stream=None):
    """FP8 forward with per-(b, h) descales: float32 device tensors of B*H elements."""
    B, H, N, d = _shape(q8)
    for t in (q_descale, k_descale, v_descale):
        if t.numel() != B * H or t.dtype.itemsize != 4 or not t.is_contiguous():
            raise ValueError("per-head descales: contiguous float32, B*H elements")
    _check(lib().fa_fwd_fp8_per_head(_ptr(q8), _ptr(k8), _ptr(v8), _ptr(o), _ptr(lse),
                                     _ptr(q_descale), _ptr(k_descale), _ptr(v_descale), B, H, N,
                                     d, float(scale), int(bool(causal)), _stream(stream)),
           "fa_fwd_fp8_per_head")


def fa_fwd_fp8_per_block(q8, k8, v8, o, lse, q_descale, k_descale, v_descale, scale, causal,
                         stream=None):
    """FP8 forward with one descale per 128-row block of each head: float32 device
    tensors of B*H*ceil(N/128) elements ([B][H][ceil(N/128)])."""
    B, H, N, d = _shape(q8)
    nb = (N + 127) // 128
    for t in (q_descale, k_descale, v_descale):
        if t.numel() != B * H * nb or t.dtype.itemsize != 4 or not t.is_contiguous():
            raise ValueError("per-block descales: contiguous float32, B*H*ceil(N/128) elements")
    _check(lib().fa_fwd_fp8_per_block(_ptr(q8), _ptr(k8), _ptr(v8), _ptr(o), _ptr(lse),
                                      _ptr(q_descale), _ptr(k_descale), _ptr(v_descale), B, H, N,
                                      d, float(scale), int(bool(causal)), _stream(stream)),
           "fa_fwd_fp8_per_block")


def fa_fwd_kv_shard(q, k, v, o_part, lse_part, scale, causal, q_offset, kv_offset,
                    dtype=FA_BF16, stream=None):
    """Forward of q [B, H, N_q, d] over one key shard k, v [B, H_kv, N_kv, d] at the
    given global offsets; o_part float32 [B, H, N_q, d], lse_part [B, H, N_q]."""
    B, H, N_q, d = _shape(q)
    H_kv, N_kv = _shape(k)[1], _shape(k)[2]
    _check(lib().fa_fwd_kv_shard(_ptr(q), _ptr(k), _ptr(v), _ptr(o_part), _ptr(lse_part), B, H,
                                 H_kv, N_q, N_kv, d, float(scale), int(bool(causal)),
                                 int(q_offset), int(kv_offset), int(dtype), _stream(stream)),
           "fa_fwd_kv_shard")


def fa_lse_merge(o_parts, lse_parts, o, lse, dtype, stream=None):
    """Merge stacked shard outputs o_parts [S, B, H, N, d] (float32), lse_parts
    [S, B, H, N] into o [B, H, N, d] (bf16 or float32 per dtype) and lse (or None)."""
    S, B, H, N, d = (int(x) for x in o_parts.shape)
    if tuple(lse_parts.shape) != (S, B, H, N) or tuple(o.shape) != (B, H, N, d):
        raise ValueError("fa_lse_merge: shapes do not match")
    _check(lib().fa_lse_merge(_ptr(o_parts), _ptr(lse_parts), S, _ptr(o), _ptr(lse), B, H, N, d,
                              int(dtype), _stream(stream)), "fa_lse_merge")


def fa_bwd_workspace_size(B, H, N, d):
    return int(lib().fa_bwd_workspace_size(int(B), int(H), int(N), int(d)))


def fa_bwd(q, k, v, o, lse, do, dq, dk, dv, workspace, scale, causal, dtype, stream=None):
    """dq, dk, dv <- backward; workspace: a device buffer of fa_bwd_workspace_size bytes."""
    B, H, N, d = _shape(q)
    nbytes = workspace.numel() * workspace.element_size()
    _check(lib().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq),
                        _ptr(dk), _ptr(dv), _ptr(workspace), nbytes, B, H, N, d, float(scale),
                        int(bool(causal)), int(dtype), _stream(stream)), "fa_bwd")


def fa_bwd_gqa(q, k, v, o, lse, do, dq, dk, dv, workspace, scale, causal, dtype, stream=None):
    """Grouped-query backward: q, o, do, dq [B, H, N, d]; k, v, dk, dv [B, H_kv, N, d]."""
    B, H, N, d = _shape(q)
    H_kv = _shape(k)[1]
    nbytes = workspace.numel() * workspace.element_size()
    _check(lib().fa_bwd_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq),
                            _ptr(dk), _ptr(dv), _ptr(workspace), nbytes, B, H, H_kv, N, d,
                            float(scale), int(bool(causal)), int(dtype), _stream(stream)),
           "fa_bwd_gqa")


def fa_bwd_noalloc(q, k, v, o, lse, do, dq, dk, dv, scale, causal, dtype, stream=None):
    """fa_bwd with the library's built-in scratch (no workspace, no allocation).
    For callers that cannot allocate device memory at call time; calls that
    overlap on the GPU race on the shared scratch."""
    B, H, N, d = _shape(q)
    _check(lib().fa_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do),
                                _ptr(dq), _ptr(dk), _ptr(dv), B, H, N, d, float(scale),
                                int(bool(causal)), int(dtype), _stream(stream)), "fa_bwd_noalloc")


# ---------------------------------------------------------------- the layer around the call
def _dense(what, dtype, shape, t):
    """Device pointer of a contiguous tensor of this dtype and shape on the current device."""
    import torch
    if t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{what}: contiguous {dtype} {list(shape)} expected, got {t.dtype} "
                         f"{list(t.shape)}")
    if not t.is_cuda or t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{what}: a tensor on the current CUDA device expected, got {t.device}")
    return t.data_ptr()


def _maybe(what, dtype, shape, t):
    return None if t is None else _dense(what, dtype, shape, t)


def _float_code(t):
    import torch
    if t.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"float32 or bfloat16 expected, got {t.dtype}")
    return FA_F32 if t.dtype == torch.float32 else FA_BF16


def _norm_rope_head(qkv, q_like, k_like, q_weight, k_weight, positions, inv_freq):
    """What fa_qk_norm_rope and its gradient have in common: pointers and sizes."""
    import torch
    code = _float_code(qkv)
    B, H, N, d = _shape(q_like)
    H_kv = _shape(k_like)[1]
    rot = 0
    if inv_freq is not None:
        if inv_freq.dtype != torch.float64 or inv_freq.is_cuda or not inv_freq.is_contiguous():
            raise ValueError("inv_freq: a contiguous float64 tensor on the host (rope_frequencies)")
        rot = 2 * inv_freq.numel()
    head = (_dense("qkv", qkv.dtype, (B, N, H + 2 * H_kv, d), qkv),
            _maybe("q_weight", torch.float32, (d,), q_weight),
            _maybe("k_weight", torch.float32, (d,), k_weight),
            _maybe("positions", torch.int32, (B, N), positions),
            inv_freq.data_ptr() if rot else None)
    return code, (B, H, H_kv, N, d), rot, head


def rope_frequencies(rot, base=10000.0):
    """The rotation's rot / 2 frequencies base^(-2 p / rot), radians per position (float64, host)."""
    import torch
    return float(base) ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)


def fa_qk_norm_rope(qkv, q_weight, k_weight, positions, inv_freq, q, k, v, eps, interleaved=False,
                    stream=None):
    """q [B, H, N, d], k, v [B, H_kv, N, d] <- norm and rotation of qkv [B, N, H + 2 H_kv, d].
    q_weight, k_weight (float32 [d]), positions (int32 [B, N]) and inv_freq (float64 host tensor
    of rot / 2) may be None: ones, the index in the sequence, no rotation."""
    code, (B, H, H_kv, N, d), rot, head = _norm_rope_head(qkv, q, k, q_weight, k_weight, positions,
                                                          inv_freq)
    t = qkv.dtype
    _check(lib().fa_qk_norm_rope(*head, _dense("q", t, (B, H, N, d), q), _dense("k", t, (B, H_kv, N, d), k),
                                 _dense("v", t, (B, H_kv, N, d), v), B, H, H_kv, N, d, rot,
                                 int(bool(interleaved)), float(eps), code, _stream(stream)),
           "fa_qk_norm_rope")


def fa_qk_norm_rope_bwd_workspace_size(B, H, H_kv, N, d):
    return int(lib().fa_qk_norm_rope_bwd_workspace_size(int(B), int(H), int(H_kv), int(N), int(d)))


def fa_qk_norm_rope_bwd(qkv, q_weight, k_weight, positions, inv_freq, dq, dk, dv, dqkv, dq_weight,
                        dk_weight, workspace, eps, interleaved=False, stream=None):
    """dqkv and (float32 [d], or None) dq_weight, dk_weight <- gradient of fa_qk_norm_rope."""
    import torch
    code, (B, H, H_kv, N, d), rot, head = _norm_rope_head(qkv, dq, dk, q_weight, k_weight, positions,
                                                          inv_freq)
    t = qkv.dtype
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().fa_qk_norm_rope_bwd(
        *head, _dense("dq", t, (B, H, N, d), dq), _dense("dk", t, (B, H_kv, N, d), dk),
        _dense("dv", t, (B, H_kv, N, d), dv), _dense("dqkv", t, (B, N, H + 2 * H_kv, d), dqkv),
        _maybe("dq_weight", torch.float32, (d,), dq_weight),
        _maybe("dk_weight", torch.float32, (d,), dk_weight), _ptr(workspace), ws_bytes, B, H, H_kv, N, d,
        rot, int(bool(interleaved)), float(eps), code, _stream(stream)), "fa_qk_norm_rope_bwd")


def fa_fwd_window(q, k, v, o, lse, scale, window, n_sink, dtype=FA_BF16, stream=None):
    """Forward under a causal window of `window` keys and the first n_sink keys: q, o
    [B, H, N, d], k, v [B, H_kv, N, d] bfloat16; lse [B, H, N] or None."""
    import torch
    B, H, N, d = _shape(q)
    H_kv = _shape(k)[1]
    t = torch.bfloat16
    _check(lib().fa_fwd_window(_dense("q", t, (B, H, N, d), q), _dense("k", t, (B, H_kv, N, d), k),
                               _dense("v", t, (B, H_kv, N, d), v), _dense("o", t, (B, H, N, d), o),
                               _maybe("lse", torch.float32, (B, H, N), lse), B, H, H_kv, N, d,
                               float(scale), int(window), int(n_sink), int(dtype), _stream(stream)),
           "fa_fwd_window")


def fa_bwd_window_workspace_size(B, H, H_kv, N, d, window, n_sink):
    return int(lib().fa_bwd_window_workspace_size(int(B), int(H), int(H_kv), int(N), int(d), int(window),
                                                  int(n_sink)))


def fa_bwd_window(q, k, v, o, lse, do, dq, dk, dv, workspace, scale, window, n_sink, dtype=FA_BF16,
                  stream=None):
    """dq, dk, dv <- backward of fa_fwd_window, from its o and lse."""
    import torch
    B, H, N, d = _shape(q)
    H_kv = _shape(k)[1]
    t, rows, kv_rows = torch.bfloat16, (B, H, N, d), (B, H_kv, N, d)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().fa_bwd_window(_dense("q", t, rows, q), _dense("k", t, kv_rows, k),
                               _dense("v", t, kv_rows, v), _dense("o", t, rows, o),
                               _dense("lse", torch.float32, (B, H, N), lse), _dense("do", t, rows, do),
                               _dense("dq", t, rows, dq), _dense("dk", t, kv_rows, dk),
                               _dense("dv", t, kv_rows, dv), workspace.data_ptr(), ws_bytes, B, H, H_kv,
                               N, d, float(scale), int(window), int(n_sink), int(dtype),
                               _stream(stream)), "fa_bwd_window")


def kv4_cache(n_pages, H_kv, page, d, device="cuda"):
    """Zeroed arrays of a 4-bit cache: k_codes, k_scales, v_codes, v_scales."""
    import torch
    codes = [torch.zeros((n_pages, H_kv, page, d // 2), dtype=torch.uint8, device=device) for _ in "kv"]
    scales = [torch.zeros((n_pages, H_kv, page, d // 32), dtype=torch.bfloat16, device=device) for _ in "kv"]
    return codes[0], scales[0], codes[1], scales[1]


def _cache_args(k_codes, k_scales, v_codes, v_scales, block_table, B, d):
    import torch
    if k_codes.dim() != 4 or block_table.dim() != 2:
        raise ValueError("4-bit cache: codes [n_pages, H_kv, page, d / 2], block_table [B, max_blocks]")
    n_pages, H_kv, page = (int(x) for x in k_codes.shape[:3])
    codes, scales = (n_pages, H_kv, page, d // 2), (n_pages, H_kv, page, d // 32)
    max_blocks = int(block_table.shape[1])
    return ((_dense("k_codes", torch.uint8, codes, k_codes),
             _dense("k_scales", torch.bfloat16, scales, k_scales),
             _dense("v_codes", torch.uint8, codes, v_codes),
             _dense("v_scales", torch.bfloat16, scales, v_scales),
             _dense("block_table", torch.int32, (B, max_blocks), block_table)), H_kv,
            (page, n_pages, max_blocks))


def fa_kv4_append(k, v, k_codes, k_scales, v_codes, v_scales, block_table, first, count=None,
                  stream=None):
    """Store k, v (bfloat16 [B, H_kv, N, d]) in the cache as tokens first[b] + 0 .. count[b] - 1
    (int32 [B]; count None: N)."""
    import torch
    B, H_kv, N, d = _shape(k)
    cache, heads, sizes = _cache_args(k_codes, k_scales, v_codes, v_scales, block_table, B, d)
    rows = (B, heads, N, d)
    _check(lib().fa_kv4_append(_dense("k", torch.bfloat16, rows, k), _dense("v", torch.bfloat16, rows, v),
                               *cache, _dense("first", torch.int32, (B,), first),
                               _maybe("count", torch.int32, (B,), count), B, H_kv, N, d, *sizes,
                               _stream(stream)), "fa_kv4_append")


def fa_kv4_read(k_codes, k_scales, v_codes, v_scales, block_table, lengths, k, v, stream=None):
    """k, v (bfloat16 [B, H_kv, N, d]) <- the cache's first N tokens of every request; rows from
    lengths[b] (int32 [B]) on are zeros."""
    import torch
    B, H_kv, N, d = _shape(k)
    cache, heads, sizes = _cache_args(k_codes, k_scales, v_codes, v_scales, block_table, B, d)
    rows = (B, heads, N, d)
    _check(lib().fa_kv4_read(*cache, _dense("lengths", torch.int32, (B,), lengths),
                             _dense("k", torch.bfloat16, rows, k), _dense("v", torch.bfloat16, rows, v),
                             B, H_kv, N, d, *sizes, _stream(stream)), "fa_kv4_read")


def fa_decode_kv4_workspace_size(B, H, H_kv, N_q, d):
    return int(lib().fa_decode_kv4_workspace_size(int(B), int(H), int(H_kv), int(N_q), int(d)))


def fa_decode_kv4(q, k_codes, k_scales, v_codes, v_scales, block_table, lengths, o, lse, workspace,
                  scale, window=0, n_sink=0, stream=None):
    """o (and lse, may be None) <- attention of the newest N_q tokens of every request, q
    [B, H, N_q, d], over the 4-bit cache; lengths int32 [B]; window 0: all earlier tokens."""
    import torch
    B, H, N_q, d = _shape(q)
    cache, H_kv, sizes = _cache_args(k_codes, k_scales, v_codes, v_scales, block_table, B, d)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().fa_decode_kv4(_dense("q", torch.bfloat16, (B, H, N_q, d), q), *cache,
                               _dense("lengths", torch.int32, (B,), lengths),
                               _dense("o", torch.bfloat16, (B, H, N_q, d), o),
                               _maybe("lse", torch.float32, (B, H, N_q), lse), workspace.data_ptr(),
                               ws_bytes, B, H, H_kv, N_q, d, *sizes, float(scale), int(window),
                               int(n_sink), _stream(stream)), "fa_decode_kv4")


def fa_last_device_error(stream=None):
    """Synchronise the stream and return (and clear) the device status word."""
    return int(lib().fa_last_device_error(_stream(stream)))


def fa_set_wait_timeout_ns(ns):
    lib().fa_set_wait_timeout_ns(int(ns))


def fa_selftest_wait_timeout(stream=None):
    _check(lib().fa_selftest_wait_timeout(_stream(stream)), "fa_selftest_wait_timeout")


# ---------------------------------------------------------------- conveniences
def attention_forward(q, k, v, scale=None, causal=False, stream=None):
    """Allocate O and lse with torch and run fa_fwd; q, k, v fp32 or bf16."""
    import torch
    dtype = {torch.float32: FA_F32, torch.bfloat16: FA_BF16}[q.dtype]
    B, H, N, d = _shape(q)
    o = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    # k, v with fewer heads than q: grouped-query attention
    fn = fa_fwd if _shape(k)[1] == H else fa_fwd_gqa
    fn(q, k, v, o, lse, 1.0 / math.sqrt(d) if scale is None else scale, causal, dtype, stream)
    return o, lse


def attention_backward(q, k, v, o, lse, do, scale=None, causal=False, stream=None):
    import torch
    B, H, N, d = _shape(q)
    ws = torch.empty(fa_bwd_workspace_size(B, H, N, d), dtype=torch.uint8, device=q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    # k, v with fewer heads than q: grouped-query attention
    fn = fa_bwd if _shape(k)[1] == H else fa_bwd_gqa
    fn(q, k, v, o, lse, do, dq, dk, dv, ws, 1.0 / math.sqrt(d) if scale is None else scale,
       causal, FA_BF16, stream)
    return dq, dk, dv
