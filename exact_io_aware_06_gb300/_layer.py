"""The layer's work around the attention call: norm and rotation of Q and K, windowed
attention, and attention over a 4-bit cache.

As the rest of the package, argument marshalling over ``include/fa.h``: the names and argument
order of the C functions.  Tensors are checked (type, shape, contiguous, on the current CUDA
device; ValueError) because a wrong one would be read out of bounds.  A call costs several
microseconds of host time, as much as the smallest kernels here, so the checks are few and plain.
"""
import torch

from . import FA_BF16, FA_F32, _check, lib

_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
_current_device = torch.cuda.current_device
# the current stream's handle without the Stream object around it (2.9 us of a 13 us call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _dense(what, t, dtype, shape, device):
    """Device pointer of a contiguous tensor of this dtype and shape on this device."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != device:
        raise ValueError(f"{what}: contiguous {dtype} {list(shape)} on the current CUDA device ({device}) "
                         f"expected, got {t.dtype} {list(t.shape)} on {t.device}, strides {t.stride()}")
    return t.data_ptr()


def _sizes(what, t):
    if t.dim() != 4:
        raise ValueError(f"{what}: four dimensions expected, got {list(t.shape)}")
    return t.shape


def _int(x):
    """x as a C int, those beyond one as the nearest: a window or a number of sinks that covers
    everything still does, and sizes are refused (ctypes would drop the upper bits without a word)."""
    return x if -0x80000000 <= x <= 0x7FFFFFFF else 0x7FFFFFFF if x > 0 else -0x80000000


def _handle(stream, device):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream if _raw_stream is None else _raw_stream(device)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _space(workspace, device):
    """Pointer and bytes of a workspace tensor of any type."""
    if not workspace.is_contiguous() or workspace.get_device() != device:
        raise ValueError(f"workspace: contiguous, on the current CUDA device ({device})")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


# ---------------------------------------------------------------- norm and rotation
def rope_frequencies(rot, base=10000.0):
    """The rotation's rot / 2 frequencies base^(-2 p / rot), radians per position (float64, host)."""
    return float(base) ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)


def _norm_rope(qkv, q_weight, k_weight, positions, inv_freq, q, k, v, device):
    """Pointers of qkv, weights, positions, frequencies, q, k, v; B, H, H_kv, N, d, rot; dtype code."""
    t = qkv.dtype
    if t is not _BF16 and t is not _F32:
        raise ValueError(f"qkv: float32 or bfloat16 expected, got {t}")
    B, H, N, d = _sizes("q", q)
    H_kv = _sizes("k", k)[1]
    rot = 0
    if inv_freq is not None:
        if inv_freq.dtype is not torch.float64 or inv_freq.is_cuda or not inv_freq.is_contiguous():
            raise ValueError("inv_freq: a contiguous float64 tensor on the host (rope_frequencies)")
        rot = 2 * inv_freq.numel()
    kv = (B, H_kv, N, d)
    return ((_dense("qkv", qkv, t, (B, N, H + 2 * H_kv, d), device),
             None if q_weight is None else _dense("q_weight", q_weight, _F32, (d,), device),
             None if k_weight is None else _dense("k_weight", k_weight, _F32, (d,), device),
             None if positions is None else _dense("positions", positions, _I32, (B, N), device),
             inv_freq.data_ptr() if rot else None, _dense("q", q, t, (B, H, N, d), device),
             _dense("k", k, t, kv, device), _dense("v", v, t, kv, device)),
            (B, H, H_kv, N, d, rot), FA_BF16 if t is _BF16 else FA_F32)


def fa_qk_norm_rope(qkv, q_weight, k_weight, positions, inv_freq, q, k, v, eps, interleaved=False,
                    stream=None):
    """q [B, H, N, d], k, v [B, H_kv, N, d] <- norm and rotation of qkv [B, N, H + 2 H_kv, d].
    q_weight, k_weight (float32 [d]), positions (int32 [B, N]) and inv_freq (float64 host tensor
    of rot / 2) may be None: ones, the index in the sequence, no rotation."""
    device = _current_device()
    pointers, sizes, code = _norm_rope(qkv, q_weight, k_weight, positions, inv_freq, q, k, v, device)
    _check(lib().fa_qk_norm_rope(*pointers, *sizes, bool(interleaved), eps, code, _handle(stream, device)),
           "fa_qk_norm_rope")


def fa_qk_norm_rope_bwd_workspace_size(B, H, H_kv, N, d):
    return int(lib().fa_qk_norm_rope_bwd_workspace_size(*map(_int, (B, H, H_kv, N, d))))


def fa_qk_norm_rope_bwd(qkv, q_weight, k_weight, positions, inv_freq, dq, dk, dv, dqkv, dq_weight,
                        dk_weight, workspace, eps, interleaved=False, stream=None):
    """dqkv and (float32 [d], or None) dq_weight, dk_weight <- gradient of fa_qk_norm_rope.
    workspace may be None if neither weight gradient is wanted."""
    device = _current_device()
    pointers, sizes, code = _norm_rope(qkv, q_weight, k_weight, positions, inv_freq, dq, dk, dv, device)
    d = sizes[4]
    space, nbytes = (None, 0) if workspace is None else _space(workspace, device)
    _check(lib().fa_qk_norm_rope_bwd(
        *pointers, _dense("dqkv", dqkv, qkv.dtype, qkv.shape, device),
        None if dq_weight is None else _dense("dq_weight", dq_weight, _F32, (d,), device),
        None if dk_weight is None else _dense("dk_weight", dk_weight, _F32, (d,), device), space, nbytes,
        *sizes, bool(interleaved), eps, code, _handle(stream, device)), "fa_qk_norm_rope_bwd")


# ---------------------------------------------------------------- windowed attention
def fa_fwd_window(q, k, v, o, lse, scale, window, n_sink, dtype=FA_BF16, stream=None):
    """Forward under a causal window of `window` keys and the first n_sink keys: q, o
    [B, H, N, d], k, v [B, H_kv, N, d] bfloat16; lse [B, H, N] or None."""
    device = _current_device()
    B, H, N, d = _sizes("q", q)
    H_kv = _sizes("k", k)[1]
    rows, kv_rows = (B, H, N, d), (B, H_kv, N, d)
    _check(lib().fa_fwd_window(_dense("q", q, _BF16, rows, device), _dense("k", k, _BF16, kv_rows, device),
                               _dense("v", v, _BF16, kv_rows, device), _dense("o", o, _BF16, rows, device),
                               None if lse is None else _dense("lse", lse, _F32, (B, H, N), device), B, H,
                               H_kv, N, d, scale, _int(window), _int(n_sink), dtype, _handle(stream, device)),
           "fa_fwd_window")


def fa_bwd_window_workspace_size(B, H, H_kv, N, d, window, n_sink):
    return int(lib().fa_bwd_window_workspace_size(*map(_int, (B, H, H_kv, N, d, window, n_sink))))


def fa_bwd_window(q, k, v, o, lse, do, dq, dk, dv, workspace, scale, window, n_sink, dtype=FA_BF16,
                  stream=None):
    """dq, dk, dv <- backward of fa_fwd_window, from its o and lse."""
    device = _current_device()
    B, H, N, d = _sizes("q", q)
    H_kv = _sizes("k", k)[1]
    rows, kv_rows = (B, H, N, d), (B, H_kv, N, d)
    _check(lib().fa_bwd_window(
        _dense("q", q, _BF16, rows, device), _dense("k", k, _BF16, kv_rows, device),
        _dense("v", v, _BF16, kv_rows, device), _dense("o", o, _BF16, rows, device),
        _dense("lse", lse, _F32, (B, H, N), device), _dense("do", do, _BF16, rows, device),
        _dense("dq", dq, _BF16, rows, device), _dense("dk", dk, _BF16, kv_rows, device),
        _dense("dv", dv, _BF16, kv_rows, device), *_space(workspace, device), B, H, H_kv, N, d, scale,
        _int(window), _int(n_sink), dtype, _handle(stream, device)), "fa_bwd_window")


# ---------------------------------------------------------------- the 4-bit cache
def kv4_cache(n_pages, H_kv, page, d, device="cuda"):
    """Zeroed arrays of a 4-bit cache: k_codes, k_scales, v_codes, v_scales."""
    codes = [torch.zeros((n_pages, H_kv, page, d // 2), dtype=_U8, device=device) for _ in "kv"]
    scales = [torch.zeros((n_pages, H_kv, page, d // 32), dtype=_BF16, device=device) for _ in "kv"]
    return codes[0], scales[0], codes[1], scales[1]


def _cache(k_codes, k_scales, v_codes, v_scales, block_table, B, H_kv, d, device):
    """Pointers of the cache and its table, and page, n_pages, max_blocks."""
    n_pages, heads, page, _ = _sizes("k_codes", k_codes)
    if block_table.dim() != 2 or (H_kv is not None and heads != H_kv):
        raise ValueError(f"4-bit cache: block_table [B, max_blocks] and {H_kv} K/V heads expected, got "
                         f"{list(block_table.shape)} and {heads}")
    max_blocks = block_table.shape[1]
    codes, scales = (n_pages, heads, page, d // 2), (n_pages, heads, page, d // 32)
    return ((_dense("k_codes", k_codes, _U8, codes, device), _dense("k_scales", k_scales, _BF16, scales, device),
             _dense("v_codes", v_codes, _U8, codes, device), _dense("v_scales", v_scales, _BF16, scales, device),
             _dense("block_table", block_table, _I32, (B, max_blocks), device)),
            (page, n_pages, _int(max_blocks)))


def fa_kv4_append(k, v, k_codes, k_scales, v_codes, v_scales, block_table, first, count=None,
                  stream=None):
    """Store k, v (bfloat16 [B, H_kv, N, d]) in the cache as tokens first[b] + 0 .. count[b] - 1
    (int32 [B]; count None: N)."""
    device = _current_device()
    B, H_kv, N, d = rows = _sizes("k", k)
    cache, pages = _cache(k_codes, k_scales, v_codes, v_scales, block_table, B, H_kv, d, device)
    _check(lib().fa_kv4_append(_dense("k", k, _BF16, rows, device), _dense("v", v, _BF16, rows, device), *cache,
                               _dense("first", first, _I32, (B,), device),
                               None if count is None else _dense("count", count, _I32, (B,), device), B, H_kv,
                               N, d, *pages, _handle(stream, device)), "fa_kv4_append")


def fa_kv4_read(k_codes, k_scales, v_codes, v_scales, block_table, lengths, k, v, stream=None):
    """k, v (bfloat16 [B, H_kv, N, d]) <- the cache's first N tokens of every request; rows from
    lengths[b] (int32 [B]) on are zeros."""
    device = _current_device()
    B, H_kv, N, d = rows = _sizes("k", k)
    cache, pages = _cache(k_codes, k_scales, v_codes, v_scales, block_table, B, H_kv, d, device)
    _check(lib().fa_kv4_read(*cache, _dense("lengths", lengths, _I32, (B,), device),
                             _dense("k", k, _BF16, rows, device), _dense("v", v, _BF16, rows, device), B, H_kv,
                             N, d, *pages, _handle(stream, device)), "fa_kv4_read")


def fa_decode_kv4_workspace_size(B, H, H_kv, N_q, d):
    return int(lib().fa_decode_kv4_workspace_size(*map(_int, (B, H, H_kv, N_q, d))))


def fa_decode_kv4(q, k_codes, k_scales, v_codes, v_scales, block_table, lengths, o, lse, workspace,
                  scale, window=0, n_sink=0, stream=None):
    """o (and lse, may be None) <- attention of the newest N_q tokens of every request, q
    [B, H, N_q, d], over the 4-bit cache; lengths int32 [B]; window 0: all earlier tokens."""
    device = _current_device()
    B, H, N_q, d = rows = _sizes("q", q)
    cache, pages = _cache(k_codes, k_scales, v_codes, v_scales, block_table, B, None, d, device)
    _check(lib().fa_decode_kv4(_dense("q", q, _BF16, rows, device), *cache,
                               _dense("lengths", lengths, _I32, (B,), device),
                               _dense("o", o, _BF16, rows, device),
                               None if lse is None else _dense("lse", lse, _F32, (B, H, N_q), device),
                               *_space(workspace, device), B, H, k_codes.shape[1], N_q, d, *pages, scale,
                               _int(window), _int(n_sink), _handle(stream, device)), "fa_decode_kv4")
