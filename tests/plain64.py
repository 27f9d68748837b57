"""Plain float64 numpy forms of the layer's operators, written from their definitions."""
import numpy as np

NEG = -np.inf


# ---------------------------------------------------------------- norm and rotation
def rope_pairs(rot, interleaved):
    p = np.arange(rot // 2)
    return (2 * p, 2 * p + 1) if interleaved else (p, p + rot // 2)


def turn(x, positions, inv_freq, interleaved, sign=1.0):
    """x [B, N, heads, d] with its pairs turned by sign * position * frequency."""
    y = x.copy()
    if inv_freq is None or len(inv_freq) == 0:
        return y
    a, b = rope_pairs(2 * len(inv_freq), interleaved)
    ang = sign * positions[:, :, None, None].astype(np.float64) * np.asarray(inv_freq)
    y[..., a] = x[..., a] * np.cos(ang) - x[..., b] * np.sin(ang)
    y[..., b] = x[..., b] * np.cos(ang) + x[..., a] * np.sin(ang)
    return y


def norm_rope(qkv, H, H_kv, qw, kw, positions, inv_freq, eps, interleaved):
    """q, k, v [B, heads, N, d] of qkv [B, N, H + 2 H_kv, d]."""
    out = []
    for x, w in ((qkv[:, :, :H], qw), (qkv[:, :, H:H + H_kv], kw)):
        r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        out.append(turn(x * r * w, positions, inv_freq, interleaved).swapaxes(1, 2))
    return out[0], out[1], qkv[:, :, H + H_kv:].swapaxes(1, 2)


def norm_rope_grad(qkv, H, H_kv, qw, kw, positions, inv_freq, eps, interleaved, dq, dk, dv):
    """dqkv, dq_weight, dk_weight."""
    parts, dw = [], []
    for x, w, dy in ((qkv[:, :, :H], qw, dq), (qkv[:, :, H:H + H_kv], kw, dk)):
        r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        g = turn(dy.swapaxes(1, 2), positions, inv_freq, interleaved, -1.0)
        dw.append((g * x * r).sum((0, 1, 2)))
        parts.append(r * (w * g - r * r * x * (w * g * x).mean(-1, keepdims=True)))
    parts.append(dv.swapaxes(1, 2))
    return np.concatenate(parts, 2), dw[0], dw[1]


# ---------------------------------------------------------------- attention under a mask
def window_mask(N_q, N_k, offset, window, n_sink):
    """Whether query i (at position offset + i) sees key j; window 0: every earlier key."""
    i, j = offset + np.arange(N_q)[:, None], np.arange(N_k)[None]
    seen = j <= i
    return seen & ((j > i - window) | (j < n_sink)) if window else seen


def attention(q, k, v, scale, seen):
    """One head: O, lse and P of q [n, d] over k, v [m, d]; rows that see nothing give 0, -inf."""
    S = np.where(seen, scale * (q @ k.T), NEG)
    m = S.max(-1, keepdims=True) if k.shape[0] else np.full((len(q), 1), NEG)
    P = np.exp(S - np.where(np.isfinite(m), m, 0.0))
    l = P.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (m + np.log(l))[:, 0]
    P = np.divide(P, l, out=np.zeros_like(P), where=l > 0)
    return P @ v, lse, P


def attention_grad(q, k, v, do, scale, seen):
    """One head: dq, dk, dv."""
    o, _, P = attention(q, k, v, scale, seen)
    dP = do @ v.T
    dS = P * (dP - (do * o).sum(-1, keepdims=True))
    return scale * dS @ k, scale * dS.T @ q, P.T @ do


# ---------------------------------------------------------------- the 4-bit cache
def bf16_round(x):
    """Nearest bfloat16 of float64 values in the normal range, ties to even."""
    x = np.asarray(x, dtype=np.float64)
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 256.0), e - 8)


def kv4_values(x):
    """What rows x [..., d] read back as: codes times scales, in groups of 32."""
    g = x.reshape(*x.shape[:-1], -1, 32)
    s = bf16_round(np.abs(g).max(-1, keepdims=True) / 7.0)
    code = np.divide(g, s, out=np.zeros_like(g), where=s > 0)
    return (np.clip(np.rint(code), -7, 7) * s).reshape(x.shape)
