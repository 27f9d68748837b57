"""Measured cases of the attention layer's operators: per-head norm and rotation of Q and K
with its gradient, windowed attention with sinks and its gradient, and attention over a
paged 4-bit K/V cache (writing it, reading it back, decoding from it).

``run`` computes a case with elementary torch operations in float32, or, where ``own`` is
true, with the library's kernels.  ``exact`` computes the same from the definitions in
float64.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
ROPE_BASE = 10000.0


# ---------------------------------------------------------------- cases
def _norm(name, grad, B, N, H, H_kv, d, rot, pos0, dtype="bf16", interleaved=False):
    return {"name": name, "op": "norm_rope_grad" if grad else "norm_rope", "B": B, "N": N, "H": H,
            "H_kv": H_kv, "d": d, "rot": rot, "pos0": pos0, "dtype": dtype,
            "interleaved": interleaved}


def _window(name, grad, B, N, H, H_kv, d, window, sinks):
    return {"name": name, "op": "window_step" if grad else "window", "B": B, "N": N, "H": H,
            "H_kv": H_kv, "d": d, "window": window, "sinks": sinks}


def _cache(name, B, old_min, old_max, new, H_kv, d, page):
    return {"name": name, "op": "cache", "B": B, "len_min": old_min, "len_max": old_max, "new": new,
            "H_kv": H_kv, "d": d, "page": page}


def _decode(name, B, len_min, len_max, N_q, H, H_kv, d, page, window=0, sinks=0):
    return {"name": name, "op": "decode", "B": B, "len_min": len_min, "len_max": len_max, "N_q": N_q,
            "H": H, "H_kv": H_kv, "d": d, "page": page, "window": window, "sinks": sinks}


def listed():
    return [
        # the projections of one decoding step of 32 requests, far into their texts
        _norm("norm_rope_one_token", False, 32, 1, 32, 8, 128, 128, 100000),
        # a whole prompt at the library's longest configuration
        _norm("norm_rope_prompt", False, 1, 16384, 32, 8, 128, 128, 0),
        # gradient in float32, ragged length, half of each head rotated, neighbouring pairs
        _norm("norm_rope_grad_f32", True, 3, 1021, 16, 16, 64, 32, 0, "f32", True),
        # gradient of a training batch
        _norm("norm_rope_grad_batch", True, 4, 4096, 32, 8, 128, 128, 0),
        # a short ragged batch under a narrow window
        _window("window_ragged", False, 4, 1000, 16, 16, 64, 256, 4),
        # the prefill of a long prompt under a wide window, grouped heads
        _window("window_long", False, 1, 16384, 32, 8, 128, 4096, 4),
        # forward and backward at the size of the library's d = 64 training configuration
        _window("window_step_b4", True, 4, 2048, 16, 16, 64, 512, 4),
        # forward and backward of one long odd sequence, grouped heads
        _window("window_step_long", True, 1, 8191, 16, 4, 128, 1024, 16),
        # a chunk of tokens added behind ragged lengths, and the caches read back
        _cache("cache_chunk", 8, 3, 700, 129, 8, 64, 16),
        # two long prompts stored and read back
        _cache("cache_prompt", 2, 0, 0, 8192, 8, 128, 64),
        # one request decoding far into its text: latency
        _decode("decode_single", 1, 16000, 16000, 1, 32, 8, 128, 64),
        # a serving batch of ragged lengths: bandwidth
        _decode("decode_batch", 64, 1000, 32768, 1, 32, 8, 128, 64),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng, most=32):
    g = rng.choice([1, 1, 2, 3, 4, 7, 8, 16])
    kv = rng.choice([k for k in (1, 2, 3, 4, 5, 8, 16, 32) if k * g <= most])
    return kv * g, kv


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_grad", "window", "window_step", "cache", "decode"])
    d = rng.choice([64, 128])
    if op in ("norm_rope", "norm_rope_grad"):
        H, H_kv = _heads(rng)
        dtype = rng.choice(["bf16", "bf16", "f32"])
        most = 16384 * 48 * 128 // ((H + 2 * H_kv) * d * (2 if dtype == "f32" else 1))
        tokens = _log_int(rng, 1, min(most, 1 << 17))
        B = min(tokens, _log_int(rng, 1, 64))
        rot = rng.choice([d, d, d // 2, 16])
        c = _norm("", op == "norm_rope_grad", B, max(1, tokens // B), H, H_kv, d, rot,
                  rng.choice([0, rng.randrange(1 << 20)]), dtype, rng.random() < 0.4)
    elif op in ("window", "window_step"):
        H, H_kv = _heads(rng)
        # a step has two keys or more to choose from: with one, Q and K have no gradient
        least = 2 if op == "window_step" else 1
        N = _log_int(rng, least, 8192 if op == "window_step" else 16384)
        # at most the pairs (B H N window d) and the scores (B H N N) of the longest listed case
        pairs, scores = (8191 * 1024 * 16 * 128, 8191 * 8191 * 16) if op == "window_step" else \
            (16384 * 4096 * 32 * 128, 16384 * 16384 * 32)
        while H * N * N > scores and H > H_kv:
            H -= H_kv
        if H * N * N > scores:
            H = H_kv = max(1, scores // (N * N))
        top = max(least, min(N + 100, 8192, pairs // (H * N * d)))
        window = _log_int(rng, least, top)
        B = _log_int(rng, 1, max(1, min(16, scores // (H * N * N), pairs // (H * N * min(window, N) * d),
                                        4 * 8191 * 16 * 128 // (H * N * d))))
        c = _window("", op == "window_step", B, N, H, H_kv, d, window, rng.choice([0, 1, 4, 4, 17, 130]))
    elif op == "cache":
        H_kv = rng.choice([1, 2, 3, 4, 8, 16])
        B = _log_int(rng, 1, 64)
        most = max(2, 2 * 8192 * 8 * 128 // (B * H_kv * d))
        new = _log_int(rng, 1, max(1, min(8192, most - 1)))
        hi = rng.randrange(0, max(1, min(8192, most - new)))
        c = _cache("", B, rng.randrange(0, hi + 1), hi, new, H_kv, d, rng.choice([16, 32, 64, 128]))
    else:
        H, H_kv = _heads(rng)
        N_q = rng.choice([1, 1, 1, 2, 5])
        B = _log_int(rng, 1, 128)
        most = 64 * 16884 * 8 * 128 // (B * H_kv * d) * 8 // max(8, H // H_kv * N_q)
        hi = _log_int(rng, 1, max(1, min(65536, most)))
        lo = rng.choice([hi, max(0, hi // 30), 0])
        window = rng.choice([0, 0, _log_int(rng, 1, 8192)])
        c = _decode("", B, lo, hi, N_q, H, H_kv, d, rng.choice([16, 32, 64, 128]), window,
                    rng.choice([0, 4, 20]) if window else 0)
    del c["name"]
    return c


def _lengths(c):
    """The requests' lengths: spread evenly over the case's range, in a mixed order."""
    B, lo, hi = c["B"], c["len_min"], c["len_max"]
    return [lo + (hi - lo) * ((b * 37 + 11) % B) // max(1, B - 1) for b in range(B)]


def _visible(length, c):
    """Keys that the N_q queries at the end of one request read between them."""
    n = length
    if c["window"]:
        lo = max(0, length - c["N_q"] + 1 - c["window"])
        n = length - lo + min(lo, c["sinks"])
    return n


def work(c):
    if c["op"] in ("norm_rope", "norm_rope_grad"):
        e = 2 if c["dtype"] == "bf16" else 4
        x = c["B"] * c["N"] * (c["H"] + 2 * c["H_kv"]) * c["d"]
        qk = c["B"] * c["N"] * (c["H"] + c["H_kv"]) * c["d"]
        if c["op"] == "norm_rope":
            return {"bytes": 2 * x * e, "flops": 8 * qk}
        return {"bytes": (2 * x + qk) * e, "flops": 18 * qk}
    if c["op"] in ("window", "window_step"):
        N, W, S = c["N"], c["window"], c["sinks"]
        i = np.arange(N, dtype=np.int64)
        lo = np.maximum(0, i - W + 1)
        pairs = float(np.sum(i - lo + 1 + np.minimum(lo, S))) * c["B"] * c["H"]
        qo, kv = c["B"] * c["H"] * N * c["d"] * 2, c["B"] * c["H_kv"] * N * c["d"] * 2
        if c["op"] == "window":
            return {"bytes": 2 * qo + 2 * kv + c["B"] * c["H"] * N * 4, "flops": 4 * pairs * c["d"]}
        return {"bytes": 4 * qo + 4 * kv, "flops": 14 * pairs * c["d"]}
    row = c["H_kv"] * (c["d"] // 2 + c["d"] // 16)  # one token's K or V in 4 bits, with its scales
    dense = c["H_kv"] * c["d"] * 2
    if c["op"] == "cache":
        new, total = c["B"] * c["new"], sum(_lengths(c)) + c["B"] * c["new"]
        return {"bytes": 2 * (new * (dense + row) + (total - new) * row + c["B"] * max(
            n + c["new"] for n in _lengths(c)) * dense), "flops": 8 * (new + total) * c["H_kv"] * c["d"]}
    keys = sum(_visible(n, c) for n in _lengths(c))
    rows = c["B"] * c["H"] * c["N_q"]
    return {"bytes": 2 * keys * row + 2 * rows * c["d"] * 2 + rows * 4,
            "flops": 4 * keys * c["N_q"] * c["H"] * c["d"]}


# ---------------------------------------------------------------- inputs
class _State:
    pass


def _normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(dtype)


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = _State()
    s.c = c
    B, H_kv, d = c["B"], c["H_kv"], c["d"]
    bf = torch.bfloat16
    if c["op"] in ("norm_rope", "norm_rope_grad"):
        N, H = c["N"], c["H"]
        dt = bf if c["dtype"] == "bf16" else torch.float32
        s.qkv = _normal(gen, (B, N, H + 2 * H_kv, d), dt, 2.0)
        s.q_weight = 1.0 + _normal(gen, (d,), torch.float32, 0.1)
        s.k_weight = 1.0 + _normal(gen, (d,), torch.float32, 0.1)
        start = torch.randint(0, 1000, (B, 1), generator=gen, device="cuda", dtype=torch.int32)
        s.positions = (c["pos0"] + start + torch.arange(N, device="cuda", dtype=torch.int32)).contiguous()
        half = c["rot"] // 2
        s.inv_freq = ROPE_BASE ** (-torch.arange(half, dtype=torch.float64) / half)
        empty = lambda *shape: torch.empty(shape, dtype=dt, device="cuda")  # noqa: E731
        if c["op"] == "norm_rope":
            s.q, s.k, s.v = empty(B, H, N, d), empty(B, H_kv, N, d), empty(B, H_kv, N, d)
        else:
            s.dq, s.dk, s.dv = (_normal(gen, (B, h, N, d), dt) for h in (H, H_kv, H_kv))
            s.dqkv = torch.empty_like(s.qkv)
            s.dq_weight, s.dk_weight = torch.empty_like(s.q_weight), torch.empty_like(s.k_weight)
            s.workspace = None
    elif c["op"] in ("window", "window_step"):
        N, H = c["N"], c["H"]
        s.q = _normal(gen, (B, H, N, d), bf)
        s.k, s.v = _normal(gen, (B, H_kv, N, d), bf), _normal(gen, (B, H_kv, N, d), bf)
        s.o = torch.empty_like(s.q)
        s.lse = torch.empty((B, H, N), dtype=torch.float32, device="cuda")
        if c["op"] == "window_step":
            s.do = _normal(gen, (B, H, N, d), bf)
            s.dq, s.dk, s.dv = torch.empty_like(s.q), torch.empty_like(s.k), torch.empty_like(s.v)
            s.workspace = None
    else:
        page, old = c["page"], _lengths(c)
        lens = [n + c.get("new", 0) for n in old]
        need = [-(-n // page) for n in lens]
        n_pages = sum(need) + 3
        perm = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32).cpu()
        table = torch.full((B, max(1, max(need))), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = perm[at:at + n]
            at += n
        s.block_table = table.cuda()
        s.old = torch.tensor(old, dtype=torch.int32, device="cuda")
        s.lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s.codes, s.scales = _full_cache(c, [_normal(gen, (n_pages, H_kv, page, d), bf) for _ in range(2)])
        if c["op"] == "cache":
            s.k_new, s.v_new = (_normal(gen, (B, H_kv, c["new"], d), bf) for _ in range(2))
            s.k, s.v = (torch.empty((B, H_kv, max(lens), d), dtype=bf, device="cuda") for _ in range(2))
        else:
            s.q = _normal(gen, (B, c["H"], c["N_q"], d), bf)
            s.o = torch.empty_like(s.q)
            s.lse = torch.empty(s.q.shape[:3], dtype=torch.float32, device="cuda")
            s.workspace = None
    return s


# ---------------------------------------------------------------- plain forms
def _norm_rope_parts(s):
    """x (q and k heads) in float32, 1/rms, weights by head, and the pairs' cos and sin."""
    c = s.c
    H, H_kv = c["H"], c["H_kv"]
    x = s.qkv[:, :, :H + H_kv].float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    w = torch.cat([s.q_weight.expand(H, -1), s.k_weight.expand(H_kv, -1)])
    angle = s.positions.double()[..., None] * s.inv_freq.cuda()
    return x, r, w, angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]


def _rotate(x, cos, sin, rot, interleaved):
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        h = rot // 2
        a, b = x[..., :h], x[..., h:rot]
        y[..., :h], y[..., h:rot] = a * cos - b * sin, b * cos + a * sin
    return y


def _plain_norm_rope(s):
    c = s.c
    x, r, w, cos, sin = _norm_rope_parts(s)
    y = _rotate(x * r * w, cos, sin, c["rot"], c["interleaved"]).to(s.qkv.dtype)
    y = y.transpose(1, 2).contiguous()
    v = s.qkv[:, :, c["H"] + c["H_kv"]:].transpose(1, 2).contiguous()
    return {"q": y[:, :c["H"]], "k": y[:, c["H"]:], "v": v}


def _plain_norm_rope_grad(s):
    c = s.c
    H = c["H"]
    x, r, w, cos, sin = _norm_rope_parts(s)
    dy = torch.cat([s.dq, s.dk], 1).transpose(1, 2).float()
    g = _rotate(dy, cos, -sin, c["rot"], c["interleaved"])
    n = x * r
    dw = (g * n).double().sum((0, 1))
    gw = g * w
    dx = r * (gw - n * (gw * n).mean(-1, keepdim=True))
    dqkv = torch.cat([dx.to(s.qkv.dtype), s.dv.transpose(1, 2)], 2)
    return {"dqkv": dqkv, "dq_weight": dw[:H].sum(0).float(), "dk_weight": dw[H:].sum(0).float()}


def _window_scores(s, k):
    """softmax of the visible scores and its logsumexp, [B, H_kv, G, N, N] and [..., N]."""
    c = s.c
    N = c["N"]
    q = s.q.float().view(c["B"], c["H_kv"], -1, N, c["d"])
    S = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(c["d"]))
    i = torch.arange(N, device="cuda")
    seen = (i[None] <= i[:, None]) & ((i[None] > i[:, None] - c["window"]) | (i[None] < c["sinks"]))
    S.masked_fill_(~seen, -math.inf)
    m = S.amax(-1, keepdim=True)
    S.sub_(m).exp_()
    total = S.sum(-1, keepdim=True)
    return S.div_(total), (m + total.log())[..., 0], q


def _plain_window(s):
    shape = s.q.shape
    P, lse, _ = _window_scores(s, s.k.float()[:, :, None])
    o = torch.matmul(P, s.v.float()[:, :, None])
    return {"o": o.to(s.q.dtype).view(shape), "lse": lse.reshape(shape[:3])}


def _plain_window_step(s):
    c, shape = s.c, s.q.shape
    k, v = s.k.float()[:, :, None], s.v.float()[:, :, None]
    P, _, q = _window_scores(s, k)
    do = s.do.float().view(q.shape)
    o = torch.matmul(P, v)
    delta = (do * o).sum(-1, keepdim=True)
    dv = torch.matmul(P.transpose(-1, -2), do).sum(2)
    dS = torch.matmul(do, v.transpose(-1, -2)).sub_(delta).mul_(P).mul_(1.0 / math.sqrt(c["d"]))
    dq = torch.matmul(dS, k)
    dk = torch.matmul(dS.transpose(-1, -2), q).sum(2)
    t = s.q.dtype
    return {"o": o.to(t).view(shape), "dq": dq.to(t).view(shape), "dk": dk.to(t), "dv": dv.to(t)}


# The cache's 4-bit form: 32 neighbouring values of a head share a bfloat16 scale
# s = bf16(amax / 7); a value's code is x / s rounded to the nearest even integer in -7..7, held
# as the nibble code + 8.
def _quantise(x):
    x = x.float().unflatten(-1, (-1, 32))
    scale = (x.abs().amax(-1) / 7.0).to(torch.bfloat16)
    s = scale.float()[..., None]
    code = torch.where(s > 0, torch.round(x / s).clamp_(-7, 7), torch.zeros_like(x))
    return (code + 8).to(torch.uint8).flatten(-2), scale


# Where a token's bytes (of two neighbouring values) and scales lie within its page, [page, d / 2]
# and [page, d / 32]: K in token rows of 32-bit words (t, group) of eight values, V in tiles of 16
# tokens of 16-bit words (half, g, pair, token of the pair, group) of four values, V's scales with
# two tokens side by side.
def _places(c, which):
    page, d = c["page"], c["d"]
    groups = d // 32
    slot = torch.arange(page, device="cuda")[:, None]
    e = torch.arange(0, d, 2, device="cuda")[None]
    group = torch.arange(groups, device="cuda")[None]
    if which == 0:
        return slot * (d // 2) + 4 * (e % 32 // 8 * groups + e // 32) + e % 8 // 2, slot * groups + group
    half, k = slot % 16 // 8, slot % 8
    word = (((half * 8 + e % 32 // 4) * 4 + k // 2) * 2 + k % 2) * groups + e // 32
    return slot // 16 * (8 * d) + 2 * word + e % 4 // 2, slot // 2 * (2 * groups) + 2 * group + slot % 2


def _store(codes, scales, nibbles, scale, places, page, slot):
    """Tokens [..., H_kv, d] and [..., H_kv, d / 32] into their pages' places."""
    for array, place, x in zip((codes, scales), places, _halves(nibbles, scale)):
        array.flatten(2)[page[..., None], :, place[slot]] = x.transpose(-1, -2)


def _full_cache(c, x):
    """Codes and scales of pages that hold x [n_pages, H_kv, page, d], K's then V's."""
    out = []
    for which in range(2):
        for data, place in zip(_halves(*_quantise(x[which])), _places(c, which)):
            order = torch.argsort(place.flatten())
            out.append(data.flatten(2)[..., order].view_as(data))
    return out[0::2], out[1::2]


def _halves(nibbles, scale):
    return nibbles[..., 0::2] | (nibbles[..., 1::2] << 4), scale


def _values(s, which):
    """The cached K (0) or V (1) of every request, [B, H_kv, positions, d] in float32."""
    c = s.c
    table = s.block_table.clamp(min=0).long()
    byte, scale = (a[which].flatten(2)[table][..., place.flatten()].unflatten(-1, place.shape).transpose(
        1, 2).flatten(2, 3) for a, place in zip((s.codes, s.scales), _places(c, which)))
    code = torch.stack([byte & 15, byte >> 4], -1).flatten(-2)
    x = (code.float() - 8).unflatten(-1, (-1, 32)) * scale.float()[..., None]
    return x.view(c["B"], c["H_kv"], -1, c["d"])


def _plain_cache(s):
    c = s.c
    pos = s.old[:, None].long() + torch.arange(c["new"], device="cuda")
    page = torch.gather(s.block_table.long(), 1, pos // c["page"])
    out = {}
    for which, (x, name) in enumerate(((s.k_new, "k"), (s.v_new, "v"))):
        nibbles, scale = _quantise(x.transpose(1, 2))
        _store(s.codes[which], s.scales[which], nibbles, scale, _places(c, which), page, pos % c["page"])
        n = s.k.shape[2]
        seen = torch.arange(n, device="cuda") < s.lengths[:, None]
        y = _values(s, which)[:, :, :n] * seen[:, None, :, None]
        out[name] = y.to(torch.bfloat16)
    return out


def _plain_decode(s):
    c = s.c
    B, H_kv, N_q, d = c["B"], c["H_kv"], c["N_q"], c["d"]
    q = s.q.float().view(B, H_kv, -1, d)  # [B, H_kv, G * N_q, d]
    S = torch.matmul(q, _values(s, 0).transpose(-1, -2)).mul_(1.0 / math.sqrt(d))
    j = torch.arange(S.shape[-1], device="cuda")
    i = s.lengths[:, None] - N_q + torch.arange(N_q, device="cuda")  # [B, N_q]
    seen = j <= i[..., None]
    if c["window"]:
        seen &= (j > i[..., None] - c["window"]) | (j < c["sinks"])
    S = S.view(B, H_kv, -1, N_q, S.shape[-1])
    S.masked_fill_(~seen[:, None, None], -math.inf)
    m = S.amax(-1, keepdim=True)
    P = S.sub_(m.clamp(min=torch.finfo(torch.float32).min)).exp_()
    total = P.sum(-1, keepdim=True)
    o = torch.matmul(P.flatten(2, 3), _values(s, 1)).view(B, H_kv, -1, N_q, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (m + total.log())[..., 0]
    return {"o": o.reshape(s.q.shape).to(s.q.dtype), "lse": lse.reshape(s.lse.shape)}


# ---------------------------------------------------------------- one pass
def run(s):
    if own:
        return _own(s)
    return {"norm_rope": _plain_norm_rope, "norm_rope_grad": _plain_norm_rope_grad,
            "window": _plain_window, "window_step": _plain_window_step, "cache": _plain_cache,
            "decode": _plain_decode}[s.c["op"]](s)


def _own(s):
    import exact_io_aware_06_gb300 as fa
    c, op = s.c, s.c["op"]
    scale = 1.0 / math.sqrt(c["d"])
    if getattr(s, "workspace", 0) is None:  # kept with the state, as a program keeps it
        if op == "norm_rope_grad":
            n = fa.fa_qk_norm_rope_bwd_workspace_size(c["B"], c["H"], c["H_kv"], c["N"], c["d"])
        elif op == "window_step":
            n = fa.fa_bwd_window_workspace_size(c["B"], c["H"], c["H_kv"], c["N"], c["d"], c["window"],
                                                c["sinks"])
        else:
            n = fa.fa_decode_kv4_workspace_size(c["B"], c["H"], c["H_kv"], c["N_q"], c["d"])
        s.workspace = torch.empty(n, dtype=torch.uint8, device="cuda")
    if op == "norm_rope":
        fa.fa_qk_norm_rope(s.qkv, s.q_weight, s.k_weight, s.positions, s.inv_freq, s.q, s.k, s.v, EPS,
                           c["interleaved"])
        return {"q": s.q, "k": s.k, "v": s.v}
    if op == "norm_rope_grad":
        fa.fa_qk_norm_rope_bwd(s.qkv, s.q_weight, s.k_weight, s.positions, s.inv_freq, s.dq, s.dk, s.dv,
                               s.dqkv, s.dq_weight, s.dk_weight, s.workspace, EPS, c["interleaved"])
        return {"dqkv": s.dqkv, "dq_weight": s.dq_weight, "dk_weight": s.dk_weight}
    if op in ("window", "window_step"):
        fa.fa_fwd_window(s.q, s.k, s.v, s.o, s.lse, scale, c["window"], c["sinks"], fa.FA_BF16)
        if op == "window":
            return {"o": s.o, "lse": s.lse}
        fa.fa_bwd_window(s.q, s.k, s.v, s.o, s.lse, s.do, s.dq, s.dk, s.dv, s.workspace, scale,
                         c["window"], c["sinks"], fa.FA_BF16)
        return {"o": s.o, "dq": s.dq, "dk": s.dk, "dv": s.dv}
    cache = (s.codes[0], s.scales[0], s.codes[1], s.scales[1], s.block_table)
    if op == "cache":
        fa.fa_kv4_append(s.k_new, s.v_new, *cache, s.old, None)
        fa.fa_kv4_read(*cache, s.lengths, s.k, s.v)
        return {"k": s.k, "v": s.v}
    fa.fa_decode_kv4(s.q, *cache, s.lengths, s.o, s.lse, s.workspace, scale, c["window"], c["sinks"])
    return {"o": s.o, "lse": s.lse}


# ---------------------------------------------------------------- definitions in 64 bits
def _exact_norm_rope(s, c):
    """Each head: x / sqrt(mean(x^2) + eps) * w, its pairs turned as complex numbers."""
    half = c["rot"] // 2
    place = torch.arange(c["rot"], device="cuda")
    place = place.view(half, 2) if c["interleaved"] else place.view(2, half).T
    turn = s.positions.double().cpu()[..., None] * s.inv_freq
    turn = torch.polar(torch.ones_like(turn), turn).cuda()
    out, dqkv, dws = {}, [], {}
    first = 0
    for name, heads, w in (("q", c["H"], s.q_weight), ("k", c["H_kv"], s.k_weight)):
        x = s.qkv[:, :, first:first + heads].double()
        first += heads
        n = x / (x.pow(2).sum(-1, keepdim=True) / c["d"] + EPS).sqrt()
        if c["op"] == "norm_rope":
            y = n * w.double()
            z = torch.complex(y[..., place[:, 0]], y[..., place[:, 1]]) * turn[:, :, None]
            y[..., place[:, 0]], y[..., place[:, 1]] = z.real, z.imag
            out[name] = y.transpose(1, 2)
            continue
        g = (s.dq if name == "q" else s.dk).double().transpose(1, 2).clone()
        z = torch.complex(g[..., place[:, 0]], g[..., place[:, 1]]) * turn[:, :, None].conj()
        g[..., place[:, 0]], g[..., place[:, 1]] = z.real, z.imag
        dws[name] = torch.einsum("bnhe,bnhe->e", g, n)
        g = g * w.double()
        # n is x over its length sqrt(d (mean + eps) / d): dn/dx = (1 - n n^T / d) / rms
        rms = (x.pow(2).sum(-1, keepdim=True) / c["d"] + EPS).sqrt()
        dqkv.append((g - n * (torch.einsum("bnhe,bnhe->bnh", g, n) / c["d"])[..., None]) / rms)
    if c["op"] == "norm_rope":
        out["v"] = s.qkv[:, :, first:].double().transpose(1, 2)
        return out
    dqkv.append(s.dv.double().transpose(1, 2))
    return {"dqkv": torch.cat(dqkv, 2), "dq_weight": dws["q"], "dk_weight": dws["k"]}


def _exact_window(s, c):
    """Query tile by query tile over the keys that it can see."""
    N, d, S, W, T = c["N"], c["d"], c["sinks"], c["window"], 512
    scale = 1.0 / math.sqrt(d)
    G = c["H"] // c["H_kv"]
    o = torch.zeros(s.q.shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s.q.shape[:3], dtype=torch.float64, device="cuda")
    grads = c["op"] == "window_step"
    if grads:
        dq = torch.zeros_like(o)
        dk, dv = (torch.zeros(s.k.shape, dtype=torch.float64, device="cuda") for _ in range(2))
    for b in range(c["B"]):
        for kv in range(c["H_kv"]):
            h = slice(kv * G, kv * G + G)
            for r0 in range(0, N, T):
                r1 = min(N, r0 + T)
                lo = max(0, r0 - W + 1)
                keys = torch.cat([torch.arange(min(S, lo)), torch.arange(lo, r1)]).cuda()
                rows = torch.arange(r0, r1, device="cuda")[:, None]
                hidden = (keys > rows) | ((keys <= rows - W) & (keys >= S))
                q, k, v = s.q[b, h, r0:r1].double(), s.k[b, kv, keys].double(), s.v[b, kv, keys].double()
                A = (q @ k.T) * scale
                A[:, hidden] = -math.inf
                L = torch.logsumexp(A, -1)
                P = (A - L[..., None]).exp()
                o[b, h, r0:r1], lse[b, h, r0:r1] = P @ v, L
                if grads:
                    do = s.do[b, h, r0:r1].double()
                    dv[b, kv].index_add_(0, keys, torch.einsum("hij,hie->je", P, do))
                    dP = do @ v.T
                    dA = P * (dP - (P * dP).sum(-1, keepdim=True)) * scale
                    dq[b, h, r0:r1] = dA @ k
                    dk[b, kv].index_add_(0, keys, torch.einsum("hij,hie->je", dA, q))
    return {"o": o, "dq": dq, "dk": dk, "dv": dv} if grads else {"o": o, "lse": lse}


def _exact_tokens(s, c, which, b, n):
    """The first n cached tokens of request b, [H_kv, n, d]: each value's nibble and scale by place."""
    d, page = c["d"], c["page"]
    i, e = torch.arange(n)[:, None], torch.arange(d)[None]
    k = i % page
    if which == 0:  # nibble of a page
        nibble = k * d + (e % 32 // 8) * (d // 4) + (e // 32) * 8 + e % 8
        scale = k * (d // 32) + e // 32
    else:
        nibble = (k // 16) * 16 * d + (k % 16 // 8) * 8 * d + (e % 32 // 4) * d + (k % 8) * (d // 8) \
            + (e // 32) * 4 + e % 4
        scale = (k // 2) * (d // 16) + (e // 32) * 2 + k % 2
    rows = s.block_table[b, torch.arange(n, device="cuda") // page].long()[:, None]
    byte = s.codes[which].flatten(2)[rows, :, (nibble // 2).cuda()].long()  # [n, d, H_kv]
    code = (byte >> (4 * (nibble % 2)).cuda()[..., None]) % 16 - 8
    x = code.double() * s.scales[which].flatten(2)[rows, :, scale.cuda()].double()
    return x.permute(2, 0, 1)


def _exact_cache(s, c):
    out = {}
    for which, (new, name) in enumerate(((s.k_new, "k"), (s.v_new, "v"))):
        x = new.double().reshape(*new.shape[:-1], -1, 32)
        scale = (x.abs().amax(-1, keepdim=True) / 7).to(torch.bfloat16).double()
        code = torch.where(scale == 0, 0.0, x / scale).round().clip(-7, 7)
        stored = (code * scale).reshape(new.shape)
        y = torch.zeros(s.k.shape, dtype=torch.float64, device="cuda")
        for b, old in enumerate(_lengths(c)):
            if old:
                y[b, :, :old] = _exact_tokens(s, c, which, b, old)
            y[b, :, old:old + c["new"]] = stored[b]
        out[name] = y
    return out


def _exact_decode(s, c):
    N_q, d = c["N_q"], c["d"]
    G = c["H"] // c["H_kv"]
    o = torch.zeros(s.q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s.q.shape[:3], -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lengths(c)):
        if n == 0:
            continue
        k, v = _exact_tokens(s, c, 0, b, n), _exact_tokens(s, c, 1, b, n)
        for i in range(N_q):
            last = n - N_q + i
            if last < 0:
                continue
            lo = max(0, last - c["window"] + 1) if c["window"] else 0
            keys = torch.cat([torch.arange(min(c["sinks"], lo)), torch.arange(lo, last + 1)]).cuda()
            q = s.q[b, :, i].double().view(c["H_kv"], G, d)
            A = torch.einsum("kge,kne->kgn", q, k[:, keys]) / math.sqrt(d)
            L = torch.logsumexp(A, -1)
            o[b, :, i] = torch.einsum("kgn,kne->kge", (A - L[..., None]).exp(), v[:, keys]).reshape(-1, d)
            lse[b, :, i] = L.reshape(-1)
    return {"o": o, "lse": lse}


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"].startswith("norm_rope"):
        return _exact_norm_rope(s, c)
    if c["op"].startswith("window"):
        return _exact_window(s, c)
    return (_exact_cache if c["op"] == "cache" else _exact_decode)(s, c)
