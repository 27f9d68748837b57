"""Measured cases of attention over another sequence's keys and of positions with several axes:
cross attention to an encoder's states with its gradient and its form for single tokens, attention
of a batch to one shared prefix, and norm and rotation of Q and K by several axes with its gradient.

``run`` computes a case with elementary torch operations in float32, or, where ``own`` is
true, with the library's kernels.  ``exact`` computes the same from the definitions in
float64.
"""
import math

import torch

own = False

EPS = 1e-6
ROPE_BASE = 10000.0


# ---------------------------------------------------------------- cases
def _axes(name, grad, B, N, H, H_kv, d, sections, grid, dtype="bf16", interleaved=False):
    """sections: rotated elements of each axis; grid: height and width of a frame of the grid."""
    return {"name": name, "op": "axes_grad" if grad else "axes", "B": B, "N": N, "H": H, "H_kv": H_kv, "d": d,
            "sections": sections, "grid": grid, "dtype": dtype, "interleaved": interleaved}


def _cross(name, op, B, B_kv, N_q, N_kv, len_min, H, H_kv, d):
    """B_kv sequences of N_kv keys, len_min to N_kv of them real; B / B_kv batches of queries to each."""
    return {"name": name, "op": op, "B": B, "B_kv": B_kv, "N_q": N_q, "N_kv": N_kv, "len_min": len_min, "H": H,
            "H_kv": H_kv, "d": d}


def listed():
    return [
        # one decoding step of 32 requests that hold images in their texts
        _axes("axes_one_token", False, 32, 1, 32, 8, 128, "32,48,48", "32x32"),
        # the tokens of a video, 16 frames of 32 x 32
        _axes("axes_video", False, 1, 16384, 32, 8, 128, "32,48,48", "32x32"),
        # gradient in float32 over images of ragged size, neighbouring pairs, half of each head rotated
        _axes("axes_grad_f32", True, 3, 1021, 16, 16, 64, "16,16", "29x36", "f32", True),
        # gradient of a training batch of short videos
        _axes("axes_grad_batch", True, 4, 4096, 32, 8, 128, "32,48,48", "16x16"),
        # one token of one request over an encoder's states: latency
        _cross("cross_one_token", "cross", 1, 1, 1, 1500, 1500, 16, 16, 64),
        # one token of a serving batch over encoded documents of ragged length: bandwidth
        _cross("cross_token_batch", "cross", 64, 64, 1, 8192, 500, 32, 8, 128),
        # the tokens of a video over an encoded text
        _cross("cross_video", "cross", 2, 2, 16384, 512, 77, 16, 16, 128),
        # training step of a decoder over ragged encoded texts
        _cross("cross_step_b4", "cross_step", 4, 4, 2048, 1000, 300, 16, 16, 64),
        # training step of a short text over a long odd sequence, grouped heads
        _cross("cross_step_long", "cross_step", 1, 1, 1021, 8191, 8191, 16, 4, 128),
        # two prompts with a few samples each, three new tokens a sample
        _cross("prefix_samples", "prefix", 10, 2, 3, 777, 500, 12, 4, 64),
        # one step of 64 requests that share a long prompt
        _cross("prefix_batch", "prefix", 64, 1, 1, 16384, 16384, 32, 8, 128),
        # continuing 32 requests behind a shared prompt by a piece of text each
        _cross("prefix_pieces", "prefix", 32, 1, 256, 4096, 4096, 32, 8, 128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng, most=32):
    g = rng.choice([1, 1, 2, 3, 4, 7, 8, 16])
    kv = rng.choice([k for k in (1, 2, 3, 4, 5, 8, 16, 32) if k * g <= most])
    return kv * g, kv


def draw(rng):
    op = rng.choice(["axes", "axes_grad", "cross", "cross", "cross_step", "prefix"])
    d = rng.choice([64, 128])
    H, H_kv = _heads(rng)
    if op in ("axes", "axes_grad"):
        dtype = rng.choice(["bf16", "bf16", "f32"])
        most = 16384 * 48 * 128 // ((H + 2 * H_kv) * d * (2 if dtype == "f32" else 1))
        tokens = _log_int(rng, 1, min(most, 1 << 17))
        B = min(tokens, _log_int(rng, 1, 64))
        eighth = d // 8
        sections = rng.choice([[d // 2, d // 2], [d // 4, d // 4], [2 * eighth, 3 * eighth, 3 * eighth],
                               [d // 4] * 4, [d - 2 * eighth, eighth, eighth], [d]])
        c = _axes("", op == "axes_grad", B, max(1, tokens // B), H, H_kv, d, ",".join(map(str, sections)),
                  f"{rng.randrange(1, 100)}x{rng.randrange(1, 100)}", dtype, rng.random() < 0.4)
    else:
        # at most the work and the queries (elements) of the kind's largest listed cases, and the keys of the
        # largest of all
        work_, queries = {"cross": (32 * 16384 * 512 * 128, 32 * 16384 * 128),
                          "cross_step": (16 * 1021 * 8191 * 128, 32 * 4096 * 128),
                          "prefix": (1024 * 256 * 4096 * 128, 1024 * 256 * 128)}[op]
        keys = 4 * 8 * 8191 * 128 if op == "cross_step" else 64 * 4346 * 8 * 128
        step = op == "cross_step"
        kind = "rows" if step else rng.choice(["tokens", "rows"])
        least = 2 if step else 1  # with one key, Q and K have no gradient
        N_kv = _log_int(rng, least, 16384 if kind == "tokens" else 8192)
        N_q = rng.choice([1, 1, 1, 2, 5]) if kind == "tokens" else _log_int(rng, 1, 16384)
        while H * N_q * d * max(N_kv, work_ // queries) > work_ and H > H_kv:
            H -= H_kv
        N_q = max(1, min(N_q, work_ // (H * d * max(N_kv, work_ // queries))))
        room = max(1, min(64, work_ // (H * N_q * N_kv * d), queries // (H * N_q * d), keys // (H_kv * N_kv * d)))
        share = _log_int(rng, 1, room) if op == "prefix" else rng.choice([1, 1, 1, min(room, 4)])
        B_kv = rng.choice([1, 1, max(1, min(4, room // share))]) if op == "prefix" else \
            _log_int(rng, 1, max(1, room // share))
        low = rng.choice([N_kv, max(least, N_kv // 8), least if step else 0])
        c = _cross("", op, share * B_kv, B_kv, N_q, N_kv, low, H, H_kv, d)
    del c["name"]
    return c


def _lengths(c):
    """The sequences' real lengths: spread evenly over the case's range, in a mixed order."""
    n, lo, hi = c["B_kv"], c["len_min"], c["N_kv"]
    return [hi - (hi - lo) * ((b * 37 + 11) % n) // max(1, n - 1) for b in range(n)]


def _sections(c):
    return [int(s) for s in c["sections"].split(",")]


def work(c):
    if c["op"] in ("axes", "axes_grad"):
        e = 2 if c["dtype"] == "bf16" else 4
        x = c["B"] * c["N"] * (c["H"] + 2 * c["H_kv"]) * c["d"]
        qk = c["B"] * c["N"] * (c["H"] + c["H_kv"]) * c["d"]
        if c["op"] == "axes":
            return {"bytes": 2 * x * e, "flops": 8 * qk}
        return {"bytes": (2 * x + qk) * e, "flops": 18 * qk}
    keys, rows = sum(_lengths(c)), c["B"] * c["H"] * c["N_q"]
    pairs = keys * (c["B"] // c["B_kv"]) * c["H"] * c["N_q"]
    q, kv = rows * c["d"] * 2, keys * c["H_kv"] * c["d"] * 2
    if c["op"] == "cross":
        return {"bytes": 2 * q + 2 * kv + rows * 4, "flops": 4 * pairs * c["d"]}
    if c["op"] == "prefix":
        return {"bytes": 3 * q + 2 * kv + 2 * rows * 4, "flops": 4 * pairs * c["d"]}
    return {"bytes": 4 * q + 2 * kv + 2 * c["B_kv"] * c["N_kv"] * c["H_kv"] * c["d"] * 2, "flops": 14 * pairs * c["d"]}


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
    B, H, H_kv, d = c["B"], c["H"], c["H_kv"], c["d"]
    bf = torch.bfloat16
    if c["op"] in ("axes", "axes_grad"):
        N = c["N"]
        dt = bf if c["dtype"] == "bf16" else torch.float32
        s.qkv = _normal(gen, (B, N, H + 2 * H_kv, d), dt, 2.0)
        s.q_weight = 1.0 + _normal(gen, (d,), torch.float32, 0.1)
        s.k_weight = 1.0 + _normal(gen, (d,), torch.float32, 0.1)
        # places in a grid, axis by axis (a single axis: the index), each sequence from a start of its own
        h, w = (int(x) for x in c["grid"].split("x"))
        i = torch.arange(N, device="cuda") + torch.randint(0, 100000, (B, 1), generator=gen, device="cuda")
        places = [i // (h * w), i // w % h, i % w, i % 7][:len(_sections(c))] if len(_sections(c)) > 1 else [i]
        s.positions = torch.stack(places).to(torch.int32).contiguous()
        # each axis has its own run of frequencies, from 1 down to about 1 / base
        f, axis = [], []
        for a, n in enumerate(_sections(c)):
            f.append(ROPE_BASE ** (-torch.arange(n // 2, dtype=torch.float64) * 2 / n))
            axis += [a] * (n // 2)
        s.inv_freq, s.axis = torch.cat(f), torch.tensor(axis, dtype=torch.int32)
        empty = lambda *shape: torch.empty(shape, dtype=dt, device="cuda")  # noqa: E731
        if c["op"] == "axes":
            s.q, s.k, s.v = empty(B, H, N, d), empty(B, H_kv, N, d), empty(B, H_kv, N, d)
        else:
            s.dq, s.dk, s.dv = (_normal(gen, (B, n, N, d), dt) for n in (H, H_kv, H_kv))
            s.dqkv = torch.empty_like(s.qkv)
            s.dq_weight, s.dk_weight = torch.empty_like(s.q_weight), torch.empty_like(s.k_weight)
            s.workspace = None
        return s
    s.q = _normal(gen, (B, H, c["N_q"], d), bf)
    s.k, s.v = (_normal(gen, (c["B_kv"], H_kv, c["N_kv"], d), bf) for _ in range(2))
    s.lengths = torch.tensor(_lengths(c), dtype=torch.int32, device="cuda")
    s.o = torch.empty_like(s.q)
    s.lse = torch.empty(s.q.shape[:3], dtype=torch.float32, device="cuda")
    s.workspace = None
    if c["op"] == "cross_step":
        s.do = _normal(gen, s.q.shape, bf)
        s.dq, s.dk, s.dv = torch.empty_like(s.q), torch.empty_like(s.k), torch.empty_like(s.v)
    if c["op"] == "prefix":
        # what the requests' own tokens gave: outputs of some dozens of keys, their number and sum
        s.o_own = _normal(gen, s.q.shape, bf, 0.2)
        s.lse_own = 3.0 + 2.0 * torch.rand(s.lse.shape, generator=gen, device="cuda")
    return s


# ---------------------------------------------------------------- plain forms
def _axes_parts(s):
    """x (q and k heads) in float32, 1/rms, weights by head, and the pairs' cos and sin."""
    H, H_kv = s.c["H"], s.c["H_kv"]
    x = s.qkv[:, :, :H + H_kv].float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    w = torch.cat([s.q_weight.expand(H, -1), s.k_weight.expand(H_kv, -1)])
    place = s.positions[s.axis.long().cuda()].permute(1, 2, 0)  # [B, N, rot / 2]
    angle = place.double() * s.inv_freq.cuda()
    return x, r, w, angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]


def _rotate(x, cos, sin, interleaved):
    y, rot = x.clone(), 2 * cos.shape[-1]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        h = rot // 2
        a, b = x[..., :h], x[..., h:rot]
        y[..., :h], y[..., h:rot] = a * cos - b * sin, b * cos + a * sin
    return y


def _plain_axes(s):
    c = s.c
    x, r, w, cos, sin = _axes_parts(s)
    y = _rotate(x * r * w, cos, sin, c["interleaved"]).to(s.qkv.dtype).transpose(1, 2).contiguous()
    v = s.qkv[:, :, c["H"] + c["H_kv"]:].transpose(1, 2).contiguous()
    return {"q": y[:, :c["H"]], "k": y[:, c["H"]:], "v": v}


def _plain_axes_grad(s):
    c = s.c
    H = c["H"]
    x, r, w, cos, sin = _axes_parts(s)
    g = _rotate(torch.cat([s.dq, s.dk], 1).transpose(1, 2).float(), cos, -sin, c["interleaved"])
    n = x * r
    dw = (g * n).double().sum((0, 1))
    gw = g * w
    dx = r * (gw - n * (gw * n).mean(-1, keepdim=True))
    dqkv = torch.cat([dx.to(s.qkv.dtype), s.dv.transpose(1, 2)], 2)
    return {"dqkv": dqkv, "dq_weight": dw[:H].sum(0).float(), "dk_weight": dw[H:].sum(0).float()}


def _rows(s, x):
    """[B, H, N_q, ...] as [B_kv, H_kv, rows of that K/V head, ...]: batches, heads and queries."""
    c = s.c
    x = x.reshape(c["B_kv"], -1, c["H_kv"], c["H"] // c["H_kv"], *x.shape[2:])
    return x.transpose(1, 2).flatten(2, 4)


def _unrows(s, x):
    c = s.c
    x = x.unflatten(2, (c["B"] // c["B_kv"], c["H"] // c["H_kv"], c["N_q"]))
    return x.transpose(1, 2).reshape(c["B"], c["H"], *x.shape[4:])


def _probabilities(s):
    """softmax over the real keys [B_kv, H_kv, rows, N_kv], 0 where there are none, and its logsumexp."""
    c = s.c
    S = torch.matmul(_rows(s, s.q.float()), s.k.float().transpose(-1, -2)).mul_(1.0 / math.sqrt(c["d"]))
    hidden = torch.arange(c["N_kv"], device="cuda") >= s.lengths[:, None]
    S.masked_fill_(hidden[:, None, None], -math.inf)
    m = S.amax(-1, keepdim=True)
    S.sub_(m.clamp(min=torch.finfo(torch.float32).min)).exp_()
    total = S.sum(-1, keepdim=True)
    return S.div_(total.clamp(min=1.0)), m + total.log()


def _plain_cross(s):
    P, lse = _probabilities(s)
    o = torch.matmul(P, s.v.float())
    return {"o": _unrows(s, o).to(s.q.dtype), "lse": _unrows(s, lse)[..., 0]}


def _plain_prefix(s):
    P, lse = _probabilities(s)
    o, lse = _unrows(s, torch.matmul(P, s.v.float())), _unrows(s, lse)
    both = torch.logaddexp(lse, s.lse_own[..., None])
    o = (lse - both).exp() * o + (s.lse_own[..., None] - both).exp() * s.o_own.float()
    return {"o": o.to(s.q.dtype), "lse": both[..., 0]}


def _plain_cross_step(s):
    c, t = s.c, s.q.dtype
    scale = 1.0 / math.sqrt(c["d"])
    P, _ = _probabilities(s)
    k, v, do = s.k.float(), s.v.float(), _rows(s, s.do.float())
    o = torch.matmul(P, v)
    dv = torch.matmul(P.transpose(-1, -2), do)
    dS = torch.matmul(do, v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(P).mul_(scale)
    dq = torch.matmul(dS, k)
    dk = torch.matmul(dS.transpose(-1, -2), _rows(s, s.q.float()))
    return {"o": _unrows(s, o).to(t), "dq": _unrows(s, dq).to(t), "dk": dk.to(t), "dv": dv.to(t)}


# ---------------------------------------------------------------- one pass
def run(s):
    if own:
        return _own(s)
    return {"axes": _plain_axes, "axes_grad": _plain_axes_grad, "cross": _plain_cross,
            "cross_step": _plain_cross_step, "prefix": _plain_prefix}[s.c["op"]](s)


def _own(s):
    import exact_io_aware_06_gb300 as fa
    c, op = s.c, s.c["op"]
    if op == "axes":
        fa.fa_qk_norm_rope_axes(s.qkv, s.q_weight, s.k_weight, s.positions, s.inv_freq, s.axis, s.q, s.k, s.v, EPS,
                                c["interleaved"])
        return {"q": s.q, "k": s.k, "v": s.v}
    if s.workspace is None:  # kept with the state, as a program keeps it
        if op == "axes_grad":
            n = fa.fa_qk_norm_rope_bwd_workspace_size(c["B"], c["H"], c["H_kv"], c["N"], c["d"])
        else:
            sizes = [c[x] for x in ("B", "B_kv", "H", "H_kv", "N_q", "N_kv", "d")]
            n = (fa.fa_fwd_prefix_workspace_size if op == "prefix" else fa.fa_fwd_cross_workspace_size)(*sizes)
            if op == "cross_step":
                n = max(n, fa.fa_bwd_cross_workspace_size(*sizes))
        s.workspace = torch.empty(n, dtype=torch.uint8, device="cuda")
    if op == "axes_grad":
        fa.fa_qk_norm_rope_axes_bwd(s.qkv, s.q_weight, s.k_weight, s.positions, s.inv_freq, s.axis, s.dq, s.dk, s.dv,
                                    s.dqkv, s.dq_weight, s.dk_weight, s.workspace, EPS, c["interleaved"])
        return {"dqkv": s.dqkv, "dq_weight": s.dq_weight, "dk_weight": s.dk_weight}
    scale = 1.0 / math.sqrt(c["d"])
    if op == "prefix":
        fa.fa_fwd_prefix(s.q, s.k, s.v, s.lengths, s.o_own, s.lse_own, s.o, s.lse, s.workspace, scale)
        return {"o": s.o, "lse": s.lse}
    fa.fa_fwd_cross(s.q, s.k, s.v, s.lengths, s.o, s.lse, s.workspace, scale)
    if op == "cross":
        return {"o": s.o, "lse": s.lse}
    fa.fa_bwd_cross(s.q, s.k, s.v, s.lengths, s.o, s.lse, s.do, s.dq, s.dk, s.dv, s.workspace, scale)
    return {"o": s.o, "dq": s.dq, "dk": s.dk, "dv": s.dv}


# ---------------------------------------------------------------- definitions in 64 bits
def _exact_axes(s, c):
    """Each head: x / sqrt(mean(x^2) + eps) * w, its pairs turned as complex numbers."""
    rot = sum(_sections(c))
    half = rot // 2
    place = torch.arange(rot, device="cuda")
    place = place.view(half, 2) if c["interleaved"] else place.view(2, half).T
    pos = s.positions.double().cpu()
    turn = torch.stack([pos[a] * f for a, f in zip(s.axis.tolist(), s.inv_freq.tolist())], -1)
    turn = torch.polar(torch.ones_like(turn), turn).cuda()
    out, dqkv, dws = {}, [], {}
    first = 0
    for name, heads, w in (("q", c["H"], s.q_weight), ("k", c["H_kv"], s.k_weight)):
        x = s.qkv[:, :, first:first + heads].double()
        first += heads
        rms = (x.pow(2).sum(-1, keepdim=True) / c["d"] + EPS).sqrt()
        n = x / rms
        if c["op"] == "axes":
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
        dqkv.append((g - n * (torch.einsum("bnhe,bnhe->bnh", g, n) / c["d"])[..., None]) / rms)
    if c["op"] == "axes":
        out["v"] = s.qkv[:, :, first:].double().transpose(1, 2)
        return out
    dqkv.append(s.dv.double().transpose(1, 2))
    return {"dqkv": torch.cat(dqkv, 2), "dq_weight": dws["q"], "dk_weight": dws["k"]}


def _exact_attention(s, c):
    """Batch by batch, query head by query head, over the real keys alone, 2048 queries at a time."""
    G, share, T = c["H"] // c["H_kv"], c["B"] // c["B_kv"], 2048
    scale = 1.0 / math.sqrt(c["d"])
    grads = c["op"] == "cross_step"
    o = torch.zeros(s.q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s.lse.shape, -math.inf, dtype=torch.float64, device="cuda")
    if grads:
        dq = torch.zeros_like(o)
        dk, dv = (torch.zeros(s.k.shape, dtype=torch.float64, device="cuda") for _ in range(2))
    for b in range(c["B"]):
        n = _lengths(c)[b // share]
        if n == 0:
            continue
        k, v = s.k[b // share, :, :n].double(), s.v[b // share, :, :n].double()
        for r0 in range(0, c["N_q"], T):
            rows = slice(r0, min(c["N_q"], r0 + T))
            for kv in range(c["H_kv"]):
                h = slice(kv * G, kv * G + G)
                q = s.q[b, h, rows].double()
                A = scale * torch.einsum("gie,je->gij", q, k[kv])
                L = torch.logsumexp(A, -1)
                P = (A - L[..., None]).exp()
                o[b, h, rows], lse[b, h, rows] = P @ v[kv], L
                if grads:
                    do = s.do[b, h, rows].double()
                    dv[b // share, kv, :n] += torch.einsum("gij,gie->je", P, do)
                    dP = do @ v[kv].T
                    dA = scale * P * (dP - (P * dP).sum(-1, keepdim=True))
                    dq[b, h, rows] = dA @ k[kv]
                    dk[b // share, kv, :n] += torch.einsum("gij,gie->je", dA, q)
    if grads:
        return {"o": o, "dq": dq, "dk": dk, "dv": dv}
    if c["op"] == "prefix":
        own_lse = s.lse_own.double()
        top = torch.maximum(lse, own_lse)
        a, b = (lse - top).exp(), (own_lse - top).exp()
        o = (a[..., None] * o + b[..., None] * s.o_own.double()) / (a + b)[..., None]
        lse = top + (a + b).log()
    return {"o": o, "lse": lse}


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] in ("axes", "axes_grad"):
        return _exact_axes(s, c)
    pairs = c["B"] * c["H"] * c["N_q"] * c["N_kv"]
    loops = c["B"] * c["H_kv"] * -(-c["N_q"] // 2048)
    if pairs * c["d"] > 3e11 or loops > 20000:
        return None
    return _exact_attention(s, c)
