"""Attention under a causal sliding window with sinks, forward and backward, against float64.

Forward tolerance, with w the softmax weights and A = sum w |v|: P is rounded to bfloat16 (2^-8
of each weight; the row sum is not, so o moves by at most 2^-8 A), o is rounded (2^-8 |o|), and
float32 scores and sums add under 1e-5 (1 + max |score|) of A.  lse: 1e-5 (1 + max |score|).

Backward tolerance, with t = 1e-5 (1 + max |score|) for the recomputed P: dV takes P in bfloat16
(2^-8 P^T |dO|); dS = P (dP - delta) is rounded to bfloat16 (2^-8), and delta = dO . o takes the o that
the forward rounded: its error is |dO| . (o's tolerance).  (Where few keys are seen it is the sum of
P dP in float32 instead: t + 1e-6 of |dO| . A.)  Each gradient adds its own rounding, 2^-8 of the value.
Group sums add up."""
import numpy as np
import pytest
import torch

import exact_io_aware_06_gb300 as fa
import plain64
from gpu_util import check_status, ensure_built, f64, scale_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def rand(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(shape, generator=g)).to(torch.bfloat16).cuda()


def inputs(B, H, H_kv, N, d, seed=0):
    return (rand((B, H, N, d), seed), rand((B, H_kv, N, d), seed + 1), rand((B, H_kv, N, d), seed + 2),
            rand((B, H, N, d), seed + 3))


def forward(q, k, v, scale, window, n_sink):
    o = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:3], float("nan"), device="cuda")
    fa.fa_fwd_window(q, k, v, o, lse, scale, window, n_sink)
    check_status()
    return o, lse


def check_forward(q, k, v, o, lse, scale, window, n_sink, heads=None):
    B, H, N, d = q.shape
    seen = plain64.window_mask(N, N, 0, window, n_sink)
    q, k, v, o, lse = (f64(t) for t in (q, k, v, o, lse))
    for b in range(B):
        for h in range(H) if heads is None else heads:
            kv = h // (H // k.shape[1])
            ref, ref_lse, P = plain64.attention(q[b, h], k[b, kv], v[b, kv], scale, seen)
            A = P @ np.abs(v[b, kv])
            top = 1e-5 * (1 + np.abs(scale) * np.abs(q[b, h] @ k[b, kv].T).max(-1))
            tol = 2.0 ** -8 * (A + np.abs(ref)) + top[:, None] * A
            err = np.abs(o[b, h] - ref)
            assert np.isfinite(o[b, h]).all() and (err <= tol).all(), (b, h, float((err / tol).max()))
            dl = np.abs(lse[b, h] - ref_lse)
            assert (dl <= top).all(), (b, h, float((dl / top).max()))


WINDOWS = [(1, 0), (1, 1), (2, 4), (7, 0), (64, 4), (127, 1), (128, 0), (128, 32), (129, 33), (200, 4), (256, 130),
           (300, 4), (5000, 0), (2 ** 31 - 1, 7), (40, 2 ** 31 - 1)]


@pytest.mark.parametrize("window,n_sink", WINDOWS)
@pytest.mark.parametrize("d", [64, 128])
def test_forward_windows(window, n_sink, d):
    q, k, v, _ = inputs(1, 2, 1, 700, d)
    o, lse = forward(q, k, v, scale_for(d), window, n_sink)
    check_forward(q, k, v, o, lse, scale_for(d), window, n_sink)


@pytest.mark.parametrize("N", [1, 2, 31, 127, 128, 129, 255, 256, 257, 384, 385, 513])
@pytest.mark.parametrize("window,n_sink", [(100, 4), (130, 0), (33, 40)])
def test_forward_lengths(N, window, n_sink):
    q, k, v, _ = inputs(2, 3, 1, N, 64, seed=N)
    o, lse = forward(q, k, v, 0.125, window, n_sink)
    check_forward(q, k, v, o, lse, 0.125, window, n_sink)


@pytest.mark.parametrize("H,H_kv", [(1, 1), (6, 3), (8, 2), (7, 1)])
def test_forward_heads_many_items(H, H_kv):
    # more items than SMs: every CTA carries its barriers from item to item
    q, k, v, _ = inputs(16, H, H_kv, 1500, 64, seed=7)
    o, lse = forward(q, k, v, 0.125, 150, 4)
    check_forward(q[::5], k[::5], v[::5], o[::5], lse[::5], 0.125, 150, 4)


@pytest.mark.parametrize("scale", [0.0, -0.125, 2.0])
def test_forward_scales(scale):
    q, k, v, _ = inputs(1, 2, 2, 400, 64, seed=3)
    o, lse = forward(q, k, v, scale, 150, 3)
    check_forward(q, k, v, o, lse, scale, 150, 3)


def test_forward_growing_scores():
    N, d = 600, 64
    unit = rand((d,), 3).float()
    k = (torch.arange(N, device="cuda")[:, None] / 40 * unit).to(torch.bfloat16)[None, None].contiguous()
    q = unit.to(torch.bfloat16).expand(1, 1, N, d).contiguous()
    v = rand((1, 1, N, d), 4)
    o, lse = forward(q, k, v, 0.125, 200, 20)
    check_forward(q, k, v, o, lse, 0.125, 200, 20)


def test_forward_is_causal_attention_when_the_window_covers_everything():
    q, k, v, _ = inputs(1, 4, 2, 1100, 128, seed=5)
    o, lse = forward(q, k, v, scale_for(128), 1100, 0)
    o2, lse2 = fa.attention_forward(q, k, v, causal=True)
    # the same arithmetic per row up to the order of blocks: both within the forward's bound
    check_forward(q, k, v, o2, lse2, scale_for(128), 1100, 0)
    assert (f64(lse) - f64(lse2)).max() < 1e-5


def test_forward_repeats_bit_for_bit_and_without_lse():
    q, k, v, _ = inputs(3, 8, 2, 2000, 128, seed=9)
    o, lse = forward(q, k, v, scale_for(128), 333, 4)
    o2 = torch.empty_like(q)
    fa.fa_fwd_window(q, k, v, o2, None, scale_for(128), 333, 4)
    assert torch.equal(o, o2)


def test_forward_large_offsets():
    # K/V beyond 2^31 bytes from the base
    B, H, N, d = 70, 8, 16384, 128
    q = torch.zeros((B, H, N, d), dtype=torch.bfloat16, device="cuda")
    k, v = torch.zeros_like(q), torch.zeros_like(q)
    small = inputs(1, 1, 1, N, d, seed=11)
    q[-1, -1], k[-1, -1], v[-1, -1] = (t[0, 0] for t in small[:3])
    o, lse = forward(q, k, v, scale_for(d), 200, 4)
    o1, lse1 = forward(*small[:3], scale_for(d), 200, 4)
    assert torch.equal(o[-1, -1], o1[0, 0]) and torch.equal(lse[-1, -1], lse1[0, 0])
    assert (o[0] == 0).all()


def test_forward_short_wait_limit_reports_and_recovers():
    q, k, v, _ = inputs(4, 16, 16, 2048, 128, seed=13)
    o, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    try:
        fa.fa_set_wait_timeout_ns(300)
        for _ in range(3):
            fa.fa_fwd_window(q, k, v, o, lse, scale_for(128), 500, 4)
            assert fa.fa_last_device_error() in (fa.FA_OK, fa.FA_ERR_DEVICE_TIMEOUT)
    finally:
        fa.fa_set_wait_timeout_ns(0)
    o, lse = forward(q, k, v, scale_for(128), 500, 4)
    check_forward(q[:1], k[:1], v[:1], o[:1], lse[:1], scale_for(128), 500, 4, heads=[0, 15])


# ---------------------------------------------------------------- backward
def backward(q, k, v, o, lse, do, scale, window, n_sink, ws=None):
    B, H, N, d = q.shape
    out = [torch.full_like(t, float("nan")) for t in (q, k, v)]
    if ws is None:
        n = fa.fa_bwd_window_workspace_size(B, H, k.shape[1], N, d, window, n_sink)
        ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    fa.fa_bwd_window(q, k, v, o, lse, do, *out, ws, scale, window, n_sink)
    check_status()
    return out


def check_backward(q, k, v, do, grads, scale, window, n_sink, kv_heads=None, few_keys=False):
    B, H, N, d = q.shape
    H_kv = k.shape[1]
    G = H // H_kv
    seen = plain64.window_mask(N, N, 0, window, n_sink)
    q, k, v, do = (f64(t) for t in (q, k, v, do))
    got = [f64(t) for t in grads]
    assert all(np.isfinite(g).all() for g in got)
    a = abs(scale)
    for b in range(B):
        for kv in range(H_kv) if kv_heads is None else kv_heads:
            K, V = k[b, kv], v[b, kv]
            aK, aV = np.abs(K), np.abs(V)
            ref_dk, ref_dv, tol_dk, tol_dv = (np.zeros((N, d)) for _ in range(4))
            for h in range(kv * G, kv * G + G):
                Q, dO = q[b, h], do[b, h]
                aQ, adO = np.abs(Q), np.abs(dO)
                o, _, P = plain64.attention(Q, K, V, scale, seen)
                t = 1e-5 * (1 + np.where(seen, a * np.abs(Q @ K.T), 0).max(-1, keepdims=True))
                dP = dO @ V.T
                diff = dP - (dO * o).sum(-1, keepdims=True)
                A = P @ aV
                o_tol = (t + 1e-6) * A if few_keys else 2.0 ** -8 * (A + np.abs(o)) + t * A
                d_delta = (adO * o_tol).sum(-1, keepdims=True)
                e_dS = (2.0 ** -8 + t) * np.abs(P * diff) + P * d_delta + 1e-6 * P * (adO @ aV.T)
                dS = P * diff
                rq, tq = scale * dS @ K, a * e_dS @ aK
                err = np.abs(got[0][b, h] - rq)
                tq += 2.0 ** -8 * np.abs(rq) + 1e-6 * a * np.abs(dS) @ aK + 1e-37
                assert (err <= tq).all(), ("dq", b, h, float((err / tq).max()))
                ref_dk += scale * dS.T @ Q
                ref_dv += P.T @ dO
                tol_dk += a * e_dS.T @ aQ + 1e-6 * a * np.abs(dS).T @ aQ
                tol_dv += (2.0 ** -8 * P + P * t + 1e-6 * P).T @ adO
            for name, g, r, tol in (("dk", got[1], ref_dk, tol_dk), ("dv", got[2], ref_dv, tol_dv)):
                tol = tol + 2.0 ** -8 * np.abs(r) + 1e-37
                err = np.abs(g[b, kv] - r)
                assert (err <= tol).all(), (name, b, kv, float((err / tol).max()))


def step(B, H, H_kv, N, d, window, n_sink, scale=None, seed=0, kv_heads=None):
    q, k, v, do = inputs(B, H, H_kv, N, d, seed)
    scale = scale_for(d) if scale is None else scale
    o, lse = forward(q, k, v, scale, window, n_sink)
    grads = backward(q, k, v, o, lse, do, scale, window, n_sink)
    check_backward(q, k, v, do, grads, scale, window, n_sink, kv_heads)
    return (q, k, v, o, lse, do), grads


@pytest.mark.parametrize("window,n_sink", WINDOWS)
@pytest.mark.parametrize("d", [64, 128])
def test_backward_windows(window, n_sink, d):
    step(1, 2, 1, 700, d, window, n_sink)


@pytest.mark.parametrize("N", [1, 2, 127, 128, 129, 256, 385, 513])
@pytest.mark.parametrize("d", [64, 128])
def test_backward_lengths(N, d):
    step(2, 3, 1, N, d, 100, 4, seed=N)
    step(2, 2, 2, N, d, 33, 40, seed=N)


@pytest.mark.parametrize("H,H_kv,d", [(6, 3, 64), (8, 1, 64), (8, 2, 128), (3, 3, 128)])
def test_backward_heads_many_items_and_pieces(H, H_kv, d):
    # more items than SMs; sinks in two blocks, whose later query blocks are dealt in pieces
    step(9, H, H_kv, 1700, d, 150, 140, kv_heads=[0])


@pytest.mark.parametrize("d", [64, 128])
def test_backward_long_with_few_heads(d):
    # one K/V head: the sink block's later query blocks in many pieces, the last one short
    step(1, 2, 1, 5000, d, 130, 4)


@pytest.mark.parametrize("scale", [0.0, -0.125, 1.0])
def test_backward_scales(scale):
    step(1, 2, 2, 400, 64, 150, 3, scale=scale)
    step(1, 2, 2, 400, 128, 150, 3, scale=scale)


def test_backward_is_causal_backward_when_the_window_covers_everything():
    (q, k, v, o, lse, do), grads = step(1, 4, 2, 900, 128, 900, 0, seed=5)
    o2, lse2 = fa.attention_forward(q, k, v, causal=True)
    grads2 = fa.attention_backward(q, k, v, o2, lse2, do, causal=True)
    for g, r in zip(grads, grads2):
        assert np.abs(f64(g) - f64(r)).max() <= 5e-2


@pytest.mark.parametrize("d", [64, 128])
def test_backward_repeats_on_a_used_workspace(d):
    (q, k, v, o, lse, do), grads = step(2, 4, 2, 1500, d, 200, 4, seed=9)
    n = fa.fa_bwd_window_workspace_size(2, 4, 2, 1500, d, 200, 4)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        again = backward(q, k, v, o, lse, do, scale_for(d), 200, 4, ws)
        assert all(torch.equal(a, g) for a, g in zip(again, grads))


def test_training_step_in_a_graph():
    # forward and backward captured together, replayed on new inputs in the same buffers
    B, H, H_kv, N, d, window, n_sink = 2, 4, 2, 600, 64, 130, 4
    q, k, v, do = inputs(B, H, H_kv, N, d)
    o, lse = torch.empty_like(q), torch.empty((B, H, N), device="cuda")
    out = [torch.empty_like(t) for t in (q, k, v)]
    ws = torch.empty(fa.fa_bwd_window_workspace_size(B, H, H_kv, N, d, window, n_sink), dtype=torch.uint8, device="cuda")
    fa.fa_fwd_window(q, k, v, o, lse, 0.125, window, n_sink)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fa_fwd_window(q, k, v, o, lse, 0.125, window, n_sink)
        fa.fa_bwd_window(q, k, v, o, lse, do, *out, ws, 0.125, window, n_sink)
    for seed in (20, 30):
        for t, new in zip((q, k, v, do), inputs(B, H, H_kv, N, d, seed)):
            t.copy_(new)
        graph.replay()
        check_status()
        check_forward(q, k, v, o, lse, 0.125, window, n_sink)
        check_backward(q, k, v, do, out, 0.125, window, n_sink)


def test_backward_short_wait_limit_reports_and_recovers():
    for d in (64, 128):
        q, k, v, do = inputs(2, 16, 16, 2048, d, seed=13)
        o, lse = forward(q, k, v, scale_for(d), 500, 4)
        out = [torch.empty_like(t) for t in (q, k, v)]
        ws = torch.empty(fa.fa_bwd_window_workspace_size(2, 16, 16, 2048, d, 500, 4), dtype=torch.uint8, device="cuda")
        try:
            fa.fa_set_wait_timeout_ns(300)
            for _ in range(3):
                fa.fa_bwd_window(q, k, v, o, lse, do, *out, ws, scale_for(d), 500, 4)
                assert fa.fa_last_device_error() in (fa.FA_OK, fa.FA_ERR_DEVICE_TIMEOUT)
        finally:
            fa.fa_set_wait_timeout_ns(0)
        grads = backward(q, k, v, o, lse, do, scale_for(d), 500, 4, ws)
        check_backward(q[:1], k[:1], v[:1], do[:1], [g[:1] for g in grads], scale_for(d), 500, 4, kv_heads=[0, 15])


def test_backward_large_offsets():
    # operands and gradients beyond 2^31 bytes from the base; without sinks no block is dealt in
    # parts, so that a head's bits do not depend on its neighbours
    B, H, N, d = 70, 8, 16384, 128
    small = inputs(1, 1, 1, N, d, seed=17)
    big = [torch.zeros((B, H, N, d), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    for t, x in zip(big, small):
        t[-1, -1] = x[0, 0]
    outs = []
    for q, k, v, do in (big, small):
        o, lse = forward(q, k, v, scale_for(d), 200, 0)
        outs.append(backward(q, k, v, o, lse, do, scale_for(d), 200, 0))
    for b, s in zip(*outs):
        assert torch.equal(b[-1, -1], s[0, 0]) and (b[0] == 0).all()


@pytest.mark.parametrize("H,H_kv,N,window,n_sink", [(4, 2, 300, 1, 0), (4, 2, 300, 2, 0), (3, 1, 389, 20, 4), (2, 2, 257, 24, 0),
                                                    (4, 4, 200, 3, 17), (2, 1, 100, 5000, 0), (2, 2, 128, 60, 4), (1, 1, 1, 1, 0)])
@pytest.mark.parametrize("d", [64, 128])
def test_backward_delta_of_few_keys(H, H_kv, N, window, n_sink, d):
    # without the share of o's rounding
    q, k, v, do = inputs(2, H, H_kv, N, d, seed=23)
    o, lse = forward(q, k, v, scale_for(d), window, n_sink)
    grads = backward(q, k, v, o, lse, do, scale_for(d), window, n_sink)
    check_backward(q, k, v, do, grads, scale_for(d), window, n_sink, few_keys=True)


@pytest.mark.parametrize("H,H_kv,N,d", [(4, 2, 1100, 128), (3, 3, 517, 64)])
def test_forward_and_the_causal_forward_where_the_window_covers_everything(H, H_kv, N, d):
    # o and lse of both calls against the same float64 form, on both sides
    q, k, v, _ = inputs(2, H, H_kv, N, d, seed=5)
    check_forward(q, k, v, *fa.attention_forward(q, k, v, causal=True), scale_for(d), N, 0)
    for window, n_sink in ((N, 0), (N + 5000, 3), (2 ** 31 - 1, 0), (1, N)):
        check_forward(q, k, v, *forward(q, k, v, scale_for(d), window, n_sink), scale_for(d), N, 0)


def until_a_wait_runs_out(call, results, ref):
    """Calls under wait limits far below a load's latency, until one reports that a wait ran out; those
    that report nothing have to be right, and so has the first one under the default limit."""
    elsewhere = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    reported = False
    try:
        for limit_ns in (300, 1, 1, 1, 1, 1, 1, 1):
            fa.fa_set_wait_timeout_ns(limit_ns)
            for t in results:
                t.fill_(float("nan"))
            elsewhere.zero_()  # the inputs leave L2: the first loads take longest
            call()
            status = fa.fa_last_device_error()
            reported = status == fa.FA_ERR_DEVICE_TIMEOUT
            if reported:
                break
            assert status == fa.FA_OK and all(torch.equal(a, b) for a, b in zip(results, ref))
    finally:
        fa.fa_set_wait_timeout_ns(0)
    assert reported
    call()
    check_status()
    assert all(torch.equal(a, b) for a, b in zip(results, ref))


@pytest.mark.parametrize("d", [64, 128])
def test_a_wait_that_runs_out_is_reported(d):
    B, H, N, window, n_sink = 2, 16, 2048, 500, 4
    q, k, v, do = inputs(B, H, H, N, d, seed=13)
    o, lse = forward(q, k, v, scale_for(d), window, n_sink)
    check_forward(q[:1], k[:1], v[:1], o[:1], lse[:1], scale_for(d), window, n_sink, heads=[0, 15])
    out = [torch.empty_like(q), torch.empty_like(lse)]
    until_a_wait_runs_out(lambda: fa.fa_fwd_window(q, k, v, *out, scale_for(d), window, n_sink), out, (o, lse))

    ws = torch.empty(fa.fa_bwd_window_workspace_size(B, H, H, N, d, window, n_sink), dtype=torch.uint8, device="cuda")
    ref = backward(q, k, v, o, lse, do, scale_for(d), window, n_sink, ws)
    check_backward(q[:1], k[:1], v[:1], do[:1], [g[:1] for g in ref], scale_for(d), window, n_sink, kv_heads=[0, 15])
    out = [torch.empty_like(t) for t in ref]
    until_a_wait_runs_out(lambda: fa.fa_bwd_window(q, k, v, o, lse, do, *out, ws, scale_for(d), window, n_sink), out, ref)
