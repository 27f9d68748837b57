"""Attention to another sequence's keys: cross attention and shared prefixes, against float64.

Forward tolerance, as in the windowed tests, with w the softmax weights and A = sum w |v|: P is
rounded to bfloat16 (2^-8 of each weight; the row sum is not, so o moves by at most 2^-8 A), o is rounded
(2^-8 |o|), and float32 scores and sums add under t = 1e-5 (1 + max |score|) of A.  lse: t.  Merging with
own attention: the two weights are off by at most t + 2^-22 (1 + |lse_own|) each, relative, which moves o
by twice that of (A + |o_own|) at most.

Backward tolerance: dV takes P in bfloat16 (2^-8 P^T |dO|); dS = P (dP - delta) is rounded to bfloat16
(2^-8), and delta = dO . o takes the o that the forward rounded: its error is |dO| . (o's tolerance).
(Where few keys are seen it is the sum of P dP in float32 instead: t + 1e-6 of |dO| . A.)  Each gradient
adds its own rounding, 2^-8 of the value.  Sums over heads and batches that share keys add up."""
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


def inputs(B, B_kv, H, H_kv, N_q, N_kv, d, seed=0):
    return (rand((B, H, N_q, d), seed), rand((B_kv, H_kv, N_kv, d), seed + 1), rand((B_kv, H_kv, N_kv, d), seed + 2),
            rand((B, H, N_q, d), seed + 3))


def sizes(q, k):
    return q.shape[0], k.shape[0], q.shape[1], k.shape[1], q.shape[2], k.shape[2], q.shape[3]


def space(nbytes):
    return torch.full((max(16, nbytes),), 255, dtype=torch.uint8, device="cuda")


def on_device(lengths):
    return None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")


def forward(q, k, v, lengths, scale, ws=None):
    o = torch.full_like(q, float("nan"))
    lse = torch.full(q.shape[:3], float("nan"), device="cuda")
    ws = space(fa.fa_fwd_cross_workspace_size(*sizes(q, k))) if ws is None else ws
    fa.fa_fwd_cross(q, k, v, on_device(lengths), o, lse, ws, scale)
    check_status()
    return o, lse


def head_reference(q, k, v, n, scale):
    """o, lse, A and t of one head's queries over the first n keys."""
    seen = np.ones((len(q), n), dtype=bool)
    ref, lse, P = plain64.attention(q, k[:n], v[:n], scale, seen)
    top = np.abs(scale) * np.abs(q @ k[:n].T).max(-1) if n else np.zeros(len(q))
    return ref, lse, P @ np.abs(v[:n]), 1e-5 * (1 + top)


def each_head(q, k, lengths, batches=None):
    share, G = q.shape[0] // k.shape[0], q.shape[1] // k.shape[1]
    for b in range(q.shape[0]) if batches is None else batches:
        n = k.shape[2] if lengths is None else min(max(lengths[b // share], 0), k.shape[2])
        for h in range(q.shape[1]):
            yield b, h, b // share, h // G, n


def check_forward(q, k, v, lengths, o, lse, scale, batches=None, own=None):
    heads = list(each_head(q, k, lengths, batches))
    q, k, v, o, lse = (f64(t) for t in (q, k, v, o, lse))
    if own is not None:
        own = [f64(t) for t in own]
    for b, h, kb, kh, n in heads:
        ref, ref_lse, A, t = head_reference(q[b, h], k[kb, kh], v[kb, kh], n, scale)
        extra = 0.0
        if own is not None:
            o2, l2 = own[0][b, h], own[1][b, h]
            both = np.logaddexp(ref_lse, l2)
            w, w2 = (np.exp(x - np.where(np.isfinite(both), both, 0))[:, None] for x in (ref_lse, l2))
            t = t + 2.0 ** -22 * (1 + np.abs(np.where(np.isfinite(l2), l2, 0)))
            A, ref, ref_lse = w * A, w * ref + w2 * np.where(w2 > 0, o2, 0), both
            extra = 2 * t[:, None] * (A + w2 * np.abs(np.where(w2 > 0, o2, 0)))
        tol = 2.0 ** -8 * (A + np.abs(ref)) + t[:, None] * A + extra
        err = np.abs(o[b, h] - ref)
        assert np.isfinite(o[b, h]).all() and (err <= tol).all(), (b, h, float((err / np.maximum(tol, 1e-30)).max()))
        empty = ref_lse == -np.inf
        assert (lse[b, h][empty] == -np.inf).all()
        dl = np.abs(lse[b, h][~empty] - ref_lse[~empty])
        assert (dl <= t[~empty]).all(), (b, h, float((dl / t[~empty]).max(initial=0)))


@pytest.mark.parametrize("N_q", [1, 2, 127, 128, 129, 256, 257, 400])
@pytest.mark.parametrize("N_kv", [1, 5, 128, 129, 300])
@pytest.mark.parametrize("d", [64, 128])
def test_forward_lengths(N_q, N_kv, d):
    q, k, v, _ = inputs(2, 2, 3, 1, N_q, N_kv, d, seed=N_q)
    o, lse = forward(q, k, v, None, scale_for(d))
    check_forward(q, k, v, None, o, lse, scale_for(d))


@pytest.mark.parametrize("lengths", [[0, 0, 0], [1, 128, 127], [300, 0, 129], [-7, 256, 10 ** 9], [257, 255, 1]])
@pytest.mark.parametrize("N_q,H,H_kv", [(1, 2, 2), (1, 8, 2), (3, 6, 2), (130, 4, 2), (300, 2, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_forward_ragged_keys(lengths, N_q, H, H_kv, d):
    q, k, v, _ = inputs(3, 3, H, H_kv, N_q, 300, d, seed=1)
    # what lies behind a sequence's end is never used
    for b, n in enumerate(lengths):
        k[b, :, max(n, 0):], v[b, :, max(n, 0):] = float("nan"), float("inf")
    o, lse = forward(q, k, v, lengths, scale_for(d))
    check_forward(q, k, v, lengths, o, lse, scale_for(d))


@pytest.mark.parametrize("B,B_kv,H,H_kv,N_q", [(1, 1, 1, 1, 1), (4, 1, 2, 2, 1), (6, 2, 8, 2, 1), (150, 1, 4, 4, 1),
                                               (70, 2, 4, 1, 2), (5, 1, 3, 1, 20), (6, 3, 2, 1, 33), (4, 2, 2, 1, 70),
                                               (130, 1, 1, 1, 1), (129, 1, 2, 1, 32), (9, 3, 6, 2, 21)])
@pytest.mark.parametrize("d", [64, 128])
def test_forward_batches_that_share_keys(B, B_kv, H, H_kv, N_q, d):
    lengths = [333, 200, 64][:B_kv]
    q, k, v, _ = inputs(B, B_kv, H, H_kv, N_q, 333, d, seed=B)
    o, lse = forward(q, k, v, lengths, scale_for(d))
    check_forward(q, k, v, lengths, o, lse, scale_for(d))


@pytest.mark.parametrize("B,H,N_q,N_kv", [(1, 1, 1, 9000), (1, 2, 300, 5000), (3, 1, 1, 4100), (2, 16, 700, 500)])
def test_forward_long_keys_divided_over_the_sms(B, H, N_q, N_kv):
    q, k, v, _ = inputs(B, B, H, H, N_q, N_kv, 128, seed=5)
    lengths = [N_kv, N_kv // 3, 130][:B]
    o, lse = forward(q, k, v, lengths, scale_for(128))
    check_forward(q, k, v, lengths, o, lse, scale_for(128))


def test_forward_of_many_sequences():
    # more than a warp's worth of lengths, most of them short; and more items than the work is cut for
    for B, H, N_q in ((100, 2, 1), (700, 2, 5)):
        g = np.random.default_rng(B)
        lengths = [int(x) for x in np.where(g.random(B) < 0.1, g.integers(200, 400, B), g.integers(0, 20, B))]
        q, k, v, _ = inputs(B, B, H, H, N_q, 400, 64, seed=B)
        o, lse = forward(q, k, v, lengths, 0.125)
        check_forward(q, k, v, lengths, o, lse, 0.125, batches=range(0, B, 7))


def test_forward_of_many_items():
    # whole items: every CTA carries its barriers from one to the next
    q, k, v, _ = inputs(8, 8, 16, 8, 2400, 200, 64, seed=7)
    lengths = [200, 1, 128, 0, 77, 199, 150, 20]
    o, lse = forward(q, k, v, lengths, 0.125)
    check_forward(q[:5], k[:5], v[:5], lengths[:5], o[:5], lse[:5], 0.125, batches=range(1, 5))


@pytest.mark.parametrize("B,H,N_q,N_kv", [(1, 8, 1, 1000), (1, 15, 130, 1100), (1, 16, 1, 700), (2, 16, 2, 600), (3, 12, 300, 300),
                                          (1, 40, 1, 400), (1, 76, 1, 256), (1, 77, 1, 256)])
@pytest.mark.parametrize("d", [64, 128])
def test_forward_of_few_items(B, H, N_q, N_kv, d):
    # an item on the CTAs of a cluster, which has more of them than the shortest sequences have blocks
    q, k, v, _ = inputs(B, B, H, H, N_q, N_kv, d, seed=H)
    for lengths in ([N_kv] * B, [130, 1, 0][:B], [N_kv // 2 + 3, N_kv - 1, 257][:B]):
        o, lse = forward(q, k, v, lengths, scale_for(d))
        check_forward(q, k, v, lengths, o, lse, scale_for(d))


@pytest.mark.parametrize("B,H,N_q,N_kv", [(5, 40, 130, 300), (32, 8, 129, 200), (33, 8, 129, 200), (2, 80, 256, 128)])
@pytest.mark.parametrize("d", [64, 128])
def test_forward_of_many_items_of_ragged_sequences(B, H, N_q, N_kv, d):
    # whole items, more than CTAs: of up to 32 sequences the longest first, some of the same length, some empty
    lengths = [(37 * b * b + 11 * b) % (N_kv + 1) if b % 7 else N_kv * (b % 2) for b in range(B)]
    assert fa.fa_fwd_cross_workspace_size(B, B, H, H, N_q, N_kv, d) == 0
    q, k, v, _ = inputs(B, B, H, H, N_q, N_kv, d, seed=B)
    for b, n in enumerate(lengths):
        k[b, :, n:], v[b, :, n:] = float("nan"), float("inf")
    o, lse = forward(q, k, v, lengths, scale_for(d))
    check_forward(q, k, v, lengths, o, lse, scale_for(d), batches=range(0, B, max(1, B // 5)))


@pytest.mark.parametrize("B,B_kv,H,H_kv,N_q", [(3, 3, 2, 2, 1), (3, 3, 4, 2, 1), (3, 3, 2, 2, 2), (3, 3, 3, 1, 1), (3, 3, 2, 2, 4),
                                                (6, 3, 2, 2, 1), (12, 3, 1, 1, 1), (6, 3, 2, 1, 1), (60, 60, 16, 16, 1)])
@pytest.mark.parametrize("N_kv", [1, 40, 128, 129, 700, 3000])
@pytest.mark.parametrize("d", [64, 128])
def test_forward_of_few_rows(B, B_kv, H, H_kv, N_q, N_kv, d):
    # of one batch, of heads that share keys, of batches that share keys; CTAs of a cluster without keys
    q, k, v, _ = inputs(B, B_kv, H, H_kv, N_q, N_kv, d, seed=N_kv)
    for lengths in (None, ([N_kv, 0, (N_kv + 1) // 2] * 20)[:B_kv], ([7, N_kv - 1, N_kv + 9] * 20)[:B_kv]):
        if lengths is not None:
            for b, n in enumerate(lengths):
                k[b, :, n:], v[b, :, n:] = float("inf"), float("nan")
        o, lse = forward(q, k, v, lengths, scale_for(d))
        check_forward(q, k, v, lengths, o, lse, scale_for(d), batches=range(0, B, max(1, B // 9)))
        again = forward(q, k, v, lengths, scale_for(d))
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
        k, v = (torch.nan_to_num(x, nan=0.5, posinf=-0.5) for x in (k, v))


@pytest.mark.parametrize("N_q,H,H_kv", [(7, 2, 2), (200, 2, 1), (130, 24, 24)])
@pytest.mark.parametrize("d", [64, 128])
def test_forward_ends_of_few_keys(N_q, H, H_kv, d):
    # the last block's keys around 32 and 64, behind none, one and two whole blocks; of lone tiles and of pairs, cut or not
    lengths = [31, 32, 33, 63, 64, 65, 1, 159, 160, 161, 191, 192, 193, 257, 288, 289, 320, 321]
    q, k, v, _ = inputs(18, 18, H, H_kv, N_q, 330, d, seed=18)
    for b, n in enumerate(lengths):
        k[b, :, n:], v[b, :, n:] = float("-inf"), float("nan")
    o, lse = forward(q, k, v, lengths, scale_for(d))
    check_forward(q, k, v, lengths, o, lse, scale_for(d), batches=range(18) if H < 24 else range(0, 18, 2))
    for n in (32, 64, 65, 160, 192):  # and of all the keys there are
        x, y = k[-1:, :, :n].contiguous(), v[-1:, :, :n].contiguous()
        o, lse = forward(q[-1:], x, y, None, -0.2)
        check_forward(q[-1:], x, y, None, o, lse, -0.2)


@pytest.mark.parametrize("scale", [0.0, -0.125, 2.0])
@pytest.mark.parametrize("N_q", [1, 200])
def test_forward_scales(scale, N_q):
    q, k, v, _ = inputs(2, 2, 2, 2, N_q, 400, 64, seed=3)
    o, lse = forward(q, k, v, [400, 250], scale)
    check_forward(q, k, v, [400, 250], o, lse, scale)


@pytest.mark.parametrize("N_q", [1, 150])
def test_forward_growing_scores(N_q):
    N, d = 1500, 64
    unit = rand((d,), 3).float()
    k = (torch.arange(N, device="cuda")[:, None] / 60 * unit).to(torch.bfloat16)[None, None].contiguous()
    q = unit.to(torch.bfloat16).expand(1, 1, N_q, d).contiguous()
    v = rand((1, 1, N, d), 4)
    o, lse = forward(q, k, v, None, 0.125)
    check_forward(q, k, v, None, o, lse, 0.125)


def test_forward_of_nan_queries_and_keys():
    q, k, v, _ = inputs(1, 1, 2, 2, 5, 200, 64, seed=8)
    q[0, 0, 3] = float("nan")
    k[0, 1, 150, 7] = float("nan")
    o, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    fa.fa_fwd_cross(q, k, v, None, o, lse, space(fa.fa_fwd_cross_workspace_size(*sizes(q, k))), 0.125)
    check_status()
    bad = torch.isnan(o).all(-1)
    assert bad[0, 0].tolist() == [False, False, False, True, False] and bad[0, 1].all()
    assert torch.equal(torch.isnan(lse), bad)


@pytest.mark.parametrize("N_q,share", [(1, 1), (1, 3), (600, 1)])
def test_forward_repeats_bit_for_bit_and_without_lse(N_q, share):
    q, k, v, _ = inputs(3 * share, 3, 8, 2, N_q, 2000, 128, seed=9)
    lengths = [2000, 77, 1300]
    o, lse = forward(q, k, v, lengths, scale_for(128))
    o2 = torch.empty_like(q)
    ws = space(fa.fa_fwd_cross_workspace_size(*sizes(q, k)))
    fa.fa_fwd_cross(q, k, v, on_device(lengths), o2, None, ws, scale_for(128))
    check_status()
    assert torch.equal(o, o2)


def test_forward_without_workspace_where_none_is_needed():
    assert fa.fa_fwd_cross_workspace_size(8, 8, 16, 16, 2400, 100, 64) == 0
    q, k, v, _ = inputs(8, 8, 16, 16, 2400, 100, 64, seed=2)
    o, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    fa.fa_fwd_cross(q, k, v, None, o, lse, None, 0.125)
    check_status()
    check_forward(q, k, v, None, o, lse, 0.125, batches=[7])


def test_forward_large_offsets():
    # queries and keys beyond 2^31 bytes from the base, of whole items and of cut ones
    for B, H, N_q, N_kv in ((70, 8, 16384, 64), (70, 8, 1, 16384), (70, 8, 5, 16384)):
        q = torch.zeros((B, H, N_q, 128), dtype=torch.bfloat16, device="cuda")
        k = torch.zeros((B, H, N_kv, 128), dtype=torch.bfloat16, device="cuda")
        v = torch.zeros_like(k)
        q1, k1, v1, _ = inputs(1, 1, 1, 1, N_q, N_kv, 128, seed=11)
        q[-1, -1], k[-1, -1], v[-1, -1] = q1[0, 0], k1[0, 0], v1[0, 0]
        o, lse = forward(q, k, v, None, scale_for(128))
        check_forward(q1, k1, v1, None, o[-1:, -1:], lse[-1:, -1:], scale_for(128))
        assert (o[0] == 0).all()


def test_rows_behind_the_queries_are_left_alone():
    q, k, v, _ = inputs(3, 1, 2, 1, 5, 150, 64, seed=6)
    o, lse = torch.full((4, 2, 5, 64), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((4, 2, 5), 7.0, device="cuda")
    ws = space(fa.fa_fwd_cross_workspace_size(*sizes(q, k)))
    fa.fa_fwd_cross(q, k, v, None, o[:3], lse[:3], ws, 0.125)
    check_status()
    check_forward(q, k, v, None, o[:3], lse[:3], 0.125)
    assert (o[3] == 7).all() and (lse[3] == 7).all()


@pytest.mark.parametrize("N_q", [1, 9, 300])
def test_two_calls_at_once(N_q):
    calls, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for i in range(2):
        q, k, v, _ = inputs(4, 4, 8, 8, N_q, 3000, 64, seed=20 + i)
        ws = space(fa.fa_fwd_cross_workspace_size(*sizes(q, k)))
        calls.append((q, k, v, torch.empty_like(q), torch.empty(q.shape[:3], device="cuda"), ws))
    torch.cuda.synchronize()
    for _ in range(5):
        for (q, k, v, o, lse, ws), s in zip(calls, streams):
            fa.fa_fwd_cross(q, k, v, None, o, lse, ws, 0.125, stream=s)
    torch.cuda.synchronize()
    check_status()
    for q, k, v, o, lse, _ in calls:
        check_forward(q, k, v, None, o, lse, 0.125)


def captured(call):
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    return graph


@pytest.mark.parametrize("H_kv,N_q", [(2, 1), (8, 1), (8, 260)])
def test_captured_call_follows_the_lengths(H_kv, N_q):
    q, k, v, _ = inputs(4, 4, 8, H_kv, N_q, 2000, 128, seed=15)
    lengths = on_device([5, 5, 5, 5])
    o, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    ws = space(fa.fa_fwd_cross_workspace_size(*sizes(q, k)))
    graph = captured(lambda: fa.fa_fwd_cross(q, k, v, lengths, o, lse, ws, scale_for(128)))
    for new in ([1999, 3, 0, 700], [1, 1, 1, 1], [2000] * 4, [0] * 4):
        lengths.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        check_status()
        check_forward(q, k, v, new, o, lse, scale_for(128))


def test_short_wait_limit_reports_and_recovers():
    q, k, v, _ = inputs(4, 4, 16, 16, 2048, 700, 128, seed=13)
    o, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    ws = space(fa.fa_fwd_cross_workspace_size(*sizes(q, k)))
    fa.fa_set_wait_timeout_ns(1)
    try:
        fa.fa_fwd_cross(q, k, v, None, o, lse, ws, scale_for(128))
        first = fa.fa_last_device_error()
    finally:
        fa.fa_set_wait_timeout_ns(0)
    assert first in (0, fa.FA_ERR_DEVICE_TIMEOUT)
    fa.fa_fwd_cross(q, k, v, None, o, lse, ws, scale_for(128))
    check_status()
    check_forward(q, k, v, None, o, lse, scale_for(128), batches=[0])


def test_binding_refuses_wrong_tensors():
    q, k, v, _ = inputs(4, 2, 4, 2, 3, 50, 64)
    n, o, lse, ws = on_device([50, 50]), torch.empty_like(q), torch.empty(q.shape[:3], device="cuda"), space(1 << 20)
    ok = dict(q=q, k=k, v=v, n=n, o=o, lse=lse, ws=ws)
    for change in (dict(q=q.float()), dict(k=k[:, :, :49]), dict(v=v.transpose(1, 2)), dict(n=n.long()), dict(n=n[:1]),
                   dict(n=n.cpu()), dict(o=o[:3]), dict(lse=lse.bfloat16()), dict(q=q[0]), dict(q=q.cpu()), dict(ws=ws.cpu()),
                   dict(ws=ws[::2])):
        a = dict(ok, **change)
        with pytest.raises(ValueError):
            fa.fa_fwd_cross(a["q"], a["k"], a["v"], a["n"], a["o"], a["lse"], a["ws"], 0.125)
    with pytest.raises(ValueError):
        fa.fa_fwd_prefix(q, k, v, n, o[:1], lse, o, lse, ws, 0.125)
    with pytest.raises(fa.FaError):
        fa.fa_fwd_cross(q[:3].contiguous(), k, v, n, o[:3], lse[:3], ws, 0.125)  # 3 batches to 2


# ---------------------------------------------------------------- backward
def backward(q, k, v, lengths, o, lse, do, scale, ws=None):
    dq, dk, dv = (torch.full_like(t, float("nan")) for t in (q, k, v))
    ws = space(fa.fa_bwd_cross_workspace_size(*sizes(q, k))) if ws is None else ws
    fa.fa_bwd_cross(q, k, v, on_device(lengths), o, lse, do, dq, dk, dv, ws, scale)
    check_status()
    return dq, dk, dv


def check_backward(q, k, v, lengths, do, grads, scale, kv_batches=None):
    share, few = q.shape[0] // k.shape[0], 24
    heads = list(each_head(q, k, lengths))
    q, k, v, do = (f64(t) for t in (q, k, v, do))
    dq, dk, dv = (f64(t) for t in grads)
    rk, rv, tk, tv = (np.zeros(k.shape) for _ in range(4))
    for b, h, kb, kh, n in heads:
        if kv_batches is not None and kb not in kv_batches:
            continue
        seen = np.ones((q.shape[2], n), dtype=bool)
        Q, K, V, dO = q[b, h], k[kb, kh, :n], v[kb, kh, :n], do[b, h]
        o, _, P = plain64.attention(Q, K, V, scale, seen)
        gq, gk, gv = plain64.attention_grad(Q, K, V, dO, scale, seen)
        rk[kb, kh, :n] += gk
        rv[kb, kh, :n] += gv
        t = 1e-5 * (1 + (np.abs(scale) * np.abs(Q @ K.T).max(initial=0)))
        A = P @ np.abs(V)
        dP, size = dO @ V.T, np.abs(dO) @ np.abs(V).T
        if n <= few:
            d_delta = (t + 1e-6) * (np.abs(dO) * A).sum(-1, keepdims=True)
        else:
            d_delta = (np.abs(dO) * (2.0 ** -8 * (A + np.abs(o)) + t * A)).sum(-1, keepdims=True)
        delta = (dO * o).sum(-1, keepdims=True)
        d_dS = P * (d_delta + 1e-6 * size + (2.0 ** -8 + t) * (np.abs(dP - delta) + d_delta))
        tq = np.abs(scale) * d_dS @ np.abs(K) + 2.0 ** -8 * np.abs(gq) + 1e-30
        err = np.abs(dq[b, h] - gq)
        assert np.isfinite(dq[b, h]).all() and (err <= tq).all(), (b, h, float((err / tq).max()))
        tk[kb, kh, :n] += np.abs(scale) * d_dS.T @ np.abs(Q)
        tv[kb, kh, :n] += (2.0 ** -8 + t) * P.T @ np.abs(dO)
    for b in range(k.shape[0]) if kv_batches is None else kv_batches:
        for got, ref, tol in ((dk[b], rk[b], tk[b]), (dv[b], rv[b], tv[b])):
            tol = tol + 2.0 ** -8 * np.abs(ref) + 1e-30 * (tol > 0)
            err = np.abs(got - ref)  # of hidden keys: zeros
            assert np.isfinite(got).all() and (err <= tol).all(), (b, float((err / np.maximum(tol, 1e-30)).max()))


def step(B, B_kv, H, H_kv, N_q, N_kv, d, lengths, seed=0, scale=None, poison=True):
    q, k, v, do = inputs(B, B_kv, H, H_kv, N_q, N_kv, d, seed)
    if poison and lengths is not None:
        for b, n in enumerate(lengths):
            k[b, :, max(n, 0):], v[b, :, max(n, 0):] = float("nan"), float("inf")
    scale = scale_for(d) if scale is None else scale
    o, lse = forward(q, k, v, lengths, scale)
    return q, k, v, do, o, lse, backward(q, k, v, lengths, o, lse, do, scale), scale


@pytest.mark.parametrize("N_q", [1, 2, 127, 128, 129, 300])
@pytest.mark.parametrize("N_kv", [1, 5, 24, 25, 128, 129, 300])
@pytest.mark.parametrize("d", [64, 128])
def test_backward_lengths(N_q, N_kv, d):
    q, k, v, do, _, _, grads, scale = step(2, 2, 3, 1, N_q, N_kv, d, None, seed=N_q)
    check_backward(q, k, v, None, do, grads, scale)


@pytest.mark.parametrize("lengths", [[0, 0, 0], [1, 128, 127], [300, 0, 129], [-7, 256, 10 ** 9], [24, 25, 2]])
@pytest.mark.parametrize("N_q,H,H_kv", [(1, 2, 2), (5, 8, 2), (130, 4, 2), (300, 2, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_backward_ragged_keys(lengths, N_q, H, H_kv, d):
    q, k, v, do, _, _, grads, scale = step(3, 3, H, H_kv, N_q, 300, d, lengths, seed=1)
    check_backward(q, k, v, lengths, do, grads, scale)


@pytest.mark.parametrize("B,B_kv,H,H_kv,N_q", [(4, 1, 2, 2, 1), (6, 2, 8, 2, 1), (6, 3, 2, 1, 33), (4, 2, 2, 1, 200)])
@pytest.mark.parametrize("d", [64, 128])
def test_backward_batches_that_share_keys(B, B_kv, H, H_kv, N_q, d):
    lengths = [333, 200, 0][:B_kv]
    q, k, v, do, _, _, grads, scale = step(B, B_kv, H, H_kv, N_q, 333, d, lengths, seed=B)
    check_backward(q, k, v, lengths, do, grads, scale)


@pytest.mark.parametrize("d", [64, 128])
def test_backward_of_pieces_and_of_many_items(d):
    # many queries on few keys: key blocks are dealt in pieces; many heads: more items than SMs
    q, k, v, do, _, _, grads, scale = step(2, 2, 2, 1, 3000, 200, d, [200, 60], seed=3)
    check_backward(q, k, v, [200, 60], do, grads, scale)
    lengths = [700, 10, 300, 0, 650, 129]
    q, k, v, do, _, _, grads, scale = step(6, 6, 16, 8, 200, 700, d, lengths, seed=4)
    check_backward(q, k, v, lengths, do, grads, scale, kv_batches=[1, 3, 5])
    lengths = [int(x) for x in np.random.default_rng(d).integers(0, 200, 70)]
    q, k, v, do, _, _, grads, scale = step(70, 70, 2, 1, 140, 200, d, lengths, seed=6)
    check_backward(q, k, v, lengths, do, grads, scale, kv_batches=range(0, 70, 9))


@pytest.mark.parametrize("B,B_kv,H,H_kv,N_q,N_kv,lengths", [(4, 4, 2, 1, 40, 4100, [4100, 130, 0, 1000]), (1, 1, 1, 1, 1, 3000, [2999]),
                                                            (6, 2, 3, 1, 70, 2600, [257, 2600]), (1, 1, 2, 2, 300, 2000, None)])
@pytest.mark.parametrize("d", [64, 128])
def test_backward_of_few_queries_on_many_keys(B, B_kv, H, H_kv, N_q, N_kv, lengths, d):
    # the keys of a query block are dealt in pieces, of which a short sequence has one, two or none
    rows = B * H_kv * (-(-H // H_kv * N_q // 128) * 128)
    assert fa.fa_bwd_cross_workspace_size(B, B_kv, H, H_kv, N_q, N_kv, d) >= 2 * rows * 4 + 2 * rows * d * 4
    q, k, v, do, o, lse, grads, scale = step(B, B_kv, H, H_kv, N_q, N_kv, d, lengths, seed=7)
    check_backward(q, k, v, lengths, do, grads, scale)
    for a, b in zip(grads, backward(q, k, v, lengths, o, lse, do, scale)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("scale", [0.0, -0.125, 1.0])
def test_backward_scales(scale):
    q, k, v, do, _, _, grads, scale = step(1, 1, 2, 2, 200, 300, 64, [270], seed=3, scale=scale)
    check_backward(q, k, v, [270], do, grads, scale)


def test_backward_against_differences():
    # the loss sum(o * do) moves by the gradient's share along a random direction: bf16 inputs a step of 2^-4
    # apart, whose o is known to 2^-8 A from float64
    B, H, H_kv, N_q, N_kv, d = 2, 2, 1, 6, 40, 64
    q, k, v, do, _, _, grads, scale = step(B, 1, H, H_kv, N_q, N_kv, d, [33], seed=9, poison=False)

    def loss(q, k, v):
        total = 0.0
        for b, h, kb, kh, n in each_head(do, k, [33]):
            o = plain64.attention(q[b, h], k[kb, kh, :n], v[kb, kh, :n], scale, np.ones((N_q, n), dtype=bool))[0]
            total += (o * f64(do[b, h])).sum()
        return total

    base = [f64(t) for t in (q, k, v)]
    for i in range(3):
        direction = np.random.default_rng(i).standard_normal(base[i].shape)
        eps = 1e-4
        sides = []
        for sign in (1, -1):
            moved = list(base)
            moved[i] = base[i] + sign * eps * direction
            sides.append(loss(*moved))
        slope = (sides[0] - sides[1]) / (2 * eps)
        got, size = (f64(grads[i]) * direction).sum(), (np.abs(f64(grads[i])) * np.abs(direction)).sum()
        # each entry is off by under 3 roundings of 2^-8 (its own, dS or P, delta) of the gradient's terms, whose
        # magnitudes add up to a few times the gradient's own
        assert abs(got - slope) <= 3 * 2.0 ** -8 * 4 * size


@pytest.mark.parametrize("d", [64, 128])
def test_backward_repeats_bit_for_bit(d):
    q, k, v, do, o, lse, grads, scale = step(3, 1, 4, 2, 500, 260, d, [260], seed=5)
    for a, b in zip(grads, backward(q, k, v, [260], o, lse, do, scale)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("B,N_q,N_kv,d", [(4, 150, 300, 64), (2, 40, 4000, 64), (2, 40, 4000, 128), (4, 3, 20, 128)])
def test_captured_step_follows_the_lengths(B, N_q, N_kv, d):
    # also where dQ, in pieces, runs beside dK and dV on rows' values that the replay before wrote in the same place
    q, k, v, do = inputs(B, 2, 4, 2, N_q, N_kv, d, seed=15)
    lengths = on_device([5, 5])
    o, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    dq, dk, dv = (torch.empty_like(t) for t in (q, k, v))
    ws = space(max(fa.fa_fwd_cross_workspace_size(*sizes(q, k)), fa.fa_bwd_cross_workspace_size(*sizes(q, k))))

    def call():
        fa.fa_fwd_cross(q, k, v, lengths, o, lse, ws, scale_for(d))
        fa.fa_bwd_cross(q, k, v, lengths, o, lse, do, dq, dk, dv, ws, scale_for(d))

    graph = captured(call)
    for new in ([N_kv, 17], [0, N_kv // 2 - 21], [N_kv - 7, N_kv]):
        q.copy_(q.flip(2)), do.copy_(do.roll(1, 2))
        lengths.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        check_status()
        check_forward(q, k, v, new, o, lse, scale_for(d))
        check_backward(q, k, v, new, do, (dq, dk, dv), scale_for(d))


def test_backward_large_offsets():
    # K/V gradients and queries beyond 2^31 bytes from the base
    for B, N_q, N_kv in ((70, 100, 16384), (70, 16384, 100)):
        q = torch.zeros((B, 8, N_q, 128), dtype=torch.bfloat16, device="cuda")
        k = torch.zeros((B, 8, N_kv, 128), dtype=torch.bfloat16, device="cuda")
        v, do = torch.zeros_like(k), torch.zeros_like(q)
        one = inputs(1, 1, 1, 1, N_q, N_kv, 128, seed=11)
        q[-1, -1], k[-1, -1], v[-1, -1], do[-1, -1] = (t[0, 0] for t in one)
        o, lse = forward(q, k, v, None, scale_for(128))
        grads = backward(q, k, v, None, o, lse, do, scale_for(128))
        check_backward(*one[:3], None, one[3], [g[-1:, -1:] for g in grads], scale_for(128))
        assert all((g[0] == 0).all() for g in grads)


def test_backward_short_wait_limit_reports_and_recovers():
    q, k, v, do, o, lse, _, scale = step(2, 2, 8, 8, 1024, 700, 128, None, seed=13)
    dq, dk, dv = (torch.empty_like(t) for t in (q, k, v))
    ws = space(fa.fa_bwd_cross_workspace_size(*sizes(q, k)))
    fa.fa_set_wait_timeout_ns(1)
    try:
        fa.fa_bwd_cross(q, k, v, None, o, lse, do, dq, dk, dv, ws, scale)
        first = fa.fa_last_device_error()
    finally:
        fa.fa_set_wait_timeout_ns(0)
    assert first in (0, fa.FA_ERR_DEVICE_TIMEOUT)
    check_backward(q, k, v, None, do, backward(q, k, v, None, o, lse, do, scale), scale, kv_batches=[0])


# ---------------------------------------------------------------- shared prefixes
def own_attention(q, seed):
    """What the queries' own tokens gave: rows of every kind, some without any."""
    g = torch.Generator().manual_seed(seed)
    o = (0.3 * torch.randn(q.shape, generator=g)).to(torch.bfloat16).cuda()
    lse = (6 * torch.randn(q.shape[:3], generator=g)).cuda()
    lse.view(-1)[::5] = -float("inf")
    o.view(-1, q.shape[-1])[::5] = float("nan")  # of no keys: not used
    return o, lse


@pytest.mark.parametrize("B,B_kv,H,H_kv,N_q,N_kv", [(8, 1, 8, 2, 1, 1500), (6, 2, 4, 4, 3, 300), (64, 1, 4, 1, 1, 130),
                                                    (4, 1, 2, 2, 300, 200), (2, 2, 3, 1, 1, 77), (16, 1, 16, 16, 1024, 130),
                                                    (2, 2, 2, 2, 1, 1500), (4, 2, 3, 3, 1, 333)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("in_place", [False, True])
def test_prefix(B, B_kv, H, H_kv, N_q, N_kv, d, in_place):
    q, k, v, _ = inputs(B, B_kv, H, H_kv, N_q, N_kv, d, seed=N_q)
    own = own_attention(q, 3)
    keep = [t.clone() for t in own]
    lengths = [N_kv, N_kv // 2][:B_kv]
    o, lse = own if in_place else (torch.full_like(q, float("nan")), torch.full(q.shape[:3], float("nan"), device="cuda"))
    ws = space(fa.fa_fwd_prefix_workspace_size(*sizes(q, k)))
    fa.fa_fwd_prefix(q, k, v, on_device(lengths), *own, o, lse, ws, scale_for(d))
    check_status()
    check_forward(q, k, v, lengths, o, lse, scale_for(d), own=keep, batches=range(min(B, 6)))


def test_empty_prefix_leaves_the_own_attention():
    q, k, v, _ = inputs(6, 2, 4, 2, 2, 40, 64)
    o_own, lse_own = own_attention(q, 4)
    o, lse = torch.empty_like(q), torch.empty_like(lse_own)
    ws = space(fa.fa_fwd_prefix_workspace_size(*sizes(q, k)))
    fa.fa_fwd_prefix(q, k, v, on_device([0, 0]), o_own, lse_own, o, lse, ws, 0.125)
    check_status()
    none = torch.isinf(lse_own)
    assert (o[none] == 0).all() and torch.equal(o[~none], o_own[~none])
    assert torch.isinf(lse[none]).all()
    # lse passes through base 2: two roundings of 2^-24
    assert torch.allclose(lse[~none], lse_own[~none], rtol=2.0 ** -22, atol=0)
