"""Attention to another sequence's keys where items are cut and their parts joined by a kernel of its own, and
where a wait inside a kernel runs out.  Tolerances: those of test_gpu_cross."""
import pytest
import torch

import exact_io_aware_06_gb300 as fa
from gpu_util import check_status, ensure_built, scale_for
from test_gpu_cross import check_forward, forward, inputs, on_device, sizes, space
from test_gpu_window import until_a_wait_runs_out

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def cut_items(ws):
    """Items that the call before has cut: the workspace begins with 152 places of four ints, the first -1 where nothing
    is cut; space() leaves it so, and calls that join none do not write there."""
    return int((ws[: 152 * 16].view(torch.int32).view(152, 4)[:, 0] >= 0).sum())


@pytest.mark.parametrize("B,H,H_kv,N_q,N_kv,d,lengths", [(16, 64, 8, 1, 16384, 128, [16384] * 12 + [5] * 4),
                                                         (140, 1, 1, 200, 16384, 64, [0] * 100 + [16384] * 40)])
def test_a_wait_that_runs_out_where_items_are_cut(B, H, H_kv, N_q, N_kv, d, lengths):
    # CTAs with more segments than the ring holds: the wait for room in it is one of those that run out, and the join
    # goes by the table all the same
    q, k, v, _ = inputs(B, B, H, H_kv, N_q, N_kv, d, seed=B)
    ws = space(fa.fa_fwd_cross_workspace_size(*sizes(q, k)))
    ref = forward(q, k, v, lengths, scale_for(d), ws)
    assert cut_items(ws) > 4
    check_forward(q, k, v, lengths, *ref, scale_for(d), batches=[0, 11, B - 1])
    n, out = on_device(lengths), [torch.empty_like(t) for t in ref]
    for _ in range(3):
        ws.fill_(255)
        until_a_wait_runs_out(lambda: fa.fa_fwd_cross(q, k, v, n, *out, ws, scale_for(d)), out, ref)


# B, B_kv, H, H_kv, N_q, N_kv, lengths; d: with rows of several batches to a tile, of one batch in two tiles and more, of
# lone tiles; a table place per item (fewer than 152 items) and per CTA
JOINED = [(64, 1, 8, 2, 1, 16384, [16384]), (64, 1, 8, 2, 1, 16384, [10101]), (64, 1, 8, 2, 1, 16384, None),
          (64, 2, 8, 2, 1, 16384, [15000, 300]), (40, 20, 8, 8, 5, 2048, [2048, 0, 1000, 1999, 1] * 4),
          (20, 20, 8, 8, 5, 2048, [2047, 1, 0, 1500, 129] * 4), (2, 2, 2, 2, 300, 5000, [4999, 0]), (3, 1, 2, 1, 200, 5000, [4097])]
SHAPES = ("B,B_kv,H,H_kv,N_q,N_kv,lengths", JOINED)


def own_attention(q, seed):
    """What the queries' own tokens gave; every fifth row has none."""
    g = torch.Generator().manual_seed(seed)
    o = (0.3 * torch.randn(q.shape, generator=g)).to(torch.bfloat16).cuda()
    lse = (6 * torch.randn(q.shape[:3], generator=g)).cuda()
    lse.view(-1)[::5] = -float("inf")
    o.view(-1, q.shape[-1])[::5] = float("nan")
    return o, lse


def poisoned(k, v, lengths):
    for b, n in enumerate(lengths or []):
        k[b, :, n:], v[b, :, n:] = float("nan"), float("inf")


@pytest.mark.parametrize(*SHAPES)
@pytest.mark.parametrize("d", [64, 128])
def test_forward_of_cut_items(B, B_kv, H, H_kv, N_q, N_kv, lengths, d):
    q, k, v, _ = inputs(B, B_kv, H, H_kv, N_q, N_kv, d, seed=N_q)
    poisoned(k, v, lengths)
    ws = space(fa.fa_fwd_cross_workspace_size(*sizes(q, k)))
    o, lse = forward(q, k, v, lengths, scale_for(d), ws)
    assert cut_items(ws) > 0
    check_forward(q, k, v, lengths, o, lse, scale_for(d), batches=range(0, B, max(1, B // 8)))


@pytest.mark.parametrize(*SHAPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("in_place", [False, True])
def test_prefix_of_cut_items(B, B_kv, H, H_kv, N_q, N_kv, lengths, d, in_place):
    # the own attention belongs to the part that has the first block; in place it is written over by the join
    q, k, v, _ = inputs(B, B_kv, H, H_kv, N_q, N_kv, d, seed=N_q)
    poisoned(k, v, lengths)
    own = own_attention(q, 3)
    keep = [t.clone() for t in own]
    o, lse = own if in_place else (torch.full_like(q, float("nan")), torch.full(q.shape[:3], float("nan"), device="cuda"))
    ws = space(fa.fa_fwd_prefix_workspace_size(*sizes(q, k)))
    fa.fa_fwd_prefix(q, k, v, on_device(lengths), *own, o, lse, ws, scale_for(d))
    check_status()
    assert cut_items(ws) > 0
    check_forward(q, k, v, lengths, o, lse, scale_for(d), own=keep, batches=range(0, B, max(1, B // 8)))


def test_empty_prefix_whose_items_might_be_cut():
    q, k, v, _ = inputs(64, 1, 8, 2, 1, 16384, 128)
    poisoned(k, v, [0])
    o_own, lse_own = own_attention(q, 4)
    o, lse = torch.full_like(q, float("nan")), torch.full_like(lse_own, float("nan"))
    ws = space(fa.fa_fwd_prefix_workspace_size(*sizes(q, k)))
    assert ws.numel() > 152 * 16
    fa.fa_fwd_prefix(q, k, v, on_device([0]), o_own, lse_own, o, lse, ws, scale_for(128))
    check_status()
    none = torch.isinf(lse_own)
    assert (o[none] == 0).all() and torch.equal(o[~none], o_own[~none]) and (lse[none] == -float("inf")).all()
    # lse passes through base 2: two roundings of 2^-24
    assert torch.allclose(lse[~none], lse_own[~none], rtol=2.0 ** -22, atol=0)
