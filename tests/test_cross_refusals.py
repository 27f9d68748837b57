"""Argument errors of attention to another sequence's keys and of positions with several axes, found on the
host before anything is launched (no GPU: the pointers are never followed)."""
import ctypes

import pytest
import torch

import exact_io_aware_06_gb300 as fa
from exact_io_aware_06_gb300 import _build
from test_layer_refusals import INF, MIS, NAN, NORM, P, freq


@pytest.fixture(scope="module")
def L():
    _build.build()
    return fa.lib()


def ints(*x):
    return (ctypes.c_int * len(x))(*x)


AXES = dict(NORM, axis=ints(*[i % 3 for i in range(32)]), n_axes=3)
AXES_BAD = [
    (dict(qkv=None), 1), (dict(pos=None), 1), (dict(pos=MIS), 1), (dict(f=None), 1), (dict(axis=None), 1), (dict(n_axes=0), 1),
    (dict(n_axes=-1), 1), (dict(n_axes=9), 1), (dict(n_axes=2), 1), (dict(axis=ints(*([0] * 31), -1)), 1),
    (dict(axis=ints(*([0] * 31), 3)), 1), (dict(f=freq(32, NAN)), 1), (dict(rot=8), 1), (dict(rot=80), 1), (dict(d=96), 2),
    (dict(eps=-1.0), 1), (dict(dtype=2), 1), (dict(N=0), 1), (dict(N=(1 << 24) + 1), 2)]


@pytest.mark.parametrize("change,status", AXES_BAD + [(dict(q=None), 1), (dict(k=MIS), 1)])
def test_axes_refusals(L, change, status):
    a = dict(AXES, **change)
    assert L.fa_qk_norm_rope_axes(a["qkv"], a["qw"], a["kw"], a["pos"], a["f"], a["axis"], a["q"], a["k"], a["v"], a["B"],
                                  a["H"], a["H_kv"], a["N"], a["d"], a["rot"], a["n_axes"], 0, a["eps"], a["dtype"],
                                  None) == status


@pytest.mark.parametrize("change,status", AXES_BAD + [
    (dict(dq=None), 1), (dict(dqkv=MIS), 1), (dict(ws=None), 1), (dict(nbytes=100), 1)])
def test_axes_bwd_refusals(L, change, status):
    n = fa.fa_qk_norm_rope_bwd_workspace_size(1, 2, 1, 8, 64)
    a = dict(AXES, dq=P, dk=P, dv=P, dqkv=P, dqw=P, dkw=P, ws=P, nbytes=n)
    a.update(change)
    assert L.fa_qk_norm_rope_axes_bwd(a["qkv"], a["qw"], a["kw"], a["pos"], a["f"], a["axis"], a["dq"], a["dk"], a["dv"],
                                      a["dqkv"], a["dqw"], a["dkw"], a["ws"], a["nbytes"], a["B"], a["H"], a["H_kv"], a["N"],
                                      a["d"], a["rot"], a["n_axes"], 0, a["eps"], a["dtype"], None) == status


def test_axes_of_sections():
    f, axis = fa.rope_axes([4, 6], base=100.0)
    assert axis.tolist() == [0, 0, 1, 1, 1] and axis.dtype == torch.int32
    assert torch.equal(f, torch.cat([fa.rope_frequencies(4, 100.0), fa.rope_frequencies(6, 100.0)]))
    f, axis = fa.rope_axes([4, 6], base=100.0, shared=True)
    assert axis.tolist() == [0, 0, 1, 1, 1] and torch.equal(f, fa.rope_frequencies(10, 100.0))
    with pytest.raises(ValueError):
        fa.rope_axes([3, 5])


CROSS = dict(q=P, k=P, v=P, n=P, o=P, lse=None, B=6, B_kv=3, H=4, H_kv=2, N_q=5, N_kv=700, d=64, scale=0.1, dtype=1)
CROSS_SIZES = ("B", "B_kv", "H", "H_kv", "N_q", "N_kv", "d")
CROSS_BAD = [
    (dict(q=None), 1), (dict(k=MIS), 1), (dict(v=None), 1), (dict(n=MIS), 1), (dict(o=None), 1), (dict(lse=MIS), 1),
    (dict(B=0), 1), (dict(B_kv=0), 1), (dict(B_kv=4), 1), (dict(B_kv=12), 1), (dict(H=0), 1), (dict(H_kv=0), 1), (dict(H_kv=3), 1),
    (dict(N_q=0), 1), (dict(N_kv=0), 1), (dict(scale=NAN), 1), (dict(scale=INF), 1), (dict(dtype=2), 1), (dict(dtype=0), 2),
    (dict(d=96), 2), (dict(d=256), 2), (dict(N_q=(1 << 24) + 1), 2), (dict(N_kv=(1 << 24) + 1), 2),
    (dict(B=3 << 12, H=1 << 13), 2), (dict(B=3, H=256, H_kv=1, N_q=1 << 23), 2)]


@pytest.mark.parametrize("change,status", CROSS_BAD + [(dict(ws=None), 1), (dict(ws=MIS), 1), (dict(short=4), 1)])
def test_cross_forward_refusals(L, change, status):
    a = dict(CROSS, ws=P, short=0)
    a.update(change)
    n = fa.fa_fwd_cross_workspace_size(*(a[x] for x in CROSS_SIZES))
    assert L.fa_fwd_cross(a["q"], a["k"], a["v"], a["n"], a["o"], a["lse"], a["ws"], max(0, n - a["short"]),
                          *(a[x] for x in CROSS_SIZES), a["scale"], a["dtype"], None) == status


@pytest.mark.parametrize("change,status", CROSS_BAD + [(dict(ws=None), 1), (dict(short=4), 1), (dict(o_own=None), 1),
                                                       (dict(lse_own=None), 1), (dict(o_own=MIS), 1), (dict(lse_own=MIS), 1)])
def test_prefix_refusals(L, change, status):
    a = dict(CROSS, ws=P, short=0, o_own=P, lse_own=P)
    a.update(change)
    n = fa.fa_fwd_prefix_workspace_size(*(a[x] for x in CROSS_SIZES))
    assert L.fa_fwd_prefix(a["q"], a["k"], a["v"], a["n"], a["o_own"], a["lse_own"], a["o"], a["lse"], a["ws"],
                           max(0, n - a["short"]), *(a[x] for x in CROSS_SIZES), a["scale"], a["dtype"], None) == status


@pytest.mark.parametrize("change,status", CROSS_BAD + [
    (dict(lse=None), 1), (dict(do=None), 1), (dict(dq=MIS), 1), (dict(dk=None), 1), (dict(dv=MIS), 1), (dict(ws=None), 1),
    (dict(short=4), 1)])
def test_cross_backward_refusals(L, change, status):
    a = dict(CROSS, lse=P, do=P, dq=P, dk=P, dv=P, ws=P, short=0)
    a.update(change)
    n = fa.fa_bwd_cross_workspace_size(*(a[x] for x in CROSS_SIZES))
    assert L.fa_bwd_cross(a["q"], a["k"], a["v"], a["n"], a["o"], a["lse"], a["do"], a["dq"], a["dk"], a["dv"], a["ws"],
                          max(0, n - a["short"]), *(a[x] for x in CROSS_SIZES), a["scale"], a["dtype"], None) == status


def test_cross_workspaces(L):
    size = fa.fa_fwd_cross_workspace_size
    # five rows of a K/V head over 12 blocks of keys: 152 places of cut items, and twelve CTAs with two parts of 32 rows
    assert size(1, 1, 5, 1, 1, 1500, 64) == 152 * 16 + 12 * 2 * 32 * (64 + 2) * 4
    # one row: none
    assert size(1, 1, 1, 1, 1, 1500, 64) == 0
    # more items than the work is cut for: none
    assert size(8, 8, 16, 16, 2400, 100, 64) == 0
    for bad in ((0, 1, 1, 1, 1, 1, 64), (3, 2, 1, 1, 1, 1, 64), (1, 1, 3, 2, 1, 1, 64), (1, 1, 1, 1, 1, 1, 80), (1, 1, 1, 1, 1 << 40, 1, 64)):
        assert size(*bad) == 0
        assert fa.fa_bwd_cross_workspace_size(*bad) == 0
    # delta and lse of the rows of a K/V head in whole blocks: 2 heads of 5 rows, in each of 6 batches and 2 heads
    assert fa.fa_bwd_cross_workspace_size(6, 6, 4, 2, 5, 700, 64) == 2 * 6 * 2 * 128 * 4
    # and the parts of the 4 key blocks' pieces
    rows = 2 * 40960 * 4
    assert (fa.fa_bwd_cross_workspace_size(1, 1, 1, 1, 40960, 512, 64) - rows) % (4 * 2 * 128 * 64 * 4) == 0
    assert fa.fa_bwd_cross_workspace_size(1, 1, 1, 1, 40960, 512, 64) > rows
