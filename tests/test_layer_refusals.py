"""Argument errors of the layer's operators, found on the host before anything is launched (no
GPU: the pointers are never followed), and their float64 references against differences."""
import ctypes

import numpy as np
import pytest

import exact_io_aware_06_gb300 as fa
import plain64
from exact_io_aware_06_gb300 import _build

P = ctypes.c_void_p(0x10000)    # aligned, never dereferenced: rejected first
MIS = ctypes.c_void_p(0x10008)  # misaligned
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def L():
    _build.build()
    return fa.lib()


def freq(n, bad=None):
    a = (ctypes.c_double * n)(*[1.0 / (i + 1) for i in range(n)])
    if bad is not None:
        a[n - 1] = bad
    return a


NORM = dict(qkv=P, qw=P, kw=P, pos=P, f=freq(32), q=P, k=P, v=P, B=1, H=2, H_kv=1, N=8, d=64, rot=64,
            eps=1e-6, dtype=1)


@pytest.mark.parametrize("change,status", [
    (dict(qkv=None), 1), (dict(q=None), 1), (dict(k=MIS), 1), (dict(v=None), 1), (dict(qw=MIS), 1),
    (dict(kw=MIS), 1), (dict(pos=MIS), 1), (dict(f=None), 1), (dict(f=freq(32, NAN)), 1),
    (dict(f=freq(32, INF)), 1), (dict(B=0), 1), (dict(H=0), 1), (dict(H_kv=0), 1), (dict(N=0), 1),
    (dict(rot=8), 1), (dict(rot=80), 1), (dict(rot=-16), 1), (dict(eps=-1.0), 1), (dict(eps=NAN), 1),
    (dict(dtype=2), 1), (dict(dtype=7), 1), (dict(d=96), 2), (dict(d=256), 2),
    (dict(N=(1 << 24) + 1), 2), (dict(B=1 << 8, N=1 << 23), 2), (dict(B=1 << 12, H=1 << 13), 2),
    (dict(B=1 << 12, H_kv=1 << 13), 2)])
def test_norm_rope_refusals(L, change, status):
    a = dict(NORM, **change)
    assert L.fa_qk_norm_rope(a["qkv"], a["qw"], a["kw"], a["pos"], a["f"], a["q"], a["k"], a["v"], a["B"],
                             a["H"], a["H_kv"], a["N"], a["d"], a["rot"], 0, a["eps"], a["dtype"],
                             None) == status


@pytest.mark.parametrize("change,status", [
    (dict(qkv=None), 1), (dict(dq=None), 1), (dict(dk=MIS), 1), (dict(dv=None), 1), (dict(dqkv=None), 1),
    (dict(dqw=MIS), 1), (dict(ws=None), 1), (dict(ws=MIS), 1), (dict(nbytes=100), 1), (dict(rot=24), 1),
    (dict(d=32), 2)])
def test_norm_rope_bwd_refusals(L, change, status):
    n = fa.fa_qk_norm_rope_bwd_workspace_size(1, 2, 1, 8, 64)
    assert n > 100
    a = dict(NORM, dq=P, dk=P, dv=P, dqkv=P, dqw=P, dkw=P, ws=P, nbytes=n)
    a.update(change)
    assert L.fa_qk_norm_rope_bwd(a["qkv"], a["qw"], a["kw"], a["pos"], a["f"], a["dq"], a["dk"], a["dv"],
                                 a["dqkv"], a["dqw"], a["dkw"], a["ws"], a["nbytes"], a["B"], a["H"],
                                 a["H_kv"], a["N"], a["d"], a["rot"], 0, a["eps"], a["dtype"], None) == status


WINDOW = dict(q=P, k=P, v=P, o=P, lse=None, B=1, H=4, H_kv=2, N=128, d=64, scale=0.1, window=16, sinks=4,
              dtype=1)
WINDOW_BAD = [
    (dict(q=None), 1), (dict(k=MIS), 1), (dict(v=None), 1), (dict(o=None), 1), (dict(lse=MIS), 1),
    (dict(B=0), 1), (dict(H=0), 1), (dict(H_kv=0), 1), (dict(H_kv=3), 1), (dict(N=0), 1),
    (dict(scale=NAN), 1), (dict(scale=INF), 1), (dict(window=0), 1), (dict(window=-5), 1),
    (dict(sinks=-1), 1), (dict(dtype=2), 1), (dict(dtype=0), 2), (dict(d=96), 2), (dict(d=256), 2),
    (dict(N=(1 << 24) + 1), 2), (dict(B=1 << 12, H=1 << 13), 2), (dict(B=1 << 8, H=1 << 8, N=1 << 22), 2)]


@pytest.mark.parametrize("change,status", WINDOW_BAD)
def test_window_forward_refusals(L, change, status):
    a = dict(WINDOW, **change)
    assert L.fa_fwd_window(a["q"], a["k"], a["v"], a["o"], a["lse"], a["B"], a["H"], a["H_kv"], a["N"], a["d"],
                           a["scale"], a["window"], a["sinks"], a["dtype"], None) == status


@pytest.mark.parametrize("change,status", WINDOW_BAD + [
    (dict(lse=None), 1), (dict(do=MIS), 1), (dict(dq=None), 1), (dict(dk=MIS), 1), (dict(dv=None), 1),
    (dict(ws=None), 1), (dict(ws=MIS), 1), (dict(short=4), 1)])
def test_window_backward_refusals(L, change, status):
    a = dict(WINDOW, lse=P, do=P, dq=P, dk=P, dv=P, ws=P, short=0)
    a.update(change)
    n = fa.fa_bwd_window_workspace_size(*(a[x] for x in ("B", "H", "H_kv", "N", "d", "window", "sinks")))
    assert L.fa_bwd_window(a["q"], a["k"], a["v"], a["o"], a["lse"], a["do"], a["dq"], a["dk"], a["dv"], a["ws"],
                           n - a["short"] if n else 0, a["B"], a["H"], a["H_kv"], a["N"], a["d"], a["scale"],
                           a["window"], a["sinks"], a["dtype"], None) == status


def test_window_workspace(L):
    # delta and lse; nothing more without sinks, or where the window covers the sequence; a sink
    # block's parts otherwise
    rows = 2 * 2 * 4 * 4096 * 4
    size = fa.fa_bwd_window_workspace_size
    assert size(2, 4, 2, 4096, 64, 512, 0) == rows
    assert size(2, 4, 2, 4096, 64, 4096, 100) == rows
    # 32 query blocks, 5 of them in reach: 27 later ones in pieces of 5 blocks, and the near part
    assert size(2, 4, 2, 4096, 64, 512, 4) == rows + 2 * 2 * (6 + 1) * 2 * 128 * 64 * 4
    assert size(1, 4, 3, 4096, 64, 512, 4) == 0
    assert size(1, 4, 2, 4096, 64, 0, 4) == 0


CACHE = dict(kc=P, ks=P, vc=P, vs=P, table=P, B=2, H_kv=2, N=4, d=64, page=16, n_pages=8, max_blocks=4)
CACHE_BAD = [
    (dict(kc=None), 1), (dict(ks=MIS), 1), (dict(vc=None), 1), (dict(vs=MIS), 1), (dict(table=None), 1),
    (dict(B=0), 1), (dict(H_kv=0), 1), (dict(N=0), 1), (dict(n_pages=0), 1), (dict(max_blocks=0), 1),
    (dict(page=8), 1), (dict(page=24), 1), (dict(page=512), 1), (dict(page=0), 1), (dict(d=96), 2),
    (dict(max_blocks=1 << 28), 2), (dict(max_blocks=(1 << 27) - 1), 2)]  # the last: 2^31 - 16 tokens


@pytest.mark.parametrize("change,status", CACHE_BAD + [
    (dict(k=None), 1), (dict(v=MIS), 1), (dict(first=None), 1), (dict(count=MIS), 1), (dict(N=(1 << 24) + 1), 2)])
def test_append_refusals(L, change, status):
    a = dict(CACHE, k=P, v=P, first=P, count=None)
    a.update(change)
    assert L.fa_kv4_append(a["k"], a["v"], a["kc"], a["ks"], a["vc"], a["vs"], a["table"], a["first"],
                           a["count"], a["B"], a["H_kv"], a["N"], a["d"], a["page"], a["n_pages"],
                           a["max_blocks"], None) == status


@pytest.mark.parametrize("change,status", CACHE_BAD + [
    (dict(k=None), 1), (dict(v=MIS), 1), (dict(lengths=None), 1)])
def test_read_refusals(L, change, status):
    a = dict(CACHE, k=P, v=P, lengths=P)
    a.update(change)
    assert L.fa_kv4_read(a["kc"], a["ks"], a["vc"], a["vs"], a["table"], a["lengths"], a["k"], a["v"], a["B"],
                         a["H_kv"], a["N"], a["d"], a["page"], a["n_pages"], a["max_blocks"], None) == status


@pytest.mark.parametrize("change,status", CACHE_BAD + [
    (dict(q=None), 1), (dict(o=MIS), 1), (dict(lengths=None), 1), (dict(lse=MIS), 1), (dict(ws=None), 1),
    (dict(nbytes=64), 1), (dict(H=3), 1), (dict(scale=NAN), 1), (dict(scale=INF), 1), (dict(window=-1), 1),
    (dict(sinks=-1), 1), (dict(N=(1 << 24) + 1), 2), (dict(B=1 << 10, H=1 << 10, N=1 << 12), 2)])
def test_decode_refusals(L, change, status):
    n = fa.fa_decode_kv4_workspace_size(2, 4, 2, 4, 64)
    assert n > 64
    a = dict(CACHE, q=P, o=P, lengths=P, lse=None, ws=P, nbytes=n, H=4, scale=0.1, window=0, sinks=0)
    a.update(change)
    assert L.fa_decode_kv4(a["q"], a["kc"], a["ks"], a["vc"], a["vs"], a["table"], a["lengths"], a["o"],
                           a["lse"], a["ws"], a["nbytes"], a["B"], a["H"], a["H_kv"], a["N"], a["d"],
                           a["page"], a["n_pages"], a["max_blocks"], a["scale"], a["window"], a["sinks"],
                           None) == status


def test_workspace_sizes_of_refused_sizes_are_zero(L):
    assert fa.fa_decode_kv4_workspace_size(1, 3, 2, 1, 64) == 0
    assert fa.fa_decode_kv4_workspace_size(1, 4, 2, 1, 96) == 0
    assert fa.fa_decode_kv4_workspace_size(0, 4, 2, 1, 64) == 0
    assert fa.fa_qk_norm_rope_bwd_workspace_size(1, 4, 2, 1, 96) == 0
    assert fa.fa_qk_norm_rope_bwd_workspace_size(1, 4, 0, 1, 64) == 0


def test_workspace_sizes_of_sizes_beyond_32_bits_are_zero(L):
    big = 2 ** 32
    for i in range(5):
        sizes = [1, 4, 2, 16, 64]
        sizes[i] += big
        assert fa.fa_decode_kv4_workspace_size(*sizes) == 0
        assert fa.fa_qk_norm_rope_bwd_workspace_size(*sizes) == 0
        assert fa.fa_bwd_window_workspace_size(*sizes, 4, 0) == 0
    size = fa.fa_bwd_window_workspace_size
    assert size(1, 4, 2, 4096, 64, big + 1, 4) == size(1, 4, 2, 4096, 64, 4096, 4) > 0
    assert size(1, 4, 2, 4096, 64, 130, big) == size(1, 4, 2, 4096, 64, 130, 4096) > 0
    assert size(1, 4, 2, 4096, 64, 5 - big, 4) == size(1, 4, 2, 4096, 64, 5, 5 - big) == 0


def test_frequencies_beyond_2_64_are_refused(L):
    for f in (2.0 ** 64 * (1 + 2.0 ** -52), -1e20, 1e300):
        a = dict(NORM, f=freq(32))
        a["f"][7] = f
        assert L.fa_qk_norm_rope(a["qkv"], a["qw"], a["kw"], a["pos"], a["f"], a["q"], a["k"], a["v"], a["B"],
                                 a["H"], a["H_kv"], a["N"], a["d"], a["rot"], 0, a["eps"], a["dtype"], None) == 1


def test_status_name(L):
    assert fa.fa_status_string(fa.FA_ERR_DEVICE_INDEX) == "FA_ERR_DEVICE_INDEX"


# ---------------------------------------------------------------- the references themselves
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_gradient_is_the_difference_quotient(interleaved):
    rng = np.random.default_rng(3)
    B, N, H, H_kv, d = 2, 3, 2, 1, 16
    x = rng.standard_normal((B, N, H + 2 * H_kv, d))
    qw, kw = 1 + 0.1 * rng.standard_normal((2, d))
    pos = rng.integers(-50, 5000, (B, N))
    f = [1.0, 0.3, 0.01]
    up = [rng.standard_normal((B, h, N, d)) for h in (H, H_kv, H_kv)]

    def loss(x, qw, kw):
        y = plain64.norm_rope(x, H, H_kv, qw, kw, pos, f, 1e-3, interleaved)
        return sum((a * b).sum() for a, b in zip(y, up))

    dx, dqw, dkw = plain64.norm_rope_grad(x, H, H_kv, qw, kw, pos, f, 1e-3, interleaved, *up)
    h = 1e-6
    for grad, args in ((dx, 0), (dqw, 1), (dkw, 2)):
        for at in rng.integers(0, grad.size, 12):
            step = np.zeros(grad.size)
            step[at] = h
            step = step.reshape(grad.shape)
            p = [x, qw, kw]
            p[args] = p[args] + step
            m = [x, qw, kw]
            m[args] = m[args] - step
            # central difference: h^2 of the third derivative, and 2^-52 |loss| / h
            assert abs((loss(*p) - loss(*m)) / (2 * h) - grad.flat[at]) < 1e-7


@pytest.mark.parametrize("window,n_sink", [(3, 0), (4, 2), (1, 1), (100, 0)])
def test_window_gradient_is_the_difference_quotient(window, n_sink):
    rng = np.random.default_rng(5)
    n, d = 9, 4
    q, k, v, do = rng.standard_normal((4, n, d))
    seen = plain64.window_mask(n, n, 0, window, n_sink)
    grads = plain64.attention_grad(q, k, v, do, 0.7, seen)
    h = 1e-6
    for i, g in enumerate(grads):
        for at in range(0, n * d, 5):
            step = np.zeros(n * d)
            step[at] = h
            step = step.reshape(n, d)
            p, m = [q, k, v], [q, k, v]
            p[i], m[i] = p[i] + step, m[i] - step
            diff = (plain64.attention(*p, 0.7, seen)[0] - plain64.attention(*m, 0.7, seen)[0]) * do
            assert abs(diff.sum() / (2 * h) - g.flat[at]) < 1e-7
