"""The 4-bit cache: what is stored and read back, and attention over it, against float64.

Stored values are defined exactly (code times scale), so they are compared for equality.

Decode tolerance, per output o = sum w v over the visible tokens with A = sum w |v|: P is
rounded to bfloat16 (2^-8 of each weight), again after V's scale (2^-8), and o itself (2^-8 of
|o|).  A score is a float32 sum over groups of 32 that starts at -136 sum q: its error e is at
most 2^-21 |scale| sum over groups of s (136 sum |q| + 15 sum |q|), and moves a weight by the
factor exp(2 e).  Together 2^-7 A + 2^-8 |o| + (2 e + 1e-5) A; lse is off by e + 1e-5 (1 + |lse|)."""
import numpy as np
import pytest
import torch

import exact_io_aware_06_gb300 as fa
import plain64
from gpu_util import check_status, ensure_built, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def rand(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(shape, generator=g)).to(torch.bfloat16).cuda()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Cache:
    """Pages in a mixed order, some of them nobody's and full of NaN scales."""

    def __init__(self, lengths, H_kv, d, page, seed=0, spare=2, max_blocks=None):
        B = len(lengths)
        need = [-(-n // page) for n in lengths]
        n_pages = sum(need) + spare
        self.arrays = fa.kv4_cache(n_pages, H_kv, page, d)
        for a in (self.arrays[1], self.arrays[3]):
            a.fill_(float("nan"))
        for a in (self.arrays[0], self.arrays[2]):
            a.random_(0, 256)
        order = np.random.default_rng(seed).permutation(n_pages)
        table = np.full((B, max_blocks or max(1, max(need))), -7, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        self.table = torch.from_numpy(table).cuda()
        self.lengths, self.H_kv, self.d, self.page = lengths, H_kv, d, page

    @property
    def args(self):
        return (*self.arrays, self.table)

    def fill(self, seed, k_scale=1.0, v_scale=1.0):
        """Random tokens for every request; their stored values [B][H_kv, n, d] in float64."""
        B, N = len(self.lengths), max(1, max(self.lengths))
        k, v = rand((B, self.H_kv, N, self.d), seed, k_scale), rand((B, self.H_kv, N, self.d), seed + 1, v_scale)
        fa.fa_kv4_append(k, v, *self.args, ints([0] * B), ints(self.lengths))
        check_status()
        return plain64.kv4_values(f64(k)), plain64.kv4_values(f64(v))


def bf16_of(x):
    return torch.from_numpy(x).to(torch.float32).to(torch.bfloat16)


# ---------------------------------------------------------------- storing and reading
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_append_and_read_ragged(d, page):
    lengths, first = [0, 1, 15, 16, 17, 130, 300], [0, 0, 3, 16, 5, 100, 299]
    B, H_kv = len(lengths), 3
    c = Cache(lengths, H_kv, d, page)
    count = [n - f for n, f in zip(lengths, first)]
    count[0] = 0
    k, v = rand((B, H_kv, 300, d), 1), rand((B, H_kv, 300, d), 2)
    zero = ints([0] * B)
    fa.fa_kv4_append(k, v, *c.args, zero, ints(first))       # what was there before
    new_k, new_v = rand((B, H_kv, 40, d), 3), rand((B, H_kv, 40, d), 4)
    count = [min(40, n) for n in count]
    fa.fa_kv4_append(new_k, new_v, *c.args, ints(first), ints(count))
    total = [f + n for f, n in zip(first, count)]
    out = [torch.full((B, H_kv, 333, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    fa.fa_kv4_read(*c.args, ints(total), *out)
    check_status()
    for got, old, new in ((out[0], k, new_k), (out[1], v, new_v)):
        old, new = plain64.kv4_values(f64(old)), plain64.kv4_values(f64(new))
        ref = np.zeros((B, H_kv, 333, d))
        for b in range(B):
            ref[b, :, :first[b]] = old[b, :, :first[b]]
            ref[b, :, first[b]:total[b]] = new[b, :, :count[b]]
        assert torch.equal(got.cpu(), bf16_of(ref))


@pytest.mark.parametrize("d,lengths", [(64, [9001, 3, 0, 8192]), (128, [5001, 5000, 1, 16])])
def test_read_many_rows(d, lengths):
    # enough rows for two a thread; odd and even lengths, and an odd number of rows
    c = Cache(lengths, 8, d, 64)
    k, v = c.fill(51)
    N = max(lengths)
    back = [torch.full((4, 8, N, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    fa.fa_kv4_read(*c.args, ints(lengths), *back)
    check_status()
    for t, values in zip(back, (k, v)):
        for b, n in enumerate(lengths):
            assert np.array_equal(f64(t[b, :, :n]), plain64.bf16_round(values[b][:, :n])) and (t[b, :, n:] == 0).all()


def test_values_at_the_format_s_edges():
    # ties, zeros, one value alone, the smallest and largest bfloat16, infinities and NaN
    d, n = 64, 12
    x = torch.zeros((1, 1, n, d))
    x[0, 0, 1] = 7.0
    x[0, 0, 2, :32] = torch.arange(32) / 2.0 - 8.0   # scale 16 / 14: many halves
    x[0, 0, 3, 5] = -3.5
    x[0, 0, 4, :14] = torch.arange(14) - 6.5         # scale bf16(7.5 / 7)
    x[0, 0, 5] = 7.0 / 2 ** torch.arange(64)
    x[0, 0, 6] = 9.183e-41                           # smallest subnormal: its scale is 0
    x[0, 0, 7] = 3.3895e38
    x[0, 0, 8, :7] = torch.tensor([7.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5])
    x[0, 0, 9, 3] = float("inf")
    x[0, 0, 10, 40] = float("nan")
    x[0, 0, 11, 0] = -float("inf")
    x = x.to(torch.bfloat16).cuda()
    c = Cache([n], 1, d, 16)
    fa.fa_kv4_append(x, x, *c.args, ints([0]))
    out = [torch.empty_like(x) for _ in "kv"]
    fa.fa_kv4_read(*c.args, ints([n]), *out)
    check_status()
    ref = plain64.kv4_values(f64(x[:, :, :9]))
    ref[0, 0, 6] = 0.0
    for got in out:
        assert torch.equal(got[:, :, :9].cpu(), bf16_of(ref))
        got = got[0, 0].float().cpu()
        for row, bad in ((9, slice(0, 32)), (10, slice(32, 64)), (11, slice(0, 32))):
            assert got[row, bad].isnan().all() and (got[row].nan_to_num(0.0) == 0).all()
            assert not got[row, 32 - bad.start:64 - bad.start].isnan().any()


def test_pages_and_positions_outside_the_cache_are_left_out_and_reported():
    d, page, H_kv = 64, 16, 2
    c = Cache([40, 40], H_kv, d, page, spare=3)
    k, v = c.fill(5)
    good = [a.clone() for a in c.arrays]
    table = c.table.clone()
    table[0, 1] = 10 ** 6
    table[1, 0] = -1
    new = rand((2, H_kv, 48, d), 6)
    # request 0's second page, request 1's first one and everything past the table are missing
    fa.fa_kv4_append(new, new, *c.arrays, table, ints([16, 0]), ints([16, 16]))
    assert fa.fa_last_device_error() == fa.FA_ERR_DEVICE_INDEX
    fa.fa_kv4_append(new, new, *c.args, ints([48, -48]))
    assert fa.fa_last_device_error() == fa.FA_ERR_DEVICE_INDEX
    for a, b in zip(c.arrays, good):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    out = [torch.empty((2, H_kv, 40, d), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    fa.fa_kv4_read(*c.arrays, table, ints([40, 40]), *out)
    assert fa.fa_last_device_error() == fa.FA_ERR_DEVICE_INDEX
    for got, ref in zip(out, (k, v)):
        ref = ref[:, :, :40].copy()
        ref[0, :, 16:32] = 0
        ref[1, :, :16] = 0
        assert torch.equal(got.cpu(), bf16_of(ref))
    # attention hides the missing tokens
    q = rand((2, 4, 1, d), 7)
    o, lse, _ = decode(q, c, [40, 40], table=table, status=fa.FA_ERR_DEVICE_INDEX)
    for b, keep in ((0, [*range(16), *range(32, 40)]), (1, range(16, 40))):
        compare(q[b:b + 1], o[b:b + 1], lse[b:b + 1], [k[b][:, keep]], [v[b][:, keep]], [len(keep)])
    # a length beyond the table is cut to it
    o, lse, _ = decode(q, c, [1000, 40], status=fa.FA_ERR_DEVICE_INDEX)
    compare(q[1:], o[1:], lse[1:], [k[1]], [v[1]], [40])


# ---------------------------------------------------------------- attention
def decode(q, c, lengths, window=0, n_sink=0, scale=None, table=None, status=0, ws=None):
    B, H, N_q, d = q.shape
    o = torch.full_like(q, float("nan"))
    lse = torch.full((B, H, N_q), float("nan"), device="cuda")
    if ws is None:
        n = fa.fa_decode_kv4_workspace_size(B, H, c.H_kv, N_q, d)
        ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    fa.fa_decode_kv4(q, *c.arrays, c.table if table is None else table, ints(lengths), o, lse, ws,
                     d ** -0.5 if scale is None else scale, window, n_sink)
    assert fa.fa_last_device_error() == status
    return o, lse, ws


def compare(q, o, lse, k, v, lengths, window=0, n_sink=0, scale=None):
    """q [B, H, N_q, d] and results against values k, v [B][H_kv, >= lengths[b], d]."""
    B, H, N_q, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    q, o, lse = f64(q), f64(o), f64(lse)
    for b in range(B):
        n = lengths[b]
        seen = plain64.window_mask(N_q, n, n - N_q, window, n_sink)
        for h in range(H):
            kv = h // (H // k[b].shape[0])
            kk, vv = k[b][kv, :n], v[b][kv, :n]
            ref, ref_lse, P = plain64.attention(q[b, h], kk, vv, scale, seen)
            A = P @ np.abs(vv)
            # s <= (largest |k|) / 7 of the group; the largest over all tokens and groups
            s = np.abs(kk).max() / 7 if n else 0.0
            e = (2.0 ** -21 * abs(scale) * s * 151 * np.abs(q[b, h]).sum(-1))[:, None]
            tol = 2.0 ** -7 * A + 2.0 ** -8 * np.abs(ref) + (2 * e + 1e-5) * A
            empty = ~seen.any(-1) if n else np.ones(N_q, bool)
            assert (o[b, h][empty] == 0).all() and np.isneginf(lse[b, h][empty]).all()
            err = np.abs(o[b, h] - ref)
            assert (err <= tol)[~empty].all(), (b, h, float((err / np.maximum(tol, 1e-300)).max()))
            dl = np.abs(lse[b, h][~empty] - ref_lse[~empty])
            assert (dl <= (e[:, 0] + 1e-5 * (1 + np.abs(ref_lse)))[~empty]).all(), (b, h, dl.max())


def run_and_compare(lengths, H, H_kv, N_q, d, page, window=0, n_sink=0, scale=None, **fill):
    c = Cache(lengths, H_kv, d, page)
    k, v = c.fill(11, **fill)
    q = rand((len(lengths), H, N_q, d), 13)
    o, lse, _ = decode(q, c, lengths, window, n_sink, scale)
    compare(q, o, lse, k, v, lengths, window, n_sink, scale)
    return c, q, o, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 128])
def test_decode_ragged_lengths(d, page):
    run_and_compare([0, 1, 2, 15, 16, 17, 63, 64, 65, 200, 1000, 5, 0], 8, 2, 1, d, page)


@pytest.mark.parametrize("H,H_kv", [(1, 1), (3, 3), (7, 1), (8, 1), (9, 1), (16, 1), (32, 1), (12, 4)])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_group_sizes(H, H_kv, d):
    run_and_compare([70, 333], H, H_kv, 1, d, 32)


@pytest.mark.parametrize("N_q", [2, 3, 5, 9])
@pytest.mark.parametrize("H,H_kv", [(2, 2), (4, 1), (6, 2)])
def test_decode_several_queries(N_q, H, H_kv):
    # requests shorter than N_q have queries at negative positions: they see nothing
    run_and_compare([0, 1, 3, 9, 16, 100], H, H_kv, N_q, 64, 16)
    run_and_compare([2, 90], H, H_kv, N_q, 128, 16, window=5, n_sink=1)


@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 1), (16, 0), (17, 4), (100, 20), (64, 64), (5000, 3), (300, 5000),
                                           (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_window_and_sinks(window, n_sink, d):
    run_and_compare([1, 16, 31, 100, 117, 777], 4, 2, 1, d, 16, window, n_sink)


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_decode_scales(scale):
    run_and_compare([40, 300], 4, 1, 1, 64, 16, scale=scale)


@pytest.mark.parametrize("v_scale", [1e-30, 1e30])
def test_decode_values_of_any_range(v_scale):
    run_and_compare([200], 4, 1, 1, 128, 16, v_scale=v_scale)


def test_decode_growing_scores_move_the_reference():
    # key j is j / 40 times one direction: scores grow along the request by far more than the
    # lazy threshold, so that every tile moves the running maximum
    n, d = 700, 64
    c = Cache([n], 1, d, 16)
    unit = rand((d,), 3).float()
    k = (torch.arange(n, device="cuda")[:, None] / 40 * unit).to(torch.bfloat16)[None, None].contiguous()
    v = rand((1, 1, n, d), 4)
    fa.fa_kv4_append(k, v, *c.args, ints([0]))
    q = unit.to(torch.bfloat16).expand(1, 2, 1, d).contiguous()
    o, lse, _ = decode(q, c, [n])
    compare(q, o, lse, [plain64.kv4_values(f64(k))[0]], [plain64.kv4_values(f64(v))[0]], [n])


def test_decode_many_requests_and_one_long_one():
    # more entries than resident CTAs, and an entry that many CTAs share
    run_and_compare([7] * 300 + [4000], 4, 2, 1, 64, 16)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,H_kv,N_q,window", [(8, 2, 1, 0), (4, 2, 5, 0), (4, 2, 5, 40), (2, 2, 1, 60)])
def test_decode_more_heads_than_sms(H, H_kv, N_q, window, d):
    # more K/V heads of requests than SMs: CTAs of two warps
    run_and_compare([(37 * i) % 300 for i in range(80)], H, H_kv, N_q, d, 32, window, 4)


def test_decode_long_single_head():
    run_and_compare([30011], 2, 1, 1, 128, 256)


def test_decode_repeats_bit_for_bit_and_follows_lengths_in_a_graph():
    lengths = [900, 33, 0, 120]
    c = Cache(lengths, 2, 128, 16)
    k, v = c.fill(21)
    q = rand((4, 8, 1, 128), 22)
    o, lse, ws = decode(q, c, lengths)
    o2, lse2, _ = decode(q, c, lengths, ws=ws)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    # two captured calls on one workspace, replayed after the lengths have changed
    n = ints(lengths)
    outs = [(torch.empty_like(q), torch.empty((4, 8, 1), device="cuda")) for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            fa.fa_decode_kv4(q, *c.args, n, *outs[0], ws, 128 ** -0.5, 0, 0)
            fa.fa_decode_kv4(q, *c.args, n, *outs[1], ws, 128 ** -0.5, 50, 2)
    torch.cuda.current_stream().wait_stream(s)
    for lens in (lengths, [1, 20, 0, 7], [500, 0, 0, 0]):
        n.copy_(ints(lens))
        graph.replay()
        check_status()
        compare(q, *outs[0], k, v, lens)
        compare(q, *outs[1], k, v, lens, 50, 2)


def test_decode_on_another_stream_after_append():
    # append, decode in order on a side stream, no host wait between them
    lengths = [513, 64]
    c = Cache(lengths, 2, 64, 64)
    k, v = c.fill(31)
    new_k, new_v = rand((2, 2, 1, 64), 33), rand((2, 2, 1, 64), 34)
    q = rand((2, 4, 1, 64), 35)
    last, full = ints([512, 63]), ints(lengths)
    o, lse = torch.empty_like(q), torch.empty((2, 4, 1), device="cuda")
    ws = torch.empty(fa.fa_decode_kv4_workspace_size(2, 4, 2, 1, 64), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    fa.fa_kv4_append(new_k, new_v, *c.args, last, stream=s)
    fa.fa_decode_kv4(q, *c.args, full, o, lse, ws, 0.125, stream=s)
    s.synchronize()
    check_status()
    for x, new in ((k, new_k), (v, new_v)):
        y = plain64.kv4_values(f64(new))
        x[0, :, 512], x[1, :, 63] = y[0, :, 0], y[1, :, 0]
    compare(q, o, lse, k, v, lengths, scale=0.125)


def test_decode_nan_in_a_visible_group_shows_and_elsewhere_does_not():
    c = Cache([64], 1, 64, 16)
    k, v = rand((1, 1, 64, 64), 1), rand((1, 1, 64, 64), 2)
    v[0, 0, 10, 40] = float("nan")
    fa.fa_kv4_append(k, v, *c.args, ints([0]))
    q = rand((1, 2, 1, 64), 3)
    o, _, _ = decode(q, c, [64])
    assert o[..., 32:].isnan().all() and not o[..., :32].isnan().any()
    o, _, _ = decode(q, c, [64], window=16)     # token 10 hidden, in another tile
    assert not o.isnan().any()
    o, _, _ = decode(q, c, [10])                # token 10 behind the end, in the same tile
    assert not o.isnan().any()


def test_pages_beyond_32_bits():
    # codes of K and V take 5 GB each; the request's pages are the last ones, in falling order
    n, d, page, H_kv, n_pages = 700, 128, 256, 8, 40000
    k, v, q = rand((1, H_kv, n, d), 41), rand((1, H_kv, n, d), 42), rand((1, 16, 1, d), 43)
    results = []
    for pages, table in ((n_pages, [39999, 39998, 39997]), (3, [0, 1, 2])):
        arrays, table = fa.kv4_cache(pages, H_kv, page, d), ints([table])
        assert pages == 3 or arrays[0].numel() > 2 ** 32
        fa.fa_kv4_append(k, v, *arrays, table, ints([0]))
        back = [torch.empty_like(k), torch.empty_like(v)]
        fa.fa_kv4_read(*arrays, table, ints([n]), *back)
        o, lse = torch.empty_like(q), torch.empty((1, 16, 1), device="cuda")
        ws = torch.empty(fa.fa_decode_kv4_workspace_size(1, 16, H_kv, 1, d), dtype=torch.uint8, device="cuda")
        fa.fa_decode_kv4(q, *arrays, table, ints([n]), o, lse, ws, d ** -0.5)
        check_status()
        results.append((*back, o, lse))
        del arrays
    assert all(torch.equal(a, b) for a, b in zip(*results))
    assert np.array_equal(f64(results[0][0]), plain64.bf16_round(plain64.kv4_values(f64(k))))
    compare(q, results[0][2], results[0][3], plain64.kv4_values(f64(k)), plain64.kv4_values(f64(v)), [n])


@pytest.mark.parametrize("N", [1, 40, 300])
@pytest.mark.parametrize("bad", [-1, -2 ** 31, 10 ** 6])
def test_read_reports_lengths_outside_the_cache(N, bad):
    # a negative length holds nothing; one beyond the table is cut to it
    d, page, H_kv = 64, 16, 2
    c = Cache([64, 64], H_kv, d, page)
    k, v = c.fill(61)
    for lengths in ([bad, 64], [64, bad]):
        out = [torch.full((2, H_kv, N, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        fa.fa_kv4_read(*c.args, ints(lengths), *out)
        assert fa.fa_last_device_error() == fa.FA_ERR_DEVICE_INDEX
        for t, values in zip(out, (k, v)):
            for b, n in enumerate(lengths):
                n = min(N, 64, max(n, 0))
                assert np.array_equal(f64(t[b, :, :n]), plain64.bf16_round(values[b][:, :n])) and (t[b, :, n:] == 0).all()
    fa.fa_kv4_read(*c.args, ints([64, 0]), *out)
    check_status()


def test_read_of_many_rows_reports_lengths_outside_the_cache():
    # two rows a thread
    c = Cache([8192, 16], 8, 64, 64)
    c.fill(63)
    back = [torch.empty((2, 8, 20000, 64), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    fa.fa_kv4_read(*c.args, ints([8192, 16]), *back)
    check_status()
    for lengths in ([8193, 16], [8192, -16]):
        fa.fa_kv4_read(*c.args, ints(lengths), *back)
        assert fa.fa_last_device_error() == fa.FA_ERR_DEVICE_INDEX


def test_append_reports_a_negative_count():
    c = Cache([40, 40], 2, 64, 16)
    c.fill(65)
    before = [a.clone() for a in c.arrays]
    new = rand((2, 2, 5, 64), 66)
    for count in ([-1, 0], [0, -2 ** 31]):
        fa.fa_kv4_append(new, new, *c.args, ints([3, 3]), ints(count))
        assert fa.fa_last_device_error() == fa.FA_ERR_DEVICE_INDEX
    fa.fa_kv4_append(new, new, *c.args, ints([3, 3]), ints([0, 0]))
    check_status()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(c.arrays, before))
    # more than there are rows: all rows
    fa.fa_kv4_append(new, new, *c.args, ints([3, 3]), ints([5, 6]))
    check_status()
    back = [torch.empty((2, 2, 8, 64), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    fa.fa_kv4_read(*c.args, ints([8, 8]), *back)
    ref = plain64.bf16_round(plain64.kv4_values(f64(new)))
    assert all(np.array_equal(f64(t[:, :, 3:]), ref) for t in back)
