"""How attention to another sequence's keys is dealt (cross_deal.cuh), its device code run on the host: the segments
that every CTA takes and the table of cut items, which the join follows, so that every place of it has to be
written in every call, also where the wait for room in the ring of segments runs out."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from exact_io_aware_06_gb300 import _build

CODE = r'''
#include "warp_on_host.h"
#include "cross_deal.cuh"

using namespace fa;

struct Call {
    const CrossArgs* a;
    int fails;      // from this segment of a CTA on no room is found
    int* segments;  // CTA, batch and head, first row of the first tile, first block, blocks, flags
    int n;
};
static void one_warp(void* p) {
    Call& c = *static_cast<Call*>(p);
    Segment s = {};
    deal_runs(*c.a, s, [&](int i, const Segment& x) {
        if (i >= c.fails) return false;
        if (threadIdx.x % 32 == 0 && x.n > 0) {
            const int row[] = {static_cast<int>(blockIdx.x), x.bh_kv, x.rows[0].b, x.rows[0].r0, x.k0, x.n, x.flags};
            for (int v : row) c.segments[c.n++] = v;
        }
        return true;
    });
}
// what[8]: stream, cluster, few, by_item, ctas, items of a batch, tile pairs of a K/V head, places
extern "C" int deal_on_host(const int* sizes, const int* lengths, int fails, int* cut, int* segments, int* what) {
    CrossArgs a = deal(sizes[0], sizes[1], sizes[2], sizes[3], sizes[4], sizes[5], sizes[6]);
    a.lengths = lengths;
    a.cut = reinterpret_cast<int4*>(cut);
    const int out[] = {a.stream, a.cluster, a.few, a.by_item, a.ctas, a.per, a.n_pairs, a.by_item ? a.B_kv * a.per : a.ctas - 1};
    for (int i = 0; i < 8; ++i) what[i] = out[i];
    if (!a.stream) return 0;
    Call c = {&a, fails, segments, 0};
    gridDim.x = a.ctas;
    for (int cta = 0; cta < a.ctas; ++cta) host_warp::run(cta, 96, one_warp, &c);
    return c.n / 7;
}
'''
UNTOUCHED = 0x5A5A5A5A


@pytest.fixture(scope="module")
def deal(tmp_path_factory):
    d = tmp_path_factory.mktemp("deal")
    src, out = d / "t.cpp", d / "t.so"
    src.write_text(CODE)
    cxx = os.environ.get("CXX") or shutil.which("g++")
    toolkit = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_build.nvcc()))), "include")
    subprocess.run([cxx, "-O1", "-std=c++17", "-shared", "-fPIC", "-I", os.path.dirname(os.path.abspath(__file__)), "-I",
                    _build.CSRC, "-isystem", toolkit, str(src), "-o", str(out)], check=True)
    fn = ctypes.CDLL(str(out)).deal_on_host

    def call(sizes, lengths, fails=1 << 30):
        sizes = np.array(sizes, dtype=np.int32)
        lengths = None if lengths is None else np.array(lengths, dtype=np.int32)
        cut, what = np.full((152, 4), UNTOUCHED, dtype=np.int32), np.zeros(8, dtype=np.int32)
        segments = np.zeros((1 << 14, 7), dtype=np.int32)
        p = lambda x: None if x is None else x.ctypes.data_as(ctypes.c_void_p)  # noqa: E731
        n = fn(p(sizes), p(lengths), int(fails), p(cut), p(segments), p(what))
        names = ("stream", "cluster", "few", "by_item", "ctas", "per", "pairs", "places")
        return cut, segments[:n], dict(zip(names, what.tolist()))

    return call


def ragged(n, seed, most, empty=0.3):
    g = np.random.default_rng(seed)
    return [int(x) for x in np.where(g.random(n) < empty, 0, g.integers(0, most + 1, n))]


# B, B_kv, H, H_kv, N_q, N_kv, d; lengths
CASES = {
    # items in places of their own; a CTA begins some 20 of the short ones at the end
    "long then short": ((16, 16, 64, 8, 1, 16384, 128), [16384] * 12 + [5] * 4),
    "many empty": ((140, 140, 1, 1, 200, 16384, 64), [0] * 100 + [16384] * 40),
    "empty among long": ((140, 140, 1, 1, 200, 16384, 64), ([0] * 5 + [16384] * 2) * 20),
    "one prompt": ((64, 1, 8, 2, 1, 16384, 64), [16384]),
    "all of one length": ((1, 1, 2, 2, 300, 5000, 128), None),
    "two batches": ((2, 2, 2, 2, 300, 5000, 128), [130, 5000]),
    # a place per CTA
    "many items": ((20, 20, 8, 8, 5, 2048, 64), ragged(20, 1, 2048)),
    "many items of more than 32 sequences": ((70, 70, 16, 8, 2, 4096, 128), ragged(70, 2, 4096)),
    "packed": ((40, 20, 8, 8, 5, 2048, 128), ragged(20, 3, 2048)),
    "no keys": ((20, 20, 8, 8, 5, 2048, 64), [0] * 20),
}


@pytest.mark.parametrize("case", CASES)
def test_segments_and_table(deal, case):
    sizes, lengths = CASES[case]
    cut, segments, what = deal(sizes, lengths)
    assert what["stream"] and not what["cluster"] and not what["few"]
    B_kv, N_kv, per = sizes[1], sizes[5], what["per"]
    blocks = [max(1, -(-min(max(n, 0), N_kv) // 128)) for n in (lengths or [N_kv] * B_kv)]
    by_item = {}
    for row in segments:
        by_item.setdefault(tuple(row[1:4]), []).append(row)
    assert len(by_item) == B_kv * per
    owners = {}  # first row of an item: batch, item
    for key in by_item:
        owners.setdefault(key[0], []).append(key)
    for bh, keys in owners.items():
        batch, h = divmod(bh, sizes[3])
        for pair, key in enumerate(sorted(keys)):
            rows, item = by_item[key], h * what["pairs"] + pair
            at = 0  # its blocks once each, in order, CTA after CTA
            for i, (cta, _, _, _, k0, n, flags) in enumerate(rows):
                assert k0 == at and n > 0 and cta == rows[0][0] + i
                assert bool(flags & 4) == (n == blocks[batch])
                at += n
            assert at == blocks[batch]
            place = batch * per + item if what["by_item"] else rows[0][0]
            if len(rows) > 1:
                assert cut[place].tolist() == [rows[-1][0], batch, item, rows[0][0]]
            elif what["by_item"]:
                assert cut[place, 0] == -1
    assert (cut[: what["places"]] != UNTOUCHED).all() and (cut[what["ctas"] if not what["by_item"] else what["places"]:] == UNTOUCHED).all()
    if not what["by_item"]:
        begun = {rows[0][0] for rows in by_item.values() if len(rows) > 1}
        assert all(cut[c, 0] == -1 for c in range(what["places"]) if c not in begun)


@pytest.mark.parametrize("fails", [0, 1, 8, 9, 15])
@pytest.mark.parametrize("case", CASES)
def test_table_where_a_wait_runs_out(deal, case, fails):
    # the join follows the table all the same, whatever the workspace held before: it has to be the whole one
    sizes, lengths = CASES[case]
    assert (deal(sizes, lengths, fails)[0] == deal(sizes, lengths)[0]).all()


def test_cases_reach_the_ring(deal):
    # that a CTA has more segments than the ring holds (8), so that a wait for room can run out
    most = {case: np.bincount(deal(*CASES[case])[1][:, 0]).max() for case in CASES}
    assert most["long then short"] > 16 and most["many empty"] > 8, most


@pytest.mark.parametrize("B,N_q", [(1 << 16, 1 << 16), (1 << 15, 1 << 16), ((1 << 16) + 1, 1 << 16), (1 << 12, 1 << 20), (3, 1 << 23), (1 << 8, 1 << 23)])
@pytest.mark.parametrize("d", [64, 128])
def test_many_rows_are_not_taken_for_few(deal, B, N_q, d):
    # the rows that share a K/V head, counted over the batches that do: beyond an int
    assert not deal((B, 1, 1, 1, N_q, 300, d), None)[2]["few"]


def test_few_rows(deal):
    assert deal((1, 1, 8, 8, 1, 300, 64), None)[2]["few"] and deal((4, 1, 1, 1, 1, 300, 128), None)[2]["few"]
    assert not deal((5, 1, 1, 1, 1, 300, 64), None)[2]["few"]
