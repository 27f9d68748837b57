// cross_deal.cuh -- attention to another sequence's keys: a call's arguments, how its rows are tiled, and how its work
// is dealt to the CTAs, by host and device.  Nothing here needs the tensor core or shared memory, so that a
// warp's part of it can be run on the host as well.
//
// No query has a place among the keys, so all rows that meet the same K/V head are alike: the G N_q
// rows of a group of heads lie side by side in q [B][H_kv][G N_q][d] (R = G N_q), and where R is small and
// batches share their keys, several batches' rows fill one tile.  Single tokens, beams over one
// encoder's states and a shared prefix are then the same tiles as a long text's.
#pragma once

#include "fwd_sizes.h"
#include "internal.h"

namespace fa {

// A K/V head's query rows in tiles of 128: nb whole batches of R rows each, or (nb = 1) runs of 128 rows
// of one batch.  Two tiles are an item, as in the plain forward: K_j and V_j are loaded once for both.
struct CrossArgs {
    const int* lengths;    // [B_kv] or null
    void* o;               // [B][H_kv][R][d] bf16
    float* lse;            // [B][H_kv][R] or null
    const void* o_own;     // as o, merged into it; null: none
    const float* lse_own;
    // Items that were cut, each by the CTA that begins it: last CTA (-1: none), batch, item, first CTA; in the
    // item's place (by_item) or the CTA's, whichever are fewer.
    int4* cut;
    float* part;           // two parts a CTA: [d / 4][part_rows][4] O, then m and l of part_rows each
    int R, share, H_kv, B_kv, N_kv;
    int nb, tiles_b, tiles, n_pairs, part_rows;
    int per;               // items of a batch, H_kv n_pairs
    int stream;            // 0: whole items; 1: equal runs of key blocks, items cut where they end
    int edge;              // an item's start and end in blocks, for these runs
    int by_item, join_rows;
    int cluster;           // 2^cluster CTAs share one item, each with its own run of the keys; 0: as `stream`
    int ctas;
    int few;               // no tiles
    float c_log2;          // scale * log2(e), not 0
    DevCtl ctl;
};

namespace {

constexpr int kMaxCtas = 152;

__device__ __forceinline__ int cross_length(const CrossArgs& a, int b) {
    return a.lengths ? min(max(__ldg(a.lengths + b), 0), a.N_kv) : a.N_kv;
}
// A sequence without keys has one block, all of it hidden: its rows get O = 0, lse = -inf from it.
__device__ __forceinline__ int cross_blocks(int len) { return len > 0 ? (len + kBN - 1) / kBN : 1; }

// The key blocks of all items and `edge` for each item's start and end ("units", the edge in front), item by item,
// batch by batch, in equal runs for the CTAs.  By a whole warp, 32 batches at a time.  Work of fewer than 8 * 152
// items of up to 2^17 blocks is dealt so: 32 bits hold all of their units.
__device__ __forceinline__ int cross_units(const CrossArgs& a, int len) { return cross_blocks(len) + a.edge; }
struct UnitPlace {
    int b, item, at, len;  // K/V batch, item of the batch, unit of the item; the batch's keys
};
struct Units {
    int len, upto;         // of batch `lane`: keys; units of an item in batches 0 .. lane
    int each, more;        // every CTA has `each`, the first `more` one more
    // batches b0 + lane
    __device__ __forceinline__ void scan(const CrossArgs& a, int b0) {
        const int lane = threadIdx.x % 32, b = b0 + lane;
        len = b < a.B_kv ? cross_length(a, b) : 0;
        upto = b < a.B_kv ? cross_units(a, len) : 0;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += x;
        }
    }
    __device__ __forceinline__ explicit Units(const CrossArgs& a) {
        uint32_t total = 0;
        if (!a.lengths) {
            total = a.B_kv * cross_units(a, a.N_kv);
        } else {
            for (int b0 = (a.B_kv - 1) & ~31; b0 >= 0; b0 -= 32) {  // the first 32 last, which place() begins with
                scan(a, b0);
                total += __shfl_sync(0xffffffffu, upto, 31);
            }
        }
        total *= a.per;
        each = total / static_cast<uint32_t>(a.ctas);
        more = total - each * a.ctas;
    }
    __device__ __forceinline__ int first(int cta) const { return each * cta + min(cta, more); }
    __device__ __forceinline__ UnitPlace place(const CrossArgs& a, uint32_t u) {
        UnitPlace p;
        uint32_t n;
        if (!a.lengths) {
            p.len = a.N_kv;
            n = cross_units(a, p.len);
            p.b = u / (a.per * n);
            u -= p.b * a.per * n;
        } else {
            for (int b0 = 0;; scan(a, b0)) {
                const unsigned behind = __ballot_sync(0xffffffffu, u < static_cast<uint32_t>(upto * a.per));
                if (behind || b0 + 32 >= a.B_kv) {
                    const int l = behind ? __ffs(behind) - 1 : 31;
                    p.b = b0 + l;
                    p.len = __shfl_sync(0xffffffffu, len, l);
                    n = cross_units(a, p.len);
                    u -= (__shfl_sync(0xffffffffu, upto, l) - n) * a.per;
                    break;
                }
                u -= __shfl_sync(0xffffffffu, upto, 31) * a.per;
                b0 += 32;
            }
        }
        p.item = u / n;
        p.at = u - p.item * n;
        return p;
    }
};

// Of up to 32 batches the one that comes in this lane's place if those of most blocks go first; by a whole warp.
__device__ __forceinline__ int batch_order(const CrossArgs& a) {
    const int lane = threadIdx.x % 32, blocks = lane < a.B_kv ? cross_blocks(cross_length(a, lane)) : 0;
    const int first = __shfl_sync(0xffffffffu, blocks, 0);
    if (__all_sync(0xffffffffu, lane >= a.B_kv || blocks == first)) return lane;
    int rank = 0, batch = 0;
    for (int j = 0; j < a.B_kv; ++j) {
        const int other = __shfl_sync(0xffffffffu, blocks, j);
        rank += other > blocks || (other == blocks && j < lane) ? 1 : 0;
    }
    for (int j = 0; j < a.B_kv; ++j)
        if (__shfl_sync(0xffffffffu, rank, j) == lane) batch = j;
    return batch;
}

// Where a tile's rows come from: its first batch and, for nb = 1, its first row there; rows in use.
struct TileRows {
    int b, r0, rows;
};
__device__ __forceinline__ TileRows tile_rows(const CrossArgs& a, int kv_batch, int tile) {
    TileRows t;
    if (a.nb > 1) {
        t.b = tile * a.nb;
        t.rows = min(a.nb, a.share - t.b) * a.R;
        t.r0 = 0;
    } else {
        t.b = a.share == 1 ? 0 : static_cast<uint32_t>(tile) / static_cast<uint32_t>(a.tiles_b);
        t.r0 = (tile - t.b * a.tiles_b) * kBM;
        t.rows = min(kBM, a.R - t.r0);
    }
    t.b += kv_batch * a.share;
    return t;
}
// Row `row` of the tile, among the rows [B][H_kv][R].
__device__ __forceinline__ size_t global_row(const CrossArgs& a, const TileRows& t, int h, int row) {
    const int over = a.nb > 1 ? row / a.R : 0;
    return (static_cast<size_t>(t.b + over) * a.H_kv + h) * a.R + (t.r0 + row - over * a.R);
}

// A run of key blocks of an item: what the kernel's roles read of it.
struct __align__(16) Segment {
    int n;       // its blocks; 0: nothing to do for this CTA
    int k0;      // the first
    int len;     // the sequence's keys
    int flags;   // 1: of one tile; 2: the CTA's last; 4: all blocks of the item
    int bh_kv, h;
    TileRows rows[2];
    __device__ __forceinline__ bool solo() const { return flags & 1; }
    __device__ __forceinline__ bool last() const { return flags & 2; }
    __device__ __forceinline__ bool whole() const { return flags & 4; }
    __device__ __forceinline__ int slot() const { return k0 > 0 ? 0 : 1; }  // of the CTA's two parts
};

// An item's place in a segment.
__device__ __forceinline__ void place_item(const CrossArgs& a, Segment& s, int batch, int item) {
    s.h = a.n_pairs == 1 ? item : static_cast<uint32_t>(item) / static_cast<uint32_t>(a.n_pairs);
    const int pair = item - s.h * a.n_pairs;
    const bool solo = 2 * pair + 1 >= a.tiles;
    s.bh_kv = batch * a.H_kv + s.h;
    s.rows[0] = tile_rows(a, batch, 2 * pair);
    if (!solo) s.rows[1] = tile_rows(a, batch, 2 * pair + 1);
    s.flags = solo ? 1 : 0;
}

// This CTA's segments, one after the other.
struct Walk {
    int b, item, kb, blocks, len;
    int left;  // units behind the edge of the item
    __device__ __forceinline__ Walk(const CrossArgs& a, Units& units) {
        const int u = units.first(blockIdx.x);
        left = units.first(blockIdx.x + 1) - u;
        if (left > 0) {
            const UnitPlace p = units.place(a, u);
            b = p.b, item = p.item, len = p.len;
            blocks = cross_blocks(len);
            kb = max(0, p.at - a.edge);
            left -= max(0, a.edge - p.at);
        }
    }
    // The next one; `batch` and `at`, its item of the batch; the item's blocks `behind` it.
    __device__ __forceinline__ void next(const CrossArgs& a, Segment& s, int& batch, int& at, int& behind) {
        batch = b, at = item, s.k0 = kb, s.len = len;
        s.n = min(left, blocks - kb);
        behind = blocks - kb - s.n;
        left -= s.n + a.edge;
        kb = 0;
        if (++item == a.per && left > 0) {
            item = 0;
            len = cross_length(a, ++b);
            blocks = cross_blocks(len);
        }
        place_item(a, s, batch, at);
        s.flags |= (left <= 0 ? 2 : 0) | (s.k0 == 0 && behind == 0 ? 4 : 0);
    }
};

// The segments of this CTA's equal run, published one after the other (`publish(i, segment)`: false when a wait for room
// ran out), and its part of the table of cut items.  By a whole warp.  The join follows the table whatever became of
// the segments, and the workspace may have held anything before: every place of it is written, also after such a wait.
template <class Publish>
__device__ __forceinline__ void deal_runs(const CrossArgs& a, Segment& s, Publish publish) {
    const int lane = threadIdx.x % 32;
    Units units(a);
    Walk walk(a, units);
    // An item that this CTA begins and leaves cut, and its last CTA, for the join.
    int4 cut = make_int4(-1, 0, 0, static_cast<int>(blockIdx.x));
    int cut_at = static_cast<int>(blockIdx.x), behind_it = 0;
    if (walk.left <= 0) {
        s.n = 0;
        s.flags = 2;
        publish(0, s);
    }
    bool room = true;
    for (int i = 0; walk.left > 0; ++i) {
        int batch, item, behind;
        walk.next(a, s, batch, item, behind);
        if (room) room = publish(i, s);
        if (s.k0 > 0 || a.ctas == 1) continue;
        const int place = batch * a.per + item;
        if (behind > 0) {
            cut = make_int4(0, batch, item, cut.w);
            behind_it = behind;
            if (a.by_item) cut_at = place;
        } else if (a.by_item && lane == 0) {
            a.cut[place] = make_int4(-1, 0, 0, 0);
        }
    }
    if (cut.x == 0) {
        const int end = units.first(blockIdx.x + 1) + behind_it;  // behind the item's last unit
        cut.x = static_cast<int>(blockIdx.x);
        for (;; cut.x += 32) {
            const int cta = cut.x + 1 + lane;
            const unsigned in = __ballot_sync(0xffffffffu, cta < a.ctas && units.first(cta) < end);
            if (in != 0xffffffffu) {
                cut.x += __popc(in);
                break;
            }
        }
    }
    // (an item's place is written by the CTA that begins it, a CTA's by itself)
    if (lane == 0 && a.ctas > 1 && (cut.x >= 0 || !a.by_item)) a.cut[cut_at] = cut;
}

// How a call's rows are tiled and its work dealt, from its sizes alone.
inline CrossArgs deal(int B, int B_kv, int H, int H_kv, int N_q, int N_kv, int d) {
    CrossArgs a = {};
    a.R = H / H_kv * N_q;
    a.share = B / B_kv;
    a.H_kv = H_kv;
    a.B_kv = B_kv;
    a.N_kv = N_kv;
    a.nb = 1;
    if (a.R <= kBM / 2 && a.share > 1) a.nb = a.share < kBM / a.R ? a.share : kBM / a.R;
    a.tiles_b = (a.R + kBM - 1) / kBM;
    a.tiles = a.nb > 1 ? (a.share + a.nb - 1) / a.nb : a.share * a.tiles_b;
    a.n_pairs = (a.tiles + 1) / 2;
    a.per = H_kv * a.n_pairs;
    const int rows = a.nb > 1 ? a.nb * a.R : a.R;  // of a lone tile
    a.part_rows = a.tiles > 1 ? 2 * kBM : round_up(rows < kBM ? rows : kBM, 32);
    const long long items = static_cast<long long>(B_kv) * a.per;
    a.join_rows = a.tiles > 1 ? 2 * kBM : rows < kBM ? rows : kBM;
    // Whole items, or key blocks in equal runs?  In blocks of the busiest CTA, an item's end counting 1.25, the
    // join's launch 2.5 and what leaves a cut item as float32 and comes back 0.022 for 256 rows at d = 128.
    // With a CTA or less an item the longest sequence would set the pace, and a batch's mean is taken for 3/4 of
    // it.  Measured, whole / cut: 138 items of 4 blocks 12.4 / 24.1 us, 512 of 4 37 / 50, 160 of 16 55 / 47,
    // 63 of up to 17 27.8 / 21.8.  Lone tiles of four rows, bound by HBM (tokens of 32 / 8 heads at d = 128 on 1500 keys):
    // 24 requests 36.2 / 33.0 us, 32 37.9 / 41.7, 40 52.2 / 47.9, 64 70.5 / 69.0; 32 on 3000 keys 67.3 / 68.7, the only
    // one of these where the slower is taken.
    const double blocks = (N_kv + kBN - 1) / kBN, even = items * blocks / kMaxCtas;
    const double whole = ((items + kMaxCtas - 1) / kMaxCtas) * (blocks + 1.25);
    const double parts = (items < kMaxCtas ? kMaxCtas + items : 2 * kMaxCtas) * a.part_rows / 256.0 * d / 128.0;
    const double cut = even * (items <= kMaxCtas ? 0.75 : 1.0) + (items / double{kMaxCtas} + 1) * 1.25 + 2.5 + 0.022 * parts;
    a.stream = N_kv > kBN && items < 8 * kMaxCtas && cut < whole;
    // A few rows: no tiles (cross_few_sm103.cu), and clusters of up to eight CTAs to fill the SMs.  One row, or two at
    // d = 64, at any length, unless the CTAs are few and have long to read (4 heads on 16000 keys 27 us, tiles 17); up
    // to four on short sequences (64 x 32 / 8 heads at d = 128 on 500 keys 27 us, tiles 30; on 500-8192 193, tiles 175).
    // Four rows without tiles / with them (tokens of 32 / 8 heads at d = 128): 1 request on 700 keys 6.5 / 7.9 us, on 1500
    // 7.5 / 8.6, on 4000 12.3 / 11.2, on 16000 30 / 21; 4 on 700 7.5 / 9.0, on 1500 11.0 / 11.3; 8 on 1500 20.8 / 15.1, on
    // 16000 90 / 86: beyond 640 keys the tiles lose up to 1.4 us to few requests and win as much as a quarter elsewhere.
    const long long few_rows = static_cast<long long>(a.R) * a.share;
    int cluster = 0;
    const bool narrow = few_rows * d <= 128;
    while (cluster < 3 && items << cluster < (narrow ? 4 : 2) * kMaxCtas && N_kv >> cluster > 256) ++cluster;
    a.few = few_rows <= 4 && (narrow ? (N_kv >> cluster) * d <= 1 << 17 || items << cluster >= 2 * kMaxCtas
                                     : N_kv <= 640);
    if (a.few) {
        a.cluster = cluster;
        a.stream = 0;
    }
    a.by_item = items < kMaxCtas;
    const long long units = a.stream ? items * ((N_kv + kBN - 1) / kBN) : items;
    a.ctas = static_cast<int>(units < kMaxCtas ? units : kMaxCtas);
    // Of packed tiles O leaves more slowly.  Counting blocks alone, some CTAs got many short sequences and few blocks:
    // 8 short and 8 long items 78 -> 36 us, 64 ragged single tokens 185 -> 175; edges of 1 and 4 were slower.
    a.edge = units <= kMaxCtas ? 0 : a.part_rows == 2 * kBM && a.nb == 1 ? 2 : 3;
    return a;
}

}  // namespace
}  // namespace fa
