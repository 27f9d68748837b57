// cross_fwd.cuh -- attention to another sequence's keys: its arguments, how the work is dealt, and the
// rows of a query tile.
//
// No query has a place among the keys, so all rows that meet the same K/V head are alike: the G N_q
// rows of a group of heads lie side by side in q [B][H_kv][G N_q][d] (R = G N_q), and where R is small and
// batches share their keys, several batches' rows fill one tile.  Single tokens, beams over one
// encoder's states and a shared prefix are then the same tiles as a long text's.
#pragma once

#include "fwd_tile.cuh"
#include "layer_ops.h"
#include "ptx.cuh"

namespace fa {

// A K/V head's query rows in tiles of 128: nb whole batches of R rows each, or (nb = 1) runs of 128 rows
// of one batch.  Two tiles are an item, as in the plain forward: K_j and V_j are loaded once for both.
struct CrossArgs {
    const int* lengths;    // [B_kv] or null
    void* o;               // [B][H_kv][R][d] bf16
    float* lse;            // [B][H_kv][R] or null
    const void* o_own;     // as o, merged into it; null: none
    const float* lse_own;
    float* part;           // two parts a CTA: [2][d / 4][part_rows][4] O, then [2][part_rows] m, l
    int R, share, H_kv, B_kv, N_kv;
    int nb, tiles_b, tiles, n_pairs, part_rows;
    int stream;            // 0: whole items; 1: equal runs of key blocks, items cut where they end
    int ctas;
    float c_log2;          // scale * log2(e), not 0
    DevCtl ctl;
};

namespace {

constexpr int kPartTile = kBM;  // rows of a part's second tile start here

__device__ __forceinline__ int cross_length(const CrossArgs& a, int b) {
    return a.lengths ? min(max(__ldg(a.lengths + b), 0), a.N_kv) : a.N_kv;
}
// A sequence without keys has one block, all of it hidden: its rows get O = 0, lse = -inf from it.
__device__ __forceinline__ int cross_blocks(int len) { return len > 0 ? (len + kBN - 1) / kBN : 1; }

// The key blocks of all items, item by item, batch by batch: their number, and where unit u lies.  By a
// whole warp, 32 batches at a time.
struct UnitPlace {
    int b, item, kb;  // K/V batch, item of the batch, key block
};
__device__ __forceinline__ long long total_units(const CrossArgs& a) {
    const long long items = static_cast<long long>(a.H_kv) * a.n_pairs;
    if (!a.lengths) return items * a.B_kv * cross_blocks(a.N_kv);
    long long n = 0;
    for (int b = threadIdx.x % 32; b < a.B_kv; b += 32) n += cross_blocks(cross_length(a, b));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) n += __shfl_xor_sync(0xffffffffu, n, off);
    return n * items;
}
__device__ __forceinline__ UnitPlace unit_place(const CrossArgs& a, long long u) {
    const long long items = static_cast<long long>(a.H_kv) * a.n_pairs;
    UnitPlace p;
    int n;
    if (!a.lengths) {
        n = cross_blocks(a.N_kv);
        p.b = static_cast<int>(u / (items * n));
        u -= p.b * items * n;
    } else {
        const int lane = threadIdx.x % 32;
        for (int b0 = 0;; b0 += 32) {
            const int mine = b0 + lane < a.B_kv ? cross_blocks(cross_length(a, b0 + lane)) : 0;
            int upto = mine;  // blocks of batches b0 .. b0 + lane
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, upto, off);
                if (lane >= off) upto += x;
            }
            const unsigned behind = __ballot_sync(0xffffffffu, u < upto * items);
            if (behind || b0 + 32 >= a.B_kv) {
                const int l = behind ? __ffs(behind) - 1 : 31;
                n = max(1, __shfl_sync(0xffffffffu, mine, l));
                u -= (__shfl_sync(0xffffffffu, upto, l) - __shfl_sync(0xffffffffu, mine, l)) * items;
                p.b = b0 + l;
                break;
            }
            u -= __shfl_sync(0xffffffffu, upto, 31) * items;
        }
    }
    p.item = static_cast<int>(u / n);
    p.kb = static_cast<int>(u - static_cast<long long>(p.item) * n);
    return p;
}
// CTA `cta`'s first unit.  No CTA is without one but those behind the last.
__device__ __forceinline__ long long first_unit(const CrossArgs& a, long long total, int cta) {
    const long long n = total < a.ctas ? total : a.ctas;
    return cta >= n ? total : total / n * cta + total % n * cta / n;
}

// A run of key blocks of an item.
struct Segment {
    int b, h, pair;     // K/V batch and head, the tiles 2 pair and 2 pair + 1
    int len;            // the sequence's keys
    int k0, n, blocks;  // key blocks k0 .. k0 + n - 1 of `blocks`
    bool solo;          // one tile
    __device__ __forceinline__ bool whole() const { return n == blocks; }
    __device__ __forceinline__ int slot() const { return k0 > 0 ? 0 : 1; }  // of the CTA's two parts
};

// This CTA's segments, one after the other: every role goes through them on its own.
struct Walk {
    int b, item, kb, blocks, len;
    long long left;
    __device__ __forceinline__ explicit Walk(const CrossArgs& a) {
        if (a.stream) {
            const long long total = total_units(a), u = first_unit(a, total, blockIdx.x);
            left = first_unit(a, total, blockIdx.x + 1) - u;
            if (left > 0) {
                const UnitPlace p = unit_place(a, u);
                b = p.b, item = p.item, kb = p.kb;
                len = cross_length(a, b);
                blocks = cross_blocks(len);
            }
        } else {
            left = 0;  // rounds
        }
    }
    __device__ __forceinline__ bool next(const CrossArgs& a, Segment& s) {
        const int per = a.H_kv * a.n_pairs;
        if (a.stream) {
            if (left <= 0) return false;
            s.b = b, s.k0 = kb, s.blocks = blocks, s.len = len;
            s.n = static_cast<int>(left < blocks - kb ? left : blocks - kb);
            place(a, s, item);
            left -= s.n;
            kb = 0;
            if (++item == per && left > 0) {
                item = 0;
                len = cross_length(a, ++b);
                blocks = cross_blocks(len);
            }
            return true;
        }
        // whole items in alternating order
        const long long G = gridDim.x, x = left * G + ((left & 1) ? G - 1 - blockIdx.x : blockIdx.x);
        if (x >= static_cast<long long>(a.B_kv) * per) return false;
        ++left;
        s.b = static_cast<int>(x / per);
        s.len = cross_length(a, s.b);
        s.k0 = 0;
        s.n = s.blocks = cross_blocks(s.len);
        place(a, s, static_cast<int>(x - static_cast<long long>(s.b) * per));
        return true;
    }
    __device__ __forceinline__ static void place(const CrossArgs& a, Segment& s, int item) {
        s.h = item / a.n_pairs;
        s.pair = item - s.h * a.n_pairs;
        s.solo = 2 * s.pair + 1 >= a.tiles;
    }
};

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
        t.b = tile / a.tiles_b;
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

// A row's state (reference maximum m in log2 units, sum l) with its own attention's: the factors of the
// unnormalised O and of the own O, and the lse of both.
struct RowEnd {
    float f, f_own, lse;
};
__device__ __forceinline__ RowEnd row_end(const CrossArgs& a, float m, float l, size_t row, bool there) {
    constexpr float kLn2 = 0.69314718055994530942f, kLog2e = 1.4426950408889634f;
    RowEnd e;
    const bool any = !(l == 0.f);  // a NaN stays one
    const float own = a.lse_own && there ? a.lse_own[row] * kLog2e : -INFINITY;
    const float mine = any ? m + log2f(l) : -INFINITY;
    if (own == -INFINITY) {
        e.f = any ? 1.f / l : 0.f;
        e.f_own = 0.f;
        e.lse = mine * kLn2;
        return e;
    }
    const float top = fmaxf(mine, own);
    const float w = any ? exp2f(mine - top) : 0.f, w_own = exp2f(own - top), sum = w + w_own;
    e.f = any ? w / (sum * l) : 0.f;
    e.f_own = w_own / sum;
    e.lse = (top + log2f(sum)) * kLn2;
    return e;
}

// Floats of one part: O of its rows, then m and l.
__host__ __device__ inline size_t part_floats(int D, int part_rows) {
    return static_cast<size_t>(part_rows) * (D + 2);
}

}  // namespace
}  // namespace fa
