// kv4_decode.cu -- attention of the newest tokens of each request over its paged 4-bit
// cache (kv4.cuh): the serving form of the attention call, with its window and sinks.
//
// For the N_q newest tokens i of request b (positions lengths[b] - N_q + i) and a K/V head's
// group of G = H / H_kv query heads: softmax over the visible tokens of scale q . k, times v,
// with one pass over the codes and the running maximum and sum of each row.
//
// Bound by memory: a cached token is d / 2 + d / 16 bytes of K and of V, read once for all
// rows of its group; nothing else grows with the length.  What that leaves to arrange:
//   * Tensor work.  mma.m16n8k16 with the 16 cache tokens as the M side and the (up to 8)
//     query rows as N: S^T = K Q^T and O^T = V^T P^T.  Eight rows then fill the instruction,
//     where rows on the M side would leave half of it empty.  tcgen05's smallest M is 64 and
//     its operands come from shared memory: the codes would have to be expanded into it, 4
//     times their bytes, which costs more than the whole multiplication here.
//   * Expanding codes, which the integer pipe bounds before memory does.  K meets Q in fp16:
//     word & 0x000F000F and word & 0x00F000F0 are pairs of the subnormals u 2^-24 and 16 u 2^-24
//     as they stand, five operations for eight values; Q is scaled to fit (exactly), and the
//     codes' offset 8 costs nothing: the accumulators start at -8 sum_d q_d of each group of 32.
//     V meets P s, whose range only bf16 holds: (word >> 4 i) & 0x000F000F | 0x43004300 is a
//     pair of 128 + u, and one packed subtraction (exact) makes it u - 8.  (Taking 136 out by a
//     further product with P is slower, and 0 * NaN would carry a NaN scale from its own group's
//     outputs into the others'.)  Scales: K's multiply the group's accumulators in float; V's
//     multiply P in float, and the product is rounded to bf16 once, by at most 2^-8 of its value.
//     The row sum, and with it lse, adds the unrounded P.
//   * S^T to P^T.  The accumulator layout of S^T transposed is the operand layout of P^T:
//     one movmatrix per 8 x 8 block.
//   * Copies.  Each warp runs its own ring of 16-token tiles, filled by 16-byte asynchronous
//     copies of its lanes (a tile never crosses a page); no barrier between warps.
//   * Splitting.  The units of 64 or 128 tokens (32 a warp) of all requests and heads form one list that is cut
//     evenly over the resident CTAs, whatever the lengths are: a CTA's share may cover several
//     requests or a part of one.  Whole requests are written at once; parts go to the
//     workspace, and decode_join_kernel adds them.  The cut depends on the lengths alone, so
//     results do not change from call to call.
// Measured (H32 H_kv8 d128): 64 requests of 1000 to 32768 tokens 294 us (4.2 TB/s, 63% of the copy
// rate).  0.61 instructions a cycle and scheduler, the integer pipe 60% busy: neither is full, and what
// limits is the latency of a step's chain (codes, product, maximum, exponentials, product) with three
// warps a scheduler (twelve of 168 registers an SM: eight took 8% longer, sixteen with spills 10%; rings of
// three steps 1%).  One request of 16000 tokens 15.1 us.
// More than 16 rows of a K/V head read and expand its codes once for every 16 of them: the same batch
// with 1, 2, 4 and 8 new tokens (4, 8, 16 and 32 rows) 294, 304, 429 and 842 us.  A window of 4096 and 4
// sinks 85 us, d = 64 193 us.
#include <atomic>
#include <cmath>
#include <type_traits>

#include "kv4.cuh"
#include "layer_ops.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kTiles = 2;                      // tiles of 16 tokens that a warp works on together
constexpr int kStages = 2;                     // ring of such steps per warp
constexpr int kNowhere = kMaxTokens;           // the "token" of a tile that is not there: hidden to every row
constexpr float kTau = 8.0f;        // lazy rescale: the reference moves by more than this (log2)
constexpr int kMaxCtas = 1024;

template <int D>
struct TileCfg {
    static constexpr int kCodes = kTileTokens * D / 2;       // bytes of K or V codes
    static constexpr int kScales = kTileTokens * (D / 32) * 2;
    static constexpr int kOffV = kCodes;
    static constexpr int kOffKs = 2 * kCodes;
    static constexpr int kOffVs = 2 * kCodes + kScales;
    static constexpr int kBytes = 2 * (kCodes + kScales);
};

// Tiles of 16 tokens that a request's queries read between them: `sink` tiles from the first
// token on, then tiles [start, end).
struct Reach {
    int len, sink, start, n_tiles, n_units;
};

template <int UNIT>  // tiles of a unit
__device__ __forceinline__ Reach reach_of(const DecodeArgs& a, long long b) {
    Reach r;
    r.len = a.lengths[b];
    const long long cap = static_cast<long long>(a.cache.max_blocks) << a.cache.page_log2;
    if (r.len < 0 || r.len > cap) {
        atomicCAS(a.ctl.status, kDevOk, kDevIndex);
        r.len = r.len < 0 ? 0 : static_cast<int>(cap);
    }
    int lo = 0;
    if (a.window > 0) lo = max(0, static_cast<int>(max(-1ll, static_cast<long long>(r.len) - a.N_q + 1 - a.window)));
    r.sink = (min(a.sinks, lo) + kTileTokens - 1) / kTileTokens;
    r.start = max(r.sink, lo / kTileTokens);
    const int end = (r.len + kTileTokens - 1) / kTileTokens;
    r.n_tiles = r.sink + max(0, end - r.start);
    if (r.len == 0) r.n_tiles = 0;
    r.n_units = (r.n_tiles + UNIT - 1) / UNIT;
    return r;
}

// Workspace: prefix sums of the requests' units, then per CTA two parts (its first and its
// last entry), each ROWS x (D + 2) floats: O unnormalised, then m and l.
struct Work {
    long long* prefix;  // [B + 1]
    float* parts;
};
__host__ __device__ inline size_t prefix_bytes(int B) {
    return (static_cast<size_t>(B) + 1 + 1) / 2 * 2 * sizeof(long long);
}

__device__ __forceinline__ long long share_start(long long total, int ctas, int c) { return total * c / ctas; }
// The CTA whose share holds unit u.
__device__ __forceinline__ int owner_of(long long total, int ctas, long long u) {
    return static_cast<int>(((u + 1) * ctas - 1) / total);
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                         const float (&c)[4]) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                        const float (&c)[4]) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// nibble i of both halves of w as bf16 pair 128 + u
__device__ __forceinline__ uint32_t expand(uint32_t w, int i) { return ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u; }
// nibbles 0 (u) and 1 (16 u) of both halves of w as fp16 pairs, times 2^-24: subnormals
__device__ __forceinline__ uint32_t tiny(uint32_t w, int i) { return w & (i ? 0x00F000F0u : 0x000F000Fu); }
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// N neighbouring words (1, 2 or 4) as one load
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
    if constexpr (N == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x;
        w[1] = v.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}

// NT: tiles of 8 query rows that share the expanded codes (1 or 2); kWarps: warps of a CTA, whose
// resident ones are twelve an SM (eight for NT = 2).
template <int D, int NT, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, (NT == 1 ? 12 : 8) / kWarps)
    decode_kv4_kernel(const __grid_constant__ DecodeArgs a, const Work work, const int row_tiles) {
    using T = TileCfg<D>;
    constexpr int G = D / 32;      // groups of 32 values
    constexpr int ROWS = 8 * NT;
    constexpr int kThreads = 32 * kWarps, kUnitTiles = kWarps * kTiles;
    extern __shared__ __align__(128) uint8_t smem[];  // the warps' rings; at an entry's end their results
    __shared__ long long s_sum[kWarps];
    __shared__ long long s_found[2];  // request of the first unit, units before it
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    uint8_t* const ring = smem + warp * (kStages * kTiles * T::kBytes);
    float* const results = reinterpret_cast<float*>(smem);
    griddep_wait();
    griddep_launch_dependents();

    // units before each request: a scan over the batch, a run of requests per thread
    const int per = (a.B + kThreads - 1) / kThreads;
    const int b0 = min(a.B, static_cast<int>(threadIdx.x) * per), b1 = min(a.B, b0 + per);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += reach_of<kUnitTiles>(a, b).n_units;
    long long incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += up;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    long long before = incl - mine, per_head = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += s_sum[w];
        per_head += s_sum[w];
    }
    const int entries = a.cache.H_kv * row_tiles;  // per request
    const long long total = per_head * entries;
    const int ctas = static_cast<int>(total < gridDim.x ? total : gridDim.x);
    if (blockIdx.x == 0) {  // for the join
        long long at = before;
        for (int b = b0; b < b1; ++b) {
            work.prefix[b] = at;
            at += reach_of<kUnitTiles>(a, b).n_units;
        }
        if (b1 == a.B && b0 < b1) work.prefix[a.B] = at;
    }
    if (static_cast<int>(blockIdx.x) >= ctas) return;
    const long long u_begin = share_start(total, ctas, blockIdx.x), u_end = share_start(total, ctas, blockIdx.x + 1);
    if (u_begin >= before * entries && u_begin < (before + mine) * entries) {
        long long at = before;
        for (int b = b0; b < b1; ++b) {
            const int n = reach_of<kUnitTiles>(a, b).n_units;
            if (u_begin < (at + n) * entries) {
                s_found[0] = b;
                s_found[1] = at;
                break;
            }
            at += n;
        }
    }
    __syncthreads();
    int b = static_cast<int>(s_found[0]);
    long long b_first = s_found[1] * entries;  // first unit of request b

    const uint32_t half_sel = (g & 1) ? 0x3244u : 0x1044u;  // this token's half of a pair's word, as a float
    const int rows_all = a.H / a.cache.H_kv * a.N_q;  // query rows of a K/V head
    for (long long u = u_begin; u < u_end;) {
        const Reach R = reach_of<kUnitTiles>(a, b);
        if (R.n_units == 0) {
            ++b;
            continue;
        }
        const long long rel = u - b_first;
        const int entry = static_cast<int>(rel / R.n_units), k0 = static_cast<int>(rel % R.n_units);
        const int take = static_cast<int>(min(static_cast<long long>(R.n_units - k0), u_end - u));
        const int kv = entry / row_tiles, row0 = (entry % row_tiles) * ROWS;
        const bool whole = k0 == 0 && take == R.n_units;
        const bool is_first = u == u_begin;

        // this warp's tiles: kTiles neighbours in every unit of the list [8 k0, 8 (k0 + take))
        const int x0 = k0 * kUnitTiles + warp * kTiles, x1 = min(R.n_tiles, (k0 + take) * kUnitTiles);
        const int n_mine = x0 < x1 ? (x1 - x0 + kUnitTiles - 1) / kUnitTiles : 0;  // steps
        const int shift = R.start - R.sink;
        const int* table = a.cache.table + static_cast<long long>(b) * a.cache.max_blocks;
        const int page_mask = (1 << a.cache.page_log2) - 1;
        const size_t head_row = static_cast<size_t>(kv) << a.cache.page_log2;
        const size_t page_rows = static_cast<size_t>(a.cache.H_kv) << a.cache.page_log2;
        const uint8_t* k_src = a.cache.codes[0] + head_row * (D / 2) + lane * 16;
        const uint8_t* v_src = a.cache.codes[1] + head_row * (D / 2) + lane * 16;
        constexpr int kPieces = T::kScales / 16;  // lanes below kPieces copy K's scales, the next ones V's
        const uint8_t* s_src = reinterpret_cast<const uint8_t*>(a.cache.scales[lane >= kPieces ? 1 : 0]) +
                               head_row * (D / 16) + (lane % kPieces) * 16;
        // first token and page of tile j of step i; kNowhere where there is none
        auto place = [&](int i, int j, int& tok, int& page) {
            const int x = x0 + i * kUnitTiles + j;
            tok = kNowhere;
            page = -1;
            if (x >= x1) return;
            const int t0 = kTileTokens * (x < R.sink ? x : x + shift);
            page = __ldg(table + (t0 >> a.cache.page_log2));
            if (static_cast<unsigned>(page) < static_cast<unsigned>(a.cache.n_pages)) {
                tok = t0;
            } else if (lane == 0) {
                atomicCAS(a.ctl.status, kDevOk, kDevIndex);
            }
        };
        // the lanes' copies of a tile from its row of the cache on, and of both tiles of a step: the
        // second is mostly the next one in the same page.  One that is not there is not copied.
        auto copy_row = [&](uint32_t dst, const uint8_t* ks, const uint8_t* vs, const uint8_t* ss) {
#pragma unroll
            for (int x = 0; x < T::kCodes; x += 512) {
                cp_async16(dst + x + lane * 16, ks + x);
                cp_async16(dst + T::kOffV + x + lane * 16, vs + x);
            }
            if (lane < 2 * kPieces) cp_async16(dst + T::kOffKs + lane * 16, ss);
        };
        auto copy = [&](uint32_t dst, const int (&tok)[kTiles], const int (&page)[kTiles]) {
            bool next = false;
#pragma unroll
            for (int j = 0; j < kTiles; ++j) {
                if (next || tok[j] == kNowhere) {
                    next = false;
                    continue;
                }
                const size_t row = page[j] * page_rows + (tok[j] & page_mask);
                const uint8_t* ks = k_src + row * (D / 2);
                const uint8_t* vs = v_src + row * (D / 2);
                const uint8_t* ss = s_src + row * (D / 16);
                copy_row(dst + j * T::kBytes, ks, vs, ss);
                if (j + 1 < kTiles && tok[j + 1] == tok[j] + kTileTokens && page[j + 1] == page[j]) {
                    copy_row(dst + (j + 1) * T::kBytes, ks + T::kCodes, vs + T::kCodes, ss + T::kScales);
                    next = true;
                }
            }
        };
        const uint32_t ring0 = smem_u32(ring);
        int toks[kStages][kTiles], next_tok[kTiles], next_page[kTiles];  // toks[s]: the s-th step from here on
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) {
#pragma unroll
            for (int j = 0; j < kTiles; ++j) place(i, j, toks[i][j], next_page[j]);
            copy(ring0 + i * kTiles * T::kBytes, toks[i], next_page);
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
#pragma unroll
        for (int j = 0; j < kTiles; ++j) place(kStages - 1, j, next_tok[j], next_page[j]);
        int stage = 0, fill = kStages - 1;  // ring positions of this step and of the one to be fetched

        // Q^T fragments in fp16, in the order of d that a lane's K words have.  A row is scaled by
        // a power of two to below 2^14 (back in c_row), and where K's nibble comes as 16 u, q is
        // divided by 16: its bf16 values are exact down to 2^-26 of the largest and off by 2^-34 of
        // it at most below.
        uint32_t qf[NT][D / 16][2];
        float q0[NT][G][2];  // -8 sum of q by group, times 2^-24: what takes the codes' 8 out
        float c_row[NT][2];  // scale * log2(e) * 2^24 over the rows' factors
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = row0 + 8 * n + g;
            const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                               ((static_cast<size_t>(b) * a.H + static_cast<size_t>(kv) * (a.H / a.cache.H_kv)) * a.N_q + r) * D);
            uint4 w[G];
            uint32_t top = 0;  // largest magnitude, as bits
#pragma unroll
            for (int c = 0; c < G; ++c) {
                w[c] = r < rows_all ? __ldg(src + 4 * c + t) : make_uint4(0, 0, 0, 0);
                const uint32_t u[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) top = max(top, max(u[i] & 0x7FFFu, (u[i] >> 16) & 0x7FFFu));
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // 2^(13 - exponent), kept within float's normal range (a row of zeros or subnormals
            // stays small; infinities and NaN stay what they are)
            const int ex = static_cast<int>(top >> 7) - 127;
            const int up = min(max(13 - ex, -100), 100);
            const float f = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
            const float back = a.c_log2 * __uint_as_float(static_cast<uint32_t>(127 - up) << 23) * 0x1p24f;
#pragma unroll
            for (int c = 0; c < G; ++c) {
                // values 32 c + 8 t + 0..7 of row g: pairs (i, i + 4) for nibble i
                const float q[8] = {bf_lo(w[c].x) * f, bf_hi(w[c].x) * f, bf_lo(w[c].y) * f, bf_hi(w[c].y) * f,
                                    bf_lo(w[c].z) * f, bf_hi(w[c].z) * f, bf_lo(w[c].w) * f, bf_hi(w[c].w) * f};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    qf[n][2 * c + i / 2][i % 2] = (i & 1) ? pack_f16x2(q[i] * 0.0625f, q[i + 4] * 0.0625f)
                                                          : pack_f16x2(q[i], q[i + 4]);
                float sum = ((q[0] + q[1]) + (q[2] + q[3])) + ((q[4] + q[5]) + (q[6] + q[7]));
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                // from row g's lanes to those of columns 2t, 2t + 1
                q0[n][c][0] = -0x1p-21f * __shfl_sync(0xffffffffu, sum, 8 * t);
                q0[n][c][1] = -0x1p-21f * __shfl_sync(0xffffffffu, sum, 8 * t + 4);
            }
            c_row[n][0] = __shfl_sync(0xffffffffu, back, 8 * t);
            c_row[n][1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);
        }
        // positions of the rows of this lane's columns
        int last[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) last[n][e] = R.len - a.N_q + (row0 + 8 * n + 2 * t + e) % a.N_q;
        // a tile from token `tok` on is seen whole by every row if it ends by the first row's
        // position, and starts inside the last row's window or ends among the sinks
        const int whole_to = R.len - a.N_q - (kTileTokens - 1);
        const int whole_from = a.window > 0 ? R.len - a.window : 0;

        float o[NT][G][2][4];   // O^T: rows 32 c + 4 g + {0, 1 | 2, 3}, columns 2t, 2t + 1
        float m[NT][2], ref[NT][2], l[NT][2];  // reference maximum; the same or 0 for -inf; sum
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int c = 0; c < G; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) o[n][c][i / 4][i % 4] = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[n][e] = -INFINITY;
                ref[n][e] = l[n][e] = 0.f;
            }
        }

        for (int i = 0; i < n_mine; ++i) {
            // the ring position that step i - 1 has left, which every lane has read, takes step
            // i + kStages - 1
            copy(ring0 + fill * kTiles * T::kBytes, next_tok, next_page);
#pragma unroll
            for (int j = 0; j < kTiles; ++j) toks[kStages - 1][j] = next_tok[j];
            asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll
            for (int j = 0; j < kTiles; ++j) place(i + kStages, j, next_tok[j], next_page[j]);
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
            __syncwarp();
            const uint8_t* st = ring + stage * (kTiles * T::kBytes);
            // S^T of the tiles' tokens, in log2 units; hidden tokens by selection, whatever their
            // bytes hold
            float x[kTiles][NT][4];
            bool edge[kTiles];
#pragma unroll
            for (int j = 0; j < kTiles; ++j) {
                const uint8_t* sj = st + j * T::kBytes;
                const int tok = toks[0][j];
                uint32_t kw[2][G], ks[2][G / 2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    load_words(sj + (g + 8 * r) * (D / 2) + t * (D / 8), kw[r]);
                    load_words(sj + T::kOffKs + (g + 8 * r) * (D / 16), ks[r]);
                }
#pragma unroll
                for (int c = 0; c < G; ++c) {
                    uint32_t f[2][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int r = 0; r < 4; ++r) f[h][r] = tiny(h ? kw[r & 1][c] >> 8 : kw[r & 1][c], r / 2);
                    const float s0 = (c & 1) ? bf_hi(ks[0][c / 2]) : bf_lo(ks[0][c / 2]);
                    const float s1 = (c & 1) ? bf_hi(ks[1][c / 2]) : bf_lo(ks[1][c / 2]);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float init[4] = {q0[n][c][0], q0[n][c][1], q0[n][c][0], q0[n][c][1]};
                        float acc[4];
                        mma_f16(acc, f[0], qf[n][2 * c][0], qf[n][2 * c][1], init);
                        mma_f16(acc, f[1], qf[n][2 * c + 1][0], qf[n][2 * c + 1][1], acc);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            x[j][n][e] = c == 0 ? acc[e] * (e < 2 ? s0 : s1) : fmaf(acc[e], e < 2 ? s0 : s1, x[j][n][e]);
                    }
                }
                edge[j] = tok > whole_to || (tok < whole_from && tok + kTileTokens > a.sinks);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[j][n][e] *= c_row[n][e & 1];
                if (edge[j]) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int key = tok + g + (e < 2 ? 0 : 8), i_pos = last[n][e & 1];
                            const bool seen = key <= i_pos && (a.window == 0 || key > i_pos - a.window || key < a.sinks);
                            if (!seen) x[j][n][e] = -INFINITY;
                        }
                }
            }
            // the rows' reference maxima, moved only when a score passes one by more than kTau
            float top[NT][2];
            bool over = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    top[n][e] = fmaxf(x[0][n][e], x[0][n][e + 2]);
#pragma unroll
                    for (int j = 1; j < kTiles; ++j) top[n][e] = fmaxf(top[n][e], fmaxf(x[j][n][e], x[j][n][e + 2]));
                    over |= top[n][e] > m[n][e] + kTau;
                }
            if (__any_sync(0xffffffffu, over)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float v = top[n][e];
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
                        if (v > m[n][e]) {
                            const float alpha = ex2_approx(m[n][e] - v);  // 0 from -inf
                            m[n][e] = ref[n][e] = v;
                            l[n][e] *= alpha;
#pragma unroll
                            for (int c = 0; c < G; ++c)
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    o[n][c][h][e] *= alpha;
                                    o[n][c][h][e + 2] *= alpha;
                                }
                        }
                    }
            }
            // P, rows of tokens g and g + 8, and O^T += V^T (P s)^T
#pragma unroll
            for (int j = 0; j < kTiles; ++j) {
                const uint8_t* sj = st + j * T::kBytes;
                float p[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        p[n][e] = ex2_approx(x[j][n][e] - ref[n][e & 1]);
                        l[n][e & 1] += p[n][e];
                    }
                uint32_t vw[2][G];  // codes: the first token's G / 2 words, then the second's
                uint32_t vs[2][G];  // scales of token pairs g / 2, 4 + g / 2
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    load_words(sj + T::kOffV + (r * 32 + lane) * (D / 8), vw[r]);
                    load_words(sj + T::kOffVs + (r * 4 + g / 2) * (D / 8), vs[r]);
                }
                // (a branch for each scale, within the loops, took 2% longer)
                auto pv = [&](auto edge_c) {
#pragma unroll
                    for (int c = 0; c < G; ++c) {
                        uint32_t f[2][4];
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            // 16-bit words of this lane's two tokens side by side
                            const uint32_t w = __byte_perm(vw[r][c / 2], vw[r][G / 2 + c / 2], (c & 1) ? 0x7632 : 0x5410);
#pragma unroll
                            for (int e = 0; e < 4; ++e) f[e / 2][2 * r + (e & 1)] = sub_bf16x2(expand(w, e), 0x43084308u);
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            // P times the group's scale, transposed into the operand of the second product
                            uint32_t ps[2];
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                const float s = __uint_as_float(__byte_perm(vs[r][c], 0u, half_sel));
                                float y0 = p[n][2 * r] * s, y1 = p[n][2 * r + 1] * s;
                                if constexpr (decltype(edge_c)::value) {  // a hidden token's scale may be anything
                                    if (x[j][n][2 * r] == -INFINITY) y0 = 0.f;
                                    if (x[j][n][2 * r + 1] == -INFINITY) y1 = 0.f;
                                }
                                ps[r] = transpose8x8(pack_bf16x2(y0, y1));
                            }
                            mma_bf16(o[n][c][0], f[0], ps[0], ps[1], o[n][c][0]);
                            mma_bf16(o[n][c][1], f[1], ps[0], ps[1], o[n][c][1]);
                        }
                    }
                };
                if (edge[j])
                    pv(std::true_type{});
                else
                    pv(std::false_type{});
            }
            __syncwarp();  // every lane has read the step
            fill = stage;
            stage = stage == kStages - 1 ? 0 : stage + 1;
#pragma unroll
            for (int s = 0; s < kStages - 1; ++s)
#pragma unroll
                for (int j = 0; j < kTiles; ++j) toks[s][j] = toks[s + 1][j];
        }

        __syncthreads();  // the results take the rings' place
        // the warps' states side by side, then one sum per value
        constexpr int kRowFloats = D + 2;
        float* mine_r = results + warp * ROWS * kRowFloats;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = l[n][e];
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                float* row = mine_r + (8 * n + 2 * t + e) * kRowFloats;
                if (g == 0) {
                    row[D] = m[n][e];
                    row[D + 1] = sum;
                }
#pragma unroll
                for (int c = 0; c < G; ++c) {
                    row[32 * c + 4 * g] = o[n][c][0][e];
                    row[32 * c + 4 * g + 1] = o[n][c][0][e + 2];
                    row[32 * c + 4 * g + 2] = o[n][c][1][e];
                    row[32 * c + 4 * g + 3] = o[n][c][1][e + 2];
                }
            }
        __syncthreads();
        for (int x = threadIdx.x; x < ROWS * (D / 4); x += kThreads) {
            const int r = x / (D / 4), c4 = 4 * (x % (D / 4));
            if (row0 + r >= rows_all) continue;
            float mm = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, results[(w * ROWS + r) * kRowFloats + D]);
            const float ref = mm == -INFINITY ? 0.f : mm;
            float acc[4] = {0.f, 0.f, 0.f, 0.f}, sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float* row = results + (w * ROWS + r) * kRowFloats;
                const float f = ex2_approx(row[D] - ref);
                sum = fmaf(f, row[D + 1], sum);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[e] = fmaf(f, row[c4 + e], acc[e]);
            }
            if (whole) {
                const size_t out = (static_cast<size_t>(b) * a.H + static_cast<size_t>(kv) * (a.H / a.cache.H_kv)) * a.N_q + row0 + r;
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + out * D + c4) =
                    make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
                if (c4 == 0 && a.lse != nullptr)
                    a.lse[out] = sum == 0.f ? -INFINITY : (mm + log2f(sum)) * 0.69314718055994530942f;
            } else {
                float* part = work.parts + (static_cast<size_t>(2 * blockIdx.x + (is_first ? 0 : 1)) * ROWS + r) * kRowFloats;
#pragma unroll
                for (int e = 0; e < 4; ++e) part[c4 + e] = acc[e];
                if (c4 == 0) {
                    part[D] = mm;
                    part[D + 1] = sum;
                }
            }
        }
        __syncthreads();
        u += take;
        if (u == b_first + static_cast<long long>(R.n_units) * entries) {
            b_first = u;
            ++b;
        }
    }
}

// One block per query row: adds the parts of requests that were cut, and writes the rows of
// requests without tokens.
template <int D>
__global__ void __launch_bounds__(256)
    decode_join_kernel(const __grid_constant__ DecodeArgs a, const Work work, const int row_tiles, const int rows_tile,
                       const int ctas_main) {
    constexpr int kRowFloats = D + 2;
    __shared__ float s_w[2 * 256];
    __shared__ float s_o[8][D];
    __shared__ float s_red[2][8];
    griddep_wait();
    const int row = blockIdx.x;  // of B * H * N_q
    const int G = a.H / a.cache.H_kv;
    const int per_b = a.H * a.N_q, per_kv = G * a.N_q;
    const int b = row / per_b, kv = row % per_b / per_kv, r = row % per_kv;
    const int entries = a.cache.H_kv * row_tiles, entry = kv * row_tiles + r / rows_tile;
    const long long p0 = work.prefix[b], p1 = work.prefix[b + 1];
    const long long n = p1 - p0, total = work.prefix[a.B] * entries;
    if (n == 0) {
        for (int x = threadIdx.x; x < D; x += blockDim.x) static_cast<uint16_t*>(a.o)[static_cast<size_t>(row) * D + x] = 0;
        if (threadIdx.x == 0 && a.lse != nullptr) a.lse[row] = -INFINITY;
        return;
    }
    const int ctas = static_cast<int>(total < ctas_main ? total : ctas_main);
    const long long u0 = p0 * entries + entry * n, u1 = u0 + n;
    const int c0 = owner_of(total, ctas, u0), c1 = owner_of(total, ctas, u1 - 1);
    if (c0 == c1) {
        return;  // written whole by its CTA
    }
    const int parts = c1 - c0 + 1;
    const bool first_of_c0 = share_start(total, ctas, c0) == u0;
    const int rt = r % rows_tile;
    auto part_at = [&](int i) {
        const int slot = 2 * (c0 + i) + (i == 0 && !first_of_c0 ? 1 : 0);
        return work.parts + (static_cast<size_t>(slot) * rows_tile + rt) * kRowFloats;
    };
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    // the row's maximum over its parts
    float mm = -INFINITY;
    for (int i = threadIdx.x; i < parts; i += blockDim.x) mm = fmaxf(mm, part_at(i)[D]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, off));
    if (lane == 0) s_red[0][warp] = mm;
    __syncthreads();
    mm = s_red[0][0];
#pragma unroll
    for (int w = 1; w < 8; ++w) mm = fmaxf(mm, s_red[0][w]);
    const float ref = mm == -INFINITY ? 0.f : mm;
    float sum = 0.f;
    for (int i = threadIdx.x; i < parts; i += blockDim.x) {
        const float* p = part_at(i);
        const float f = ex2_approx(p[D] - ref);
        if (i < 512) s_w[i] = f;
        sum = fmaf(f, p[D + 1], sum);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (lane == 0) s_red[1][warp] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) sum += s_red[1][w];
    // warps take parts in turn, a lane D / 32 neighbouring values
    constexpr int V = D / 32;
    float acc[V];
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.f;
#pragma unroll 4
    for (int i = warp; i < parts; i += 8) {
        const float* p = part_at(i);
        const float f = i < 512 ? s_w[i] : ex2_approx(p[D] - ref);
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            const float2 x = *reinterpret_cast<const float2*>(p + lane * V + e);
            acc[e] = fmaf(f, x.x, acc[e]);
            acc[e + 1] = fmaf(f, x.y, acc[e + 1]);
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) s_o[warp][lane * V + e] = acc[e];
    __syncthreads();
    if (threadIdx.x < D / 2) {
        float x = 0.f, y = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            x += s_o[w][2 * threadIdx.x];
            y += s_o[w][2 * threadIdx.x + 1];
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        reinterpret_cast<uint32_t*>(a.o)[static_cast<size_t>(row) * (D / 2) + threadIdx.x] = pack_bf16x2(x * inv, y * inv);
        if (threadIdx.x == 0 && a.lse != nullptr)
            a.lse[row] = sum == 0.f ? -INFINITY : (mm + log2f(sum)) * 0.69314718055994530942f;
    }
}

template <int D, int NT, int kWarps>
cudaError_t launch_impl(const DecodeArgs& a, cudaStream_t s) {
    constexpr int kRings = kWarps * kStages * kTiles * TileCfg<D>::kBytes;
    constexpr int kResults = kWarps * 8 * NT * (D + 2) * static_cast<int>(sizeof(float));
    constexpr int kSmem = kRings > kResults ? kRings : kResults;
    // CTAs that are resident together, per device; asked once
    static std::atomic<int> resident[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int ctas = dev < 64 ? resident[dev].load() : 0;
    if (ctas == 0) {
        int sms = 0, per_sm = 0;
        e = cudaFuncSetAttribute(decode_kv4_kernel<D, NT, kWarps>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess)
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, decode_kv4_kernel<D, NT, kWarps>, 32 * kWarps, kSmem);
        if (e != cudaSuccess) return e;
        ctas = sms * (per_sm < 1 ? 1 : per_sm);
        if (ctas > kMaxCtas) ctas = kMaxCtas;
        if (dev < 64) resident[dev].store(ctas);
    }
    const int rows = a.H / a.cache.H_kv * a.N_q;
    const int row_tiles = (rows + 8 * NT - 1) / (8 * NT);
    // no more CTAs than units that the tables could hold
    const long long most_units = ((static_cast<long long>(a.cache.max_blocks) << a.cache.page_log2) / (16 * kWarps * kTiles) + 1) *
                                 a.B * a.cache.H_kv * row_tiles;
    const long long grid = ctas < most_units ? ctas : most_units;
    Work w;
    w.prefix = static_cast<long long*>(a.workspace);
    w.parts = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + prefix_bytes(a.B));
    e = launch_pdl(decode_kv4_kernel<D, NT, kWarps>, dim3(static_cast<unsigned>(grid)), dim3(32 * kWarps), kSmem, s, a, w,
                   row_tiles);
    if (e != cudaSuccess) return e;
    return launch_pdl(decode_join_kernel<D>, dim3(static_cast<unsigned>(a.B * a.H * a.N_q)), dim3(256), 0, s, a, w,
                      row_tiles, 8 * NT, static_cast<int>(grid));
}

}  // namespace

size_t decode_kv4_workspace_bytes(int B, int H, int H_kv, int N_q, int d) {
    const int rows = H / H_kv * N_q;
    return prefix_bytes(B) + static_cast<size_t>(2 * kMaxCtas) * (rows <= 8 ? 8 : 16) * (d + 2) * sizeof(float);
}

namespace {
// With about as many heads to attend to as SMs or more, CTAs of two warps (their entries end apart
// from one another); with fewer, of four, which leave half the parts to join.  Two against four, 8
// K/V heads of d = 128: 64 requests of 1000 to 32768 tokens 294 us against 301, 64 of 100 to 1000 32
// against 37, 16 of 2000 to 8000 34.1 against 34.8; 8 of 4000 to 8000 26.8 against 25.8, 4 of 8000
// 22.1 against 21.8, one of 16000 16.6 against 15.1.
template <int D, int NT>
cudaError_t launch_warps(const DecodeArgs& a, cudaStream_t s) {
    const bool many = static_cast<long long>(a.B) * a.cache.H_kv >= 128;
    return many ? launch_impl<D, NT, 2>(a, s) : launch_impl<D, NT, 4>(a, s);
}
}  // namespace

cudaError_t launch_decode_kv4(const DecodeArgs& a, int d, cudaStream_t s) {
    const int rows = a.H / a.cache.H_kv * a.N_q;
    if (d == 64) return rows <= 8 ? launch_warps<64, 1>(a, s) : launch_warps<64, 2>(a, s);
    return rows <= 8 ? launch_warps<128, 1>(a, s) : launch_warps<128, 2>(a, s);
}

}  // namespace fa
