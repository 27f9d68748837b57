// cross_fwd_sm103.cu -- forward of attention to another sequence's keys (an encoder's states, a prefix
// that requests share) on the sm_103a tensor core (tcgen05 + TMEM + TMA).
//
//     O = softmax(scale Q K^T over the keys j < len_b) V,  lse = m + ln l,
// by the online softmax of the plain forward (fwd_sm103.cu): a running reference maximum, sum and
// unnormalised output a row, lazily rescaled.  Optionally merged with (o_own, lse_own), the same queries'
// attention to other keys: lse = ln(e^lse + e^lse_own), O weighted by e^(lse_x - lse).  That state is the one that
// the rows begin with (m = lse_own log2 e, l = 1, O = o_own), which costs a load of o_own and no pass of its own.
//
// What bounds it, and the split taken for it:
//   * Many rows on many keys: the tensor pipe.  Two query tiles a CTA in ping-pong share every K and V block, as
//     in the plain forward: 3,050 cycles for a pair of blocks at d = 128 (2,048 of the pipe), 1,640 TFLOP/s at
//     16 x 16384 x 16384.
//   * Many rows on few keys (2 x 16384 video tokens on 77 to 512, one to four blocks): an item's end, 3,600 cycles of
//     its softmax warpgroups (O's last product, its way out, the next scores), beside 3,050 for each block of keys.  O
//     leaves in boxes by TMA, so that the warps go on while it is stored: 101 -> 95 us by that step, 88 now, floor 42.
//   * Few rows on many keys: HBM, at the rate that 152 SMs can have loads in flight.  The key blocks of all items
//     are cut into equal runs (64 ragged single tokens on 500-8192 keys: 175 us, 96% of the copy rate), whose
//     float32 parts a join adds up in a fixed order.
//   * Few rows on few keys: latency: 7.3 us for 10 x 3 tokens of 12 / 4 heads on 500 to 777 keys, 8.6 for one token of
//     32 / 8 heads on 1500.  Of 8.2 us (one token of 16 heads on 1500 keys, which takes no tiles any more) the start
//     took 0.3, the segments 0.7, the first loads 0.7 to 1.5, a block 1, joining in a cluster 1.  Much of each is
//     instructions fetched for the first time.
#include <type_traits>

#include "cross_fwd.cuh"
#include "tma_host.h"

namespace fa {
namespace {

constexpr int kThreads = 384;
constexpr size_t kCutBytes = kMaxCtas * sizeof(int4);

template <int D>
struct Cfg {
    static constexpr int kStages = D == 64 ? 4 : 2;  // 128 KB of K and V either way
    static constexpr int kChunks = D / 64;           // 128-byte swizzle columns per row
    static constexpr int kChunkBytes = 128 * 128;
    static constexpr int kTileBytes = kChunks * kChunkBytes;
    static constexpr int kOffQ = 0;                  // two tiles
    static constexpr int kOffK = 2 * kTileBytes;
    static constexpr int kOffV = kOffK + kStages * kTileBytes;
    static constexpr int kOffO = kOffV + kStages * kTileBytes;  // two boxes of 32 rows x 64 bytes a softmax warp
    static constexpr int kSmemAlloc = kOffO + 8 * 4096 + 1024;
    static constexpr uint32_t kColS = 0, kColO = 256;  // + 128, + D for the second warpgroup
    static constexpr uint32_t kTmemCols = 512;
    static constexpr uint32_t kIdescS = idesc_bf16(kBM, kBN, false, false);
    static constexpr uint32_t kIdescO = idesc_bf16(kBM, D, false, true);
};
static_assert(Cfg<128>::kSmemAlloc + 2000 <= 232448, "smem");

// Columns of S and P that a block with `valid` keys takes: a sequence's end of up to 32 or 64 keys has its own softmax
// (6 x 2629 queries of 16 heads on 4 keys 26.6 -> 19.2 us, 2 x 16384 on 50 62.4 -> 52.1; one for 64 alone 22.3 and
// 51.7; asked for before the usual one 2 x 8192 on 2048 keys take 177.8 us instead of 175.4).
__device__ __forceinline__ int columns_of(int valid) { return valid <= 32 ? 32 : valid <= 64 ? 64 : kBN; }

constexpr int kSegments = 8;   // ring of segments
constexpr int kReaders = 10;   // the loading thread, the MMA thread, 8 softmax warps
template <int STAGES>
struct Bars {
    uint64_t seg_full[kSegments], seg_empty[kSegments];
    uint64_t q_full[2], q_free[2];  // of a tile's Q: landed; read by its last S
    uint64_t kv_full[STAGES], kv_empty[STAGES];
    uint64_t s_full[2], p_half[2], p_full[2], o_done[2];
    uint64_t merge_ml, merge_done;  // one tile: warpgroup 1's state is in shared memory; its O was read
    uint64_t drain;
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z, int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

// 32 columns of this thread's row of the accumulator at `first`, weighted, and with w1 != 0 for any row (two) of
// that at `second`.
__device__ __forceinline__ void weighted32(uint32_t first, float w0, uint32_t second, float w1, bool two, float (&x)[32]) {
    uint32_t r[32];
    tmem_ld32(first, r);
#pragma unroll
    for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(r[e]) * w0;
    if (two) {
        tmem_ld32(second, r);
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = fmaf(__uint_as_float(r[e]), w1, x[e]);
    }
}

// A warp's rows of O as bf16 from TMEM to global memory, each lane its own: row `at` of o (-1: none), the weights of
// the accumulator(s) its own.  For tiles that are packed or alone, which a warp stores once or twice: the time is
// that of fetching the instructions.  (Through lanes that exchange their columns for runs of 64 bytes 64 tokens of
// 16 heads took 25.7 us instead of 23.7, of 32 / 8 heads 27.0 instead of 24.4, both on keys so few that they take no
// tiles any more; a lone tile of 128 rows 31.3 instead of 32.4.)
template <int D>
__device__ __forceinline__ void store_lanes(uint32_t first, float w0, uint32_t second, float w1, bool two, void* o, long long at) {
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
        float x[32];
        weighted32(first + 32 * c, w0, second + 32 * c, w1, two, x);
        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(o) + at * D) + 4 * c;
#pragma unroll
        for (int g = 0; g < 4; ++g)
            if (at >= 0)
                dst[g] = make_uint4(pack_bf16x2(x[8 * g], x[8 * g + 1]), pack_bf16x2(x[8 * g + 2], x[8 * g + 3]),
                                    pack_bf16x2(x[8 * g + 4], x[8 * g + 5]), pack_bf16x2(x[8 * g + 6], x[8 * g + 7]));
    }
}

// O of whole tiles of one batch, by TMA: 32 columns a box, two boxes in turn, so that one is filled
// while the other is stored, and the warp goes on with its next block while the last ones leave.  16-byte
// granule g of row r lies at g ^ (r / 2 % 4).
template <int D>
__device__ __forceinline__ void store_boxes(const CUtensorMap& tm_o, uint32_t boxes, uint32_t taddr, float f, int row0, int bh,
                                            int N) {
    const int lane = threadIdx.x % 32;
    uint32_t r[2][32];
    tmem_ld32_async(taddr, r[0]);
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
        const uint32_t box = boxes + (c & 1) * 2048;
        tmem_wait_ld();
        reg_fence(r[c & 1]);
        if (c + 1 < D / 32) tmem_ld32_async(taddr + 32 * (c + 1), r[(c + 1) & 1]);
        // the store before the last has read this box
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        __syncwarp();
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const uint32_t* x = r[c & 1] + 8 * g;
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(box + lane * 64 + ((g ^ (lane >> 1 & 3)) << 4)),
                         "r"(pack_bf16x2(__uint_as_float(x[0]) * f, __uint_as_float(x[1]) * f)),
                         "r"(pack_bf16x2(__uint_as_float(x[2]) * f, __uint_as_float(x[3]) * f)),
                         "r"(pack_bf16x2(__uint_as_float(x[4]) * f, __uint_as_float(x[5]) * f)),
                         "r"(pack_bf16x2(__uint_as_float(x[6]) * f, __uint_as_float(x[7]) * f))
                         : "memory");
        }
        fence_proxy_async_smem();  // the lanes' writes -> visible to the TMA unit
        __syncwarp();
        if (lane == 0) {
            if (row0 < N) tma_store_3d(&tm_o, box, 32 * c, row0, bh);
            bulk_commit_group();
        }
    }
}

// A row's state over some of its keys: reference maximum, sum, eight columns of the unnormalised O.
struct JoinState {
    float m, l, x[8];
    // this and another state over other keys
    __device__ __forceinline__ void add(float mk, float lk, const float (&y)[8]) {
        const float top = fmaxf(m, mk);
        // of a part whose keys' scores are all -inf nothing; a NaN in l stays
        const float keep = m == -INFINITY && l == 0.f ? 0.f : ex2_approx(m == top ? 0.f : m - top);
        const float w = mk == -INFINITY && lk == 0.f ? 0.f : ex2_approx(mk == top ? 0.f : mk - top);
        m = top;
        l = fmaf(w, lk, keep * l);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = fmaf(w, y[e], keep * x[e]);
    }
};
// Blocks of an item's run for CTA r of its cluster: up to this.
__device__ __forceinline__ int cluster_run(int blocks, int r, int log2_size) { return blocks * r >> log2_size; }

// The parts of an item on a cluster's CTAs, joined by the threads t = 0 .. 255 of each, a share of the rows a CTA:
// eight columns of a row a thread, four parts' loads in flight.
template <int D>
__device__ __forceinline__ void cluster_join(const CrossArgs& args, int t) {
    const int size = 1 << args.cluster, rank = static_cast<int>(blockIdx.x) & (size - 1);
    const int item = static_cast<int>(blockIdx.x) >> args.cluster, batch = item / args.per, at_item = item - batch * args.per;
    const int h = at_item / args.n_pairs, pair = at_item - h * args.n_pairs;
    const int blocks = cross_blocks(cross_length(args, batch));
    const int share = (args.join_rows + size - 1) / size;
    const int first = rank * share, end = min(args.join_rows, first + share);
    for (int x = t; x < share * (D / 8); x += 256) {
        // a warp takes 8 rows x 32 columns where there are so many rows
        const int vec = x / share, at = first + x % share;
        if (at >= end) continue;
        const int tile = 2 * pair + at / kPartTile, row = at % kPartTile;
        if (tile >= args.tiles) continue;
        const TileRows T = tile_rows(args, batch, tile);
        if (row >= T.rows) continue;
        const size_t size_floats = part_floats(D, args.part_rows), ml = static_cast<size_t>(args.part_rows) * D + at;
        const size_t o_at = static_cast<size_t>(2 * vec) * args.part_rows + at;
        JoinState s = {-INFINITY, 0.f, {}};
        for (int r0 = 0; r0 < size; r0 += 4) {
            float mk[4], lk[4];
            float4 y[4], z[4];
            bool there[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = r0 + i;
                there[i] = r < size && cluster_run(blocks, r, args.cluster) < cluster_run(blocks, r + 1, args.cluster);
                const float* src = args.part + static_cast<size_t>(item * size + (there[i] ? r : 0)) * size_floats;
                mk[i] = __ldcg(src + ml);
                lk[i] = __ldcg(src + ml + args.part_rows);
                y[i] = __ldcg(reinterpret_cast<const float4*>(src) + o_at);
                z[i] = __ldcg(reinterpret_cast<const float4*>(src) + o_at + args.part_rows);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float c[8] = {y[i].x, y[i].y, y[i].z, y[i].w, z[i].x, z[i].y, z[i].z, z[i].w};
                if (there[i]) s.add(mk[i], lk[i], c);
            }
        }
        const size_t out = global_row(args, T, h, row);
        const float f = row_factor(s.l);
        reinterpret_cast<uint4*>(args.o)[out * (D / 8) + vec] =
            make_uint4(pack_bf16x2(s.x[0] * f, s.x[1] * f), pack_bf16x2(s.x[2] * f, s.x[3] * f),
                       pack_bf16x2(s.x[4] * f, s.x[5] * f), pack_bf16x2(s.x[6] * f, s.x[7] * f));
        if (vec == 0 && args.lse != nullptr) args.lse[out] = row_lse(s.m, s.l);
    }
}

// Persistent.  A warp of its own works out the CTA's segments (some hundred instructions each, which
// took the other roles 1400 to 2000 cycles) and hands them to the others through a ring in shared memory.
// Every barrier counts its phases across segments: q_* per tile, kv_* per bundle, s_full and p_full per block
// of a warpgroup, o_done per segment in which the warpgroup has any.
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    cross_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                     const CrossArgs args) {
    using C = Cfg<D>;
    constexpr int kStages = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Segment segments[kSegments];
    __shared__ __align__(8) Bars<kStages> bars;
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;
    __shared__ float merge_m[kBM], merge_l[kBM];

    const uint32_t smem_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < kSegments; ++s) {
            mbar_init(smem_u32(&bars.seg_full[s]), 1);
            mbar_init(smem_u32(&bars.seg_empty[s]), kReaders);
        }
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&bars.kv_full[s]), 1);
            mbar_init(smem_u32(&bars.kv_empty[s]), 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(smem_u32(&bars.q_full[t]), 1);
            mbar_init(smem_u32(&bars.q_free[t]), 1);
            mbar_init(smem_u32(&bars.s_full[t]), 1);
            mbar_init(smem_u32(&bars.p_half[t]), 128);
            mbar_init(smem_u32(&bars.p_full[t]), 128);
            mbar_init(smem_u32(&bars.o_done[t]), 1);
        }
        mbar_init(smem_u32(&bars.merge_ml), 128);
        mbar_init(smem_u32(&bars.merge_done), 128);
        mbar_init(smem_u32(&bars.drain), 1);
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
        tma_prefetch_desc(&tm_o);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&tmem_slot), C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const uint64_t lim = args.ctl.wait_ns;
    griddep_wait();
    griddep_launch_dependents();

    // Waits for the i-th segment; taken(i) after it was read.
    auto segment_there = [&](int i) -> bool {
        return mbar_wait(smem_u32(&bars.seg_full[i % kSegments]), (i / kSegments) & 1, lim, &abort_flag);
    };
    auto segment_taken = [&](int i) { mbar_arrive(smem_u32(&bars.seg_empty[i % kSegments])); };

    // 384 threads x 168 registers at launch: 128 * 120 + 256 * 184 <= 384 * 168
    if (warp < 4) {
        regs_dec<120>();
        if (warp == 3) {
            // ============================================================ segments
            // Hands over the i-th; waits until the ring has room for it.
            auto publish = [&](int i, const Segment& s) -> bool {
                const int u = i % kSegments;
                if (i >= kSegments) {
                    const bool free = mbar_wait(smem_u32(&bars.seg_empty[u]), ((i / kSegments) & 1) ^ 1, lim, &abort_flag);
                    if (!__all_sync(0xffffffffu, free)) {
                        if (lane == 0) record_timeout(args.ctl, &abort_flag);
                        return false;
                    }
                }
                if (lane == 0) {
                    segments[u] = s;
                    mbar_arrive(smem_u32(&bars.seg_full[u]));
                }
                return true;
            };
            Segment s;
            if (args.cluster > 0) {
                const int rank = static_cast<int>(blockIdx.x) & ((1 << args.cluster) - 1);
                const int item = static_cast<int>(blockIdx.x) >> args.cluster;
                const int batch = args.B_kv == 1 ? 0 : static_cast<uint32_t>(item) / static_cast<uint32_t>(args.per);
                s.len = cross_length(args, batch);
                const int blocks = cross_blocks(s.len);
                s.k0 = cluster_run(blocks, rank, args.cluster);
                s.n = cluster_run(blocks, rank + 1, args.cluster) - s.k0;
                place_item(args, s, batch, item - batch * args.per);
                s.flags |= 2;
                publish(0, s);
            } else if (!args.stream) {
                // Whole items in alternating order, of up to 32 sequences the longest first (4 x 2048 queries on
                // 300-1000 keys 45.7 -> 39.5 us, 8 x 512 on 100-512 19.0 -> 16.7).
                int order = lane;  // lane r: the batch of rank r
                if (args.lengths != nullptr && args.B_kv <= 32 && gridDim.x < args.B_kv * args.per) order = batch_order(args);
                const uint32_t G = gridDim.x, per = args.per, all = args.B_kv * per;  // (up to 2^30 + 2^24)
                auto item_of = [&](uint32_t i) { return i * G + ((i & 1) ? G - 1 - blockIdx.x : blockIdx.x); };
                uint32_t x = item_of(0);
                for (int i = 0;; ++i) {
                    const int place = x / per, batch = args.B_kv <= 32 ? __shfl_sync(0xffffffffu, order, place) : place;
                    s.len = cross_length(args, batch);
                    s.k0 = 0;
                    s.n = cross_blocks(s.len);
                    place_item(args, s, batch, x - place * per);
                    x = item_of(i + 1);
                    s.flags |= 4 | (x >= all ? 2 : 0);
                    if (!publish(i, s) || s.last()) break;
                }
            } else {
                deal_runs(args, s, publish);
            }
        } else if (warp == 0) {
            // ============================================================ TMA producer
            if (lane == 0) {
                const int q_rows = args.nb > 1 ? args.nb * args.R : kBM;  // of a box
                int gb = 0, kq[2] = {0, 0};  // bundles and tiles issued
                bool ok = true;
                const volatile int never = 0;
                for (int i = 0; ok; ++i) {
                    ok = segment_there(i);
                    if (!ok) break;
                    const Segment s = segments[i % kSegments];
                    segment_taken(i);
                    if (s.n == 0) break;
                    auto load_q = [&](int t) -> bool {
                        if (kq[t] > 0 && !mbar_wait(smem_u32(&bars.q_free[t]), (kq[t] - 1) & 1, lim, &abort_flag)) return false;
                        const uint32_t qf = smem_u32(&bars.q_full[t]);
                        mbar_arrive_expect_tx(qf, C::kChunks * q_rows * 128);
                        for (int c = 0; c < C::kChunks; ++c)
                            tma_load_4d(smem_base + C::kOffQ + t * C::kTileBytes + c * C::kChunkBytes, &tm_q, qf, c * 64,
                                        s.rows[t].r0, s.h, s.rows[t].b);
                        ++kq[t];
                        return true;
                    };
                    ok = load_q(0);
                    // bundle n = {K of block n (n < s.n), V of block n - 1 (n >= 1)}
                    for (int n = 0; ok && n <= s.n; ++n) {
                        const int u = gb % kStages;
                        if (gb >= kStages &&
                            !mbar_wait(smem_u32(&bars.kv_empty[u]), ((gb / kStages) & 1) ^ 1, lim, &abort_flag)) {
                            ok = false;
                            break;
                        }
                        const uint32_t fb = smem_u32(&bars.kv_full[u]);
                        mbar_arrive_expect_tx(fb, ((n < s.n ? 1 : 0) + (n >= 1 ? 1 : 0)) * C::kTileBytes);
                        ++gb;
                        if (n < s.n)
                            for (int c = 0; c < C::kChunks; ++c)
                                tma_load_3d(smem_base + C::kOffK + u * C::kTileBytes + c * C::kChunkBytes, &tm_k, fb, c * 64,
                                            (s.k0 + n) * kBN, s.bh_kv);
                        if (n >= 1)
                            for (int c = 0; c < C::kChunks; ++c)
                                tma_load_3d(smem_base + C::kOffV + u * C::kTileBytes + c * C::kChunkBytes, &tm_v, fb, c * 64,
                                            (s.k0 + n - 1) * kBN, s.bh_kv);
                        if (n == 0 && !s.solo()) ok = load_q(1);
                    }
                    if (s.last()) break;
                }
                if (!ok) record_timeout(args.ctl, &abort_flag);
                // the newest load of every slot has landed before exit
                for (int t = 0; t < 2; ++t)
                    if (kq[t] > 0) mbar_wait(smem_u32(&bars.q_full[t]), (kq[t] - 1) & 1, kDrainWaitNs, &never);
                for (int n = max(0, gb - kStages); n < gb; ++n)
                    mbar_wait(smem_u32(&bars.kv_full[n % kStages]), (n / kStages) & 1, kDrainWaitNs, &never);
            }
        } else if (warp == 1) {
            // ============================================================ MMA issuer
            if (lane == 0) {
                constexpr uint32_t kDescHi = sdesc_sw128_hi(1024);
                const uint32_t q_lo = sdesc_sw128_lo(smem_base + C::kOffQ, 16);
                const uint32_t k_lo = sdesc_sw128_lo(smem_base + C::kOffK, 16);
                const uint32_t v_lo = sdesc_sw128_lo(smem_base + C::kOffV, C::kChunkBytes);
                // S in the columns of warpgroup t from query tile q and K in slot u
                auto issue_s = [&](int t, int q, int u) {
                    const uint32_t ql = q_lo + q * (C::kTileBytes >> 4), kl = k_lo + u * (C::kTileBytes >> 4);
                    const uint32_t col = tmem + C::kColS + 128 * t;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off16 = ((kk * 32) / 128 * C::kChunkBytes + (kk * 32) % 128) >> 4;
                        if (kk == 0)
                            mma_ss_w<false, -1>(col, ql, kl, kDescHi, C::kIdescS, 0u);
                        else
                            mma_ss_w<false, 1>(col, ql + off16, kl + off16, kDescHi, C::kIdescS);
                    }
                    mma_commit(smem_u32(&bars.s_full[t]));
                };
                // O_t += P_t V, each half of the keys as soon as its P is there
                auto issue_pv = [&](int t, int u, bool acc, uint32_t par, auto steps) -> bool {  // of 16 keys
                    const uint32_t vl = v_lo + u * (C::kTileBytes >> 4);
                    const uint32_t colO = tmem + C::kColO + D * t, colP = tmem + C::kColS + 128 * t;
#pragma unroll
                    for (int kk = 0; kk < kBN / 16; ++kk) {
                        if (kk >= steps) break;
                        if (kk % (kBN / 32) == 0) {
                            if (!mbar_wait(smem_u32(kk == 0 ? &bars.p_half[t] : &bars.p_full[t]), par, lim, &abort_flag)) return false;
                            tc_fence_after();
                        }
                        if (kk == 0)
                            mma_ts_w<false, -1>(colO, colP, vl, kDescHi, C::kIdescO, acc ? 1u : 0u);
                        else
                            mma_ts_w<false, 1>(colO, colP + kk * 8, vl + ((kk * 16 * 128) >> 4), kDescHi, C::kIdescO);
                    }
                    return true;
                };
                int gb = 0, kq0 = 0, kq1 = 0;
                int c0 = 0, c1 = 0;    // blocks of warpgroup 0 / 1 before the segment
                bool ok = true, begun;  // O begins with the own attention's
                // Block j of two tiles: P_t V_j, then the next block's scores, tile by tile; the last two
                // blocks run outside the loop, which keeps its body free of branches.
                auto block = [&](int j, int g1, uint32_t p0, uint32_t p1, auto more_c, auto last2_c, auto steps) -> bool {
                    constexpr bool more = decltype(more_c)::value, last2 = decltype(last2_c)::value;
                    const int u = g1 % kStages;
                    if (!mbar_wait(smem_u32(&bars.kv_full[u]), (g1 / kStages) & 1, lim, &abort_flag)) return false;
                    if (!issue_pv(0, u, j > 0 || begun, p0, steps)) return false;
                    if constexpr (more)
                        issue_s(0, 0, u);
                    else
                        mma_commit(smem_u32(&bars.o_done[0]));
                    if constexpr (last2) mma_commit(smem_u32(&bars.q_free[0]));
                    if (!issue_pv(1, u, j > 0 || begun, p1, steps)) return false;
                    if constexpr (more)
                        issue_s(1, 1, u);
                    else
                        mma_commit(smem_u32(&bars.o_done[1]));
                    if constexpr (last2) mma_commit(smem_u32(&bars.q_free[1]));
                    mma_commit(smem_u32(&bars.kv_empty[u]));
                    return true;
                };
                using T = std::true_type;
                using F = std::false_type;
                using All = std::integral_constant<int, kBN / 16>;
                for (int x = 0; ok; ++x) {
                    ok = segment_there(x);
                    if (!ok) break;
                    const int n = segments[x % kSegments].n;
                    const bool solo = segments[x % kSegments].solo(), last = segments[x % kSegments].last();
                    begun = args.o_own != nullptr && segments[x % kSegments].k0 == 0;
                    const int steps = columns_of(segments[x % kSegments].len - (segments[x % kSegments].k0 + n - 1) * kBN) / 16;
                    segment_taken(x);
                    if (n == 0) break;
                    ok = mbar_wait(smem_u32(&bars.q_full[0]), kq0++ & 1, lim, &abort_flag);
                    if (ok) ok = mbar_wait(smem_u32(&bars.kv_full[gb % kStages]), (gb / kStages) & 1, lim, &abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    const int u0 = gb % kStages;
                    issue_s(0, 0, u0);
                    if (n == 1) mma_commit(smem_u32(&bars.q_free[0]));
                    if (!solo) {
                        ok = mbar_wait(smem_u32(&bars.q_full[1]), kq1++ & 1, lim, &abort_flag);
                        if (!ok) break;
                        tc_fence_after();
                        issue_s(1, 1, u0);
                        if (n == 1) mma_commit(smem_u32(&bars.q_free[1]));
                    }
                    mma_commit(smem_u32(&bars.kv_empty[u0]));
                    if (solo) {
                        // One tile: block i belongs to warpgroup i % 2, whose S, P and O columns it uses.
                        for (int i = 1; i <= n; ++i) {
                            const int g = gb + i, u = g % kStages;
                            ok = mbar_wait(smem_u32(&bars.kv_full[u]), (g / kStages) & 1, lim, &abort_flag);
                            if (!ok) break;
                            tc_fence_after();
                            if (i < n) {
                                issue_s(i & 1, 0, u);
                                if (i == n - 1) mma_commit(smem_u32(&bars.q_free[0]));
                            }
                            const int j = i - 1, t = j & 1;
                            ok = issue_pv(t, u, j >= 2 || (j == 0 && begun), ((t ? c1 : c0) + j / 2) & 1, i < n ? kBN / 16 : steps);
                            if (!ok) break;
                            if (j + 2 >= n) mma_commit(smem_u32(&bars.o_done[t]));  // the warpgroup's last
                            mma_commit(smem_u32(&bars.kv_empty[u]));
                        }
                        c0 += (n + 1) / 2;
                        c1 += n / 2;
                    } else {
                        int j = 0;
                        for (; j + 2 < n && ok; ++j) ok = block(j, gb + j + 1, (c0 + j) & 1, (c1 + j) & 1, T{}, F{}, All{});
                        if (ok && n >= 2) ok = block(n - 2, gb + n - 1, (c0 + n - 2) & 1, (c1 + n - 2) & 1, T{}, T{}, All{});
                        if (ok) ok = block(n - 1, gb + n, (c0 + n - 1) & 1, (c1 + n - 1) & 1, F{}, F{}, steps);
                        c0 += n;
                        c1 += n;
                    }
                    gb += n + 1;
                    if (last) break;
                }
                if (!ok) record_timeout(args.ctl, &abort_flag);
                mma_commit(smem_u32(&bars.drain));
                const volatile int never = 0;
                mbar_wait(smem_u32(&bars.drain), 0, kDrainWaitNs, &never);
            }
        }
        // warp 2 has no role
    } else {
        regs_inc<184>();
        // ================================================================ softmax warpgroups
        const int t = (warp - 4) / 4;
        const int wq = warp % 4;
        const int row = wq * 32 + lane;  // of the tile
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(wq * 32) << 16);
        const uint32_t colS = C::kColS + 128 * t, colO = C::kColO + D * t;
        const float c = args.c_log2;
        const bool c_pos = c >= 0.f;
        const uint32_t mask_bits = c_pos ? 0xff800000u : 0x7f800000u;  // -inf after the multiply by c
        int gb = 0;          // bundles before the segment
        int gj = 0, kd = 0;  // this warpgroup's blocks before the segment, and segments with any
        int ns = 0;          // solo segments
        bool ok = true;
        // Of a segment only what the loop over its blocks needs is kept in registers, of which that has none to
        // spare; the rest is read from the ring again after it.
        auto place = [&](const Segment& s, int tile) -> long long {  // the thread's row among o's rows, or -1
            const TileRows T = s.rows[tile];
            return row < T.rows ? static_cast<long long>(global_row(args, T, s.h, row)) : -1;
        };
        for (int x = 0;; ++x) {
            ok = segment_there(x);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const Segment& seg = segments[x % kSegments];
            const int n = seg.n, k0 = seg.k0, len = seg.len;
            if (n == 0) break;
            const bool solo = seg.solo();
            const int tile = solo ? 0 : t;
            const bool busy = wq * 32 < seg.rows[tile].rows;  // some of the warp's rows are in use
            float m_ref = -INFINITY, l = 0.f;
            const bool begun = args.o_own != nullptr && k0 == 0 && (!solo || t == 0);
            if (begun && busy) {
                // The queries' own attention is the state to begin with: m = lse_own, l = 1, O = o_own (where
                // there is any: nothing of a row with lse_own = -inf).
                const long long at = place(seg, tile);
                m_ref = at >= 0 ? args.lse_own[at] * 1.4426950408889634f : -INFINITY;
                const bool any = m_ref != -INFINITY;
                l = any ? 1.f : 0.f;
                const uint4* own = static_cast<const uint4*>(args.o_own) + (any ? at : 0) * (D / 8);
                uint4 v[D / 8];
#pragma unroll
                for (int e = 0; e < D / 8; ++e) v[e] = any ? own[e] : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int q = 0; q < D / 32; ++q) {
                    uint32_t r[32];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t u[4] = {v[4 * q + e].x, v[4 * q + e].y, v[4 * q + e].z, v[4 * q + e].w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) r[8 * e + 2 * k] = u[k] << 16, r[8 * e + 2 * k + 1] = u[k] & 0xFFFF0000u;
                    }
                    tmem_st32(lane_base + colO + 32 * q, r);
                }
                tmem_st_wait();
            }
            int i = 0;
            for (int j = solo ? t : 0; j < n; j += solo ? 2 : 1, ++i) {
                ok = mbar_wait(smem_u32(&bars.s_full[t]), (gj + i) & 1, lim, &abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const int kv0 = (k0 + j) * kBN, valid = len - kv0;
                if (valid < kBN && len < args.N_kv) {
                    // What the caller left behind the sequence's end (an infinity, a NaN) would reach O as
                    // 0 * V: the block's rows of V from there on are made zeros before P V.
                    const int g = gb + j + 1, u = g % kStages;
                    ok = mbar_wait(smem_u32(&bars.kv_full[u]), (g / kStages) & 1, lim, &abort_flag);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    const uint32_t vb = smem_base + C::kOffV + u * C::kTileBytes;
                    const int r1 = min(kBN, args.N_kv - kv0);
                    for (int y = max(valid, 0) * 8 + row; y < r1 * 8; y += 128)
#pragma unroll
                        for (int ch = 0; ch < C::kChunks; ++ch)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vb + ch * C::kChunkBytes + y * 16), "r"(0)
                                         : "memory");
                    fence_proxy_async_smem();
                }
                auto softmax = [&](auto columns) {
                    softmax_block<D, decltype(columns)::value>(lane_base, colS, colS, colO, c, c_pos, mask_bits, valid - 1, -1, 0,
                                                               i == 0 && !begun, m_ref, l, [] {}, [] { return true; }, [&] {
                                                                   tc_fence_before();
                                                                   mbar_arrive(smem_u32(&bars.p_half[t]));
                                                               });
                };
                if (!busy)
                    mbar_arrive(smem_u32(&bars.p_half[t]));
                else if (__builtin_expect(valid > 64, 1))
                    softmax(std::integral_constant<int, kBN>{});
                else if (valid > 32)
                    softmax(std::integral_constant<int, 64>{});
                else
                    softmax(std::integral_constant<int, 32>{});
                tc_fence_before();
                mbar_arrive(smem_u32(&bars.p_full[t]));
            }
            gj += i;
            gb += n + 1;
            // a whole item's lse, while its last P V runs
            const bool by_box = !solo && args.nb == 1 && seg.whole();
            if (by_box && args.lse != nullptr && row < seg.rows[tile].rows) {
                const TileRows T = seg.rows[tile];
                args.lse[static_cast<size_t>(T.b * args.H_kv + seg.h) * args.R + (T.r0 + row)] = row_lse(m_ref, l);
            }
            if (ok && i > 0) {
                ok = mbar_wait(smem_u32(&bars.o_done[t]), kd & 1, lim, &abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                ++kd;
            }
            if (!ok) break;
            tc_fence_after();
            float w0 = 1.f, w1 = 0.f;
            const bool two = solo && n >= 2;
            if (solo) {
                // Two states over disjoint keys: m = max(m_0, m_1), l and O weighted by 2^(m_t - m).
                if (t == 1) {
                    merge_m[row] = m_ref;
                    merge_l[row] = l;
                    mbar_arrive(smem_u32(&bars.merge_ml));
                    // O_1 stays in TMEM until warpgroup 0 has read it
                    ok = mbar_wait(smem_u32(&bars.merge_done), ns & 1, lim, &abort_flag);
                    ok = __all_sync(0xffffffffu, ok);
                    ++ns;
                    if (!ok) break;
                    const bool last = seg.last();
                    __syncwarp();
                    if (lane == 0) segment_taken(x);
                    if (last) break;
                    continue;
                }
                ok = mbar_wait(smem_u32(&bars.merge_ml), ns & 1, lim, &abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                ++ns;
                if (!ok) break;
                tc_fence_after();
                const float m1 = merge_m[row], l1 = merge_l[row], mm = fmaxf(m_ref, m1);
                w0 = m_ref == -INFINITY ? 0.f : ex2_approx(m_ref - mm);
                w1 = m1 == -INFINITY ? 0.f : ex2_approx(m1 - mm);
                l = w0 * l + w1 * l1;
                m_ref = mm;
            }
            // O_t is read before this warp publishes the next segment's first P, so the next segment's
            // first P V (which overwrites O_t) comes after these loads
            const uint32_t col = lane_base + colO, col1 = lane_base + C::kColO + D;
            if (busy && !seg.whole()) {
                const int slot = args.cluster > 0 ? static_cast<int>(blockIdx.x) : static_cast<int>(blockIdx.x) * 2 + seg.slot();
                float* part = args.part + slot * part_floats(D, args.part_rows);
                const int to = row + (solo ? 0 : t * kPartTile);
#pragma unroll
                for (int q = 0; q < D / 32; ++q) {
                    float y[32];
                    weighted32(col + 32 * q, w0, col1 + 32 * q, w1, two, y);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        reinterpret_cast<float4*>(part)[static_cast<size_t>(8 * q + e) * args.part_rows + to] =
                            make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
                }
                float* ml = part + static_cast<size_t>(args.part_rows) * D;
                ml[to] = m_ref;
                ml[args.part_rows + to] = l;
            } else if (busy) {
                const float f = row_factor(l);
                if (by_box) {
                    const TileRows T = seg.rows[tile];
                    store_boxes<D>(tm_o, smem_base + C::kOffO + (warp - 4) * 4096, col, f, T.r0 + wq * 32,
                                   T.b * args.H_kv + seg.h, args.R);
                } else {
                    const long long at = place(seg, tile);
                    store_lanes<D>(col, w0 * f, col1, w1 * f, two, args.o, at);
                    if (at >= 0 && args.lse != nullptr) args.lse[at] = row_lse(m_ref, l);
                }
            }
            if (solo) {
                tc_fence_before();
                mbar_arrive(smem_u32(&bars.merge_done));
            }
            const bool last = seg.last();
            __syncwarp();
            if (lane == 0) segment_taken(x);
            if (last) break;
        }
        if (!ok && lane == 0) record_timeout(args.ctl, &abort_flag);
        // the stores complete before the CTA's shared memory goes away
        if (lane == 0) bulk_wait_all();
    }

    tc_fence_before();
    if (args.cluster > 0) {  // every thread gets here, also from a wait that ran out
        __syncwarp();
        cluster_sync();
        if (warp >= 4) cluster_join<D>(args, static_cast<int>(threadIdx.x) - 128);
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

// Items that were cut: the parts of the one in place blockIdx.x of the table, some of its rows at a time
// (blockIdx.y), in a fixed order.  A warp takes 8 rows x 32 columns (128-byte runs of the parts, 64-byte runs of
// the result) of every GROUPS-th part; the groups' states meet in shared
// memory.  Items of many parts take four groups (16 items of 9 parts each 7.0 -> 3.5 us, 8 of 19 13.7 -> 8.8; a lone
// tile's rows from four parts on, 27 of 48 rows 14.8 -> 13.3 with the attention);
// where there are two to four parts four groups are idle and in the way (64 items 8 -> 34 us), and the reads
// of 128 KB a part at d = 128 count.
// Parts in flight: four in four groups take 73 registers, one CTA an SM instead of two (64 requests on 16384 keys
// 30.6 us, three 28.0).
template <int GROUPS>
constexpr int kTogetherOf = GROUPS == 1 ? 2 : 3;
template <int GROUPS>
constexpr int kJoinRows = GROUPS == 1 ? 16 : 8;
template <int D, int GROUPS>
__global__ void __launch_bounds__(GROUPS == 1 ? 2 * D : GROUPS * D) cross_join_kernel(const CrossArgs args) {
    constexpr int kCols = D / 32, kWarpRows = kJoinRows<GROUPS> / 8, kTogether = kTogetherOf<GROUPS>;
    __shared__ JoinState states[GROUPS > 1 ? GROUPS - 1 : 1][GROUPS > 1 ? kCols * 32 : 1];
    griddep_wait();
    griddep_launch_dependents();
    const int4 cut = args.cut[blockIdx.x];  // last CTA (-1: not cut), batch, item, first CTA
    if (cut.x < 0) return;
    const int c = cut.w;
    const int h = cut.z / args.n_pairs, pair = cut.z - h * args.n_pairs;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int group = warp / (kCols * kWarpRows), vec = warp % kCols * 4 + lane / 8;  // 8 columns
    const int at = blockIdx.y * kJoinRows<GROUPS> + warp / kCols % kWarpRows * 8 + lane % 8;
    const int tile = 2 * pair + at / kPartTile, row = at % kPartTile;
    TileRows T = {0, 0, 0};
    if (tile < args.tiles && at < args.part_rows) T = tile_rows(args, cut.y, tile);
    const bool mine = row < T.rows;
    if (GROUPS == 1 ? !mine : !__syncthreads_or(mine)) return;
    const size_t size = part_floats(D, args.part_rows), ml = static_cast<size_t>(args.part_rows) * D + at;
    const size_t o_at = static_cast<size_t>(2 * vec) * args.part_rows + at;
    JoinState s = {-INFINITY, 0.f, {}};
    for (int k0 = c + group; mine && k0 <= cut.x; k0 += GROUPS * kTogether) {
        float mk[kTogether], lk[kTogether];
        float4 y[kTogether], z[kTogether];
#pragma unroll
        for (int i = 0; i < kTogether; ++i) {
            const int k = k0 + GROUPS * i;
            const bool there = k <= cut.x;
            // the item's first part is its CTA's second slot, the others are their CTAs' first
            const float* src = args.part + static_cast<size_t>(2 * k + (k == c)) * size;
            const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
            mk[i] = there ? src[ml] : -INFINITY;
            lk[i] = there ? src[ml + args.part_rows] : 0.f;
            y[i] = there ? reinterpret_cast<const float4*>(src)[o_at] : none;
            z[i] = there ? reinterpret_cast<const float4*>(src)[o_at + args.part_rows] : none;
        }
#pragma unroll
        for (int i = 0; i < kTogether; ++i) {
            const float x[8] = {y[i].x, y[i].y, y[i].z, y[i].w, z[i].x, z[i].y, z[i].z, z[i].w};
            if (k0 + GROUPS * i <= cut.x) s.add(mk[i], lk[i], x);
        }
    }
    if constexpr (GROUPS > 1) {
        const int place = threadIdx.x % (kCols * 32);
        if (group > 0) states[group - 1][place] = s;
        __syncthreads();
        if (group > 0 || !mine) return;
#pragma unroll
        for (int g = 0; g < GROUPS - 1; ++g)
            if (c + g + 1 <= cut.x) s.add(states[g][place].m, states[g][place].l, states[g][place].x);
    }
    const size_t out = global_row(args, T, h, row);
    const float f = row_factor(s.l);
#pragma unroll
    for (int i = 0; i < 8; ++i) s.x[i] *= f;
    reinterpret_cast<uint4*>(args.o)[out * (D / 8) + vec] =
        make_uint4(pack_bf16x2(s.x[0], s.x[1]), pack_bf16x2(s.x[2], s.x[3]), pack_bf16x2(s.x[4], s.x[5]), pack_bf16x2(s.x[6], s.x[7]));
    if (vec == 0 && args.lse != nullptr) args.lse[out] = row_lse(s.m, s.l);
}

// q as [B][H_kv][R][d] in boxes of `rows` rows of nb batches, 64 columns, or o in boxes of a warp's 32 rows, 32
// columns.
int row_map(CUtensorMap* map, const void* base, int D, const CrossArgs& a, int cols, int rows, int nb) {
    EncodeTiledFn fn = encode_tiled_fn();
    if (fn == nullptr) return -1;
    const cuuint64_t line = static_cast<cuuint64_t>(D) * 2;
    cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(a.R), static_cast<cuuint64_t>(a.H_kv),
                          static_cast<cuuint64_t>(a.B_kv) * a.share};
    cuuint64_t strides[3] = {line, line * a.R, line * a.R * a.H_kv};
    cuuint32_t box[4] = {static_cast<cuuint32_t>(cols), static_cast<cuuint32_t>(rows), 1, static_cast<cuuint32_t>(nb)};
    int rank = 4;
    if (cols == 32) {  // heads and batches as one dimension
        dims[2] *= dims[3];
        rank = 3;
    }
    cuuint32_t one[4] = {1, 1, 1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, one,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? 0 : static_cast<int>(r);
}

template <int D, int GROUPS>
cudaError_t join(const CrossArgs& x, int places, cudaStream_t s) {
    return launch_pdl(cross_join_kernel<D, GROUPS>, dim3(places, (x.join_rows + kJoinRows<GROUPS> - 1) / kJoinRows<GROUPS>),
                      dim3(GROUPS == 1 ? 2 * D : GROUPS * D), 0, s, x);
}

// Few items take a cluster each, whose CTAs meet at its barrier, which spares the launch of the join (one token of 32 / 8
// heads on 1500 keys, 8 items on clusters of eight, 9.25 -> 8.6 us; 8 queries of 16 heads there 10.3 -> 8.55, of 36 on 700,
// clusters of four, 10.6 -> 8.2; 10 x 3 tokens on two prompts 8.2 -> 7.8; but 15 x 130 queries on 1100 keys 13.0 -> 14.4,
// where 15 clusters of eight leave 32 SMs out): the largest clusters of which the device holds
// as many at once as there are items (36 of four, 15 of eight).  Those leave some SMs out, so not where that costs
// more blocks a CTA than the join is worth (a ragged batch's mean again taken for 3/4).  Sizes that are no powers of two and those beyond eight were
// slower than their numbers of blocks say (8 items of 7 blocks: four 8.3 us, seven 9.2, the join's launch 9.0;
// 1 item of 32: sixteen 13.6, the launch 11.3).  0: none.
constexpr int kMaxCluster = 8, kJoinBlocks = 3;  // blocks of keys in the time of a join
template <int D>
cudaError_t cluster_size(const CrossArgs& a, int dev, int* log2_size) {
    static std::atomic<int> known[64][kMaxCluster + 1];  // clusters of a size, + 1; 0: not asked
    *log2_size = 0;
    const long long items = static_cast<long long>(a.B_kv) * a.per;
    const int blocks = (a.N_kv + kBN - 1) / kBN;
    if (!a.stream || items * 2 > kMaxCtas || dev >= 64) return cudaSuccess;
    for (int s = kMaxCluster; s > 1; s /= 2) {
        if (s > blocks || items * s > kMaxCtas) continue;
        if ((blocks + s - 1) / s > 0.75 * items * blocks / kMaxCtas + kJoinBlocks) return cudaSuccess;
        int n = known[dev][s].load();
        if (n == 0) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(s);
            cfg.blockDim = dim3(kThreads);
            cfg.dynamicSmemBytes = Cfg<D>::kSmemAlloc;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim = {static_cast<unsigned>(s), 1, 1};
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&n, cross_fwd_kernel<D>, &cfg) != cudaSuccess) {
                cudaGetLastError();  // no such cluster: not the caller's error
                n = 0;
            }
            known[dev][s].store(++n);
        }
        if (n > items) {
            *log2_size = s == 8 ? 3 : s / 2;
            return cudaSuccess;
        }
    }
    return cudaSuccess;
}

template <int D>
cudaError_t launch_clusters(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& to,
                            const CrossArgs& x, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(x.B_kv * x.per << x.cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Cfg<D>::kSmemAlloc;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {1u << x.cluster, 1, 1};
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, cross_fwd_kernel<D>, tq, tk, tv, to, x);
}

template <int D>
int launch_impl(const void* q, const void* k, const void* v, const CrossArgs& a, cudaStream_t s) {
    const int BH_kv = a.B_kv * a.H_kv;
    CUtensorMap tq, tk, tv, to;
    const CUtensorMapDataType dt = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    int rc = row_map(&tq, q, D, a, 64, a.nb > 1 ? a.R : kBM, a.nb);
    if (rc == 0) rc = row_map(&to, a.o, D, a, 32, 32, 1);
    if (rc == 0) rc = make_map_3d(&tk, k, dt, 2, D, a.N_kv, BH_kv, 64, kBN);
    if (rc == 0) rc = make_map_3d(&tv, v, dt, 2, D, a.N_kv, BH_kv, 64, kBN);
    if (rc != 0) return rc;
    static std::atomic<uint64_t> smem_done;
    cudaError_t e = allow_smem(cross_fwd_kernel<D>, Cfg<D>::kSmemAlloc, smem_done);
    int dev = 0, sms = 0;
    if (e == cudaSuccess) e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return static_cast<int>(e);
    CrossArgs x = a;
    if (x.ctas > sms) x.ctas = sms;
    e = cluster_size<D>(a, dev, &x.cluster);
    if (e != cudaSuccess) return static_cast<int>(e);
    if (x.cluster > 0) return static_cast<int>(launch_clusters<D>(tq, tk, tv, to, x, s));
    e = launch_pdl(cross_fwd_kernel<D>, dim3(x.ctas), dim3(kThreads), Cfg<D>::kSmemAlloc, s, tq, tk, tv, to, x);
    const int items = x.by_item ? x.B_kv * x.per : x.ctas - 1;  // places of cut items
    if (e == cudaSuccess && x.stream && x.ctas > 1)
        e = x.ctas >= (x.join_rows > kBM ? 6 : 4) * items ? join<D, 4>(x, items, s) : join<D, 1>(x, items, s);
    return static_cast<int>(e);
}

}  // namespace

size_t fwd_cross_workspace_bytes(int B, int B_kv, int H, int H_kv, int N_q, int N_kv, int d) {
    const CrossArgs a = deal(B, B_kv, H, H_kv, N_q, N_kv, d);
    return a.stream && a.ctas > 1 ? kCutBytes + 2 * a.ctas * part_floats(d, a.part_rows) * sizeof(float) : 0;
}

int launch_fwd_cross(const void* q, const void* k, const void* v, const int* lengths, const void* o_own,
                     const float* lse_own, void* o, float* lse, void* workspace, int B, int B_kv, int H, int H_kv, int N_q,
                     int N_kv, int d, float c_log2, DevCtl ctl, cudaStream_t s) {
    CrossArgs a = deal(B, B_kv, H, H_kv, N_q, N_kv, d);
    a.lengths = lengths;
    a.o = o;
    a.lse = lse;
    a.o_own = o_own;
    a.lse_own = lse_own;
    a.cut = static_cast<int4*>(workspace);
    a.part = static_cast<float*>(workspace) + kCutBytes / sizeof(float);
    // a scale of 0 makes all scores 0; the mask multiplies -inf by c, which has to stay -inf
    a.c_log2 = c_log2 == 0.f ? 1e-30f : c_log2;
    a.ctl = ctl;
    if (a.few) return static_cast<int>(launch_cross_few(a, d, q, k, v, s));
    return d == 64 ? launch_impl<64>(q, k, v, a, s) : launch_impl<128>(q, k, v, a, s);
}

}  // namespace fa
