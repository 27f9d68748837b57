// kv4_cache.cu -- writing tokens into the paged 4-bit K/V cache, and reading them back as
// bf16 (the dense prefix that a chunked prompt's attention reads).
//
// Both are bound by memory: 2 d bytes of bf16 against 9 d / 16 of codes and scales per row.
// d / 8 lanes hold a row, eight values (16 bytes of bf16) each, four lanes a group of 32 whose
// maximum is two shuffles.  A thread takes a row of K and the same row of V: the way to their
// bytes (request, its first token, its page: three dependent loads) is gone once for both.
// Instructions bound these kernels next to memory, hence the arithmetic below.  Measured for two
// prompts of 8192 tokens, 8 heads of d = 128 (67 MB of bf16): append and read 31.2 us together for 153 MB,
// 4.9 TB/s (the codes counted once: what the read finds in L2 is not traffic).
#include <cuda_bf16.h>

#include "kv4.cuh"
#include "layer_ops.h"
#include "ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void record_index(const DevCtl& ctl) { atomicCAS(ctl.status, kDevOk, kDevIndex); }

// Page of token `pos` of request b, or -1 where the table has none (recorded).
__device__ __forceinline__ int page_of(const Kv4Cache& c, const DevCtl& ctl, long long b, int pos) {
    const int blk = pos >> c.page_log2;
    int p = -1;
    if (pos >= 0 && blk < c.max_blocks) p = __ldg(c.table + b * c.max_blocks + blk);
    if (p < 0 || p >= c.n_pages) {
        record_index(ctl);
        p = -1;
    }
    return p;
}

__device__ __forceinline__ float bf16_at(uint32_t w, int i) {
    return __uint_as_float(i ? w & 0xFFFF0000u : w << 16);
}

// Codes + 8 of eight bf16 values (pairs w) with a scale s > 0, as nibbles.
//
// x / s has to round as the quotient itself does, halves to even.  x and s have 8 bits each, so a
// quotient below 8 that is no half of an odd integer is at least 2^-10 from one: x times the
// reciprocal of s (off by 2^-20), rounded to a multiple of 2^-12 by adding 1.5 2^11, is on a half
// exactly where the quotient is, and on the quotient's side of it elsewhere.  Adding the rest of
// 1.5 2^23 + 8 rounds to the integer, and leaves the nibble in the low bits.  Division took 260
// operations a row and 32 us for 131072 rows of K and V, where memory needs 13.  A subnormal s, which
// has fewer bits and whose reciprocal may overflow, divides.
__device__ __forceinline__ uint32_t codes_of(const uint32_t (&w)[4], float s) {
    constexpr float kSnap = 0x1.8p11f, kInt = 0x1.8p23f + 8.f;
    float q[8];
    if (s >= 0x1p-120f) {
        float inv;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
        const float2 inv2 = make_float2(inv, inv);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 t = __ffma2_rn(make_float2(bf16_at(w[i], 0), bf16_at(w[i], 1)), inv2, make_float2(kSnap, kSnap));
            t = __fadd2_rn(t, make_float2(kInt - kSnap, kInt - kSnap));
            q[2 * i] = t.x;
            q[2 * i + 1] = t.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            q[i] = fminf(fmaxf(rintf(__fdiv_rn(bf16_at(w[i / 2], i & 1), s)), -7.f), 7.f) + kInt;
    }
    // sum of bits 16^i; what kInt's own bits, 0x4B400008 without the 8, add to it comes off again
    uint32_t word = __float_as_uint(q[7]);
#pragma unroll
    for (int i = 6; i >= 0; --i) word = word * 16 + __float_as_uint(q[i]);
    return word - 0x3F400000u;
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Where a row is: request, head and the index among the request's rows.
struct Row {
    uint32_t b, h, n;
};
__device__ __forceinline__ Row row_at(uint32_t row, const Div& by_n, const Div& by_heads) {
    Row r;
    const uint32_t bh = by_n.of(row);
    r.n = row - bh * by_n.d;
    r.b = by_heads.of(bh);
    r.h = bh - r.b * by_heads.d;
    return r;
}

template <int D>
__global__ void __launch_bounds__(kThreads)
    kv4_append_kernel(const Kv4Cache c, const uint4* __restrict__ k, const uint4* __restrict__ v,
                      const int* __restrict__ first, const int* __restrict__ count, const Div by_n, const Div by_heads,
                      uint32_t rows, DevCtl ctl) {
    constexpr int kLanes = D / 8;
    const int j = threadIdx.x % kLanes;  // this lane's eight values: 8 j ..
    const int grp = j / 4, t = j % 4;
    const uint32_t row = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
    griddep_wait();
    griddep_launch_dependents();
    uint4 raw[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    int page = -1, pos = 0, head = 0;
    if (row < rows) {
        const size_t at = static_cast<size_t>(row) * kLanes + j;
        raw[0] = __ldcs(k + at);
        raw[1] = __ldcs(v + at);
        const Row r = row_at(row, by_n, by_heads);
        head = r.h;
        if (count == nullptr || static_cast<int>(r.n) < count[r.b]) {
            const long long p = static_cast<long long>(first[r.b]) + r.n;
            pos = p < 0 || p > 0x7fffffff ? -1 : static_cast<int>(p);
            page = page_of(c, ctl, r.b, pos);
        } else if (count[r.b] < 0) {
            record_index(ctl);
        }
    }
    uint32_t word[2], sbits[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        // the largest magnitude as bits: ordered as integers, infinities and NaN above all else
        uint32_t top = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                                __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
        top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
        top = max(top & 0xFFFFu, top >> 16);
        const bool finite = top < 0x7F80u;
        // max / 7 has the binary period 001, so no max of 8 bits comes near a tie of bf16: the
        // product with 1/7 rounds as the quotient does
        const float s = __bfloat162float(__float2bfloat16_rn(__uint_as_float(top << 16) * (1.f / 7.f)));
        word[i] = finite && s > 0.f ? codes_of(w, s) : 0x88888888u;
        sbits[i] = finite ? __float_as_uint(s) >> 16 : 0x7FC0u;
    }
    if (page < 0) return;
    const int slot = pos & ((1 << c.page_log2) - 1);
    const size_t base = (static_cast<size_t>(page) * c.H_kv + head) << c.page_log2;  // in tokens
    *reinterpret_cast<uint32_t*>(c.codes[0] + (base + slot) * (D / 2) + kv4_k_word(D, t, grp)) = word[0];
    uint8_t* dst = c.codes[1] + base * (D / 2) + kv4_v_half(D, slot, 2 * t, grp);
    *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(word[1]);
    *reinterpret_cast<uint16_t*>(dst + kv4_v_half(D, 0, 1, 0)) = static_cast<uint16_t>(word[1] >> 16);
    if (t == 0) {
        c.scales[0][(base + slot) * (D / 32) + grp] = static_cast<uint16_t>(sbits[0]);
        c.scales[1][base * (D / 32) + kv4_v_scale(D, slot, grp)] = static_cast<uint16_t>(sbits[1]);
    }
}

// Eight values back from their codes and scale.
__device__ __forceinline__ uint4 values_of(uint32_t word, uint32_t scale) {
    // pairs of values m and m + 4 as 128 + code + 8, less 136 (exact), times the scale: the product
    // of 4 and 8 bits, rounded once
    const uint32_t s2 = scale | scale << 16;
    uint32_t e[4];
#pragma unroll
    for (int m = 0; m < 4; ++m)
        e[m] = mul_bf16x2(sub_bf16x2(((word >> (4 * m)) & 0x000F000Fu) | 0x43004300u, 0x43084308u), s2);
    return make_uint4(__byte_perm(e[0], e[1], 0x5410), __byte_perm(e[2], e[3], 0x5410),
                      __byte_perm(e[0], e[1], 0x7632), __byte_perm(e[2], e[3], 0x7632));
}

// Bad lengths are recorded by CTAs of their own behind those of the rows, which do not meet them all.
// (A test in the rows' threads took 1 to 4% longer.)
__device__ __forceinline__ void check_lengths(const Kv4Cache& c, const int* __restrict__ lengths, int B, uint32_t row_ctas,
                                              const DevCtl& ctl) {
    const uint32_t step = (gridDim.x - row_ctas) * kThreads;
    for (uint32_t b = (blockIdx.x - row_ctas) * kThreads + threadIdx.x; b < static_cast<uint32_t>(B); b += step)
        if (lengths[b] < 0 || lengths[b] > c.max_blocks << c.page_log2) record_index(ctl);
}

// A thread reads ROWS (1 or 2) rows of K and of V from row n = ROWS i on: an even token and the next
// one are in the same tile of the same page.
template <int D, int ROWS>
__global__ void __launch_bounds__(kThreads)
    kv4_read_kernel(const Kv4Cache c, const int* __restrict__ lengths, uint4* __restrict__ k,
                    uint4* __restrict__ v, const Div by_runs, const Div by_heads, uint32_t N, uint32_t runs, int B,
                    uint32_t row_ctas, DevCtl ctl) {
    constexpr int kLanes = D / 8;
    const int j = threadIdx.x % kLanes;
    const int grp = j / 4, t = j % 4;
    const uint32_t run = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
    griddep_wait();
    griddep_launch_dependents();
    if (run >= runs) {
        if (blockIdx.x >= row_ctas) check_lengths(c, lengths, B, row_ctas, ctl);
        return;
    }
    const Row r = row_at(run, by_runs, by_heads);
    const uint32_t n = ROWS * r.n;
    const int len = lengths[r.b];
    const int page = static_cast<int>(n) < len ? page_of(c, ctl, r.b, n) : -1;
    const size_t at = (ROWS == 1 ? run : (static_cast<size_t>(r.b) * by_heads.d + r.h) * N + n) * kLanes + j;
    if (ROWS == 1 && page < 0) {
        k[at] = v[at] = make_uint4(0, 0, 0, 0);
        return;
    }
    const int slot = n & ((1 << c.page_log2) - 1);
    const size_t base = (static_cast<size_t>(max(page, 0)) * c.H_kv + r.h) << c.page_log2;
    const uint8_t* ks = c.codes[0] + (base + slot) * (D / 2) + kv4_k_word(D, t, grp);
    const uint8_t* vs = c.codes[1] + base * (D / 2) + kv4_v_half(D, slot, 2 * t, grp);
    const uint16_t* kscale = c.scales[0] + (base + slot) * (D / 32) + grp;
    const uint16_t* vscale = c.scales[1] + base * (D / 32) + kv4_v_scale(D, slot, grp);
    constexpr int kNextV = static_cast<int>(kv4_v_half(D, 1, 0, 0)), kNextG = static_cast<int>(kv4_v_half(D, 0, 1, 0));
    constexpr int kNextScale = static_cast<int>(kv4_v_scale(D, 1, 0));
#pragma unroll
    for (int x = 0; x < ROWS; ++x) {
        if (x > 0 && n + x >= N) break;
        uint4 out[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        if (page >= 0 && (x == 0 || static_cast<int>(n) + x < len)) {
            const uint8_t* q = vs + x * kNextV;
            const uint32_t vw = *reinterpret_cast<const uint16_t*>(q) |
                                static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(q + kNextG)) << 16;
            out[0] = values_of(*reinterpret_cast<const uint32_t*>(ks + x * (D / 2)), kscale[x * (D / 32)]);
            out[1] = values_of(vw, vscale[x * kNextScale]);
        }
        k[at + x * kLanes] = out[0];
        v[at + x * kLanes] = out[1];
    }
}

uint32_t ctas_of(uint32_t rows, int lanes) {
    const uint32_t per = kThreads / lanes;
    return (rows + per - 1) / per;
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4Cache& c, const void* k, const void* v, const int* first,
                              const int* count, int B, int N, int d, DevCtl ctl, cudaStream_t s) {
    const uint32_t rows = static_cast<uint32_t>(B) * c.H_kv * N;
    return launch_pdl(d == 64 ? kv4_append_kernel<64> : kv4_append_kernel<128>, dim3(ctas_of(rows, d / 8)), dim3(kThreads),
                      0, s, c, static_cast<const uint4*>(k), static_cast<const uint4*>(v), first, count, make_div(N),
                      make_div(c.H_kv), rows, ctl);
}

namespace {
template <int D, int ROWS>
cudaError_t launch_read(const Kv4Cache& c, const int* lengths, void* k, void* v, int B, int N, DevCtl ctl, cudaStream_t s) {
    const uint32_t per_head = (static_cast<uint32_t>(N) + ROWS - 1) / ROWS;
    const uint32_t runs = static_cast<uint32_t>(B) * c.H_kv * per_head;
    const uint32_t row_ctas = ctas_of(runs, D / 8);
    const uint32_t checks = B < 64 * kThreads ? (B + kThreads - 1) / kThreads : 64;  // CTAs of check_lengths
    return launch_pdl(kv4_read_kernel<D, ROWS>, dim3(row_ctas + checks), dim3(kThreads), 0, s, c, lengths,
                      static_cast<uint4*>(k), static_cast<uint4*>(v), make_div(per_head), make_div(c.H_kv),
                      static_cast<uint32_t>(N), runs, B, row_ctas, ctl);
}
}  // namespace

// Two rows a thread share the way to their page, once there are rows for all threads that an SM
// holds: two prompts of 8192 tokens, 8 heads, d = 128, append and read, 32.5 us against 34.5; 8
// ragged ones of up to 829 tokens, d = 64 (53000 rows of 8 threads) 7.0 against 6.0.
cudaError_t launch_kv4_read(const Kv4Cache& c, const int* lengths, void* k, void* v, int B, int N, int d,
                            DevCtl ctl, cudaStream_t s) {
    const bool two = static_cast<long long>(B) * c.H_kv * N * (d / 8) >= 4ll * 152 * 2048;
    if (d == 64)
        return two ? launch_read<64, 2>(c, lengths, k, v, B, N, ctl, s) : launch_read<64, 1>(c, lengths, k, v, B, N, ctl, s);
    return two ? launch_read<128, 2>(c, lengths, k, v, B, N, ctl, s) : launch_read<128, 1>(c, lengths, k, v, B, N, ctl, s);
}

}  // namespace fa
