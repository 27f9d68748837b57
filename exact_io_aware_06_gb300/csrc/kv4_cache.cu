// kv4_cache.cu -- writing tokens into the paged 4-bit K/V cache, and reading them back as
// bf16 (the dense prefix that a chunked prompt's attention reads).
//
// Both are bound by memory: 2 d bytes of bf16 against 9 d / 16 of codes and scales per row.
// d / 8 lanes hold a row, eight values (16 bytes of bf16) each, four lanes a group of 32 whose
// maximum is two shuffles; a warp takes 32 / (d / 8) rows of one array and strides over them.
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

template <int D>
__global__ void __launch_bounds__(kThreads)
    kv4_append_kernel(const Kv4Cache c, const uint4* __restrict__ k, const uint4* __restrict__ v,
                      const int* __restrict__ first, const int* __restrict__ count, int N, long long rows,
                      DevCtl ctl) {
    constexpr int kLanes = D / 8;
    griddep_wait();
    griddep_launch_dependents();
    const int j = threadIdx.x % kLanes;  // this lane's eight values: 8 j ..
    const int which = blockIdx.y;        // K or V
    const uint4* src = which ? v : k;
    const long long step = static_cast<long long>(gridDim.x) * (kThreads / kLanes);
    // rows of a warp go round together: the shuffles below need every lane
    const long long r0 = static_cast<long long>(blockIdx.x) * (kThreads / kLanes) + threadIdx.x / kLanes;
    const long long w0 = r0 - (threadIdx.x % 32) / kLanes;
    for (long long off = 0; w0 + off < rows; off += step) {
        const long long row = r0 + off;
        bool in = row < rows;
        int page = -1, pos = 0, h = 0;
        if (in) {
            const long long bh = row / N;
            const int n = static_cast<int>(row % N);
            const long long b = bh / c.H_kv;
            h = static_cast<int>(bh % c.H_kv);
            in = count == nullptr || n < count[b];
            if (in) {
                const long long at = static_cast<long long>(first[b]) + n;
                pos = at < 0 || at > 0x7fffffff ? -1 : static_cast<int>(at);
                page = page_of(c, ctl, b, pos);
                in = page >= 0;
            }
        }
        const uint4 raw = in ? __ldcs(src + row * kLanes + j) : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
        // the largest magnitude as bits: ordered as integers, infinities and NaN above all else
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const bool finite = top < 0x7F80u;
        const float s = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(__uint_as_float(top << 16), 7.f)));
        uint32_t word = 0x88888888u;
        if (finite && s > 0.f) {
            word = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float q = rintf(__fdiv_rn(bf16_at(w[i / 2], i & 1), s));
                word |= static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(q, -7.f), 7.f)) + 8) << (4 * i);
            }
        }
        if (!in) continue;
        const uint16_t sbits = finite ? static_cast<uint16_t>(__float_as_uint(s) >> 16) : 0x7FC0u;
        const int slot = pos & ((1 << c.page_log2) - 1);
        const size_t base = (static_cast<size_t>(page) * c.H_kv + h) << c.page_log2;  // in tokens
        const int grp = j / 4, t = j % 4;
        if (which == 0) {
            *reinterpret_cast<uint32_t*>(c.codes[0] + (base + slot) * (D / 2) + kv4_k_word(D, t, grp)) = word;
            if (t == 0) c.scales[0][(base + slot) * (D / 32) + grp] = sbits;
        } else {
            uint8_t* dst = c.codes[1] + base * (D / 2);
            *reinterpret_cast<uint16_t*>(dst + kv4_v_half(D, slot, 2 * t, grp)) = static_cast<uint16_t>(word);
            *reinterpret_cast<uint16_t*>(dst + kv4_v_half(D, slot, 2 * t + 1, grp)) =
                static_cast<uint16_t>(word >> 16);
            if (t == 0) c.scales[1][base * (D / 32) + kv4_v_scale(D, slot, grp)] = sbits;
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads)
    kv4_read_kernel(const Kv4Cache c, const int* __restrict__ lengths, uint4* __restrict__ k,
                    uint4* __restrict__ v, int N, long long rows, DevCtl ctl) {
    constexpr int kLanes = D / 8;
    griddep_wait();
    griddep_launch_dependents();
    const int j = threadIdx.x % kLanes;
    const int which = blockIdx.y;
    uint4* dst = which ? v : k;
    const int grp = j / 4, t = j % 4;
    const long long step = static_cast<long long>(gridDim.x) * (kThreads / kLanes);
    for (long long row = static_cast<long long>(blockIdx.x) * (kThreads / kLanes) + threadIdx.x / kLanes;
         row < rows; row += step) {
        const long long bh = row / N, b = bh / c.H_kv;
        const int n = static_cast<int>(row % N), h = static_cast<int>(bh % c.H_kv);
        uint4 out = make_uint4(0, 0, 0, 0);
        const int page = n < lengths[b] ? page_of(c, ctl, b, n) : -1;
        if (page >= 0) {
            const int slot = n & ((1 << c.page_log2) - 1);
            const size_t base = (static_cast<size_t>(page) * c.H_kv + h) << c.page_log2;
            uint32_t word, sbits;
            if (which == 0) {
                word = *reinterpret_cast<const uint32_t*>(c.codes[0] + (base + slot) * (D / 2) + kv4_k_word(D, t, grp));
                sbits = c.scales[0][(base + slot) * (D / 32) + grp];
            } else {
                const uint8_t* src = c.codes[1] + base * (D / 2);
                word = *reinterpret_cast<const uint16_t*>(src + kv4_v_half(D, slot, 2 * t, grp));
                word |= static_cast<uint32_t>(
                            *reinterpret_cast<const uint16_t*>(src + kv4_v_half(D, slot, 2 * t + 1, grp))) << 16;
                sbits = c.scales[1][base * (D / 32) + kv4_v_scale(D, slot, grp)];
            }
            const float s = __uint_as_float(sbits << 16);
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float lo = static_cast<float>(static_cast<int>((word >> (8 * i)) & 15u) - 8) * s;
                const float hi = static_cast<float>(static_cast<int>((word >> (8 * i + 4)) & 15u) - 8) * s;
                o[i] = pack_bf16x2(lo, hi);
            }
            out = make_uint4(o[0], o[1], o[2], o[3]);
        }
        dst[row * kLanes + j] = out;
    }
}

dim3 grid_of(long long rows, int lanes) {
    int sms = 152, dev = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const long long per = kThreads / lanes, blocks = (rows + per - 1) / per, cap = static_cast<long long>(sms) * 8;
    return dim3(static_cast<unsigned>(blocks < cap ? blocks : cap), 2);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4Cache& c, const void* k, const void* v, const int* first,
                              const int* count, int B, int N, int d, DevCtl ctl, cudaStream_t s) {
    const long long rows = static_cast<long long>(B) * c.H_kv * N;
    const uint4* k4 = static_cast<const uint4*>(k);
    const uint4* v4 = static_cast<const uint4*>(v);
    if (d == 64)
        return launch_pdl(kv4_append_kernel<64>, grid_of(rows, 8), dim3(kThreads), 0, s, c, k4, v4, first, count, N,
                          rows, ctl);
    return launch_pdl(kv4_append_kernel<128>, grid_of(rows, 16), dim3(kThreads), 0, s, c, k4, v4, first, count, N,
                      rows, ctl);
}

cudaError_t launch_kv4_read(const Kv4Cache& c, const int* lengths, void* k, void* v, int B, int N, int d,
                            DevCtl ctl, cudaStream_t s) {
    const long long rows = static_cast<long long>(B) * c.H_kv * N;
    uint4* k4 = static_cast<uint4*>(k);
    uint4* v4 = static_cast<uint4*>(v);
    if (d == 64)
        return launch_pdl(kv4_read_kernel<64>, grid_of(rows, 8), dim3(kThreads), 0, s, c, lengths, k4, v4, N, rows,
                          ctl);
    return launch_pdl(kv4_read_kernel<128>, grid_of(rows, 16), dim3(kThreads), 0, s, c, lengths, k4, v4, N, rows,
                      ctl);
}

}  // namespace fa
