// layer_ops.h -- declarations of the operators around the attention call: norm and
// rotation of Q and K, windowed attention with sinks, and the 4-bit K/V cache.
#pragma once

#include <atomic>

#include "internal.h"

namespace fa {

// The current device's status word and wait limit; false with *err set on failure.
bool device_ctl(DevCtl* ctl, int* err);

// Lets a kernel use `bytes` of dynamic shared memory on the current device; asked once per
// kernel and device (`done`: one bit per device, of the kernel's own).
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (bit & done.load()) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit);
    return e;
}

// n / d for n < 2^31 by a multiplication: with l = ceil(log2 d) and mul = 2^32 (2^l - d) / d + 1,
// (n + (n mul >> 32)) >> l, whose sum stays below 2^32.
struct Div {
    uint32_t d, mul, shift;
#ifdef __CUDACC__
    __device__ __forceinline__ uint32_t of(uint32_t n) const { return (__umulhi(n, mul) + n) >> shift; }
#endif
};
inline Div make_div(uint32_t d) {
    uint32_t l = 0;
    while ((1ull << l) < d) ++l;
    return {d, static_cast<uint32_t>((((1ull << l) - d) << 32) / d + 1), l};
}

// Angle of position t in rotation pair p, in turns: frac(t * f[p] / 2^64).
struct RopeFreq {
    uint64_t f[64];
};

struct NormRopeArgs {
    const void* qkv;        // [B][N][H + 2 H_kv][d]
    const float* weight[2]; // q, k; null: ones
    const int* pos;         // [B][N]; null: the index in the sequence
    void* out[3];           // forward: q, k, v
    const void* grad[3];    // backward: dq, dk, dv
    void* dqkv;             // backward
    float* part;            // backward: [grid][2][d] partial weight gradients
    int heads[3];           // H, H_kv, H_kv
    int N, rot;
    uint32_t tokens;        // B * N, below 2^31
    float eps;
    RopeFreq freq;
};

// d in {64, 128}; rot a multiple of 16, at most d.
cudaError_t launch_qk_norm_rope(const NormRopeArgs& a, int d, int f32, int interleaved, cudaStream_t s);
// dweight[0/1]: d floats each, or null.
cudaError_t launch_qk_norm_rope_bwd(const NormRopeArgs& a, float* const (&dweight)[2], int d, int f32,
                                    int interleaved, cudaStream_t s);
size_t qk_norm_rope_bwd_workspace_bytes(int d);

// The paged 4-bit cache (layout and code in kv4.cuh).  The four arrays, and where a
// request's tokens are: token i of request b in page table[b * max_blocks + i / page].
struct Kv4Cache {
    uint8_t* codes[2];   // K, V: [n_pages][H_kv][page][d / 2]
    uint16_t* scales[2]; // bfloat16: [n_pages][H_kv][page][d / 32]
    const int* table;
    int H_kv, page_log2, n_pages, max_blocks;
};

// Rows [B][H_kv][N][d] bf16 of K and V into the cache at tokens first[b] + 0 .. count[b] - 1
// (count null: N).
cudaError_t launch_kv4_append(const Kv4Cache& c, const void* k, const void* v, const int* first,
                              const int* count, int B, int N, int d, DevCtl ctl, cudaStream_t s);
// Tokens 0 .. N - 1 out of the cache as bf16 rows [B][H_kv][N][d]; rows from lengths[b] on are zeros.
cudaError_t launch_kv4_read(const Kv4Cache& c, const int* lengths, void* k, void* v, int B, int N, int d,
                            DevCtl ctl, cudaStream_t s);

struct DecodeArgs {
    Kv4Cache cache;
    const void* q;       // [B][H][N_q][d] bf16
    const int* lengths;  // [B], the queries' own tokens included
    void* o;             // [B][H][N_q][d] bf16
    float* lse;          // [B][H][N_q], or null
    int B, H, N_q;
    int window;          // 0: every earlier key
    int sinks;
    float c_log2;        // scale * log2(e)
    void* workspace;
    DevCtl ctl;
};
size_t decode_kv4_workspace_bytes(int B, int H, int H_kv, int N_q, int d);
cudaError_t launch_decode_kv4(const DecodeArgs& a, int d, cudaStream_t s);

// Forward under a causal window of `window` keys and the first `sinks` keys: bf16, d in {64, 128}.
int launch_fwd_window(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int H_kv, int N,
                      int d, float c_log2, int window, int sinks, DevCtl ctl, cudaStream_t s);

int launch_fwd_window64(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int H_kv, int N,
                        float c_log2, int window, int sinks, DevCtl ctl, cudaStream_t s);

// The windowed backward's deal: key block j meets query blocks j .. j + reach; the first
// n_part blocks (those with sinks and more query blocks after that) leave the rest to
// `pieces` pieces of `per` query blocks.
struct WinSplit {
    int window, sinks, reach, n_part, per, pieces;
};
WinSplit win_split(int B, int H_kv, int N, int window, int sinks);
size_t bwd_window_workspace_bytes(int B, int H, int H_kv, int N, int d, int window, int sinks);
int launch_bwd_window(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
                      void* dq, void* dk, void* dv, void* workspace, int B, int H, int H_kv, int N, int d, float scale,
                      int window, int sinks, DevCtl ctl, cudaStream_t s);

constexpr int kDevIndex = 5;  // == FA_ERR_DEVICE_INDEX: a page or length outside the cache

}  // namespace fa
