// layer_api.cu -- the extern "C" entry points of the layer's work around the attention call:
// argument checks and dispatch.
#include <cmath>
#include <cstdint>

#include "../../include/fa.h"
#include "internal.h"
#include "kv4.cuh"
#include "layer_ops.h"
#include "rope_turns.h"

namespace fa {
namespace {

template <typename... P>
bool pointers_ok(const P*... p) {  // non-null and 16-byte aligned
    for (const void* x : {static_cast<const void*>(p)...})
        if (x == nullptr || (reinterpret_cast<uintptr_t>(x) & 15u) != 0) return false;
    return true;
}
template <typename... P>
bool optional_ok(const P*... p) {  // null, or 16-byte aligned
    for (const void* x : {static_cast<const void*>(p)...})
        if ((reinterpret_cast<uintptr_t>(x) & 15u) != 0) return false;
    return true;
}

int from_cuda(cudaError_t e) { return e == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

// Sizes of the norm and rotation: B tokens' rows times H + 2 H_kv heads.
int norm_rope_sizes(int B, int H, int H_kv, int N, int d) {
    if (B < 1 || H < 1 || H_kv < 1 || N < 1) return FA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
    if (!sizes_supported(B, H, N) || !sizes_supported(B, H_kv, N)) return FA_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(B) * N > 0x7fffffffll) return FA_ERR_UNSUPPORTED;
    return FA_OK;
}

int norm_rope_args(NormRopeArgs* a, const void* qkv, const float* qw, const float* kw, const int* pos,
                   const double* inv_freq, int B, int H, int H_kv, int N, int d, int rot, float eps, int dtype) {
    if (!pointers_ok(qkv) || !optional_ok(qw, kw, pos)) return FA_ERR_INVALID_ARG;
    const int rc = norm_rope_sizes(B, H, H_kv, N, d);
    if (rc != FA_OK) return rc;
    if (rot < 0 || rot > d || rot % 16 != 0 || (rot > 0 && inv_freq == nullptr)) return FA_ERR_INVALID_ARG;
    if (!std::isfinite(eps) || eps < 0.f) return FA_ERR_INVALID_ARG;
    if (dtype != FA_F32 && dtype != FA_BF16) return FA_ERR_INVALID_ARG;
    *a = NormRopeArgs{};
    for (int p = 0; p < rot / 2; ++p) {
        if (!(std::fabs(inv_freq[p]) <= kMaxRopeFreq)) return FA_ERR_INVALID_ARG;  // nor NaN
        a->freq.f[p] = rope_turns(inv_freq[p]);
    }
    a->qkv = qkv;
    a->weight[0] = qw;
    a->weight[1] = kw;
    a->pos = pos;
    a->axes = 1;
    a->any_order = false;
    a->heads[0] = H;
    a->heads[1] = a->heads[2] = H_kv;
    a->N = N;
    a->rot = rot;
    a->tokens = static_cast<uint32_t>(B) * N;
    a->eps = eps;
    return FA_OK;
}

int cache_args(Kv4Cache* c, const void* kc, const void* ks, const void* vc, const void* vs, const int* table, int B,
               int H_kv, int d, int page, int n_pages, int max_blocks) {
    if (!pointers_ok(kc, ks, vc, vs, table)) return FA_ERR_INVALID_ARG;
    if (B < 1 || H_kv < 1 || n_pages < 1 || max_blocks < 1) return FA_ERR_INVALID_ARG;
    int log2 = 4;
    while (log2 < 8 && (1 << log2) != page) ++log2;
    if ((1 << log2) != page) return FA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(max_blocks) * page > kMaxTokens) return FA_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(B) * H_kv > (1ll << 24)) return FA_ERR_UNSUPPORTED;
    c->codes[0] = static_cast<uint8_t*>(const_cast<void*>(kc));
    c->codes[1] = static_cast<uint8_t*>(const_cast<void*>(vc));
    c->scales[0] = static_cast<uint16_t*>(const_cast<void*>(ks));
    c->scales[1] = static_cast<uint16_t*>(const_cast<void*>(vs));
    c->table = table;
    c->H_kv = H_kv;
    c->page_log2 = log2;
    c->n_pages = n_pages;
    c->max_blocks = max_blocks;
    return FA_OK;
}

int decode_sizes(int B, int H, int H_kv, int N_q, int d) {
    if (B < 1 || H < 1 || H_kv < 1 || N_q < 1 || H % H_kv != 0) return FA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
    if (!sizes_supported(B, H, N_q) || static_cast<int64_t>(B) * H * N_q > 0x7fffffffll) return FA_ERR_UNSUPPORTED;
    return FA_OK;
}

// Sizes and parameters of the windowed attention, forward and backward.
int window_args(int B, int H, int H_kv, int N, int d, float scale, int window, int n_sink, int dtype) {
    if (B < 1 || H < 1 || N < 1 || H_kv < 1 || H % H_kv != 0) return FA_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || window < 1 || n_sink < 0) return FA_ERR_INVALID_ARG;
    if (dtype != FA_F32 && dtype != FA_BF16) return FA_ERR_INVALID_ARG;
    if (dtype != FA_BF16 || (d != 64 && d != 128) || !sizes_supported(B, H, N)) return FA_ERR_UNSUPPORTED;
    return FA_OK;
}

// Sizes of attention to another sequence's keys.
int cross_sizes(int B, int B_kv, int H, int H_kv, int N_q, int N_kv, int d) {
    if (B < 1 || B_kv < 1 || H < 1 || H_kv < 1 || N_q < 1 || N_kv < 1 || B % B_kv != 0 || H % H_kv != 0)
        return FA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
    if (!sizes_supported(B, H, N_q) || !sizes_supported(B_kv, H_kv, N_kv)) return FA_ERR_UNSUPPORTED;
    // the rows that share a K/V head in one batch are counted in an int, a tile's past the end included
    if (static_cast<int64_t>(H / H_kv) * N_q > 0x7fffffffll - 256) return FA_ERR_UNSUPPORTED;
    return FA_OK;
}
int cross_args(int B, int B_kv, int H, int H_kv, int N_q, int N_kv, int d, float scale, int dtype) {
    if (!std::isfinite(scale) || (dtype != FA_F32 && dtype != FA_BF16)) return FA_ERR_INVALID_ARG;
    const int rc = cross_sizes(B, B_kv, H, H_kv, N_q, N_kv, d);
    if (rc != FA_OK) return rc;
    return dtype == FA_BF16 ? FA_OK : FA_ERR_UNSUPPORTED;
}

}  // namespace
}  // namespace fa

using namespace fa;

#define FA_API extern "C" __attribute__((visibility("default")))

namespace {

// Positions' axes and each pair's own.
int norm_rope_axes(NormRopeArgs* a, const int* axis, int n_axes) {
    if (n_axes < 1 || n_axes > kMaxRopeAxes) return FA_ERR_INVALID_ARG;
    if (a->rot > 0 && (axis == nullptr || a->pos == nullptr)) return FA_ERR_INVALID_ARG;
    a->axes = n_axes;
    a->any_order = true;  // (fa_qk_norm_rope_bwd keeps its own)
    for (int p = 0; p < a->rot / 2; ++p) {
        if (axis[p] < 0 || axis[p] >= n_axes) return FA_ERR_INVALID_ARG;
        a->axis[p] = static_cast<uint8_t>(axis[p]);
    }
    return FA_OK;
}

int norm_rope_forward(NormRopeArgs& a, void* q, void* k, void* v, int d, int interleaved, int dtype, void* stream) {
    a.out[0] = q;
    a.out[1] = k;
    a.out[2] = v;
    return from_cuda(launch_qk_norm_rope(a, d, dtype == FA_F32, interleaved ? 1 : 0, static_cast<cudaStream_t>(stream)));
}

int norm_rope_backward(NormRopeArgs& a, const void* dq, const void* dk, const void* dv, void* dqkv, float* dq_weight,
                       float* dk_weight, void* workspace, size_t workspace_bytes, int d, int interleaved, int dtype,
                       void* stream) {
    if ((dq_weight != nullptr || dk_weight != nullptr) &&
        (workspace == nullptr || workspace_bytes < qk_norm_rope_bwd_workspace_bytes(d)))
        return FA_ERR_INVALID_ARG;
    a.grad[0] = dq;
    a.grad[1] = dk;
    a.grad[2] = dv;
    a.dqkv = dqkv;
    a.part = static_cast<float*>(workspace);
    float* const dw[2] = {dq_weight, dk_weight};
    return from_cuda(
        launch_qk_norm_rope_bwd(a, dw, d, dtype == FA_F32, interleaved ? 1 : 0, static_cast<cudaStream_t>(stream)));
}

}  // namespace

FA_API int fa_qk_norm_rope(const void* qkv, const float* q_weight, const float* k_weight, const int* positions,
                           const double* inv_freq, void* q, void* k, void* v, int B, int H, int H_kv, int N, int d,
                           int rot, int interleaved, float eps, int dtype, void* stream) {
    if (!pointers_ok(q, k, v)) return FA_ERR_INVALID_ARG;
    NormRopeArgs a;
    const int rc = norm_rope_args(&a, qkv, q_weight, k_weight, positions, inv_freq, B, H, H_kv, N, d, rot, eps, dtype);
    if (rc != FA_OK) return rc;
    return norm_rope_forward(a, q, k, v, d, interleaved, dtype, stream);
}

FA_API int fa_qk_norm_rope_axes(const void* qkv, const float* q_weight, const float* k_weight, const int* positions,
                                const double* inv_freq, const int* axis, void* q, void* k, void* v, int B, int H,
                                int H_kv, int N, int d, int rot, int n_axes, int interleaved, float eps, int dtype,
                                void* stream) {
    if (!pointers_ok(q, k, v)) return FA_ERR_INVALID_ARG;
    NormRopeArgs a;
    int rc = norm_rope_args(&a, qkv, q_weight, k_weight, positions, inv_freq, B, H, H_kv, N, d, rot, eps, dtype);
    if (rc == FA_OK) rc = norm_rope_axes(&a, axis, n_axes);
    if (rc != FA_OK) return rc;
    return norm_rope_forward(a, q, k, v, d, interleaved, dtype, stream);
}

FA_API size_t fa_qk_norm_rope_bwd_workspace_size(int B, int H, int H_kv, int N, int d) {
    return norm_rope_sizes(B, H, H_kv, N, d) == FA_OK ? qk_norm_rope_bwd_workspace_bytes(d) : 0;
}

FA_API int fa_qk_norm_rope_bwd(const void* qkv, const float* q_weight, const float* k_weight, const int* positions,
                               const double* inv_freq, const void* dq, const void* dk, const void* dv, void* dqkv,
                               float* dq_weight, float* dk_weight, void* workspace, size_t workspace_bytes, int B,
                               int H, int H_kv, int N, int d, int rot, int interleaved, float eps, int dtype,
                               void* stream) {
    if (!pointers_ok(dq, dk, dv, dqkv) || !optional_ok(dq_weight, dk_weight, workspace)) return FA_ERR_INVALID_ARG;
    NormRopeArgs a;
    const int rc = norm_rope_args(&a, qkv, q_weight, k_weight, positions, inv_freq, B, H, H_kv, N, d, rot, eps, dtype);
    if (rc != FA_OK) return rc;
    return norm_rope_backward(a, dq, dk, dv, dqkv, dq_weight, dk_weight, workspace, workspace_bytes, d, interleaved,
                              dtype, stream);
}

FA_API int fa_qk_norm_rope_axes_bwd(const void* qkv, const float* q_weight, const float* k_weight,
                                    const int* positions, const double* inv_freq, const int* axis, const void* dq,
                                    const void* dk, const void* dv, void* dqkv, float* dq_weight, float* dk_weight,
                                    void* workspace, size_t workspace_bytes, int B, int H, int H_kv, int N, int d,
                                    int rot, int n_axes, int interleaved, float eps, int dtype, void* stream) {
    if (!pointers_ok(dq, dk, dv, dqkv) || !optional_ok(dq_weight, dk_weight, workspace)) return FA_ERR_INVALID_ARG;
    NormRopeArgs a;
    int rc = norm_rope_args(&a, qkv, q_weight, k_weight, positions, inv_freq, B, H, H_kv, N, d, rot, eps, dtype);
    if (rc == FA_OK) rc = norm_rope_axes(&a, axis, n_axes);
    if (rc != FA_OK) return rc;
    return norm_rope_backward(a, dq, dk, dv, dqkv, dq_weight, dk_weight, workspace, workspace_bytes, d, interleaved,
                              dtype, stream);
}

FA_API int fa_fwd_window(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int H_kv,
                         int N, int d, float scale, int window, int n_sink, int dtype, void* stream) {
    if (!pointers_ok(q, k, v, o) || !optional_ok(lse)) return FA_ERR_INVALID_ARG;
    const int rc = window_args(B, H, H_kv, N, d, scale, window, n_sink, dtype);
    if (rc != FA_OK) return rc;
    DevCtl ctl;
    int err = FA_OK;
    if (!device_ctl(&ctl, &err)) return err;
    const int e = launch_fwd_window(q, k, v, o, lse, B, H, H_kv, N, d, scale * 1.4426950408889634f, window, n_sink, ctl,
                                    static_cast<cudaStream_t>(stream));
    return e == 0 ? FA_OK : FA_ERR_CUDA;
}

FA_API size_t fa_bwd_window_workspace_size(int B, int H, int H_kv, int N, int d, int window, int n_sink) {
    return window_args(B, H, H_kv, N, d, 1.f, window, n_sink, FA_BF16) == FA_OK
               ? bwd_window_workspace_bytes(B, H, H_kv, N, d, window, n_sink) : 0;
}

FA_API int fa_bwd_window(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
                         void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes, int B, int H, int H_kv,
                         int N, int d, float scale, int window, int n_sink, int dtype, void* stream) {
    if (!pointers_ok(q, k, v, o, lse, dO, dq, dk, dv, workspace)) return FA_ERR_INVALID_ARG;
    const int rc = window_args(B, H, H_kv, N, d, scale, window, n_sink, dtype);
    if (rc != FA_OK) return rc;
    if (workspace_bytes < bwd_window_workspace_bytes(B, H, H_kv, N, d, window, n_sink)) return FA_ERR_INVALID_ARG;
    DevCtl ctl;
    int err = FA_OK;
    if (!device_ctl(&ctl, &err)) return err;
    const int e = launch_bwd_window(q, k, v, o, lse, dO, dq, dk, dv, workspace, B, H, H_kv, N, d, scale, window, n_sink,
                                    ctl, static_cast<cudaStream_t>(stream));
    return e == 0 ? FA_OK : FA_ERR_CUDA;
}

FA_API int fa_kv4_append(const void* k, const void* v, void* k_codes, void* k_scales, void* v_codes, void* v_scales,
                         const int* block_table, const int* first, const int* count, int B, int H_kv, int N, int d,
                         int page, int n_pages, int max_blocks, void* stream) {
    if (!pointers_ok(k, v, first) || !optional_ok(count) || N < 1) return FA_ERR_INVALID_ARG;
    Kv4Cache c;
    const int rc = cache_args(&c, k_codes, k_scales, v_codes, v_scales, block_table, B, H_kv, d, page, n_pages, max_blocks);
    if (rc != FA_OK) return rc;
    if (!sizes_supported(B, H_kv, N) || static_cast<int64_t>(B) * H_kv * N > 0x7fffffffll) return FA_ERR_UNSUPPORTED;
    DevCtl ctl;
    int err = FA_OK;
    if (!device_ctl(&ctl, &err)) return err;
    return from_cuda(launch_kv4_append(c, k, v, first, count, B, N, d, ctl, static_cast<cudaStream_t>(stream)));
}

FA_API int fa_kv4_read(const void* k_codes, const void* k_scales, const void* v_codes, const void* v_scales,
                       const int* block_table, const int* lengths, void* k, void* v, int B, int H_kv, int N, int d,
                       int page, int n_pages, int max_blocks, void* stream) {
    if (!pointers_ok(k, v, lengths) || N < 1) return FA_ERR_INVALID_ARG;
    Kv4Cache c;
    const int rc = cache_args(&c, k_codes, k_scales, v_codes, v_scales, block_table, B, H_kv, d, page, n_pages, max_blocks);
    if (rc != FA_OK) return rc;
    if (!sizes_supported(B, H_kv, N) || static_cast<int64_t>(B) * H_kv * N > 0x7fffffffll) return FA_ERR_UNSUPPORTED;
    DevCtl ctl;
    int err = FA_OK;
    if (!device_ctl(&ctl, &err)) return err;
    return from_cuda(launch_kv4_read(c, lengths, k, v, B, N, d, ctl, static_cast<cudaStream_t>(stream)));
}

FA_API size_t fa_decode_kv4_workspace_size(int B, int H, int H_kv, int N_q, int d) {
    return decode_sizes(B, H, H_kv, N_q, d) == FA_OK ? decode_kv4_workspace_bytes(B, H, H_kv, N_q, d) : 0;
}

FA_API int fa_decode_kv4(const void* q, const void* k_codes, const void* k_scales, const void* v_codes,
                         const void* v_scales, const int* block_table, const int* lengths, void* o, float* lse,
                         void* workspace, size_t workspace_bytes, int B, int H, int H_kv, int N_q, int d, int page,
                         int n_pages, int max_blocks, float scale, int window, int n_sink, void* stream) {
    if (!pointers_ok(q, lengths, o, workspace) || !optional_ok(lse)) return FA_ERR_INVALID_ARG;
    int rc = decode_sizes(B, H, H_kv, N_q, d);
    if (rc != FA_OK) return rc;
    if (!std::isfinite(scale) || window < 0 || n_sink < 0) return FA_ERR_INVALID_ARG;
    DecodeArgs a;
    rc = cache_args(&a.cache, k_codes, k_scales, v_codes, v_scales, block_table, B, H_kv, d, page, n_pages, max_blocks);
    if (rc != FA_OK) return rc;
    if (workspace_bytes < decode_kv4_workspace_bytes(B, H, H_kv, N_q, d)) return FA_ERR_INVALID_ARG;
    a.q = q;
    a.lengths = lengths;
    a.o = o;
    a.lse = lse;
    a.B = B;
    a.H = H;
    a.N_q = N_q;
    a.window = window;
    a.sinks = n_sink;
    a.c_log2 = scale * 1.4426950408889634f;
    a.workspace = workspace;
    int err = FA_OK;
    if (!device_ctl(&a.ctl, &err)) return err;
    return from_cuda(launch_decode_kv4(a, d, static_cast<cudaStream_t>(stream)));
}

namespace {

int cross_forward(const void* q, const void* k, const void* v, const int* lengths, const void* o_own,
                  const float* lse_own, void* o, float* lse, void* workspace, size_t workspace_bytes, int B, int B_kv,
                  int H, int H_kv, int N_q, int N_kv, int d, float scale, int dtype, void* stream) {
    if (!pointers_ok(q, k, v, o) || !optional_ok(lengths, lse, workspace)) return FA_ERR_INVALID_ARG;
    int rc = cross_args(B, B_kv, H, H_kv, N_q, N_kv, d, scale, dtype);
    if (rc != FA_OK) return rc;
    const size_t need = fwd_cross_workspace_bytes(B, B_kv, H, H_kv, N_q, N_kv, d);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return FA_ERR_INVALID_ARG;
    DevCtl ctl;
    if (!device_ctl(&ctl, &rc)) return rc;
    const int e = launch_fwd_cross(q, k, v, lengths, o_own, lse_own, o, lse, workspace, B, B_kv, H, H_kv, N_q, N_kv, d,
                                   scale * 1.4426950408889634f, ctl, static_cast<cudaStream_t>(stream));
    return e == 0 ? FA_OK : FA_ERR_CUDA;
}

}  // namespace

FA_API int fa_fwd_cross(const void* q, const void* k, const void* v, const int* kv_lengths, void* o, float* lse,
                        void* workspace, size_t workspace_bytes, int B, int B_kv, int H, int H_kv, int N_q, int N_kv,
                        int d, float scale, int dtype, void* stream) {
    return cross_forward(q, k, v, kv_lengths, nullptr, nullptr, o, lse, workspace, workspace_bytes, B, B_kv, H, H_kv,
                         N_q, N_kv, d, scale, dtype, stream);
}

FA_API size_t fa_fwd_cross_workspace_size(int B, int B_kv, int H, int H_kv, int N_q, int N_kv, int d) {
    return cross_sizes(B, B_kv, H, H_kv, N_q, N_kv, d) == FA_OK
               ? fwd_cross_workspace_bytes(B, B_kv, H, H_kv, N_q, N_kv, d)
               : 0;
}

FA_API int fa_bwd_cross(const void* q, const void* k, const void* v, const int* kv_lengths, const void* o,
                        const float* lse, const void* dO, void* dq, void* dk, void* dv, void* workspace,
                        size_t workspace_bytes, int B, int B_kv, int H, int H_kv, int N_q, int N_kv, int d, float scale,
                        int dtype, void* stream) {
    if (!pointers_ok(q, k, v, o, lse, dO, dq, dk, dv, workspace) || !optional_ok(kv_lengths)) return FA_ERR_INVALID_ARG;
    int rc = cross_args(B, B_kv, H, H_kv, N_q, N_kv, d, scale, dtype);
    if (rc != FA_OK) return rc;
    if (workspace_bytes < bwd_cross_workspace_bytes(B, B_kv, H, H_kv, N_q, N_kv, d)) return FA_ERR_INVALID_ARG;
    DevCtl ctl;
    if (!device_ctl(&ctl, &rc)) return rc;
    const int e = launch_bwd_cross(q, k, v, kv_lengths, o, lse, dO, dq, dk, dv, workspace, B, B_kv, H, H_kv, N_q, N_kv, d,
                                   scale, ctl, static_cast<cudaStream_t>(stream));
    return e == 0 ? FA_OK : FA_ERR_CUDA;
}

FA_API size_t fa_bwd_cross_workspace_size(int B, int B_kv, int H, int H_kv, int N_q, int N_kv, int d) {
    return cross_sizes(B, B_kv, H, H_kv, N_q, N_kv, d) == FA_OK
               ? bwd_cross_workspace_bytes(B, B_kv, H, H_kv, N_q, N_kv, d)
               : 0;
}

FA_API int fa_fwd_prefix(const void* q, const void* k, const void* v, const int* kv_lengths, const void* o_own,
                         const float* lse_own, void* o, float* lse, void* workspace, size_t workspace_bytes, int B,
                         int B_kv, int H, int H_kv, int N_q, int N_kv, int d, float scale, int dtype, void* stream) {
    if (!pointers_ok(o_own, lse_own)) return FA_ERR_INVALID_ARG;
    return cross_forward(q, k, v, kv_lengths, o_own, lse_own, o, lse, workspace, workspace_bytes, B, B_kv, H, H_kv,
                         N_q, N_kv, d, scale, dtype, stream);
}

FA_API size_t fa_fwd_prefix_workspace_size(int B, int B_kv, int H, int H_kv, int N_q, int N_kv, int d) {
    return fa_fwd_cross_workspace_size(B, B_kv, H, H_kv, N_q, N_kv, d);
}
