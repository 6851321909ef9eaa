// qmv_kv.h -- parameters and host-side launch hooks of the paged-cache calls
// (internal; the public interface is include/qmv.h).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace qmv {

// Device status bits (mirror QMV_DEV_* in include/qmv.h).
constexpr int kDevBadPage = 0x4;
constexpr int kDevNoPages = 0x8;
constexpr int kDevBadLength = 0x10;

// The current device's status word and SM count, and the launch mode.
cudaError_t call_env(int **status, int *sms, bool *pdl);

// How cached rows are held (QMV_KV_* in include/qmv.h).
constexpr int kKvF16 = 0;
constexpr int kKvQ8 = 1;

struct PagesParams {
    const int32_t *len, *n_new, *free_pages, *head, *tree, *held;
    int32_t *table, *start, *kv_len, *slots, *pos, *request, *head_out, *held_out;
    int64_t n_free, R, width, T;
    int tree_words, page_shift;
    int64_t n_pages;
    int *status;
};

struct AppendParams {
    const void *x;               // [T][Hq + 2 Hkv][D], fp32 or fp16
    const float *cos_t, *sin_t;  // [n_pos][rot / 2]
    const int32_t *slots, *pos;
    __half *q;                   // [T][Hq][D]
    void *k, *v;                 // [n_pages][Hkv][page][D]
    float *k_scale, *v_scale;    // [n_pages][Hkv][page] (8-bit cache)
    int64_t T, x_stride, page_stride, n_pos, n_slots;
    int Hq, Hkv, rot, page_shift;
    int *status;
};

// The cache write with norms and with positions of several axes.
struct NormAppendParams {
    AppendParams a;
    const float *q_norm, *k_norm;        // [1 or heads][D], or null
    int q_norm_stride, k_norm_stride;    // 0: one row for all heads
    float eps;
    int axes;                            // rows of a.pos, pos_stride apart
    int64_t pos_stride;
    uint32_t axis_bits[4];               // two bits to each of rot / 2 frequencies: its axis
    int units;                           // warps that share a token's rows (set by the launcher)
};

// The accepted path of each request's drafted tree.
struct AcceptParams {
    const int32_t *tokens, *sampled, *start, *kv_len, *tree;
    const int32_t *slots;                // [T], negative where a node has no cache row; or null
    int32_t *path, *count, *next, *lens;
    int64_t R, T;
    int tree_words;
    int *status;
};

// Rows of kept nodes moved to the front of their request's new places, in several caches at once.
constexpr int kKeepCaches = 64;
struct KeepParams {
    void *k[kKeepCaches], *v[kKeepCaches];
    float *k_scale[kKeepCaches], *v_scale[kKeepCaches];
    const int32_t *slots, *start, *path, *count;
    int64_t R, T, page_stride, n_slots;
    int caches, Hkv, page_shift;
    int *status;
};

struct AttnParams {
    const __half *q;             // [T][Hq][D], token stride q_stride
    const void *k, *v;           // [n_pages][Hkv][page][D], page stride page_stride (elements)
    const float *k_scale, *v_scale;
    const int32_t *table, *start, *kv_len, *tree;
    __half *out;                 // [T][Hq][D]
    void *workspace;
    int64_t q_stride, page_stride, R, T, width, n_pages;
    int Hq, Hkv, group, tree_words, page_shift;
    float scale_log2;            // softmax scale times log2(e)
    int *status;
    int test_skip_copy;          // failure-detection test only: CTA 0 never requests its first keys
};

cudaError_t launch_kv_pages(const PagesParams &p, int sms, cudaStream_t s, bool pdl);
cudaError_t launch_kv_append(const AppendParams &p, int D, bool x_f32, int kind, bool interleaved, int sms,
                             cudaStream_t s, bool pdl);
cudaError_t launch_kv_append_norm(NormAppendParams p, int D, bool x_f32, int kind, bool interleaved, int sms,
                                  cudaStream_t s, bool pdl);
cudaError_t launch_tree_accept(const AcceptParams &p, cudaStream_t s, bool pdl);
cudaError_t launch_kv_keep(const KeepParams &p, int D, int kind, cudaStream_t s, bool pdl);
cudaError_t launch_tree_attn(const AttnParams &p, int D, int kind, int sms, cudaStream_t s, bool pdl);
// Bytes of workspace launch_tree_attn needs on a device with `sms` SMs.
int64_t tree_attn_workspace_bytes(int sms);

}  // namespace qmv
