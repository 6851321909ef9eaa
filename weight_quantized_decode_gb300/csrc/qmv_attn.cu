// qmv_attn.cu -- attention of new tokens (a chain, or a tree of drafted
// tokens) over the paged key/value cache.
//
//   o = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale q . k_j - max_j)
//
// over the places j that a token sees: everything cached before the request's
// new tokens, and of those the ones its mask row names (no mask: itself and
// the ones before it).  A row that sees nothing gives zeros.
#include <cstdint>

#include "qmv_common.cuh"
#include "qmv_kv.h"
#include "qmv_launch.h"

namespace qmv {

namespace {

constexpr int kWarps = 4;

template <int D, int KIND>
__global__ void __launch_bounds__(kWarps * 32) tree_attn_kernel(const AttnParams p)
{
    constexpr int PER = D / 32;
    pdl_allow_next_grid();
    pdl_wait_prior_grid();
    const int lane = threadIdx.x & 31;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int64_t t = unit / p.Hq;
    const int h = static_cast<int>(unit - t * p.Hq);
    if (t >= p.T || t >= p.start[p.R]) return;
    int64_t lo = 0, hi = p.R;
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) >> 1;
        if (p.start[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    const int64_t r = lo;
    const int node = static_cast<int>(t - p.start[r]);
    const int nodes = p.start[r + 1] - p.start[r];
    const int page = 1 << p.page_shift;
    bool bad = false;
    int64_t len = p.kv_len[r];
    if (len < nodes || len > (p.width << p.page_shift)) {
        bad = true;
        len = 0;
    }
    const int64_t ctx = len - nodes;
    const int kvh = h / p.group;
    float q[D];
    for (int d = 0; d < D; ++d) q[d] = __half2float(p.q[t * p.q_stride + static_cast<int64_t>(h) * D + d]);
    float m = -INFINITY, l = 0.0f, o[PER] = {};
    for (int64_t j0 = 0; j0 < len; j0 += 32) {
        const int64_t j = j0 + lane;
        bool sees = j < len;
        if (sees && j >= ctx) {
            const int n = static_cast<int>(j - ctx);
            sees = p.tree ? (n < 32 * p.tree_words && (p.tree[t * p.tree_words + (n >> 5)] >> (n & 31) & 1)) : n <= node;
        }
        int64_t row = 0;
        if (sees) {
            const int32_t id = p.table[r * p.width + (j >> p.page_shift)];
            if (id < 0 || id >= p.n_pages) {
                bad = true;
                sees = false;
            } else {
                row = static_cast<int64_t>(id) * p.page_stride +
                      ((static_cast<int64_t>(kvh) << p.page_shift) + (j & (page - 1))) * D;
            }
        }
        const int64_t cell = sees ? (static_cast<int64_t>(p.table[r * p.width + (j >> p.page_shift)]) * p.Hkv + kvh) * page +
                                        (j & (page - 1))
                                  : 0;
        float s = -INFINITY;
        if (sees) {
            s = 0.0f;
            for (int d = 0; d < D; ++d)
                s += q[d] * (KIND == kKvF16 ? __half2float(static_cast<const __half *>(p.k)[row + d])
                                            : static_cast<float>(static_cast<const int8_t *>(p.k)[row + d]));
            if (KIND == kKvQ8) s *= p.k_scale[cell];
            s *= p.scale_log2;
        }
        float top = s;
        for (int i = 16; i; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
        if (top == -INFINITY) continue;
        const float mn = fmaxf(m, top);
        const float fix = exp2f(m - mn);
        const float w = sees ? exp2f(s - mn) : 0.0f;
        float ws = w;
        for (int i = 16; i; i >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, i);
        l = l * fix + ws;
        m = mn;
        for (int k = 0; k < PER; ++k) o[k] *= fix;
        for (int i = 0; i < 32; ++i) {
            const float wi = __shfl_sync(0xffffffffu, w, i);
            const int64_t ri = __shfl_sync(0xffffffffu, row, i), ci = __shfl_sync(0xffffffffu, cell, i);
            if (!__shfl_sync(0xffffffffu, sees ? 1 : 0, i)) continue;
            for (int k = 0; k < PER; ++k) {
                const int d = k * 32 + lane;
                const float v = KIND == kKvF16 ? __half2float(static_cast<const __half *>(p.v)[ri + d])
                                               : static_cast<const int8_t *>(p.v)[ri + d] * p.v_scale[ci];
                o[k] += wi * v;
            }
        }
    }
    bad = __any_sync(0xffffffffu, bad);
    if (bad && lane == 0) atomicOr(p.status, kDevBadPage);
    for (int k = 0; k < PER; ++k)
        p.out[(t * p.Hq + h) * D + k * 32 + lane] =
            __float2half_rn(bad ? __int_as_float(0x7fffffff) : (l > 0.0f || l != l ? o[k] / l : 0.0f));
}

}  // namespace

int64_t tree_attn_workspace_bytes(int) { return 0; }

cudaError_t launch_tree_attn(const AttnParams &p, int D, int kind, int, cudaStream_t s, bool pdl)
{
    const int64_t units = p.T * p.Hq;
    const dim3 grid(static_cast<unsigned>((units + kWarps - 1) / kWarps));
    if (D == 64)
        return kind == kKvF16 ? launch_ex(tree_attn_kernel<64, kKvF16>, grid, dim3(kWarps * 32), 0, s, pdl, p)
                              : launch_ex(tree_attn_kernel<64, kKvQ8>, grid, dim3(kWarps * 32), 0, s, pdl, p);
    return kind == kKvF16 ? launch_ex(tree_attn_kernel<128, kKvF16>, grid, dim3(kWarps * 32), 0, s, pdl, p)
                          : launch_ex(tree_attn_kernel<128, kKvQ8>, grid, dim3(kWarps * 32), 0, s, pdl, p);
}

}  // namespace qmv
