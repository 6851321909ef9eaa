// qmv_kv_api.cu -- C entry points of the paged-cache calls (include/qmv.h):
// argument validation and the hand-over to the launchers.
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <cstring>

#include "../../include/qmv.h"
#include "qmv_kv.h"

namespace qmv {

namespace {

constexpr int64_t kInt32Max = 0x7fffffff;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// log2 of a page size the calls take (a power of two, 16 .. 256), or -1.
int page_shift_of(int64_t page)
{
    for (int s = 4; s <= 8; ++s)
        if (page == (int64_t(1) << s)) return s;
    return -1;
}

// Shape of a cache: pages whose slots fit int32, head layouts the kernels take.
qmv_status check_cache(int64_t n_pages, int64_t Hkv, int64_t page, int64_t D, int64_t page_stride, int kind)
{
    if (page_shift_of(page) < 0 || (D != 64 && D != 128) || Hkv < 1 || Hkv > 1024) return QMV_ERR_SHAPE;
    if (n_pages < 1 || n_pages * page > kInt32Max) return QMV_ERR_SHAPE;
    if (kind != QMV_KV_F16 && kind != QMV_KV_Q8) return QMV_ERR_SHAPE;
    if (page_stride < Hkv * page * D || page_stride > (int64_t(1) << 38)) return QMV_ERR_SHAPE;
    // 16-byte rows of every page: the strides the copies need
    if ((page_stride * (kind == QMV_KV_F16 ? 2 : 1)) % 16 != 0) return QMV_ERR_ALIGN;
    return QMV_OK;
}

// Failure detection is tested without a GPU fault: QMV_TEST_SKIP_COPY="attn:N"
// makes the N-th attention launch (counted from 1) of this process skip a copy
// whose bytes a barrier still expects.  The waits on it run out, the kernel
// records QMV_DEV_TIMEOUT, gives that CTA's outputs as NaN and returns.  Unset
// in every normal run.
bool test_skip_this_launch()
{
    static const long long armed = [] {
        const char *e = std::getenv("QMV_TEST_SKIP_COPY");
        return e && !std::strncmp(e, "attn:", 5) ? std::atoll(e + 5) : 0ll;
    }();
    static std::atomic<long long> seen{0};
    return armed > 0 && seen.fetch_add(1) + 1 == armed;
}

}  // namespace

}  // namespace qmv

using namespace qmv;

extern "C" {

qmv_status qmv_kv_pages(const int32_t *len, const int32_t *n_new, const int32_t *free_pages, int64_t n_free,
                        const int32_t *head, const int32_t *tree, int64_t tree_words, int32_t *table,
                        int32_t *start, int32_t *kv_len, int32_t *slots, int32_t *pos, int32_t *request,
                        int32_t *head_out, int64_t R, int64_t width, int64_t page, int64_t n_pages, int64_t T,
                        qmv_stream_t stream)
{
    return qmv_kv_pages_held(len, n_new, free_pages, n_free, head, tree, tree_words, table, nullptr, start, kv_len, slots,
                             pos, request, head_out, nullptr, R, width, page, n_pages, T, stream);
}

qmv_status qmv_kv_pages_held(const int32_t *len, const int32_t *n_new, const int32_t *free_pages, int64_t n_free,
                             const int32_t *head, const int32_t *tree, int64_t tree_words, int32_t *table,
                             const int32_t *held, int32_t *start, int32_t *kv_len, int32_t *slots, int32_t *pos,
                             int32_t *request, int32_t *head_out, int32_t *held_out, int64_t R, int64_t width,
                             int64_t page, int64_t n_pages, int64_t T, qmv_stream_t stream)
{
    const int shift = page_shift_of(page);
    if (shift < 0 || R < 0 || R > kInt32Max || width < 0 || width > kInt32Max || T < 0 || T > kInt32Max ||
        n_free < 0 || n_free > kInt32Max || n_pages < 1 || n_pages > kInt32Max / page || tree_words < 0 ||
        tree_words > 65536 || (tree && tree_words == 0))
        return QMV_ERR_SHAPE;
    if (R == 0 && T == 0 && !start && !head_out) return QMV_OK;
    if ((R > 0 && (!len || !n_new || !start || !kv_len)) || (R > 0 && width > 0 && !table) || (n_free > 0 && !free_pages) ||
        (T > 0 && (!slots || !pos || !request)))
        return QMV_ERR_NULL;
    for (const void *p : {static_cast<const void *>(len), static_cast<const void *>(n_new),
                          static_cast<const void *>(free_pages), static_cast<const void *>(head),
                          static_cast<const void *>(tree), static_cast<const void *>(table),
                          static_cast<const void *>(start), static_cast<const void *>(kv_len),
                          static_cast<const void *>(slots), static_cast<const void *>(pos),
                          static_cast<const void *>(request), static_cast<const void *>(head_out),
                          static_cast<const void *>(held), static_cast<const void *>(held_out)})
        if (!aligned(p, 4)) return QMV_ERR_ALIGN;
    PagesParams p = {};
    int sms = 0;
    bool pdl = false;
    if (call_env(&p.status, &sms, &pdl) != cudaSuccess) return QMV_ERR_CUDA;
    p.len = len;
    p.n_new = n_new;
    p.free_pages = free_pages;
    p.head = head;
    p.tree = tree;
    p.table = table;
    p.start = start;
    p.kv_len = kv_len;
    p.slots = slots;
    p.pos = pos;
    p.request = request;
    p.head_out = head_out;
    p.held = held;
    p.held_out = held_out;
    p.n_free = n_free;
    p.R = R;
    p.width = width;
    p.T = T;
    p.tree_words = static_cast<int>(tree_words);
    p.page_shift = shift;
    p.n_pages = n_pages;
    if (launch_kv_pages(p, sms, reinterpret_cast<cudaStream_t>(stream), pdl) != cudaSuccess) {
        (void)cudaGetLastError();
        return QMV_ERR_LAUNCH;
    }
    return QMV_OK;
}

qmv_status qmv_kv_append(const void *qkv, int64_t stride, int qkv_f32, const int32_t *slots, const int32_t *pos,
                         const float *cos_table, const float *sin_table, int64_t n_pos, int64_t rot,
                         int interleaved, void *q, void *k, void *v, float *k_scale, float *v_scale, int kind,
                         int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t n_pages, int64_t page,
                         int64_t page_stride, qmv_stream_t stream)
{
    const qmv_status st = check_cache(n_pages, Hkv, page, D, page_stride, kind);
    if (st != QMV_OK) return st;
    if (T < 0 || T > kInt32Max || Hq < 0 || Hq > 65536 || rot < 0 || rot > D || rot % 8 != 0 ||
        stride < (Hq + 2 * Hkv) * D || stride > (int64_t(1) << 31) || n_pos < 0 || (rot > 0 && n_pos > kInt32Max))
        return QMV_ERR_SHAPE;
    if (T == 0) return QMV_OK;
    if (!qkv || !slots || !k || !v || (Hq > 0 && !q) || (kind == QMV_KV_Q8 && (!k_scale || !v_scale)) ||
        (rot > 0 && (!pos || !cos_table || !sin_table)))
        return QMV_ERR_NULL;
    if (!aligned(qkv, qkv_f32 ? 16 : 8) || stride % 4 != 0 || !aligned(k, 16) || !aligned(v, 16) || !aligned(q, 16) ||
        !aligned(slots, 4) || !aligned(pos, 4) || !aligned(cos_table, 16) || !aligned(sin_table, 16) ||
        !aligned(k_scale, 16) || !aligned(v_scale, 16))
        return QMV_ERR_ALIGN;
    AppendParams p = {};
    int sms = 0;
    bool pdl = false;
    if (call_env(&p.status, &sms, &pdl) != cudaSuccess) return QMV_ERR_CUDA;
    p.x = qkv;
    p.cos_t = cos_table;
    p.sin_t = sin_table;
    p.slots = slots;
    p.pos = pos;
    p.q = static_cast<__half *>(q);
    p.k = k;
    p.v = v;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.T = T;
    p.x_stride = stride;
    p.page_stride = page_stride;
    p.n_pos = n_pos;
    p.n_slots = n_pages * page;
    p.Hq = static_cast<int>(Hq);
    p.Hkv = static_cast<int>(Hkv);
    p.rot = static_cast<int>(rot);
    p.page_shift = page_shift_of(page);
    if (launch_kv_append(p, static_cast<int>(D), qkv_f32 != 0, kind, interleaved != 0, sms,
                         reinterpret_cast<cudaStream_t>(stream), pdl) != cudaSuccess) {
        (void)cudaGetLastError();
        return QMV_ERR_LAUNCH;
    }
    return QMV_OK;
}

qmv_status qmv_kv_append_norm(const void *qkv, int64_t stride, int qkv_f32, const int32_t *slots, const int32_t *pos,
                              int64_t axes, int64_t pos_stride, const int8_t *axis_of, const float *cos_table,
                              const float *sin_table, int64_t n_pos, int64_t rot, int interleaved, const float *q_norm,
                              int64_t q_norm_stride, const float *k_norm, int64_t k_norm_stride, const float *eps,
                              void *q, void *k, void *v, float *k_scale, float *v_scale, int kind, int64_t T, int64_t Hq,
                              int64_t Hkv, int64_t D, int64_t n_pages, int64_t page, int64_t page_stride,
                              qmv_stream_t stream)
{
    const qmv_status st = check_cache(n_pages, Hkv, page, D, page_stride, kind);
    if (st != QMV_OK) return st;
    if (T < 0 || T > kInt32Max || Hq < 0 || Hq > 65536 || rot < 0 || rot > D || rot % 8 != 0 ||
        stride < (Hq + 2 * Hkv) * D || stride > (int64_t(1) << 31) || n_pos < 0 ||
        (rot > 0 && (n_pos > kInt32Max || axes < 1 || axes > 4 || pos_stride < 0 || pos_stride > (int64_t(1) << 40))) ||
        (q_norm && q_norm_stride != 0 && q_norm_stride != D) || (k_norm && k_norm_stride != 0 && k_norm_stride != D) ||
        (eps && !(*eps >= 1e-30f && *eps <= 1e30f)))
        return QMV_ERR_SHAPE;
    NormAppendParams p = {};
    for (int64_t i = 0; rot > 0 && axis_of && i < rot / 2; ++i) {
        if (axis_of[i] < 0 || axis_of[i] >= axes) return QMV_ERR_SHAPE;
        p.axis_bits[i / 16] |= static_cast<uint32_t>(axis_of[i]) << (2 * (i % 16));
    }
    if (T == 0) return QMV_OK;
    if (!qkv || !slots || !k || !v || (Hq > 0 && !q) || (kind == QMV_KV_Q8 && (!k_scale || !v_scale)) ||
        (rot > 0 && (!pos || !cos_table || !sin_table)))
        return QMV_ERR_NULL;
    if (!aligned(qkv, qkv_f32 ? 16 : 8) || stride % 4 != 0 || !aligned(k, 16) || !aligned(v, 16) || !aligned(q, 16) ||
        !aligned(slots, 4) || !aligned(pos, 4) || !aligned(cos_table, 16) || !aligned(sin_table, 16) ||
        !aligned(k_scale, 16) || !aligned(v_scale, 16) || !aligned(q_norm, 16) || !aligned(k_norm, 16))
        return QMV_ERR_ALIGN;
    int sms = 0;
    bool pdl = false;
    if (call_env(&p.a.status, &sms, &pdl) != cudaSuccess) return QMV_ERR_CUDA;
    p.a.x = qkv;
    p.a.cos_t = cos_table;
    p.a.sin_t = sin_table;
    p.a.slots = slots;
    p.a.pos = pos;
    p.a.q = static_cast<__half *>(q);
    p.a.k = k;
    p.a.v = v;
    p.a.k_scale = k_scale;
    p.a.v_scale = v_scale;
    p.a.T = T;
    p.a.x_stride = stride;
    p.a.page_stride = page_stride;
    p.a.n_pos = n_pos;
    p.a.n_slots = n_pages * page;
    p.a.Hq = static_cast<int>(Hq);
    p.a.Hkv = static_cast<int>(Hkv);
    p.a.rot = static_cast<int>(rot);
    p.a.page_shift = page_shift_of(page);
    p.q_norm = q_norm;
    p.k_norm = k_norm;
    p.q_norm_stride = static_cast<int>(q_norm_stride);
    p.k_norm_stride = static_cast<int>(k_norm_stride);
    p.eps = eps ? *eps : 1e-6f;
    p.axes = rot > 0 ? static_cast<int>(axes) : 0;
    p.pos_stride = pos_stride;
    if (launch_kv_append_norm(p, static_cast<int>(D), qkv_f32 != 0, kind, interleaved != 0, sms,
                              reinterpret_cast<cudaStream_t>(stream), pdl) != cudaSuccess) {
        (void)cudaGetLastError();
        return QMV_ERR_LAUNCH;
    }
    return QMV_OK;
}

qmv_status qmv_tree_accept_slots(const int32_t *tokens, const int32_t *sampled, const int32_t *start,
                                 const int32_t *kv_len, const int32_t *tree, int64_t tree_words,
                                 const int32_t *slots, int32_t *path, int32_t *count, int32_t *next, int32_t *lens,
                                 int64_t R, int64_t T, qmv_stream_t stream)
{
    if (R < 0 || R > kInt32Max || T < 0 || T > kInt32Max || tree_words < 0 || tree_words > 65536 ||
        (tree && tree_words == 0))
        return QMV_ERR_SHAPE;
    if (R == 0 && T == 0) return QMV_OK;
    if ((R > 0 && (!start || !kv_len || !count || !next || !lens)) || (T > 0 && (!tokens || !sampled || !path)))
        return QMV_ERR_NULL;
    for (const int32_t *a : {tokens, sampled, start, kv_len, tree, slots, static_cast<const int32_t *>(path),
                             static_cast<const int32_t *>(count), static_cast<const int32_t *>(next),
                             static_cast<const int32_t *>(lens)})
        if (!aligned(a, 4)) return QMV_ERR_ALIGN;
    AcceptParams p = {};
    int sms = 0;
    bool pdl = false;
    if (call_env(&p.status, &sms, &pdl) != cudaSuccess) return QMV_ERR_CUDA;
    p.tokens = tokens;
    p.sampled = sampled;
    p.start = start;
    p.kv_len = kv_len;
    p.tree = tree;
    p.slots = slots;
    p.path = path;
    p.count = count;
    p.next = next;
    p.lens = lens;
    p.R = R;
    p.T = T;
    p.tree_words = static_cast<int>(tree_words);
    if (launch_tree_accept(p, reinterpret_cast<cudaStream_t>(stream), pdl) != cudaSuccess) {
        (void)cudaGetLastError();
        return QMV_ERR_LAUNCH;
    }
    return QMV_OK;
}

qmv_status qmv_tree_accept(const int32_t *tokens, const int32_t *sampled, const int32_t *start, const int32_t *kv_len,
                           const int32_t *tree, int64_t tree_words, int32_t *path, int32_t *count, int32_t *next,
                           int32_t *lens, int64_t R, int64_t T, qmv_stream_t stream)
{
    return qmv_tree_accept_slots(tokens, sampled, start, kv_len, tree, tree_words, nullptr, path, count, next, lens, R, T,
                                 stream);
}

qmv_status qmv_kv_keep(const void *rows, int64_t caches, int kind, const int32_t *slots, const int32_t *start,
                       const int32_t *path, const int32_t *count, int64_t R, int64_t T, int64_t Hkv, int64_t D,
                       int64_t n_pages, int64_t page, int64_t page_stride, qmv_stream_t stream)
{
    const qmv_status st = check_cache(n_pages, Hkv, page, D, page_stride, kind);
    if (st != QMV_OK) return st;
    if (R < 0 || R > kInt32Max || T < 0 || T > kInt32Max || caches < 0 || caches > 4096) return QMV_ERR_SHAPE;
    if (R == 0 || T == 0 || caches == 0) return QMV_OK;
    if (!rows || !slots || !start || !path || !count) return QMV_ERR_NULL;
    const qmv_kv_rows *c = static_cast<const qmv_kv_rows *>(rows);
    for (int64_t i = 0; i < caches; ++i) {
        if (!c[i].k || !c[i].v || (kind == QMV_KV_Q8 && (!c[i].k_scale || !c[i].v_scale))) return QMV_ERR_NULL;
        if (!aligned(c[i].k, 16) || !aligned(c[i].v, 16)) return QMV_ERR_ALIGN;
        if (kind == QMV_KV_Q8 && (!aligned(c[i].k_scale, 16) || !aligned(c[i].v_scale, 16))) return QMV_ERR_ALIGN;
        // rows that are named twice would be moved twice, at the same time
        if (c[i].k == c[i].v) return QMV_ERR_SHAPE;
        for (int64_t j = 0; j < i; ++j)
            if (c[i].k == c[j].k || c[i].v == c[j].v || c[i].k == c[j].v || c[i].v == c[j].k) return QMV_ERR_SHAPE;
    }
    if (!aligned(slots, 4) || !aligned(start, 4) || !aligned(path, 4) || !aligned(count, 4)) return QMV_ERR_ALIGN;
    KeepParams p = {};
    int sms = 0;
    bool pdl = false;
    if (call_env(&p.status, &sms, &pdl) != cudaSuccess) return QMV_ERR_CUDA;
    p.slots = slots;
    p.start = start;
    p.path = path;
    p.count = count;
    p.R = R;
    p.T = T;
    p.page_stride = page_stride;
    p.n_slots = n_pages * page;
    p.Hkv = static_cast<int>(Hkv);
    p.page_shift = page_shift_of(page);
    for (int64_t first = 0; first < caches; first += kKeepCaches) {
        p.caches = static_cast<int>(caches - first < kKeepCaches ? caches - first : kKeepCaches);
        for (int i = 0; i < p.caches; ++i) {
            p.k[i] = c[first + i].k;
            p.v[i] = c[first + i].v;
            p.k_scale[i] = kind == QMV_KV_Q8 ? c[first + i].k_scale : nullptr;
            p.v_scale[i] = kind == QMV_KV_Q8 ? c[first + i].v_scale : nullptr;
        }
        if (launch_kv_keep(p, static_cast<int>(D), kind, reinterpret_cast<cudaStream_t>(stream), pdl) != cudaSuccess) {
            (void)cudaGetLastError();
            return QMV_ERR_LAUNCH;
        }
    }
    return QMV_OK;
}

int64_t qmv_tree_attn_workspace(void)
{
    int *status = nullptr;
    int sms = 0;
    bool pdl = false;
    if (call_env(&status, &sms, &pdl) != cudaSuccess) {
        (void)cudaGetLastError();
        return -1;
    }
    return tree_attn_workspace_bytes(sms);
}

qmv_status qmv_tree_attn(const void *q, int64_t q_stride, const void *k, const void *v, const float *k_scale,
                         const float *v_scale, int kind, int64_t n_pages, int64_t page, int64_t page_stride,
                         const int32_t *table, int64_t width, const int32_t *start, const int32_t *kv_len,
                         const int32_t *tree, int64_t tree_words, const float *scale, void *out, void *workspace,
                         int64_t workspace_bytes, int64_t R, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                         qmv_stream_t stream)
{
    const qmv_status st = check_cache(n_pages, Hkv, page, D, page_stride, kind);
    if (st != QMV_OK) return st;
    if (T < 0 || T > (1 << 24) || R < 0 || R > (1 << 20) || Hq < 1 || Hq > 65536 || Hq % Hkv != 0 || T * Hq > kInt32Max ||
        width < 0 || width > kInt32Max || q_stride < Hq * D || q_stride > (int64_t(1) << 31) || tree_words < 0 ||
        tree_words > 65536 || (tree && tree_words == 0) || (scale && !std::isfinite(*scale)))
        return QMV_ERR_SHAPE;
    if (T == 0 || R == 0) return QMV_OK;
    if (!q || !k || !v || !start || !kv_len || !out || (width > 0 && !table) ||
        (kind == QMV_KV_Q8 && (!k_scale || !v_scale)))
        return QMV_ERR_NULL;
    if (!aligned(q, 16) || q_stride % 8 != 0 || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) ||
        !aligned(table, 4) || !aligned(start, 4) || !aligned(kv_len, 4) || !aligned(tree, 4) ||
        !aligned(k_scale, 16) || !aligned(v_scale, 16) || !aligned(workspace, 16))
        return QMV_ERR_ALIGN;
    AttnParams p = {};
    int sms = 0;
    bool pdl = false;
    if (call_env(&p.status, &sms, &pdl) != cudaSuccess) return QMV_ERR_CUDA;
    const int64_t need = tree_attn_workspace_bytes(sms);
    if (workspace_bytes < need) return QMV_ERR_SHAPE;
    if (need > 0 && !workspace) return QMV_ERR_NULL;
    p.q = static_cast<const __half *>(q);
    p.k = k;
    p.v = v;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.table = table;
    p.start = start;
    p.kv_len = kv_len;
    p.tree = tree;
    p.out = static_cast<__half *>(out);
    p.workspace = workspace;
    p.q_stride = q_stride;
    p.page_stride = page_stride;
    p.R = R;
    p.T = T;
    p.width = width;
    p.n_pages = n_pages;
    p.Hq = static_cast<int>(Hq);
    p.Hkv = static_cast<int>(Hkv);
    p.group = static_cast<int>(Hq / Hkv);
    p.tree_words = static_cast<int>(tree_words);
    p.page_shift = page_shift_of(page);
    p.test_skip_copy = test_skip_this_launch() ? 1 : 0;
    p.scale_log2 = (scale ? *scale : 1.0f / std::sqrt(static_cast<float>(D))) * 1.4426950408889634f;
    if (launch_tree_attn(p, static_cast<int>(D), kind, sms, reinterpret_cast<cudaStream_t>(stream), pdl) !=
        cudaSuccess) {
        (void)cudaGetLastError();
        return QMV_ERR_LAUNCH;
    }
    return QMV_OK;
}

}  // extern "C"
