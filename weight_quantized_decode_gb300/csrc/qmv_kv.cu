// qmv_kv.cu -- the paged key/value cache: page and slot maps from request
// lengths, and the rotary write of new rows into the cache.
#include <cstdint>

#include "qmv_common.cuh"
#include "qmv_kv.h"
#include "qmv_launch.h"

namespace qmv {

namespace {

// ---- page and slot maps -------------------------------------------------------
//
//   start[r]  = sum over s < r of n[s]
//   have, need = ceil(len / page) or the pages it holds, if more; ceil((len + n) / page) per request
//   table[r][have .. need) = free[head + sum over s < r of (need - have) ..]
//   slot of request r's i-th new token = table[r][(len + i) / page] * page + (len + i) % page
//   pos  = len + i, or with a tree mask len + (nodes its row sees) - 1: its depth
//
// One launch.  Every CTA scans the request counts by itself (a chunk of 1024
// at a time: two loads and a block scan, all from L2), so that no CTA waits
// for another; it then writes the tokens of its own slice of the output, and
// the table rows of the chunks that fall to it.  A token finds its request by
// binary search in the chunk's offsets in shared memory and takes a fresh page
// from the free list itself, not from the table row another CTA may be writing.
// Bound by latency: 4.1 us for one tree of 8 nodes, 9.7 us for 1000 prompts of
// 1 to 509 tokens (255 thousand in all, 3.1 MB).
constexpr int kPagesThreads = 1024;
constexpr int kPagesTokens = 1024;   // tokens of a CTA, at the least

struct PagesChunk {
    int64_t start[kPagesThreads + 1];   // offset of each request's first token
    int64_t base[kPagesThreads + 1];    // offset of its first fresh page in the free list
    int32_t len[kPagesThreads];
    int32_t have[kPagesThreads];
};

// Inclusive scan over the block of two sums at once.
__device__ __forceinline__ void block_scan2(int64_t &a, int64_t &b, int64_t (*warp_sums)[2])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t ua = __shfl_up_sync(0xffffffffu, a, d), ub = __shfl_up_sync(0xffffffffu, b, d);
        if (lane >= d) {
            a += ua;
            b += ub;
        }
    }
    if (lane == 31) {
        warp_sums[warp][0] = a;
        warp_sums[warp][1] = b;
    }
    __syncthreads();
    if (warp == 0) {
        int64_t wa = warp_sums[lane][0], wb = warp_sums[lane][1];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t ua = __shfl_up_sync(0xffffffffu, wa, d), ub = __shfl_up_sync(0xffffffffu, wb, d);
            if (lane >= d) {
                wa += ua;
                wb += ub;
            }
        }
        warp_sums[lane][0] = wa;
        warp_sums[lane][1] = wb;
    }
    __syncthreads();
    if (warp > 0) {
        a += warp_sums[warp - 1][0];
        b += warp_sums[warp - 1][1];
    }
}

// The last i in [0, n) with off[i] <= t, for off ascending and off[0] <= t.
__device__ __forceinline__ int last_at_or_below(const int64_t *off, int n, int64_t t)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPagesThreads) kv_pages_kernel(const PagesParams p)
{
    __shared__ PagesChunk c;
    __shared__ int64_t warp_sums[32][2];
    pdl_allow_next_grid();
    pdl_wait_prior_grid();
    const int tid = threadIdx.x;
    const int page = 1 << p.page_shift;
    const int64_t head = p.head ? *p.head : 0;
    const int64_t t_lo = p.T * blockIdx.x / gridDim.x, t_hi = p.T * (blockIdx.x + 1) / gridDim.x;
    int64_t tokens = 0, pages = head;   // before this chunk
    int bad = head < 0 || head > p.n_free ? kDevNoPages : 0;
    for (int64_t r0 = 0; r0 < p.R; r0 += kPagesThreads) {
        const int n = static_cast<int>(p.R - r0 < kPagesThreads ? p.R - r0 : kPagesThreads);
        int64_t len = 0, fresh = 0, cnt = 0, hold = 0;
        if (tid < n) {
            len = p.len[r0 + tid];
            cnt = p.n_new[r0 + tid];
            if (len < 0 || cnt < 0 || len + cnt > 0x7fffffff) {
                bad |= kDevBadLength;
                len = len < 0 ? 0 : len;
                cnt = 0;
            }
            if (p.held) {
                hold = p.held[r0 + tid];
                if (hold < 0 || hold > p.width) {
                    bad |= kDevBadLength;
                    hold = hold < 0 ? 0 : p.width;
                }
            }
        }
        // Tokens past T are dropped: the counts are cut so that the offsets end at T.
        int64_t sum = cnt, none = 0;
        block_scan2(sum, none, warp_sums);
        int64_t first = tokens + sum - cnt;
        if (first > p.T) first = p.T;
        if (first + cnt > p.T) {
            bad |= kDevNoPages;
            cnt = p.T - first;
        }
        int64_t have = (len + page - 1) >> p.page_shift;
        if (have < hold) have = hold;
        int64_t need = (len + cnt + page - 1) >> p.page_shift;
        if (p.held && need > p.width) need = p.width;   // no page is taken that the row has no entry for
        if (tid < n && need > have) fresh = need - have;
        int64_t last = first + cnt, upto = fresh;
        __syncthreads();   // warp_sums again
        none = 0;
        block_scan2(upto, none, warp_sums);
        const int64_t base = pages + upto - fresh;
        if (tid < n) {
            c.start[tid] = first;
            c.base[tid] = base;
            c.len[tid] = static_cast<int32_t>(len);
            c.have[tid] = static_cast<int32_t>(have);
            if (tid == n - 1) {
                c.start[n] = last;
                c.base[n] = base + fresh;
            }
        }
        __syncthreads();
        if ((r0 / kPagesThreads) % gridDim.x == blockIdx.x) {
            if (tid < n) {
                p.start[r0 + tid] = static_cast<int32_t>(first);
                p.kv_len[r0 + tid] = static_cast<int32_t>(len + cnt);
                if (p.held_out) {   // with the fresh pages that the list had
                    const int64_t left = p.n_free - base, got = base < 0 || left < 0 ? 0 : (fresh < left ? fresh : left);
                    p.held_out[r0 + tid] = static_cast<int32_t>(have + got < p.width ? have + got : p.width);
                }
                if (r0 + tid == p.R - 1) {
                    p.start[p.R] = static_cast<int32_t>(last);
                    if (p.head_out)
                        *p.head_out = static_cast<int32_t>(base + fresh < p.n_free ? base + fresh : p.n_free);
                }
            }
            for (int64_t e = c.base[0] + tid; e < c.base[n]; e += kPagesThreads) {
                const int r = last_at_or_below(c.base, n, e);
                const int64_t j = c.have[r] + (e - c.base[r]);
                const int32_t id = e >= 0 && e < p.n_free ? p.free_pages[e] : -1;
                if (id < 0 || id >= p.n_pages) bad |= e >= 0 && e < p.n_free ? kDevBadPage : kDevNoPages;
                if (j < p.width)
                    p.table[(r0 + r) * p.width + j] = id;
                else
                    bad |= kDevNoPages;
            }
        }
        const int64_t lo = t_lo > c.start[0] ? t_lo : c.start[0], hi = t_hi < c.start[n] ? t_hi : c.start[n];
        for (int64_t t = lo + tid; t < hi; t += kPagesThreads) {
            const int r = last_at_or_below(c.start, n, t);
            const int64_t i = t - c.start[r], at = c.len[r] + i, j = at >> p.page_shift;
            int32_t id = -1;
            if (j < p.width) {
                if (j < c.have[r]) {
                    id = p.table[(r0 + r) * p.width + j];
                } else {
                    const int64_t e = c.base[r] + (j - c.have[r]);
                    if (e >= 0 && e < p.n_free) id = p.free_pages[e];
                }
            }
            const bool ok = id >= 0 && id < p.n_pages;
            if (!ok) bad |= j >= p.width ? kDevNoPages : (j < c.have[r] ? kDevBadPage : 0);
            p.slots[t] = ok ? static_cast<int32_t>((static_cast<int64_t>(id) << p.page_shift) | (at & (page - 1))) : -1;
            int64_t pos = at;
            if (p.tree) {
                const int64_t nodes = c.start[r + 1] - c.start[r];
                int depth = -1;
                for (int w = 0; w < p.tree_words && 32 * w < nodes; ++w) {
                    uint32_t m = static_cast<uint32_t>(p.tree[t * p.tree_words + w]);
                    if (nodes - 32 * w < 32) m &= (1u << (nodes - 32 * w)) - 1u;
                    depth += __popc(m);
                }
                pos = c.len[r] + (depth < 0 ? 0 : depth);
            }
            p.pos[t] = static_cast<int32_t>(pos);
            p.request[t] = static_cast<int32_t>(r0 + r);
        }
        tokens = c.start[n];
        pages = c.base[n];
        __syncthreads();   // the chunk's shared memory is rewritten
    }
    if (p.R == 0 && blockIdx.x == 0 && tid == 0) {
        if (p.start) p.start[0] = 0;
        if (p.head_out) *p.head_out = static_cast<int32_t>(head < p.n_free ? head : p.n_free);
    }
    // Output places past the last token: padding that the cache write skips.
    for (int64_t t = (t_lo > tokens ? t_lo : tokens) + tid; t < t_hi; t += kPagesThreads) {
        p.slots[t] = -1;
        p.pos[t] = 0;
        p.request[t] = -1;
    }
    if (bad) atomicOr(p.status, bad);
}

// ---- rotary write of new rows ---------------------------------------------------
//
// For each token: its query heads, rotated, as fp16 to q; its key heads,
// rotated, and its value heads to the cache row of its slot, as fp16 or as
// 8-bit codes with one fp32 scale d = max |y| / 127 to the row,
// code = round(y / d); a row that is not finite has a scale that is not, and codes of
// 0.  A rotation of pair (a, b) by the position's (cos, sin)
// is (a cos - b sin, b cos + a sin); products and sums are rounded one by one
// in fp32, so that a code does not depend on how a compiler fuses them.
//
// G = D / 4 lanes hold one head's row, four neighbouring values each, so a
// warp carries 32 / G rows; the partner of a half-split pair sits rot / 8
// lanes away.  A warp takes kAppendRows rows of one token and loads them all
// before it uses one.  Bound by the bytes: 16381 tokens of 32 heads on 8 of 128,
// fp32 in, fp16 out, 612 MB in 100 us, 6.1 TB/s, 0.90 of the measured copy
// bandwidth; one token 1.9 us.  8-bit rows, 580 MB, take 147 us: a reduction, a division
// and a reciprocal to a row, and a lane stores one word.
constexpr int kAppendThreads = 128;
constexpr int kAppendRows = 4;

template <int D, bool XF32, int KIND, bool INTER>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendParams p)
{
    constexpr int G = D / 4;
    constexpr int PER = 32 / G;   // rows a warp holds at a time
    pdl_allow_next_grid();
    pdl_wait_prior_grid();
    const int lane = threadIdx.x & 31;
    const int g = lane % G, sub = lane / G;
    const int heads = p.Hq + 2 * p.Hkv;
    const int per_token = (heads + kAppendRows * PER - 1) / (kAppendRows * PER);
    const int64_t units = p.T * per_token;
    const int page = 1 << p.page_shift;
    for (int64_t u = (static_cast<int64_t>(blockIdx.x) * kAppendThreads + threadIdx.x) >> 5; u < units;
         u += (static_cast<int64_t>(gridDim.x) * kAppendThreads) >> 5) {
        const int64_t t = u / per_token;
        const int h0 = static_cast<int>(u - t * per_token) * (kAppendRows * PER);
        const int slot = p.slots[t];
        float x[kAppendRows][4];
#pragma unroll
        for (int i = 0; i < kAppendRows; ++i) {
            const int h = h0 + i * PER + sub;
            if (h < heads) {
                const int64_t at = t * p.x_stride + static_cast<int64_t>(h) * D + 4 * g;
                if constexpr (XF32) {
                    const float4 f = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.x) + at);
                    x[i][0] = f.x; x[i][1] = f.y; x[i][2] = f.z; x[i][3] = f.w;
                } else {
                    const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const __half *>(p.x) + at);
                    x[i][0] = half_lo_to_float(w.x); x[i][1] = half_hi_to_float(w.x);
                    x[i][2] = half_lo_to_float(w.y); x[i][3] = half_hi_to_float(w.y);
                }
            } else {
                x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.0f;
            }
        }
        // This lane's share of the position's cosines and sines: INTER: its two
        // pairs (x[0], x[1]) and (x[2], x[3]); half split: its four values are
        // the first (partner rot / 2 further on) or the second half of pairs.
        float cs[4], sn[4];
        const bool turns = 4 * g < p.rot;
        const bool second = !INTER && 8 * g >= p.rot;
        bool pos_ok = true;
        if (p.rot > 0) {
            const int64_t pos = p.pos[t];
            pos_ok = pos >= 0 && pos < p.n_pos;
            if (turns && pos_ok) {
                const int64_t row = pos * (p.rot / 2);
                if constexpr (INTER) {
                    const float2 c2 = *reinterpret_cast<const float2 *>(p.cos_t + row + 2 * g);
                    const float2 s2 = *reinterpret_cast<const float2 *>(p.sin_t + row + 2 * g);
                    cs[0] = c2.x; cs[1] = c2.y;
                    sn[0] = s2.x; sn[1] = s2.y;
                } else {
                    const int64_t at = row + 4 * g - (second ? p.rot / 2 : 0);
                    const float4 c4 = *reinterpret_cast<const float4 *>(p.cos_t + at);
                    const float4 s4 = *reinterpret_cast<const float4 *>(p.sin_t + at);
                    cs[0] = c4.x; cs[1] = c4.y; cs[2] = c4.z; cs[3] = c4.w;
                    sn[0] = s4.x; sn[1] = s4.y; sn[2] = s4.z; sn[3] = s4.w;
                }
            }
        }
        const bool slot_ok = slot >= 0 && slot < p.n_slots;
        if (lane == 0 && ((!slot_ok && slot != -1) || !pos_ok))
            atomicOr(p.status, (!pos_ok ? kDevBadLength : 0) | (!slot_ok && slot != -1 ? kDevBadPage : 0));
        const int64_t cell = slot_ok ? slot >> p.page_shift : 0;
        const int row_in_page = slot & (page - 1);
#pragma unroll
        for (int i = 0; i < kAppendRows; ++i) {
            const int h = h0 + i * PER + sub;
            float y[4] = {x[i][0], x[i][1], x[i][2], x[i][3]};
            if (p.rot > 0) {
                float other[4];
                if constexpr (!INTER) {
                    // every lane takes part in the exchange; rows past `heads` exchange zeros
                    const int from = turns ? (second ? lane - p.rot / 8 : lane + p.rot / 8) : lane;
#pragma unroll
                    for (int j = 0; j < 4; ++j) other[j] = __shfl_sync(0xffffffffu, x[i][j], from);
                }
                if (h < p.Hq + p.Hkv && turns) {
                    if constexpr (INTER) {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const float a = x[i][2 * j], b = x[i][2 * j + 1];
                            y[2 * j] = __fsub_rn(__fmul_rn(a, cs[j]), __fmul_rn(b, sn[j]));
                            y[2 * j + 1] = __fadd_rn(__fmul_rn(b, cs[j]), __fmul_rn(a, sn[j]));
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float s = __fmul_rn(other[j], sn[j]);
                            y[j] = second ? __fadd_rn(__fmul_rn(x[i][j], cs[j]), s)
                                          : __fsub_rn(__fmul_rn(x[i][j], cs[j]), s);
                        }
                    }
                }
                if (!pos_ok && h < p.Hq + p.Hkv) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) y[j] = __int_as_float(0x7fffffff);   // no such position: NaN
                }
            }
            const uint2 packed = make_uint2(float2_to_half2_bits(make_float2(y[0], y[1])),
                                            float2_to_half2_bits(make_float2(y[2], y[3])));
            if (h < p.Hq) {
                *reinterpret_cast<uint2 *>(p.q + (t * p.Hq + h) * D + 4 * g) = packed;
            }
            const bool is_v = h >= p.Hq + p.Hkv;
            const int kvh = h - p.Hq - (is_v ? p.Hkv : 0);
            const int64_t in_page = (static_cast<int64_t>(kvh) << p.page_shift) + row_in_page;
            const bool writes = h >= p.Hq && h < heads && slot_ok && pos_ok;
            if constexpr (KIND == kKvF16) {
                if (writes)
                    *reinterpret_cast<uint2 *>(static_cast<__half *>(is_v ? p.v : p.k) + cell * p.page_stride +
                                               in_page * D + 4 * g) = packed;
            } else {
                // largest magnitude, by its bits: NaN counts as larger than any number
                uint32_t most = 0u;
#pragma unroll
                for (int j = 0; j < 4; ++j) most = max(most, __float_as_uint(y[j]) & 0x7fffffffu);
#pragma unroll
                for (int d = 1; d < G; d <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
                const float d = __fdiv_rn(__uint_as_float(most), 127.0f);
                // (a row whose largest value is below 2^-119 is stored as zeros: 1 / d would overflow)
                const float id = d >= 1.17549435e-38f ? __frcp_rn(d) : 0.0f;
                uint32_t word = 0u;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float code = __fmul_rn(y[j], id);
                    // nearest, ties away from zero, as trunc(code +- 1/2) has it
                    const int c = static_cast<int>(truncf(__fadd_rn(code, copysignf(0.5f, code))));
                    word |= (static_cast<uint32_t>(c) & 0xffu) << (8 * j);
                }
                if (writes) {
                    *reinterpret_cast<uint32_t *>(static_cast<int8_t *>(is_v ? p.v : p.k) + cell * p.page_stride +
                                                  in_page * D + 4 * g) = word;
                    if (g == 0)
                        (is_v ? p.v_scale : p.k_scale)[((cell * p.Hkv) << p.page_shift) + in_page] = d;
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_kv_pages(const PagesParams &p, int sms, cudaStream_t s, bool pdl)
{
    int64_t grid = (p.T + kPagesTokens - 1) / kPagesTokens;
    if (grid > sms) grid = sms;
    if (grid < 1) grid = 1;
    return launch_ex(kv_pages_kernel, dim3(static_cast<unsigned>(grid)), dim3(kPagesThreads), 0, s, pdl, p);
}

namespace {

template <int D, bool XF32, int KIND>
cudaError_t append_with(const AppendParams &p, bool interleaved, dim3 grid, cudaStream_t s, bool pdl)
{
    if (interleaved)
        return launch_ex(kv_append_kernel<D, XF32, KIND, true>, grid, dim3(kAppendThreads), 0, s, pdl, p);
    return launch_ex(kv_append_kernel<D, XF32, KIND, false>, grid, dim3(kAppendThreads), 0, s, pdl, p);
}

}  // namespace

cudaError_t launch_kv_append(const AppendParams &p, int D, bool x_f32, int kind, bool interleaved, int sms,
                             cudaStream_t s, bool pdl)
{
    const int rows = kAppendRows * (32 / (D / 4));
    const int64_t units = p.T * ((p.Hq + 2 * p.Hkv + rows - 1) / rows);
    int64_t g = (units + kAppendThreads / 32 - 1) / (kAppendThreads / 32);
    if (g > 16LL * sms) g = 16LL * sms;   // 2048 threads to an SM
    const dim3 grid(static_cast<unsigned>(g));
    if (D == 64) {
        if (x_f32)
            return kind == kKvF16 ? append_with<64, true, kKvF16>(p, interleaved, grid, s, pdl)
                                  : append_with<64, true, kKvQ8>(p, interleaved, grid, s, pdl);
        return kind == kKvF16 ? append_with<64, false, kKvF16>(p, interleaved, grid, s, pdl)
                              : append_with<64, false, kKvQ8>(p, interleaved, grid, s, pdl);
    }
    if (x_f32)
        return kind == kKvF16 ? append_with<128, true, kKvF16>(p, interleaved, grid, s, pdl)
                              : append_with<128, true, kKvQ8>(p, interleaved, grid, s, pdl);
    return kind == kKvF16 ? append_with<128, false, kKvF16>(p, interleaved, grid, s, pdl)
                          : append_with<128, false, kKvQ8>(p, interleaved, grid, s, pdl);
}

}  // namespace qmv
