// qmv_kv_norm.cu -- the cache write with norms of queries and keys and with
// positions of several axes: qmv_kv_append_norm.
#include <cstdint>

#include "qmv_common.cuh"
#include "qmv_kv.h"
#include "qmv_launch.h"

namespace qmv {

namespace {

// For each head's row x of D values (queries with q_norm, keys with k_norm):
//
//   n_i = x_i / sqrt(mean x^2 + eps) * w_i
//   pair i of n is turned by (cos, sin)[pos[axis(i)][t]][i]
//
// then rounded to fp16 (queries; an fp16 cache) or to 8-bit codes with one scale
// to the row, as the plain cache write does it.  All in fp32; every product and
// sum is rounded by itself, so that a code does not depend on what a compiler fuses.
//
// D / 8 lanes hold one row, lane l its chunks l and l + D/8 of four values each.  So a
// warp instruction loads whole 128-byte lines, and where all D values are turned the two
// values of a half-split pair lie in one lane; fewer turned ones exchange them by shuffles.
//
// Bound by the bytes in fp32: 16381 tokens of 32 heads on 8 of 128 with norms and three
// axes, fp16 cache, 613 MB in 100 us, 6.1 TB/s, 0.90 of the measured copy bandwidth.  fp16
// rows in: 88 us for 60 of bytes; an 8-bit cache: 111 for 85.  There some 180 and 220 instructions to
// two rows (fp16: 71 million, 61 us if every issue slot were used) stand beside fewer bytes, and fp16
// rows have half the bytes under way that fp32 rows have.  4099 tokens of 28 heads on 4, fp16,
// 16.8 us; one token 2.9.
// Measured and not taken: rows through rings of asynchronous copies (107 to 145 us), 16
// values to a lane (200), the norms' weights kept in registers (108 to 116).
constexpr int kThreads = 128;
constexpr int kGroups = 3;   // row groups of a warp that are loaded before one is used
constexpr int kBlocks = 7;   // blocks to an SM

enum Turn { kAllHalves = 0, kHalves = 1, kNeighbours = 2 };

struct Axes {
    int pos[4];

    __device__ __forceinline__ int at(int axis) const
    {
        const int lo = axis & 1 ? pos[1] : pos[0], hi = axis & 1 ? pos[3] : pos[2];
        return axis & 2 ? hi : lo;
    }
};

// N neighbouring values f .. of `table`, each from the row of its own axis (two bits to a frequency in `code`).
template <int N>
__device__ __forceinline__ void load_turns(float *to, const float *table, int f, uint32_t code, const Axes &ax, int half)
{
    constexpr uint32_t kAll = N == 4 ? 0x55u : 0x5u;
    const int first = code & 3;
    if (code == first * kAll) {
        const float *from = table + static_cast<int64_t>(ax.at(first)) * half + f;
        if constexpr (N == 4) {
            const float4 v = *reinterpret_cast<const float4 *>(from);
            to[0] = v.x; to[1] = v.y; to[2] = v.z; to[3] = v.w;
        } else {
            const float2 v = *reinterpret_cast<const float2 *>(from);
            to[0] = v.x; to[1] = v.y;
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) to[j] = table[static_cast<int64_t>(ax.at((code >> (2 * j)) & 3)) * half + f + j];
    }
}

// Sums over the lanes of a row.
template <int LPR>
__device__ __forceinline__ float row_sum(float x)
{
#pragma unroll
    for (int d = 1; d < LPR; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

template <int D, bool XF32, int KIND, int TURN>
__global__ void __launch_bounds__(kThreads, kBlocks) kv_append_norm_kernel(const __grid_constant__ NormAppendParams p)
{
    constexpr int LPR = D / 8;     // lanes to a row
    constexpr int PER = 32 / LPR;  // rows of a group
    pdl_allow_next_grid();
    pdl_wait_prior_grid();
    const int lane = threadIdx.x & 31;
    const int l = lane % LPR, sub = lane / LPR;
    const int heads = p.a.Hq + 2 * p.a.Hkv, groups = (heads + PER - 1) / PER;
    const int page = 1 << p.a.page_shift;
    const int half = p.a.rot / 2, h = p.a.rot / 8;   // values, and chunks, from one of a half-split pair to the other
    // Chunk i's frequencies: the first one (-1: not turned) and the axes of them.
    constexpr int NT = TURN == kNeighbours ? 2 : 4;   // frequencies of a chunk
    constexpr int SETS = TURN == kAllHalves ? 1 : 2;  // chunks of a lane with frequencies of their own
    int freq[SETS];
    uint32_t code[SETS];
#pragma unroll
    for (int i = 0; i < SETS; ++i) {
        const int c = l + i * LPR;
        if constexpr (TURN == kNeighbours)
            freq[i] = c < 2 * h ? 2 * c : -1;
        else
            freq[i] = c < h ? 4 * c : c < 2 * h ? 4 * (c - h) : -1;
        code[i] = freq[i] < 0 ? 0u : (p.axis_bits[freq[i] >> 4] >> (2 * (freq[i] & 15))) & (NT == 4 ? 0xffu : 0xfu);
    }
    const int64_t units = p.a.T * p.units;
    for (int64_t u = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5; u < units;
         u += (static_cast<int64_t>(gridDim.x) * kThreads) >> 5) {
        const int64_t t = p.units == 1 ? u : u / p.units;
        const int part = p.units == 1 ? 0 : static_cast<int>(u - t * p.units);
        const int g_lo = groups * part / p.units, g_hi = groups * (part + 1) / p.units;
        const int slot = p.a.slots[t];
        Axes ax = {};
        bool pos_ok = true;
        if (p.a.rot > 0) {
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                if (a < p.axes) {
                    ax.pos[a] = p.a.pos[a * p.pos_stride + t];
                    pos_ok = pos_ok && ax.pos[a] >= 0 && ax.pos[a] < p.a.n_pos;
                }
            }
        }
        const bool slot_ok = slot >= 0 && slot < p.a.n_slots;
        if (lane == 0 && ((!slot_ok && slot != -1) || !pos_ok))
            atomicOr(p.a.status, (!pos_ok ? kDevBadLength : 0) | (!slot_ok && slot != -1 ? kDevBadPage : 0));
        const bool writes = slot_ok && pos_ok;
        const int64_t cell = slot_ok ? slot >> p.a.page_shift : 0;
        const int row_in_page = slot & (page - 1);
        float cs[SETS][NT], sn[SETS][NT];
        for (int g0 = g_lo; g0 < g_hi; g0 += kGroups) {
            float x[kGroups][8];
#pragma unroll
            for (int k = 0; k < kGroups; ++k) {
                const int head = (g0 + k) * PER + sub;
                const bool there = g0 + k < g_hi && head < heads;
                const int64_t at = t * p.a.x_stride + head * D + 4 * l;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if constexpr (XF32) {
                        float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        if (there) f = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.a.x) + at + 4 * LPR * i);
                        x[k][4 * i] = f.x; x[k][4 * i + 1] = f.y; x[k][4 * i + 2] = f.z; x[k][4 * i + 3] = f.w;
                    } else {
                        uint2 w = make_uint2(0u, 0u);
                        if (there) w = *reinterpret_cast<const uint2 *>(static_cast<const __half *>(p.a.x) + at + 4 * LPR * i);
                        x[k][4 * i] = half_lo_to_float(w.x); x[k][4 * i + 1] = half_hi_to_float(w.x);
                        x[k][4 * i + 2] = half_lo_to_float(w.y); x[k][4 * i + 3] = half_hi_to_float(w.y);
                    }
                }
            }
            if (g0 == g_lo) {
#pragma unroll
                for (int i = 0; i < SETS; ++i) {
                    if (freq[i] >= 0 && pos_ok) {
                        load_turns<NT>(cs[i], p.a.cos_t, freq[i], code[i], ax, half);
                        load_turns<NT>(sn[i], p.a.sin_t, freq[i], code[i], ax, half);
                    } else {
#pragma unroll
                        for (int j = 0; j < NT; ++j) cs[i][j] = sn[i][j] = 0.0f;
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < kGroups; ++k) {
                const int head = (g0 + k) * PER + sub;
                const bool there = g0 + k < g_hi && head < heads;
                const bool is_q = head < p.a.Hq, turned = head < p.a.Hq + p.a.Hkv;
                float(&y)[8] = x[k];
                if (p.q_norm || p.k_norm) {
                    float ss = 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) ss = fmaf(y[i], y[i], ss);
                    ss = row_sum<LPR>(ss);
                    const float *w = is_q ? p.q_norm : p.k_norm;
                    const bool normed = there && turned && w;
                    float eps = p.eps;
                    if constexpr (XF32) {
                        // Squares that leave fp32's range: the row is taken times 2^-70, which is exact but for
                        // values that the sum does not see.
                        const bool wide = normed && !(ss < 1e38f);
                        if (__any_sync(0xffffffffu, wide)) {
                            float big = 0.0f;
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float z = y[i] * 0x1p-70f;
                                big = fmaf(z, z, big);
                                if (wide) y[i] = z;
                            }
                            big = row_sum<LPR>(big);
                            if (wide) {
                                ss = big;
                                eps = eps * 0x1p-100f * 0x1p-40f;
                            }
                        }
                    }
                    if (normed) {
                        const float r = rsqrtf(__fadd_rn(ss * (1.0f / D), eps));
                        w += (is_q ? head * p.q_norm_stride : (head - p.a.Hq) * p.k_norm_stride) + 4 * l;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float4 f = *reinterpret_cast<const float4 *>(w + 4 * LPR * i);
                            y[4 * i] = __fmul_rn(__fmul_rn(y[4 * i], r), f.x);
                            y[4 * i + 1] = __fmul_rn(__fmul_rn(y[4 * i + 1], r), f.y);
                            y[4 * i + 2] = __fmul_rn(__fmul_rn(y[4 * i + 2], r), f.z);
                            y[4 * i + 3] = __fmul_rn(__fmul_rn(y[4 * i + 3], r), f.w);
                        }
                    }
                }
                if constexpr (TURN == kAllHalves) {
                    if (turned) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float a = y[j], b = y[4 + j];
                            y[j] = __fsub_rn(__fmul_rn(a, cs[0][j]), __fmul_rn(b, sn[0][j]));
                            y[4 + j] = __fadd_rn(__fmul_rn(b, cs[0][j]), __fmul_rn(a, sn[0][j]));
                        }
                    }
                } else if constexpr (TURN == kNeighbours) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (turned && freq[i] >= 0) {
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const float a = y[4 * i + 2 * j], b = y[4 * i + 2 * j + 1];
                                y[4 * i + 2 * j] = __fsub_rn(__fmul_rn(a, cs[i][j]), __fmul_rn(b, sn[i][j]));
                                y[4 * i + 2 * j + 1] = __fadd_rn(__fmul_rn(b, cs[i][j]), __fmul_rn(a, sn[i][j]));
                            }
                        }
                    }
                } else {
                    // h < LPR chunks from one of a pair to the other: chunk l (i = 0) has its partner in chunk l + h, which
                    // may be a second one (lane l + h - LPR), or l - h; chunk l + LPR (i = 1) in chunk l + LPR - h, a first one.
                    // Every lane takes part in each exchange.
                    const int row = sub * LPR;
                    const bool second0 = l >= h, over = l < h && l + h >= LPR;
                    const int from0 = row + (second0 ? (l < 2 * h ? l - h : l) : (l + h) % LPR);
                    const int from1 = row + (l + LPR < 2 * h ? l + LPR - h : l);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float a0 = y[j], a1 = y[4 + j];
                        float b0 = __shfl_sync(0xffffffffu, a0, from0), b1 = 0.0f;
                        if (2 * h > LPR) {
                            const float o = __shfl_sync(0xffffffffu, a1, from0);
                            if (over) b0 = o;
                            b1 = __shfl_sync(0xffffffffu, a0, from1);
                        }
                        if (turned && freq[0] >= 0) {
                            const float c = __fmul_rn(a0, cs[0][j]), s = __fmul_rn(b0, sn[0][j]);
                            y[j] = second0 ? __fadd_rn(c, s) : __fsub_rn(c, s);
                        }
                        if (turned && freq[1] >= 0) y[4 + j] = __fadd_rn(__fmul_rn(a1, cs[1][j]), __fmul_rn(b1, sn[1][j]));
                    }
                }
                if (!pos_ok && turned) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = __int_as_float(0x7fffffff);   // no such position: NaN
                }
                const bool is_v = !turned;
                const int in_page = ((head - p.a.Hq - (is_v ? p.a.Hkv : 0)) << p.a.page_shift) + row_in_page;
                if (KIND == kKvF16 || is_q) {
                    __half *to = is_q ? p.a.q + (t * p.a.Hq + head) * D
                                      : static_cast<__half *>(is_v ? p.a.v : p.a.k) + cell * p.a.page_stride + in_page * D;
                    if (there && (is_q || writes)) {
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            *reinterpret_cast<uint2 *>(to + 4 * l + 4 * LPR * i) =
                                make_uint2(float2_to_half2_bits(make_float2(y[4 * i], y[4 * i + 1])),
                                           float2_to_half2_bits(make_float2(y[4 * i + 2], y[4 * i + 3])));
                    }
                }
                if constexpr (KIND == kKvQ8) {
                    // largest magnitude, by its bits: NaN counts as larger than any number
                    uint32_t most = 0u;
#pragma unroll
                    for (int i = 0; i < 8; ++i) most = max(most, __float_as_uint(y[i]) & 0x7fffffffu);
#pragma unroll
                    for (int d = 1; d < LPR; d <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
                    if (there && !is_q && writes) {
                        const float d = __fdiv_rn(__uint_as_float(most), 127.0f);
                        // (a row whose largest value is below 2^-119 is stored as zeros: 1 / d would overflow)
                        const float id = d >= 1.17549435e-38f ? __frcp_rn(d) : 0.0f;
                        int8_t *to = static_cast<int8_t *>(is_v ? p.a.v : p.a.k) + cell * p.a.page_stride + in_page * D;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t word = 0u;
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float v = __fmul_rn(y[4 * i + j], id);
                                // nearest, ties away from zero, as trunc(v +- 1/2) has it
                                const int c = static_cast<int>(truncf(__fadd_rn(v, copysignf(0.5f, v))));
                                word |= (static_cast<uint32_t>(c) & 0xffu) << (8 * j);
                            }
                            *reinterpret_cast<uint32_t *>(to + 4 * l + 4 * LPR * i) = word;
                        }
                        if (l == 0)
                            (is_v ? p.a.v_scale : p.a.k_scale)[((cell * p.a.Hkv) << p.a.page_shift) + in_page] = d;
                    }
                }
            }
        }
    }
}

template <int D, bool XF32, int KIND>
cudaError_t append_with(const NormAppendParams &p, bool interleaved, dim3 grid, cudaStream_t s, bool pdl)
{
    if (interleaved || p.a.rot == 0)
        return launch_ex(kv_append_norm_kernel<D, XF32, KIND, kNeighbours>, grid, dim3(kThreads), 0, s, pdl, p);
    if (p.a.rot == D)
        return launch_ex(kv_append_norm_kernel<D, XF32, KIND, kAllHalves>, grid, dim3(kThreads), 0, s, pdl, p);
    return launch_ex(kv_append_norm_kernel<D, XF32, KIND, kHalves>, grid, dim3(kThreads), 0, s, pdl, p);
}

}  // namespace

cudaError_t launch_kv_append_norm(NormAppendParams p, int D, bool x_f32, int kind, bool interleaved, int sms,
                                  cudaStream_t s, bool pdl)
{
    const int per = 32 / (D / 8);
    const int groups = (p.a.Hq + 2 * p.a.Hkv + per - 1) / per;
    // Few tokens: their rows go to all the warps that the GPU holds.  Many: a warp takes whole tokens, so that it fetches a
    // token's cosines once (16381 tokens, three axes: 153 us with 4 rows to a unit, 104 with 48).  The warps that run at
    // once (4256 on 152 SMs) take a token each, and a few tokens more begin another wave: 48 heads, fp32 in, three axes,
    // 2128 tokens 17 us, 2129 (a warp to each) 23, 4256 29, 4257 39, 8192 53, for 12, 12, 23, 23 and 45 of bytes.
    const int64_t share = kThreads / 32 * kBlocks * sms / p.a.T;
    p.units = static_cast<int>(share < 1 ? 1 : share > groups ? groups : share);
    int64_t g = (p.a.T * p.units + kThreads / 32 - 1) / (kThreads / 32);
    if (g > 16LL * sms) g = 16LL * sms;
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
