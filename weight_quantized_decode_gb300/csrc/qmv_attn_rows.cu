// qmv_attn_rows.cu -- attention over the paged cache for few query rows to a
// key/value head (up to 16 in a tile): one pass over the cached rows, bound by
// their bytes.
//
// Four warps to a CTA, two CTAs to an SM.  A block of 128 places is 32 to each
// warp; a warp keeps 16 rows' running maximum, sum and output in registers and
// streams its own places through its own ring of shared-memory slots (tensor
// copies, one mbarrier to a slot, refilled by the warp as it empties them), so
// that warps wait for each other only at the end of a segment.  There the four
// outputs are brought to a common maximum and added in shared memory.
//   s = q k^T and o += p v are m16n8k16 products with fp32 accumulators: at 16
// rows they take a third of the time that the bytes take, and rows that a tile
// lacks cost nothing else.  p = 2^(s - max + 10): the factor 2^10 keeps small
// weights out of fp16's subnormals, and cancels against the sum.
//   8-bit rows: codes become exact fp16 integers in registers.  The key scale
// multiplies the score, the value scale the weight, both in fp32; weights are
// held below fp16's largest value by a running power of two of the largest
// value scale, handled like the running maximum.
#include <cstdint>

#include "qmv_attn.cuh"
#include "qmv_launch.h"

namespace qmv {

namespace {

constexpr int kRows = 16;
constexpr int kBlock = 128;
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStep = 32;           // places of a warp's step
constexpr float kShift = 10.0f;     // weights are 2^10 times exp(s - max)

template <int D, int KIND>
struct Ring {
    static constexpr int kRowBytes = KIND == kKvF16 ? 2 * D : D;
    static constexpr int kBoxBytes = kRowBytes < 128 ? kRowBytes : 128;   // inner extent of a copy
    static constexpr int kHalves = kRowBytes / kBoxBytes;
    static constexpr int kDataBytes = kStep * kRowBytes;
    static constexpr int kScaleBytes = KIND == kKvQ8 ? kStep * 4 : 0;
    static constexpr int kSlots = kDataBytes >= 8192 ? 3 : (kDataBytes >= 4096 ? 6 : 10);   // 24 KB to a warp or so
    // data slots of all warps, scale slots of all warps, P scratch (fp16 rows with non-finite values), barriers
    static constexpr int kDataAll = kWarps * kSlots * kDataBytes;
    static constexpr int kScaleAll = kWarps * kSlots * kScaleBytes;
    static constexpr int kPBytes = KIND == kKvF16 ? kWarps * kRows * 33 * 4 : 0;
    static constexpr int kOut = kWarps * kRows * (D + 8) * 4;             // joins the warps' outputs over the rings
    static constexpr int kBytes = (kDataAll > kOut ? kDataAll : kOut) + kScaleAll + kPBytes;
    static constexpr size_t kSmem = 1024 + kBytes;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four int8 codes of a word as fp16 integers: bytes (i, j) of the four.
__device__ __forceinline__ uint32_t codes_to_half2(uint32_t flipped, uint32_t sel)
{
    // a byte b ^ 0x80 under the exponent byte 0x64 is 1024 + 128 + code, exactly
    const __half2 h = __hsub2(as_h2(__byte_perm(flipped, 0x64646464u, sel)), as_h2(0x64806480u));
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ float quad_max(float v)
{
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}

__device__ __forceinline__ float quad_sum(float v)
{
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

__device__ __forceinline__ uint32_t h2_bits(float a, float b) { return float2_to_half2_bits(make_float2(a, b)); }

template <int D, int KIND>
__global__ void __launch_bounds__(kThreads, 2)
    tree_attn_rows_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                          const AttnParams p)
{
    using R = Ring<D, KIND>;
    constexpr int KS = D / 16;    // 16-wide steps of a score product
    constexpr int NT = D / 8;     // 8-wide tiles of the output
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ Share sh;
    __shared__ uint64_t bars[kWarps][R::kSlots];
    __shared__ float ml[2][kWarps][kRows];
    __shared__ int last_flag;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t4 = lane & 3;
    uint8_t *ring = smem + warp * R::kSlots * R::kDataBytes;
    constexpr int kFirst = R::kDataAll > R::kOut ? R::kDataAll : R::kOut;
    float *scales = reinterpret_cast<float *>(smem + kFirst) + warp * R::kSlots * kStep;
    float *pscr = reinterpret_cast<float *>(smem + kFirst + R::kScaleAll) + warp * kRows * 33;
    float *oscr = reinterpret_cast<float *>(smem);
    uint64_t *bar = bars[warp];

    if (lane == 0) {
        for (int i = 0; i < R::kSlots; ++i) mbar_init(&bar[i], 1);
        mbar_init_fence();
    }
    pdl_allow_next_grid();
    pdl_wait_prior_grid();
    find_share<kRows, kBlock, false, kThreads>(p, &sh);

    SegmentWalk<kRows, kBlock, false> walk;
    walk.begin(p, sh);
    Segment seg;
    uint32_t entry = 0;       // ring entries consumed so far, this warp's
    uint32_t asked = 0;       // entries requested so far
    bool gave_up = false;     // a wait ran out: nothing more is requested, outputs become NaN
    while (walk.next(p, seg)) {
        const int64_t len = seg.w.len;
        const int nodes = seg.w.nodes;
        const int64_t first_place = seg.b0 * kBlock + warp * kStep;
        // this warp's steps: places first_place + 128 s, those that begin before len
        int64_t steps64 = len > first_place ? (len - first_place + kBlock - 1) / kBlock : 0;
        if (steps64 > seg.nb) steps64 = seg.nb;
        const int steps = static_cast<int>(steps64);
        bool bad = seg.w.bad;

        // Page ids ahead of their use: lane l holds chunk l of a group of 32
        // (a step is one chunk, or two of 16-place pages).
        const int page = 1 << p.page_shift;
        const int cps = page < kStep ? 2 : 1;       // chunks of a step
        const int box_rows = page < kStep ? page : kStep;
        const int32_t *trow = p.table + seg.r * p.width;
        const int64_t n_pages_used = (len + page - 1) >> p.page_shift;
        auto load_ids = [&](int group) -> int {
            const int c = group * 32 + lane;
            const int s = c / cps;
            const int64_t idx = (first_place + static_cast<int64_t>(s) * kBlock + (c - s * cps) * box_rows) >> p.page_shift;
            if (s >= steps || idx >= n_pages_used) return -1;
            const int id = trow[idx];
            if (id < 0 || id >= p.n_pages) {
                bad = true;
                return 0;
            }
            return id;
        };
        int ids = load_ids(0), ids_next = load_ids(1), group = 0;
        // Requests entry e of this segment (even: keys of step e / 2; odd: values).
        auto request = [&](int e) {
            const int s = e >> 1;
            const int c0 = s * cps;
            if ((c0 >> 5) != group) {
                ids = ids_next;
                group = c0 >> 5;
                ids_next = load_ids(group + 1);
            }
            if (gave_up) return;
            asked = entry + static_cast<uint32_t>(e) + 1u;
            const int id0 = __shfl_sync(0xffffffffu, ids, c0 & 31), id1 = __shfl_sync(0xffffffffu, ids, (c0 + cps - 1) & 31);
            if (lane == 0) {
                const uint32_t slot = (entry + static_cast<uint32_t>(e)) % R::kSlots;
                const CUtensorMap *map = (e & 1) ? &vmap : &kmap;
                const int chunks = cps == 2 && id1 >= 0 ? 2 : 1;
                uint8_t *dst = ring + slot * R::kDataBytes;
                mbar_arrive_expect_tx(&bar[slot], chunks * box_rows * (R::kRowBytes + (KIND == kKvQ8 ? 4 : 0)));
                const int64_t j0 = first_place + static_cast<int64_t>(s) * kBlock;
                for (int c = 0; c < chunks; ++c) {
                    const int id = c ? id1 : id0;
                    const int y = (seg.kvh << p.page_shift) + (static_cast<int>(j0 & (page - 1)) & ~(box_rows - 1));
#pragma unroll
                    for (int h = 0; h < R::kHalves; ++h)
                        copy_box(dst + h * kStep * R::kBoxBytes + c * box_rows * R::kBoxBytes, map, h * 64, y, id, &bar[slot]);
                    if constexpr (KIND == kKvQ8) {
                        const float *src = ((e & 1) ? p.v_scale : p.k_scale) +
                                           ((static_cast<int64_t>(id) * p.Hkv) << p.page_shift) + y;
                        bulk_g2s(scales + slot * kStep + c * box_rows, src, box_rows * 4, &bar[slot]);
                    }
                }
            }
        };
        const int entries = 2 * steps;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the last segment's reads and writes of the ring
        for (int e = 0; e < R::kSlots && e < entries; ++e) request(e);

        // Rows g and g + 8 of the tile: their queries as product operands.
        const int64_t row_base = static_cast<int64_t>(seg.tile) * kRows;
        const int64_t all_rows = static_cast<int64_t>(nodes) * p.group;
        const int valid = static_cast<int>(all_rows - row_base < kRows ? all_rows - row_base : kRows);
        const int64_t first_token = p.start[seg.r];
        uint32_t qf[KS][4];
        {
            const __half *q0 = nullptr, *q1 = nullptr;
            if (g < valid && !seg.w.bad) {
                const int64_t i = (row_base + g) / p.group;
                q0 = p.q + (first_token + i) * p.q_stride + (seg.kvh * p.group + (row_base + g - i * p.group)) * D;
            }
            if (g + 8 < valid && !seg.w.bad) {
                const int64_t i = (row_base + g + 8) / p.group;
                q1 = p.q + (first_token + i) * p.q_stride + (seg.kvh * p.group + (row_base + g + 8 - i * p.group)) * D;
            }
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                if constexpr (KIND == kKvF16) {
                    // columns 16 s + 2 t4 and + 8
                    qf[s][0] = q0 ? *reinterpret_cast<const uint32_t *>(q0 + 16 * s + 2 * t4) : 0u;
                    qf[s][1] = q1 ? *reinterpret_cast<const uint32_t *>(q1 + 16 * s + 2 * t4) : 0u;
                    qf[s][2] = q0 ? *reinterpret_cast<const uint32_t *>(q0 + 16 * s + 8 + 2 * t4) : 0u;
                    qf[s][3] = q1 ? *reinterpret_cast<const uint32_t *>(q1 + 16 * s + 8 + 2 * t4) : 0u;
                } else {
                    // a lane's four codes are columns 16 s + 4 t4 ..: the same order of columns on both sides
                    const uint2 a = q0 ? *reinterpret_cast<const uint2 *>(q0 + 16 * s + 4 * t4) : make_uint2(0u, 0u);
                    const uint2 b = q1 ? *reinterpret_cast<const uint2 *>(q1 + 16 * s + 4 * t4) : make_uint2(0u, 0u);
                    qf[s][0] = a.x; qf[s][1] = b.x; qf[s][2] = a.y; qf[s][3] = b.y;
                }
            }
        }
        float o[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
        int ve = -126;        // 8-bit: 2^ve is at least the largest value scale so far

        auto wait_entry = [&](int e) {
            const uint32_t n = entry + static_cast<uint32_t>(e);
            if (!gave_up && !mbar_wait_warp(&bar[n % R::kSlots], (n / R::kSlots) & 1u, p.status)) gave_up = true;
            return smem_u32(ring) + (n % R::kSlots) * R::kDataBytes;
        };
        // Address of 16-byte chunk c of row r in a slot.
        auto at = [&](uint32_t base, int r, int c) -> uint32_t {
            if constexpr (R::kBoxBytes == 128)
                return base + (c >> 3) * (kStep * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
            else
                return base + r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
        };
        for (int s = 0; s < steps; ++s) {
            const int64_t j0 = first_place + static_cast<int64_t>(s) * kBlock;
            const bool masked = j0 + kStep > len - nodes;
            // ---- scores of 16 rows x 32 places ----
            const uint32_t kb = wait_entry(2 * s);
            float sc[4][4];
#pragma unroll
            for (int n = 0; n < 4; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.0f;
            if constexpr (KIND == kKvF16) {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int np = 0; np < 2; ++np) {
                        uint32_t b[4];   // places 16 np .. + 7 (columns 0-7, 8-15), + 8 .. + 15
                        ldsm4(b, at(kb, 16 * np + (lane & 7) + ((lane >> 4) << 3), 2 * ks + ((lane >> 3) & 1)));
                        mma16816(sc[2 * np], qf[ks], b[0], b[1]);
                        mma16816(sc[2 * np + 1], qf[ks], b[2], b[3]);
                    }
            } else {
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int kq = 0; kq < KS / 4; ++kq) {
                        uint32_t b[4];   // 16-column chunks 4 kq .. + 3 of places 8 n .. + 7
                        ldsm4(b, at(kb, 8 * n + (lane & 7), 4 * kq + (lane >> 3)));
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t f = b[i] ^ 0x80808080u;
                            mma16816(sc[n], qf[4 * kq + i], codes_to_half2(f, 0x4140u), codes_to_half2(f, 0x4342u));
                        }
                    }
            }
            float kd[4][2], vd[4][2];
            if constexpr (KIND == kKvQ8) {
                const float *ksl = scales + ((entry + 2u * s) % R::kSlots) * kStep;
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const float2 d = *reinterpret_cast<const float2 *>(ksl + 8 * n + 2 * t4);
                    kd[n][0] = d.x * p.scale_log2;
                    kd[n][1] = d.y * p.scale_log2;
                }
            }
            // ---- the keys' slot is free: request what comes kSlots entries later ----
            __syncwarp();
            if (2 * s + R::kSlots < entries) {
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                request(2 * s + R::kSlots);
            }
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[n][i] *= KIND == kKvQ8 ? kd[n][i & 1] : p.scale_log2;
            uint32_t see0 = 0xffffffffu, see1 = 0xffffffffu;
            if (masked) {
                uint32_t mine = 0u;
                if (lane < valid) {
                    const int node = static_cast<int>((row_base + lane) / p.group);
                    mine = seen_places(p.tree ? p.tree + (first_token + node) * p.tree_words : nullptr, p.tree_words,
                                       node, nodes, len, j0);
                }
                see0 = __shfl_sync(0xffffffffu, mine, g);
                see1 = __shfl_sync(0xffffffffu, mine, g + 8);
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (!(see0 >> (8 * n + 2 * t4 + i) & 1u)) sc[n][i] = -INFINITY;
                        if (!(see1 >> (8 * n + 2 * t4 + i) & 1u)) sc[n][2 + i] = -INFINITY;
                    }
            }
            // ---- running maximum; outputs follow where it rises ----
            float t0 = m0, t1 = m1;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                t0 = fmaxf(t0, fmaxf(sc[n][0], sc[n][1]));
                t1 = fmaxf(t1, fmaxf(sc[n][2], sc[n][3]));
            }
            t0 = quad_max(t0);
            t1 = quad_max(t1);
            const uint32_t vb = wait_entry(2 * s + 1);
            float vfix = 1.0f;
            if constexpr (KIND == kKvQ8) {
                const float *vsl = scales + ((entry + 2u * s + 1u) % R::kSlots) * kStep;
                float mine = vsl[lane];
                if (masked && j0 + lane >= len) mine = 0.0f;
                const uint32_t bits = __float_as_uint(mine) & 0x7fffffffu;
                // largest finite scale of the step; a non-finite one makes its own weights non-finite
                const uint32_t top = __reduce_max_sync(0xffffffffu, bits < 0x7f800000u ? bits : 0u);
                int e = static_cast<int>(top >> 23) - 126;
                e = e > 120 ? 120 : e;
                if (e > ve) {
                    vfix = exp2_fast(static_cast<float>(ve - e));
                    ve = e;
                }
                const float unit = __uint_as_float(static_cast<uint32_t>(127 - ve) << 23);   // 2^-ve
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const float2 d = *reinterpret_cast<const float2 *>(vsl + 8 * n + 2 * t4);
                    vd[n][0] = d.x * unit;
                    vd[n][1] = d.y * unit;
                }
            }
            if (__any_sync(0xffffffffu, t0 > m0 || t1 > m1 || vfix != 1.0f)) {
                const float f0 = t0 > m0 ? exp2_fast(m0 - t0) : 1.0f, f1 = t1 > m1 ? exp2_fast(m1 - t1) : 1.0f;
                l0 *= f0;
                l1 *= f1;
                const float a = f0 * vfix, b = f1 * vfix;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    o[n][0] *= a; o[n][1] *= a;
                    o[n][2] *= b; o[n][3] *= b;
                }
                m0 = t0;
                m1 = t1;
            }
            const float c0 = (m0 == -INFINITY ? 0.0f : m0) - kShift, c1 = (m1 == -INFINITY ? 0.0f : m1) - kShift;
            uint32_t pf[2][4];   // weights as operands of two 16-place products
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                float w[4] = {exp2_fast(sc[n][0] - c0), exp2_fast(sc[n][1] - c0), exp2_fast(sc[n][2] - c1),
                              exp2_fast(sc[n][3] - c1)};
                l0 += w[0] + w[1];
                l1 += w[2] + w[3];
                if constexpr (KIND == kKvQ8) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float x = w[i] * vd[n][i & 1];
                        // an unseen place weighs nothing, whatever its scale
                        w[i] = masked && !((i < 2 ? see0 : see1) >> (8 * n + 2 * t4 + (i & 1)) & 1u) ? 0.0f : x;
                    }
                }
                pf[n >> 1][(n & 1) * 2] = h2_bits(w[0], w[1]);
                pf[n >> 1][(n & 1) * 2 + 1] = h2_bits(w[2], w[3]);
                sc[n][0] = w[0]; sc[n][1] = w[1]; sc[n][2] = w[2]; sc[n][3] = w[3];
            }
            // ---- output += weights x values ----
            if constexpr (KIND == kKvF16) {
                if (masked) {
                    // Values no row sees (past the end) are cleared; a node
                    // whose value row is not finite is added by hand to the
                    // rows that see it, and cleared for the product.
                    uint4 *vrow[R::kRowBytes / 16];
#pragma unroll
                    for (int c = 0; c < R::kRowBytes / 16; ++c)
                        vrow[c] = reinterpret_cast<uint4 *>(ring + (at(vb, lane, c) - smem_u32(ring)));
                    bool strange = false;
                    const bool past = j0 + lane >= len;
                    if (j0 + lane >= len - nodes && !past)
#pragma unroll
                        for (int c = 0; c < R::kRowBytes / 16; ++c) {
                            const uint4 x = *vrow[c];
                            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                strange |= (w[k] & 0x7c00u) == 0x7c00u || (w[k] & 0x7c000000u) == 0x7c000000u;
                        }
                    uint32_t odd = __ballot_sync(0xffffffffu, strange);
                    if (odd) {
#pragma unroll
                        for (int n = 0; n < 4; ++n)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                pscr[(g + (i & 2) * 4) * 33 + 8 * n + 2 * t4 + (i & 1)] = sc[n][i];
                        __syncwarp();
                        for (; odd; odd &= odd - 1u) {
                            const int j = __ffs(odd) - 1;
                            const float w0 = pscr[g * 33 + j], w1 = pscr[(g + 8) * 33 + j];
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                const uint32_t v2 =
                                    *reinterpret_cast<const uint32_t *>(ring + (at(vb, j, n) - smem_u32(ring)) + 4 * t4);
                                if (see0 >> j & 1u) {
                                    o[n][0] += w0 * half_lo_to_float(v2);
                                    o[n][1] += w0 * half_hi_to_float(v2);
                                }
                                if (see1 >> j & 1u) {
                                    o[n][2] += w1 * half_lo_to_float(v2);
                                    o[n][3] += w1 * half_hi_to_float(v2);
                                }
                            }
                        }
                        __syncwarp();
                    }
                    if (past || strange)
#pragma unroll
                        for (int c = 0; c < R::kRowBytes / 16; ++c) *vrow[c] = make_uint4(0u, 0u, 0u, 0u);
                    __syncwarp();
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int np = 0; np < NT / 2; ++np) {
                        uint32_t b[4];   // columns 16 np .. + 7 (places 16 h + 0-7, 8-15), + 8 .. + 15
                        ldsm4_t(b, at(vb, 16 * h + (lane & 15), 2 * np + (lane >> 4)));
                        mma16816(o[2 * np], pf[h], b[0], b[1]);
                        mma16816(o[2 * np + 1], pf[h], b[2], b[3]);
                    }
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int np = 0; np < NT / 4; ++np) {
                        uint32_t b[4];   // chunks of 16 columns 2 np (places 16 h + 0-7, 8-15), 2 np + 1
                        ldsm4_t(b, at(vb, 16 * h + (lane & 15), 2 * np + (lane >> 4)));
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            // a word is two places' neighbouring columns: even ones to
                            // one product, odd ones to the next
                            const uint32_t lo = b[2 * i] ^ 0x80808080u, hi = b[2 * i + 1] ^ 0x80808080u;
                            mma16816(o[4 * np + 2 * i], pf[h], codes_to_half2(lo, 0x4240u), codes_to_half2(hi, 0x4240u));
                            mma16816(o[4 * np + 2 * i + 1], pf[h], codes_to_half2(lo, 0x4341u),
                                     codes_to_half2(hi, 0x4341u));
                        }
                    }
            }
            __syncwarp();
            if (2 * s + 1 + R::kSlots < entries) {
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                request(2 * s + 1 + R::kSlots);
            }
        }
        entry += static_cast<uint32_t>(entries);

        // ---- the four warps' outputs to one ----
        l0 = quad_sum(l0);
        l1 = quad_sum(l1);
        if (__any_sync(0xffffffffu, bad || gave_up)) {
            l0 = l1 = __int_as_float(0x7fffffff);
            if (lane == 0 && !gave_up) atomicOr(p.status, kDevBadPage);
        }
        if (t4 == 0) {
            ml[0][warp][g] = m0;
            ml[0][warp][g + 8] = m1;
            ml[1][warp][g] = l0;
            ml[1][warp][g + 8] = l1;
        }
        __syncthreads();    // also: every warp is done with the ring
        {
            float a = -INFINITY, b = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                a = fmaxf(a, ml[0][w][g]);
                b = fmaxf(b, ml[0][w][g + 8]);
            }
            const float back = KIND == kKvQ8 ? __uint_as_float(static_cast<uint32_t>(ve + 127) << 23) : 1.0f;   // 2^ve
            const float f0 = m0 == -INFINITY ? 0.0f : exp2_fast(m0 - a) * back;
            const float f1 = m1 == -INFINITY ? 0.0f : exp2_fast(m1 - b) * back;
            float *r0 = oscr + (warp * kRows + g) * (D + 8), *r1 = r0 + 8 * (D + 8);
            if constexpr (KIND == kKvF16) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    *reinterpret_cast<float2 *>(r0 + 8 * n + 2 * t4) = make_float2(o[n][0] * f0, o[n][1] * f0);
                    *reinterpret_cast<float2 *>(r1 + 8 * n + 2 * t4) = make_float2(o[n][2] * f1, o[n][3] * f1);
                }
            } else {
#pragma unroll
                for (int n = 0; n < NT; n += 2) {
                    *reinterpret_cast<float4 *>(r0 + 8 * n + 4 * t4) =
                        make_float4(o[n][0] * f0, o[n + 1][0] * f0, o[n][1] * f0, o[n + 1][1] * f0);
                    *reinterpret_cast<float4 *>(r1 + 8 * n + 4 * t4) =
                        make_float4(o[n][2] * f1, o[n + 1][2] * f1, o[n][3] * f1, o[n + 1][3] * f1);
                }
            }
        }
        __syncthreads();
        const bool whole = seg.nb == seg.blocks;
        const int first = whole ? 0 : owner_of(seg.unit_first, sh);
        const int last = whole ? 0 : owner_of(seg.unit_first + seg.blocks - 1, sh);
        float *part = whole ? nullptr : workspace_partial(p, blockIdx.x, seg.b0 == 0 ? 1 : 0, kRows, D);
        for (int i = tid; i < valid * (D / 8); i += kThreads) {
            const int row = i / (D / 8), d = (i - row * (D / 8)) * 8;
            float m = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) m = fmaxf(m, ml[0][w][row]);
            float l = 0.0f, v[8] = {};
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float mw = ml[0][w][row];
                l += ml[1][w][row] * (mw == -INFINITY ? 1.0f : exp2_fast(mw - m));
                const float *src = oscr + (w * kRows + row) * (D + 8) + d;
                const float4 a = *reinterpret_cast<const float4 *>(src), b = *reinterpret_cast<const float4 *>(src + 4);
                v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
                v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
            }
            if (whole) {
                const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = l == l ? v[k] * inv : l;
                store_half8(out_row<kRows, D>(p, seg, row) + d, v);
            } else {
                if (d == 0) {
                    part[row] = m;
                    part[kRows + row] = l;
                }
                *reinterpret_cast<float4 *>(part + 2 * kRows + row * D + d) = make_float4(v[0], v[1], v[2], v[3]);
                *reinterpret_cast<float4 *>(part + 2 * kRows + row * D + d + 4) = make_float4(v[4], v[5], v[6], v[7]);
            }
        }
        if (!whole) {
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                int *count = workspace_counters(p) + first;
                const int seen = atomicAdd(count, 1);
                last_flag = seen == last - first;
                if (last_flag) *count = 0;   // ready for the next call
            }
            __syncthreads();
            if (last_flag) {
                __threadfence();
                join_parts<kRows, D, kThreads>(p, seg, first, last - first + 1, valid, tid);
            }
        }
        __syncthreads();    // the scratch is the ring again
    }
    if (gave_up && lane == 0)   // copies still in flight land before the CTA leaves
        for (uint32_t n = asked > R::kSlots ? asked - R::kSlots : 0u; n < asked; ++n)
            mbar_wait_bounded(&bar[n % R::kSlots], (n / R::kSlots) & 1u, nullptr);
}

template <int D, int KIND>
cudaError_t launch_with(const AttnParams &p, int sms, cudaStream_t s, bool pdl)
{
    const int page = 1 << p.page_shift;
    CUtensorMap kmap, vmap;
    const int rows = page < kStep ? page : kStep;
    if (!encode_rows(&kmap, p, p.k, D, KIND, rows) || !encode_rows(&vmap, p, p.v, D, KIND, rows))
        return cudaErrorInvalidValue;
    auto kernel = tree_attn_rows_kernel<D, KIND>;
    cudaError_t e = ensure_smem_optin(reinterpret_cast<const void *>(kernel), Ring<D, KIND>::kSmem);
    if (e != cudaSuccess) return e;
    return launch_ex(kernel, dim3(static_cast<unsigned>(2 * sms)), dim3(kThreads), Ring<D, KIND>::kSmem, s, pdl, kmap,
                     vmap, p);
}

}  // namespace

int64_t attn_rows_workspace_floats(int sms) { return 2 * (2 * static_cast<int64_t>(sms)) * partial_floats(kRows, 128); }

cudaError_t launch_attn_rows(const AttnParams &p, int D, int kind, int sms, cudaStream_t s, bool pdl)
{
    if (2 * sms > kMaxGrid) return cudaErrorInvalidConfiguration;
    if (D == 64)
        return kind == kKvF16 ? launch_with<64, kKvF16>(p, sms, s, pdl) : launch_with<64, kKvQ8>(p, sms, s, pdl);
    return kind == kKvF16 ? launch_with<128, kKvF16>(p, sms, s, pdl) : launch_with<128, kKvQ8>(p, sms, s, pdl);
}

}  // namespace qmv
