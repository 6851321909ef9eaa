// qmv_attn_rows.cu -- attention over the paged cache for few query rows to a
// key/value head (8, 16 or 32 in a tile): one pass over the cached rows, bound
// by their bytes.
//
// Four warps to a CTA, two CTAs to an SM (four for 8 rows of 8-bit places).  A
// block of 128 places is 32 to each warp; a warp keeps all rows' running
// maximum, sum and output in registers and streams its own places through its
// own ring of shared-memory slots (tensor copies, one mbarrier to a slot,
// refilled by the warp as it empties them), so that warps wait for each other
// only at the end of a segment.  There the four outputs are brought to a common
// maximum and added in shared memory.
//   Products are m16n8k16 with fp32 accumulators, cached places or columns on
// the 16 side and query rows on the 8 side: s^T = k q^T, o^T += v^T p^T.  One
// token of four to eight heads a group then wastes half as much as with rows
// on the 16 side, and needs half the registers.  p = 2^(s - max + 10): the
// factor 2^10 keeps small weights out of fp16's subnormals, and cancels against
// the sum.  The maximum may lag by 2^5 before the outputs are rescaled.
//   8-bit rows: codes become exact fp16 integers in registers.  The key scale
// multiplies the score, the value scale the weight, both in fp32; weights are
// held below fp16's largest value by a running power of two of the largest value
// scale, handled like the running maximum.  It is one for all rows as long as they
// see the same places; from the first step on where some see a larger scale than
// before and others may not, each row has its own, in shared memory (the last steps
// of a request; in registers for every step: 60 for 56 us, 16 requests with 32 rows).
//   Weights are rounded to fp16 for the value product (fp16 x fp16 with fp32
// accumulators; a wider type would take twice the matrix instructions or more):
// with fp16 outputs, whose own rounding is 2.1e-4 of the result, that makes 2.4e-4
// to 2.9e-4.  Scores, maxima, sums, outputs and parts are fp32.
//   Measured: 64 requests of 100 to 16383 8-bit places, one token of 32 heads on
// 8 of 128: 186 us, 6.1 TB/s, 0.90 of the measured copy bandwidth; 16 uneven
// trees of up to 24 nodes over 511 to 8191 fp16 places, 16 heads on 8: 63 us,
// 0.68.  One request has little to stream and pays for the start, the ragged
// end and the join: 8 nodes over 30001 places 36.5 us where the bytes take 18,
// one token over 4095 places 10.3 us where they take 2.5.
#include <cstdint>

#include "qmv_attn.cuh"
#include "qmv_launch.h"

namespace qmv {

namespace {

constexpr int kBlock = RowsSplit::kBlock;
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kCost = RowsSplit::kCost;
constexpr int kStep = 32;           // places of a warp's step
constexpr float kShift = 10.0f;     // weights are 2^10 times exp(s - max)

constexpr float kLazy = 5.0f;       // a maximum may lag this far (log2): 2^(10 + 5) < 65504

template <int D, int KIND, int NR>
struct Ring {
    static constexpr int kRows = 8 * NR;
    static constexpr int kRowBytes = KIND == kKvF16 ? 2 * D : D;
    static constexpr int kBoxBytes = kRowBytes < 128 ? kRowBytes : 128;   // inner extent of a copy
    static constexpr int kHalves = kRowBytes / kBoxBytes;
    static constexpr int kDataBytes = kStep * kRowBytes;
    static constexpr int kScaleBytes = KIND == kKvQ8 ? kStep * 4 : 0;
    // 8 rows of 8-bit places leave registers for four CTAs to an SM.
    static constexpr int kCtas = KIND == kKvQ8 && NR == 1 ? 4 : 2;
    static constexpr int kSlots = (kCtas == 4 ? 12288 : 24576) / kDataBytes < 10 ? (kCtas == 4 ? 12288 : 24576) / kDataBytes : 10;
    // Shared memory: the warps' slots (at a segment's end their outputs), their
    // scale slots, weights of fp16 steps that hold non-finite values, queries
    // (32 rows: they are read from here at every step).
    static constexpr int kOutPitch = D + 4;
    static constexpr int kDataAll = kWarps * kSlots * kDataBytes;
    static constexpr int kOut = kWarps * kRows * kOutPitch * 4;
    static constexpr int kScaleAt = kDataAll > kOut ? kDataAll : kOut;
    static constexpr int kPAt = kScaleAt + kWarps * kSlots * kScaleBytes;
    static constexpr int kQAt = kPAt + (KIND == kKvF16 ? (kWarps * 8 * 34 * 2 + 15) / 16 * 16 : 0);
    static constexpr size_t kSmem = 1024 + kQAt + (NR > 2 ? kRows * D * 2 : 0);
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

// Bits of the magnitude of a finite value scale, else 0; the exponent e of 2^e
// above a scale of these bits (-126 .. 126); 2^-e and back.
__device__ __forceinline__ uint32_t finite_bits(float v)
{
    const uint32_t bits = __float_as_uint(v) & 0x7fffffffu;
    return bits < 0x7f800000u ? bits : 0u;
}
__device__ __forceinline__ int exponent_above(uint32_t bits)
{
    const int e = static_cast<int>(bits >> 23) - 126;
    return e > 126 ? 126 : e;
}
__device__ __forceinline__ float unit_of(int e) { return __uint_as_float(static_cast<uint32_t>(127 - e) << 23); }
__device__ __forceinline__ int exponent_of_unit(float u) { return 127 - static_cast<int>(__float_as_uint(u) >> 23); }

// Over the eight lanes that hold a column of a product's tile.
__device__ __forceinline__ float column_max(float v)
{
#pragma unroll
    for (int i = 4; i < 32; i <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, i));
    return v;
}

__device__ __forceinline__ float column_sum(float v)
{
#pragma unroll
    for (int i = 4; i < 32; i <<= 1) v += __shfl_xor_sync(0xffffffffu, v, i);
    return v;
}

// Transpose of an 8 x 8 matrix of fp16, two neighbours of a row to a lane's word.
__device__ __forceinline__ uint32_t transpose8(uint32_t v)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ uint32_t h2_bits(float a, float b) { return float2_to_half2_bits(make_float2(a, b)); }

template <int D, int KIND, int NR>
__global__ void __launch_bounds__(kThreads, Ring<D, KIND, NR>::kCtas)
    tree_attn_rows_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                          const AttnParams p)
{
    using R = Ring<D, KIND, NR>;
    constexpr int kRows = R::kRows;
    constexpr int KS = D / 16;    // 16-wide steps of a score product, 16-wide tiles of the output
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ Share sh;
    __shared__ uint64_t bars[kWarps][R::kSlots];
    __shared__ float ml[2][kWarps][kRows];
    __shared__ float units[kWarps][kRows];   // 8-bit rows: each row's 2^-ve, once they have their own
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t4 = lane & 3;
    uint8_t *ring = smem + warp * R::kSlots * R::kDataBytes;
    const uint32_t ring_at = smem_u32(ring);
    float *scales = reinterpret_cast<float *>(smem + R::kScaleAt) + warp * R::kSlots * kStep;
    const uint32_t scales_at = smem_u32(scales);
    __half *pscr = reinterpret_cast<__half *>(smem + R::kPAt) + warp * 8 * 34;
    uint8_t *qbuf = smem + R::kQAt;
    float *oscr = reinterpret_cast<float *>(smem);
    uint64_t *bar = bars[warp];

    if (tid == 0) {
        prefetch_map(&kmap);
        prefetch_map(&vmap);
    }
    if (lane == 0) {
        for (int i = 0; i < R::kSlots; ++i) mbar_init(&bar[i], 1);
        mbar_init_fence();
    }
    pdl_wait_prior_grid();
    find_share<kRows, kBlock, kCost, false, kThreads>(p, &sh);

    SegmentWalk<kRows, kBlock, kCost, false> walk;
    walk.begin(p, sh, static_cast<int>(blockIdx.x));
    Segment seg;
    // The ring: the slot that is consumed next and its phase; requests refill
    // the slot just consumed.
    uint32_t slot = 0, phase = 0;
    uint32_t asked = 0, taken = 0;
    bool gave_up = false;     // a wait ran out: nothing more is requested, outputs become NaN
    bool left_unit = false;   // word of a shared unit left for the second kernel
    while (walk.next(p, seg)) {
        const int64_t len = seg.w.len;
        const int nodes = seg.w.nodes;
        const int64_t first_place = seg.b0 * kBlock + warp * kStep;
        // this warp's steps: places first_place + 128 s, those that begin before len
        int64_t steps64 = len > first_place ? (len - first_place + kBlock - 1) / kBlock : 0;
        if (steps64 > seg.nb) steps64 = seg.nb;
        const int steps = static_cast<int>(steps64), entries = 2 * steps;
        bool bad = seg.w.bad;

        // ---- the tile's queries as product operands ----
        // (row indices of a request fit 32 bits: T * Hq does)
        const uint32_t row_base = static_cast<uint32_t>(seg.tile) * kRows, group_size = p.group;
        const uint32_t rows_left = static_cast<uint32_t>(nodes) * group_size - row_base;
        const int valid = rows_left < static_cast<uint32_t>(kRows) ? static_cast<int>(rows_left) : kRows;
        const int64_t first_token = p.start[seg.r];
        auto q_row = [&](int row) -> const __half * {
            if (row >= valid || seg.w.bad) return nullptr;
            const uint32_t i = (row_base + row) / group_size;
            return p.q + (first_token + i) * p.q_stride + (seg.kvh * p.group + (row_base + row - i * group_size)) * D;
        };
        constexpr bool kQRegs = NR <= 2;   // queries in registers
        uint32_t qreg[kQRegs ? NR : 1][kQRegs ? KS : 1][2];
        if constexpr (kQRegs) {
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                const __half *q0 = q_row(8 * n + g);
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    qreg[n][s][0] = qreg[n][s][1] = 0u;
                    if (!q0) continue;
                    if constexpr (KIND == kKvF16) {
                        // columns 16 s + 2 t4 and + 8
                        qreg[n][s][0] = *reinterpret_cast<const uint32_t *>(q0 + 16 * s + 2 * t4);
                        qreg[n][s][1] = *reinterpret_cast<const uint32_t *>(q0 + 16 * s + 8 + 2 * t4);
                    } else {
                        // a lane's four codes are columns 16 s + 4 t4 ..: the same order of columns on both sides
                        const uint2 a = *reinterpret_cast<const uint2 *>(q0 + 16 * s + 4 * t4);
                        qreg[n][s][0] = a.x;
                        qreg[n][s][1] = a.y;
                    }
                }
            }
        }
        // 32 rows: two 16-column groups to a thread, on their way to shared memory.
        // (Asked for here, ahead of the page ids, whose latency then covers theirs.)
        constexpr int kQItems = kQRegs ? 1 : kRows * KS / kThreads;
        uint4 qv[kQItems][2];
        if constexpr (!kQRegs) {
#pragma unroll
            for (int k = 0; k < kQItems; ++k) {
                const int i = tid + k * kThreads, row = i / KS, s = i - row * KS;
                const __half *q0 = q_row(row);
                qv[k][0] = qv[k][1] = make_uint4(0u, 0u, 0u, 0u);
                if (q0) {
                    qv[k][0] = *reinterpret_cast<const uint4 *>(q0 + 16 * s);
                    qv[k][1] = *reinterpret_cast<const uint4 *>(q0 + 16 * s + 8);
                }
            }
        }

        // Page ids ahead of their use: lane l holds chunk l of a group of 32
        // (a step is one chunk, or two of 16-place pages).
        const int page = 1 << p.page_shift;
        const int cps = page < kStep ? 2 : 1;       // chunks of a step
        const int box_rows = page < kStep ? page : kStep;
        const int32_t *trow = p.table + seg.r * p.width;
        const int64_t n_pages_used = (len + page - 1) >> p.page_shift;
        auto load_ids = [&](int group) -> int {
            const int c = group * 32 + lane;
            const int s = cps == 2 ? c >> 1 : c;
            const int64_t idx = (first_place + static_cast<int64_t>(s) * kBlock + (cps == 2 ? (c & 1) * 16 : 0)) >> p.page_shift;
            if (s >= steps || idx >= n_pages_used) return -1;
            const int id = trow[idx];
            if (id < 0 || id >= p.n_pages) {
                bad = true;
                return 0;
            }
            return id;
        };
        int ids = load_ids(0), ids_next = load_ids(1), group = 0;
        const int y_head = seg.kvh << p.page_shift, y_first = static_cast<int>(first_place & (page - 1));
        // Requests entry e of this segment (even: keys of step e / 2; odd: values) into slot `to`.
        auto request = [&](int e, uint32_t to) {
            if (gave_up) return;
            const int s = e >> 1;
            const int c0 = s * cps;
            if ((c0 >> 5) != group) {
                ids = ids_next;
                group = c0 >> 5;
                ids_next = load_ids(group + 1);
            }
            ++asked;
            const int id0 = __shfl_sync(0xffffffffu, ids, c0 & 31), id1 = __shfl_sync(0xffffffffu, ids, (c0 + cps - 1) & 31);
            if (lane == 0) {
                const CUtensorMap *map = (e & 1) ? &vmap : &kmap;
                uint8_t *dst = ring + to * R::kDataBytes;
                const int chunks = cps == 2 && id1 >= 0 ? 2 : 1;
                mbar_arrive_expect_tx(&bar[to], chunks * box_rows * (R::kRowBytes + (KIND == kKvQ8 ? 4 : 0)));
                // the step's place within its page
                const int y = y_head + (page > kStep ? (y_first + s * kBlock) & (page - 1) : 0);
                // (test only) the first entry of CTA 0 is expected but never requested
                const bool skip = p.test_skip_copy && blockIdx.x == 0 && warp == 0 && asked == 1u;
                for (int c = 0; c < chunks && !skip; ++c) {
                    const int id = c ? id1 : id0;
#pragma unroll
                    for (int h = 0; h < R::kHalves; ++h)
                        copy_box(dst + h * kStep * R::kBoxBytes + c * 16 * R::kBoxBytes, map, h * 64, y, id, &bar[to]);
                    if constexpr (KIND == kKvQ8) {
                        const float *src = ((e & 1) ? p.v_scale : p.k_scale) +
                                           ((static_cast<int64_t>(id) * p.Hkv) << p.page_shift) + y;
                        bulk_g2s(scales + to * kStep + c * 16, src, box_rows * 4, &bar[to]);
                    }
                }
            }
        };
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the last segment's reads and writes of the ring
        {
            uint32_t to = slot;
            for (int e = 0; e < R::kSlots && e < entries; ++e) {
                request(e, to);
                if (++to == R::kSlots) to = 0;
            }
        }

        if constexpr (!kQRegs) {
            // Rows of D fp16, 16-byte chunk c of row r at chunk c ^ (r & 7); for 8-bit
            // keys each group of 16 columns is ordered as its codes are used.
#pragma unroll
            for (int k = 0; k < kQItems; ++k) {
                const int i = tid + k * kThreads, row = i / KS, s = i - row * KS;
                uint4 a = qv[k][0], b = qv[k][1];
                if constexpr (KIND == kKvQ8) {
                    const uint4 lo = make_uint4(a.x, a.z, b.x, b.z), hi = make_uint4(a.y, a.w, b.y, b.w);
                    a = lo;
                    b = hi;
                }
                uint8_t *dst = qbuf + row * (D * 2);
                *reinterpret_cast<uint4 *>(dst + (((2 * s) ^ (row & 7)) << 4)) = a;
                *reinterpret_cast<uint4 *>(dst + (((2 * s + 1) ^ (row & 7)) << 4)) = b;
            }
            __syncthreads();
        }
        // Operands of step ks for all row tiles.
        auto q_operands = [&](int ks, uint32_t (&b)[NR][2]) {
            if constexpr (kQRegs) {
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    b[n][0] = qreg[n][ks][0];
                    b[n][1] = qreg[n][ks][1];
                }
            } else {
#pragma unroll
                for (int n = 0; n < NR; n += 2) {
                    uint32_t x[4];
                    const int row = 8 * (n + (lane >> 4)) + (lane & 7);
                    ldsm4(x, smem_u32(qbuf) + row * (D * 2) + (((2 * ks + ((lane >> 3) & 1)) ^ (row & 7)) << 4));
                    b[n][0] = x[0];
                    b[n][1] = x[1];
                    b[n + 1][0] = x[2];
                    b[n + 1][1] = x[3];
                }
            }
        };
        // o[n][dt]: columns 16 dt + g (0, 1) and + 8 (2, 3) of rows 8 n + 2 t4, + 1
        float o[NR][KS][4];
        float m[NR][2], l[NR][2];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
#pragma unroll
            for (int dt = 0; dt < KS; ++dt) o[n][dt][0] = o[n][dt][1] = o[n][dt][2] = o[n][dt][3] = 0.0f;
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.0f;
        }
        int ve = -126;        // 8-bit: 2^ve is at least the largest value scale so far
        bool own_units = false;

        // The entry that is due, as the address of its slot.
        auto wait_entry = [&]() {
            if (!gave_up && !mbar_wait_warp(&bar[slot], phase, p.status)) gave_up = true;
            return ring_at + slot * R::kDataBytes;
        };
        // Done with entry e: its slot takes the entry kSlots further on.
        auto release = [&](int e) {
            __syncwarp();
            if (gave_up) return;
            if (e + R::kSlots < entries) {
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                request(e + R::kSlots, slot);
            }
            ++taken;
            if (++slot == R::kSlots) {
                slot = 0;
                phase ^= 1u;
            }
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
            // ---- scores: sc[n][pm], places 16 pm + g (0, 1) and + 8 (2, 3) of rows 8 n + 2 t4, + 1 ----
            const uint32_t kb = wait_entry();
            float sc[NR][2][4];
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int pm = 0; pm < 2; ++pm) sc[n][pm][0] = sc[n][pm][1] = sc[n][pm][2] = sc[n][pm][3] = 0.0f;
            if constexpr (KIND == kKvF16) {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    uint32_t b[NR][2];
                    q_operands(ks, b);
#pragma unroll
                    for (int pm = 0; pm < 2; ++pm) {
                        uint32_t a[4];
                        ldsm4(a, at(kb, 16 * pm + (lane & 15), 2 * ks + (lane >> 4)));
#pragma unroll
                        for (int n = 0; n < NR; ++n) mma16816(sc[n][pm], a, b[n][0], b[n][1]);
                    }
                }
            } else {
#pragma unroll
                for (int ks = 0; ks < KS; ks += 2) {
                    uint32_t b[2][NR][2];
                    q_operands(ks, b[0]);
                    q_operands(ks + 1, b[1]);
#pragma unroll
                    for (int pm = 0; pm < 2; ++pm) {
                        uint32_t x[4];   // 16 codes of places 16 pm + 0-7, 8-15; the next 16 codes of both
                        ldsm4(x, at(kb, 16 * pm + (lane & 15), ks + (lane >> 4)));
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t lo = x[2 * i] ^ 0x80808080u, hi = x[2 * i + 1] ^ 0x80808080u;
                            const uint32_t a[4] = {codes_to_half2(lo, 0x4140u), codes_to_half2(hi, 0x4140u),
                                                   codes_to_half2(lo, 0x4342u), codes_to_half2(hi, 0x4342u)};
#pragma unroll
                            for (int n = 0; n < NR; ++n) mma16816(sc[n][pm], a, b[i][n][0], b[i][n][1]);
                        }
                    }
                }
            }
#pragma unroll
            for (int pm = 0; pm < 2; ++pm) {
                float d0 = p.scale_log2, d1 = p.scale_log2;
                if constexpr (KIND == kKvQ8) {
                    d0 *= lds1(scales_at + 4 * (slot * kStep + 16 * pm + g));
                    d1 *= lds1(scales_at + 4 * (slot * kStep + 16 * pm + 8 + g));
                }
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    sc[n][pm][0] *= d0;
                    sc[n][pm][1] *= d0;
                    sc[n][pm][2] *= d1;
                    sc[n][pm][3] *= d1;
                }
            }
            release(2 * s);
            // ---- places a row does not see ----
            uint32_t see[NR][2];   // of rows 8 n + 2 t4, + 1; shifted so that bit 0 is place g
            uint32_t mine = 0u;    // of row `lane`
            if (masked) {
                if (lane < valid) {
                    const int node = static_cast<int>((row_base + lane) / group_size);
                    mine = seen_places(p.tree ? p.tree + (first_token + node) * p.tree_words : nullptr, p.tree_words,
                                       node, nodes, len, j0);
                }
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        see[n][i] = __shfl_sync(0xffffffffu, mine, 8 * n + 2 * t4 + i) >> g;
#pragma unroll
                        for (int pm = 0; pm < 2; ++pm) {
                            if (!(see[n][i] >> (16 * pm) & 1u)) sc[n][pm][i] = -INFINITY;
                            if (!(see[n][i] >> (16 * pm + 8) & 1u)) sc[n][pm][2 + i] = -INFINITY;
                        }
                    }
            }
            // ---- running maximum; it may lag, and outputs follow when it moves ----
            float top[NR][2];
            bool rises = false;
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    top[n][i] = column_max(fmaxf(fmaxf(sc[n][0][i], sc[n][0][2 + i]), fmaxf(sc[n][1][i], sc[n][1][2 + i])));
                    // (no maximum yet: -inf + 5 < any score)
                    rises |= top[n][i] > m[n][i] + kLazy;
                }
            const uint32_t vb = wait_entry();
            float vfix = 1.0f;
            if constexpr (KIND == kKvQ8) {
                float d = lds1(scales_at + 4 * (slot * kStep + lane));
                if (masked && j0 + lane >= len) d = 0.0f;
                // largest finite scale of the step; a non-finite one makes its own weights non-finite
                const int e = exponent_above(__reduce_max_sync(0xffffffffu, finite_bits(d)));
                if (e > ve && !masked) {
                    vfix = exp2_fast(static_cast<float>(ve - e));
                    ve = e;
                    rises = true;
                } else if (e > ve) {
#pragma unroll
                    for (int n = 0; n < NR; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float &unit = units[warp][8 * n + 2 * t4 + i];
                            const int before = own_units ? exponent_of_unit(unit) : ve;
                            uint32_t most = 0u;   // of the places that this row sees
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const uint32_t bits = finite_bits(lds1(scales_at + 4 * (slot * kStep + 8 * k + g)));
                                if ((see[n][i] >> (8 * k) & 1u) && bits > most) most = bits;
                            }
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1) {
                                const uint32_t other = __shfl_xor_sync(0xffffffffu, most, d);
                                most = other > most ? other : most;
                            }
                            const int seen = exponent_above(most), now = seen > before ? seen : before;
                            const float f = exp2_fast(static_cast<float>(before - now));
#pragma unroll
                            for (int dt = 0; dt < KS; ++dt) {
                                o[n][dt][i] *= f;
                                o[n][dt][2 + i] *= f;
                            }
                            __syncwarp();         // every lane has read it
                            if (g == 0) unit = unit_of(now);
                        }
                    own_units = true;
                    __syncwarp();
                }
            }
            if (__any_sync(0xffffffffu, rises)) {
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float f = 1.0f;
                        if (top[n][i] > m[n][i]) {
                            f = exp2_fast(m[n][i] - top[n][i]);
                            m[n][i] = top[n][i];
                            l[n][i] *= f;
                        }
                        f *= vfix;
#pragma unroll
                        for (int dt = 0; dt < KS; ++dt) {
                            o[n][dt][i] *= f;
                            o[n][dt][2 + i] *= f;
                        }
                    }
            }
            // ---- weights ----
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float c = kShift - (m[n][i] == -INFINITY ? 0.0f : m[n][i]);
#pragma unroll
                    for (int pm = 0; pm < 2; ++pm) {
                        sc[n][pm][i] = exp2_fast(sc[n][pm][i] + c);
                        sc[n][pm][2 + i] = exp2_fast(sc[n][pm][2 + i] + c);
                        l[n][i] += sc[n][pm][i] + sc[n][pm][2 + i];
                    }
                }
            if constexpr (KIND == kKvQ8) {
#pragma unroll
                for (int pm = 0; pm < 2; ++pm) {
                    const float d0 = lds1(scales_at + 4 * (slot * kStep + 16 * pm + g));
                    const float d1 = lds1(scales_at + 4 * (slot * kStep + 16 * pm + 8 + g));
                    if (!own_units) {
                        const float e0 = d0 * unit_of(ve), e1 = d1 * unit_of(ve);
#pragma unroll
                        for (int n = 0; n < NR; ++n) {
                            sc[n][pm][0] *= e0;
                            sc[n][pm][1] *= e0;
                            sc[n][pm][2] *= e1;
                            sc[n][pm][3] *= e1;
                        }
                    } else {
#pragma unroll
                        for (int n = 0; n < NR; ++n)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const float unit = units[warp][8 * n + 2 * t4 + i];
                                sc[n][pm][i] *= d0 * unit;
                                sc[n][pm][2 + i] *= d1 * unit;
                            }
                    }
                }
                if (masked) {
                    // an unseen place weighs nothing, whatever its scale
#pragma unroll
                    for (int n = 0; n < NR; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int pm = 0; pm < 2; ++pm) {
                                if (!(see[n][i] >> (16 * pm) & 1u)) sc[n][pm][i] = 0.0f;
                                if (!(see[n][i] >> (16 * pm + 8) & 1u)) sc[n][pm][2 + i] = 0.0f;
                            }
                }
            }
            // Two rows' weights of a place to a word; the transpose of 8 x 8 of
            // them is the operand (two places of a row to a word).
            uint32_t pf[NR][2][2];
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int pm = 0; pm < 2; ++pm) {
                    pf[n][pm][0] = transpose8(h2_bits(sc[n][pm][0], sc[n][pm][1]));
                    pf[n][pm][1] = transpose8(h2_bits(sc[n][pm][2], sc[n][pm][3]));
                }
            // ---- output += weights x values ----
            if constexpr (KIND == kKvF16) {
                if (masked) {
                    // Values no row sees (past the end) are cleared; a node
                    // whose value row is not finite is added by hand to the
                    // rows that see it, and cleared for the product.
                    bool strange = false;
                    const bool past = j0 + lane >= len;
                    auto chunk = [&](int r, int c) { return reinterpret_cast<uint4 *>(ring + (at(vb, r, c) - ring_at)); };
                    if (j0 + lane >= len - nodes && !past)
#pragma unroll 4
                        for (int c = 0; c < R::kRowBytes / 16; ++c) {
                            const uint4 x = *chunk(lane, c);
                            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                strange |= (w[k] & 0x7c00u) == 0x7c00u || (w[k] & 0x7c000000u) == 0x7c000000u;
                        }
                    const uint32_t odd = __ballot_sync(0xffffffffu, strange);
                    if (odd) {
#pragma unroll
                        for (int n = 0; n < NR; ++n) {
#pragma unroll
                            for (int pm = 0; pm < 2; ++pm)
#pragma unroll
                                for (int k = 0; k < 2; ++k)   // row g, places 16 pm + 8 k + 2 t4, + 1
                                    *reinterpret_cast<uint32_t *>(pscr + g * 34 + 16 * pm + 8 * k + 2 * t4) = pf[n][pm][k];
                            __syncwarp();
                            for (uint32_t left = odd; left; left &= left - 1u) {
                                const int j = __ffs(left) - 1;
                                // (a weight of 0 counts as well: seen infinities and NaN show)
                                const bool s0 = __shfl_sync(0xffffffffu, mine, 8 * n + 2 * t4) >> j & 1u;
                                const bool s1 = __shfl_sync(0xffffffffu, mine, 8 * n + 2 * t4 + 1) >> j & 1u;
                                const float w0 = __half2float(pscr[2 * t4 * 34 + j]);
                                const float w1 = __half2float(pscr[(2 * t4 + 1) * 34 + j]);
#pragma unroll
                                for (int dt = 0; dt < KS; ++dt) {
                                    const float va = __half2float(reinterpret_cast<const __half *>(chunk(j, 2 * dt))[g]);
                                    const float vc = __half2float(reinterpret_cast<const __half *>(chunk(j, 2 * dt + 1))[g]);
                                    if (s0) {
                                        o[n][dt][0] += w0 * va;
                                        o[n][dt][2] += w0 * vc;
                                    }
                                    if (s1) {
                                        o[n][dt][1] += w1 * va;
                                        o[n][dt][3] += w1 * vc;
                                    }
                                }
                            }
                            __syncwarp();
                        }
                    }
                    if (past || strange)
#pragma unroll 4
                        for (int c = 0; c < R::kRowBytes / 16; ++c) *chunk(lane, c) = make_uint4(0u, 0u, 0u, 0u);
                    __syncwarp();
                }
#pragma unroll
                for (int pm = 0; pm < 2; ++pm)
#pragma unroll
                    for (int dt = 0; dt < KS; ++dt) {
                        uint32_t a[4];   // columns 16 dt + 0-7, 8-15 of places 16 pm + 0-7; of places + 8 .. + 15
                        ldsm4_t(a, at(vb, 16 * pm + (lane & 7) + ((lane >> 4) << 3), 2 * dt + ((lane >> 3) & 1)));
#pragma unroll
                        for (int n = 0; n < NR; ++n) mma16816(o[n][dt], a, pf[n][pm][0], pf[n][pm][1]);
                    }
            } else {
#pragma unroll
                for (int pm = 0; pm < 2; ++pm)
#pragma unroll
                    for (int dt = 0; dt < KS; dt += 2) {
                        uint32_t x[4];   // chunk dt of places 16 pm + 0-7, 8-15; chunk dt + 1
                        ldsm4_t(x, at(vb, 16 * pm + (lane & 15), dt + (lane >> 4)));
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            // a word is two places' neighbouring columns: even ones are rows
                            // 0-7 of the product's tile, odd ones rows 8-15
                            const uint32_t lo = x[2 * i] ^ 0x80808080u, hi = x[2 * i + 1] ^ 0x80808080u;
                            const uint32_t a[4] = {codes_to_half2(lo, 0x4240u), codes_to_half2(lo, 0x4341u),
                                                   codes_to_half2(hi, 0x4240u), codes_to_half2(hi, 0x4341u)};
#pragma unroll
                            for (int n = 0; n < NR; ++n) mma16816(o[n][dt + i], a, pf[n][pm][0], pf[n][pm][1]);
                        }
                    }
            }
            release(2 * s + 1);
        }

        // ---- the four warps' outputs to one ----
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) l[n][i] = column_sum(l[n][i]);
        const bool poison = __any_sync(0xffffffffu, bad || gave_up);
        if (poison && lane == 0 && !gave_up) atomicOr(p.status, kDevBadPage);
        if (g == 0)
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    ml[0][warp][8 * n + 2 * t4 + i] = m[n][i];
                    ml[1][warp][8 * n + 2 * t4 + i] = poison ? __int_as_float(0x7fffffff) : l[n][i];
                }
        __syncthreads();    // also: every warp is done with the ring
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int row = 8 * n + 2 * t4 + i;
                float most = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) most = fmaxf(most, ml[0][w][row]);
                float back = 1.0f;            // 8-bit: the row's 2^ve
                if constexpr (KIND == kKvQ8) back = unit_of(-(own_units ? exponent_of_unit(units[warp][row]) : ve));
                const float f = m[n][i] == -INFINITY ? 0.0f : exp2_fast(m[n][i] - most) * back;
                float *dst = oscr + (warp * kRows + row) * R::kOutPitch;
#pragma unroll
                for (int dt = 0; dt < KS; ++dt) {
                    if constexpr (KIND == kKvF16) {
                        dst[16 * dt + g] = o[n][dt][i] * f;
                        dst[16 * dt + 8 + g] = o[n][dt][2 + i] * f;
                    } else {
                        *reinterpret_cast<float2 *>(dst + 16 * dt + 2 * g) = make_float2(o[n][dt][i] * f, o[n][dt][2 + i] * f);
                    }
                }
            }
        __syncthreads();
        const bool whole = seg.whole;
        const int64_t first_out = first_token < 0 ? 0 : first_token;
        float *part = whole ? nullptr : workspace_partial(p, blockIdx.x, seg.b0 == 0 ? 1 : 0, kRows, D);
        for (int i = tid; i < valid * (D / 8); i += kThreads) {
            const int row = i / (D / 8), d = (i - row * (D / 8)) * 8;
            float most = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) most = fmaxf(most, ml[0][w][row]);
            float sum = 0.0f, v[8] = {};
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float mw = ml[0][w][row];
                sum += ml[1][w][row] * (mw == -INFINITY ? 1.0f : exp2_fast(mw - most));
                const float *src = oscr + (w * kRows + row) * R::kOutPitch + d;
                const float4 a = *reinterpret_cast<const float4 *>(src), b = *reinterpret_cast<const float4 *>(src + 4);
                v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
                v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
            }
            if (whole) {
                const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = sum == sum ? v[k] * inv : sum;
                store_half8(out_row<kRows, D>(p, first_out, seg.kvh, seg.tile, row) + d, v);
            } else {
                if (d == 0) {
                    part[row] = most;
                    part[kRows + row] = sum;
                }
                *part_columns<kRows>(part, row, d) = make_float4(v[0], v[1], v[2], v[3]);
                *part_columns<kRows>(part, row, d + 4) = make_float4(v[4], v[5], v[6], v[7]);
            }
        }
        if (seg.parts > 0) {
            left_unit = true;
            if (tid == 0) leave_unit(p, seg, valid, first_out);
        }
        __syncthreads();    // the scratch is the ring again
    }
    pdl_allow_next_grid();
    if (tid == 0 && !left_unit) workspace_units(p)[blockIdx.x].parts = 0;
    if (gave_up && lane == 0) {
        // copies still in flight land before the CTA leaves: entries taken .. asked - 1
        for (uint32_t n = taken; n < asked && n < taken + R::kSlots; ++n) {
            mbar_wait_bounded(&bar[slot], phase, nullptr);
            if (++slot == R::kSlots) {
                slot = 0;
                phase ^= 1u;
            }
        }
    }
}

template <int D, int KIND, int NR>
cudaError_t launch_with(const AttnParams &p, int sms, cudaStream_t s, bool pdl)
{
    const int page = 1 << p.page_shift;
    CUtensorMap kmap, vmap;
    const int rows = page < kStep ? page : kStep;
    if (!encode_rows(&kmap, p, p.k, D, KIND, rows) || !encode_rows(&vmap, p, p.v, D, KIND, rows))
        return cudaErrorInvalidValue;
    auto kernel = tree_attn_rows_kernel<D, KIND, NR>;
    cudaError_t e = ensure_smem_optin(reinterpret_cast<const void *>(kernel), Ring<D, KIND, NR>::kSmem);
    if (e != cudaSuccess) return e;
    const int grid = Ring<D, KIND, NR>::kCtas * sms;
    e = launch_ex(kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), Ring<D, KIND, NR>::kSmem, s, pdl, kmap, vmap, p);
    if (e != cudaSuccess) return e;
    return launch_join<8 * NR, D>(p, grid, kBlock, s, pdl);
}

template <int D, int KIND>
cudaError_t launch_for(const AttnParams &p, int64_t rows, int sms, cudaStream_t s, bool pdl)
{
    if (rows <= 8) return launch_with<D, KIND, 1>(p, sms, s, pdl);
    return rows <= 16 ? launch_with<D, KIND, 2>(p, sms, s, pdl) : launch_with<D, KIND, 4>(p, sms, s, pdl);
}

}  // namespace

int64_t attn_rows_workspace_floats(int sms)
{
    // two CTAs to an SM with 32 rows each, or four with 8
    return 2 * (2 * static_cast<int64_t>(sms)) * partial_floats(32, 128);
}

cudaError_t launch_attn_rows(const AttnParams &p, int D, int kind, int64_t rows, int sms, cudaStream_t s, bool pdl)
{
    if (4 * sms > kMaxGrid) return cudaErrorInvalidConfiguration;
    if (D == 64)
        return kind == kKvF16 ? launch_for<64, kKvF16>(p, rows, sms, s, pdl) : launch_for<64, kKvQ8>(p, rows, sms, s, pdl);
    return kind == kKvF16 ? launch_for<128, kKvF16>(p, rows, sms, s, pdl) : launch_for<128, kKvQ8>(p, rows, sms, s, pdl);
}

}  // namespace qmv
