// qmv_attn_tiles.cu -- attention over the paged cache for many query rows to a
// key/value head (trees of drafted tokens, chunks of prompts): 128-row tiles on
// the 5th-generation tensor cores (tcgen05.mma), scores and outputs in tensor
// memory.
//
// A CTA (one to an SM) works on up to 256 rows of one (request, key/value
// head) as two streams, each with a softmax warpgroup, a 128 x 128 score tile
// and a 128 x D output in tensor memory:
//   * more than 128 rows: a stream to each 128-row tile, both over every block
//     of 128 places, so that a block is read once for 256 rows;
//   * up to 128 rows: both streams hold the same rows, one takes the even and
//     one the odd blocks, and their outputs are joined at the end of a segment.
//   s = q k^T: queries and keys from shared memory (K-major, 128-byte swizzle,
// as the tensor copies deliver them).  The weights p go back to tensor memory
// over the scores they came from, as fp16, and are the A operand of o += p v;
// values are read N-major from the same kind of tile.  Both go by halves of 64
// places: as soon as a half's weights are there, their product and that half of
// the next block's scores are issued, beside the softmax of the other half (by
// whole blocks two prompt chunks took 190 us, by halves 161).  A thread owns a row:
// its maximum and sum need no exchange.  The output in tensor memory is rescaled
// only where a row's maximum has risen by more than 2^5 since it last was; until
// then the weights simply come out larger, p <= 2^(10 + 5) < 65504.
//   8-bit rows: a fourth warpgroup expands codes to fp16 tiles (exact integers);
// scales multiply scores and weights in fp32, weights are held below fp16's
// largest value by each row's running power of two of the largest value scale that
// the row sees, which enters through the exponent.
// The scales' arithmetic makes the softmax longer still: the chunks and the eight
// trees of the figures below take 234 and 135 us, the 16 nodes 186.
//   Weights are rounded to fp16 for the value product, as in the kernel for few rows
// (2.1e-4 of the result from the output's rounding alone, 2.9e-4 with it).
//   Value rows that no product may see (past the end; nodes' rows that are not finite)
// are cleared in shared memory by the stream that owns the tile, and in units of more
// than 128 rows, where both streams read it, by the first for both.
//   Warps: 0-3 and 4-7 the two softmax groups, 8 and 10 issue their products, 9
// the copies, 11 brings the next segment's queries as soon as the last products
// have read this one's (loaded by the softmax groups at a segment's start instead,
// the two prompt chunks took 161 us, not 151), 12-15 expand codes.  All waits are
// bounded.
//   What bounds it: up to 128 rows the bytes (16 nodes of 4 heads a group over
// 262147 places of 128: 172 us, 6.2 TB/s, 0.92 of the measured copy bandwidth);
// more rows the softmax: each half of a block is a chain of some 1700 cycles for
// its warp (about 850 of arithmetic, the rest waiting for scores to arrive from
// and weights to arrive in tensor memory), two warps share a scheduler, and the
// products, 2048 cycles a block of 256 rows at 128 columns, pass beside it (two
// chunks of 1400 and 1500 tokens behind 2000 and 2800, 32 heads on 8: 152 us,
// 970 TFLOP/s of useful products, 0.51 of the measured bf16 peak; 64 columns:
// eight trees of 64 nodes over 4001 to 8001 places, 64 heads on 8: 90 us).  A
// share of the exponentials as polynomials in place of the special-function unit
// made it slower (a quarter of them: 105 for 91 us), and so did passing a half's
// weights on only after asking for the next scores (170 for 155).
#include <cstdint>

#include "qmv_attn.cuh"
#include "qmv_launch.h"

namespace qmv {

namespace {

constexpr int kTile = 128;           // rows of a stream
constexpr int kRows = TilesSplit::kRows;
constexpr int kBlock = TilesSplit::kBlock;
constexpr int kCost = TilesSplit::kCost;
static_assert(kRows == 2 * kTile && kBlock == kTile, "two streams of a tile, and a thread of each to a place");
constexpr int kMmaWarp = 8, kCopyWarp = 9;   // and 10: the second stream's products
constexpr int kQueryWarp = 11;
constexpr int kExpandWarp = 12;      // 12-15, for 8-bit rows only
constexpr float kShift = 10.0f;      // weights are 2^10 times exp(s - max)
constexpr float kLazy = 5.0f;        // a maximum may lag this far (log2)

template <int D, int KIND>
struct Ring {
    static constexpr int kHalves = D / 64;                      // 64-column halves of a tile
    static constexpr int kHalfBytes = kBlock * 128;
    static constexpr int kTileBytes = kHalves * kHalfBytes;     // 128 rows of fp16
    // fp16: 128 KB of keys and values.  8-bit rows: 96 KB of expanded tiles, the
    // copies' own ring of codes (a tile, and with keys the block's two vectors of
    // scales), and the blocks' scales as the softmax reads them.
    static constexpr int kSlots = (KIND == kKvF16 ? 131072 : 98304) / kTileBytes;
    static constexpr int kCodeBytes = kBlock * D;
    static constexpr int kRawBytes = kCodeBytes + 2 * kBlock * 4;
    static constexpr int kRaw = KIND == kKvF16 ? 1 : kSlots;
    // Blocks whose scales are kept: those that the copies and the expanding warps
    // may be ahead, two tiles to a block, and the two in work.
    static constexpr int kScales = KIND == kKvF16 ? 1 : (D == 128 ? 8 : 16);
    static constexpr int kRawAt = (2 + kSlots) * kTileBytes;
    static constexpr int kScaleAt = kRawAt + kRaw * kRawBytes;
    static constexpr size_t kSmem = 1024 + (KIND == kKvF16 ? kRawAt : kScaleAt + kScales * 2 * kBlock * 4);
    // Registers of a thread: at launch, and after the softmax groups have taken
    // what the others give up (the shares add up to the launch's; these leave least in
    // local memory, and 224 and 56, or 176, 64 and 96, measured up to 1 % slower).
    static constexpr int kThreads = KIND == kKvF16 ? 384 : 512;
    static constexpr int kLaunchRegs = KIND == kKvF16 ? 168 : 128;
    static constexpr int kSoftmaxRegs = KIND == kKvF16 ? 208 : 176, kOtherRegs = KIND == kKvF16 ? 88 : 80;
    static constexpr int kExpandRegs = 80;
    static_assert(2 * kSoftmaxRegs + kOtherRegs + (KIND == kKvF16 ? 0 : kExpandRegs) == kThreads / 128 * kLaunchRegs,
                  "shares of the launch's registers");
};

// ---- tensor memory and products -----------------------------------------------

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 32 columns of this thread's lane; the values are there after ld_wait.
__device__ __forceinline__ void ld_32cols(uint32_t taddr, uint32_t *v)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr));
}

// The wait names the registers it makes valid, so that no use moves before it.
__device__ __forceinline__ void ld_wait(uint32_t *v)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]),
                   "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]),
                   "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]),
                   "+r"(v[30]), "+r"(v[31])
                 :
                 : "memory");
}

__device__ __forceinline__ void st_32cols(uint32_t taddr, const uint32_t *v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
        ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
          "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]),
          "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]),
          "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}

__device__ __forceinline__ void st_16cols(uint32_t taddr, const uint32_t *v)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
          "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

__device__ __forceinline__ void st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory matrix descriptors, 128-byte swizzle.  Rows of 128 bytes, eight
// of them to a swizzle atom of 1024 bytes.  K-major (queries, keys): the row is
// an M or N index, atoms follow each other along it.  N-major (values): the row
// is a K index and carries 64 columns; `next64` bytes lead to the next 64.
__device__ __forceinline__ uint64_t tile_desc(uint32_t saddr, uint32_t next64)
{
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFF) | static_cast<uint64_t>((next64 >> 4) & 0x3FFF) << 16 |
           static_cast<uint64_t>(1024 >> 4) << 32 | static_cast<uint64_t>(1) << 46 | static_cast<uint64_t>(2) << 61;
}

// Instruction descriptor, kind::f16: fp16 operands, fp32 accumulator, M = 128.
__device__ __forceinline__ constexpr uint32_t mma_desc(int n, bool b_n_major)
{
    return (1u << 4) | (b_n_major ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(kTile >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
        "r"(add ? 1 : 0)
        : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
        "r"(add ? 1 : 0)
        : "memory");
}

__device__ __forceinline__ void mma_commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

// Two fp32 values to a 64-bit register, and arithmetic on both at once.
__device__ __forceinline__ uint64_t pair(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float power_of_2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }   // -126 .. 127
__device__ __forceinline__ float low(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float high(uint64_t v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// 8-bit rows.  The value scales of 32 places are kept over a power of two, 2^e, e the
// exponent above the largest of them or the nearer of these limits; weights carry
// 2^(e - ve), ve the row's own.  So no step leaves fp32's range (2^(15 + 60 + 40) at
// the most, where a node that the row does not see has a far larger scale), and what
// lies below the lower limit is lost in the output's rounding to fp16.
constexpr int kLeastExponent = -40, kMostKept = 60, kMostExponent = 126;

// Barrier `id` among `n` threads.
__device__ __forceinline__ void group_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }

// Order of a segment's tiles in the ring: step i asks for the values of block
// i - lag and the keys of block i (lag 1: both streams on every block; 2: a
// stream on every second one).
__device__ __forceinline__ uint32_t seq_k(int i, int lag) { return static_cast<uint32_t>(i + (i >= lag ? i - lag + 1 : 0)); }
__device__ __forceinline__ uint32_t seq_v(int i, int lag, int nb)
{
    return static_cast<uint32_t>(i + (i + lag < nb ? i + lag : nb));
}

// Page ids of a segment's blocks ahead of their use, 32 chunks to a warp's
// register (a chunk is the part of a block that lies in one page).
struct PageAhead {
    int cur, next, group;
};

struct Barriers {
    uint64_t kv_full[8], kv_empty[8];
    uint64_t raw_full[8], raw_empty[8];   // 8-bit rows: the copies' ring of codes
    uint64_t scale_full[16];              // and the blocks' scales
    uint64_t clean[8];                    // fp16 rows: the value tile in a slot has been looked over (the second stream waits)
    // Segments by their number's parity: a role that lags by one is never taken for one that does not.
    uint64_t q_full[2];       // a segment's queries are in shared memory
    uint64_t q_empty;         // both streams' products have read them
    uint64_t seg_done[2];     // a segment's outputs are written
    uint64_t s_full[2][2];    // a half of a stream's scores is in tensor memory
    uint64_t p_full[2][2];    // a half of its weights is
    uint64_t o_full[2][2];    // that half's product with values is done
    uint64_t drain[2];        // (after a wait ran out) the stream's products in flight are done
};

// Where a role is: one of its threads walks, and the segment lies in shared
// memory, out of the registers that the loops over the blocks need.
struct Where {
    Segment seg;
    SegmentWalk<kRows, kBlock, kCost, true> walk;
    int more;
    __device__ __forceinline__ bool next_for_warp(const AttnParams &p)
    {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) more = walk.next(p, seg) ? 1 : 0;
        __syncwarp();
        return more != 0;
    }
};

struct Shared {
    Barriers b;
    Share share;
    uint32_t tmem;
    int gave_up;              // volatile use: a wait ran out somewhere
    int strange;              // a value row of the segment's nodes is not finite
    int bad[2];               // a page id of the segment is out of range, or its request's length
    Where where[6];           // the softmax groups, the streams' products, the copies, the expanding warps, the queries
    float m[kTile], l[kTile];
    int ve[kTile];
    // 8-bit rows, of each block kept: by 32 places, whose scales are not finite,
    // whose key scales are negative, the exponent above the largest of the finite
    // value scales, and the one that they are kept over
    uint32_t odd[16][4];
    uint32_t below[16][4];
    int exponent[16][4];
    int kept[16][4];
};

// Places below this one are seen by every row from `row` of the unit on.
__device__ __forceinline__ int64_t open_places(const AttnParams &p, const Segment &s, int row)
{
    const int64_t ctx = s.w.len - s.w.nodes;
    return p.tree ? ctx : ctx + (static_cast<uint32_t>(s.tile) * kRows + row) / static_cast<uint32_t>(p.group) + 1;
}

// The first block of a unit, of fp16 rows, whose value tile is looked over before
// either stream multiplies it: the first that holds a place some row of the unit
// does not see.  There rows past the end, and nodes' rows that are not finite, are
// cleared, and the latter are what add_strange_nodes adds; both streams read the
// tile, so which tiles these are does not depend on the stream.
__device__ __forceinline__ int64_t first_cleaned(const AttnParams &p, const Segment &s) { return open_places(p, s, 0) / kBlock; }

// Adds by hand what nodes with a non-finite value row (cleared for the products)
// give to columns d0 .. d0 + 31 of a row: exact, and rare.
template <int D>
__device__ __forceinline__ void add_strange_nodes(const AttnParams &p, const Segment &seg, const __half *q,
                                               const int32_t *tree_row, int node, float c, int d0, float (&o)[32])
{
    const int64_t ctx = seg.w.len - seg.w.nodes, cleaned = first_cleaned(p, seg);
    const int64_t lo = (seg.b0 > cleaned ? seg.b0 : cleaned) * kBlock, hi = (seg.b0 + seg.nb) * kBlock;
    const int page = 1 << p.page_shift;
    for (int64_t j = lo > ctx ? lo : ctx; j < hi && j < seg.w.len; ++j) {
        if (!(seen_places(tree_row, p.tree_words, node, seg.w.nodes, seg.w.len, j) & 1u)) continue;
        const int id = p.table[seg.r * p.width + (j >> p.page_shift)];
        if (id < 0 || id >= p.n_pages) continue;
        const int64_t row = id * p.page_stride +
                            ((static_cast<int64_t>(seg.kvh) << p.page_shift) + (j & (page - 1))) * D;
        const __half *v = static_cast<const __half *>(p.v) + row, *k = static_cast<const __half *>(p.k) + row;
        bool odd = false;
        for (int d = 0; d < D; ++d) odd |= (__half_as_ushort(v[d]) & 0x7c00u) == 0x7c00u;
        if (!odd) continue;
        float s = 0.0f;
        for (int d = 0; d < D; ++d) s += __half2float(q[d]) * __half2float(k[d]);
        const float w = exp2_fast(s * p.scale_log2 - c);
#pragma unroll
        for (int d = 0; d < 32; ++d) o[d] += w * __half2float(v[d0 + d]);
    }
}

// 8-bit rows: the exponent above the largest value scale that a row sees in a block of
// 128 places (kept from vd on over the exponents from `over` on), not below `ve` and not
// above `most_e`.
__device__ __forceinline__ int seen_exponent(uint32_t vd, uint32_t over, int most_e, const int32_t *tree_row, int tree_words,
                                          int node, int nodes, int64_t len, int64_t j0, int ve)
{
    int e = ve;
#pragma unroll 1
    for (int w = 0; w < 4; ++w) {
        const uint32_t see = seen_places(tree_row, tree_words, node, nodes, len, j0 + 32 * w);
        float most = 0.0f;
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
            const float4 d = lds4(vd + 128 * w + 4 * k);
            if (see >> k & 1u) most = fmaxf(most, fabsf(d.x));
            if (see >> k & 2u) most = fmaxf(most, fabsf(d.y));
            if (see >> k & 4u) most = fmaxf(most, fabsf(d.z));
            if (see >> k & 8u) most = fmaxf(most, fabsf(d.w));
        }
        const int own = static_cast<int>(__float_as_uint(most) >> 23) - 126 + static_cast<int>(__float_as_uint(lds1(over + 4 * w)));
        if (own > e) e = own;
    }
    return e < most_e ? e : most_e;
}

template <int D, int KIND>
__global__ void __launch_bounds__(Ring<D, KIND>::kThreads, 1)
    tree_attn_tiles_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                           const AttnParams p)
{
    using R = Ring<D, KIND>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ Shared sh;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *qbuf = smem;                          // two 128-row tiles of queries
    uint8_t *ring = smem + 2 * R::kTileBytes;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Barriers &b = sh.b;
    volatile int *gave_up = &sh.gave_up;

    if (tid == 0) {
        prefetch_map(&kmap);
        prefetch_map(&vmap);
        for (int i = 0; i < R::kSlots; ++i) {
            mbar_init(&b.kv_full[i], KIND == kKvF16 ? 1 : 4);
            mbar_init(&b.kv_empty[i], 2);
            mbar_init(&b.clean[i], 4);
        }
        for (int i = 0; KIND == kKvQ8 && i < R::kRaw; ++i) {
            mbar_init(&b.raw_full[i], 1);
            mbar_init(&b.raw_empty[i], 4);
        }
        for (int i = 0; KIND == kKvQ8 && i < R::kScales; ++i) mbar_init(&b.scale_full[i], 4);
        mbar_init(&b.q_empty, 2);
        for (int x = 0; x < 2; ++x) {
            mbar_init(&b.q_full[x], 1);
            mbar_init(&b.seg_done[x], 8);
            mbar_init(&b.drain[x], 1);
            for (int h = 0; h < 2; ++h) {
                mbar_init(&b.s_full[x][h], 1);
                mbar_init(&b.p_full[x][h], 4);
                mbar_init(&b.o_full[x][h], 1);
            }
        }
        sh.gave_up = 0;
        mbar_init_fence();
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    pdl_wait_prior_grid();
    find_share<kRows, kBlock, kCost, true, R::kThreads>(p, &sh.share);   // ends with a block barrier
    fence_after();
    const uint32_t tmem = sh.tmem;
    constexpr uint32_t kCopyRing = KIND == kKvF16 ? R::kSlots : R::kRaw;
    // Columns: scores of stream x (its weights over them, half by half) at 128 x,
    // outputs at 256 + D x.

    auto rows_of = [&](const Segment &s) -> int {
        const int64_t left = static_cast<int64_t>(s.w.nodes) * p.group - static_cast<int64_t>(s.tile) * kRows;
        return static_cast<int>(left < kRows ? left : kRows);
    };

    if (KIND == kKvQ8 && warp >= kExpandWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::kExpandRegs));
        // ---------------- codes to fp16 tiles: a thread to a row ----------------
        const int wt = tid & 127;
        const float scale = p.scale_log2 == 0.0f ? 1.0f : fabsf(p.scale_log2);   // as the softmax groups have it
        Where &at = sh.where[4];
        const Segment &seg = at.seg;
        uint32_t entry = 0;
        bool ok = true;
        if (wt == 0) at.walk.begin(p, sh.share, static_cast<int>(blockIdx.x));
        while (true) {
            group_sync(2, 128);
            if (wt == 0) at.more = at.walk.next(p, at.seg) ? 1 : 0;
            group_sync(2, 128);
            if (!at.more) break;
            if (seg.w.bad) continue;
            const int nb = static_cast<int>(seg.nb);
            const int lag = rows_of(seg) > kTile ? 1 : 2;
            const int64_t len = seg.w.len, b0 = seg.b0;
            const uint32_t first_block = entry / 2;      // blocks of the segments before
            for (int i = 0; ok && i < nb + lag; ++i)
                for (int k = 0; k < 2; ++k) {            // values of block i - lag, keys of block i
                    if (k == 0 ? i < lag : i >= nb) continue;
                    const uint32_t r = entry % R::kRaw, slot = entry % R::kSlots;
                    ok = ok && warp_wait_or_give_up(&b.raw_full[r], (entry / R::kRaw) & 1u, gave_up, p.status);
                    const uint32_t raw = smem_u32(smem + R::kRawAt) + r * R::kRawBytes;
                    if (ok && k == 1) {
                        // This block's scales, fit for use.  Keys: times the softmax scale.
                        // Values: over a power of two to 32 places, which goes into the
                        // exponent of the weights.  Ones that are not finite are listed and
                        // replaced, so that they reach no row that does not see them.  The
                        // -inf of a place that a row does not see has to survive its key scale:
                        // one of 0 becomes the least normal number, whose scores are below
                        // 2^-90 and so 0 beside any other, and negative ones are listed.
                        const uint32_t kept = (first_block + static_cast<uint32_t>(i)) % R::kScales;
                        const uint32_t src = raw + R::kCodeBytes + 4 * wt;
                        const uint32_t dst = smem_u32(smem + R::kScaleAt) + kept * (2 * kBlock * 4) + 4 * wt;
                        const bool there = (b0 + i) * kBlock + wt < len;
                        float kd = lds1(src), vd = lds1(src + 4 * kBlock);
                        const bool k_finite = (__float_as_uint(kd) & 0x7f800000u) != 0x7f800000u;
                        const bool v_finite = (__float_as_uint(vd) & 0x7f800000u) != 0x7f800000u;
                        kd = fminf(fmaxf(kd * scale, -3.402823466e38f), 3.402823466e38f);
                        if (kd == 0.0f) kd = 1.175494351e-38f;
                        if (!there || !k_finite) kd = 1.0f;
                        if (!there || !v_finite) vd = 0.0f;
                        const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(vd) & 0x7fffffffu);
                        const uint32_t odd = __ballot_sync(0xffffffffu, there && !(k_finite && v_finite));
                        const uint32_t below = __ballot_sync(0xffffffffu, kd < 0.0f);
                        const int e = static_cast<int>(most >> 23) - 126;
                        const int over = e > kMostKept ? kMostKept : (e < kLeastExponent ? kLeastExponent : e);
                        asm volatile("st.shared.f32 [%0], %1;" ::"r"(dst), "f"(kd) : "memory");
                        asm volatile("st.shared.f32 [%0], %1;" ::"r"(dst + 4 * kBlock), "f"(vd * power_of_2(-over)) : "memory");
                        if (lane == 0) {
                            sh.exponent[kept][warp & 3] = e;
                            sh.kept[kept][warp & 3] = over;
                            sh.odd[kept][warp & 3] = odd;
                            sh.below[kept][warp & 3] = below;
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&b.scale_full[kept]);
                    }
                    ok = ok && warp_wait_or_give_up(&b.kv_empty[slot], ((entry / R::kSlots) & 1u) ^ 1u, gave_up, p.status);
                    if (!ok) break;
                    // All of the row's codes first: no load can move above a store.
                    const uint32_t dst = smem_u32(ring) + slot * R::kTileBytes + wt * 128;
                    uint4 codes[D / 16];
#pragma unroll
                    for (int c = 0; c < D / 16; ++c)   // as the copies' swizzle of 128 or 64 bytes has them
                        codes[c] = lds4u(raw + wt * D + ((D == 128 ? c ^ (wt & 7) : c ^ ((wt >> 1) & 3)) << 4));
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        const uint4 q = codes[c];
                        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
                        uint32_t f[8];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            // a byte b ^ 0x80 under the exponent byte 0x64 is 1024 + 128 + code, exactly
                            const uint32_t u = w[j] ^ 0x80808080u;
                            const __half2 lo = __hsub2(as_h2(__byte_perm(u, 0x64646464u, 0x4140u)), as_h2(0x64806480u));
                            const __half2 hi = __hsub2(as_h2(__byte_perm(u, 0x64646464u, 0x4342u)), as_h2(0x64806480u));
                            f[2 * j] = *reinterpret_cast<const uint32_t *>(&lo);
                            f[2 * j + 1] = *reinterpret_cast<const uint32_t *>(&hi);
                        }
                        const uint32_t half = dst + (c >> 2) * R::kHalfBytes;
                        sts4u(half + ((((2 * c) & 7) ^ (wt & 7)) << 4), make_uint4(f[0], f[1], f[2], f[3]));
                        sts4u(half + ((((2 * c + 1) & 7) ^ (wt & 7)) << 4), make_uint4(f[4], f[5], f[6], f[7]));
                    }
                    fence_async();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&b.raw_empty[r]);
                        mbar_arrive(&b.kv_full[slot]);
                    }
                    ++entry;
                }
        }
    } else if (warp >= kMmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R::kOtherRegs));
    if (warp == kCopyWarp) {
        // ---------------- copies: one lane to each box ----------------
        Where &at = sh.where[3];
        const Segment &seg = at.seg;
        if (lane == 0) at.walk.begin(p, sh.share, static_cast<int>(blockIdx.x));
        const int page = 1 << p.page_shift;
        const int box_rows = page < kBlock ? page : kBlock;
        const int chunks = kBlock / box_rows;      // of a block: 1 .. 8
        uint32_t entry = 0;
        bool ok = true;
        while (ok && at.next_for_warp(p)) {
            if (seg.w.bad) continue;               // its outputs are NaN, nothing is read
            const int nb = static_cast<int>(seg.nb);
            const int64_t b0 = seg.b0;
            const int y_head = seg.kvh << p.page_shift;
            const int lag = rows_of(seg) > kTile ? 1 : 2;
            const int64_t used = (seg.w.len + page - 1) >> p.page_shift;
            const int32_t *trow = p.table + seg.r * p.width;
            auto load_ids = [&](int group) -> int {
                const int c = group * 32 + lane;
                const int i = c / chunks;
                const int64_t idx =
                    ((b0 + i) * kBlock + static_cast<int64_t>(c - i * chunks) * box_rows) >> p.page_shift;
                if (i >= nb || idx >= used) return -1;
                const int id = trow[idx];
                return id < 0 || id >= p.n_pages ? 0 : id;   // a bad page: read another, the softmax side sees it too
            };
            PageAhead pk = {load_ids(0), load_ids(1), 0}, pv = pk;
            auto ask = [&](int i, bool values) {
                PageAhead &a = values ? pv : pk;
                const int c0 = i * chunks;
                if ((c0 >> 5) != a.group) {
                    a.cur = a.next;
                    a.group = c0 >> 5;
                    a.next = load_ids(a.group + 1);
                }
                // fp16 tiles land where they are used; codes in a ring of their own
                const uint32_t slot = entry % kCopyRing;
                uint64_t *full = KIND == kKvF16 ? &b.kv_full[slot] : &b.raw_full[slot];
                uint64_t *empty = KIND == kKvF16 ? &b.kv_empty[slot] : &b.raw_empty[slot];
                uint8_t *dst = KIND == kKvF16 ? ring + slot * R::kTileBytes : smem + R::kRawAt + slot * R::kRawBytes;
                if (!warp_wait_or_give_up(empty, ((entry / kCopyRing) & 1u) ^ 1u, gave_up, p.status)) {
                    ok = false;
                    return;
                }
                // lane l: kind l / chunks of chunk l % chunks (the 64-column halves of an fp16
                // tile; or the codes and, with a block's keys, its key and value scales)
                const int c = lane % chunks, h = lane / chunks;
                const int id = __shfl_sync(0xffffffffu, a.cur, (c0 + c) & 31);
                const uint32_t there = __ballot_sync(0xffffffffu, h == 0 && id >= 0);
                const int row_bytes = KIND == kKvF16 ? 2 * D : (values ? D : D + 8);
                if (lane == 0) mbar_arrive_expect_tx(full, __popc(there) * box_rows * row_bytes);
                __syncwarp();
                const int64_t j = (b0 + i) * kBlock + c * box_rows;
                const int y = y_head + (static_cast<int>(j & (page - 1)) & ~(box_rows - 1));
                const CUtensorMap *map = values ? &vmap : &kmap;
                // (test only) the first tile of CTA 0 is expected but never requested
                const bool skip = p.test_skip_copy && blockIdx.x == 0 && entry == 0u;
                if constexpr (KIND == kKvF16) {
                    if (h < R::kHalves && id >= 0 && !skip)
                        copy_box(dst + h * R::kHalfBytes + c * box_rows * 128, map, 64 * h, y, id, full);
                } else {
                    if (h == 0 && id >= 0 && !skip) copy_box(dst + c * box_rows * D, map, 0, y, id, full);
                    if (!values && (h == 1 || h == 2) && id >= 0) {
                        const float *src = (h == 1 ? p.k_scale : p.v_scale) + ((static_cast<int64_t>(id) * p.Hkv) << p.page_shift) + y;
                        bulk_g2s(dst + R::kCodeBytes + (h - 1) * kBlock * 4 + c * box_rows * 4, src, box_rows * 4, full);
                    }
                }
                __syncwarp();
                ++entry;
            };
            for (int i = 0; ok && i < nb + lag; ++i) {
                if (i >= lag) ask(i - lag, true);
                if (ok && i < nb) ask(i, false);
            }
        }
        if (!ok && lane == 0)   // copies in flight land before the CTA leaves
            for (uint32_t n = entry > kCopyRing ? entry - kCopyRing : 0u; n < entry; ++n)
                mbar_wait_bounded(KIND == kKvF16 ? &b.kv_full[n % kCopyRing] : &b.raw_full[n % kCopyRing],
                                  (n / kCopyRing) & 1u, nullptr);
    } else if (warp == kMmaWarp || warp == kMmaWarp + 2) {
        // ---------------- products: a warp to each stream runs the loop, one elected lane issues ----------------
        const int x = (warp - kMmaWarp) >> 1;
        constexpr uint32_t kOutDesc = mma_desc(D, true);
        // A negative softmax scale turns the queries' signs (bit 13 negates A).
        const uint32_t score_desc = mma_desc(64, false) | (p.scale_log2 < 0.0f ? 1u << 13 : 0u);
        const uint64_t qd = tile_desc(smem_u32(qbuf), 16), kd = tile_desc(smem_u32(ring), 16);
        const uint64_t vd = tile_desc(smem_u32(ring), R::kHalfBytes);
        const uint32_t s_at = tmem + 128 * x, o_at = tmem + 256 + D * x;
        Where &at = sh.where[1 + x];
        const Segment &seg = at.seg;
        if (lane == 0) at.walk.begin(p, sh.share, static_cast<int>(blockIdx.x));
        uint32_t entry = 0, segs = 0, np = 0, commits = 0;   // np: phase of this stream's blocks
        uint32_t cleans = 0;                       // phases of the slots' barriers `clean`, a bit to a slot
        bool ok = true;
        while (ok && at.next_for_warp(p)) {
            if (!warp_wait_or_give_up(&b.q_full[segs & 1u], (segs >> 1) & 1u, gave_up, p.status)) {
                ok = false;
                break;
            }
            ++segs;
            if (seg.w.bad) {           // nothing to multiply, its outputs are NaN
                if (lane == 0) mbar_arrive(&b.q_empty);
                continue;
            }
            fence_after();
            const int nb = static_cast<int>(seg.nb);
            const bool two = rows_of(seg) > kTile;
            const int lag = two ? 1 : 2, step = lag;
            const uint64_t qx = qd + (two ? x : 0) * (R::kTileBytes >> 4);
            auto wait_tile = [&](uint32_t n) {
                const uint32_t e = entry + n;
                ok = ok && warp_wait_or_give_up(&b.kv_full[e % R::kSlots], (e / R::kSlots) & 1u, gave_up, p.status);
                return static_cast<uint64_t>((e % R::kSlots) * (R::kTileBytes >> 4));
            };
            // Both streams' products free a slot; a stream that has the block alone does it twice.
            auto free_tile = [&](uint32_t n) {
                uint64_t *empty = &b.kv_empty[(entry + n) % R::kSlots];
                mma_commit(empty);
                if (!two) mma_commit(empty);
            };
            // s = q k^T of half h of a block (64 places); the segment's last ones free the queries.
            auto scores = [&](uint64_t off, uint32_t sk, int h, bool last) {
                if (elect_one()) {
                    const uint64_t kx = kd + off + h * (64 * 128 >> 4);
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const uint32_t k16 = (ks >> 2) * (R::kHalfBytes >> 4) + (ks & 3) * 2;
                        mma_ss(s_at + 64 * h, qx + k16, kx + k16, score_desc, ks > 0);
                    }
                    mma_commit(&b.s_full[x][h]);
                    if (h == 1) free_tile(sk);
                    if (h == 1 && last) mma_commit(&b.q_empty);
                }
                __syncwarp();
                ++commits;
            };
            // Blocks from here on: the first stream's softmax group looks the value tile over for both.
            int64_t looked = 0;
            if constexpr (KIND == kKvF16) looked = two && x == 1 ? first_cleaned(p, seg) - seg.b0 : nb;
            const int i0 = two ? 0 : x;
            if (i0 >= nb && lane == 0) mbar_arrive(&b.q_empty);
            if (i0 < nb) {
                const uint32_t sk = seq_k(i0, lag);
                const uint64_t off = wait_tile(sk);
                if (!ok) break;
                fence_after();
                scores(off, sk, 0, false);
                scores(off, sk, 1, i0 + step >= nb);
            }
            for (int i = i0; ok && i < nb; i += step, np ^= 1u) {
                const uint32_t sv = seq_v(i, lag, nb), sk = seq_k(i + step, lag);
                const bool more = i + step < nb;
                const uint64_t v_off = wait_tile(sv);
                if (KIND == kKvF16 && i >= looked) {
                    const uint32_t slot = (entry + sv) % R::kSlots;
                    ok = ok && warp_wait_or_give_up(&b.clean[slot], cleans >> slot & 1u, gave_up, p.status);
                    cleans ^= 1u << slot;
                }
                uint64_t k_off = 0;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // o += p v, half a block, as its weights arrive
                    ok = ok && warp_wait_or_give_up(&b.p_full[x][h], np, gave_up, p.status);
                    if (!ok) break;
                    fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int ks = 4 * h; ks < 4 * h + 4; ++ks)
                            mma_ts(o_at, s_at + 64 * h + 8 * (ks - 4 * h), vd + v_off + ks * (2048 >> 4),
                                   kOutDesc, i > i0 || ks > 0);
                        mma_commit(&b.o_full[x][h]);
                        if (h == 1) free_tile(sv);
                    }
                    __syncwarp();
                    ++commits;
                    // that half's scores of the next block, over the weights that the product
                    // just issued reads first (a thread's products run in the order of issue)
                    if (more) {
                        if (h == 0) k_off = wait_tile(sk);
                        if (!ok) break;
                        fence_after();
                        scores(k_off, sk, h, i + 2 * step >= nb);
                    }
                }
            }
            entry += 2u * static_cast<uint32_t>(nb);
        }
        if (!ok && commits > 0) {   // products in flight end before the tensor memory is given back
            if (elect_one()) mma_commit(&b.drain[x]);
            __syncwarp();
            if (lane == 0) mbar_wait_bounded(&b.drain[x], 0, nullptr);
            __syncwarp();
        }
    } else if (warp == kQueryWarp) {
        // ---------------- queries: to shared memory as the last segment's products are done with it ----------------
        Where &at = sh.where[5];
        const Segment &seg = at.seg;
        if (lane == 0) at.walk.begin(p, sh.share, static_cast<int>(blockIdx.x));
        uint32_t segs = 0;
        bool joined = false;                       // the last segment's end uses the queries' memory
        int64_t blocks = 0;                        // of the last segment
        while (at.next_for_warp(p)) {
            if (segs > 0) {
                const uint32_t last = segs - 1;
                // This wait lasts as long as the last segment does, some 2 us a block (each
                // other role's waits are for one step of the pipeline): its limit grows with it.
                const unsigned long long limit = kWaitLimitNs + static_cast<unsigned long long>(blocks) * 100000ull;
                bool ok = warp_wait_or_give_up(&b.q_empty, last & 1u, gave_up, p.status, limit);
                if (segs > 1)                      // the one before it has long ended: at most two are in work
                    ok = ok && warp_wait_or_give_up(&b.seg_done[(last - 1) & 1u], ((last - 1) >> 1) & 1u, gave_up, p.status);
                if (joined) ok = ok && warp_wait_or_give_up(&b.seg_done[last & 1u], (last >> 1) & 1u, gave_up, p.status);
                if (!ok) break;
            }
            const int valid = rows_of(seg);
            bool bad = seg.w.bad;
            joined = bad || valid <= kTile;
            blocks = seg.nb;
            if (!bad) {
                // Rows past the last one are zeros, and all are for a scale of 0.  A lane copies
                // whole rows, 16 bytes at a time: the addresses are worked out once to a row.
                const int64_t first_token = p.start[seg.r] < 0 ? 0 : p.start[seg.r];
                const uint32_t group = static_cast<uint32_t>(p.group), base = static_cast<uint32_t>(seg.tile) * kRows;
                const int rows = valid > kTile ? kRows : kTile;
                const int there = p.scale_log2 == 0.0f ? 0 : valid;
#pragma unroll 1
                for (int r = lane; r < rows; r += 32) {
                    const uint32_t rho = base + r, t = rho / group;
                    const __half *src = r < there ? p.q + (first_token + t) * p.q_stride +
                                                        (static_cast<int64_t>(seg.kvh) * group + (rho - t * group)) * D
                                                  : p.q;
                    const uint32_t dst = smem_u32(qbuf) + (r >> 7) * R::kTileBytes + (r & 127) * 128 + ((r & 7) << 4);
                    const int bytes = r < there ? 16 : 0;
#pragma unroll
                    for (int c = 0; c < D / 8; ++c)
                        asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"((dst ^ ((c & 7) << 4)) + (c >> 3) * R::kHalfBytes),
                                     "l"(src + 8 * c), "r"(bytes)
                                     : "memory");
                }
                const int64_t used = (seg.w.len + (1 << p.page_shift) - 1) >> p.page_shift;
                const int64_t lo = (seg.b0 * kBlock) >> p.page_shift;
                const int64_t hi = (((seg.b0 + seg.nb) * kBlock - 1) >> p.page_shift) + 1;
                for (int64_t i = lo + lane; i < hi && i < used; i += 32) {
                    const int id = p.table[seg.r * p.width + i];
                    bad |= id < 0 || id >= p.n_pages;
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
            }
            fence_async();
            bad = __any_sync(0xffffffffu, bad);
            __syncwarp();                          // all lanes' copies before lane 0 says so (a vote orders no memory)
            if (lane == 0) {
                if (bad) atomicOr(p.status, kDevBadPage);
                sh.bad[segs & 1u] = bad ? 1 : 0;
                mbar_arrive(&b.q_full[segs & 1u]);
            }
            ++segs;
        }
    }
    } else {
        // ---------------- softmax: a thread to a row ----------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R::kSoftmaxRegs));
        const int x = warp >> 2;                   // stream
        const int wt = tid & 127;                  // lane of tensor memory: row within the stream's tile
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t s_at = tmem + lanes + 128 * x, o_at = tmem + lanes + 256 + D * x;
        // A negative scale turns the queries' signs in the products; scale 0 clears them.
        const float scale = p.scale_log2 == 0.0f ? 1.0f : fabsf(p.scale_log2);
        uint32_t entry = 0, ns = 0, segs = 0;      // ring entries so far; phase of this stream's blocks; segments
        bool ok = true;
        Where &at = sh.where[0];
        const Segment &seg = at.seg;
        bool left_unit = false;                    // word of a shared unit left for the second kernel
        if (tid == 0) at.walk.begin(p, sh.share, static_cast<int>(blockIdx.x));
        while (true) {
            if (tid == 0) {
                at.more = at.walk.next(p, at.seg) ? 1 : 0;
                sh.strange = 0;                    // (all have read the last segment's)
            }
            group_sync(1, 256);
            if (!at.more) break;
            const int valid = rows_of(seg);
            const bool two = valid > kTile;
            const int lag = two ? 1 : 2;
            const int nb = seg.w.bad ? 0 : static_cast<int>(seg.nb);
            const int64_t len = seg.w.len, ctx = len - seg.w.nodes, b0 = seg.b0;
            const int64_t first_token = p.start[seg.r] < 0 ? 0 : p.start[seg.r];
            const int64_t row_base = static_cast<int64_t>(seg.tile) * kRows;
            ok = warp_wait_or_give_up(&b.q_full[segs & 1u], (segs >> 1) & 1u, gave_up, p.status) && ok;
            const bool bad = seg.w.bad || !ok || sh.bad[segs & 1u] != 0;

            const int row = (two ? kTile * x : 0) + wt;              // row of the unit
            const int64_t rho = row_base + row;
            const int node = row < valid ? static_cast<int>(static_cast<uint32_t>(rho) / static_cast<uint32_t>(p.group)) : 0;
            const int32_t *tree_row = p.tree ? p.tree + (first_token + node) * p.tree_words : nullptr;
            // A warp whose rows all lie past the last one leaves its weights as they are:
            // what they give goes to rows that nobody reads.
            const bool idle = row - lane >= valid;
            // Places below `open` are seen by every row of this stream.
            const int64_t open = open_places(p, seg, two ? kTile * x : 0);
            float m = -INFINITY, l = 0.0f;
            bool first = true;
            int ve = kLeastExponent;               // 8-bit rows: 2^ve is at least the largest value scale seen so far
            for (int i = two ? 0 : x; ok && i < nb; i += two ? 1 : 2, ns ^= 1u) {
                const int64_t j0 = (b0 + i) * kBlock;
                const bool masked = j0 + kBlock > open;
                uint32_t kd = 0u, vd = 0u;                  // 8-bit rows: the block's scales, in shared memory
                const int *over = nullptr;                  // and the exponents that its value scales are kept over
                int e_block = kLeastExponent;               // the largest exponent of its value scales
                if constexpr (KIND == kKvQ8) {
                    const uint32_t block = entry / 2 + static_cast<uint32_t>(i), kept = block % R::kScales;
                    ok = warp_wait_or_give_up(&b.scale_full[kept], (block / R::kScales) & 1u, gave_up, p.status);
                    kd = smem_u32(smem + R::kScaleAt) + kept * (2 * kBlock * 4);
                    vd = kd + kBlock * 4;
                    over = sh.kept[kept];
                    const int *ev = sh.exponent[kept];
#pragma unroll
                    for (int w = 0; w < 4; ++w) e_block = ev[w] > e_block ? ev[w] : e_block;
                    // a scale that is not finite makes the rows that see its place NaN
#pragma unroll 1
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t odd = sh.odd[kept][w];
                        if (odd && (odd & seen_places(tree_row, p.tree_words, node, seg.w.nodes, len, j0 + 32 * w)))
                            l = __int_as_float(0x7fffffff);
                    }
                }
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    ok = ok && warp_wait_or_give_up(&b.s_full[x][h], ns, gave_up, p.status);
                    if (!ok) break;
                    fence_after();
                    if (!idle) {
                        uint32_t s[64];
                        ld_32cols(s_at + 64 * h, s);
                        ld_32cols(s_at + 64 * h + 32, s + 32);
                        ld_wait(s);
                        ld_wait(s + 32);
                        if (masked) {
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const uint32_t see =
                                    seen_places(tree_row, p.tree_words, node, seg.w.nodes, len, j0 + 64 * h + 32 * c);
                                const uint32_t kept = (entry / 2 + static_cast<uint32_t>(i)) % R::kScales;
                                const uint32_t below = KIND == kKvQ8 ? sh.below[kept][2 * h + c] : 0u;
#pragma unroll
                                for (int k = 0; k < 32; ++k)   // -inf, once the scale has multiplied it
                                    if (!(see >> k & 1u)) s[32 * c + k] = 0xff800000u ^ (below >> k & 1u) << 31;
                            }
                        }
                        uint32_t w[32];
                        float l_half;
                        // Weights by the maximum so far, beside the maximum of these
                        // scores; where one lies past the lag, the outputs follow the new
                        // maximum and the weights are taken again.
                        while (true) {
                            const float c0 = kShift - (m == -INFINITY ? 0.0f : m);
                            float top;
                            if constexpr (KIND == kKvF16) {
                                const uint64_t scale2 = pair(scale, scale), c2 = pair(c0, c0);
                                float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                                uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
                                for (int k = 0; k < 32; ++k) {
                                    const float s0 = __uint_as_float(s[2 * k]), s1 = __uint_as_float(s[2 * k + 1]);
                                    const uint64_t e = fma2(pair(s0, s1), scale2, c2);
                                    const float a = exp2_fast(low(e)), c = exp2_fast(high(e));
                                    sum[k & 1] = add2(sum[k & 1], pair(a, c));
                                    w[k] = float2_to_half2_bits(make_float2(a, c));
                                    t[k & 3] = fmaxf(t[k & 3], fmaxf(s0, s1));
                                }
                                sum[0] = add2(sum[0], sum[1]);
                                l_half = low(sum[0]) + high(sum[0]);
                                top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * scale;
                            } else {
                                // Weights carry their 32 places' power of two, 2^(e - ve), in the
                                // exponent (not below 2^-100: such weights are 0 as fp16 either
                                // way), and the sum is taken without it.
                                l_half = 0.0f;
                                float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                                for (int g = 0; g < 2; ++g) {
                                    const int drop = over[2 * h + g] - ve;
                                    const float by = drop < -100 ? -100.0f : static_cast<float>(drop);
                                    const uint64_t c2 = pair(c0 + by, c0 + by);
                                    float u[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                                    uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
                                    for (int k4 = 0; k4 < 8; ++k4) {
                                        const float4 d = lds4(kd + 256 * h + 128 * g + 16 * k4), dv = lds4(vd + 256 * h + 128 * g + 16 * k4);
#pragma unroll
                                        for (int i2 = 0; i2 < 2; ++i2) {
                                            const int k = 16 * g + 2 * k4 + i2;
                                            const uint64_t e = fma2(pair(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])),
                                                                    i2 ? pair(d.z, d.w) : pair(d.x, d.y), c2);
                                            const float a = exp2_fast(low(e)), c = exp2_fast(high(e));
                                            sum[i2] = add2(sum[i2], pair(a, c));
                                            const uint64_t q = mul2(pair(a, c), i2 ? pair(dv.z, dv.w) : pair(dv.x, dv.y));
                                            w[k] = float2_to_half2_bits(make_float2(low(q), high(q)));
                                            u[k & 3] = fmaxf(u[k & 3], fmaxf(low(e), high(e)));
                                        }
                                    }
                                    sum[0] = add2(sum[0], sum[1]);
                                    l_half += (low(sum[0]) + high(sum[0])) * exp2_fast(-by);
                                    t[g] = fmaxf(fmaxf(u[0], u[1]), fmaxf(u[2], u[3])) - (c0 + by);
                                    // stored at once: fewer registers (eight trees 146 -> 138 us; fp16
                                    // rows, which have them, gain nothing)
                                    st_16cols(s_at + 64 * h + 16 * g, w + 16 * g);
                                }
                                top = fmaxf(t[0], t[1]);
                            }
                            const bool rises = top > m + kLazy;   // (no maximum yet: -inf + 5 < any score)
                            if (!__any_sync(0xffffffffu, rises || e_block > ve)) break;
                            float vfix = 1.0f;
                            if (KIND == kKvQ8 && e_block > ve) {
                                // As far as this row sees them.  (In this branch, which a block seldom
                                // takes, and not ahead of the block's halves, where it made every
                                // block of 8-bit rows 4 to 20 % slower.)
                                int e = e_block > kMostExponent ? kMostExponent : e_block;
                                if (masked)
                                    e = seen_exponent(vd, smem_u32(over), e, tree_row, p.tree_words, node, seg.w.nodes, len, j0, ve);
                                vfix = exp2_fast(static_cast<float>(ve - e));
                                ve = e;
                                e_block = kLeastExponent;
                            }
                            __syncwarp();
                            if (!first) {
                                // of the products before these weights only the last may still run
                                ok = warp_wait_or_give_up(&b.o_full[x][1 - h], h == 1 ? ns : ns ^ 1u, gave_up, p.status);
                                if (!ok) break;
                                fence_after();
                                float f = rises ? exp2_fast(m - top) : 1.0f;
                                l *= f;
                                f *= vfix;
#pragma unroll 1
                                for (int c = 0; c < D / 32; ++c) {
                                    uint32_t v[32];
                                    ld_32cols(o_at + 32 * c, v);
                                    ld_wait(v);
#pragma unroll
                                    for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * f);
                                    st_32cols(o_at + 32 * c, v);
                                }
                            }
                            if (rises) m = top;
                        }
                        if (!ok) break;
                        if constexpr (KIND == kKvF16) st_32cols(s_at + 64 * h, w);
                        l += l_half;
                    }
                    if (KIND == kKvF16 && masked && h == 0 && (x == 0 || !two)) {
                        // Value rows past the end are cleared, and so are nodes' rows
                        // that are not finite (add_strange_nodes adds those): before this
                        // stream's product, and where the other reads the tile as well,
                        // before it is told that the tile is clean.
                        const uint32_t e = entry + seq_v(i, lag, nb), slot = e % R::kSlots;
                        if (j0 + wt >= ctx) {
                            ok = ok && wait_or_give_up(&b.kv_full[slot], (e / R::kSlots) & 1u, gave_up, p.status);
                            uint8_t *v = ring + slot * R::kTileBytes + wt * 128;
                            bool clear = j0 + wt >= len;
                            if (ok && !clear) {
#pragma unroll
                                for (int hh = 0; hh < R::kHalves; ++hh)
#pragma unroll
                                    for (int c = 0; c < 8; ++c) {
                                        const uint4 q4 =
                                            *reinterpret_cast<const uint4 *>(v + hh * R::kHalfBytes + ((c ^ (wt & 7)) << 4));
                                        const uint32_t u[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
                                        for (int k = 0; k < 4; ++k)
                                            clear |= (u[k] & 0x7c00u) == 0x7c00u || (u[k] & 0x7c000000u) == 0x7c000000u;
                                    }
                                if (clear) sh.strange = 1;
                            }
                            if (ok && clear)
#pragma unroll
                                for (int hh = 0; hh < R::kHalves; ++hh)
#pragma unroll
                                    for (int c = 0; c < 8; ++c)
                                        *reinterpret_cast<uint4 *>(v + hh * R::kHalfBytes + (c << 4)) = make_uint4(0u, 0u, 0u, 0u);
                            fence_async();
                        }
                        ok = __all_sync(0xffffffffu, ok);
                        __syncwarp();
                        if (two && ok && lane == 0) mbar_arrive(&b.clean[slot]);
                    }
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    st_wait();
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&b.p_full[x][h]);
                    first = false;
                }
            }
            entry += 2u * static_cast<uint32_t>(nb);
            // ---- this stream's outputs are complete once its last product is ----
            if (!first && ok) ok = warp_wait_or_give_up(&b.o_full[x][1], ns ^ 1u, gave_up, p.status);
            fence_after();
            if (__any_sync(0xffffffffu, bad || !ok || *gave_up)) {
                l = __int_as_float(0x7fffffff);
                first = true;
            }
            group_sync(1, 256);                    // every value row has been looked at
            const bool strange = sh.strange != 0;
            float f = 1.0f;
            if (!two) {
                // Stream 1 hands its rows to stream 0 over the queries' shared memory.
                float *xo = reinterpret_cast<float *>(qbuf);
                if (x == 1) {
                    sh.m[wt] = m;
                    sh.l[wt] = l;
                    sh.ve[wt] = ve;
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t v[32];
                        if (!first) {
                            ld_32cols(o_at + 32 * c, v);
                            ld_wait(v);
                        }
                        if (wt < valid)
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const int at = ((c * 8 + k) + wt) & (D / 4 - 1);   // rows begin at different banks
                                *reinterpret_cast<uint4 *>(xo + wt * D + 4 * at) =
                                    first ? make_uint4(0u, 0u, 0u, 0u)
                                          : make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                            }
                    }
                }
                group_sync(1, 256);
            }
            const bool whole = seg.whole;
            float *part = whole ? nullptr : workspace_partial(p, blockIdx.x, seg.b0 == 0 ? 1 : 0, kRows, D);
            if (two || x == 0) {
                float f1 = 0.0f;
                bool own = !first, other = false;  // outputs of this stream, and of stream 1, are to be added
                if (KIND == kKvQ8 && two) f = power_of_2(ve);
                if (!two) {
                    const float m1 = sh.m[wt], top = fmaxf(m, m1);
                    own = own && m != -INFINITY;   // (also those whose factor is 0: infinities and NaN show)
                    other = m1 != -INFINITY;
                    f = m == -INFINITY ? 0.0f : exp2_fast(m - top);
                    f1 = m1 == -INFINITY ? 0.0f : exp2_fast(m1 - top);
                    const float l1 = sh.l[wt];
                    l = (m == -INFINITY ? l : l * f) + (m1 == -INFINITY ? l1 : l1 * f1);
                    m = top;
                    if constexpr (KIND == kKvQ8) {
                        f *= power_of_2(ve);
                        f1 *= power_of_2(sh.ve[wt]);
                    }
                }
                const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
                const __half *q = nullptr;
                if (KIND == kKvF16 && strange && row < valid && !seg.w.bad)
                    q = p.q + (first_token + node) * p.q_stride + (seg.kvh * p.group + (rho - static_cast<int64_t>(node) * p.group)) * D;
                if (!whole && row < valid) {
                    part[row] = m;
                    part[kRows + row] = l;
                }
                __half *dst = whole && row < valid ? out_row<kRows, D>(p, first_token, seg.kvh, seg.tile, row) : nullptr;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t v[32];
                    float o[32];
                    __syncwarp();
                    if (!first) {
                        ld_32cols(o_at + 32 * c, v);
                        ld_wait(v);
                    }
                    if (row >= valid) continue;
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = own ? __uint_as_float(v[k]) * f : 0.0f;
                    if (other) {
                        const float *xo = reinterpret_cast<const float *>(qbuf) + wt * D;
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const float4 a = *reinterpret_cast<const float4 *>(xo + 4 * (((c * 8 + k) + wt) & (D / 4 - 1)));
                            o[4 * k] += a.x * f1; o[4 * k + 1] += a.y * f1;
                            o[4 * k + 2] += a.z * f1; o[4 * k + 3] += a.w * f1;
                        }
                    }
                    if (q) add_strange_nodes<D>(p, seg, q, tree_row, node, (m == -INFINITY ? 0.0f : m) - kShift, 32 * c, o);
                    if (whole) {
#pragma unroll
                        for (int k = 0; k < 32; k += 8) {
                            float o8[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) o8[i] = l == l ? o[k + i] * inv : l;
                            store_half8(dst + 32 * c + k, o8);
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            *part_columns<kRows>(part, row, 32 * c + k) = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
                    }
                }
            }
            if (tid == 0 && seg.parts > 0) {
                left_unit = true;
                leave_unit(p, seg, valid, first_token);
            }
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&b.seg_done[segs & 1u]);
            ++segs;
            group_sync(1, 256);                    // nobody reads this segment's record any more
        }
        if (tid == 0 && !left_unit) workspace_units(p)[blockIdx.x].parts = 0;
    }
    fence_before();
    pdl_allow_next_grid();
    __syncthreads();
    if (warp == kMmaWarp) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

template <int D, int KIND>
cudaError_t launch_with(const AttnParams &p, int sms, cudaStream_t s, bool pdl)
{
    const int page = 1 << p.page_shift;
    const int rows = page < kBlock ? page : kBlock;
    CUtensorMap kmap, vmap;
    using R = Ring<D, KIND>;
    if (!encode_rows(&kmap, p, p.k, D, KIND, rows) || !encode_rows(&vmap, p, p.v, D, KIND, rows))
        return cudaErrorInvalidValue;
    auto kernel = tree_attn_tiles_kernel<D, KIND>;
    cudaError_t e = ensure_smem_optin(reinterpret_cast<const void *>(kernel), R::kSmem);
    if (e != cudaSuccess) return e;
    // The softmax groups' share of the registers exists only if the launch brings it.
    static const int regs = [] {
        cudaFuncAttributes a;
        return cudaFuncGetAttributes(&a, tree_attn_tiles_kernel<D, KIND>) == cudaSuccess ? a.numRegs : 0;
    }();
    if (regs < R::kLaunchRegs) return cudaErrorInvalidConfiguration;
    e = launch_ex(kernel, dim3(static_cast<unsigned>(sms)), dim3(R::kThreads), R::kSmem, s, pdl, kmap, vmap, p);
    if (e != cudaSuccess) return e;
    return launch_join<kRows, D>(p, sms, kBlock, s, pdl);
}

}  // namespace

int64_t attn_tiles_workspace_floats(int sms) { return 2 * static_cast<int64_t>(sms) * partial_floats(kRows, 128); }

cudaError_t launch_attn_tiles(const AttnParams &p, int D, int kind, int sms, cudaStream_t s, bool pdl)
{
    if (sms > kMaxGrid) return cudaErrorInvalidConfiguration;
    if (D == 64) return kind == kKvF16 ? launch_with<64, kKvF16>(p, sms, s, pdl) : launch_with<64, kKvQ8>(p, sms, s, pdl);
    return kind == kKvF16 ? launch_with<128, kKvF16>(p, sms, s, pdl) : launch_with<128, kKvQ8>(p, sms, s, pdl);
}

}  // namespace qmv
