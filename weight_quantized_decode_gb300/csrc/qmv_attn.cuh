// qmv_attn.cuh -- what the attention kernels over the paged cache share: the
// split of the work over the CTAs of a persistent grid, the mask of a row, and
// the join of partial results.
//
// A unit is one (request, key/value head, tile of ROWS query rows); a row is
// one (new token, query head of the group).  Its places are cut into blocks of
// BLOCK.  All units' blocks, in order, are one long list, and CTA c of g takes
// blocks [c B / g, (c + 1) B / g): the same share for each, however uneven the
// requests are, with no plan made on the host.  A CTA's share is a run of
// segments, each a range of one unit's blocks.  A unit that several CTAs share
// is joined by the last of them to finish: each writes its rows' running
// maximum, sum and unnormalised output (fp32) to its own place of the
// workspace, and the last one adds them in CTA order, so that the result does
// not depend on which one it was.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "qmv_common.cuh"
#include "qmv_kv.h"

namespace qmv {

// Request r's share of the work.
struct RequestWork {
    int nodes;         // new tokens
    int tiles;         // row tiles
    int64_t len;       // places
    bool bad;          // a length the cache cannot have: one block that gives NaN
    int64_t per_head;  // blocks of the units of one key/value head
    int64_t total;     // blocks of all its units
};

// Blocks of the unit of row tile `tile`.  CUT: the rows of a chain see nothing
// past the tile's last token, and the blocks there are left out.
template <int ROWS, int BLOCK, bool CUT>
__device__ __forceinline__ int64_t unit_blocks(const AttnParams &p, const RequestWork &w, int tile)
{
    if (w.bad) return 1;
    int64_t places = w.len;
    if (CUT && !p.tree) {
        const int64_t last = ((static_cast<int64_t>(tile) + 1) * ROWS - 1) / p.group;   // the tile's last token
        if (last < w.nodes) places = w.len - w.nodes + last + 1;
    }
    return (places + BLOCK - 1) / BLOCK;
}

template <int ROWS, int BLOCK, bool CUT>
__device__ __forceinline__ RequestWork request_work(const AttnParams &p, int64_t r)
{
    RequestWork w;
    // offsets past the T rows of q are cut off
    const int64_t lo = p.start[r], hi = p.start[r + 1];
    const int64_t a = lo < 0 ? 0 : lo, b = hi > p.T ? p.T : hi;
    w.nodes = b > a ? static_cast<int>(b - a) : 0;
    w.len = p.kv_len[r];
    w.bad = lo < 0 || hi > p.T || w.len < w.nodes || w.len > (p.width << p.page_shift);
    if (w.bad) w.len = 0;
    w.tiles = static_cast<int>((static_cast<int64_t>(w.nodes) * p.group + ROWS - 1) / ROWS);
    if (CUT && !p.tree) {
        w.per_head = 0;
        for (int t = 0; t < w.tiles; ++t) w.per_head += unit_blocks<ROWS, BLOCK, CUT>(p, w, t);
    } else {
        w.per_head = w.tiles * unit_blocks<ROWS, BLOCK, CUT>(p, w, 0);
    }
    w.total = w.per_head * p.Hkv;
    return w;
}

// Where a CTA's share begins, in shared memory (find_share).
struct Share {
    int64_t lo, hi;      // blocks [lo, hi) of the list
    int64_t total;       // all blocks
    int64_t r;           // the request block lo falls into
    int64_t before;      // blocks of the requests before it
    int g;               // CTAs that have a share
    int64_t sums[32];
    int64_t found[2];
};

// Every thread of the block calls this (THREADS of them, a multiple of 32).
template <int ROWS, int BLOCK, bool CUT, int THREADS>
__device__ __forceinline__ void find_share(const AttnParams &p, Share *sh)
{
    constexpr int W = THREADS / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // inclusive scan of v over the block; *all = the block's sum
    auto scan = [&](int64_t v, int64_t *all) {
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, v, d);
            if (lane >= d) v += u;
        }
        __syncthreads();
        if (lane == 31) sh->sums[warp] = v;
        __syncthreads();
        int64_t add = 0, sum = 0;
        for (int i = 0; i < W; ++i) {
            if (i < warp) add += sh->sums[i];
            sum += sh->sums[i];
        }
        *all = sum;
        return v + add;
    };
    int64_t mine = 0, total = 0;
    for (int64_t r = tid; r < p.R; r += THREADS) mine += request_work<ROWS, BLOCK, CUT>(p, r).total;
    scan(mine, &total);
    const int64_t g = total < gridDim.x ? total : static_cast<int64_t>(gridDim.x);
    const int64_t lo = g > 0 && blockIdx.x < g ? total * blockIdx.x / g : 0;
    const int64_t hi = g > 0 && blockIdx.x < g ? total * (blockIdx.x + 1) / g : 0;
    int64_t before = 0;
    for (int64_t r0 = 0; r0 < p.R && before <= lo && lo < hi; r0 += THREADS) {
        const int64_t cnt = r0 + tid < p.R ? request_work<ROWS, BLOCK, CUT>(p, r0 + tid).total : 0;
        int64_t all = 0;
        const int64_t upto = before + scan(cnt, &all);
        if (cnt > 0 && upto - cnt <= lo && lo < upto) {
            sh->found[0] = r0 + tid;
            sh->found[1] = upto - cnt;
        }
        before += all;
    }
    __syncthreads();
    if (tid == 0) {
        sh->lo = lo;
        sh->hi = hi;
        sh->total = total;
        sh->g = static_cast<int>(g);
        if (lo < hi) {
            sh->r = sh->found[0];
            sh->before = sh->found[1];
        }
    }
    __syncthreads();
}

// A CTA's part of one unit.
struct Segment {
    int64_t r;            // request
    int kvh, tile;        // key/value head, row tile
    int64_t b0, nb;       // its blocks [b0, b0 + nb) of the unit
    int64_t blocks;       // blocks of the unit
    int64_t unit_first;   // the list's index of the unit's first block
    RequestWork w;
};

// Walks a CTA's segments (begin, then next until it is false).  Any number of
// threads may each keep one.
template <int ROWS, int BLOCK, bool CUT>
struct SegmentWalk {
    int64_t at, hi;
    Segment u;            // the unit that `at` falls into (b0, nb unused)
    __device__ __forceinline__ void begin(const AttnParams &p, const Share &sh)
    {
        at = sh.lo;
        hi = sh.hi;
        if (at >= hi) return;
        u.r = sh.r;
        u.w = request_work<ROWS, BLOCK, CUT>(p, u.r);
        u.kvh = static_cast<int>((at - sh.before) / u.w.per_head);
        u.unit_first = sh.before + u.kvh * u.w.per_head;
        u.tile = 0;
        u.blocks = unit_blocks<ROWS, BLOCK, CUT>(p, u.w, 0);
        if (!CUT) {   // units of one size
            u.tile = static_cast<int>((at - u.unit_first) / u.blocks);
            u.unit_first += u.tile * u.blocks;
        }
        while (at >= u.unit_first + u.blocks) step(p);
    }
    // To the unit that follows.
    __device__ __forceinline__ void step(const AttnParams &p)
    {
        u.unit_first += u.blocks;
        if (++u.tile == u.w.tiles) {
            u.tile = 0;
            if (++u.kvh == p.Hkv) {
                u.kvh = 0;
                do u.w = request_work<ROWS, BLOCK, CUT>(p, ++u.r);
                while (u.w.total == 0);
            }
        }
        u.blocks = unit_blocks<ROWS, BLOCK, CUT>(p, u.w, u.tile);
    }
    __device__ __forceinline__ bool next(const AttnParams &p, Segment &s)
    {
        if (at >= hi) return false;
        if (at >= u.unit_first + u.blocks) step(p);
        s = u;
        s.b0 = at - u.unit_first;
        s.nb = u.blocks - s.b0 < hi - at ? u.blocks - s.b0 : hi - at;
        at += s.nb;
        return true;
    }
};

// The CTA whose share holds block b of the list.
__device__ __forceinline__ int owner_of(int64_t b, const Share &sh)
{
    return static_cast<int>(((b + 1) * sh.g - 1) / sh.total);
}

// Which of the 32 places j0 .. j0 + 31 a row's token sees, as bits.  node: its
// index among the request's `nodes` new tokens; tree_row its mask, or NULL.
__device__ __forceinline__ uint32_t seen_places(const int32_t *tree_row, int tree_words, int node, int nodes,
                                                int64_t len, int64_t j0)
{
    const int64_t ctx = len - nodes;
    const int64_t left = len - j0;
    const uint32_t there = left >= 32 ? 0xffffffffu : (left <= 0 ? 0u : (1u << left) - 1u);
    const int64_t lo = j0 - ctx;   // the node at place j0; below zero: cached before
    if (lo <= -32) return there;
    uint32_t m;
    if (!tree_row) {
        const int64_t cnt = node + 1 - lo;   // places up to its own
        m = cnt >= 32 ? 0xffffffffu : (cnt <= 0 ? 0u : (1u << cnt) - 1u);
    } else if (lo < 0) {
        const int k = static_cast<int>(-lo);
        m = (static_cast<uint32_t>(tree_row[0]) << k) | ((1u << k) - 1u);
    } else {
        const int64_t w = lo >> 5;
        const uint32_t a = w < tree_words ? static_cast<uint32_t>(tree_row[w]) : 0u;
        const uint32_t b = w + 1 < tree_words ? static_cast<uint32_t>(tree_row[w + 1]) : 0u;
        m = __funnelshift_r(a, b, static_cast<uint32_t>(lo & 31));
    }
    return m & there;
}

// Bounded wait that also gives up when another role of the CTA has.
__device__ __forceinline__ bool wait_or_give_up(uint64_t *bar, uint32_t parity, volatile int *gave_up, int *status)
{
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = global_timer_ns();
    while (true) {
        if (mbar_try_wait_sleep(bar, parity, kSuspendHintNs)) return true;
        if (*gave_up) return false;
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            *gave_up = 1;
            atomicOr(status, kDevTimeout);
            return false;
        }
    }
}

// The same for a whole warp: every lane calls it and gets the same answer.
__device__ __forceinline__ bool warp_wait_or_give_up(uint64_t *bar, uint32_t parity, volatile int *gave_up, int *status)
{
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    bool ok = true;
    if ((threadIdx.x & 31) == 0) ok = wait_or_give_up(bar, parity, gave_up, status);
    ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
    if (ok)   // the phase has completed: every lane observes it before going on
        while (!mbar_try_wait(bar, parity)) {
        }
    return ok;
}

// 2^x (the hardware's approximation; 2^-inf = 0).
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Workspace: a counter to each CTA of the grid, then for each CTA two places
// for partial results (a unit it finishes for others, and one it begins).
// A place: m[ROWS], l[ROWS], o[ROWS][D], fp32.
constexpr int kMaxGrid = 4096;
__host__ __device__ constexpr int64_t partial_floats(int rows, int D) { return static_cast<int64_t>(rows) * (D + 2); }

__device__ __forceinline__ int *workspace_counters(const AttnParams &p) { return static_cast<int *>(p.workspace); }
__device__ __forceinline__ float *workspace_partial(const AttnParams &p, int cta, int which, int rows, int D)
{
    return reinterpret_cast<float *>(static_cast<int *>(p.workspace) + kMaxGrid) +
           (2 * static_cast<int64_t>(cta) + which) * partial_floats(rows, D);
}

// The output row of row `row` of a segment's unit.
template <int ROWS, int D>
__device__ __forceinline__ __half *out_row(const AttnParams &p, const Segment &s, int row)
{
    const int64_t rho = static_cast<int64_t>(s.tile) * ROWS + row;
    const int64_t token = rho / p.group;
    const int head = s.kvh * p.group + static_cast<int>(rho - token * p.group);
    const int64_t first = p.start[s.r] < 0 ? 0 : p.start[s.r];
    return p.out + ((first + token) * p.Hq + head) * D;
}

__device__ __forceinline__ void store_half8(__half *dst, const float (&v)[8])
{
    uint4 w;
    w.x = float2_to_half2_bits(make_float2(v[0], v[1]));
    w.y = float2_to_half2_bits(make_float2(v[2], v[3]));
    w.z = float2_to_half2_bits(make_float2(v[4], v[5]));
    w.w = float2_to_half2_bits(make_float2(v[6], v[7]));
    *reinterpret_cast<uint4 *>(dst) = w;
}

// Joins a unit of `rows` valid rows whose parts are in the workspace: called by
// the THREADS threads (tid 0 ..) of the CTA that finished last, which has seen
// the others' parts published.  Part i lies with CTA first + i; the first one
// in its second place, the others in their first.
template <int ROWS, int D, int THREADS>
__device__ __forceinline__ void join_parts(const AttnParams &p, const Segment &s, int first, int parts, int rows, int tid)
{
    constexpr int CH = D / 8;   // 8 values to a thread at a time
    for (int i = tid; i < rows * CH; i += THREADS) {
        const int row = i / CH, d = (i - row * CH) * 8;
        float m = -INFINITY;
        for (int c = 0; c < parts; ++c)
            m = fmaxf(m, __ldcg(workspace_partial(p, first + c, c == 0, ROWS, D) + row));
        const float mm = m == -INFINITY ? 0.0f : m;
        float l = 0.0f, o[8] = {};
#pragma unroll 4
        for (int c = 0; c < parts; ++c) {
            const float *part = workspace_partial(p, first + c, c == 0, ROWS, D);
            const float f = exp2_fast(__ldcg(part + row) - mm);
            l += __ldcg(part + ROWS + row) * f;
            const float4 a = __ldcg(reinterpret_cast<const float4 *>(part + 2 * ROWS + row * D + d));
            const float4 b = __ldcg(reinterpret_cast<const float4 *>(part + 2 * ROWS + row * D + d + 4));
            if (f > 0.0f) {   // a part whose rows saw nothing adds nothing
                o[0] += a.x * f; o[1] += a.y * f; o[2] += a.z * f; o[3] += a.w * f;
                o[4] += b.x * f; o[5] += b.y * f; o[6] += b.z * f; o[7] += b.w * f;
            }
        }
        const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = l == l ? o[k] * inv : l;
        store_half8(out_row<ROWS, D>(p, s, row) + d, o);
    }
}

// Tensor copy of one box of cached rows: x the first column, y the row within
// the page, z the page.
__device__ __forceinline__ void copy_box(void *dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// Tensor map of a cache's rows: [n_pages][Hkv * page][D], boxes of `rows` rows
// and up to 128 bytes, swizzled over that width.  False where the driver has
// no such call or refuses the shape.
bool encode_rows(CUtensorMap *map, const AttnParams &p, const void *base, int D, int kind, int rows);

// The two kernels' launches (qmv_attn_rows.cu, qmv_attn_tiles.cu) and the
// workspace each needs.
cudaError_t launch_attn_rows(const AttnParams &p, int D, int kind, int sms, cudaStream_t s, bool pdl);
cudaError_t launch_attn_tiles(const AttnParams &p, int D, int kind, int sms, cudaStream_t s, bool pdl);
int64_t attn_rows_workspace_floats(int sms);
int64_t attn_tiles_workspace_floats(int sms);

}  // namespace qmv
