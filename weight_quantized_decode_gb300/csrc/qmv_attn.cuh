// qmv_attn.cuh -- what the attention kernels over the paged cache share: the
// split of the work over the CTAs of a persistent grid, the mask of a row, and
// the join of partial results.
//
// A unit is one (request, key/value head, tile of ROWS query rows); a row is
// one (new token, query head of the group).  Its places are cut into blocks of
// BLOCK.  All units' blocks, in order, are one long list, and CTA c of g takes
// entries [c B / g, (c + 1) B / g): the same share for each, however uneven the
// requests are, with no plan made on the host.  A unit begins with COST entries
// that stand for no block but for what a CTA spends on a unit besides its
// blocks (queries, start and end of the pipeline).  A CTA's share is a run of
// segments, each a range of one unit's blocks.  A CTA writes its part of a unit
// that several CTAs share (its rows' running maximum, sum and unnormalised
// output, fp32) to its own place of the workspace, and a second kernel adds a
// unit's parts, in CTA order: the sum is the same on every run.  (Joined by the
// last CTA to finish instead, 38 parts of 32 rows took 40 us, in two levels of
// eight 14 us, each CTA reading alone; one tree of 8 nodes over 30001 places,
// whose keys and values take 18 us.)
#pragma once

#include <cuda.h>

#include <cstdint>

#include "qmv_common.cuh"
#include "qmv_kv.h"
#include "qmv_launch.h"

namespace qmv {

// How each kernel cuts its work: rows of a unit (for few rows: 8, 16 or 32), places of a
// block, and what a unit costs besides its blocks, in blocks (tiles: 3 .. 6 measured
// within 3 %).  Stated here for the kernels and for the check of the split alike.
struct RowsSplit {
    static constexpr int kBlock = 128, kCost = 2;
};
struct TilesSplit {
    static constexpr int kRows = 256, kBlock = 128, kCost = 5;
};

// a / b for a, b >= 0, in 32 bits where they fit (a 64-bit division is a long
// sequence of dependent instructions).
__host__ __device__ __forceinline__ int64_t quotient(int64_t a, int64_t b)
{
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// Request r's share of the work.
struct RequestWork {
    int nodes;         // new tokens
    int tiles;         // row tiles
    int64_t len;       // places
    bool bad;          // a length the cache cannot have: one block that gives NaN
    int64_t per_head;  // entries of the units of one key/value head
    int64_t total;     // entries of all its units
};

// Entries of the unit of row tile `tile`: COST and its blocks.  CUT: the rows of a chain see nothing
// past the tile's last token, and the blocks there are left out.
template <int ROWS, int BLOCK, int COST, bool CUT>
__host__ __device__ __forceinline__ int64_t unit_entries(const AttnParams &p, const RequestWork &w, int tile)
{
    if (w.bad) return COST + 1;
    int64_t places = w.len;
    if (CUT && !p.tree) {
        const uint32_t last = ((static_cast<uint32_t>(tile) + 1) * ROWS - 1) / static_cast<uint32_t>(p.group);   // the tile's last token
        if (last < static_cast<uint32_t>(w.nodes)) places = w.len - w.nodes + last + 1;
    }
    return COST + (places + BLOCK - 1) / BLOCK;
}

template <int ROWS, int BLOCK, int COST, bool CUT>
__host__ __device__ __forceinline__ RequestWork request_work(const AttnParams &p, int64_t r)
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
    if (CUT && !p.tree && !w.bad) {
        // the tiles' last tokens, ((t + 1) * ROWS - 1) / group, without the divisions
        const uint32_t group = static_cast<uint32_t>(p.group), by = ROWS / group, over = ROWS % group;
        uint32_t last = (ROWS - 1) / group, rest = (ROWS - 1) % group;
        const int64_t ctx = w.len - w.nodes;
        w.per_head = 0;
        for (int t = 0; t < w.tiles; ++t) {
            const int64_t places = ctx + (last < static_cast<uint32_t>(w.nodes) ? last + 1 : w.nodes);
            w.per_head += COST + static_cast<int64_t>(static_cast<uint64_t>(places + BLOCK - 1) / BLOCK);
            last += by;
            rest += over;
            if (rest >= group) {
                rest -= group;
                ++last;
            }
        }
    } else {
        w.per_head = w.tiles * unit_entries<ROWS, BLOCK, COST, CUT>(p, w, 0);
    }
    w.total = w.per_head * p.Hkv;
    return w;
}

// Where a CTA's share begins, in shared memory (find_share).
struct Share {
    int64_t lo, hi;      // entries [lo, hi) of the list
    int64_t total;       // all entries
    int64_t r;           // the request entry lo falls into
    int64_t before;      // entries of the requests before it
    RequestWork w;       // that request's work
    int g;               // CTAs that have a share
    int64_t sums[32];
};

// CTA `cta`'s entries [lo, hi) of `total`, on a grid of which g CTAs have some.
__host__ __device__ __forceinline__ void share_of(int64_t total, int grid, int cta, int *g, int64_t *lo, int64_t *hi)
{
    *g = total < grid ? static_cast<int>(total) : grid;
    *lo = cta < *g ? quotient(total * cta, *g) : 0;
    *hi = cta < *g ? quotient(total * (cta + 1), *g) : 0;
}

// Every thread of the block calls this (THREADS of them, a multiple of 32).
// With up to THREADS requests each thread looks at one, once.
template <int ROWS, int BLOCK, int COST, bool CUT, int THREADS>
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
        if (lane == 31) sh->sums[warp] = v;
        __syncthreads();
        int64_t add = 0, sum = 0;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if (i < warp) add += sh->sums[i];
            sum += sh->sums[i];
        }
        __syncthreads();
        *all = sum;
        return v + add;
    };
    RequestWork w;
    w.total = 0;
    if (tid < p.R) w = request_work<ROWS, BLOCK, COST, CUT>(p, tid);
    int64_t total = 0;
    int64_t upto = scan(w.total, &total);          // of the first THREADS requests
    const int64_t chunk0 = total;
    if (p.R > THREADS) {
        int64_t more = 0, rest = 0;
        for (int64_t r = THREADS + tid; r < p.R; r += THREADS) more += request_work<ROWS, BLOCK, COST, CUT>(p, r).total;
        scan(more, &rest);
        total += rest;
    }
    int g;
    int64_t lo, hi;
    share_of(total, gridDim.x, blockIdx.x, &g, &lo, &hi);
    const bool mine = lo < hi;
    if (tid == 0) {
        sh->lo = lo;
        sh->hi = hi;
        sh->total = total;
        sh->g = g;
    }
    int64_t before = chunk0;
    for (int64_t r = tid;;) {
        if (w.total > 0 && upto - w.total <= lo && lo < upto && mine) {
            sh->r = r;
            sh->before = upto - w.total;
            sh->w = w;
        }
        r += THREADS;
        if (r - tid >= p.R || before > lo || !mine) break;
        w.total = 0;
        if (r < p.R) w = request_work<ROWS, BLOCK, COST, CUT>(p, r);
        int64_t all = 0;
        upto = before + scan(w.total, &all);
        before += all;
    }
    __syncthreads();
}

// The CTA of g whose share holds entry e of the list's `total`.
__host__ __device__ __forceinline__ int owner_of(int64_t e, int g, int64_t total)
{
    return static_cast<int>(quotient((e + 1) * g - 1, total));
}

// A CTA's part of one unit.
struct Segment {
    int64_t r;            // request
    int kvh, tile;        // key/value head, row tile
    int64_t b0, nb;       // its blocks [b0, b0 + nb) of the unit
    bool whole;           // they are all
    int parts;            // CTAs that share the unit, if this one begins it; else 0
    int64_t entries;      // entries of the unit
    int64_t unit_first;   // the list's index of the first of them
    RequestWork w;
};

// Walks a CTA's segments (begin, then next until it is false).  Any number of
// threads may each keep one.
template <int ROWS, int BLOCK, int COST, bool CUT>
struct SegmentWalk {
    int64_t at, hi, total;
    int g, cta;
    Segment u;            // the unit that `at` falls into
    __host__ __device__ __forceinline__ void begin(const AttnParams &p, const Share &sh, int cta_)
    {
        cta = cta_;
        at = sh.lo;
        hi = sh.hi;
        total = sh.total;
        g = sh.g;
        if (at >= hi) return;
        u.r = sh.r;
        u.w = sh.w;
        u.kvh = static_cast<int>(quotient(at - sh.before, u.w.per_head));
        u.unit_first = sh.before + u.kvh * u.w.per_head;
        u.tile = 0;
        u.entries = unit_entries<ROWS, BLOCK, COST, CUT>(p, u.w, 0);
        if (!CUT) {   // units of one size
            u.tile = static_cast<int>(quotient(at - u.unit_first, u.entries));
            u.unit_first += u.tile * u.entries;
        }
        while (at >= u.unit_first + u.entries) step(p);
    }
    // To the unit that follows.
    __host__ __device__ __forceinline__ void step(const AttnParams &p)
    {
        u.unit_first += u.entries;
        if (++u.tile == u.w.tiles) {
            u.tile = 0;
            if (++u.kvh == p.Hkv) {
                u.kvh = 0;
                do u.w = request_work<ROWS, BLOCK, COST, CUT>(p, ++u.r);
                while (u.w.total == 0);
            }
        }
        u.entries = unit_entries<ROWS, BLOCK, COST, CUT>(p, u.w, u.tile);
    }
    __host__ __device__ __forceinline__ bool next(const AttnParams &p, Segment &s)
    {
        while (at < hi) {
            if (at >= u.unit_first + u.entries) step(p);
            const int64_t unit_end = u.unit_first + u.entries, end = unit_end < hi ? unit_end : hi;
            const int64_t from = at - u.unit_first - COST, to = end - u.unit_first - COST;
            at = end;
            if (to <= 0) continue;   // none of its blocks
            s = u;
            s.b0 = from > 0 ? from : 0;
            s.nb = to - s.b0;
            s.whole = s.nb == u.entries - COST;
            s.parts = 0;
            if (!s.whole && s.b0 == 0) s.parts = owner_of(unit_end - 1, g, total) - cta + 1;
            return true;
        }
        return false;
    }
};

// Which of the 32 places j0 .. j0 + 31 a row's token sees, as bits.  node: its
// index among the request's `nodes` new tokens; tree_row its mask, or NULL.
__host__ __device__ __forceinline__ uint32_t seen_places(const int32_t *tree_row, int tree_words, int node, int nodes,
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
        m = static_cast<uint32_t>((static_cast<uint64_t>(b) << 32 | a) >> (lo & 31));
    }
    return m & there;
}

// Bounded wait that also gives up when another role of the CTA has.
__device__ __forceinline__ bool wait_or_give_up(uint64_t *bar, uint32_t parity, volatile int *gave_up, int *status,
                                                unsigned long long limit_ns = kWaitLimitNs)
{
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = global_timer_ns();
    while (true) {
        if (mbar_try_wait_sleep(bar, parity, kSuspendHintNs)) return true;
        if (*gave_up) return false;
        if (global_timer_ns() - t0 > limit_ns) {
            *gave_up = 1;
            atomicOr(status, kDevTimeout);
            return false;
        }
    }
}

// The same for a whole warp: every lane calls it and gets the same answer.
__device__ __forceinline__ bool warp_wait_or_give_up(uint64_t *bar, uint32_t parity, volatile int *gave_up, int *status,
                                                     unsigned long long limit_ns = kWaitLimitNs)
{
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    bool ok = true;
    if ((threadIdx.x & 31) == 0) ok = wait_or_give_up(bar, parity, gave_up, status, limit_ns);
    ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
    if (ok)   // the phase has completed: every lane observes it before going on
        while (!mbar_try_wait(bar, parity)) {
        }
    return ok;
}

// Shared-memory accesses by 32-bit address: through a pointer whose memory the
// compiler cannot tell they would be generic ones, and several times as slow.
__device__ __forceinline__ float lds1(uint32_t at)
{
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ float4 lds4(uint32_t at)
{
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint4 lds4u(uint32_t at)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void sts4u(uint32_t at, uint4 v)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// 2^x (the hardware's approximation; 2^-inf = 0).
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The same, not below 2^-149.
__device__ __forceinline__ float exp2_least(float x)
{
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(fmaxf(x, -149.0f)));
    return y;
}

// Workspace: what each CTA of the grid leaves to join, then for each CTA two
// places for partial results (a unit it ends or passes on, and one it begins).
// A place: m[ROWS], l[ROWS], o[D / 4][ROWS][4], fp32 (neighbouring threads hold
// neighbouring rows or neighbouring columns: either way they write whole lines).
constexpr int kMaxGrid = 1024;

// The shared unit that a CTA begins (parts 0: none).
struct alignas(32) SharedUnit {
    int parts;          // CTAs that share it, this one first
    int valid;          // its rows
    int kvh, tile;
    int64_t first_row;  // its request's first token
    int64_t pad;
};
constexpr int64_t kUnitBytes = kMaxGrid * sizeof(SharedUnit);

__host__ __device__ constexpr int64_t partial_floats(int rows, int D) { return static_cast<int64_t>(rows) * (D + 2); }

__device__ __forceinline__ SharedUnit *workspace_units(const AttnParams &p) { return static_cast<SharedUnit *>(p.workspace); }
__device__ __forceinline__ float *workspace_partial(const AttnParams &p, int cta, int which, int rows, int D)
{
    return reinterpret_cast<float *>(static_cast<uint8_t *>(p.workspace) + kUnitBytes) +
           (2 * static_cast<int64_t>(cta) + which) * partial_floats(rows, D);
}

// The output row of row `row` of a unit.
template <int ROWS, int D>
__device__ __forceinline__ __half *out_row(const AttnParams &p, int64_t first_token, int kvh, int tile, int row)
{
    const uint32_t rho = static_cast<uint32_t>(tile) * ROWS + row;   // T * Hq fits 32 bits
    const uint32_t token = rho / static_cast<uint32_t>(p.group);
    const int head = kvh * p.group + static_cast<int>(rho - token * p.group);
    return p.out + ((first_token + token) * p.Hq + head) * D;
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

// Columns d .. d + 3 of row `row` in such a place.
template <int ROWS>
__device__ __forceinline__ float4 *part_columns(float *part, int row, int d)
{
    return reinterpret_cast<float4 *>(part + 2 * ROWS) + (d >> 2) * ROWS + row;
}

// Leaves word of the shared unit that segment s begins.
__device__ __forceinline__ void leave_unit(const AttnParams &p, const Segment &s, int valid, int64_t first_token)
{
    SharedUnit u;
    u.parts = s.parts;
    u.valid = valid;
    u.kvh = s.kvh;
    u.tile = s.tile;
    u.first_row = first_token;
    u.pad = 0;
    workspace_units(p)[blockIdx.x] = u;
}

// ---- the second kernel: adds the parts of shared units ----
//
// Block x looks at what CTAS CTAs of the first kernel left; block y takes every
// gridDim.y-th run of a unit's pieces (8 columns of a row each, rows next to
// each other).  A unit of up to four parts: each thread adds a piece.  More:
// the four warps take every fourth part of the same 32 pieces, and their sums
// are added in shared memory.  Eight parts' loads are in flight at a time.
constexpr int kJoinThreads = 128;

template <int ROWS, int D, int CTAS>
__global__ void __launch_bounds__(kJoinThreads) join_units_kernel(const AttnParams p, int grid)
{
    constexpr int CH = D / 8;
    constexpr int kAhead = 8;
    __shared__ float sums[4][32][12];
    pdl_wait_prior_grid();
    pdl_allow_next_grid();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c0 = blockIdx.x * CTAS;
    const int mine = lane < CTAS && c0 + lane < grid ? __ldcg(&workspace_units(p)[c0 + lane].parts) : 0;
    for (uint32_t left = __ballot_sync(0xffffffffu, mine > 1); left; left &= left - 1u) {
        const int cta = c0 + __ffs(left) - 1;
        const SharedUnit u = workspace_units(p)[cta];
        const int pieces = u.valid * CH;
        const bool split = u.parts > 4;                  // a piece's parts over the warps
        const int run = split ? 32 : kJoinThreads, stride = split ? 4 : 1;
        for (int base = run * blockIdx.y; base < pieces; base += run * gridDim.y) {
            const int at = base + (split ? lane : static_cast<int>(threadIdx.x));
            const bool on = at < pieces;
            const int piece = on ? at : pieces - 1;
            const int chunk = piece / u.valid, row = piece - chunk * u.valid, d = 8 * chunk;
            float m = -INFINITY, l = 0.0f, o[8] = {};
            for (int k0 = split ? warp : 0; k0 < u.parts; k0 += stride * kAhead) {
                float mc[kAhead], lc[kAhead];
                float4 a[kAhead], b[kAhead];
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    mc[k] = -INFINITY;
                    lc[k] = 0.0f;
                    a[k] = b[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    const int part_no = k0 + stride * k;
                    if (part_no < u.parts) {
                        float *part = workspace_partial(p, cta + part_no, part_no == 0, ROWS, D);
                        mc[k] = __ldcg(part + row);
                        lc[k] = __ldcg(part + ROWS + row);
                        a[k] = __ldcg(part_columns<ROWS>(part, row, d));
                        b[k] = __ldcg(part_columns<ROWS>(part, row, d + 4));
                    }
                }
                float top = m;
#pragma unroll
                for (int k = 0; k < kAhead; ++k) top = fmaxf(top, mc[k]);
                const float tt = top == -INFINITY ? 0.0f : top;
                const float f0 = exp2_fast(m - tt);
                l *= f0;
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] *= f0;
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const float f = exp2_least(mc[k] - tt);
                    // A part whose rows saw nothing holds zeros (but a NaN sum says that the
                    // request cannot be read).  f is never 0, so that an infinity or NaN that
                    // a row saw shows in the output however small its weight; the condition
                    // keeps the loads together ahead of it (without it 0.6 us more a launch).
                    l += lc[k] != lc[k] ? lc[k] : lc[k] * f;
                    if (f > 0.0f) {
                        o[0] += a[k].x * f; o[1] += a[k].y * f; o[2] += a[k].z * f; o[3] += a[k].w * f;
                        o[4] += b[k].x * f; o[5] += b[k].y * f; o[6] += b[k].z * f; o[7] += b[k].w * f;
                    }
                }
                m = top;
            }
            if (split) {
                float *mine4 = sums[warp][lane];
                *reinterpret_cast<float2 *>(mine4) = make_float2(m, l);
                *reinterpret_cast<float4 *>(mine4 + 4) = make_float4(o[0], o[1], o[2], o[3]);
                *reinterpret_cast<float4 *>(mine4 + 8) = make_float4(o[4], o[5], o[6], o[7]);
                __syncthreads();
                if (warp == 0) {
                    float top = m;
#pragma unroll
                    for (int w = 1; w < 4; ++w) top = fmaxf(top, sums[w][lane][0]);
                    const float tt = top == -INFINITY ? 0.0f : top;
                    l = 0.0f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = 0.0f;
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const float *x = sums[w][lane];
                        const float f = exp2_fast(x[0] - tt);
                        l += x[1] != x[1] ? x[1] : x[1] * f;
#pragma unroll
                        for (int j = 0; j < 8; ++j) o[j] += x[4 + j] * f;
                    }
                }
                __syncthreads();
            }
            if (on && (!split || warp == 0)) {
                const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = l == l ? o[j] * inv : l;
                store_half8(out_row<ROWS, D>(p, u.first_row, u.kvh, u.tile, row) + d, o);
            }
        }
    }
}

// Launches it behind a kernel of `grid` CTAs, unless no unit can have had more
// than one block.
template <int ROWS, int D>
cudaError_t launch_join(const AttnParams &p, int grid, int block, cudaStream_t s, bool pdl)
{
    if ((p.width << p.page_shift) <= block) return cudaSuccess;
    // 32 rows: 16 runs of pieces; 256 rows: a block to each CTA, 16 runs of 256
    constexpr int kCtas = ROWS > 64 ? 1 : 2, kRuns = ROWS * D / 8 / 32 < 16 ? ROWS * D / 8 / 32 : 16;
    return launch_ex(join_units_kernel<ROWS, D, kCtas>, dim3((grid + kCtas - 1) / kCtas, kRuns), dim3(kJoinThreads), 0, s, pdl,
                     p, grid);
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
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
// rows: query rows that share a key/value head in the average request.
cudaError_t launch_attn_rows(const AttnParams &p, int D, int kind, int64_t rows, int sms, cudaStream_t s, bool pdl);
cudaError_t launch_attn_tiles(const AttnParams &p, int D, int kind, int sms, cudaStream_t s, bool pdl);
int64_t attn_rows_workspace_floats(int sms);
int64_t attn_tiles_workspace_floats(int sms);

}  // namespace qmv
