// qmv_sample.cu -- a token from each row of logits: temperature, top-k, top-p,
// min-p, and one given uniform number to a row.
#include <cooperative_groups.h>
#include <atomic>
#include <cstdint>

#include "../../include/qmv.h"
#include "qmv_common.cuh"
#include "qmv_kv.h"
#include "qmv_launch.h"
#include "qmv_sample.h"
#include "qmv_sample_plan.h"
#include "qmv_sample_weight.h"

namespace qmv {

namespace {

namespace cg = cooperative_groups;

// With w_i = exp((l_i - max l) / T) and the row's tokens in order of l, largest
// first, equal ones lowest index first:
//
//   K     the first top_k tokens
//   P     of K, the tokens before which less than top_p * sum_K w lies
//   kept  of P, the tokens with w >= min_p
//   token the lowest index i with sum_{j <= i, kept} w_j > u * sum_kept w
//
// K and P are prefixes of the order.  Such a prefix is held as a bound (key, index):
// the tokens with a larger key (the logit's bits, in the order of its value), and of
// those with the same key the ones up to the index.  No row is sorted.  A prefix is
// found from a histogram over 2048 steps of the distance to the largest logit; the
// tokens of the step it ends in are gathered and sorted by one CTA, or, where they are more
// than 1024 (equal logits), counted by the digits of their keys.  A small top-k needs no
// histogram of the logits: of the threads' own largest ones the k-th is a bound, and few
// tokens lie above it.  Weights are whole numbers (qmv_sample_weight.h), so sums are
// exact, and the same whatever their order.
//
// A cluster of up to 16 CTAs holds the row in shared memory, a slice to each: the
// logits are read once from memory, and what the steps exchange goes through
// distributed shared memory.  Many rows, or longer ones, are read from memory again
// instead, by clusters of one to eight (qmv_sample_plan.h has both sides measured).
//
// Where rows are many, latency that nothing overlaps and instructions share the time (512
// text-like rows of 128256, 39 us of bytes; in brackets the issue slots in use): greedy 59
// (0.28: waits for loads and barriers; 1024 CTAs on 304 places are 3.4 waves), top-k 50 84
// (0.35), unfiltered 135 (0.58: a token's weight takes 30 instructions), top-p 0.9 323
// (0.65: the row is passed over three times).  Where they are few, a chain of latencies:
// one row with top-k and top-p 11 us, of which the logits' way into shared memory is 1.6
// and each of six barriers of the cluster 0.5 to 1; eight rows with top-p 28 us (barriers
// 6, histogram 2.5, the bin it gives 2.5, weights 6, sorting 350 tokens 3, loads 1.6; the
// rest is in none of these), and 39 where its instructions have to be fetched first.
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kAhead = 8;         // 16-byte loads that a thread has under way as a slice is first read
constexpr int kMany = 2;          // and as it is read again from memory
constexpr int kGather = 2 * kThreads;   // tokens that one CTA sorts
constexpr int kGatherTopK = kThreads;   // the largest top-k that is taken from a gathered list

struct Find {
    uint32_t bin;
    uint64_t before, inside;   // weight before the bin, and in it
    uint64_t target;
};

// (the slice lies behind it, read 16 bytes at a time)
struct alignas(16) Shared {
    WeightStep table[kWeightTable];
    union {
        struct {
            uint32_t lo[kBins], hi[kBins];   // a histogram's sums, in halves: 64-bit additions to shared memory are loops
        };
        uint64_t sorted[kGather];            // gathered tokens: inverted key above the index
    };
    uint64_t warp_sum[kWarps];
    unsigned long long run_sum[kWarps];   // of the runs that the warps draw from
    uint64_t total, above;                // this CTA's shares of sums
    Find found;
    float top, low;
    uint32_t gathered, first, bound_key, bound_index;
    uint32_t listed;                      // threads of this CTA that have ...
    uint16_t threads[kThreads];           // ... a token of the gathered ones
};
static_assert(sizeof(Shared) % 16 == 0 && sizeof(Shared) <= kSampleShared, "the slice's alignment, and room for it");

// The logit's bits in the order of its value (both zeros alike).
__device__ __forceinline__ uint32_t key_of(float l)
{
    const uint32_t b = __float_as_uint(l == 0.0f ? 0.0f : l);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float logit_of(uint32_t key)
{
    return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// The larger one; NaN if there is one.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// A CTA's slice of a row, in places: place j holds token base + j, where there is one.  The places begin on a 16-byte
// boundary of the row in memory, so the first slice has up to 15 bytes of places before its first token.
struct Row {
    const float *v;            // the slice in shared memory (-inf in places without a token), or null:
    const unsigned char *x;    // in memory, place 0 (not read where there is no token)
    int places, base, V;
    WeightRow w;
    float steps;          // histogram steps to an octave of weight
    bool bound;           // whether there is a prefix: logits above ...
    float last;           // ... this one, and this one
    uint32_t upto;        // up to this index
};

__device__ __forceinline__ bool in_prefix(const Row &row, float l, int j)
{
    return !row.bound || l > row.last || (l == row.last && static_cast<uint32_t>(row.base + j) <= row.upto);
}

// Logits of places j .. j + VEC - 1, j a multiple of VEC, from memory; `none` in places without a token.
template <bool F32, int VEC>
__device__ __forceinline__ void read_places(const Row &row, int j, float none, float (&f)[VEC])
{
    static_assert(VEC == (F32 ? 4 : 8), "16 bytes");
    const int i = row.base + j;
    if (i >= 0 && i + VEC <= row.V) {
        const uint4 x = reinterpret_cast<const uint4 *>(row.x)[j / VEC];
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (F32) {
                f[k] = __uint_as_float(w[k]);
            } else {
                f[2 * k] = half_lo_to_float(w[k]);
                f[2 * k + 1] = half_hi_to_float(w[k]);
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            f[k] = none;
            if (i + k >= 0 && i + k < row.V) {
                if constexpr (F32)
                    f[k] = reinterpret_cast<const float *>(row.x)[j + k];
                else
                    f[k] = __half2float(reinterpret_cast<const __half *>(row.x)[j + k]);
            }
        }
    }
}

constexpr float kNone = -__builtin_inff();

template <bool F32, bool SMEM>
__device__ __forceinline__ float read_place(const Row &row, int j)
{
    if constexpr (SMEM) return row.v[j];
    const int i = row.base + j;
    if (i < 0 || i >= row.V) return kNone;
    return F32 ? reinterpret_cast<const float *>(row.x)[j] : __half2float(reinterpret_cast<const __half *>(row.x)[j]);
}

// Calls f(logits, first place) for places lo .. hi - 1 (lo a multiple of 32), STRIDE / 32 warps wide, this thread the
// `lane`-th: four logits (from memory in fp16: eight) at a time, kMany such reads under way.  Every lane of a
// warp makes the same number of calls; past hi a place has no token.
template <bool F32, bool SMEM, int STRIDE, typename F>
__device__ __forceinline__ void each(const Row &row, int lo, int hi, int lane, F f)
{
    constexpr int VEC = SMEM || F32 ? 4 : 8, MANY = SMEM ? 2 : F32 ? kMany : kMany / 2;
    for (int j0 = lo + (lane & ~31) * VEC; j0 < hi; j0 += MANY * STRIDE * VEC) {
        float l[MANY][VEC];
#pragma unroll
        for (int m = 0; m < MANY; ++m) {
            const int j = j0 + (m * STRIDE + (lane & 31)) * VEC;
            if (j + VEC <= hi) {
                if constexpr (SMEM) {
                    const float4 x = *reinterpret_cast<const float4 *>(row.v + j);
                    l[m][0] = x.x; l[m][1] = x.y; l[m][2] = x.z; l[m][3] = x.w;
                } else {
                    read_places<F32>(row, j, kNone, l[m]);
                }
            } else {
#pragma unroll
                for (int k = 0; k < VEC; ++k) l[m][k] = j + k < hi ? read_place<F32, SMEM>(row, j + k) : kNone;
            }
        }
#pragma unroll
        for (int m = 0; m < MANY; ++m) f(l[m], j0 + (m * STRIDE + (lane & 31)) * VEC);
    }
}

__device__ __forceinline__ int step_of(const Row &row, float t)
{
    return static_cast<int>(fmaxf(fminf(t * row.steps, kBins - 1.0f), 0.0f));
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t x)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

__device__ __forceinline__ uint64_t warp_scan(uint64_t x)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    return x;
}

// Sums of `mine` over the block's threads before this one, and over all.
__device__ __forceinline__ uint64_t block_scan(Shared &s, uint64_t mine, uint64_t *all)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint64_t upto = warp_scan(mine);
    __syncthreads();
    if (lane == 31) s.warp_sum[warp] = upto;
    __syncthreads();
    const uint64_t sums = warp_scan(lane < kWarps ? s.warp_sum[lane] : 0);
    *all = __shfl_sync(0xffffffffu, sums, 31);
    const uint64_t before = __shfl_sync(0xffffffffu, sums, warp > 0 ? warp - 1 : 0);
    return upto - mine + (warp > 0 ? before : 0);
}

// A share of each CTA, summed: those of the ranks before this one, and of all.
__device__ __forceinline__ uint64_t cluster_scan(Shared &s, cg::cluster_group &c, uint64_t mine, uint64_t *all)
{
    const int ranks = c.num_blocks(), rank = c.block_rank(), lane = threadIdx.x & 31;
    if (ranks == 1) {
        *all = mine;
        return 0;
    }
    if (threadIdx.x == 0) s.total = mine;
    c.sync();
    const uint64_t x = lane < ranks ? *c.map_shared_rank(&s.total, lane) : 0;
    *all = warp_sum(x);
    return warp_sum(lane < rank ? x : 0);
}

// x * 2^64 for 0 <= x < 1, what is below 2^-64 cut off.  (Products with sums are made of
// these: a double's multiplication is exact enough too, but this GPU makes two a cycle on an SM.)
__device__ __forceinline__ uint64_t fraction(float x)
{
    const uint32_t b = __float_as_uint(x) & 0x7fffffffu;   // (-0 is 0)
    const int e = static_cast<int>(b >> 23) - 127;         // of a normal number, -1 at most
    const uint64_t m = (b & 0x7fffffu) | 0x800000u;
    return e < -64 ? 0 : e >= -41 ? m << (41 + e) : m >> (-41 - e);
}

__device__ __forceinline__ uint64_t share_down(uint64_t sum, uint64_t share) { return __umul64hi(sum, share); }

__device__ __forceinline__ uint64_t share_up(uint64_t sum, uint64_t share)
{
    return __umul64hi(sum, share) + (sum * share != 0 ? 1 : 0);
}

// Begins a histogram, and a list (which is gathered after the histogram has been used: they share their memory).
__device__ __forceinline__ void clear_bins(Shared &s)
{
    for (int i = threadIdx.x; i < kBins; i += kThreads) s.lo[i] = s.hi[i] = 0;
    if (threadIdx.x == 0) s.gathered = s.listed = 0;
    __syncthreads();
}

// Adds w to a bin of this CTA's histogram.  (64-bit additions to shared memory are loops of compare and swap.)
__device__ __forceinline__ void add_to_bin(Shared &s, int bin, uint64_t w)
{
    const uint32_t low = static_cast<uint32_t>(w);
    const uint32_t old = atomicAdd(&s.lo[bin], low);
    const uint32_t up = static_cast<uint32_t>(w >> 32) + (old + low < low ? 1u : 0u);
    if (up) atomicAdd(&s.hi[bin], up);
}

// From the CTAs' histograms: the bin in which the sum over bins reaches `target`, at
// least 1 (0: `share` of the whole sum, rounded up).  False where the whole sum does not.  each(b): what the sum in bin b
// is multiplied by.
// COUNTS: the sums are below 2^32.
template <bool COUNTS, typename Each>
__device__ bool find_bin(Shared &s, cg::cluster_group &c, uint64_t target, uint64_t share, Find *found, Each each)
{
    const int ranks = c.num_blocks(), rank = c.block_rank(), per = kBins / ranks;
    c.sync();   // every CTA's histogram is complete
    // This CTA's share of the bins, `run` neighbouring ones to a thread.  No other CTA reads these of this
    // CTA's own histogram, so that their sums go there.
    const int run = per > kThreads ? per / kThreads : 1;
    const bool has = static_cast<int>(threadIdx.x) * run < per;
    uint64_t mine = 0;
    for (int i = 0; i < run && has; ++i) {
        const int b = rank * per + threadIdx.x * run + i;
        uint64_t sum = 0;
        // (eight other CTAs' sums under way at a time)
        for (int k0 = 0; k0 < ranks; k0 += 8) {
            uint32_t lo[8], hi[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const Shared *of = c.map_shared_rank(&s, k0 + k < ranks ? k0 + k : rank);
                lo[k] = of->lo[b];
                hi[k] = COUNTS ? 0u : of->hi[b];
            }
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k0 + k < ranks) sum += (static_cast<uint64_t>(hi[k]) << 32) + lo[k];
        }
        sum *= each(b);
        s.lo[b] = static_cast<uint32_t>(sum);
        s.hi[b] = static_cast<uint32_t>(sum >> 32);
        mine += sum;
    }
    uint64_t in_cta, whole;
    uint64_t before = block_scan(s, mine, &in_cta);
    before += cluster_scan(s, c, in_cta, &whole);
    if (target == 0) {
        target = share_up(whole, share);
        if (target == 0) target = 1;
    }
    if (whole < target) {
        c.sync();   // (every CTA has read the shares)
        return false;
    }
    if (has && before < target && target <= before + mine) {
        for (int i = 0; i < run; ++i) {
            const int b = rank * per + threadIdx.x * run + i;
            const uint64_t w = static_cast<uint64_t>(s.hi[b]) << 32 | s.lo[b];
            if (target <= before + w) {
                // the answer goes to every CTA
                const Find f = {static_cast<uint32_t>(b), before, w, target};
                for (int k = 0; k < ranks; ++k) c.map_shared_rank(&s, k)->found = f;
                break;
            }
            before += w;
        }
    }
    c.sync();
    *found = s.found;
    return true;
}

// Appends the tokens of a warp's logits l[k], places j + k, whose bit is set in `which`, to the list of the first CTA;
// past kGather they are only counted.  The list is complete after a cluster barrier.
template <int N>
__device__ __forceinline__ void append(Shared *to, const Row &row, const float (&l)[N], int j, uint32_t which)
{
    const int lane = threadIdx.x & 31;
    if (!__any_sync(0xffffffffu, which != 0)) return;
    int before = __popc(which);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, before, d);
        if (lane >= d) before += o;
    }
    uint32_t at = 0;
    if (lane == 31) at = atomicAdd(&to->gathered, static_cast<uint32_t>(before));
    at = __shfl_sync(0xffffffffu, at, 31) + before - __popc(which);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if (which >> k & 1) {
            if (at < kGather)
                to->sorted[at] = static_cast<uint64_t>(~key_of(l[k])) << 32 | static_cast<uint32_t>(row.base + j + k);
            ++at;
        }
    }
}

// Gathers this row's tokens for which `wanted(l, j)` holds in the first CTA.  Returns their number; where
// that is above kGather, the list is not complete.
template <bool F32, bool SMEM, typename Wanted>
__device__ uint32_t gather(Shared &s, cg::cluster_group &c, const Row &row, Wanted wanted)
{
    Shared *to = c.map_shared_rank(&s, 0);
    each<F32, SMEM, kThreads>(row, 0, row.places, threadIdx.x, [&](const auto &l, int j) {
        uint32_t which = 0;
#pragma unroll
        for (int k = 0; k < sizeof(l) / sizeof(float); ++k) which |= wanted(l[k], j + k) ? 1u << k : 0u;
        append(to, row, l, j, which);
    });
    c.sync();
    const uint32_t n = to->gathered;
    if (n > kGather) c.sync();   // (its number is not cleared before all have it)
    return n;
}

// Gathers the tokens with weight whose distance times row.steps is below `to`, given this thread's largest logit: only the
// threads that have one are looked at, a warp to each, a lane to each of its reads (512 rows of 128256 with top-k 50: 109 us
// by a pass over the row, 84 so).
template <bool F32, bool SMEM>
__device__ uint32_t gather_below(Shared &s, cg::cluster_group &c, const Row &row, float mine, float to)
{
    constexpr int VEC = F32 ? 4 : 8;   // as first_read reads
    Shared *const first = c.map_shared_rank(&s, 0);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const auto wanted = [&](float l) {
        const float t = weight_distance(l, row.w);
        return t < kWeightEnd && t * row.steps < to;
    };
    const bool has = wanted(mine);
    const uint32_t who = __ballot_sync(0xffffffffu, has);
    uint32_t at = 0;
    if (lane == 0 && who) at = atomicAdd(&s.listed, static_cast<uint32_t>(__popc(who)));
    at = __shfl_sync(0xffffffffu, at, 0) + __popc(who & ((1u << lane) - 1u));
    if (has) s.threads[at] = static_cast<uint16_t>(threadIdx.x);
    __syncthreads();
    const int listed = s.listed;
    for (int i = warp; i < listed; i += kWarps) {
        for (int j0 = s.threads[i] * VEC; j0 < row.places; j0 += 32 * kThreads * VEC) {
            const int j = j0 + lane * kThreads * VEC;
            float l[VEC];
            uint32_t which = 0;
            if (j < row.places) {
                if constexpr (SMEM) {
#pragma unroll
                    for (int k = 0; k < VEC; ++k) l[k] = row.v[j + k];
                } else {
                    read_places<F32>(row, j, kNone, l);
                }
#pragma unroll
                for (int k = 0; k < VEC; ++k) which |= wanted(l[k]) ? 1u << k : 0u;
            }
            append(first, row, l, j, which);
        }
    }
    c.sync();
    const uint32_t n = first->gathered;
    if (n > kGather) c.sync();   // (its number is not cleared before all have it)
    return n;
}

template <bool COUNTS>
__device__ __forceinline__ bool find_bin(Shared &s, cg::cluster_group &c, uint64_t target, uint64_t share, Find *found)
{
    return find_bin<COUNTS>(s, c, target, share, found, [](int) { return uint64_t(1); });
}

// Bitonic steps of 32 and fewer on 64 neighbouring tokens, lane l those at first + l and first + l + 32.
__device__ __forceinline__ void merge_in_warp(uint64_t &x, uint64_t &y, int first, int k, int from)
{
    const int lane = threadIdx.x & 31;
    const bool up_x = ((first + lane) & k) == 0, up_y = ((first + lane + 32) & k) == 0;
    if (from == 32) {
        if ((x > y) == up_x) {
            const uint64_t t = x;
            x = y;
            y = t;
        }
        from = 16;
    }
    for (int d = from; d; d >>= 1) {
        const bool lower = (lane & d) == 0;
        const uint64_t ox = __shfl_xor_sync(0xffffffffu, x, d), oy = __shfl_xor_sync(0xffffffffu, y, d);
        x = (lower == up_x) == (ox < x) ? ox : x;
        y = (lower == up_y) == (oy < y) ? oy : y;
    }
}

// Sorts the n gathered tokens of this CTA into the row's order: bitonic, by 64 in a warp's registers, the steps between
// warps in shared memory.
__device__ void sort_gathered(Shared &s, int n)
{
    const int lane = threadIdx.x & 31, first = (threadIdx.x >> 5) * 64;
    int size = 64;
    while (size < n) size *= 2;
    uint64_t x = 0, y = 0;
    __syncthreads();
    if (first < size) {
        x = first + lane < n ? s.sorted[first + lane] : ~uint64_t(0);
        y = first + lane + 32 < n ? s.sorted[first + lane + 32] : ~uint64_t(0);
        for (int k = 2; k <= 64; k *= 2) merge_in_warp(x, y, first, k, k / 2);
        s.sorted[first + lane] = x;
        s.sorted[first + lane + 32] = y;
    }
    __syncthreads();
    for (int k = 128; k <= size; k *= 2) {
        for (int d = k / 2; d > 32; d /= 2) {
            const int i = threadIdx.x, a = 2 * i - (i & (d - 1)), b = a + d;
            if (i < size / 2) {
                const uint64_t p = s.sorted[a], q = s.sorted[b];
                if ((p > q) == ((a & k) == 0)) {
                    s.sorted[a] = q;
                    s.sorted[b] = p;
                }
            }
            __syncthreads();
        }
        if (first < size) {
            x = s.sorted[first + lane];
            y = s.sorted[first + lane + 32];
            merge_in_warp(x, y, first, k, 32);
            s.sorted[first + lane] = x;
            s.sorted[first + lane + 32] = y;
        }
        __syncthreads();
    }
}

__device__ __forceinline__ uint64_t weight_of_key(Shared &s, const Row &row, uint32_t key)
{
    return weight_of(logit_of(key), row.w, s.table);
}

// Adds the prefix's tokens that have weight to the bins of their steps (COUNT: one to each, else their weights).
template <bool F32, bool SMEM, bool COUNT>
__device__ __forceinline__ void add_all(Shared &s, const Row &row)
{
    each<F32, SMEM, kThreads>(row, 0, row.places, threadIdx.x, [&](const auto &l, int j) {
#pragma unroll
        for (int k = 0; k < sizeof(l) / sizeof(float); ++k) {
            const float t = weight_distance(l[k], row.w);
            const bool in = t < kWeightEnd && in_prefix(row, l[k], j + k);
            const int step = step_of(row, t);
            if constexpr (COUNT) {
                if (in) atomicAdd(&s.lo[step], 1u);
            } else {
                if (in) add_to_bin(s, step, weight_of(l[k], row.w, s.table));
            }
        }
    });
}

// This thread's two of the first CTA's n sorted tokens, which begin behind a weight of `before`: whether the sum
// reaches `target` among them, and then the token that it does so at.
template <bool COUNT>
__device__ __forceinline__ bool last_of(Shared &s, const Row &row, uint32_t n, uint64_t before, uint64_t target, uint64_t *last)
{
    const uint32_t a = 2 * threadIdx.x;
    const uint64_t t0 = a < n ? s.sorted[a] : 0, t1 = a + 1 < n ? s.sorted[a + 1] : 0;
    const uint64_t w0 = a >= n ? 0 : COUNT ? 1 : weight_of_key(s, row, ~static_cast<uint32_t>(t0 >> 32));
    const uint64_t w1 = a + 1 >= n ? 0 : COUNT ? 1 : weight_of_key(s, row, ~static_cast<uint32_t>(t1 >> 32));
    uint64_t all;
    before += block_scan(s, w0 + w1, &all);
    *last = target <= before + w0 ? t0 : t1;
    return before < target && target <= before + w0 + w1;
}

__device__ __forceinline__ void tell_bound(Shared &s, cg::cluster_group &c, uint64_t last)
{
    for (unsigned k = 0; k < c.num_blocks(); ++k) {
        Shared *to = c.map_shared_rank(&s, k);
        to->bound_key = ~static_cast<uint32_t>(last >> 32);
        to->bound_index = static_cast<uint32_t>(last);
    }
}

__device__ __forceinline__ void take_bound(Shared &s, Row &row)
{
    row.last = logit_of(s.bound_key);
    row.upto = s.bound_index;
    row.bound = true;
}

// Narrows the prefix to the shortest one of weight `target` (0: `share` of the whole).
// COUNT: every token weighs 1.
template <bool F32, bool SMEM, bool COUNT>
__device__ void narrow(Shared &s, cg::cluster_group &c, Row &row, uint64_t target, uint64_t share)
{
    clear_bins(s);
    add_all<F32, SMEM, COUNT>(s, row);
    Find f;
    if (!find_bin<COUNT>(s, c, target, share, &f)) return;   // (more tokens than have weight)
    const int step = f.bin;
    target = f.target - f.before;
    // (step_of(t) == step, without the conversion)
    const float from = step == 0 ? kNone : static_cast<float>(step), to = step == kBins - 1 ? -kNone : step + 1.0f;
    const auto in_step = [&](float l, int j) {
        const float t = weight_distance(l, row.w), at = t * row.steps;
        return at >= from && at < to && t < kWeightEnd && in_prefix(row, l, j);
    };
    const uint32_t n = gather<F32, SMEM>(s, c, row, in_step);
    if (n <= kGather) {
        if (c.block_rank() == 0) {
            sort_gathered(s, n);
            uint64_t last;
            if (last_of<COUNT>(s, row, n, 0, target, &last)) tell_bound(s, c, last);
        }
        c.sync();
        take_bound(s, row);
        return;
    }
    // Many tokens of nearly one logit: three digits of their keys, larger ones first.
    uint32_t digits = 0;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, known = pass == 1 ? 21 : 10;
        clear_bins(s);
        each<F32, SMEM, kThreads>(row, 0, row.places, threadIdx.x, [&](const auto &l, int j) {
            for (int k = 0; k < sizeof(l) / sizeof(float); ++k) {
                const uint32_t turned = ~key_of(l[k]);
                if (!in_step(l[k], j + k) || (pass > 0 && (turned >> known) != digits)) continue;
                const uint64_t w = COUNT ? 1 : weight_of(l[k], row.w, s.table);
                if (w) add_to_bin(s, (turned >> shift) & (pass == 2 ? 1023 : 2047), w);
            }
        });
        find_bin<false>(s, c, target, 0, &f);
        digits = (digits << (pass == 2 ? 10 : 11)) | f.bin;
        target -= f.before;
    }
    const uint32_t key = ~digits;
    const float last = logit_of(key);
    const uint64_t one = COUNT ? 1 : weight_of_key(s, row, key);
    const uint64_t admitted = (target + one - 1) / one, tied = f.inside / one;
    uint32_t upto = row.bound && last == row.last ? row.upto : 0xffffffffu;
    if (admitted < tied) {
        // the admitted-th of the tied tokens by index
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        const int per = (row.places + kThreads - 1) / kThreads * 32;   // neighbouring places of a warp
        const int lo = min(warp * per, row.places), hi = min(lo + per, row.places);
        const auto is_tied = [&](int j) {
            const float l = j < hi ? read_place<F32, SMEM>(row, j) : kNone;
            return l == last && in_prefix(row, l, j);
        };
        uint64_t mine = 0;
        for (int j = lo + lane; j < hi; j += 32) mine += is_tied(j);
        uint64_t in_cta, whole;
        const uint64_t thread_before = block_scan(s, mine, &in_cta);
        const uint64_t before = __shfl_sync(0xffffffffu, thread_before, 0) + cluster_scan(s, c, in_cta, &whole);
        const uint64_t in_warp = warp_sum(mine);
        if (before < admitted && admitted <= before + in_warp) {
            uint64_t at = before;
            for (int j = lo + lane; j - lane < hi; j += 32) {
                const bool is = is_tied(j);
                const uint32_t who = __ballot_sync(0xffffffffu, is);
                if (is && at + __popc(who & ((2u << lane) - 1u)) == admitted)
                    for (unsigned k = 0; k < c.num_blocks(); ++k) c.map_shared_rank(&s, k)->bound_index = row.base + j;
                at += __popc(who);
            }
        }
        c.sync();
        upto = s.bound_index;
    }
    row.last = last;
    row.upto = upto;
    row.bound = true;
}

// The places of a warp's run, by which the sums of a draw are held: neighbouring ones, a multiple of 32.
__device__ __forceinline__ int run_of(int slice) { return (slice + kThreads - 1) / kThreads * 32; }

// Narrows the prefix to the shortest one of `share` of its weight, with one pass over the weights: the step it ends in is
// told beforehand by counts (times the weight of a step's middle), and the tokens of that step, and of a neighbour that
// the end is near to, are gathered as the sums of all and of those above are taken.  s.run_sum receives the sums of the
// warps' runs over the new prefix.  False where the prefix did not end there after all, or the tokens there are too many
// (nothing is changed).
template <bool F32, bool SMEM>
__device__ bool narrow_once(Shared &s, cg::cluster_group &c, Row &row, uint64_t share, int slice)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ranks = c.num_blocks();
    clear_bins(s);
    add_all<F32, SMEM, true>(s, row);
    Find f;
    const float step = 1.0f / row.steps;
    find_bin<true>(s, c, 0, share, &f, [&](int b) {
        return static_cast<uint64_t>(exp2f(kWeightBits - (static_cast<float>(b) + 0.5f) * step)) + 1;
    });
    // (the counts are right to far less than a quarter of a step, unless its tokens lie on one side of it)
    const uint64_t in = f.target - f.before;
    const bool early = in < f.inside / 4, late = in > f.inside - f.inside / 4;
    const float from = f.bin <= (early ? 1 : 0) ? kNone : f.bin - (early ? 1.0f : 0.0f), to = f.bin + (late ? 2.0f : 1.0f);
    Shared *first = c.map_shared_rank(&s, 0);
    const int run = run_of(slice), lo = min(warp * run, row.places), hi = min(lo + run, row.places);
    uint64_t all = 0, above = 0;
    each<F32, SMEM, 32>(row, lo, hi, lane, [&](const auto &l, int j) {
        constexpr int N = sizeof(l) / sizeof(float);
        WeightParts sums = {0u, 0u}, over = {0u, 0u};
        uint32_t which = 0, n_over = 0, n = 0;
        const auto one = [&](int k, WeightParts w) {
            const float t = weight_distance(l[k], row.w), at = t * row.steps;
            if (!in_prefix(row, l[k], j + k)) return;
            sums.high += w.high;
            sums.low += w.low;
            ++n;
            if (at < from) {
                over.high += w.high;
                over.low += w.low;
                ++n_over;
            } else if (at < to && t < kWeightEnd) {
                which |= 1u << k;
            }
        };
#pragma unroll
        for (int k = 0; k < N; k += 2) {
            WeightParts w0, w1;
            weight_parts_pair(l[k], l[k + 1], row.w, s.table, w0, w1);
            one(k, w0);
            one(k + 1, w1);
        }
        all += weight_sum(sums, n);
        above += weight_sum(over, n_over);
        append(first, row, l, j, which);
    });
    all = warp_sum(all);
    above = warp_sum(above);
    if (lane == 0) {
        s.run_sum[warp] = above;
        s.warp_sum[warp] = all;
    }
    if (threadIdx.x == 0) s.bound_key = 0;   // (no key of a token with weight)
    __syncthreads();
    if (warp == 0) {
        all = warp_sum(lane < kWarps ? s.warp_sum[lane] : 0);
        above = warp_sum(lane < kWarps ? s.run_sum[lane] : 0);
        if (lane == 0) {
            s.total = all;
            s.above = above;
        }
    }
    c.sync();
    const uint32_t n = first->gathered;
    if (n > kGather) {
        c.sync();   // (its number is not cleared before all have it)
        return false;
    }
    if (c.block_rank() == 0) {
        const Shared *of = c.map_shared_rank(&s, lane < ranks ? lane : 0);
        const uint64_t whole = warp_sum(lane < ranks ? of->total : 0), before = warp_sum(lane < ranks ? of->above : 0);
        uint64_t target = share_up(whole, share), last;
        if (target == 0) target = 1;
        sort_gathered(s, n);
        if (last_of<false>(s, row, n, before, target, &last)) tell_bound(s, c, last);
        __syncthreads();
        // the gathered tokens up to the bound belong to the runs that they lie in
        if (s.bound_key != 0) {
            for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
                const uint64_t token = s.sorted[i];
                if (token > (static_cast<uint64_t>(~s.bound_key) << 32 | s.bound_index)) break;
                const int place = static_cast<int>(static_cast<uint32_t>(token)) - row.base;   // (this CTA's places, carried on)
                const int rank = place / slice;
                atomicAdd(&c.map_shared_rank(&s, rank)->run_sum[(place - rank * slice) / run],
                          static_cast<unsigned long long>(weight_of_key(s, row, ~static_cast<uint32_t>(token >> 32))));
            }
        }
    }
    c.sync();
    if (s.bound_key == 0) return false;
    take_bound(s, row);
    return true;
}

__device__ __forceinline__ void answer(const SampleParams &p, int64_t r, uint32_t token, uint64_t w, uint64_t whole)
{
    p.token[r] = static_cast<int32_t>(token);
    if (p.prob) p.prob[r] = static_cast<float>(static_cast<double>(w) / static_cast<double>(whole));
}

// The draw from a gathered list of n tokens that begins with the row's first top_k ones: one CTA's work.
__device__ void draw_gathered(Shared &s, const SampleParams &p, int64_t r, const Row &row, int n, int top_k, float top_p,
                              uint64_t least, float u)
{
    const int tid = threadIdx.x;
    sort_gathered(s, n);
    const uint64_t token = tid < top_k ? s.sorted[tid] : 0;
    uint64_t w = tid < top_k ? weight_of_key(s, row, ~static_cast<uint32_t>(token >> 32)) : 0;
    uint64_t whole;
    const uint64_t before = block_scan(s, w, &whole);
    bool kept = tid < top_k && w >= least;
    if (top_p < 1.0f) kept = kept && (before < share_up(whole, fraction(top_p)) || tid == 0);
    if (!kept) w = 0;
    block_scan(s, w, &whole);
    const uint64_t target = share_down(whole, fraction(u));
    // sums in index order: over the kept ones up to this index
    uint64_t *const weights = s.sorted + kGather / 2;   // the upper half is free: top_k <= kGather / 2
    if (tid < top_k) weights[tid] = w;
    __syncthreads();
    if (w > 0) {
        uint64_t upto = 0;
        for (int j = 0; j < top_k; ++j)
            if (static_cast<uint32_t>(s.sorted[j]) <= static_cast<uint32_t>(token)) upto += weights[j];
        if (upto - w <= target && target < upto) answer(p, r, static_cast<uint32_t>(token), w, whole);
    }
}

// The slice's largest (NaN if there is one) and smallest logit among this thread's, and with SMEM the slice into shared
// memory.  kAhead loads of a thread are under way, each with a bound of its own (a loop's rest would load one after the
// other).
template <bool F32, bool SMEM>
__device__ __forceinline__ void first_read(const Row &row, float *v, float &top, float &low)
{
    constexpr int VEC = F32 ? 4 : 8;
    for (int j0 = threadIdx.x * VEC; j0 < row.places; j0 += kAhead * kThreads * VEC) {
        float f[kAhead][VEC];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int j = j0 + k * kThreads * VEC;
            if (j < row.places) read_places<F32>(row, j, kNone, f[k]);
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int j = j0 + k * kThreads * VEC, i = row.base + j;
            if (j >= row.places) break;
#pragma unroll
            for (int n = 0; n < VEC; ++n) top = max_nan(top, f[k][n]);
            if (i >= 0 && i + VEC <= row.V) {
#pragma unroll
                for (int n = 0; n < VEC; ++n) low = fminf(low, f[k][n]);
            } else {
#pragma unroll
                for (int n = 0; n < VEC; ++n)
                    if (i + n >= 0 && i + n < row.V) low = fminf(low, f[k][n]);
            }
            if constexpr (SMEM) {
#pragma unroll
                for (int n = 0; n < VEC; n += 4)
                    *reinterpret_cast<float4 *>(v + j + n) = make_float4(f[k][n], f[k][n + 1], f[k][n + 2], f[k][n + 3]);
            }
        }
    }
}

template <bool F32, bool SMEM>
__global__ void __launch_bounds__(kThreads, kSampleBlocks) sample_kernel(const SampleParams p)
{
    extern __shared__ __align__(16) unsigned char raw[];
    Shared &s = *reinterpret_cast<Shared *>(raw);
    cg::cluster_group c = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ranks = c.num_blocks(), rank = c.block_rank();
    int64_t r = blockIdx.x / ranks;
    constexpr float kInf = __builtin_inff();
    // (one 16-byte copy to a thread; nobody waits for it before the row's largest logit is known)
    static_assert(sizeof(s.table) == kThreads * 16, "the table's copy");
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(smem_u32(s.table + 2 * tid)), "l"(kWeightSteps32.step + 2 * tid)
                 : "memory");
    pdl_allow_next_grid();
    pdl_wait_prior_grid();

    if (p.reorder) {
        // Of kThreads neighbouring rows the ones with the most work come first: a row whose top-p takes all its tokens
        // twice, begun last, would run alone (512 rows of 128256 with settings of their own: 189 us as they stand, 153 in
        // this order).
        const int64_t first = r - r % kThreads, mine = first + tid;
        bool heavy = false;
        if (mine < p.R) {
            const int k = p.top_k ? p.top_k[mine] : p.top_k_all;
            heavy = (p.top_p ? p.top_p[mine] : p.top_p_all) < 1.0f && !(k > 0 && k <= kGatherTopK) &&
                    (p.temperature ? p.temperature[mine] : p.temperature_all) != 0.0f;
        }
        uint64_t all;
        const uint64_t before = block_scan(s, heavy ? 1 : 0, &all);
        if (mine < p.R && (heavy ? before : all + tid - before) == static_cast<uint64_t>(r - first)) s.first = tid;
        __syncthreads();
        r = first + s.first;
        __syncthreads();
    }
    const float T = p.temperature ? p.temperature[r] : p.temperature_all;
    const float top_p = p.top_p ? p.top_p[r] : p.top_p_all;
    const float min_p = p.min_p ? p.min_p[r] : p.min_p_all;
    const int top_k = p.top_k ? p.top_k[r] : p.top_k_all;
    const float u = p.u[r];

    // ---- the slice, and the row's largest and smallest logit
    constexpr int kElem = F32 ? 4 : 2, kVec = 16 / kElem;
    const unsigned char *const x = static_cast<const unsigned char *>(p.logits) + r * p.stride * kElem;
    const int early = static_cast<int>(reinterpret_cast<uintptr_t>(x) % 16) / kElem;   // places before the first token
    float *const v = reinterpret_cast<float *>(raw + sizeof(Shared));
    Row row;
    row.v = SMEM ? v : nullptr;
    row.V = p.V;
    row.base = rank * p.slice - early;
    row.x = x + static_cast<int64_t>(row.base) * kElem;
    row.places = (max(0, min(p.slice, p.V - row.base)) + kVec - 1) / kVec * kVec;
    float mine = kNone, low = kInf;
    first_read<F32, SMEM>(row, v, mine, low);
    float top = mine;
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, d));
        low = fminf(low, __shfl_xor_sync(0xffffffffu, low, d));
    }
    if (lane == 0) s.warp_sum[warp] = static_cast<uint64_t>(__float_as_uint(top)) << 32 | __float_as_uint(low);
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    const auto both = [&](uint64_t x, int count) {
        top = __uint_as_float(static_cast<uint32_t>(x >> 32));
        low = __uint_as_float(static_cast<uint32_t>(x));
        for (int d = count / 2; d; d >>= 1) {
            top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, d));
            low = fminf(low, __shfl_xor_sync(0xffffffffu, low, d));
        }
    };
    both(s.warp_sum[lane % kWarps], 32);
    if (ranks > 1) {
        if (tid == 0) {
            s.top = top;
            s.low = low;
            s.first = 0xffffffffu;
        }
        c.sync();
        const Shared *of = c.map_shared_rank(&s, lane % ranks);
        both(static_cast<uint64_t>(__float_as_uint(of->top)) << 32 | __float_as_uint(of->low), 32);
    } else if (tid == 0) {
        s.first = 0xffffffffu;
    }

    bool arrived = false;
    const bool bad = !(top < kInf) || !(T == 0.0f || (T >= 0x1p-64f && T <= 0x1p64f)) || !(top_p >= 0.0f) ||
                     !(min_p >= 0.0f && min_p <= 1.0f) || !(u >= 0.0f && u < 1.0f);
    if (bad || top == kNone) {
        if (rank == 0 && tid == 0) {
            p.token[r] = -1;
            if (p.prob) p.prob[r] = bad ? __int_as_float(0x7fffffff) : 0.0f;
            if (bad) atomicOr(p.status, kDevBadValue);
        }
    } else if (T == 0.0f) {
        __syncthreads();   // s.first is set
        if (mine == top) {   // this thread has one of the largest
            uint32_t first = 0xffffffffu;
            for (int j0 = tid * kVec; j0 < row.places && first == 0xffffffffu; j0 += kThreads * kVec)
                for (int j = j0 + kVec - 1; j >= j0; --j)
                    if (read_place<F32, SMEM>(row, j) == top) first = row.base + j;
            atomicMin(&s.first, first);
        }
        c.sync();
        if (rank == 0 && warp == 0) {
            uint32_t first = lane < ranks ? c.map_shared_rank(&s, lane)->first : 0xffffffffu;
            first = __reduce_min_sync(0xffffffffu, first);
            if (lane == 0) {
                p.token[r] = static_cast<int32_t>(first);
                if (p.prob) p.prob[r] = 1.0f;
            }
        }
    } else {
        float ch, cl;
        weight_scale(T, &ch, &cl);
        row.w = weight_row(top, ch, cl);
        // steps over what the row's distances span, 44 octaves at most (weights end there)
        const float span = fminf((top - low) * ch, kWeightEnd);
        row.steps = fminf(kBins / (span + 1e-3f), 1e6f);
        row.bound = false;
        const uint64_t largest = weight_of(top, row.w, s.table);
        const uint64_t least = min_p < 1.0f ? share_up(largest, fraction(min_p)) : largest;

        bool done = false;
        if (top_k > 0 && top_k < p.V) {
            if (top_k <= kGatherTopK) {
                // The k-th of the threads' largest logits: at least k tokens lie in its step or before it.
                clear_bins(s);
                const float t = weight_distance(mine, row.w);
                if (t < kWeightEnd) atomicAdd(&s.lo[step_of(row, t)], 1u);
                Find f;
                if (find_bin<true>(s, c, top_k, 0, &f)) {
                    const int step = f.bin;
                    const float to = step == kBins - 1 ? -kNone : step + 1.0f;   // (step_of(t) <= step)
                    const uint32_t n = gather_below<F32, SMEM>(s, c, row, mine, to);
                    if (n <= kGather) {
                        if (rank == 0) draw_gathered(s, p, r, row, n, top_k, top_p, least, u);
                        done = true;
                    }
                }
            }
            if (!done) narrow<F32, SMEM, true>(s, c, row, top_k, 0);
        }
        if (!done) {
            bool summed = false;   // whether s.run_sum has the sums already
            if (top_p < 1.0f) {
                summed = narrow_once<F32, SMEM>(s, c, row, fraction(top_p), p.slice);
                if (!summed) narrow<F32, SMEM, false>(s, c, row, 0, fraction(top_p));
                summed = summed && min_p == 0.0f;
            }

            // ---- the draw: sums in index order, by slices, then by ever shorter runs of the slice that has the token
            const bool plain = !row.bound && min_p == 0.0f;   // every token weighs in
            const float end = fminf(kWeightEnd, min_p > 0.0f ? 0.01f - log2f(min_p) : kWeightEnd);   // no weight of `least` beyond
            const auto weight = [&](float l, int j) {
                if (!(weight_distance(l, row.w) < end) || !in_prefix(row, l, j)) return uint64_t(0);
                const uint64_t w = weight_of(l, row.w, s.table);
                return w >= least ? w : uint64_t(0);
            };
            const auto sum_of_run = [&](int lo, int hi) {
                uint64_t sum = 0;
                if (plain)
                    each<F32, SMEM, 32>(row, lo, hi, lane, [&](const auto &l, int) {
                        WeightParts sums = {0u, 0u};
                        constexpr int N = sizeof(l) / sizeof(float);
#pragma unroll
                        for (int k = 0; k < N; k += 2) {
                            WeightParts w0, w1;
                            weight_parts_pair(l[k], l[k + 1], row.w, s.table, w0, w1);
                            sums.high += w0.high + w1.high;
                            sums.low += w0.low + w1.low;
                        }
                        sum += weight_sum(sums, N);
                    });
                else
                    each<F32, SMEM, 32>(row, lo, hi, lane, [&](const auto &l, int j) {
                        constexpr int N = sizeof(l) / sizeof(float);
                        bool in[N], any = false;
#pragma unroll
                        for (int k = 0; k < N; ++k) {
                            in[k] = weight_distance(l[k], row.w) < end && in_prefix(row, l[k], j + k);
                            any = any || in[k];
                        }
                        if (!any) return;
#pragma unroll
                        for (int k = 0; k < N; ++k) {
                            const uint64_t w = weight_of(l[k], row.w, s.table);
                            if (in[k] && w >= least) sum += w;
                        }
                    });
                return warp_sum(sum);
            };
            int lo = 0, hi = row.places, run = run_of(p.slice);   // a run to each warp
            uint64_t in_run = summed ? s.run_sum[warp] : sum_of_run(min(warp * run, hi), min((warp + 1) * run, hi));
            uint64_t all, whole;
            uint64_t before = block_scan(s, lane == 0 ? in_run : 0, &all);
            const uint64_t of_slices = cluster_scan(s, c, all, &whole);
            if (ranks > 1) {   // nothing of another CTA is read from here on
                c.barrier_arrive();
                arrived = true;
            }
            const uint64_t target = share_down(whole, fraction(u));   // below the whole, as u < 1
            if (of_slices <= target && target < of_slices + all) {
                before = __shfl_sync(0xffffffffu, before, 0) + of_slices;
                for (;;) {
                    // the run that has the token is the next round's whole
                    if (before <= target && target < before + in_run) {
                        if (lane == 0) {
                            s.first = lo + warp * run;
                            s.found.before = before;
                        }
                    }
                    __syncthreads();
                    lo = s.first;
                    hi = min(lo + run, hi);
                    before = s.found.before;
                    if (run == 32) break;
                    run = (run / 32 + kWarps - 1) / kWarps * 32;
                    uint64_t sum = 0;
#pragma unroll 1
                    for (int j = lo + warp * run + lane; j < min(lo + (warp + 1) * run, hi); j += 32)
                        sum += weight(read_place<F32, SMEM>(row, j), j);
                    in_run = warp_sum(sum);
                    before += __shfl_sync(0xffffffffu, block_scan(s, lane == 0 ? in_run : 0, &all), 0);
                }
                if (warp == 0) {
                    const uint64_t w = lo + lane < hi ? weight(read_place<F32, SMEM>(row, lo + lane), lo + lane) : 0;
                    const uint64_t upto = before + warp_scan(w);
                    if (upto - w <= target && target < upto) answer(p, r, row.base + lo + lane, w, whole);
                }
            }
        }
    }
    // no CTA leaves while another may read its shared memory
    if (ranks > 1) {
        if (!arrived) c.barrier_arrive();
        c.barrier_wait();
    }
}

}  // namespace

namespace {

template <bool F32, bool SMEM>
cudaError_t launch_with(SampleParams p, int64_t R, int ranks, cudaStream_t s, bool pdl)
{
    const size_t smem = sizeof(Shared) + (SMEM ? static_cast<size_t>(p.slice) * 4 : 0);
    const void *f = reinterpret_cast<const void *>(&sample_kernel<F32, SMEM>);
    cudaError_t e = ensure_smem_optin(f, 64 * 1024);
    if (e != cudaSuccess) return e;
    if (ranks > 8) {   // clusters of 16 are to be asked for, once on a device
        static std::atomic<uint64_t> asked;
        int dev = 0;
        e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const uint64_t bit = uint64_t(1) << (dev & 63);
        if (dev > 63 || !(asked.load(std::memory_order_relaxed) & bit)) {
            e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return e;
            asked.fetch_or(bit, std::memory_order_relaxed);
        }
    }
    return launch_ex_cluster(sample_kernel<F32, SMEM>, dim3(static_cast<unsigned>(R * ranks)), dim3(kThreads), smem, s, pdl, ranks, p);
}

}  // namespace

cudaError_t launch_sample(SampleParams p, int64_t R, bool f32, int sms, cudaStream_t s, bool pdl)
{
    const SamplePlan plan = plan_sample(R, p.V, sms);
    p.slice = plan.slice;
    p.R = R;
    p.reorder = R * plan.ranks > static_cast<int64_t>(kSampleBlocks) * sms && (p.temperature || p.top_p || p.top_k);
    const int ranks = plan.ranks;
    const bool smem = plan.smem;
    if (f32) return smem ? launch_with<true, true>(p, R, ranks, s, pdl) : launch_with<true, false>(p, R, ranks, s, pdl);
    return smem ? launch_with<false, true>(p, R, ranks, s, pdl) : launch_with<false, false>(p, R, ranks, s, pdl);
}

}  // namespace qmv

using namespace qmv;

extern "C" {

qmv_status qmv_sample(const void *logits, int64_t stride, int logits_f32, const float *u, const float *temperature,
                      const float *top_p, const float *min_p, const float *all, const int32_t *top_k, int64_t top_k_all,
                      int32_t *token, float *prob, int64_t R, int64_t V, qmv_stream_t stream)
{
    if (R < 0 || R > (int64_t(1) << 26) || V < 1 || V > kSampleVocab || stride < 0 || stride > (int64_t(1) << 40))
        return QMV_ERR_SHAPE;
    // (arrays of settings are checked row by row on the device)
    if (all && ((!temperature && !(all[0] == 0.0f || (all[0] >= 0x1p-64f && all[0] <= 0x1p64f))) ||
                (!top_p && !(all[1] >= 0.0f)) || (!min_p && !(all[2] >= 0.0f && all[2] <= 1.0f))))
        return QMV_ERR_SHAPE;
    if (R == 0) return QMV_OK;
    if (!logits || !u || !token) return QMV_ERR_NULL;
    for (const void *a : {static_cast<const void *>(u), static_cast<const void *>(temperature),
                          static_cast<const void *>(top_k), static_cast<const void *>(top_p),
                          static_cast<const void *>(min_p), static_cast<const void *>(token),
                          static_cast<const void *>(prob)})
        if (reinterpret_cast<uintptr_t>(a) % 4 != 0) return QMV_ERR_ALIGN;
    if (reinterpret_cast<uintptr_t>(logits) % (logits_f32 ? 4 : 2) != 0) return QMV_ERR_ALIGN;
    SampleParams p = {};
    int sms = 0;
    bool pdl = false;
    if (call_env(&p.status, &sms, &pdl) != cudaSuccess) return QMV_ERR_CUDA;
    p.logits = logits;
    p.u = u;
    p.temperature = temperature;
    p.top_k = top_k;
    p.top_p = top_p;
    p.min_p = min_p;
    p.temperature_all = all ? all[0] : 1.0f;
    p.top_p_all = all ? all[1] : 1.0f;
    p.min_p_all = all ? all[2] : 0.0f;
    p.top_k_all = static_cast<int32_t>(top_k_all < 0 ? 0 : top_k_all > kSampleVocab ? kSampleVocab : top_k_all);
    p.token = token;
    p.prob = prob;
    p.stride = stride;
    p.V = static_cast<int>(V);
    if (launch_sample(p, R, logits_f32 != 0, sms, reinterpret_cast<cudaStream_t>(stream), pdl) != cudaSuccess) {
        (void)cudaGetLastError();
        return QMV_ERR_LAUNCH;
    }
    return QMV_OK;
}

}  // extern "C"
