// qmv_kv_tree.cu -- after the nodes of a drafted tree have been sampled: the path
// that the samples accept, and the move of its rows in the caches.
#include <cstdint>

#include "qmv_common.cuh"
#include "qmv_kv.h"
#include "qmv_launch.h"

namespace qmv {

namespace {

// ---- the accepted path ----------------------------------------------------------
//
//   node 0 is accepted; behind an accepted node c the lowest j > c with
//   row(j) = row(c) + {j} (chain: j = c + 1) and token[j] = sampled[c] is.  Where slots
//   are given, only nodes that have one, and a place of the path to be moved to.
//
// One warp to a request: its lanes look at 32 nodes at a time, the token first,
// and the mask words only of those that have it.  Bound by latency: a few loads
// one behind the other for each accepted node (one tree of 8 nodes 2.7 us, 1000 trees
// of 9 to 64 6.9 us, both mostly the launch).
constexpr int kAcceptThreads = 128;

__device__ __forceinline__ uint32_t row_word(const AcceptParams &p, int64_t t, int w, int64_t nodes)
{
    uint32_t m = static_cast<uint32_t>(p.tree[t * p.tree_words + w]);
    const int64_t left = nodes - 32LL * w;
    if (left < 32) m &= left > 0 ? (1u << left) - 1u : 0u;
    return m;
}

// Whether node j's row is node c's with j added.
__device__ __forceinline__ bool is_child(const AcceptParams &p, int64_t lo, int64_t nodes, int64_t c, int64_t j)
{
    if (!p.tree) return j == c + 1;
    if (j >= 32LL * p.tree_words) return false;   // no row names it
    for (int w = 0; w < p.tree_words && 32LL * w < nodes; ++w) {
        const uint32_t own = (j >> 5) == w ? 1u << (j & 31) : 0u;
        const uint32_t of_c = row_word(p, lo + c, w, nodes);
        if ((of_c & own) || row_word(p, lo + j, w, nodes) != (of_c | own)) return false;
    }
    return true;
}

__global__ void __launch_bounds__(kAcceptThreads) tree_accept_kernel(const AcceptParams p)
{
    pdl_allow_next_grid();
    pdl_wait_prior_grid();
    const int lane = threadIdx.x & 31;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kAcceptThreads / 32);
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (kAcceptThreads / 32) + (threadIdx.x >> 5);
    for (int64_t r = first; r < p.R; r += warps) {
        const int64_t lo = p.start[r], hi = p.start[r + 1], len = p.kv_len[r], nodes = hi - lo;
        if (lo < 0 || hi < lo || hi > p.T || len < nodes) {
            if (lane == 0) {
                p.count[r] = 0;
                p.next[r] = -1;
                p.lens[r] = static_cast<int32_t>(len);
                atomicOr(p.status, kDevBadLength);
            }
            continue;
        }
        // (a request whose first node has no row keeps nothing)
        const bool begins = nodes > 0 && !(p.slots && p.slots[lo] < 0);
        int64_t c = 0, taken = begins ? 1 : 0;
        int32_t want = -1;
        if (begins) {
            want = p.sampled[lo];
            if (lane == 0) p.path[lo] = 0;
        }
        while (begins && want >= 0) {
            int64_t found = -1;
            const int64_t upto = p.tree ? nodes : (c + 2 < nodes ? c + 2 : nodes);
            for (int64_t base = c + 1; base < upto && found < 0; base += 32) {
                const int64_t j = base + lane;
                const bool hit = j < upto && p.tokens[lo + j] == want && is_child(p, lo, nodes, c, j) &&
                                 !(p.slots && (p.slots[lo + j] < 0 || p.slots[lo + taken] < 0));
                const uint32_t who = __ballot_sync(0xffffffffu, hit);
                if (who) found = base + __ffs(who) - 1;
            }
            if (found < 0) break;
            c = found;
            if (lane == 0) p.path[lo + taken] = static_cast<int32_t>(c);
            ++taken;
            want = p.sampled[lo + c];
        }
        for (int64_t i = taken + lane; i < nodes; i += 32) p.path[lo + i] = -1;
        if (lane == 0) {
            p.count[r] = static_cast<int32_t>(taken);
            p.next[r] = want < 0 ? -1 : want;
            p.lens[r] = static_cast<int32_t>(len - nodes + taken);
        }
    }
    // Places past the last request's nodes are padding.  Where offsets fall, other requests' may lie there: past all of
    // theirs.
    const int64_t last = p.R > 0 ? p.start[p.R] : 0;
    if (last >= 0 && last + first * 32 < p.T) {
        int end = static_cast<int>(last);
#pragma unroll 4
        for (int64_t r = lane; r < p.R; r += 32) {
            const int lo = p.start[r], hi = p.start[r + 1];
            if (lo >= 0 && hi >= lo && hi <= p.T) end = max(end, hi);
        }
        end = __reduce_max_sync(0xffffffffu, end);
        for (int64_t i = end + first * 32 + lane; i < p.T; i += warps * 32) p.path[i] = -1;
    }
}

// ---- kept rows --------------------------------------------------------------------
//
//   row(slot[path[i]]) -> row(slot[i]),  i < count,  for all heads, keys and values,
//   in every cache of the call
//
// A group of lanes carries one head's row of one cache, 16 bytes to a lane, along
// the whole path: as path[i] > path[i - 1], a place is written only after its own
// row has been read, whatever else runs.  kAhead rows are read before any of them is
// written: more shorten a lone long path and cost a batch its occupancy (64 requests
// in 32 caches of 8 heads of 128, 69 MB, and one path of 40 rows in 32 caches, us: 1 ahead
// 19.3 and 19.5, 2 21.3 and 18.4, 4 21.5 and 17.5, 8 32 and 15.8).  Bound by the latency of
// scattered rows of 256 bytes, four loads one behind the other for each; one request's
// path of a few nodes in 32 caches 2.7 us; the batch with 8-bit rows 12.7 for 5.2 of bytes.
constexpr int kKeepThreads = 128;
constexpr int kAhead = 1;

template <int LANES>   // lanes to a row, 16 bytes each
__global__ void __launch_bounds__(kKeepThreads) kv_keep_kernel(const __grid_constant__ KeepParams p, int row_elems)
{
    constexpr int ROWS = kKeepThreads / LANES;
    pdl_allow_next_grid();
    pdl_wait_prior_grid();
    const int sub = threadIdx.x / LANES, l = threadIdx.x % LANES;
    const int64_t tasks = p.R * p.Hkv;   // of a cache's keys or values (blockIdx.y)
    const int page = 1 << p.page_shift;
    const int row_bytes = LANES * 16, elem = row_bytes / row_elems;
    const int cache = blockIdx.y >> 1;
    const bool is_v = blockIdx.y & 1;
    for (int64_t task = static_cast<int64_t>(blockIdx.x) * ROWS + sub; task < tasks;
         task += static_cast<int64_t>(gridDim.x) * ROWS) {
        const int64_t r = tasks <= 0xffffffffll ? static_cast<uint32_t>(task) / static_cast<uint32_t>(p.Hkv) : task / p.Hkv;
        const int head = static_cast<int>(task - r * p.Hkv);
        const bool tells = blockIdx.y == 0 && head == 0 && l == 0;   // one thread of a request
        const int64_t lo = p.start[r], hi = p.start[r + 1];
        const int count = p.count[r], nodes = static_cast<int>(hi - lo);
        if (lo < 0 || hi < lo || hi > p.T || count < 0 || count > nodes) {
            if (tells) atomicOr(p.status, kDevBadLength);
            continue;
        }
        char *rows = static_cast<char *>(is_v ? p.v[cache] : p.k[cache]);
        float *scales = is_v ? p.v_scale[cache] : p.k_scale[cache];
        int bad = 0;
        int last = -1;
        for (int i0 = 0; i0 < count && !(bad & kDevBadLength); i0 += kAhead) {
            // all indices of one kind at a time: four loads one behind the other for kAhead rows
            int node[kAhead], to[kAhead], from[kAhead];
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                const bool there = i0 + a < count;
                node[a] = there ? p.path[lo + i0 + a] : -1;
                to[a] = there ? p.slots[lo + i0 + a] : -1;
            }
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                if (i0 + a < count && (node[a] <= last || node[a] >= nodes)) bad |= kDevBadLength;
                if (i0 + a >= count || (bad & kDevBadLength)) node[a] = -1;   // not ascending, or no node: nothing from here on
                if (node[a] >= 0) last = node[a];
                if (node[a] == i0 + a) node[a] = -1;                          // stays where it is
                from[a] = node[a] >= 0 ? p.slots[lo + node[a]] : 0;
            }
            uint4 data[kAhead];
            float scale[kAhead];
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                if (node[a] < 0) continue;
                if (from[a] < 0 || from[a] >= p.n_slots || to[a] < 0 || to[a] >= p.n_slots) {
                    bad |= from[a] == -1 || to[a] == -1 ? kDevNoPages : kDevBadPage;   // (a token that its step had no page for)
                    node[a] = -1;
                    continue;
                }
                const int64_t cell = from[a] >> p.page_shift;
                const int row = (head << p.page_shift) + (from[a] & (page - 1));
                data[a] = *reinterpret_cast<const uint4 *>(rows + cell * p.page_stride * elem + row * row_bytes + 16 * l);
                if (scales && l == 0) scale[a] = scales[((cell * p.Hkv) << p.page_shift) + row];
            }
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                if (node[a] < 0) continue;
                const int64_t cell = to[a] >> p.page_shift;
                const int row = (head << p.page_shift) + (to[a] & (page - 1));
                *reinterpret_cast<uint4 *>(rows + cell * p.page_stride * elem + row * row_bytes + 16 * l) = data[a];
                if (scales && l == 0) scales[((cell * p.Hkv) << p.page_shift) + row] = scale[a];
            }
        }
        if (bad && tells) atomicOr(p.status, bad);
    }
}

}  // namespace

cudaError_t launch_tree_accept(const AcceptParams &p, cudaStream_t s, bool pdl)
{
    int64_t grid = (p.R + kAcceptThreads / 32 - 1) / (kAcceptThreads / 32);
    if (grid < 1) grid = 1;
    if (grid > 1 << 20) grid = 1 << 20;
    return launch_ex(tree_accept_kernel, dim3(static_cast<unsigned>(grid)), dim3(kAcceptThreads), 0, s, pdl, p);
}

cudaError_t launch_kv_keep(const KeepParams &p, int D, int kind, cudaStream_t s, bool pdl)
{
    const int lanes = D * (kind == kKvF16 ? 2 : 1) / 16;
    const int64_t rows = kKeepThreads / lanes;
    int64_t grid = (p.R * p.Hkv + rows - 1) / rows;
    if (grid > 1 << 16) grid = 1 << 16;
    const dim3 g(static_cast<unsigned>(grid), static_cast<unsigned>(2 * p.caches)), b(kKeepThreads);
    if (lanes == 4) return launch_ex(kv_keep_kernel<4>, g, b, 0, s, pdl, p, D);
    if (lanes == 8) return launch_ex(kv_keep_kernel<8>, g, b, 0, s, pdl, p, D);
    return launch_ex(kv_keep_kernel<16>, g, b, 0, s, pdl, p, D);
}

}  // namespace qmv
