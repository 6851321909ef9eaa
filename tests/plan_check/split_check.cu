// split_check.cu -- host-only check of how attention over the paged cache
// splits its work over CTAs.  No GPU is needed and no kernel runs: for many
// batches of uneven requests the program walks every CTA's share with the
// kernels' own code and checks that every block of every unit is taken once and
// in order, that a shared unit's parts lie with neighbouring CTAs the way the
// joining kernel looks for them, that no CTA needs more than its two places of
// the workspace, and that blocks left out for a chain's row tile hold nothing
// its rows see.  seen_places is checked bit by bit against the definition.
//
// Built and run by tests/test_split_check.py.
#include "../../weight_quantized_decode_gb300/csrc/qmv_attn.cuh"

#include <cstdio>
#include <map>
#include <random>
#include <vector>

using namespace qmv;

namespace {

long g_bad = 0, g_checked = 0;

#define CHECK(cond, ...)                                   \
    do {                                                   \
        ++g_checked;                                       \
        if (!(cond)) {                                     \
            if (g_bad < 20) {                              \
                std::printf("FAIL %s: ", #cond);           \
                std::printf(__VA_ARGS__);                  \
                std::printf("\n");                         \
            }                                              \
            ++g_bad;                                       \
        }                                                  \
    } while (0)

struct Batch {
    std::vector<int32_t> start, kv_len;
    AttnParams p = {};
};

Batch make(std::mt19937 &rng, int R, int len_hi, int new_hi, int group, int hkv, bool tree, bool spoil)
{
    Batch b;
    b.start.push_back(0);
    for (int r = 0; r < R; ++r) {
        const int n = static_cast<int>(rng() % (new_hi + 1)), len = static_cast<int>(rng() % (len_hi + 1));
        b.start.push_back(b.start.back() + n);
        b.kv_len.push_back(len + n);
        if (spoil && rng() % 5 == 0) b.kv_len.back() = rng() % 2 ? -3 : 1 << 30;
    }
    b.p.start = b.start.data();
    b.p.kv_len = b.kv_len.data();
    static const int32_t words[1] = {0};
    b.p.tree = tree ? words : nullptr;   // (not read here: only whether there is one)
    b.p.R = R;
    b.p.T = b.start.back() - (spoil ? new_hi / 2 : 0);
    if (b.p.T < 0) b.p.T = 0;
    b.p.page_shift = 4;
    b.p.width = (len_hi + new_hi) / 16 + 2;
    b.p.Hkv = hkv;
    b.p.group = group;
    return b;
}

struct Unit {
    int64_t blocks = 0, taken = 0;
    int lead = -1, last = -1, parts = 0, seen = 0;
};

template <int ROWS, int BLOCK, int COST, bool CUT>
void check(const Batch &b, int grid)
{
    const AttnParams &p = b.p;
    int64_t total = 0;
    std::vector<int64_t> before(p.R + 1, 0);
    for (int64_t r = 0; r < p.R; ++r) {
        const RequestWork w = request_work<ROWS, BLOCK, COST, CUT>(p, r);
        int64_t sum = 0;
        for (int t = 0; t < w.tiles; ++t) sum += unit_entries<ROWS, BLOCK, COST, CUT>(p, w, t);
        CHECK(sum == w.per_head && w.total == sum * p.Hkv, "request %ld", static_cast<long>(r));
        total += w.total;
        before[r + 1] = total;
    }
    std::map<std::vector<int64_t>, Unit> units;
    for (int64_t r = 0; r < p.R; ++r) {
        const RequestWork w = request_work<ROWS, BLOCK, COST, CUT>(p, r);
        for (int h = 0; h < p.Hkv; ++h)
            for (int t = 0; t < w.tiles; ++t) {
                Unit u;
                u.blocks = unit_entries<ROWS, BLOCK, COST, CUT>(p, w, t) - COST;
                units[{r, h, t}] = u;
                if (CUT && !p.tree && !w.bad) {
                    // the last token of the tile sees nothing past its own place
                    int64_t last = ((static_cast<int64_t>(t) + 1) * ROWS - 1) / p.group;
                    if (last >= w.nodes) last = w.nodes - 1;
                    CHECK(w.len - w.nodes + last < u.blocks * BLOCK, "cut too far: tile %d", t);
                    CHECK(u.blocks * BLOCK < w.len - w.nodes + last + 1 + BLOCK, "cut too little: tile %d", t);
                }
            }
    }
    for (int cta = 0; cta < grid; ++cta) {
        Share sh = {};
        share_of(total, grid, cta, &sh.g, &sh.lo, &sh.hi);
        sh.total = total;
        if (sh.lo < sh.hi) {
            sh.r = 0;
            while (!(before[sh.r] <= sh.lo && sh.lo < before[sh.r + 1])) ++sh.r;
            sh.before = before[sh.r];
            sh.w = request_work<ROWS, BLOCK, COST, CUT>(p, sh.r);
        }
        SegmentWalk<ROWS, BLOCK, COST, CUT> walk;
        walk.begin(p, sh, cta);
        Segment s;
        int begun = 0, continued = 0;
        while (walk.next(p, s)) {
            auto it = units.find({s.r, s.kvh, s.tile});
            CHECK(it != units.end(), "no such unit: %ld %d %d", static_cast<long>(s.r), s.kvh, s.tile);
            if (it == units.end()) return;
            Unit &u = it->second;
            CHECK(s.nb > 0 && s.b0 == u.taken && s.b0 + s.nb <= u.blocks, "blocks %ld + %ld, %ld taken of %ld",
                  static_cast<long>(s.b0), static_cast<long>(s.nb), static_cast<long>(u.taken), static_cast<long>(u.blocks));
            CHECK(s.whole == (s.nb == u.blocks), "whole");
            if (s.b0 == 0) u.lead = cta;
            if (!s.whole) {
                if (s.b0 == 0) {
                    ++begun;
                    u.parts = s.parts;
                    CHECK(s.parts > 1, "parts %d", s.parts);
                } else {
                    ++continued;
                    CHECK(s.parts == 0 && cta == u.last + 1, "part of CTA %d after %d", cta, u.last);
                }
            } else {
                CHECK(s.parts == 0, "parts of a whole unit");
            }
            u.taken += s.nb;
            u.last = cta;
            ++u.seen;
        }
        CHECK(begun <= 1 && continued <= 1, "CTA %d begins %d and continues %d", cta, begun, continued);
    }
    for (const auto &kv : units) {
        const Unit &u = kv.second;
        CHECK(u.taken == u.blocks, "unit with %ld of %ld blocks", static_cast<long>(u.taken), static_cast<long>(u.blocks));
        if (u.seen > 1) CHECK(u.parts == u.seen && u.last == u.lead + u.parts - 1, "parts %d, seen %d", u.parts, u.seen);
    }
}

void check_seen(std::mt19937 &rng)
{
    for (int i = 0; i < 20000; ++i) {
        const int nodes = 1 + static_cast<int>(rng() % 150), ctx = static_cast<int>(rng() % 200);
        const int words = 1 + static_cast<int>(rng() % 5), node = static_cast<int>(rng() % nodes);
        std::vector<int32_t> row(words);
        for (auto &w : row) w = static_cast<int32_t>(rng());
        const bool tree = rng() % 2;
        const int64_t len = ctx + nodes, j0 = static_cast<int64_t>(rng() % (len + 40));
        const uint32_t got = seen_places(tree ? row.data() : nullptr, words, node, nodes, len, j0);
        for (int k = 0; k < 32; ++k) {
            const int64_t j = j0 + k, n = j - ctx;
            bool want = j < len;
            if (want && n >= 0)
                want = tree ? n < 32 * words && (static_cast<uint32_t>(row[n >> 5]) >> (n & 31) & 1u) : n <= node;
            CHECK((got >> k & 1u) == (want ? 1u : 0u), "place %ld", static_cast<long>(j));
        }
    }
}

}  // namespace

int main()
{
    std::mt19937 rng(7);
    for (int i = 0; i < 400; ++i) {
        const int R = 1 + static_cast<int>(rng() % (i % 4 == 0 ? 300 : 12));
        const int len_hi = i % 3 == 0 ? 40 : (i % 3 == 1 ? 3000 : 40000 / R);
        const int new_hi = i % 5 == 0 ? 1 : (i % 5 == 1 ? 2000 / R : 40);
        const int groups[] = {1, 2, 3, 4, 5, 8, 20};
        const Batch b = make(rng, R, len_hi, new_hi, groups[rng() % 7], 1 + static_cast<int>(rng() % 8), rng() % 2, i % 7 == 0);
        const int grids[] = {152, 304, 608, 1, 7};
        const int grid = grids[rng() % 5];
        check<8, 128, 2, false>(b, grid);
        check<16, 128, 2, false>(b, grid);
        check<32, 128, 2, false>(b, grid);
        check<256, 128, 6, true>(b, grid);
    }
    check_seen(rng);
    std::printf("%ld checked, %ld failures\n", g_checked, g_bad);
    return g_bad ? 1 : 0;
}
