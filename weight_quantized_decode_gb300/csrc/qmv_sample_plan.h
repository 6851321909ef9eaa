// qmv_sample_plan.h -- how qmv_sample cuts a row: CTAs of a cluster, places of a slice, and where the slices are held (host
// code without CUDA, which a test compiles for the CPU).
#pragma once

#include <cstdint>

namespace qmv {

constexpr int kSampleBlocks = 2;        // CTAs to an SM
constexpr int kSampleShared = 26624;    // bytes of shared memory that a CTA has beside its slice, at the most

struct SamplePlan {
    int ranks;    // CTAs to a row
    int slice;    // places of a CTA: a multiple of 32, all of them the row and up to 7 places before it
    bool smem;    // slices in shared memory, fp32
};

inline SamplePlan plan_sample(int64_t R, int64_t V, int sms)
{
    // A slice of up to 16384 logits leaves room in shared memory for two CTAs on an SM, one of up to 49152 for one.
    // Few rows: as many CTAs to a row as run at once, the row in shared memory.  More rows, or longer ones, are read again
    // from memory (which for the rows under way is the L2), so that a row needs fewer CTAs, which wait for each other.
    // Measured, us, unfiltered / top-k 50 / top-p 0.9, in shared memory (s) or from memory (m) by clusters of:
    //   rows x logits     1 x 128256   8 x 128256   32 x 128256  64 x 128256  256 x 128256  512 x 128256  128 x 32003  256 x 32003
    //     16 s            9/11/21      13/15/27     27/38/66     50/67/117    189/253/439   373/496/863   82/125/182   158/240/348
    //      8 s            11/10/25     11/11/25     16/15/34     30/26/63     105/103/225   202/193/436   32/45/71     60/86/132
    //      4 s            14/11/33     14/12/33     15/12/34     28/23/65     102/94/246    197/176/464   21/24/44     37/45/77
    //      2 s                                                                                            16/16/32     30/28/60
    //      8 m            12/11/25     12/11/27     17/14/36     31/26/67     109/99/242    209/186/469
    //      4 m            17/12/38     16/12/38     22/14/46     25/15/51     87/62/179     158/107/337   22/25/46     39/45/85
    //      2 m            25/14/57     26/14/58     26/15/61     34/17/75     81/45/167     136/85/290    17/15/34     31/29/65
    //      1 m            41/18/99     42/18/99     42/19/99     43/19/99     81/35/167     148/72/312    19/15/43     22/16/48
    // (rows of normal logits times 1.7; text-like rows take longer with top-p: 512 of 128256 323 for 290.)  The rule knows
    // rows and logits only: where all rows have top-k, one CTA to a row would be faster (512 x 128256: 72 for 85).
    // Rows of very different settings, more than run at once, end more evenly with two CTAs to a row (512 x 128256, each
    // row with settings of its own: 154 us, by one 266).
    const int64_t slots = static_cast<int64_t>(kSampleBlocks) * sms;
    const auto slice_of = [&](int ranks) { return (V + ranks - 1) / ranks; };
    int ranks = R <= 4 ? 16 : 8;
    while (ranks > 1 && (R * ranks > slots || slice_of(ranks) < 2048)) ranks /= 2;
    // one CTA to an SM, and clusters of eight find room for less than the whole GPU
    while (ranks > 1 && slice_of(ranks) > 16384 && R * ranks > (ranks == 8 ? 7 * sms / 10 : 9 * sms / 10)) ranks /= 2;
    bool smem = slice_of(ranks) <= 16384 || (slice_of(ranks) <= 49152 && R * ranks <= 9 * sms / 10);
    if (!smem) {
        ranks = 8;
        while (ranks > 1 && R * ranks > slots) ranks /= 2;
        if (R > slots && V > 65536) ranks = 2;
    }
    // (and the places before a row's first token)
    return {ranks, static_cast<int>(((V + 7 + ranks - 1) / ranks + 31) / 32 * 32), smem};
}

}  // namespace qmv
