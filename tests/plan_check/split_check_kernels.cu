// split_check_kernels.cu -- the split of work of split_check.cu with the block
// sizes, unit rows and fixed costs that the kernels are compiled with.
//
// Built and run by tests/test_split_check_kernels.py.
#define main other_sizes
#include "split_check.cu"
#undef main

int main()
{
    std::mt19937 rng(11);
    for (int i = 0; i < 400; ++i) {
        const int R = 1 + static_cast<int>(rng() % (i % 4 == 0 ? 300 : 12));
        const int len_hi = i % 3 == 0 ? 40 : (i % 3 == 1 ? 3000 : 40000 / R);
        const int new_hi = i % 5 == 0 ? 1 : (i % 5 == 1 ? 2000 / R : 40);
        const int groups[] = {1, 2, 3, 4, 5, 8, 20, 300};
        const Batch b = make(rng, R, len_hi, new_hi, groups[rng() % 8], 1 + static_cast<int>(rng() % 8), rng() % 2, i % 7 == 0);
        const int grids[] = {152, 304, 608, 1, 7};
        const int grid = grids[rng() % 5];
        check<8, RowsSplit::kBlock, RowsSplit::kCost, false>(b, grid);
        check<16, RowsSplit::kBlock, RowsSplit::kCost, false>(b, grid);
        check<32, RowsSplit::kBlock, RowsSplit::kCost, false>(b, grid);
        check<TilesSplit::kRows, TilesSplit::kBlock, TilesSplit::kCost, true>(b, grid);
    }
    std::printf("%ld checked, %ld failures\n", g_checked, g_bad);
    return g_bad ? 1 : 0;
}
