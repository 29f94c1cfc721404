// Checks the rules by which the adapters' work is cut up (built without optimisation and with traps on signed overflow, and run, by tests/test_adapter_cuts.py):
// every cut is one that the kernels have, and no rule reads what it has not written, which here would be numbers whose sum overflows.
#include <cstdio>
#include <initializer_list>

#include "adapter_cuts.h"

using namespace sgb::ad;

__attribute__((noinline)) void fill_stack()
{
    volatile unsigned char below[8192];
    for (unsigned i = 0; i < sizeof below; ++i) below[i] = 0x7f;
}

int main()
{
    unsigned long long bad = 0, checks = 0;
    const auto want = [&](bool ok, const char* what, long long rows, long long adapters, int rank, long long cols, long long outs) {
        ++checks;
        if (!ok && bad++ < 10) std::printf("%s: %lld rows, %lld adapters, rank %d, %lld -> %lld\n", what, rows, adapters, rank, cols, outs);
    };
    for (const int64_t rows : {int64_t(0), int64_t(1), int64_t(20), int64_t(641), int64_t(12544), int64_t(1) << 24, (int64_t(1) << 31) - (1 << 16)})
        for (const int64_t adapters : {int64_t(1), int64_t(16), int64_t(4000), int64_t(65535)})
            for (const int rank : {1, 16, 64, 65, 128})
                for (const int64_t cols : {int64_t(1), int64_t(256), int64_t(4097), int64_t(1) << 30})
                    for (const int64_t outs : {int64_t(1), int64_t(777), int64_t(1) << 30}) {
                        fill_stack();
                        const SumCut s = cut_sums(rows, adapters, rank, cols, outs);
                        want(s.da >= 1 && s.da <= SUM_TILES && s.db >= 1 && s.db <= SUM_TILES, "tiles to a piece", rows, adapters, rank, cols, outs);
                        want(rows > 0 || (s.da == 1 && s.db == 1), "no rows", rows, adapters, rank, cols, outs);
                        for (const bool vec : {false, true}) {
                            const PassCut p = cut_pass(rows, adapters, rank, static_cast<int>(cols), static_cast<int>(outs), 4, 2, vec);
                            want(p.splits == 1 || p.splits == 2 || p.splits == 4 || p.splits == 8, "splits", rows, adapters, rank, cols, outs);
                            // without a result there are no more CTAs to a tile than the first product has steps
                            const PassCut alone = cut_pass(rows, adapters, rank, static_cast<int>(cols), static_cast<int>(outs), 4, 0, vec);
                            want(alone.splits >= 1 && (alone.splits == 1 || alone.splits <= blocks_of(cols, P_STEP)), "splits of the first product", rows, adapters, rank, cols, outs);
                        }
                    }
    std::printf("%llu checks, %llu wrong\n", checks, bad);
    return bad ? 1 : 0;
}
