// Checks sgb::ln::row_copy (built and run by tests/test_row_copy.py): over rows of every alignment, each copy of the row kernels reads
// from an aligned address inside the tensor, empty copies too, and a row's copies together bring each of its elements once.
#include <cstdint>
#include <cstdio>
#include <vector>

#include "row_copy.h"

int main()
{
    unsigned long long bad = 0, checks = 0;
    auto want = [&](bool ok, const char* what, int64_t cols, int64_t stride, int64_t r, int c) {
        ++checks;
        if (!ok && bad++ < 10) std::printf("%s: cols %lld stride %lld row %lld column %d\n", what, (long long)cols, (long long)stride, (long long)r, c);
    };
    // elements to a vector, to a copy: bf16 and fp32 rows in 16-byte copies, a bf16 dy beside an fp32 x in 8-byte ones, an fp32
    // dy beside a bf16 x in two copies a vector
    const struct { int vec, per; } kinds[] = {{8, 8}, {4, 4}, {8, 4}};
    const int shapes[][2] = {{4, 16}, {8, 8}, {8, 16}, {16, 8}, {32, 8}, {32, 16}, {64, 8}, {64, 16}, {96, 32}};
    for (const auto& k : kinds)
        for (const auto& s : shapes) {
            const int group = s[0], elems = s[1], most = group * elems;
            for (int cols : {1, 2, 5, most / 2 + 1, most - 9, most - 8, most - 7, most / 8 * 8})
                for (int extra : {0, 1, 3, 8, 13}) {
                    const int64_t stride = cols + extra, rows = 11;
                    const bool whole = cols % 8 == 0 && stride % 8 == 0;
                    if (cols < 1 || (!whole && cols + 7 > most)) continue;
                    for (int64_t r = 0; r < rows + 2; ++r) {
                        const bool live = r < rows;
                        const int front = live ? static_cast<int>(r * stride % k.vec) : 0;
                        const int64_t row = live ? r * stride : 0;
                        std::vector<int> seen(cols);
                        for (int t = 0; t < group; ++t)
                            for (int u = 0; u < elems / k.vec; ++u)
                                for (int j = 0; j < k.vec / k.per; ++j) {
                                    const int c = t * k.vec - front + u * group * k.vec + j * k.per;
                                    const sgb::ln::RowCopy copy = sgb::ln::row_copy(c, k.per, live ? cols : 0, front, whole);
                                    const int64_t at = row + copy.at;
                                    want(at % k.per == 0, "unaligned", cols, stride, r, c);
                                    want(copy.count >= 0 && copy.count <= k.per, "count", cols, stride, r, c);
                                    want(at >= 0 && at + copy.count <= (rows - 1) * stride + cols, "outside", cols, stride, r, c);
                                    for (int i = 0; i < copy.count; ++i)
                                        if (copy.at + i >= 0 && copy.at + i < cols) ++seen[copy.at + i];
                                }
                        for (int c = 0; c < cols; ++c) want(seen[c] == (live ? 1 : 0), "times read", cols, stride, r, c);
                    }
                }
        }
    std::printf("%llu checks, %llu wrong\n", checks, bad);
    return bad ? 1 : 0;
}
