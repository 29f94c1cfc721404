// How the adapters' work is cut up over the SMs, in plain C++ so that the host can check it.
#pragma once

#include <cstdint>

namespace sgb {
namespace ad {

constexpr int CARD_SMS = 152;

constexpr int TILE = 128;      // rows of a tile of the plan, at most
constexpr int P_STEP = 128;    // of `from`: in a stage of a pass
constexpr int P_COLS = 128;    // of `to`: in a chunk of a pass
constexpr int SUM_TILES = 32;  // of a piece of the sums, at most

inline int64_t blocks_of(int64_t n, int64_t size) { return n / size + (n % size != 0); }

// About how many pieces of up to `tile` rows there are: one to an adapter at least, and half a piece more to each than its rows fill.
inline int64_t tiles_about(int64_t rows, int64_t groups, int tile)
{
    groups = groups < rows ? groups : rows;
    const int64_t filled = rows / tile + (groups + 1) / 2;
    return filled > groups ? filled : groups;
}

// Blocks of 128 columns that a CTA of the sums takes: what tensor memory holds of the rank.
constexpr int sum_blocks(int rank) { return rank <= 64 ? 2 : 1; }

struct PassCut {
    int splits;   // CTAs that share a tile
    bool halved;  // tiles of 64 rows, not 128
};

// How a pass is cut up: tiles of 128 or 64 rows, and the CTAs that share one, one CTA to an SM.  A CTA costs some 3 us beside its rows, 3 more where sums
// are joined over a cluster, and takes its bytes at 60 a ns at best (12 where they are not whole vectors) and at its share of HBM's 6600; weights come
// from L2.  Without a result (out_bytes = 0) there is the first product alone to share.
inline PassCut cut_pass(int64_t rows, int64_t adapters, int rank, int from, int to, int base_bytes, int out_bytes, bool vec)
{
    if (out_bytes == 0) to = 0;
    PassCut cut{1, false};
    double best = 1e30;
    const int parts = static_cast<int>(blocks_of(from, P_STEP)), chunks = static_cast<int>(blocks_of(to, P_COLS));
    for (int h = 0; h < 2; ++h)
        for (int splits = 1; splits <= 8; splits *= 2) {
            if (splits > 1 && splits > parts && splits > chunks) break;
            const int tile = TILE >> h;
            const int64_t ctas = tiles_about(rows, adapters, tile) * splits;
            const double held = splits == 8 ? 120.0 : splits == 4 ? 144.0 : 152.0;  // CTAs of clusters that the SMs hold at once
            const double waves = static_cast<double>(blocks_of(ctas, static_cast<int64_t>(held)));
            const double on = static_cast<double>(ctas) < held ? static_cast<double>(ctas) : held;
            const double from_each = static_cast<double>(from) / (splits < parts ? splits : parts), to_each = to ? static_cast<double>(to) / (splits < chunks ? splits : chunks) : 0.0;
            const double bytes = tile * (2.0 * from_each + (base_bytes + out_bytes) * to_each);
            const double weights = 2.0 * rank * (from_each + to_each);
            const double fast = vec ? 60.0 : 12.0, rate = 6600.0 / on < fast ? 6600.0 / on : fast;
            const double own = (bytes + weights) / fast / 1000.0, hbm = bytes / rate / 1000.0;
            const double us = waves * (3.0 + (splits > 1 ? 3.0 : 0.0) + (own > hbm ? own : hbm));
            if (us < best) {
                best = us;
                cut = {splits, h == 1};
            }
        }
    return cut;
}

struct SumCut {
    int da, db;  // tiles to a piece
};

// How many tiles a CTA takes for each gradient: as few as fill the SMs in whole waves, against some 4 us that a CTA costs beside its tiles'
// 1.2 us each (that of ranks up to 64; above, 3.5 would suit some sizes and spoil others): both gradients together, as where the pass leaves no SMs free, and
// then da's, which waits for the pass, once more.  12544 x 256 -> 1024, rank 16: 32.4 us, with the same pieces for both 36.9.
inline SumCut cut_sums(int64_t rows, int64_t adapters, int rank, int64_t cols, int64_t outs)
{
    const int columns = 128 * sum_blocks(rank);
    const int64_t tiles = tiles_about(rows, adapters, TILE);
    if (tiles == 0) return SumCut{1, 1};  // no rows
    const int most = static_cast<int>(tiles < SUM_TILES ? tiles : SUM_TILES);
    int64_t a_ctas[SUM_TILES + 1], b_ctas[SUM_TILES + 1];
    for (int i = 1; i <= most; ++i) {
        const int64_t pieces = blocks_of(tiles, i);
        a_ctas[i] = pieces * blocks_of(cols, columns);
        b_ctas[i] = pieces * blocks_of(outs, columns);
    }
    const auto waves = [](int64_t ctas) { return blocks_of(ctas, CARD_SMS); };
    const auto time = [](int each) { return 4.0 + 1.2 * each; };
    SumCut best{1, 1};
    double best_us = 1e30;
    for (int a = 1; a <= most; ++a) {
        const double own = static_cast<double>(waves(a_ctas[a])) * time(a);
        if (own >= best_us) continue;
        for (int b = a; b <= most; ++b) {  // fewer for db than for da do not shorten the two
            const double us = static_cast<double>(waves(a_ctas[a] + b_ctas[b])) * time(b) + own;
            if (us < best_us) best = {a, b}, best_us = us;
        }
    }
    // but cost nothing where they need no further wave, together or alone
    const int64_t whole = waves(a_ctas[best.da] + b_ctas[best.db]), alone = waves(b_ctas[best.db]);
    while (best.db > 1 && waves(a_ctas[best.da] + b_ctas[best.db - 1]) == whole && waves(b_ctas[best.db - 1]) == alone) --best.db;
    return best;
}

}  // namespace ad
}  // namespace sgb
