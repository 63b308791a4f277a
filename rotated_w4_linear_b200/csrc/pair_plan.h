// Which form of the CTA-pair GEMM (gemm_pair_sm100.cu) a product takes: plain
// host arithmetic on its sizes and on how many clusters are resident at once.
#pragma once

#include <algorithm>

namespace paro {

constexpr int kMaxPairs = 4;                            // pairs that may split a tile's channels (cluster of 8)

struct PairPlan {
    long cost = 0;              // SM cycles
    int form = 0;               // 64, 128: tiles of as many tokens, channels split; 256: persistent
    int bn = 0;                 // tokens per tile: the form's, or for 256 a multiple of 32 up to it
    int pairs = 1;              // pairs per cluster
};

// Tokens of a tile of the 256-token form: the batch in as few tiles as it
// takes, of equal size in steps of 32 (333 tokens: two tiles of 192, not of 256).
inline int balanced_tile(int T) {
    const int tiles = (T + 255) / 256;
    return (((T + tiles - 1) / tiles) + 31) / 32 * 32;
}

// What a product of mt 256-row tiles, T tokens and nk 128-channel stages takes
// in one form, in SM cycles: rounds of tiles that do not fit at once, times a
// tile's stages and its start and end. resident(form, pairs): clusters of
// `pairs` CTA pairs on the device at once. The figures are
// measured (4096 -> 28672 and 14336 -> 4096, 17 to 512 tokens): a stage of the
// 256-token form 1250 (less for smaller tiles, down to the dequantisation's
// 900) and a tile's change-over 4000; a stage of the split form
// 800, its start, exchange and end 11000, 1500 more with several pairs. Taking
// the cheaper one, 4096 -> 4096 at 256 tokens runs in the split form (32 tiles
// of 128 tokens, two pairs each) and 4096 -> 28672 at 256 in the other.
template <class Resident>
PairPlan plan_form(int form, int mt, int T, int nk, const Resident& resident) {
    const bool split = form < 256;
    PairPlan best;
    best.form = form;
    best.bn = split ? form : balanced_tile(T);
    const int tiles = mt * ((T + best.bn - 1) / best.bn);
    for (int p = 1; p <= (split ? std::min(kMaxPairs, nk) : 1); ++p) {
        const int n = std::max(1, resident(form, p));
        const long rounds = (tiles + n - 1) / n, stages = (nk + p - 1) / p;
        const long cost = split ? rounds * (stages * 800 + 11000 + (p > 1 ? 1500 : 0))
                                : rounds * (stages * std::max(900, 1250 * best.bn / 256) + 4000) + 6000;
        if (best.cost == 0 || cost < best.cost) {
            best.cost = cost;
            best.pairs = p;
        }
    }
    return best;
}

// 17 to 64 tokens: tiles of 64; to 128: tiles of 128; above: the cheaper of
// the split form with tiles of 128 and the persistent one with tiles of 256.
template <class Resident>
PairPlan plan_pairs(int mt, int T, int nk, const Resident& resident) {
    const PairPlan split = plan_form(T <= 64 ? 64 : 128, mt, T, nk, resident);
    if (T <= 128) return split;
    const PairPlan whole = plan_form(256, mt, T, nk, resident);
    return split.cost < whole.cost ? split : whole;
}

}  // namespace paro
