// Which kernel takes an MXFP4 product, and into how many parts its K loop is split (host only).
#pragma once
#include <algorithm>
#include <cstdint>

namespace tpmlp {
namespace mx {

inline constexpr int kMaxSplit = 8;

// What runs at once on a device: CTA pairs, and clusters of s single CTAs with one CTA an SM (with two CTAs an SM,
// twice as many).  Not every SM is in a cluster: on a GB300 of 152 SMs there are 76 clusters of two, 46 of three, 36 of
// four and 15 of eight.
struct Machine {
    int pairs;
    int clusters[kMaxSplit + 1];
};

// A single CTA's epilogue: chunks of 32 columns in `parts` accumulators each, and shared memory for the partial sums that
// it receives from the other CTAs of a split tile.
struct Exchange {
    int chunks, parts, room;

    // Bytes that one CTA of a split tile receives: the chunks it finishes, from every other CTA.
    int bytes(int split, int rows) const {
        const int owners = std::min(split, chunks);
        return (chunks + owners - 1) / owners * (split - 1) * parts * 128 * rows;
    }
    bool fits(int split, int rows, int kb) const { return split <= kb && bytes(split, std::min((rows + 31) / 32 * 32, 128)) <= room; }
};

struct Extent {
    int64_t M, tiles, pair_tiles;  // rows; tiles of a single CTA (128 x 128) and of a pair (256 x 256)
    int kb;                        // ring stages of K, 256 values each
};

struct Choice {
    bool pair;
    int split;
    double us;
};

constexpr double kPairStart = 4.0;
inline double pair_tile_us(int kb) { return 0.265 * kb + 1.05; }

// By the expected time in microseconds, weights out of L2:
//   pairs    4 + waves (0.265 kb + 1.05)
//   single   4 + 0.34 kb                          at most one CTA an SM,
//            5.3 + 0.38 kb                        at most two (4.8 + 0.3 kb with at most 32 rows: they copy less of A),
//            2.5 + waves (0.38 kb + 3)            else
//   split    the same of kb / split, and 1.5 (one CTA an SM) or 2.3 (two) log2(split) for the exchange; only where all
//            clusters run at once, since a second wave of a few of them takes as long as the first
// Against one GB300's times of 1581 products in every form (1 to 2048 rows, N 768 to 20480, K 1024 to 20480) the choice
// costs 1 % on average against the best form, more than 10 % in 19 of them and 17 % at most (2048 x 768 x 4096: pairs 8.7,
// single 7.5).  Both sides of the limits, 128 rows and K 20480: 45 tiles, three ways 18.8 and four 20.2; 48 tiles, two
// clusters of three too many for one CTA an SM, 20.5 and 20.9; 64 tiles, two ways 24.0, three 23.9, four 23.9; 76 tiles, four
// clusters of four too many for two CTAs an SM, 25.8, 25.8 and 37.0.  512 x 5120 x 20480: pairs 26.7, single 33.7, two
// ways 41.6; 800 rows: single 35.9, pairs 48.2 (80 tiles, two waves).
// At most 32 rows: single CTAs, which copy no more rows of A than there are (4 x 40960 x 5120: 23 against 31).
inline Choice choose(const Machine& on, const Exchange& ex, const Extent& p) {
    const int rows = static_cast<int>(std::min<int64_t>(p.M, 128));
    const bool few = p.M <= 32;
    Choice c{false, 1, 0.0};
    for (int s : {1, 2, 3, 4, 8}) {
        const int64_t at_once = on.clusters[s];
        if (s > 1 && (p.tiles > 2 * at_once || !ex.fits(s, rows, p.kb))) break;
        const int64_t waves = at_once > 0 ? (p.tiles + 2 * at_once - 1) / (2 * at_once) : p.tiles;
        const double k = static_cast<double>(p.kb) / s, log = s == 3 ? 1.6 : s == 8 ? 3.0 : s / 2;
        const double t = p.tiles <= at_once ? 4.0 + 0.34 * k + 1.5 * log
                         : waves > 1        ? 2.5 + waves * (0.38 * k + 3.0)
                         : few              ? 4.8 + 0.3 * k + 2.3 * log
                                            : 5.3 + 0.38 * k + 2.3 * log;
        if (s == 1 || t < c.us) {
            c.us = t;
            c.split = s;
        }
    }
    if (on.pairs > 0 && !few) {
        const int64_t waves = (p.pair_tiles + on.pairs - 1) / on.pairs;
        const double t = kPairStart + waves * pair_tile_us(p.kb);
        if (t < c.us) {
            c.us = t;
            c.pair = true;
        }
    }
    return c;
}

}  // namespace mx
}  // namespace tpmlp
