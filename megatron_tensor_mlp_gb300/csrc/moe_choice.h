// Which kernel takes a product grouped by expert (host only).  The row ranges are on the device: the rules go by sizes alone and
// take the rows as spread over the experts.  They were fitted on up to 64 experts; a plan that is skewed, or has more experts,
// changes what a choice costs, not what it computes.
#pragma once
#include <algorithm>
#include <cmath>
#include <cstdint>

namespace tpmlp {
namespace moe {

enum Kernel { FEW, NARROW, WIDE };
constexpr int64_t kFeatures = 256, kGatedFeatures = 128;  // of a pair's narrow tile (gated: gate and up features of each)
constexpr int64_t kContraction = 64;                      // of a stage

inline int64_t blocks(int64_t n, int64_t size) { return (n + size - 1) / size; }

// Whether a product runs on the few-rows kernel.  The row ranges are on the device, so this goes by the tiles that the pairs
// would have if the rows were spread over the experts: where they fill about half of the pairs, or, with at most 16 rows an
// expert, up to four rounds of them (which do not come out even).  4 tokens, 8 of 64 experts, 1024 x 8192 gated (256 tiles):
// 28.0 us, pairs 33.8; 4096 x 1024 (32 tiles): 14.6, 26.0; 128 rows on 8 experts of that size 16.6, 23.8; 666 rows (40 tiles)
// 19.3, 24.7.  But 128 rows on 34 of 64 experts, gated (2112 tiles): 112, pairs 91; 1024 rows on 16 experts, 4096 x 1024 (80
// tiles): 36.1, 27.4.  Gradients of the inputs: 30 rows on 8 experts, 3840 -> 624 (24 tiles) 11.5, 22.3; 1000 rows, 2048 -> 1024
// (44 tiles) 17.1, 15.8.  Through the gated activation a thread handles a feature's pre-activations one by one, so for fewer
// tiles: 8 rows, 5120 -> 4096 (128 tiles) 43, 61; 1400 rows, 1024 -> 512 (26 tiles) 14.7, 17.1; but 600 rows on 64 experts,
// 1024 -> 1024 (264 tiles) 33, 27; 400 rows on 8 (36 tiles) 14.6, 13.5.
inline bool few_rows(int64_t rows, int64_t experts, int64_t m_blocks, int pairs, bool gated_dx = false) {
    const int64_t tiles = m_blocks * (std::min(rows, experts) + rows / 256);
    if (gated_dx) return rows <= 8 * experts ? tiles <= 2 * pairs : 20 * tiles <= 8 * pairs;
    return rows <= 16 * experts ? tiles <= 4 * pairs : 20 * tiles <= 11 * pairs;
}

// Whether tiles of twice the size keep the pairs as busy: they come in half as many rounds, or in so many that the last, partly
// empty one weighs little.  (36 of them instead of 72, on 76 pairs: 1.6 times as long; 128 instead of 256: 0.95; 102 instead of
// 204, two rounds for three: 1.16.)
inline bool busy(double wide, double narrow, int pairs) {
    const double w = std::ceil(wide / pairs), n = std::ceil(narrow / pairs);
    return 2 * w <= n || w >= 3;
}

// Whether the rows kernel runs on wide tiles (m_blocks: of narrow ones), if they keep the pairs busy.  For gathered rows, whose
// copies they halve: 16384 rows on 8 experts, 5120 x 8192 735 us, narrow 811; 8192 rows on 64 experts, 1024 x 2048 gated 57, 79;
// in 30 of 33 other cases 2-18 % less.  For rows in order where much is done for each byte, since a tile's epilogue is not
// hidden: 6000 rows on 8 experts, 5120 x 8192 gated 314, 342, plain 287, 318, its gradient of the inputs 330, 362; but 16384
// rows on 16 experts, 1024 x 4096 gated 102, 98, plain 103, 92, and 8192 rows on 8 experts, 2048 x 4096 gated 94, 97, plain 98, 95.
inline bool wide_tiles(int64_t rows, int64_t experts, int64_t m_blocks, int64_t k_blocks, bool gated, bool gathered, int pairs) {
    if (!gathered && k_blocks < (gated ? 32 : 64)) return false;
    // tiles of tokens: of one expert, or, as the ranges are on the device, with the last of each half full
    const double t = experts == 1 ? static_cast<double>((rows + 255) / 256) : rows / 256.0 + std::min(experts, rows) / 2.0;
    return busy(t * ((m_blocks + 1) / 2), t * m_blocks, pairs);
}

// Y = X W, features N (gated: N / 2 and as many up features).
inline Kernel forward_kernel(int64_t rows, int64_t experts, int64_t K, int64_t N, bool gated, bool gathered, int pairs) {
    const int64_t m = gated ? blocks(N / 2, kGatedFeatures) : blocks(N, kFeatures);
    if (few_rows(rows, experts, m, pairs)) return FEW;
    return wide_tiles(rows, experts, m, blocks(K, kContraction), gated, gathered, pairs) ? WIDE : NARROW;
}

// dX = dY W^T, features K; through the gated activation no wide tiles, whose epilogue has no second staging.
inline Kernel dx_kernel(int64_t rows, int64_t experts, int64_t K, int64_t N, bool gated, int pairs) {
    const int64_t m = blocks(K, kFeatures);
    if (few_rows(rows, experts, m, pairs, gated)) return FEW;
    return !gated && wide_tiles(rows, experts, m, blocks(N, kContraction), false, false, pairs) ? WIDE : NARROW;
}

// dW = X^T dY.  Wide tiles for gathered rows (see wide_tiles; 16384 rows on 8 experts, 5120 x 8192: 793 us, narrow 1230) and where
// contractions are long (the same in order: 739, 804; 8192 rows on 16 experts, 4096 x 2048: 119, 116), if they keep the pairs busy.
inline Kernel dw_kernel(int64_t rows, int64_t experts, int64_t K, int64_t N, bool gathered, int pairs) {
    const double m = static_cast<double>(experts) * blocks(K, 256);
    return (gathered || rows >= 1280 * experts) && busy(m * blocks(N, 512), m * blocks(N, 256), pairs) ? WIDE : NARROW;
}

}  // namespace moe
}  // namespace tpmlp
