// sv_lmhead_fp4_plan.h -- which shape of the 4-bit LM head a product takes (host code
// without CUDA, so that the rule can be asked by itself).
#pragma once

#include <cstdint>

namespace sv {

constexpr int kL4MaxNB = 192; // ids of a tile: 512 tensor-memory columns are 2 x 192 of sums and 2 x 64 of scales
constexpr int kL4Rows = 128;  // rows of a CTA's tile

inline int64_t l4_ceil(int64_t a, int64_t b) { return (a + b - 1) / b; }

// How a product is cut: a function of (M, V).  A stage (256 hidden dims) of a tile
// costs an SM the largest of
//   the MMAs' time, 2 cycles an id and row tile (4 steps of 64 dims);
//   what it loads, 128 bytes and 16 of scales for each row of h and of W, at the rate
//   that was measured of each shape: 55 bytes a cycle for lone CTAs, 45 for pairs, 42
//   for pairs with two row tiles (whose accumulators are not read behind the next
//   tile's MMAs: half a tile more at the end);
//   with one row tile, where W comes from memory once, 23 bytes a cycle for W.
// d is not looked at: what a tile costs besides its stages (40 cycles a stage here) was
// fitted at d 4096, and weighs more at small d, where the choice was measured at M 1024,
// V 32003, d 1056 only.  Narrower tiles on ties: they reach more SMs.  The three shapes, replayed, d 4096
// (two row tiles, pairs, lone CTAs; the rule's choice starred):
//   V 128256: M 384 98* 105 101 us; M 576 182 154 149*; M 1024 184* 204 244; M 2304 397* 462 519;
//   V 32000: M 257 37 35 31*; M 576 48 44 45*; M 1024 60 56* 65; M 2304 113* 116 135;
//   M 131, V 128256: pairs 59*, lone CTAs 69.
struct Lm4Plan {
    bool pair;
    int32_t H;          // row tiles that share a pair's tile of W
    int32_t RT, MT;     // row tiles, groups of H of them
    int32_t NT, NB;
};

inline Lm4Plan lm4_plan(int64_t M, int32_t V, int32_t sms)
{
    Lm4Plan p = {};
    const int64_t rows = M < kL4Rows ? M : kL4Rows;
    int64_t best = INT64_MAX;
    for (int shape = M > 2 * kL4Rows ? 2 : (M > kL4Rows ? 1 : 0); shape >= 0; --shape) { // H 2, pair, lone CTA
        const bool pair = shape > 0;
        const int32_t H = shape == 2 ? 2 : 1;
        const int64_t units = pair ? sms / 2 : sms, rate = shape == 2 ? 42 : (pair ? 45 : 55);
        const int32_t rt = static_cast<int32_t>(l4_ceil(M > 0 ? M : 1, pair ? 2 * kL4Rows : kL4Rows));
        const int32_t mt = static_cast<int32_t>(l4_ceil(rt, H));
        int64_t low = INT64_MAX;
        int32_t NB = 0;
        for (int32_t nb = kL4MaxNB; nb >= 64; nb -= 64) {
            const int64_t w = 144 * (pair ? nb / 2 : nb);
            auto stage = [&](int64_t h) { // of a group of h row tiles
                int64_t c = (h * 144 * rows + w) / rate;
                c = c > 2 * nb * h ? c : 2 * nb * h;
                return mt == 1 && c < w / 23 ? w / 23 : c;
            };
            // the mean of a unit's tiles; where the units are a multiple of the groups, some units
            // get full groups only
            const int64_t tile =
                (units % mt == 0 ? stage(H) : (rt / H * stage(H) + (rt % H ? stage(1) : 0)) / mt) + 40;
            const int64_t cost = l4_ceil(mt * l4_ceil(V, nb), units) * tile + (H == 2 ? tile / 2 : 0);
            if (cost <= low) {
                low = cost;
                NB = nb;
            }
        }
        if (low < best) { // two row tiles, then a pair, on ties
            best = low;
            p.pair = pair;
            p.H = H;
            p.RT = rt;
            p.MT = mt;
            p.NB = NB;
        }
    }
    p.NT = static_cast<int32_t>(l4_ceil(V, p.NB));
    return p;
}

} // namespace sv
