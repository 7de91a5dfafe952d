// pair_schedule.cuh -- schedule of k_pair_gemm.  (Plain C++ too, so that a test can ask which schedule a
// shape gets.)
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace qlora {

// Most ways that a tile is split along K.
constexpr int kPairMaxSplit = 4;

// Pairs of SMs, tiles of 256 x 256 or (bf16) 256 x 128, and how many ways the tiles of an incomplete last
// wave are split along K.
struct PairSched {
    int bn = 256, pairs = 1, tail = 0, split = 1;
    size_t part_bytes = 0;         // fp32 partials of the split tiles
    int n_cnt = 0;                 // their tickets
    size_t cnt_bytes() const { return (static_cast<size_t>(n_cnt) * sizeof(int) + 255) & ~static_cast<size_t>(255); }
    size_t bytes() const { return part_bytes + cnt_bytes(); }
};

// The shortest by the measured costs in microseconds, on `slots` pairs of SMs.  A bf16 stage takes 0.27 on a
// 256-wide tile and 0.2 on a 128-wide one, joining two parts 7 (4) and each further part 1.  An MXFP4 tile
// is done in 5 to 20 us and is never split (4096^3: 49.9 us whole, 56.5 us with its last wave split in two).
inline PairSched pair_schedule(int64_t M, int64_t N, int64_t k_steps, bool mx, int64_t slots) {
    PairSched g;
    double best = 0;
    for (int bn = 256; bn >= (mx ? 256 : 128); bn -= 128) {
        const int64_t tiles = ((M + 255) / 256) * ((N + bn - 1) / bn), whole = tiles / slots, rem = tiles % slots;
        const double step = bn == 256 ? 0.27 : 0.2, join = bn == 256 ? 5 : 2;
        for (int c = 1; c <= (rem && !mx ? kPairMaxSplit : 1); ++c) {
            if (c > 1 && (c * rem > slots || c > k_steps)) break;
            const double t = step * static_cast<double>(k_steps * whole + (rem ? (k_steps + c - 1) / c : 0)) +
                             (c > 1 ? join + c : 0);
            if (best > 0 && t >= best) continue;
            best = t;
            g.bn = bn;
            g.split = c;
            g.tail = c > 1 ? static_cast<int>(rem) : 0;
            g.pairs = static_cast<int>(whole ? slots : rem * c);
        }
    }
    if (g.split > 1) {
        g.part_bytes = static_cast<size_t>(g.tail) * 8 * g.split * (g.bn * 8) * 16;
        g.n_cnt = g.tail * 8;
    }
    return g;
}

}  // namespace qlora
