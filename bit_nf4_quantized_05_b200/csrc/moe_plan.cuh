// moe_plan.cuh -- host side of the experts kernel: how many warps share a work
// item. Plain C++, without CUDA.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>

namespace nf4 {

constexpr int kMoeChunk = 8;                       // tokens of one work item
constexpr int kMoeWarps = 16;                      // of a CTA

// Expected number of chunks (up to kMoeChunk tokens of one expert) of a router that
// spreads its tokens evenly: E times the mean of ceil(n / kMoeChunk), n the tokens of an
// expert, binomial in M tokens of probability top_k / E. How many there are in a call,
// only the device knows.
inline double moe_expected_chunks(int M, int E, int top_k) {
    const double p = static_cast<double>(top_k) / E;
    if (p >= 1.0) return static_cast<double>(E) * ((M + kMoeChunk - 1) / kMoeChunk);
    double pn = std::pow(1.0 - p, M), mean = 0.0;
    for (int n = 1; n <= M; ++n) {
        pn *= static_cast<double>(M - n + 1) / n * (p / (1.0 - p));
        mean += pn * ((n + kMoeChunk - 1) / kMoeChunk);
    }
    return std::max(1.0, E * mean);
}

// Warps of a group: the choice with the smallest estimate of (items x (steps of
// a warp per item + 1) over the groups, plus 1.75 items of each kind for the uneven
// end), the 1 standing for what an item costs beside its steps. Small groups are ahead
// where there are many items (us with 4 / 8 / 16 warps: 64 tokens at 8 of 32 experts,
// 2048 x 1024, 112 / 115 / 149), larger ones where few items are left to the end (64 at
// 2 of 8, 59 / 50 / 55; 3 at 2 of 8, 5120 x 2112, 52 / 45 / 40). Over 46 measurements,
// 18 at shapes drawn after the 1.75 was set, the choice is 0.8% above the best of the three in
// the mean and 13% at worst (4 tokens at 2 of 96, 1408 x 3456: 16 warps 46, 8 warps 41); with
// the number of chosen experts for the chunks and 1 for the 1.75 it was 2.5% and 22%.
inline int pick_moe_group(double chunks, int64_t tiles_gu, int64_t steps_gu, int64_t tiles_dn, int64_t steps_dn, int sms) {
    int best = 4;
    double best_cost = -1;
    for (int gw : {4, 8, 16}) {
        const double groups = double(sms) * (kMoeWarps / gw);
        const double gu = double((steps_gu + gw - 1) / gw + 1), dn = double((steps_dn + gw - 1) / gw + 1);
        const double cost = (chunks * tiles_gu / groups + 1.75) * gu + (chunks * tiles_dn / groups + 1.75) * dn;
        if (best_cost < 0 || cost < best_cost) {
            best = gw;
            best_cost = cost;
        }
    }
    return best;
}

}  // namespace nf4
