// q4_mx_runs.cuh -- how the k units of all output tiles of a product are cut
// into one run for each CTA or pair (q4_mx_gemm.cu).  Whole numbers only: every
// role of every CTA works the cut out for itself and waits on what the others
// make of it, so it must not depend on how a compiler rounds or contracts.  No
// CUDA header is needed: the tests compile it for the host.
#pragma once

#include <stdint.h>

#include "q4_wait.cuh"

namespace q4 {

// What the cut of few tiles goes by, in ns: `whole` for all of a tile's k, and
// for adding its parts up `join` and `part` for each sharer.  `sharers`: the
// number that makes whole / sharers + part * sharers least.
struct RunCost {
    int whole, join, part, sharers;
};

inline RunCost run_cost(int64_t whole, int join, int part, int Ku) {
    RunCost c{static_cast<int>(whole), join, part, 1};
    while (c.sharers < Ku && static_cast<int64_t>(c.sharers + 1) * (c.sharers + 1) * part <= whole) ++c.sharers;
    return c;
}

// With fewer output tiles than groups (CTAs or pairs), as many groups share a
// tile as make the time least: its k, divided by the sharers, plus adding the
// parts up.  With one group a tile nothing is added up.  Measured on B200 (us;
// equal runs over all groups, whole tiles): 64 tokens, 4096 x 4096 17.1, 13.5;
// 100 tokens 23.4, 15.8; 40 tokens, 2048 x 2048 11.3, 8.9; 12 tokens 11.0, 10.6.
struct RunCut {
    int units, ctas, each, more;  // CTAs below `more` take one unit beyond `each`
    Q4_HOST_DEVICE RunCut(int tiles, int groups, int Ku, const RunCost& cost) {
        units = tiles * Ku;
        ctas = groups < units ? groups : units;
        if (ctas < 1) ctas = 1;
        if (tiles > 0 && tiles < groups) {
            if (tiles * cost.sharers < groups) ctas = tiles * cost.sharers;
            // whole <= whole / n + join + part * n for n = ctas / tiles sharers
            const int64_t c = ctas, t = tiles;
            if (cost.whole * c * t <= cost.whole * t * t + cost.join * c * t + cost.part * c * c) ctas = tiles;
        }
        each = units / ctas;
        more = units - each * ctas;
    }
    // the first unit of CTA c's run, which ends where the next begins
    Q4_HOST_DEVICE int start(int c) const { return each * c + (c < more ? c : more); }
    // the CTA whose run holds unit v
    Q4_HOST_DEVICE int owner(int v) const {
        const int longer = more * (each + 1);
        return v < longer ? v / (each + 1) : more + (v - longer) / each;
    }
};

}  // namespace q4
