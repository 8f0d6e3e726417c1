// shares.cuh -- how the attention over a paged cache is divided among the
// CTAs (see cached_attn_kernel.cuh): what a unit of work costs, which CTA does
// which of it, and how many parts a unit that is cut leaves.  Whole numbers
// only, and compiled by the host's compiler too: the tests run it there.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define VGGT_SHARES_FN __host__ __device__ __forceinline__
#else
#define VGGT_SHARES_FN inline
#endif

namespace vggt {

constexpr int kMaxCtas = 148;
enum : int { kTaskSingle = 0, kTaskPair = 1, kTaskFew = 2 };
// What a unit costs beside its steps (Q load, first score, epilogue), in
// steps, and the fewest steps a CTA is used for.  Measured over fourteen small
// and middle calls, geometric mean: (1, 4) for the last two 20.3 us, (3, 4)
// 19.1, (3, 3) 18.8, (3, 2) 18.9, (1, 1) 19.5, (6, 4) 19.1; 3, 10 and 16 for the
// first within 0.3% of 6.
constexpr int kUnitCost = 6, kFewUnitCost = 3, kMinSteps = 3;

// Points of a unit of `tiles` key tiles: a point is 2^shift steps.  A unit
// without keys counts one, so that some CTA writes its rows.
VGGT_SHARES_FN int unit_points(int kind, int tiles, int shift)
{
    const int steps = (kind == kTaskPair ? 2 * tiles : tiles) + (kind == kTaskFew ? kFewUnitCost : kUnitCost);
    return tiles == 0 ? 1 : ((steps - 1) >> shift) + 1;
}

// Key tiles of a unit before point x of it.
VGGT_SHARES_FN int tiles_before(int kind, int tiles, int x, int shift)
{
    int steps = (x << shift) - (kind == kTaskFew ? kFewUnitCost : kUnitCost);
    if (kind == kTaskPair)
        steps >>= 1;
    return steps < 0 ? 0 : (steps > tiles ? tiles : steps);
}

// `work` points in `ctas` shares as equal as they can be: share i starts at
// floor(i work / ctas).  A unit's parts are counted as one per CTA from its
// first part to its last, so no share in between may be without a key tile.
// Hence at least kMinSteps (3) steps each, which is a key tile of a pair
// wherever they lie, and at least one point, which for shift > 0 is that too:
// 2^shift steps from an even one.
struct Shares {
    int work, ctas, each, rest;

    VGGT_SHARES_FN Shares(int total, int shift, int grid) : work(total), ctas(grid)
    {
        const int64_t most = (static_cast<int64_t>(total) << shift) / kMinSteps;
        if (most < ctas)
            ctas = static_cast<int>(most);
        if (total < ctas)
            ctas = total;
        if (ctas < 1)
            ctas = 1;
        each = work / ctas;
        rest = work - each * ctas;
    }
    VGGT_SHARES_FN int start(int i) const { return i * each + i * rest / ctas; }
    // The share with the last point before `end`, a point behind share `first`'s start.
    VGGT_SHARES_FN int last(int first, int end) const
    {
        int i = static_cast<int>(static_cast<float>(end) * ctas / work) + 1;
        i = i < ctas - 1 ? i : ctas - 1;
        while (i > first && start(i) >= end)
            --i;
        return i;
    }
};

} // namespace vggt
