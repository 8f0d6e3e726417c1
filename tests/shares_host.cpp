// The walk of cached_attn_kernel's CTAs along a line of units, on the host, with the kernel's own arithmetic
// (csrc/shares.cuh): which parts are written, and which the joins count.
#include <cstdint>
#include <vector>

#include "shares.cuh"

using namespace vggt;

// 0, or what is wrong: 1 a key tile not covered once and in order, 2 a join that counts a part that nobody writes,
// 3 a part that is written and not joined, 4 a workspace slot written twice, 5 a unit without keys not dealt with
// once, 6 a share outside the line.
extern "C" int walk(int n_units, const int *kind, const int *tiles, int shift, int grid)
{
    std::vector<int> begin(n_units + 1, 0);
    for (int u = 0; u < n_units; ++u)
        begin[u + 1] = begin[u] + unit_points(kind[u], tiles[u], shift);
    const Shares shares(begin[n_units], shift, grid);
    if (shares.ctas < 1 || shares.ctas > grid || shares.start(0) != 0 || shares.start(shares.ctas) != begin[n_units])
        return 6;
    std::vector<int> done(n_units, 0), parts(n_units, 0), seen(n_units, 0), empty(n_units, 0);
    std::vector<int> first(n_units, -1);
    std::vector<int> wrote(2 * grid, 0);
    std::vector<std::vector<int>> at(n_units);  // CTAs that wrote a part of the unit
    int u0 = 0;
    for (int cta = 0; cta < shares.ctas; ++cta) {
        const int w0 = shares.start(cta), w1 = shares.start(cta + 1);
        if (w1 < w0 || w1 > begin[n_units])
            return 6;
        while (u0 < n_units && begin[u0 + 1] <= w0)
            ++u0;
        for (int u = u0; u < n_units && begin[u] < w1; ++u) {
            const int x0 = w0 > begin[u] ? w0 - begin[u] : 0;
            const int x1 = (w1 < begin[u + 1] ? w1 : begin[u + 1]) - begin[u];
            if (x1 <= x0)
                continue;
            if (tiles[u] == 0) {
                empty[u] += x0 == 0;
                continue;
            }
            const int k0 = tiles_before(kind[u], tiles[u], x0, shift);
            const int n = tiles_before(kind[u], tiles[u], x1, shift) - k0;
            if (n == 0)
                continue;
            if (n < 0 || k0 != done[u])
                return 1;
            done[u] += n;
            if (n < tiles[u]) {
                int &slot = wrote[2 * cta + (k0 == 0)];
                if (slot++)
                    return 4;
                at[u].push_back(cta);
                if (k0 == 0) {
                    first[u] = cta;
                    parts[u] = shares.last(cta, begin[u + 1]) - cta + 1;
                }
            }
        }
    }
    for (int u = 0; u < n_units; ++u) {
        if (tiles[u] == 0) {
            if (empty[u] != 1)
                return 5;
            continue;
        }
        if (done[u] != tiles[u])
            return 1;
        if (parts[u] > static_cast<int>(at[u].size()))
            return 2;
        if (parts[u] < static_cast<int>(at[u].size()))
            return 3;
        for (int c = 0; c < parts[u]; ++c)
            if (at[u][c] != first[u] + c)
                return 2;
    }
    return 0;
}
