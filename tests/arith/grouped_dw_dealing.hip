/*
 * How gemm_grouped_dw deals the tiles of its output to workgroups, run on the
 * host with the library's own plan and dealing (csrc/spg_grouped_dw.h): every
 * workgroup's list is walked as the kernel walks it, up to its first place
 * past the last expert, and every (expert's place, part of its rows, row of
 * tiles, tile) has to come up exactly once.
 *
 * Reads "experts N K rows" a line; prints, for each, tiles, tiles that no
 * workgroup has, tiles dealt more than once, and the plan (parts of the rows,
 * rows of tiles a unit and parts of a row of tiles, as powers of two).
 */
#include <stdio.h>
#include <string.h>

#include <vector>

#include "spg_grouped_dw.h"

using namespace spg;

int main()
{
    long E, N, K, R;
    while (scanf("%ld %ld %ld %ld", &E, &N, &K, &R) == 4) {
        spg_grouped_dw_desc d;
        memset(&d, 0, sizeof(d));
        d.rows = d.x_rows = R;
        d.N = N;
        d.K = K;
        d.experts = (int32_t)E;
        GroupedDwArgs a;
        memset(&a, 0, sizeof(a));
        a.E = (int32_t)E;
        plan_grouped_dw(d, a);
        const unsigned grid = dw_grid(a);
        const size_t tiles = (size_t)E * a.slices * a.tiles_n * a.tiles_k;
        std::vector<unsigned char> seen(tiles);
        size_t twice = 0, missing = 0;
        for (unsigned b = 0; b < grid; ++b)
            for (uint32_t k = 0;; ++k) {
                const DwPlace p = dw_place(a, b & 7u, dw_item(grid, b, k));
                if (p.place >= (uint32_t)E) break;
                const size_t at = (((size_t)p.place * a.slices + p.slice) * a.tiles_n + p.tn) * a.tiles_k + p.tk;
                if (p.slice >= (uint32_t)a.slices || p.tn >= a.tiles_n || p.tk >= a.tiles_k || seen[at])
                    ++twice;
                else
                    seen[at] = 1;
            }
        for (size_t i = 0; i < tiles; ++i) missing += !seen[i];
        printf("%ld %ld %ld %ld: tiles %zu missing %zu twice %zu plan %d %d %d\n", E, N, K, R, tiles, missing, twice, a.slices,
               a.unit_n, a.unit_k);
    }
    return 0;
}
