// gdn_adapter_index.cuh -- where a tile's h lies in the adapters' workspace, and which of it each column of adapter_up's
// operand reads.  Plain C++ too: the host's tests go through every pair of ranks.
#pragma once

#include <cstddef>

#ifdef __CUDACC__
#define GDN_HD __host__ __device__ __forceinline__
#else
#define GDN_HD inline
#endif

namespace gdn {

constexpr int kAdapterTile = 128;  // tokens
constexpr int kAdapterTeams = 2;   // of adapter_up's workers
constexpr int kAdapterParts = kAdapterTeams * 2;  // threads that share a row of the operand

// The h of one range's part of a tile that begins at token `start`: [rank][the tile's tokens], in the tokens' places for the
// range that the tile begins in, in a place of its own behind all tokens for every other.
GDN_HD size_t h_place(int T, int room, int range, int start, bool begins)
{
    return (begins ? (size_t)start : (size_t)T + (size_t)range * kAdapterTile) * room;
}

// A tile's products take 16 rows of `up` a step.  Where the last step has only 8 rows of its own (the rank rounded up to
// 8s) it takes the 8 in front of them again, with zeros for their h: rows behind the rank may not be finite.
struct Steps {
    int count, last;  // steps; the first row of the last one
    GDN_HD explicit Steps(int rank)
    {
        const int rows = (rank + 7) & ~7;
        count = (rows + 15) / 16;
        last = rows > 8 ? rows - 16 : 0;
    }
    GDN_HD int first_row(int step) const { return step == count - 1 ? last : step * 16; }
    // the row whose h stands in column j of the operand; -1: none
    GDN_HD int row_of(int j) const
    {
        if (j < (count - 1) * 16 || last == (count - 1) * 16) return j;
        return j >= count * 16 ? -1 : j >= count * 16 - 8 ? j - 8 : -1;
    }
};

// What a block of columns from `column` on (up to 8, which stand in one step's half) reads: rows `at` and the ones behind it,
// as many as the adapter's own rank leaves (none or fewer: zeros).  Rows behind the rank lie in another tile's place, or
// behind the workspace.
struct OperandRows {
    int at, left;
    GDN_HD OperandRows(const Steps& steps, int rank, int column) : at(steps.row_of(column)), left(at >= 0 ? rank - at : 0) {}
};

}  // namespace gdn
