// Every read of h that adapter_up makes for its operand, for every pair of an adapter's rank and the room for ranks, counted
// against where adapter_down wrote.  Built and called by test_adapter_index.py.
#include <cstdint>
#include <cstdio>
#include <vector>

#include "gdn_adapter_index.cuh"

using namespace gdn;

static char g_first[256];

static void note(long& bad, const char* what, int room, int rank, int n, int range, int column, size_t index)
{
    if (bad++ == 0) std::snprintf(g_first, sizeof g_first, "%s: room %d rank %d tokens %d range %d column %d index %zu", what, room, rank, n, range, column, index);
}

extern "C" const char* first_mistake() { return g_first; }

// unguarded: the mistake to be found, a block of columns that reads all its rows whatever the adapter's rank
extern "C" long mistakes(int unguarded)
{
    long bad = 0;
    g_first[0] = 0;
    const int ctas = 152;
    for (int room = 8; room <= 128; room += 8) {
        const int built = room <= 16 ? 16 : room <= 32 ? 32 : room <= 64 ? 64 : 128;  // columns of the operand
        const int mine = built / kAdapterParts, block = mine < 8 ? mine : 8;
        for (int rank = 1; rank <= room; ++rank) {
            const Steps steps(rank);
            std::vector<int> times(room, 0);
            for (int part = 0; part < kAdapterParts; ++part)
                for (int j = 0; j < mine; j += block) {
                    const int column = part * mine + j;
                    const OperandRows rows(steps, rank, column);
                    const int left = unguarded && rows.at >= 0 ? block : rows.left;
                    for (int e = 0; e < block; ++e) {
                        const int row = steps.row_of(column + e);
                        if (e >= left) {  // a zero
                            if (row >= 0 && row < rank) note(bad, "a row is left out", room, rank, 0, 0, column + e, row);
                            continue;
                        }
                        if (row != rows.at + e) note(bad, "not the column's row", room, rank, 0, 0, column + e, rows.at + e);
                        if (rows.at + e < rank) ++times[rows.at + e];
                        for (int n : {1, 2, 31, 32, 127, 128})
                            for (int range : {-1, 0, ctas - 1}) {  // -1: the range that the tile begins in
                                const int T = 1000 + n, start = 1000;  // the last tile
                                const size_t place = h_place(T, room, range, start, range < 0), all = ((size_t)T + (size_t)ctas * kAdapterTile) * room;
                                for (int token : {0, n - 1}) {
                                    const size_t index = place + (size_t)(rows.at + e) * n + token;
                                    if (index >= all) note(bad, "behind the workspace", room, rank, n, range, column + e, index);
                                    // adapter_down writes rows below the rank, the tile's tokens of each
                                    else if (index >= place + (size_t)rank * n) note(bad, "not written for this tile", room, rank, n, range, column + e, index);
                                }
                            }
                    }
                }
            for (int r = 0; r < rank; ++r)
                if (times[r] != 1) note(bad, "a row enters the product not once", room, rank, 0, 0, r, times[r]);
            // the steps' rows of `up` are the adapter's, rounded up to 8s, or to the 16 that a step takes of at most 8
            for (int s = 0; s < steps.count; ++s)
                if (steps.first_row(s) < 0 || (rank > 8 && steps.first_row(s) + 16 > ((rank + 7) & ~7))) note(bad, "rows that nobody copied", room, rank, 0, 0, s, 0);
        }
    }
    return bad;
}
