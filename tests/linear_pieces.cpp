// Every tile of either list is worked on once, whole or in pieces that make it
// up, by a block of the grid: for all lists of up to 70 tiles and 9 small ones
// and up to 33 units.
#include "linear_pieces.hpp"

#include <cstdio>
#include <vector>

int main()
{
    for (int slots = 0; slots <= 33; ++slots)
        for (int n = 0; n <= 70; ++n)
            for (int small = 0; small <= 9; ++small) {
                const int blocks = n + small + (slots * 3 + 3) / 4 + small;
                std::vector<int> seen(n + small, 0);   // which quarters
                for (int j = 0; j < blocks + 40; ++j) {
                    const dg::Piece p = dg::xcd_piece(j, n, small, slots);
                    if (p.at < 0) continue;
                    const int parts = p.which < 0 ? 15 : p.which < 4 ? 1 << p.which : p.which == 4 ? 5 : 10;
                    if (j >= blocks || p.at >= n + small || p.which > 5 || (seen[p.at] & parts)) {
                        std::printf("slots %d, %d tiles, %d small: block %d has place %d, piece %d\n", slots, n, small,
                                    j, p.at, p.which);
                        return 1;
                    }
                    seen[p.at] |= parts;
                }
                for (int t = 0; t < n + small; ++t)
                    // of a small tile the upper half of the rows is all there is
                    if ((t < n ? seen[t] : seen[t] & 5) != (t < n ? 15 : 5)) {
                        std::printf("slots %d, %d tiles, %d small: tile %d is not covered\n", slots, n, small, t);
                        return 1;
                    }
            }
    return 0;
}
