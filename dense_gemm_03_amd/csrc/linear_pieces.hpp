// Which tile, or which piece of one, a block of a linear-layer kernel works on.
// Plain C++, for the host and the device.
#pragma once

namespace dg {

// The list position and the piece of this block, the j-th of its XCD, in a list
// of n tiles and `small` small ones behind them.
//
// One block of a large tile fills a compute unit, so n tiles take n / slots
// rounds of the XCD's `slots` units, and a last round that is not full leaves
// units idle for a whole tile's time.  If its r = n % slots tiles make no more
// than one round of quarters or of halves, they are cut into those (K = 4096 on
// 256 units: 64 tiles take 38 us in quarters, 128 tiles 65 in halves, 77 whole
// and 82 in two rounds of quarters).  A small tile is two quarters.  slots == 0
// (entries without pieces, or a device of fewer than 8 units): every tile whole,
// the small ones too.  There are at most 3/4 slots + small pieces more than tiles.
struct Piece {
    int at;       // position in the list, or -1
    int which;    // -1: the whole tile; quarter 0 .. 3: row half + 2 * column half; 4, 5: row half
};

// Inlined whatever its size: behind a call the compiler would take the place for
// one that differs from lane to lane, and addresses made from it with it.
__attribute__((always_inline)) constexpr inline Piece xcd_piece(int j, int n, int small, int slots)
{
    if (slots == 0) return {j < n + small ? j : -1, -1};
    const int r = n % slots, of = 4 * r <= slots ? 4 : 2 * r <= slots ? 2 : 1;
    const int whole = of > 1 ? n - r : n;
    if (j < whole) return {j, -1};
    const int h = j - whole - of * (n - whole);   // among the small tiles' quarters
    if (h < 0) return {whole + (j - whole) / of, (j - whole) % of + (of == 2 ? 4 : 0)};
    return {h < 2 * small ? n + h / 2 : -1, h % 2 * 2};
}

}  // namespace dg
