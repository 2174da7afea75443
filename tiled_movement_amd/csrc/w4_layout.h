// What a wave of the 4-bit product (kernels_w4_gemm.hip) holds in LDS and where, in
// bytes from its own area's start.  Host code as well, so that a test can hold
// every read of every variant to what the same wave has written.
#pragma once

namespace swz {

// Which 8 values of k (of 16 in a block of 128) lane g = lane / 16 has in product s.
template <int GROUP>
constexpr int w4_unit_of(int s, int g) {
    if constexpr (GROUP == 128) return 4 * g + s;
    // words s and s + 2 exchanged between lanes g and g ^ 2: lanes 0, 1 keep the
    // first group's, lanes 2, 3 take theirs
    if constexpr (GROUP == 64) return 8 * (s / 2) + 4 * (g & 1) + 2 * (g / 2) + s % 2;
    // and words s and s + 1 between lanes g and g ^ 1
    return 4 * s + 2 * (g / 2) + (g & 1);
}

// MATS: weights (2 for a gated block); NB: 16 rows of each; XL: X's rows in fours.
template <int GROUP, bool ZERO, int MATS, int NB, int XL>
struct W4Layout {
    static constexpr int MB = XL < 4 ? 1 : XL / 4;             // blocks of 16 rows of X
    static constexpr int PER = 128 / GROUP, COLS = MATS * NB;  // groups of a block of k; blocks of 16 rows of either W
    // the scales and zero points of kRun groups, each row's behind the other's with a
    // gap; a block of W; of X
    static constexpr int kRun = 32, kScaleRow = 2 * kRun + 4, kZeroRow = kRun + 4, kZero = COLS * 16 * kScaleRow;
    static constexpr int kW = (kZero + (ZERO ? COLS * 16 * kZeroRow : 0) + 15) / 16 * 16, kX = kW + COLS * 1024;
    static constexpr int kRed = MB * COLS * 1024, kOwn = kX + XL * 1024;

    // Row r's (of 16) 16-byte piece c (of 4) of block o of W, and row r's unit u (of 16)
    // of block a of X: the rows of a fragment fall on different banks.
    static constexpr int w_at(int o, int r, int c) { return kW + o * 1024 + 16 * (4 * r + (c ^ (r / 4))); }
    static constexpr int x_at(int a, int r, int u) { return kX + a * 4096 + 16 * (16 * r + (u ^ r)); }
    // The row of X that is read for row r of a fragment.  Fewer than 16 are held where
    // XL < 4, and the others are those over again: their products are rows of
    // their own, which are not stored.
    static constexpr int x_row(int r) { return XL < 4 ? r % (4 * XL) : r; }
    static_assert(x_at(MB - 1, x_row(15), 15 ^ x_row(15)) + 16 == kOwn && w_at(COLS - 1, 15, 0) + 16 == kX,
                  "the last row's last unit ends the wave's area, the last piece of W the codes'");
};

}  // namespace swz
