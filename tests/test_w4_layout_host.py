"""Every LDS read of the 4-bit products lies in the reading wave's own area, on bytes that the same wave has loaded, and finds
the row and columns that it means.  w4_layout.h is compiled with g++; no kernel is built or run."""

import subprocess

import pytest

from test_sanitized_host import CSRC, _gxx

# The loads as the kernel issues them, 16 bytes a lane from a base on; then all reads of a block.
PROGRAM = f"""
#include "{CSRC}/w4_layout.h"
#include <cstdio>
#include <vector>
template <int GROUP, bool ZERO, int MATS, int NB, int XL>
int check() {{
    using L = swz::W4Layout<GROUP, ZERO, MATS, NB, XL>;
    std::vector<int> w(L::kOwn, -1), x(L::kOwn, -1);  // 16 * row + piece (unit) where one begins
    int bad = 0;
    for (int lane = 0; lane < 64; ++lane) {{
        const int g = lane / 16, l16 = lane % 16;
        for (int o = 0; o < L::COLS; ++o) w.at(L::kW + o * 1024 + 16 * lane) = 1000 * o + 16 * (lane / 4) + ((lane % 4) ^ g);
        for (int a = 0; a < XL; ++a) x.at(L::kX + a * 1024 + 16 * lane) = 16 * (4 * a + g) + (l16 ^ ((4 * a + g) % 16));
    }}
    for (int lane = 0; lane < 64; ++lane) {{
        const int g = lane / 16, l16 = lane % 16;
        for (int o = 0; o < L::COLS; ++o) {{
            const int at = L::w_at(o, l16, g);
            bad += at < L::kW || at + 16 > L::kX || w.at(at) != 1000 * o + 16 * l16 + g;
            const int row = o * 16 + l16, last = L::kRun - L::PER;
            bad += row * L::kScaleRow + 2 * last + 2 * L::PER > L::kZero;
            bad += ZERO && L::kZero + row * L::kZeroRow + last + L::PER > L::kW;
        }}
        for (int a = 0; a < L::MB; ++a)
            for (int s = 0; s < 4; ++s) {{
                const int row = L::x_row(l16), unit = swz::w4_unit_of<GROUP>(s, g), at = L::x_at(a, row, unit);
                bad += at < L::kX || at + 16 > L::kOwn || row != (XL < 4 && l16 >= 4 * XL ? row : l16);
                bad += at + 16 <= L::kOwn && x.at(at) != 16 * (16 * a + row) + unit;
            }}
    }}
    // read for all 16 rows, an area of fewer is left
    const bool leaves = L::x_at(0, 15, 15) + 16 > L::kOwn;
    printf("%d %d %d %d %d: %d %d\\n", GROUP, ZERO, MATS, NB, XL, bad, leaves == (XL < 4));
    return bad;
}}
template <int GROUP, bool ZERO, int MATS, int NB>
int rows() {{
    return check<GROUP, ZERO, MATS, NB, 1>() + check<GROUP, ZERO, MATS, NB, 2>() + check<GROUP, ZERO, MATS, NB, 4>() +
           check<GROUP, ZERO, MATS, NB, 8>() + check<GROUP, ZERO, MATS, NB, 16>();
}}
template <int GROUP, bool ZERO>
int all() {{ return rows<GROUP, ZERO, 2, 1>() + rows<GROUP, ZERO, 1, 1>() + rows<GROUP, ZERO, 1, 2>(); }}
int main() {{
    all<32, false>(), all<32, true>(), all<64, false>(), all<64, true>(), all<128, false>(), all<128, true>();
    return 0;
}}
"""


@pytest.fixture(scope="module")
def variants(tmp_path_factory):
    d = tmp_path_factory.mktemp("w4_layout")
    (d / "layout.cpp").write_text(PROGRAM)
    subprocess.run([_gxx(), "-std=c++17", "-O1", "-D_GLIBCXX_ASSERTIONS", "-o", str(d / "layout"), str(d / "layout.cpp")], check=True)
    return subprocess.run([str(d / "layout")], capture_output=True, text=True, check=True).stdout.splitlines()


def test_reads_stay_in_a_waves_own_loads(variants):
    assert len(variants) == 6 * 3 * 5
    for line in variants:
        assert line.split(": ")[1] == "0 1", line
