"""Which tile the products of a gated block take by their sizes: every tile is reached, by the shapes that the GPU test
runs (gated_cases.py).  The rules are compiled with g++ from the library's host code; no kernel is built or run."""

import subprocess

import pytest

from gated_cases import DW, DX, FORWARD
from test_sanitized_host import CSRC, HOST_SOURCES, ROOT, _gxx

TILES = ["k64x64", "k64x256", "k128x128", "k128x256", "k256x256"]
GATED = ["k64x32", "k128x32", "k64x128", "k128x128", "k256x128"]

PROGRAM = f"""
#include "{CSRC}/capi.cpp"
#include <cstdio>
#include <cstdlib>
int main(int argc, char** argv) {{
    const int64_t n = atoll(argv[1]), k = atoll(argv[2]), f = atoll(argv[3]);
    const swz::GatedPlan p = plan_gated(n, f, k);
    printf("%d %d %d %lld %d %lld %d\\n", swz::gated_few(n, f, k) ? 1 : 0, static_cast<int>(swz::gated_tile(n, f)),
           static_cast<int>(p.dx_tile), static_cast<long long>(p.dx_parts), static_cast<int>(p.dw_tile),
           static_cast<long long>(p.dw_parts), p.rest != 0);
}}
"""


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    d = tmp_path_factory.mktemp("gated_rules")
    (d / "rules.cpp").write_text(PROGRAM)
    others = [f"{CSRC}/{s}" for s in HOST_SOURCES if s != "capi.cpp"]
    others += [f"{ROOT}/tests/{s}" for s in ("host_stubs.cpp", "host_stubs_feed_forward.cpp")]
    subprocess.run([_gxx(), "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", f"-I{ROOT}/include", f"-I{CSRC}",
                    "-o", str(d / "rules"), str(d / "rules.cpp"), *others], check=True)

    def run(shape):
        out = subprocess.run([str(d / "rules"), *map(str, shape)], capture_output=True, text=True, check=True).stdout
        few, gated, dx, dxp, dw, dwp, two = (int(x) for x in out.split())
        return "few" if few else GATED[gated], (TILES[dx], dxp > 1, two == 1), (TILES[dw], dwp > 1, two == 1)

    return run


@pytest.mark.parametrize("tile", FORWARD)
def test_forward_shapes_take_their_tiles(rules, tile):
    assert all(rules(shape)[0] == tile for shape in FORWARD[tile])


@pytest.mark.parametrize("kind", DX)
def test_dx_shapes_take_their_tiles(rules, kind):
    assert rules(DX[kind])[1] == kind


@pytest.mark.parametrize("kind", DW)
def test_dw_shapes_take_their_tiles(rules, kind):
    assert rules(DW[kind])[2] == kind


def test_cases_reach_every_tile():
    assert set(FORWARD) == {"few", *GATED}
    tiles = {(t, split, False) for t in TILES for split in (False, True)}
    assert set(DX) == set(DW) == tiles | {("k64x64", False, True), ("k64x64", True, True), ("k128x256", False, True)}


def test_small_products_take_two_terms(rules):
    for n, k, f in ((1, 8, 1), (1, 8, 1 << 20), (256, 256, 128), (255, 8, 4112)):
        assert rules((n, k, f))[1][2] and rules((n, k, f))[2][2]
    for n, k, f in ((256, 256, 129), (1 << 20, 16, 1), (1, 1032, 8192)):
        assert not rules((n, k, f))[1][2] and not rules((n, k, f))[2][2]
