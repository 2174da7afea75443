"""The rules that choose product tiles, compiled from the library's sources: the shapes of tile_cases.py take
the tiles that they are meant to (no GPU)."""

import subprocess

import pytest

from test_sanitized_host import CSRC, HOST_SOURCES, ROOT, _gxx
from tile_cases import GEMM, LOSS

# the entry points' file itself, for its plan of the gradients' pieces
PROGRAM = r"""
#include "capi.cpp"

#include <cstdio>
#include <cstdlib>

int main(int argc, char** argv) {
    for (int i = 1; i + 3 < argc; i += 4) {
        const int64_t n = atoll(argv[i + 1]), v = atoll(argv[i + 2]), k = atoll(argv[i + 3]);
        if (argv[i][0] == 'g') {
            const int rows[] = {64, 64, 128, 256}, cols[] = {64, 128, 128, 256}, t = static_cast<int>(swz::gemm_f8_tile(n, v));
            printf("%d %d\n", n <= swz::kFewRows ? 0 : rows[t], cols[t]);
        } else {
            printf("%lld", static_cast<long long>(swz::loss_tile_rows(n, (v + 255) / 256)));
            const int64_t piece = plan_loss(n, v, k, 1).piece;
            for (int64_t at = 0; at < v; at += piece) {
                const int64_t words = v - at < piece ? v - at : piece;
                printf(" %lld %lld", static_cast<long long>(swz::loss_tile_rows(n, (words + 255) / 256)),
                       static_cast<long long>(swz::loss_tile_rows(words, (k + 255) / 256)));
            }
            printf("\n");
        }
    }
}
"""


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    d = tmp_path_factory.mktemp("rules")
    (d / "rules.cpp").write_text(PROGRAM)
    others = [f"{CSRC}/{s}" for s in HOST_SOURCES if s != "capi.cpp"] + [f"{ROOT}/tests/host_stubs.cpp"]
    subprocess.run([_gxx(), "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", f"-I{ROOT}/include", f"-I{CSRC}",
                    "-o", str(d / "rules"), str(d / "rules.cpp"), *others], check=True)

    def run(kind, *shape):
        out = subprocess.run([str(d / "rules"), kind, *map(str, shape)], capture_output=True, text=True, check=True).stdout
        return [int(x) for x in out.split()]

    return run


@pytest.mark.parametrize("tile", GEMM)
def test_product_shapes_take_their_tiles(rules, tile):
    assert tuple(rules("g", *GEMM[tile], 1)) == tile


@pytest.mark.parametrize("shape", LOSS)
def test_loss_shapes_take_their_tiles(rules, shape):
    forward, logits, dw = LOSS[shape]
    got = rules("l", *shape)
    assert got[0] == forward and got[1::2] == logits and got[2::2] == dw
