"""Which rows' states a thread of the gated recurrence asks for, followed on the host: the kernels' own tile header is compiled
with the host compiler, and for every thread of every tile the states it would read and write are counted.

Every element of a [rows, C] array is asked for by exactly one thread where its row begins and by one where it ends (rows
without tokens: by none), and nothing else is, before the array or past it."""
from __future__ import annotations

import shutil
import subprocess

import pytest

from gated_delta_rule_sm_gb300 import build as kbuild

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "kda_gated.h"
using namespace kda;

template <int VEC> int follow(int C, const std::vector<int>& off) {
    const int rows = (int)off.size() - 1, tokens = off[rows];
    std::vector<int> begun((size_t)rows * C), ended((size_t)rows * C);
    int wrong = 0;
    auto ask = [&](std::vector<int>& seen, int row, int c) {
        for (int v = 0; v < VEC; ++v) {
            const long at = (long)row * C + c + v;
            if (row < 0 || row >= rows || c + v >= C || at >= (long)seen.size()) ++wrong;      // another row's element, or nobody's
            else ++seen[at];
        }
    };
    for (int tile = 0; tile * kGatedTile < tokens; ++tile) {
        GatedEdges e;
        for (int k = 0; k < kGatedTile; ++k) e.first[k] = e.last[k] = -1;
        const int t0 = tile * kGatedTile;
        for (int m = 0; m < rows; ++m) {
            if (off[m + 1] == off[m]) continue;
            if (off[m] >= t0 && off[m] < t0 + kGatedTile) e.first[off[m] - t0] = m;
            if (off[m + 1] > t0 && off[m + 1] <= t0 + kGatedTile) e.last[off[m + 1] - 1 - t0] = m;
        }
        for (int col = 0; col * 32 * VEC < C; ++col)
            for (int thread = 0; thread < kGatedThreads; ++thread) {
                const GatedSpot s = gated_spot<VEC>(tokens, C, tile, col, thread);
                for (int k = 0; k < kGatedTok; ++k) {
                    if (e.begins(s, k) >= 0) ask(begun, e.begins(s, k), s.c);
                    if (e.ends(s, k) >= 0) ask(ended, e.ends(s, k), s.c);
                }
            }
    }
    for (int m = 0; m < rows; ++m)
        for (int c = 0; c < C; ++c) {
            const int want = off[m + 1] > off[m];
            wrong += begun[(size_t)m * C + c] != want || ended[(size_t)m * C + c] != want;
        }
    return wrong;
}

int main(int argc, char** argv) {      // channels at once, C, offsets
    std::vector<int> off;
    for (int k = 3; k < argc; ++k) off.push_back(std::atoi(argv[k]));
    const int C = std::atoi(argv[2]);
    std::printf("%d\n", std::atoi(argv[1]) == 2 ? follow<2>(C, off) : follow<1>(C, off));
}
"""


@pytest.fixture(scope="module")
def follow(tmp_path_factory):
    at = tmp_path_factory.mktemp("rows")
    (at / "rows.cpp").write_text(PROGRAM)
    cmd = [shutil.which("g++") or "g++", "-std=c++17", "-O1", "-I", kbuild.CSRC, str(at / "rows.cpp"), "-o", str(at / "rows")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(vec, C, offsets):
        return int(subprocess.run([str(at / "rows"), str(vec), str(C), *map(str, offsets)], capture_output=True, text=True, check=True).stdout)
    return run


OFFSETS = {"one": [0, 1], "short": [0, 37], "tiles": [0, 64, 128], "rows": [0, 100, 200, 300], "batch": list(range(0, 201)),
           "ragged": [0, 0, 3, 3, 3, 203, 331, 332, 396, 396], "last empty": [0, 40, 40]}


@pytest.mark.parametrize("vec,C", [(1, 1), (1, 31), (1, 32), (1, 33), (1, 515), (2, 2), (2, 8), (2, 62), (2, 64), (2, 66), (2, 130)])
@pytest.mark.parametrize("offsets", OFFSETS.values(), ids=OFFSETS.keys())
def test_states_are_asked_for_by_their_own_threads(follow, vec, C, offsets):
    assert follow(vec, C, offsets) == 0
