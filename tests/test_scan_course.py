"""The order in which the blocks of a scan go through their tiles, on the CPU, by the kernels' own code (csrc/kda_scan_course.h) between a
loader's asks and the waits for what it asked for: every tile once, nothing asked for that no turn waits for, and no tile
behind the end however often one asks."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "linear_attention_kda_gb300", "csrc")

# argv: chains back grid blocks length...; prints "block sequence position first-token" of every tile that a block's turns take, then
# "asked waited more" of each block, more being the tiles that three more calls find
PROGRAM = r"""
#include <stdio.h>
#include <stdlib.h>
#include <vector>
#include "kda_scan_course.h"
using kda::scan::tile;
constexpr int L = 64;
int main(int argc, char **argv) {
    const bool chains = atoi(argv[1]), back = atoi(argv[2]);
    const int grid = atoi(argv[3]), blocks = atoi(argv[4]), N = argc - 5;
    std::vector<int> at(1, 0);
    for (int n = 0; n < N; ++n) at.push_back(at.back() + atoi(argv[5 + n]));
    const int items = (chains ? N : at[N] / L + N) * blocks;
    for (int b = 0; b < grid; ++b) {
        int item = -1, asked = 0, waited = 0, more = 0;
        tile t{0, -1, 0, 0, 0, 0, 0}, stage[2];
        auto next = [&] {
            kda::scan::next_tile<L>(t, chains, back, [&](tile *to) {
                item = item < 0 ? b : item + grid;
                if (item >= items) return false;
                const int r = back && !chains ? items - 1 - item : item, i = r / blocks;
                to->block = r - i * blocks;
                int n = i, p = 0;
                if (!chains) {
                    for (n = N - 1; n > 0 && at[n] / L + n > i; --n) {}
                    p = i - (at[n] / L + n);
                }
                to->n = n, to->a = at[n], to->b = at[n + 1];
                to->p = p == 0 || p < (to->b - to->a + L - 1) / L ? p : -1;
                return true;
            });
        };
        auto ask = [&](int s) {
            next();
            stage[s] = t;
            asked += t.p >= 0;
        };
        ask(0);
        ask(1);
        for (int turn = 0; turn < 1 << 20; ++turn) {
            const tile u = stage[turn & 1];
            if (u.p < 0) break;
            ++waited;
            printf("%d %d %d %d\n", u.block, u.n, u.p, u.first);
            ask(turn & 1);
        }
        for (int i = 0; i < 3; ++i) {
            next();
            more += t.p >= 0;
        }
        printf("%d %d %d\n", asked, waited, more);
    }
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("course")
    (d / "course.cc").write_text(PROGRAM)
    exe = str(d / "course")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-I", CSRC, str(d / "course.cc"), "-o", exe])
    return exe


@pytest.mark.parametrize("chains", (0, 1))
@pytest.mark.parametrize("back", (0, 1))
@pytest.mark.parametrize("grid,blocks", [(1, 1), (2, 3), (7, 2), (40, 1)])
@pytest.mark.parametrize("lens", [[1], [0], [64], [1000], [65, 0, 64, 200], [500] * 6, [1] * 9, [700, 3, 0, 0, 129]])
def test_every_tile_once_and_none_behind_the_end(program, chains, back, grid, blocks, lens):
    out = subprocess.run([program] + [str(v) for v in (chains, back, grid, blocks, *lens)], capture_output=True, text=True, check=True).stdout
    rows = [tuple(map(int, x.split())) for x in out.splitlines()]
    ends = [r for r in rows if len(r) == 3]
    assert len(ends) == grid and all(asked == waited and more == 0 for asked, waited, more in ends)
    want, at = [], 0
    for n, m in enumerate(lens):
        want += [(c, n, p, at // 64 + n) for p in range(max(1, -(-m // 64))) for c in range(blocks)]
        at += m
    got = sorted(r for r in rows if len(r) == 4)
    assert got == sorted(want)
