"""The work list of pa_chunk_fp8 on the host: the closed forms that the kernel
compiles (chunk_schedule.h) against a plain enumeration, and the cut into
equal ranges: every unit once, pieces of an item in consecutive ranges."""
import os
import random
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "quantized_paged_attention_gb300", "csrc")

with open(os.path.join(CSRC, "chunk_schedule.h")) as f:
    COST = int(re.search(r"ITEM_COST = (\d+);", f.read()).group(1))

MAIN = r"""
#include "chunk_schedule.h"
#include <cstdio>
using namespace qpa::chunk;
// reads: bt q0 q1 L T maxlen -> prints q0 ql L nt units, then tiles and prefix of every item
// the kernel's search, a warp's 32 probes in a loop
static int find(const Req& r, long long off, int bt) {
  int lo = 0, hi = r.nt;
  while (hi - lo > 1) {
    int c = 0;
    for (int i = 0; i < 32; ++i) c += r.before(Req::split(lo, hi, i), bt) <= off;
    const int l = c ? Req::split(lo, hi, c - 1) : lo, h = c < 32 ? Req::split(lo, hi, c) : hi;
    lo = l;
    hi = h;
  }
  return lo;
}
int main() {
  int bt, a, b, L, T, M;
  while (scanf("%d %d %d %d %d %d", &bt, &a, &b, &L, &T, &M) == 6) {
    Req r = make_req(a, b, L, T, M, bt);
    printf("%d %d %d %d %lld", r.q0, r.ql, r.L, r.nt, r.units(bt));
    long long u = 0;
    bool found = true;
    for (int j = 0; j < r.nt; ++j) {
      printf(" %d %lld", r.tiles(j, bt), r.before(j, bt));
      if (r.nt < 300 || j % 97 == 0) found = found && find(r, u, bt) == j && find(r, u + r.tiles(j, bt) + ITEM_COST - 1, bt) == j;
      u += r.tiles(j, bt) + ITEM_COST;
    }
    printf(" %d\n", (int)found);
  }
}
"""


@pytest.fixture(scope="module")
def prog(tmp_path_factory):
    d = tmp_path_factory.mktemp("sched")
    src, exe = str(d / "s.cpp"), str(d / "s")
    with open(src, "w") as f:
        f.write(MAIN)
    subprocess.run(["g++", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover", "-std=c++17", "-I", CSRC, src,
                    "-o", exe], check=True)
    return exe


def _rows(bt, ql, L):
    """Key tiles of every item by looking at every row."""
    out = []
    for j in range(0, ql, bt):
        last = max(L - ql + min(j + bt, ql) - 1, 0)
        out.append(last // 128 + 1)
    return out


def test_closed_forms(prog):
    r = random.Random(1)
    cases = []
    for _ in range(3000):
        g = r.randint(1, 64)
        bt = 256 // g
        T = r.choice([5, 300, 20000])
        a = r.randint(-3, T)
        b = min(r.randint(a - 3, a + r.choice([3, 300, 6000])), T + 3)
        L = r.choice([0, r.randint(0, 200), r.randint(0, 9000), r.randint(-5, 5)])
        cases.append((bt, a, b, L, T, 8192))
    # the ends of the range
    cases += [(256, 0, 1, 2 ** 31 - 1, 1, 2 ** 31 - 1), (4, 0, 40000, 2 ** 31 - 1, 40000, 2 ** 31 - 1),
              (4, 0, 100000, 50, 100000, 1 << 20)]
    out = subprocess.run([prog], input="\n".join(" ".join(map(str, c)) for c in cases), capture_output=True, text=True,
                         check=True).stdout.splitlines()
    assert len(out) == len(cases)
    for (bt, a, b, L, T, M), line in zip(cases, out):
        q0, ql, LL, nt, units, *rest = map(int, line.split())
        assert q0 == max(0, min(a, T)) and ql == max(0, max(0, min(b, T)) - q0) and LL == max(0, min(L, M))
        tiles = _rows(bt, ql, LL)
        assert nt == len(tiles) and units == sum(tiles) + COST * nt and rest[-1] == 1
        assert rest[:-1:2] == tiles
        assert rest[1:-1:2] == [sum(tiles[:j]) + COST * j for j in range(nt)] if nt < 200 else True


def test_ranges_cover_every_unit_once_and_pieces_are_found():
    """The cut and the merge's walk, restated: every CTA's first piece that
    began earlier lies in its slot 2c, and following the pieces from the CTA
    where an item starts meets all of its units, over CTAs without units."""
    r = random.Random(2)
    for _ in range(300):
        grid = r.choice([1, 2, 5, 152])
        items = [r.randint(1, r.choice([1, 4, 60])) for _ in range(r.randint(1, 40))]
        cost = r.choice([0, COST, 9])
        U = sum(n + cost for n in items)
        first = [0]
        for n in items:
            first.append(first[-1] + n + cost)
        pieces, start, cont, tiles = {}, {}, {}, [0] * len(items)
        active = min(grid, -(-U // r.choice([1, 4])))
        for c in range(grid):
            u, u1 = U * min(c, active) // active, U * min(c + 1, active) // active
            cont[c] = dict(empty=True, x=False, ends=False)
            k = 0
            while u < u1:
                i = max(j for j in range(len(items)) if first[j] <= u)
                e = min(first[i + 1], u1)
                t0, t1 = max(0, u - first[i] - cost), max(0, e - first[i] - cost)
                u = e
                if t0 == t1:
                    continue
                tiles[i] += t1 - t0
                starts, ends = t0 == 0, t1 == items[i]
                if not (starts and ends):
                    slot = 2 * c + (k > 0)
                    assert slot not in pieces
                    pieces[slot] = (i, t0, t1)
                    if starts:
                        start[c] = (i, slot)
                    else:
                        assert k == 0
                        cont[c].update(x=True, ends=ends)
                cont[c]["empty"] = False
                k += 1
        assert tiles == items
        met = 0
        for c, (i, slot) in start.items():
            got = [pieces[slot]]
            for d in range(c + 1, grid):
                if cont[d]["empty"]:
                    continue
                if not cont[d]["x"]:
                    break
                got.append(pieces[2 * d])
                if cont[d]["ends"]:
                    break
            assert all(p[0] == i for p in got)
            assert got[0][1] == 0 and got[-1][2] == items[i]
            assert all(x[2] == y[1] for x, y in zip(got, got[1:]))
            met += len(got)
        assert met == len(pieces)
