"""The ranges that pa_decode_nvfp4 cuts its work into, restated: every tile once, at
most one piece before and one behind a range's whole items, and the number of
pieces that the joining kernel is told."""
import random

import pytest

TILE = 128


def _ranges(lens, heads, ctas, begin, whole):
    """Per CTA: [(sequence, head, first tile, end, units before its first tile)], and {item: pieces} of cut items."""
    tiles = [-(-n // TILE) for n in lens]
    work = [min(t, 1) if whole else (t + begin if t else 0) for t in tiles]
    W = sum(work)
    U = W * heads
    per, rem = divmod(U, ctas)
    first = [per * c + min(c, rem) for c in range(ctas + 1)]
    out, told = [], {}
    for c in range(ctas):
        u, u1, items = first[c], first[c + 1], []
        while u < u1:
            head, x = divmod(u, W)
            s = off = 0
            while off + work[s] <= x:
                off += work[s]
                s += 1
            t, v = (0, 0) if whole else (max(0, x - off - begin), max(0, begin - (x - off)))
            if u1 - u <= v:
                break
            te = tiles[s] if whole else min(tiles[s], t + u1 - u - v)
            items.append((s, head, t, te))
            if t == 0 and te < tiles[s]:
                last, cut = u + v + tiles[s] - 1, rem * (per + 1)
                told[s, head] = (last // (per + 1) if last < cut else rem + (last - cut) // per) - c + 1
            u += 1 if whole else v + te - t
        out.append(items)
    return tiles, out, told


@pytest.mark.parametrize("seed", range(300))
def test_ranges(seed):
    r = random.Random(seed)
    top = r.choice([130, 600, 5000, 100000])
    lens = [r.choice([0, 1, 128, r.randint(0, top)]) for _ in range(r.randint(1, 70))]
    if not any(lens):
        lens[0] = 1
    heads, ctas, begin = r.choice([1, 2, 8, 40]), r.choice([1, 2, 7, 152]), r.choice([5, 8])
    whole = max(lens) <= 512 and r.random() < 0.5
    tiles, ranges, told = _ranges(lens, heads, ctas, begin, whole)
    seen = {}
    for c, items in enumerate(ranges):
        cut_here = [(t > 0, te < tiles[s]) for s, _, t, te in items]
        # a continued piece comes first, one that goes on comes last: a slot of the workspace each
        assert all(not a for a, _ in cut_here[1:]) and all(not b for _, b in cut_here[:-1])
        for s, h, t, te in items:
            assert te > t
            seen.setdefault((s, h), []).append((c, t, te))
    assert len(seen) == heads * sum(1 for t in tiles if t)
    for (s, h), pieces in seen.items():
        assert [p[1] for p in pieces] == [0] + [p[2] for p in pieces[:-1]] and pieces[-1][2] == tiles[s]
        # in consecutive ranges, as many as the joining kernel is told
        assert [p[0] for p in pieces] == list(range(pieces[0][0], pieces[0][0] + len(pieces)))
        assert told.get((s, h), 1) == len(pieces)
