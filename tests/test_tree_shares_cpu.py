"""Where the tree attention's blocks leave the shares of items that the launch cuts: replayed on the
host for many shapes, with the rule of who leaves a share read from the kernels' source."""
import os
import random
import re

import pytest

from transposed_conv_implicit_gb300 import build


def _source(name):
    with open(os.path.join(build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


FEW, MANY = _source("tree_few.cu"), _source("tree_many.cu")
KEYS = 128


def _whole(source):
    """What a block calls an item that it writes itself."""
    text = re.search(r"const bool whole = ([^;,]+)[;,]", source).group(1)
    return text.replace("w.whole()", "held").replace("&&", "and").replace("!single", "not single").strip()


def _replay(source, requests, kv_heads, group, tile_rows, ctas):
    """requests: (keys, drafts).  Slots that blocks write, and those that the join reads, by item."""
    many, whole = tile_rows == 256, _whole(source)
    items = []       # (first step, tiles, rows)
    total = 0
    for keys, drafts in requests:
        rows, tiles = drafts * group, -(-keys // KEYS)
        for _ in range(kv_heads):
            for r0 in range(0, rows, tile_rows):
                items.append((total, tiles, min(tile_rows, rows - r0)))
                total += tiles
    begin = [total * c // ctas for c in range(ctas + 1)]
    written, at = {}, 0
    for c in range(ctas):
        lo, hi = begin[c], begin[c + 1]
        while lo < hi:
            while items[at][0] + items[at][1] <= lo:
                at += 1
            first, tiles, rows = items[at]
            t0, t1 = lo - first, min(tiles, hi - first)
            single = many and rows <= tile_rows // 2
            if not eval(whole, {"held": t0 == 0 and t1 == tiles, "single": single}):
                for half in range(2 if single else 1):
                    slot = (2 * c + (t0 == 0), half)
                    assert slot not in written, "slot %s of items %d and %d" % (slot, written[slot], at)
                    written[slot] = at
            lo = first + t1
    share_of = lambda s: ((s + 1) * ctas - 1) // total
    read = {}
    for i, (first, tiles, rows) in enumerate(items):
        c0, c1 = share_of(first), share_of(first + tiles - 1)
        if c0 == c1:
            continue
        for c in range(c0, c1 + 1):
            if total < ctas and begin[c] == begin[c + 1]:
                continue
            for half in range(2 if many and rows <= tile_rows // 2 else 1):
                read[(2 * c + (c == c0), half)] = i
    assert written == read
    return len(items), len(written)


MANY_CASES = [   # requests, kv_heads, group
    ([(4096, 24)] * 64, 8, 4), ([(928, 24)] * 25, 8, 4), ([(100, 30)] * 40, 8, 3), ([(77, 100)] * 3, 1, 1),
    ([(900, 75)] * 40, 4, 4), ([(300, 94), (2000, 94), (128, 94)] * 20, 2, 4), ([(129, 17)] * 152, 1, 8),
    ([(8192, 64)] * 16, 8, 4), ([(2531, 29), (30, 20), (333, 7)], 4, 3), ([(0, 0), (5, 5), (700, 65)] * 30, 3, 1),
]


@pytest.mark.parametrize("ctas", [152, 148, 7])
@pytest.mark.parametrize("case", MANY_CASES, ids=lambda c: "%dx%s" % (len(c[0]), c[0][0]))
def test_many_rows(case, ctas):
    _replay(MANY, *case, 256, ctas)


def test_drawn_shapes():
    rng = random.Random(5)
    joined = held = 0
    for _ in range(300):
        b, kv_heads, group = rng.randint(1, 64), rng.choice([1, 2, 3, 8, 16]), rng.choice([1, 2, 3, 4, 8])
        most, t = int(2 ** rng.uniform(0, 13)), rng.choice([1, 2, 7, 24, 64, 100, 256])
        requests = []
        for _ in range(b):
            keys = rng.choice([most, rng.randint(0, most)])
            requests.append((keys, min(keys, rng.choice([t, rng.randint(0, t)]))))
        if not any(d for _, d in requests):
            continue
        requests = [(k, d) for k, d in requests if d]
        rows = t * group
        tile = 256 if rows > 64 else 16 if rows <= 16 else 32
        source = MANY if tile == 256 else FEW
        items, shares = _replay(source, requests, kv_heads, group, tile, {256: 152, 32: 304, 16: 456}[tile])
        joined += shares > 0
        held += shares < items
    assert joined > 50 and held > 50


def test_the_join_leaves_out_what_one_block_holds():
    assert "shares = range[1] == c0 ? 1 : (range[1] - c0 + 1) * halves;" in FEW
    assert "if (shares <= 1) return;" in FEW
