"""The order in which the tree attention's kernel for many rows takes its barriers, walked over every
interleaving of the widening, the product warp, the tensor core and a softmax group: a run shows one
of them.  Which barriers and parities are waited for is read from the source."""
import os
import re

import pytest

from transposed_conv_implicit_gb300 import build

with open(os.path.join(build.CSRC, "tree_many.cu")) as f:
    SOURCE = re.sub(r"//[^\n]*", "", f.read())


def _index(text):
    return [i.replace("half ^ 1", "1 - half") for i in re.findall(r"\[([^\]]+)\]", text)][1:]   # (behind [g])


def _waits():
    """((barrier's half, parity) in front of rescaling an output, those at an item's end), as expressions."""
    found = [(m.start(), _index(m.group(1)), m.group(2)) for m in
             re.finditer(r"wait\(&sh\.o_done((?:\[[^\]]+\])+), ([^,]+), kAttnSoftmaxTimeout\)", SOURCE)]
    end = SOURCE.index("if (ok && !first)")
    parse = lambda w: (w[1][0] if w[1] else "0", w[2].replace("1u", "1").replace("half ^ 1", "1 - half"))
    return [parse(w) for w in found if w[0] < end], [parse(w) for w in found if w[0] > end]


RESCALE, END = _waits()
DONE = _index(re.search(r"mma_commit_warp\(smem_u32\(&sh\.o_done((?:\[[^\]]+\])+)\)\)", SOURCE).group(1))
DONE = DONE[0] if DONE else "0"


def _product_warp(items, in_turn):
    """What the product warp does for items of so many tiles: waits, products and commits.  in_turn: the
    next tile's scores are issued behind the last product of the one before (tiles go to two groups in turn)."""
    steps, tile, words = [], 0, 0
    for count in items:
        def scores(half):
            return [("issue", ("scores", None)), ("issue", ("arrive", ("s", half)))]

        steps.append(("word", words))
        words += 1
        steps += scores(0) + scores(1)
        for t in range(count):
            steps.append(("word", words))                   # the values
            words += 1
            more = t + 1 < count
            for half in range(2):
                steps.append(("wait", ("p", half), tile & 1))
                if more and half == 0 and not in_turn:
                    steps.append(("word", words))
                    words += 1
                steps.append(("issue", ("product", (tile, half))))
                steps.append(("issue", ("arrive", ("o", eval(DONE, {"half": half})))))
                if more and not in_turn:
                    steps += scores(half)
            if more and in_turn:
                steps.append(("word", words))
                words += 1
                steps += scores(0) + scores(1)
            tile += 1
    return steps, words


def _softmax(items, rescale, end):
    """What a softmax warp does: a set of halves (own tile, half) is rescaled in front of."""
    steps, tiles, halves = [], 0, 0
    for count in items:
        for t in range(count):
            for half in range(2):
                names = {"half": half, "tiles": tiles, "halves": halves}
                steps.append(("wait", ("s", half), tiles & 1))
                if (t, half) != (0, 0) and (tiles, half) in rescale:
                    for at, parity in RESCALE:
                        steps.append(("wait", ("o", eval(at, names)), eval(parity, names)))
                    steps.append(("read", 2 * tiles + half))       # products that have to be done
                steps.append(("arrive", ("p", half)))
                halves += 1
            tiles += 1
        names = {"tiles": tiles, "halves": halves}
        for at, parity in end:
            steps.append(("wait", ("o", eval(at, names)), eval(parity, names)))
        steps.append(("read", 2 * tiles))
    return steps


def _walk(items, in_turn, rescale, end):
    """(whether a read comes before a product it needs, whether anything can wait for ever)."""
    warp, words = _product_warp(items, in_turn)
    soft = _softmax(items, rescale, end)
    queue = [s[1] for s in warp if s[0] == "issue"]
    bars = [("s", 0), ("s", 1), ("p", 0), ("p", 1), ("o", 0), ("o", 1)]
    issued_at = [0]
    for s in warp:
        issued_at.append(issued_at[-1] + (s[0] == "issue"))

    def phases(done, at):
        """Completed phases of each barrier: what the tensor core and softmax have arrived at."""
        c = dict.fromkeys(bars, 0)
        for kind, arg in queue[:done]:
            if kind == "arrive":
                c[arg] += 1
        for s in soft[:at]:
            if s[0] == "arrive":
                c[s[1]] += 1
        return c

    def through(c, bar, parity):
        return (c[bar] & 1) != parity          # (the phase before has this parity, or nothing has yet)

    early = stuck = False
    seen, todo = set(), [(0, 0, 0, 0)]         # widened tiles, the product warp, the tensor core, softmax
    while todo:
        state = todo.pop()
        if state in seen:
            continue
        seen.add(state)
        w, pc, done, at = state
        c = phases(done, at)
        nexts = []
        if w < words:
            nexts.append((w + 1, pc, done, at))
        if pc < len(warp):
            s = warp[pc]
            if s[0] == "issue" or (s[0] == "word" and w > s[1]) or (s[0] == "wait" and through(c, s[1], s[2])):
                nexts.append((w, pc + 1, done, at))
        if done < issued_at[pc]:
            nexts.append((w, pc, done + 1, at))
        if at < len(soft):
            s = soft[at]
            if s[0] == "read":
                early |= sum(kind == "product" for kind, _ in queue[:done]) < s[1]
            if s[0] != "wait" or through(c, s[1], s[2]):
                nexts.append((w, pc, done, at + 1))
        if not nexts and (pc, at) != (len(warp), len(soft)):
            stuck = True
        todo += nexts
    return early, stuck


ITEMS = [(1,), (2,), (3,), (1, 1), (1, 2), (2, 1), (3, 1), (1, 1, 1), (2, 3)]


@pytest.mark.parametrize("in_turn", [False, True])
@pytest.mark.parametrize("items", ITEMS, ids=str)
def test_no_output_is_read_before_its_products(items, in_turn):
    for rescale in (set(), {(t, h) for t in range(8) for h in range(2)}, {(t, 1) for t in range(8)},
                    {(t, 0) for t in range(8)}, {(1, 0)}, {(0, 1), (2, 0)}):
        assert _walk(items, in_turn, rescale, END) == (False, False), rescale


def test_the_walk_sees_what_is_missing():
    """Without the waits at an item's end the walk finds the early read; with a wait for a phase that
    nothing completes, the standstill."""
    assert _walk((2,), False, set(), [])[0]
    assert _walk((2,), False, set(), END + [("0", "tiles & 1")])[1]


def _meet(pairs, read_wait):
    """Two softmax groups over items of which pairs[i] are held by both and written here: what each does,
    over every interleaving.  Returns (whether one reads the other's statistics or output of another item,
    whether anything can wait for ever)."""
    steps = []
    for i, pair in enumerate(pairs):
        if i and pairs[i - 1] and read_wait:
            steps.append(("wait", 1))
        steps.append(("products", i))            # writes the group's output
        if pair:
            steps += [("stat", i), ("arrive",), ("wait", 0), ("read", i), ("arrive",)]
    early = stuck = False
    seen, todo = set(), [(0, 0)]
    while todo:
        state = todo.pop()
        if state in seen:
            continue
        seen.add(state)
        done = [steps[:at] for at in state]
        phase = sum(s[0] == "arrive" for d in done for s in d) // 2
        # (An arrival counts for the phase that is incomplete: nobody may be two ahead.)
        counts = [sum(s[0] == "arrive" for s in d) for d in done]
        assert abs(counts[0] - counts[1]) <= 1 or not read_wait
        nexts = []
        for g in range(2):
            if state[g] == len(steps):
                continue
            s = steps[state[g]]
            if s[0] == "read":
                other = done[1 - g]
                last = lambda kind: max([x[1] for x in other if x[0] == kind], default=-1)
                early |= last("stat") != s[1] or last("products") != s[1]
            if s[0] != "wait" or (phase & 1) != s[1]:
                nexts.append((state[0] + (g == 0), state[1] + (g == 1)))
        stuck |= not nexts and state != (len(steps), len(steps))
        todo += nexts
    return early, stuck


@pytest.mark.parametrize("pairs", [(1,), (1, 1), (1, 0, 1), (0, 1, 1, 0), (1, 1, 1, 1), (1, 0, 0, 1, 1)], ids=str)
def test_groups_read_one_anothers_output_of_their_item(pairs):
    assert "ok = (!met || wait(&sh.meet, 1u, kAttnSoftmaxTimeout)) &&" in SOURCE
    assert "ok = wait(&sh.meet, 0u, kAttnSoftmaxTimeout);" in SOURCE
    assert SOURCE.count("mbar_arrive(smem_u32(&sh.meet))") == 2
    assert _meet(pairs, True) == (False, False)
    if len(pairs) > 1 and pairs[0]:
        assert _meet(pairs, False)[0]


def test_groups_that_meet_leave_an_item_together():
    """Behind the wait for the other group, whose end each warp sees for itself, the group's warps agree."""
    for wait in ("ok = wait(&sh.meet, 0u, kAttnSoftmaxTimeout);",
                 "wait(&sh.q_empty[g], (items & 1u) ^ 1u, kAttnSoftmaxTimeout);"):
        after = SOURCE[SOURCE.index(wait) + len(wait):]
        assert after.lstrip().startswith("ok = barrier_all(bar_id, 128, ok);")
