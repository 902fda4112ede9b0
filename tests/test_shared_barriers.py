"""Waits of the attention over shared prefixes, from its source: each lane of a warp comes to
the same end of a wait, and no barrier's phase can be missed at an item's end."""
import itertools
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_mla_decode_04_gb300", "csrc")


@pytest.fixture(scope="module")
def source():
    with open(os.path.join(CSRC, "shared_decode.cu")) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_waits_that_may_give_up_are_a_warps_or_a_threads(source):
    """mbar_wait ends for each lane by itself. Where the others would meet lanes that have given up (at a shuffle
    or a barrier of the warp), the lanes vote; a wait without a flag to give up for is one lane's alone."""
    waits = [m.start() for m in re.finditer(r"\bmbar_wait\s*\(", source)]
    assert waits
    for at in waits:
        depth, end = 1, source.index("(", at) + 1
        while depth:
            depth += {"(": 1, ")": -1}.get(source[end], 0)
            end += 1
        if "abort_flag" in source[at:end]:
            assert re.search(r"__all_sync\(0xffffffffu, $", source[:at]), source[at:end]
        else:
            assert "nullptr" in source[at:end]


def item_end(source):
    """What a softmax warp does at an item's end, in the source's order: (what, barrier, who)."""
    body = source[source.index("if (k >= item0) {\n", source.index("kBarQ));\n")):]
    body = body[:body.index("if (k + 1 >= item1) break;")]
    marks = {r"warp_wait\(bar\(kBarStatsFree\)": ("wait", "free", "both"),
             r"mbar_arrive\(sum_bar\)": ("arrive", "sum", "other"),
             r"warp_wait_block\(sum_bar": ("wait", "sum", "last"),
             r"peer\(kBarStats\), 32 \* 8": ("arrive", "stats", "last")}
    found = sorted((m.start(), what) for pattern, what in marks.items() for m in re.finditer(pattern, body))
    assert len(found) == len(marks)
    return [what for _, what in found]


@pytest.mark.parametrize("last", list(itertools.product((0, 1), repeat=5)))
def test_no_phase_passes_a_waiter_by(source, last):
    """Every order in which a quarter's two softmax warps and the accumulators' warps can come to the ends of five
    items, the last block of item k being group last[k]'s: a wait tells phases apart by their parity only, and has
    to end with its own."""
    ends = item_end(source)
    warps = []
    for group in (0, 1):
        steps = []
        for k, g in enumerate(last):
            for what, barrier, who in ends:
                if who == "both" or (who == "last") == (group == g):
                    # (of the sums' two barriers each has every other item; the room's first phase counts as complete)
                    name, phase = ("sum%d" % (k & 1), k >> 1) if barrier == "sum" else (barrier, k - 1 if barrier == "free" else k)
                    steps.append((what, name, phase))
        warps.append(steps)
    warps.append([s for k in range(len(last)) for s in (("wait", "stats", k), ("arrive", "free", k))])
    names = ["free", "stats", "sum0", "sum1"]  # (one arrival completes a phase of each)
    start = (0,) * len(warps) + (0,) * len(names)
    seen, todo = {start}, [start]
    while todo:
        state = todo.pop()
        at, done = state[:len(warps)], state[len(warps):]
        moved = False
        for w, steps in enumerate(warps):
            if at[w] == len(steps):
                continue
            what, name, phase = steps[at[w]]
            b = names.index(name)
            after = list(done)
            if what == "arrive":
                after[b] += 1
            elif (done[b] & 1) == (phase & 1):  # this phase, or one as even, is not complete
                assert done[b] <= phase, (name, phase, state)
                continue
            else:
                assert done[b] == phase + 1, (name, phase, state)
            moved = True
            to = at[:w] + (at[w] + 1,) + at[w + 1:] + tuple(after)
            if to not in seen:
                seen.add(to)
                todo.append(to)
        assert moved or all(at[w] == len(s) for w, s in enumerate(warps)), state
