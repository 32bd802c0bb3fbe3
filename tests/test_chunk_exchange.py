"""The exchanges of the softmax warps in the tcgen05 chunk attention, played through on the CPU: four
warps (two groups, two halves of a row) leave one another their halves' maxima in every step and their
sums at a run's end, each in a place of its own. Every order of their actions that the barriers allow is
tried; each warp has to read what was written for the exchange it is in. No GPU."""
import os
import re

import pytest

KERNEL = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "paged_kv_cache_271_gb300", "csrc", "chunk_attn_tc.cu")
WIDE = "wide"  # a run of more than 128 rows with one tile; a number: a narrower one of that many tiles
WARPS = [(g, h) for g in (0, 1) for h in (0, 1)]


def settles():
    """Whether the kernel's warps, at a wide run's end, arrive at their pair's barrier once more when they
    have read the other's sums, and wait there before the next run."""
    text = open(KERNEL).read()
    end = text[text.index("= exchange(l);"):text.index("base.skip(run.n);")]
    arrive, wait = end.find("mbar_arrive(pair)"), end.find("mbar_wait(pair, ph_pair")
    return 0 <= arrive < wait and len(re.findall(r"ph_pair \^= 1u", end)) == 1


def program(runs, g, h, settled):
    """Actions of warp (group g, half h). ("wait", mark, warps): until all of them have done ``mark``."""
    pair = ((g, 0), (g, 1))
    acts = []

    def swap(u, what):
        return [("write", (u, what)), ("do", ("pair", u, what)), ("wait", ("pair", u, what), pair),
                ("read", (g, 1 - h), (u, what))]

    acts.append(("do", ("queries", 0)))
    for u, tiles in enumerate(runs):
        wide = tiles == WIDE
        steps = 1 if wide else len(range(g, tiles, 2))
        for i in range(steps):  # scores: behind the group's queries, or both warps' last P
            acts += [("wait", ("queries", u) if i == 0 else ("p", u, i - 1), pair)]
            acts += swap(u, i) + [("do", ("p", u, i))]
        acts.append(("do", ("queries", u + 1)))
        if steps:  # the weighted values are done: both warps' last P was ready
            acts.append(("wait", ("p", u, steps - 1), pair))
        if wide:
            acts += swap(u, "end")
            if settled:
                acts += [("do", ("settled", u)), ("wait", ("settled", u), pair)]
        else:
            acts += [("write", (u, "end")), ("do", ("met", u)), ("wait", ("met", u), WARPS)]
            acts += [("read", who, (u, "end")) for who in WARPS]
            acts += [("do", ("parted", u)), ("wait", ("parted", u), WARPS)]
    return acts


def stale_reads(runs, settled):
    programs = [program(runs, *w, settled) for w in WARPS]
    when = [{a[1]: i for i, a in enumerate(p) if a[0] == "do"} for p in programs]
    wrong, seen, todo = set(), set(), [((0, 0, 0, 0), ((), (), (), ()))]
    while todo:
        at, places = todo.pop()
        if (at, places) in seen:
            continue
        seen.add((at, places))
        moves = []
        for k, p in enumerate(programs):
            if at[k] < len(p):
                act = p[at[k]]
                if act[0] != "wait" or all(at[WARPS.index(w)] > when[WARPS.index(w)][act[1]]
                                           for w in act[2]):
                    moves.append((k, act))
        assert moves or all(at[k] == len(p) for k, p in enumerate(programs)), "they wait for one another"
        # (marks and passed waits change no place and stop nobody: done first, the same reads remain)
        silent = [m for m in moves if m[1][0] in ("do", "wait")]
        for k, act in (silent[:1] or moves):
            after = list(places)
            if act[0] == "write":
                after[k] = act[1]
            elif act[0] == "read" and places[WARPS.index(act[1])] != act[2]:
                wrong.add((WARPS[k], act[2]))
            todo.append((tuple(a + (i == k) for i, a in enumerate(at)), tuple(after)))
    return wrong


RUNS = [[WIDE] * 3, [WIDE, 1, WIDE], [WIDE, 1, 1, WIDE], [1, WIDE, 2], [2, 3, 1], [WIDE, 2, WIDE, 1]]


@pytest.mark.parametrize("runs", RUNS, ids=str)
def test_warps_read_the_exchange_they_are_in_in_every_order(runs):
    assert not stale_reads(runs, settles())


def test_without_a_word_after_the_sums_they_would_be_read_stale():
    """(the model tells the difference: a wide run's sums, overwritten by the next run's first maxima or,
    in a group without a step there, by its sums)"""
    assert {w[1] for w in stale_reads([WIDE, WIDE], False)} == {(0, "end")}
    assert ((1, 0), (0, "end")) in stale_reads([WIDE, 1], False)
    assert not stale_reads([2, 3, 1], False)
