"""The end of a unit in the tcgen05 tree attention, played through on the CPU: two groups of threads
exchange their rows' maxima and sums through places that exchange_slot names. Every order of
their actions that the barriers allow is tried; each group has to read what both wrote for the
unit it is in. No GPU."""
import ctypes
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "paged_kv_cache_271_gb300", "csrc")


@pytest.fixture(scope="module")
def exchange(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("exchange")
    (d / "x.cpp").write_text(
        '#include "tree_exchange.h"\n'
        'extern "C" int slot(unsigned u, int g, int r) { return pkv::exchange_slot(u, g, r); }\n'
        'extern "C" int slots() { return pkv::kExchangeSlots; }\n'
        'extern "C" int rows() { return pkv::kExchangeRows; }\n')
    subprocess.run([cxx, "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(d / "x.cpp"), "-o",
                    str(d / "x.so")], check=True)
    return ctypes.CDLL(str(d / "x.so"))


def stale_reads(tiles, slot):
    """Orders of the groups' actions over units of these tile counts in which a group reads another
    unit's values. A group's actions in a unit: wait for the queries of both (only with a step in
    it: group g takes tiles g, g + 2, ..), write its place, arrive at `met`, wait for the other
    there, read its own place and the other's (one after the other), store its next queries."""
    acts = [[("queries", u) for _ in range(tiles[u] > g)] +
            [("write", u), ("arrive", u), ("met", u), ("read", u, g), ("read", u, 1 - g),
             ("store", u + 1)] for g in (0, 1) for u in range(len(tiles))]
    n = len(tiles)
    program = [sum(acts[g * n:(g + 1) * n], []) for g in (0, 1)]
    wrong, seen, todo = set(), set(), [(0, 0, ())]
    while todo:
        state = todo.pop()
        if state in seen:
            continue
        seen.add(state)
        at, places = state[:2], dict(state[2])
        done = [set(program[g][:at[g]]) for g in (0, 1)]
        for g in (0, 1):
            if at[g] == len(program[g]):
                continue
            act, u = program[g][at[g]][:2]
            if act == "queries" and u > 0 and any(("store", u) not in d for d in done):
                continue
            if act == "met" and any(("arrive", u) not in d for d in done):
                continue
            after = dict(places)
            if act == "write":
                after[slot(u, g)] = (u, g)
            if act == "read":
                whose = program[g][at[g]][2]
                if places.get(slot(u, whose)) != (u, whose):
                    wrong.add((u, g, whose))
            nxt = (at[0] + (g == 0), at[1] + (g == 1))
            todo.append((*nxt, tuple(sorted(after.items()))))
    return wrong


@pytest.mark.parametrize("tiles", [[1] * 5, [3, 1, 1, 2, 1], [2, 2, 2], [1, 4, 1, 1, 1]])
def test_groups_read_the_units_own_sums_in_every_order(exchange, tiles):
    assert not stale_reads(tiles, lambda u, g: exchange.slot(u, g, 5))


def test_one_place_for_all_units_would_be_read_stale():
    """(the model tells the difference: group 1 overwrites what group 0 has still to read)"""
    one_place = lambda u, g: g
    assert stale_reads([1, 1], one_place) == {(0, 0, 1)}
    assert not stale_reads([2, 2, 2], one_place)


def test_places_are_distinct_and_fit(exchange):
    slots = [exchange.slot(u, g, r) for u in (6, 7) for g in (0, 1) for r in range(exchange.rows())]
    assert sorted(slots) == list(range(exchange.slots()))
