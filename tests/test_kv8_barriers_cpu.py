"""The barriers that units of the 8-bit attention kernel pass through, searched over every order in which its roles can run.

A barrier counts completed phases; a wait names a phase and passes by parity alone (as mbarrier.try_wait.parity
does), so a waiter that lags two whole phases behind waits for a phase to come.  The roles are those of
csrc/attn_kv8_gqa.cu with units without tiles, which give the weakest order: nothing but the unit descriptors, the
query's barriers and the softmax warps' meeting holds them together.  A CTA that has given up goes through its remaining
units all the same; waits that heed that pass at any time then, and what the split warps write of a unit (where its rows
go) still has to be there before a softmax warp uses it."""

from __future__ import annotations

import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "context_decode_attention_paged_gb300",
                      "csrc", "attn_kv8_gqa.cu")


def query_barriers():
    """How many q_full barriers the kernel has."""
    with open(SOURCE) as f:
        found = re.search(r"uint64_t [^;]*\bq_full(?:\[(\d+)\])?", f.read())
    return int(found.group(1) or 1)


def softmax_heeds():
    """Whether the softmax warps' wait for a unit's query ends when the CTA has given up."""
    with open(SOURCE) as f:
        text = f.read()
    call = re.search(r"(wait|wait_at)\((?:smem_u32\(&)?sm\.q_full[^;]*", text[text.index("softmax and epilogue ----"):])
    return call.group(1) == "wait" or not re.search(r"\bfalse\b", call.group(0))


def roles(units, nq, softmax_warps=2, gave_up=False, heeds=False):
    """(programs, barriers): a program is a list of (kind, barrier or cell, phase or unit) steps, barriers {name: arrivals
    a phase}.  gave_up: waits that heed it are left out."""
    readers = 2 + softmax_warps
    barriers = {"meet": softmax_warps, "q_free": 1}
    barriers.update({f"full{s}": 1 for s in range(2)})
    barriers.update({f"empty{s}": readers for s in range(2)})
    barriers.update({f"q{s}": 1 for s in range(nq)})
    scheduler, split, issuer, softmax = [], [], [], []
    for u in range(units):
        s, phase = u % 2, u // 2
        if u >= 2:
            scheduler.append(("wait", f"empty{s}", phase - 1))
        scheduler.append(("arrive", f"full{s}", phase))
        for program in (split, issuer, softmax):
            program.append(("wait", f"full{s}", phase))
        q = (f"q{u % nq}", u // nq)
        if u > 0 and not gave_up:
            split.append(("wait", "q_free", u - 1))
        split += [("write", s, u), ("arrive", *q)]
        issuer += [] if gave_up else [("wait", *q)]
        issuer.append(("arrive", "q_free", u))
        softmax += [] if gave_up and heeds else [("wait", *q)]
        softmax += [("arrive", "meet", u), ("wait", "meet", u), ("use", s, u)]
        for program in (split, issuer, softmax):
            program.append(("arrive", f"empty{s}", phase))
    return [scheduler, split, issuer] + [softmax] * softmax_warps, barriers


def orders(programs, barriers):
    """(number of states, some state in which nobody can go on or a cell that is used is not its unit's, or None), over
    every order of the steps."""
    names = list(barriers)
    at = {n: k for k, n in enumerate(names)}
    # barrier: (completed phases, arrivals since); cells: the unit that wrote them last
    start = (tuple(0 for _ in programs), tuple((0, 0) for _ in names), (None, None))
    seen, todo = {start}, [start]
    while todo:
        where, bars, cells = todo.pop()
        moved = False
        for r, program in enumerate(programs):
            if where[r] == len(program):
                continue
            kind, name, phase = program[where[r]]
            nbars, ncells = bars, cells
            if kind == "wait":
                if (bars[at[name]][0] & 1) == (phase & 1):
                    continue
            elif kind == "write":
                ncells = cells[:name] + (phase,) + cells[name + 1:]
            elif kind == "use":
                if cells[name] != phase:
                    return len(seen), where
            else:
                done, here = bars[at[name]]
                here += 1
                if here == barriers[name]:
                    done, here = done + 1, 0
                nbars = bars[:at[name]] + ((done, here),) + bars[at[name] + 1:]
            moved = True
            state = (where[:r] + (where[r] + 1,) + where[r + 1:], nbars, ncells)
            if state not in seen:
                seen.add(state)
                todo.append(state)
        if not moved and any(where[r] < len(p) for r, p in enumerate(programs)):
            return len(seen), where
    return len(seen), None


@pytest.mark.parametrize("units", [2, 5])
@pytest.mark.parametrize("softmax_warps", [1, 2, 3])
def test_no_order_of_the_roles_stops_the_units(units, softmax_warps):
    states, stuck = orders(*roles(units, query_barriers(), softmax_warps))
    assert stuck is None, (states, stuck)


def test_one_query_barrier_would_let_a_softmax_warp_fall_two_phases_behind():
    assert orders(*roles(4, 1))[1] is not None


@pytest.mark.parametrize("units", [1, 2, 5])
def test_a_ctas_units_have_their_rows_places_after_it_gave_up(units):
    states, stuck = orders(*roles(units, query_barriers(), gave_up=True, heeds=softmax_heeds()))
    assert stuck is None, (states, stuck)


def test_a_wait_that_heeds_would_let_places_be_used_that_are_not_there():
    assert orders(*roles(2, 2, gave_up=True, heeds=True))[1] is not None


def test_warps_that_may_give_up_alone_meet_at_no_barrier():
    """The warps that convert values wait each for themselves, and one of them may give up where the others do not: a
    barrier of theirs would then wait for ever."""
    with open(SOURCE) as f:
        text = f.read()
    part = text[text.index("query split, then value tiles"):text.index("softmax and epilogue ----")]
    assert not re.search(r"named_bar_sync|bar_red_or|__syncthreads", part)


def test_the_copies_in_flight_land_whoever_gives_up():
    """The producer waits for its last copies whether or not it has seen that the CTA has given up: another role may do so
    behind its last look."""
    with open(SOURCE) as f:
        text = f.read()
    part = text[text.index("TMA producer ----"):text.index("QK issuer: S^T")]
    tail = part[part.rindex("unit_done(u);"):]
    assert tail.count("wait_at(") == 2 and "abort_flag" not in tail
