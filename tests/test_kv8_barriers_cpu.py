"""The barriers that units of the 8-bit attention kernel pass through, searched over every order in which its roles can run.

A barrier counts completed phases; a wait names a phase and passes by parity alone (as mbarrier.try_wait.parity
does), so a waiter that lags two whole phases behind waits for a phase to come.  The roles are those of
csrc/attn_kv8_gqa.cu with units without tiles, which give the weakest order: nothing but the unit descriptors, the
query's barriers and the softmax warps' meeting holds them together."""

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


def roles(units, nq, softmax_warps=2):
    """(programs, barriers): a program is a list of (wait | arrive, barrier, phase) steps, barriers {name: arrivals a phase}."""
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
        if u > 0:
            split.append(("wait", "q_free", u - 1))
        split.append(("arrive", *q))
        issuer += [("wait", *q), ("arrive", "q_free", u)]
        softmax += [("wait", *q), ("arrive", "meet", u), ("wait", "meet", u)]
        for program in (split, issuer, softmax):
            program.append(("arrive", f"empty{s}", phase))
    return [scheduler, split, issuer] + [softmax] * softmax_warps, barriers


def orders(programs, barriers):
    """(number of states, some state in which nobody can go on, or None), over every order of the steps."""
    names = list(barriers)
    at = {n: k for k, n in enumerate(names)}
    start = (tuple(0 for _ in programs), tuple((0, 0) for _ in names))     # barrier: (completed phases, arrivals since)
    seen, todo = {start}, [start]
    while todo:
        where, bars = todo.pop()
        moved = False
        for r, program in enumerate(programs):
            if where[r] == len(program):
                continue
            kind, name, phase = program[where[r]]
            done, here = bars[at[name]]
            nbars = bars
            if kind == "wait":
                if (done & 1) == (phase & 1):
                    continue
            else:
                here += 1
                if here == barriers[name]:
                    done, here = done + 1, 0
                nbars = bars[:at[name]] + ((done, here),) + bars[at[name] + 1:]
            moved = True
            state = (where[:r] + (where[r] + 1,) + where[r + 1:], nbars)
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
