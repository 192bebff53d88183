"""The weight gradient's stage ring, its hand-over from role to role explored on
the CPU in every order that the barriers allow.

One SM's share of dw_gemm (grouped_tc.cuh): a producer fills the stages, a warp
zeroes the rows behind a group's end in the blocks that have such rows (`fix`),
the issuer multiplies and gives the stage back.  The barriers are mbarriers: a
phase ends after `count` arrivals, and a wait knows the phase by one parity bit.
Who arrives on `empty`, and its count, are read from the source."""
import os
import re

import pytest

from conftest import ROOT

STAGES = 2


def source_protocol():
    """(count of `empty`, whether the warp of the tail rows arrives on it)"""
    text = open(os.path.join(ROOT, "sparse_moe_layer_sum_b200", "csrc", "grouped_tc.cuh")).read()
    dw = text[text.index("dw_gemm(const __grid_constant__"):]
    count = int(re.search(r"mbar_init\(empty \+ s, (\d)\)", dw).group(1))
    warp = dw[dw.index("warp == 2"):dw.index("regs_high()")]
    return count, "mbar_arrive(empty + r.stage)" in warp


def explore(fixes, count, passes_on):
    """What can go wrong with blocks of which fixes[i] needs zeroing: a set of
    'wrong block' (zeroed, or multiplied before it was zeroed) and 'stuck'."""
    n = len(fixes)
    counts = {"full": 1, "tail": 1, "empty": count}

    # barriers: (phases ended, arrivals of the present one) by name and stage
    def arrive(bars, name, s):
        k = (name, s)
        ended, got = bars[k]
        got += 1
        out = dict(bars)
        out[k] = (ended + 1, 0) if got == counts[name] else (ended, got)
        return out

    def passed(bars, name, s, parity):  # the phase of that parity is over
        return (bars[name, s][0] & 1) != parity

    faults, seen = set(), set()
    start = {(b, s): (0, 0) for b in counts for s in range(STAGES)}
    # holds[s]: (block, zeroed)
    todo = [((0, 0, 0), start, tuple((-1, False) for _ in range(STAGES)))]
    while todo:
        pcs, bars, holds = todo.pop()
        key = (pcs, tuple(sorted(bars.items())), holds)
        if key in seen:
            continue
        seen.add(key)
        moved = False
        prod, fixer, mma = pcs
        if prod < n:
            s, phase = prod % STAGES, prod // STAGES & 1
            if passed(bars, "empty", s, phase ^ 1):
                moved = True
                h = list(holds)
                h[s] = (prod, False)
                b = arrive(bars, "tail", s)
                if not fixes[prod]:
                    b = arrive(b, "full", s)
                todo.append(((prod + 1, fixer, mma), b, tuple(h)))
        if fixer < n:
            s, phase = fixer % STAGES, fixer // STAGES & 1
            if passed(bars, "tail", s, phase):
                moved = True
                h, b = list(holds), bars
                if fixes[fixer]:
                    if holds[s][0] != fixer:
                        faults.add("wrong block")
                    h[s] = (holds[s][0], True)
                    b = arrive(b, "full", s)
                if passes_on:
                    b = arrive(b, "empty", s)
                todo.append(((prod, fixer + 1, mma), b, tuple(h)))
        if mma < n:
            s, phase = mma % STAGES, mma // STAGES & 1
            if passed(bars, "full", s, phase):
                moved = True
                if holds[s] != (mma, fixes[mma]):
                    faults.add("wrong block")
                todo.append(((prod, fixer, mma + 1), arrive(bars, "empty", s), holds))
        if not moved and pcs != (n, n, n):
            faults.add("stuck")
    return faults


# the last block of a group's rows is the one to fix: runs of other blocks
# before it, several groups, the six passes of split operands
RUNS = [[0, 0, 0, 0, 0, 0, 1], [0] * 5 + [1], [1] * 6, [0, 1, 0, 1, 0, 1], [0, 0, 1, 0, 0, 0, 0, 1, 0, 0],
        [0, 0, 0, 1] * 3, [0] * 9]


@pytest.mark.parametrize("run", RUNS, ids=lambda r: "".join(map(str, r)))
def test_no_order_zeroes_another_block(run):
    assert explore([bool(f) for f in run], *source_protocol()) == set()


def test_the_exploration_sees_an_overrun():
    """Without the zeroing warp's arrivals the producer may lap it: its wait
    misses a whole turn of the ring."""
    assert explore([False] * 6 + [True], 1, False) == {"stuck"}
