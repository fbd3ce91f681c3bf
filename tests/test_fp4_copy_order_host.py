"""The order in which the 4-bit product's warps wait for one another, over every interleaving.

A stage's slot of the ring is loaded (FULL), its scales are copied by one of two warps in turn (SF), the
products of the stage run in order and free the slot (EMPTY). A barrier knows the parity of its open phase and
no more, so a wait that looks too early, or after the phase behind the one it means is over too, takes one phase
for another. The states of such a pipeline are few enough to visit all: loads land in any order, and each warp may
be held at any point for as long as it likes."""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dit_transformer_block_gb300", "csrc",
                      "h3_fp4_gemm.cu")


def constant(name):
    with open(SOURCE) as f:
        return int(re.search(rf"\b{name} = (\d+)\b", f.read()).group(1))


SLOTS, WARPS = constant("STAGES4"), constant("COPY_WARPS")


def passes(over, phase):
    """Whether a wait for the phase numbered `phase` passes at a barrier with `over` phases over."""
    return (over & 1) != (phase & 1)


# What a copy warp waits for before stage `it`: ((barrier, phase) ..., whether it then copies).
def only_its_own(it, warp):
    return ([("full", it // SLOTS)], True) if it % WARPS == warp else ([], False)


def all_loads(it, warp):
    return [("full", it // SLOTS)], it % WARPS == warp


def the_slots_copies_before(it, warp):
    return ([("sf", it // SLOTS - 1), ("full", it // SLOTS)], True) if it % WARPS == warp else ([], False)


def explore(rule, total):
    """Faults that some interleaving reaches: 'early' (a stage's scales copied, or its products run, before they are
    there) and 'stall' (nothing can go on before the end)."""
    steps = []   # per warp: (kind, barrier or None, slot, phase, stage)
    for w in range(WARPS):
        mine = []
        for it in range(total):
            waits, copies = rule(it, w)
            mine += [("wait", b, it % SLOTS, p, it) for b, p in waits]
            if copies:
                mine.append(("copy", None, 0, 0, it))
        steps.append(mine)

    def over(n, slot, done):   # phases of a slot's barrier that are over, `done`: stages it counts
        return sum(1 for it in range(slot, n, SLOTS) if it in done)

    # loaded: loads issued; landed: those that landed; at: the copy warps' places; sent, copied: copies issued, done;
    # run, ran: stages whose products are issued, done (they end in order)
    none = frozenset()
    start = (0, none, (0,) * WARPS, none, none, 0, 0)
    seen, todo, faults = {start}, [start], set()
    while todo:
        loaded, landed, at, sent, copied, run, ran = todo.pop()
        after = []
        if loaded < total and passes(len(range(loaded % SLOTS, ran, SLOTS)), loaded // SLOTS - 1):
            after.append((loaded + 1, landed, at, sent, copied, run, ran))
        after += [(loaded, landed | {it}, at, sent, copied, run, ran) for it in range(loaded) if it not in landed]
        after += [(loaded, landed, at, sent - {it}, copied | {it}, run, ran) for it in sent]
        for w in range(WARPS):
            if at[w] < len(steps[w]):
                kind, barrier, slot, phase, it = steps[w][at[w]]
                ahead = at[:w] + (at[w] + 1,) + at[w + 1:]
                if kind == "copy":
                    if it not in landed or it - SLOTS >= ran:
                        faults.add("early")
                    else:
                        after.append((loaded, landed, ahead, sent | {it}, copied, run, ran))
                elif passes(over(total, slot, landed if barrier == "full" else copied), phase):
                    after.append((loaded, landed, ahead, sent, copied, run, ran))
        if run < total and passes(over(total, run % SLOTS, landed), run // SLOTS) and \
                passes(over(total, run % SLOTS, copied), run // SLOTS):
            if run in landed and run in copied:
                after.append((loaded, landed, at, sent, copied, run + 1, ran))
            else:
                faults.add("early")
        if ran < run:
            after.append((loaded, landed, at, sent, copied, run, ran + 1))
        if not after and ran < total:
            faults.add("stall")
        for t in after:
            if t not in seen:
                seen.add(t)
                todo.append(t)
    return faults


@pytest.mark.parametrize("total", [1, SLOTS, SLOTS + 1, 2 * SLOTS + 1, 3 * SLOTS + 2])
def test_every_interleaving_ends_and_reads_what_was_loaded(total):
    assert explore(the_slots_copies_before, total) == set()


def test_other_orders_fail():
    # without waiting for the slot's stage between, a load that lands late is taken for one that has; with waits for
    # the other warp's loads, a warp that is held for long misses one
    assert "early" in explore(only_its_own, 3 * SLOTS)
    assert "stall" in explore(all_loads, 3 * SLOTS)


def test_the_kernel_waits_in_this_order():
    with open(SOURCE) as f:
        copies = f.read().split("scale copies\n")[1].split("epilogue warps")[0]
    waits = re.findall(r"wait\((B4_\w+) \+ st, ([^)]*)\)", copies)
    assert waits == [("B4_SF", "phase ^ 1"), ("B4_FULL", "phase")], waits
