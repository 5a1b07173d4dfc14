"""The barrier protocol of the received weights' kernel, checked as a graph (see
test_cache_attn_barriers.py, whose conditions on waits and buffers hold here)."""
import os
import re

import pytest

from test_cache_attn_barriers import CSRC, Graph

WARPS = 2           # warps of a role that may drift apart


def _constants():
    with open(os.path.join(CSRC, "cache_mass_tc.cuh")) as f:
        src = re.sub(r"//[^\n]*", "", f.read())
    return (int(re.search(r"kQSlots = (\d+)", src).group(1)), int(re.search(r"kAhead = (\d+)", src).group(1)))


def _kernel(steps):
    """The kernel's graph for a cluster that is handed these steps: pairs of what
    a step has ("k" columns on the tile's keys, "" none) and whether it is the
    last of the cluster's share of a tile."""
    slots, ahead = _constants()
    slabs = 9
    g = Graph()

    def take(role, c, n):
        g.wait(role, f"STEP{c}.{n % ahead}", n // ahead)
        g.use(role, f"info{c}.{n % ahead}", n // ahead, False)
        g.arrive(role, f"STEPFREE{c}.{n % ahead}", n // ahead)

    for c in (0, 1):
        role, place, tile, fresh = f"loads{c}", 0, 0, True
        for n, (has, last) in enumerate(steps):
            take(role, c, n)
            if has:
                for k in range(slabs):
                    s, u = place % slots, place // slots
                    g.wait(role, f"QEMPTY{c}.{s}", u - 1)
                    if fresh:
                        g.wait(role, f"KEMPTY{c}.{k}", tile - 1)
                        g.use(role, f"K{c}.{k}", tile, True)
                        g.arrive(role, f"KFULL.{k}", tile)
                    g.use(role, f"ring{c}.{s}", u, True)
                    g.arrive(role, f"QFULL.{s}", u)
                    place += 1
                tile += fresh
                fresh = last
        take(role, c, len(steps))

    role, place, tile, step, fresh = "mma", 0, 0, 0, True
    for n, (has, last) in enumerate(steps):
        take(role, 0, n)
        if not has:
            continue
        for k in range(slabs):
            s, u = place % slots, place // slots
            g.wait(role, f"QFULL.{s}", u)
            if fresh:
                g.wait(role, f"KFULL.{k}", tile)
            if k == 0:
                g.wait(role, f"DFREE.{step & 1}", (step >> 1) - 1)
            for c in (0, 1):
                g.use(role, f"D{c}.{step & 1}", step >> 1, True)
                g.use(role, f"ring{c}.{s}", u, False)
                g.use(role, f"K{c}.{k}", tile, False)
                g.arrive(role, f"QEMPTY{c}.{s}", u)
                if last:
                    g.arrive(role, f"KEMPTY{c}.{k}", tile)
            place += 1
        for c in (0, 1):
            g.arrive(role, f"DFULL{c}.{step & 1}", step >> 1)
        tile, step, fresh = tile + last, step + 1, last
    take(role, 0, len(steps))

    for c in (0, 1):
        for n in range(len(steps) + 1):
            g.wait(f"steps{c}", f"STEPFREE{c}.{n % ahead}", n // ahead - 1)
            g.use(f"steps{c}", f"info{c}.{n % ahead}", n // ahead, True)
            g.arrive(f"steps{c}", f"STEP{c}.{n % ahead}", n // ahead)

    for c in (0, 1):
        for hs in (0, 1):
            for w in range(WARPS):
                role, step, tile = f"sums{c}.{hs}.{w}", 0, 0
                for n, (has, last) in enumerate(steps):
                    g.wait(role, f"STEP{c}.{n % ahead}", n // ahead)
                    if has:
                        g.wait(role, f"DFULL{c}.{step & 1}", step >> 1)
                        g.use(role, f"D{c}.{step & 1}", step >> 1, False)
                        g.arrive(role, f"DFREE.{step & 1}", step >> 1)
                        step += 1
                    if last:
                        half = f"half{c}.{w}.{tile % ahead}"       # a warp of each half shares its keys
                        if hs == 1:
                            g.use(role, half, tile // ahead, True)
                            g.arrive(role, f"HALF{c}.{tile % ahead}", tile // ahead)
                        else:
                            g.wait(role, f"HALF{c}.{tile % ahead}", tile // ahead)
                            g.use(role, half, tile // ahead, False)
                        tile += 1
                    g.use(role, f"info{c}.{n % ahead}", n // ahead, False)
                    g.arrive(role, f"STEPFREE{c}.{n % ahead}", n // ahead)
                g.wait(role, f"STEP{c}.{len(steps) % ahead}", len(steps) // ahead)
    return g


K, END, DUE, IDLE = ("k", False), ("k", True), ("", True), ("", False)
WALKS = {
    "one step": [END],
    "one step a tile": [END] * 11,
    "several": [K, K, END, K, END, END, K, K, K, K, K, END, END],
    "shares without steps": [DUE, END, DUE, K, END, DUE, DUE],
    "empty steps": [IDLE, END, IDLE, IDLE, K, IDLE, END, IDLE, IDLE, IDLE, IDLE, IDLE, IDLE, END, IDLE],
    "only empty steps": [IDLE] * 7,
    "nothing": [],
}


@pytest.mark.parametrize("name", WALKS)
def test_no_wait_can_miss_its_phase(name):
    assert _kernel(WALKS[name]).check() == []
