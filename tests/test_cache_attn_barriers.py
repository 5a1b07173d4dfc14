"""The barrier protocol of the paged latent attention kernel, checked as a graph.

A wait on an mbarrier names its phase by parity alone, so it is right only if,
whatever the speed of each warp,
  * the phase before the awaited one is complete when the wait begins, and
  * the phase behind it cannot complete until the wait is over.
Both are questions of reachability: the roles' programs (loads, MMA issue,
parts, softmax, Q and O) are written down as sequences of waits and arrivals,
a wait follows every arrival of its phase, and each condition is a path in that
graph. Buffers that warps hand to one another are held to the same rule. How
many barriers a role takes in turn comes from the kernel's source.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_20_b200", "csrc")
WARPS = 2           # warps of a role that may drift apart


def _source():
    with open(os.path.join(CSRC, "cache_attn_tc.cuh")) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _constants():
    src = _source()
    enum = re.search(r"enum : int \{(.*?)\}", src, re.S).group(1)
    at = {n: int(v) for n, v in re.findall(r"(B_\w+) = (\d+)", enum)}
    order = sorted(at.values())
    span = {n: (order[order.index(v) + 1] - v if n != "B_COUNT" else 0) for n, v in at.items()}
    slots = int(re.search(r"kSlots = (\d+)", src).group(1))
    ahead = int(re.search(r"kAhead = (\d+)", src).group(1))
    return span, slots, ahead


def _full_first(name):
    """Whether the load of a box with a barrier of its own arrives for the MMA
    before it announces its bytes."""
    body = re.search(r"auto " + name + r" = .*?\n        \};", _source(), re.S).group(0)
    own = body[body.index("if (own)"):body.index("} else {")]
    return own.index("mbar_arrive(bar(B_") < own.index("mbar_arrive_expect_tx(own")


class Graph:
    """Events in program order per role; arrivals and waits of (barrier, phase)."""

    def __init__(self):
        self.before = []            # predecessors of each event
        self.last = {}              # last event of each role
        self.arrivals, self.waits = {}, []
        self.reads, self.writes = {}, {}

    def event(self, role):
        e = len(self.before)
        self.before.append([self.last[role]] if role in self.last else [])
        self.last[role] = e
        return e

    def arrive(self, role, bar, phase):
        self.arrivals.setdefault((bar, phase), []).append(self.event(role))

    def wait(self, role, bar, phase):
        if phase >= 0:              # the phase "before the first" of a free buffer is always complete
            self.waits.append((self.event(role), bar, phase, role))

    def use(self, role, buf, turn, write):
        (self.writes if write else self.reads).setdefault((buf, turn), []).append((self.event(role), role))

    def close(self):
        for e, bar, phase, role in self.waits:
            assert (bar, phase) in self.arrivals, f"{role} waits for {bar} phase {phase}: no arrival"
            self.before[e] += self.arrivals[(bar, phase)]
        n = len(self.before)
        after, need = [[] for _ in range(n)], [0] * n
        for e, p in enumerate(self.before):
            need[e] = len(p)
            for q in p:
                after[q].append(e)
        past, ready, seen = [0] * n, [e for e in range(n) if need[e] == 0], 0
        while ready:                # past[e]: every event that comes before e, as a bit set
            e = ready.pop()
            seen += 1
            for q in self.before[e]:
                past[e] |= past[q] | (1 << q)
            for a in after[e]:
                need[a] -= 1
                if need[a] == 0:
                    ready.append(a)
        assert seen == n, "a cycle of waits"
        return past

    def check(self):
        past = self.close()
        wrong = []
        for e, bar, phase, role in self.waits:
            if not all(past[e] >> a & 1 for a in self.arrivals.get((bar, phase - 1), [])):
                wrong.append(f"{role}: {bar} may still be in phase {phase - 1} when {phase} is awaited")
            nxt = self.arrivals.get((bar, phase + 1), [])
            if nxt and not any(past[a] >> e & 1 for a in nxt):
                wrong.append(f"{role}: {bar} may be through phase {phase + 1} while {phase} is awaited")
        for (bar, phase), ar in self.arrivals.items():
            for a in ar:
                if not all(past[a] >> b & 1 for b in self.arrivals.get((bar, phase - 1), [])):
                    wrong.append(f"{bar}: an arrival of phase {phase} may fall into phase {phase - 1}")
        for (buf, turn), ws in self.writes.items():
            for w, who in ws:
                for r, reader in self.reads.get((buf, turn - 1), []):
                    if not past[w] >> r & 1:
                        wrong.append(f"{who} may write {buf} (turn {turn}) before {reader} has read it")
            for r, reader in self.reads.get((buf, turn), []):
                if not all(past[r] >> w & 1 for w, _ in ws):
                    wrong.append(f"{reader} may read {buf} (turn {turn}) before it is written")
        return sorted(set(wrong))


def _kernel(parts):
    """The kernel's graph for a cluster whose parts have these tiles: a list of
    lists of truth values (a tile that not every row sees whole), [] without keys."""
    span, slots, ahead = _constants()
    g = Graph()
    parts = [list(p) for p in parts]
    units = [p for p in parts if p]

    def take(role, c, n):
        g.wait(role, f"PART{c}.{n % ahead}", n // ahead)
        g.use(role, f"info{c}.{n % ahead}", n // ahead, False)
        g.arrive(role, f"PARTFREE{c}.{n % ahead}", n // ahead)

    def in_turn(name, c, n):
        return f"{name}{c}.{n % span['B_' + name]}", n // span["B_" + name]

    full_first = _full_first("push"), _full_first("push_rope")

    def signal(role, c, own, full, first):
        if own and not first:
            g.arrive(role, *own)
        if c == 0 or not own:
            g.arrive(role, *full)
        if own and first:
            g.arrive(role, *own)

    # ring places: Q K(0) K(1) V(0) ... V(n-1) as the loads push them
    for c in (0, 1):
        role, place, rope, own_of, cut, keys = f"loads{c}", 0, 0, {}, [], 0

        def push(own):
            nonlocal place
            s, u = place % slots, place // slots
            g.wait(role, f"EMPTY{c}.{s}", u - 1)
            g.use(role, f"ring{c}.{s}", u, True)
            if own == "slot":
                own = f"OWN{c}.{s}", own_of.setdefault(s, 0)
                own_of[s] += 1
            signal(role, c, own, (f"FULL.{s}", u), full_first[0])
            place += 1

        def push_rope(own):
            nonlocal rope
            s, u = rope % 2, rope // 2
            g.wait(role, f"REMPTY{c}.{s}", u - 1)
            g.use(role, f"rope{c}.{s}", u, True)
            signal(role, c, own, (f"RFULL.{s}", u), full_first[1])
            rope += 1

        values = None
        for n, p in enumerate(parts):
            take(role, c, n)
            if not p:
                continue
            here = in_turn("QLOAD", c, keys)
            keys += 1
            push(here)
            push(here)
            push_rope(here)
            for masked in p:
                push(None)
                push(None)
                push_rope(None)
                if values is not None:
                    push("slot" if values else None)
                    push("slot" if values else None)
                values = masked
        if values is not None:
            push("slot" if values else None)
            push("slot" if values else None)
        take(role, c, len(parts))

    # MMA issue: a commit arrives in both CTAs
    role, place, rope, tile, u, last_nt = "mma", 0, 0, 0, 0, 0

    def commit(name, n):
        for c in (0, 1):
            g.arrive(role, f"{name}{c}", n)

    def done(read=True):
        nonlocal place
        for c in (0, 1):
            if read:
                g.use(role, f"ring{c}.{place % slots}", place // slots, False)
            g.arrive(role, f"EMPTY{c}.{place % slots}", place // slots)
        place += 1

    def rdone(read=True):
        nonlocal rope
        for c in (0, 1):
            if read:
                g.use(role, f"rope{c}.{rope % 2}", rope // 2, False)
            g.arrive(role, f"REMPTY{c}.{rope % 2}", rope // 2)
        rope += 1

    def full():
        g.wait(role, f"FULL.{place % slots}", place // slots)

    def qk():
        g.wait(role, "SFREE", tile - 1)
        full()
        done()
        full()
        g.wait(role, f"RFULL.{rope % 2}", rope // 2)
        for c in (0, 1):
            g.use(role, f"Q{c}", u, False)
        done()
        rdone()
        commit("SFULL", tile)

    def pv(gp, first, of):
        g.wait(role, "PFULL", gp)
        if first:
            g.wait(role, "OFREE", of - 1)
        full()
        done()
        full()
        done()
        for c in (0, 1):
            g.use(role, f"P{c}", gp, False)
            g.use(role, f"O{c}", of, True)
        commit("PVDONE", gp)

    for n, p in enumerate(parts):
        take(role, 0, n)
        if not p:
            continue
        g.wait(role, "QT", u)
        done(read=False)
        done(read=False)
        rdone(read=False)
        for j in range(len(p)):
            qk()
            if j == len(p) - 1:
                commit("QFREE", u)
            if tile > 0:
                if j > 0:
                    pv(tile - 1, j == 1, u)
                else:
                    pv(tile - 1, last_nt == 1, u - 1)
            tile += 1
        last_nt = len(p)
        u += 1
    if u:
        pv(tile - 1, last_nt == 1, u - 1)
        g.wait(role, "SFREE", tile - 1)
        g.wait(role, "OFREE", u - 1)
    take(role, 0, len(parts))

    # parts
    for c in (0, 1):
        for n in range(len(parts) + 1):
            g.wait(f"parts{c}", f"PARTFREE{c}.{n % ahead}", n // ahead - 1)
            g.use(f"parts{c}", f"info{c}.{n % ahead}", n // ahead, True)
            g.arrive(f"parts{c}", f"PART{c}.{n % ahead}", n // ahead)

    # softmax, and Q in / O out
    for c in (0, 1):
        for w in range(WARPS):
            role, np, tile, uc, own_n = f"softmax{c}.{w}", 0, 0, 0, {}
            ring = -2

            def advance():
                nonlocal np
                while True:
                    take(role, c, np)
                    np += 1
                    if np > len(parts):
                        return None
                    if parts[np - 1]:
                        return parts[np - 1]

            unit = advance()
            while unit is not None:
                nt, nxt = len(unit), None
                for j in range(nt):
                    g.wait(role, f"SFULL{c}", tile)
                    g.arrive(role, "SFREE", tile)
                    g.use(role, f"red{c}.{tile & 1}", tile >> 1, True)
                    g.use(role, f"bad{c}.{tile & 1}", tile >> 1, True)
                    g.arrive(role, *in_turn("RED", c, tile))
                    g.wait(role, *in_turn("RED", c, tile))
                    g.use(role, f"red{c}.{tile & 1}", tile >> 1, False)
                    g.wait(role, f"PVDONE{c}", tile - 1)
                    g.use(role, f"P{c}", tile, True)
                    if j == 0:
                        nxt = advance()
                    if unit[j]:
                        v0 = ring + 4 * j + (8 if j < nt - 1 else 10 if nxt is not None else 6)
                        for b in (0, 1):
                            s = (v0 + b) % slots
                            g.wait(role, f"OWN{c}.{s}", own_n.setdefault(s, 0))
                            own_n[s] += 1
                            g.use(role, f"ring{c}.{s}", (v0 + b) // slots, False)
                    g.use(role, f"bad{c}.{tile & 1}", tile >> 1, False)
                    g.arrive(role, "PFULL", tile)
                    tile += 1
                ring += 2 + 4 * nt
                g.use(role, f"sums{c}.{uc & 1}", uc >> 1, True)
                g.arrive(role, *in_turn("LSUM", c, uc))
                unit, uc = nxt, uc + 1

            role, np, uc, tile, ring, rope = f"qo{c}.{w}", 0, 0, 0, 0, 0

            def write_q(n):
                g.wait(role, *in_turn("QLOAD", c, n))
                for b in (0, 1):
                    g.use(role, f"ring{c}.{(ring + b) % slots}", (ring + b) // slots, False)
                g.use(role, f"rope{c}.{rope % 2}", rope // 2, False)
                g.use(role, f"Q{c}", n, True)
                g.arrive(role, "QT", n)

            unit = advance()
            if unit is not None:
                write_q(0)
            while unit is not None:
                nxt = advance()
                ring += 4 * len(unit) + (2 if uc > 0 else 0)
                rope += 1 + len(unit)
                if nxt is not None:
                    g.wait(role, f"QFREE{c}", uc)
                    write_q(uc + 1)
                tile += len(unit)
                g.wait(role, *in_turn("LSUM", c, uc))
                g.use(role, f"sums{c}.{uc & 1}", uc >> 1, False)
                g.wait(role, f"PVDONE{c}", tile - 1)
                g.use(role, f"O{c}", uc, False)
                g.arrive(role, "OFREE", uc)
                unit, uc = nxt, uc + 1
    assert len(units) == u
    return g


T, F = True, False
WALKS = {
    "one tile": [[T]],
    "units of one tile": [[T]] * 9,
    "whole tiles, one a unit": [[F]] * 9,
    "one, two and three tiles": [[T], [F, T], [T, F, T], [T], [T], [F, F], [T], [F, F, F, T], [T]],
    "long units": [[F] * 12 + [T], [F] * 7, [T] + [F] * 9],
    "padding between": [[], [], [T], [], [T], [], [T], [T], [], [F, T], [], [T], []],
    "only padding": [[], []],
    "nothing": [],
}


@pytest.mark.parametrize("name", WALKS)
def test_no_wait_can_miss_its_phase(name):
    assert _kernel(WALKS[name]).check() == []


def test_tensor_memory_is_written_behind_a_fence():
    """The warps that bring Q in overwrite columns that earlier MMAs read: their
    wait for those MMAs has to be followed by the fence that orders tcgen05
    accesses behind it."""
    body = re.search(r"auto write_q = .*?return true;\s*\};", _source(), re.S).group(0)
    assert "tmem_st32(" in body
    assert "tc_fence_after();" in body[:body.index("tmem_st32(")]
