"""The order of the tcgen05 attention kernel's roles (CPU only).

A CTA of `attn_many_kernel` passes blocks of keys between converter warps, an
MMA thread, softmax warps and a scale warp through shared memory and mbarriers.
A missing wait there shows in no result as long as the timing is kind, so the
roles' loops are written down here as programs of waits, arrivals, reads and
writes, and every reuse of a buffer has to be ordered by them behind the last
use of what it held.  The sizes of the page ring come from the source.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "invariant_numerics_b200", "csrc")
SRC = os.path.join(CSRC, "attn_paged.cu")
SCALE_RING = 4  # blocks of scales held


def page_ring():
    m = re.search(r"PAGE_RING = (\d+), PAGE_AHEAD = (\d+)", open(SRC).read())
    return int(m.group(1)), int(m.group(2))


def roles(n, ring, ahead):
    """The programs of one warp of each role for n blocks: ("wait" | "arrive", barrier, phase) and ("read" | "write",
    buffer, what it holds)."""
    conv, mma, soft, scale = [], [], [], []

    def operand(s):  # K 0, K 1, V 0, K 2, V 1, .., V n-1
        is_v = s > 0 and (s % 2 == 0 or s == 2 * n - 1)
        if s == 0:
            return 0, is_v
        return (n - 1 if s == 2 * n - 1 else (s + 1) // 2) if s % 2 else s // 2 - 1, is_v

    def load(i):
        conv.append(("read", ("pages", i % ring), i))

    conv.append(("wait", ("pg_full", 0), 0))
    load(0), load(0)
    for s in range(4 * n):
        i, is_v = operand(s // 2)
        if s % 2 == 0 and i > 0:
            conv.append(("wait", ("v_empty" if is_v else "k_empty",), i - 1))
        conv.append(("write", ("v" if is_v else "k",), i))
        if s % 2:
            conv.append(("arrive", ("v_full" if is_v else "k_full",), i))
        if s + 2 < 4 * n:
            ni, next_v = operand((s + 2) // 2)
            if not next_v and s % 2 == 0:
                conv.append(("wait", ("pg_full", ni % ring), ni // ring))
            load(ni)

    for i in range(n + 1):
        if i < n:
            mma += [("wait", ("k_full",), i), ("read", ("k",), i), ("write", ("scores", i % 2), i),
                    ("arrive", ("k_empty",), i), ("arrive", ("s_full", i % 2), i // 2)]
        if i > 0:
            j = i - 1
            mma += [("wait", ("p_full", j % 2), j // 2), ("wait", ("v_full",), j)]
            if j > 0:
                mma.append(("wait", ("o_empty",), j - 1))
            mma += [("read", ("scores", j % 2), j), ("read", ("v",), j), ("write", ("o",), j), ("arrive", ("v_empty",), j),
                    ("arrive", ("o_full",), j)]

    for i in range(n + 1):
        if i < n:
            sl = i % SCALE_RING
            soft += [("wait", ("sc_full", sl), i // SCALE_RING), ("wait", ("s_full", i % 2), i // 2),
                     ("read", ("scales", sl), i), ("read", ("scores", i % 2), i), ("arrive", ("p_full", i % 2), i // 2),
                     ("arrive", ("sc_empty", sl), i // SCALE_RING)]
        if i > 0:
            soft += [("wait", ("o_full",), i - 1), ("read", ("o",), i - 1), ("arrive", ("o_empty",), i - 1)]

    def put_pages(j):
        scale.extend([("write", ("pages", j % ring), j), ("arrive", ("pg_full", j % ring), j // ring)])

    for j in range(min(n, ahead)):
        put_pages(j)
    for i in range(n):
        sl = i % SCALE_RING
        if i >= SCALE_RING:
            scale.append(("wait", ("sc_empty", sl), (i - SCALE_RING) // SCALE_RING))
        if i + ahead < n:
            put_pages(i + ahead)
        scale += [("write", ("scales", sl), i), ("arrive", ("sc_full", sl), i // SCALE_RING)]
    return {"conv": conv, "mma": mma, "soft": soft, "scale": scale}


def clocks(prog):
    """Vector clock of every step: how many steps of each role are ordered before it by program order and barriers.
    Raises if the programs wait for one another for good."""
    arrived, at = {}, {r: 0 for r in prog}
    now = {r: {q: 0 for q in prog} for r in prog}
    done = {r: [] for r in prog}
    moved = True
    while moved:
        moved = False
        for r, steps in prog.items():
            while at[r] < len(steps):
                kind, name, x = steps[at[r]]
                if kind == "wait":
                    if (name, x) not in arrived:
                        break
                    for q, t in arrived[name, x].items():
                        now[r][q] = max(now[r][q], t)
                at[r] += 1
                now[r][r] = at[r]
                if kind == "arrive":
                    assert (name, x) not in arrived and (x == 0 or (name, x - 1) in arrived)
                    arrived[name, x] = dict(now[r])
                done[r].append(dict(now[r]))
                moved = True
    assert all(at[r] == len(s) for r, s in prog.items()), "the roles wait for one another"
    return done


def unordered(n, ring, ahead):
    """Reuses of a buffer, and phases of a barrier, that overtake a step that still needs the one before."""
    prog = roles(n, ring, ahead)
    done = clocks(prog)
    bad = []
    uses, waits = {}, {}
    for r, steps in prog.items():
        for t, (kind, name, x) in enumerate(steps):
            if kind in ("read", "write"):
                uses.setdefault(name, []).append((x, kind, r, t))
            elif kind == "wait":
                waits.setdefault((name, x), []).append((r, t))
    before = lambda r, t, q, u: done[q][u][r] > t  # step t of role r comes before step u of role q
    for name, us in uses.items():
        for x, kind, r, t in us:
            for y, other, q, u in us:
                # a value is written before it is read (once per half for the operands), and its place is written
                # again behind its last use
                if other == "write" and y > x and not before(r, t, q, u):
                    bad.append((name, x, kind, r, "overtaken by", y, q))
                if kind == "write" and other == "read" and x == y and not before(r, t, q, u):
                    bad.append((name, x, "read before it is written", q))
    for r, steps in prog.items():
        for t, (kind, name, x) in enumerate(steps):
            if kind == "arrive" and x > 0:
                for q, u in waits.get((name, x - 1), []):
                    if not before(q, u, r, t):  # the waiter would take the phase after next for this one
                        bad.append((name, x, "completes before the wait for the phase before it", q))
    return bad


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 7, 8, 9, 10, 15, 16, 17, 18, 19, 31, 32, 33, 40, 64])
def test_every_buffer_is_reused_behind_its_last_use(n):
    assert unordered(n, *page_ring()) == []


def test_the_model_sees_a_missing_wait():
    """Eight slots written three blocks ahead: the second half of V of block m is read behind the arrival that lets
    the slot's next pages in, from nine blocks on."""
    assert unordered(8, 8, 3) == [] and unordered(9, 8, 3) != []
    bad = unordered(40, 8, 3)
    assert bad and {b[0][0] for b in bad} == {"pages"}
    assert unordered(40, 8, 2) == [] and unordered(40, 16, 3) == []
    with pytest.raises(AssertionError, match="wait for one another"):
        clocks({"a": [("wait", ("x",), 0), ("arrive", ("y",), 0)], "b": [("wait", ("y",), 0), ("arrive", ("x",), 0)]})


@pytest.mark.parametrize("name", ["attn_paged.cu", "kv_append.cu", "sampling.cu"])
def test_barriers_do_not_count_on_converged_warps(name):
    """Barriers stand behind branches on the lane; in PTX's aligned forms (`bar` is one) a warp's threads must come
    together, which such a branch does not promise."""
    asm = " ".join(re.findall(r'"((?:[^"\\]|\\.)*)"', open(os.path.join(CSRC, name)).read()))
    barriers = re.findall(r"\b(?:bar|barrier)\.[\w.:]+", asm)
    assert [b for b in barriers if ".aligned" in b or b.startswith("bar.")] == []
    assert barriers or name == "kv_append.cu"
