"""Roles of the dense attention that give up a wait: no partner is left at a hardware barrier.

The kernel's waits on mbarriers are bounded; its hardware barriers between warps are not.
On the CPU: the source leaves a role that meets others there only by way of the barriers
still owed, and a model of those roles ends for every pair of places to give up.
"""
import itertools
import os
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "compressed_sparse_attention_fp4_gb300",
                   "csrc", "dense.cu")


def body(name):
    """Source of function `name`, comments taken out."""
    text = re.sub(r"//[^\n]*", "", open(SRC).read())
    at = re.search(r"__device__ inline \w+ " + name + r"\([^{]*\{", text).end()
    depth, i = 1, at
    while depth:
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        i += 1
    return text[at:i]


def gives_up(text):
    """What follows each failed wait."""
    return [m.group(1) for m in re.finditer(r"!wait_warp(?:<\w+>)?\([^;{]*?\)\)\s*(\{[^}]*\}|[^;]*;)", text)]


@pytest.mark.parametrize("role,waits", [("softmax_role", 3), ("widen_role", 6)])
def test_roles_with_hardware_barriers_leave_by_them(role, waits):
    text = body(role)
    assert "some_sync(" in text
    out = gives_up(text)
    assert len(out) >= waits
    for o in out:
        assert "goto leave" in o and "return" not in o, o
    assert re.search(r"return;\s*leave", text)                # the ordinary end does not pass the owed barriers


def test_queries_give_up_before_their_barriers_only():
    text = body("queries_to_tmem")
    assert text.rindex("wait_warp(") < text.index("some_sync(")
    assert "!queries_to_tmem" not in re.sub(r"!queries_to_tmem<\w+>\([^;]*\)\) goto leave_queries;", "", body("widen_role"))


def test_no_other_role_uses_hardware_barriers():
    text = re.sub(r"//[^\n]*", "", open(SRC).read())
    inside = sum(len(re.findall(r"some_(?:sync|arrive)\(k", body(n))) for n in ("softmax_role", "widen_role", "queries_to_tmem"))
    assert len(re.findall(r"some_(?:sync|arrive)\(", text)) == inside + 2       # and the two definitions
    assert len(re.findall(r'"bar\.\w+', text)) == 2


# --- a model of the roles: each step is a wait that may be given up, or a meeting at a barrier ----------------------
def softmax_warp(half, items, owed):
    """Steps of the warp of the even (0) or odd (1) blocks of one lane quarter; send(True) gives the wait up."""
    n1 = 0
    for at, (blocks, live) in enumerate(items):
        yield "sync", "turn"
        n0, n1 = n1, n1 + blocks
        n = n0 + ((half ^ n0) & 1)
        while n < n1:
            left = yield "wait", None                         # scores of the block
            if not left and not live:
                left = yield "wait", None                     # slot of P
            if not left and live:
                if n != n0:
                    yield "sync", ("ref", half ^ 1)
                if n + 1 != n1:
                    yield "arrive", ("ref", half)
                left = yield "wait", None                     # slot of P
                if left:
                    n += 2
            if left:
                if not owed:
                    return
                rest = list(items[at + 1:])
                while True:
                    while live and n < n1:
                        if n != n0:
                            yield "sync", ("ref", half ^ 1)
                        if n + 1 != n1:
                            yield "arrive", ("ref", half)
                        n += 2
                    if not rest:
                        return
                    blocks, live = rest.pop(0)
                    yield "sync", "turn"
                    n0, n1 = n1, n1 + blocks
                    n = n0 + ((half ^ n0) & 1)
            n += 2


def query_warp(items, owed):
    for at, (blocks, _) in enumerate(items):
        left = yield "wait", None
        for _ in range(0 if left else 2):
            yield "sync", "q"
        tiles = 1 if left else 0
        for _ in range(blocks):
            if left:
                break
            left = yield "wait", None
        if left:
            for _ in range(2 * (tiles + len(items) - at - 1) if owed else 0):
                yield "sync", "q"
            return


def ends(warps, give_up):
    """Whether all warps end; warp w gives its give_up[w]-th wait up.  A barrier opens when all `warps` have come."""
    step = [next(w) for w in warps]
    waits, come, held = [0] * len(warps), {}, [None] * len(warps)
    moved = True
    while moved:
        moved = False
        for i, w in enumerate(warps):
            while step[i] is not None and held[i] is None:
                moved = True
                kind, bar = step[i]
                answer = None
                if kind == "wait":
                    answer = waits[i] == give_up[i]
                    waits[i] += 1
                else:
                    assert i not in come.setdefault(bar, set())                # never twice in one phase
                    come[bar].add(i)
                    if len(come[bar]) == len(warps):
                        come[bar] = set()
                        held = [None if h == bar else h for h in held]
                    elif kind == "sync":
                        held[i] = bar
                try:
                    step[i] = w.send(answer)
                except StopIteration:
                    step[i] = None
    return all(s is None for s in step)


ITEMS = [[(1, True)], [(2, True), (3, True)], [(5, True), (1, True), (4, False), (2, True)], [(3, False), (4, True), (7, True)]]


@pytest.mark.parametrize("items", ITEMS)
def test_softmax_warps_end_wherever_they_give_up(items):
    stuck = 0
    for give_up in itertools.product(range(-1, 2 * sum(b for b, _ in items) + 1), repeat=2):
        assert ends([softmax_warp(h, items, True) for h in (0, 1)], give_up), give_up
        stuck += not ends([softmax_warp(h, items, False) for h in (0, 1)], give_up)
    assert stuck > 0 or items == ITEMS[0]                    # without the owed barriers some do not


@pytest.mark.parametrize("items", ITEMS)
def test_query_warps_end_wherever_they_give_up(items):
    stuck = 0
    for give_up in itertools.product(range(-1, sum(b + 1 for b, _ in items)), repeat=3):
        assert ends([query_warp(items, True) for _ in range(3)], give_up), give_up
        stuck += not ends([query_warp(items, False) for _ in range(3)], give_up)
    assert stuck > 0
