"""The hand-overs between the roles of the linear attention passes, read from their source.

A missing fence shows in no result that a test could compare (the hardware mostly orders what the memory model leaves
open), so the order is read from the text of linear_walk.cuh, function by function, in the order in which it stands.
"""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = os.path.join(ROOT, "gated_deltanet_recurrence_prefill_b200", "csrc", "linear_walk.cuh")


def functions():
    """{name: body} of the source's device functions and kernels, without comments."""
    text = re.sub(r"/\*.*?\*/", "", re.sub(r"//[^\n]*", "", open(SRC).read()), flags=re.S)
    out = {}
    for m in re.finditer(r"^(?:GDN_DEVICE [^;{}]*?|lin_walk_kernel)\b(\w+)?\([^;{}]*\)\s*(?:const )?\{", text, re.M):
        name = re.findall(r"(\w+)\(", m.group(0))[0]
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        out[name] = text[m.end():i - 1]
    return out


BODIES = functions()
# (function, barrier): what the waiter lets the asynchronous proxy (TMA, the tensor cores) read or overwrite in shared
# memory, the threads that arrive have written with ordinary stores
ASYNC_NEXT = [("state_role", "bStateIn"), ("weight_role", "bZeroed"), ("weight_role", "bZDone"),
              ("score_role", "bPReady"), ("out_role", "bRows")]


def test_all_roles_are_read():
    assert {"load_role", "decay_role", "kv_role", "out_products_role", "weight_role", "score_role", "put_state",
            "state_role", "out_role", "lin_walk_kernel"} <= set(BODIES)


@pytest.mark.parametrize("role,barrier", ASYNC_NEXT)
def test_ordinary_stores_are_fenced_before_the_asynchronous_proxy_may_have_the_bytes(role, barrier):
    """Every thread runs fence.proxy.async between its last ordinary access and the arrival: the fence, then the warp
    together, then one lane's arrival."""
    body = BODIES[role]
    arrivals = list(re.finditer(r"mbar_arrive\(c\.bar\(L::kBars, L::%s\b[^;]*;" % barrier, body))
    assert arrivals
    for a in arrivals:
        before = body[:a.start()]
        sync = before.rindex("__syncwarp()")
        assert re.fullmatch(r"__syncwarp\(\);[\s}]*if \(lane == 0\) \{?\s*", before[sync:]), "the warp, then one lane"
        fence = before.rfind("fence_async_smem()")
        assert fence >= 0, f"{role} arrives on {barrier} without a proxy fence"
        between = before[fence:sync]
        assert not re.search(r"\*reinterpret_cast|load_state|store_state|clear_rows|stmatrix|ldmatrix", between)


TMEM = re.compile(r"c\.wait\(|wait_set<|tc_fence_after\(\)|\btmem_(?:ld|st)\w*\(|\bput_state<|\bmma_bf16\w*\(|\bscores\(|"
                  r"__syncthreads\(\)|\btmem_dealloc\(")


@pytest.mark.parametrize("role", ["kv_role", "out_products_role", "weight_role", "score_role", "state_role", "out_role",
                                  "lin_walk_kernel"])
def test_tensor_memory_is_touched_behind_a_fence(role):
    """After a wait tcgen05.fence::after_thread_sync comes before the next tcgen05 operation (tmem_st_wait orders the
    thread's own stores and needs none)."""
    waited = False
    for m in TMEM.finditer(BODIES[role]):
        what = m.group(0)
        if "wait(" in what and "tmem" not in what or "wait_set" in what or "syncthreads" in what:
            waited = True
        elif "tc_fence_after" in what:
            waited = False
        elif what != "tmem_st_wait(":
            assert not waited, f"{role}: {what} after a wait without tcgen05.fence::after_thread_sync"


class Barrier:
    """An mbarrier: a phase ends with its last arrival."""

    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def passed(self, parity):                    # what mbarrier.try_wait.parity tells
        return self.phase & 1 != parity & 1


def output_rows(sets, slow, order, chunks=12):
    """The output's four warps of one half and the thread that issues the products, one step of one of them at a time:
    `slow` gets a step only when nobody else can take one.  Returns the chunks whose rows warp 0 sent away before all
    four warps had put theirs in place."""
    full, free, rows = Barrier(1), Barrier(4), [Barrier(4) for _ in range(sets)]
    placed, early = [0] * 4, []

    def products():
        for n in range(chunks):
            while n > 0 and not free.passed(n - 1):
                yield False
            full.arrive()
            yield True

    def warp(w):
        for n in range(chunks):
            while not full.passed(n):
                yield False
            free.arrive()                        # its part of the products is read ...
            yield True
            placed[w] = n + 1                    # ... and only then are its rows in place
            yield True
            rows[n % sets].arrive()
            yield True
            if w == 0:
                while not rows[n % sets].passed(n // sets):
                    yield False
                if min(placed) <= n:
                    early.append(n)
                yield True

    agents = {"products": products(), **{w: warp(w) for w in range(4)}}
    while agents:
        for name in sorted(agents, key=lambda a: (a == slow, order.index(a))):
            step = next(agents[name], None)
            if step is None:
                del agents[name]
                break
            if step:
                break
        else:
            raise AssertionError("nobody can take a step")
    return early


def test_the_output_leaves_when_all_warps_have_it_in_place():
    """Whichever warp falls behind: with the barriers that the source has, and not with one."""
    layout = re.search(r"bRows = (\w+) \+ 1, bDrain = bRows \+ (\d+),", open(SRC).read())
    sets = int(layout.group(2)) // 2             # (of each half)
    names = ["products", 0, 1, 2, 3]
    found = []
    for count in (1, sets):
        found.append([early for slow in names for order in (names, names[::-1]) for early in [output_rows(count, slow, order)]
                      if early])
    assert found[0] and not found[1]
