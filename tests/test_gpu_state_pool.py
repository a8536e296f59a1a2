"""The state cache's page operations on the GPU, bit for bit against the same moves in numpy."""
import numpy as np
import pytest

from tests.helpers import dev_i32

pytestmark = pytest.mark.gpu


def cache(n_slots, seed=0, big=False):
    """Buffers of several types and slot sizes: a last item of 16 bytes, one below an item, one of several items."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(n_slots, *s, generator=g, device="cuda")  # noqa: E731
    out = [r(2, 3, 64, 65), r(4), r(20, 36).bfloat16(), r(3, 128 * 12, 3)]
    if big:
        out.append(r(5, 128, 128).bfloat16())
    return out


def pages(buffers):
    import torch
    return [b.clone().view(torch.uint8).reshape(b.shape[0], -1).cpu().numpy() for b in buffers]


def same(buffers, want):
    return all(np.array_equal(a, b) for a, b in zip(pages(buffers), want))


def copy_ref(old, src, dst):
    n = old[0].shape[0]
    new = [b.copy() for b in old]
    for s, d in zip(src, dst):
        if 0 <= s < n and 0 <= d < n:
            for x, y in zip(old, new):
                y[d] = x[s]
    return new


@pytest.mark.parametrize("n_slots,src,dst", [
    (1, [0], [0]),
    (2, [1, 0], [0, 1]),                                   # a swap
    (6, [1, 2, 3, 4, 5, 0], [0, 1, 2, 3, 4, 5]),           # a rotation
    (6, [2, 2, 2, 0], [0, 1, 3, 2]),                       # one page to several, while it is overwritten
    (5, [0, 1, 2], [4, 4, 4]),                             # one destination: the last holds
    (5, [0, 3], [3, 3]),                                   # the last leaves it as it was
    (5, [0, 7, -1, 2, 9], [4, 4, 1, 5, -3]),               # void entries
    (5, [0, 7], [4, 4]),                                   # a void entry does not hide an earlier one
    (4, [], []),
], ids=str)
def test_copy(n_slots, src, dst):
    import gated_deltanet_recurrence_prefill_b200 as gdn
    b = cache(n_slots)
    want = copy_ref(pages(b), src, dst)
    gdn.state_copy(b, dev_i32(src), dev_i32(dst))
    assert same(b, want)


@pytest.mark.parametrize("n_slots,n", [(50, 50), (300, 257), (1100, 1024), (40, 700)])
def test_copy_many(n_slots, n):
    import gated_deltanet_recurrence_prefill_b200 as gdn
    rng = np.random.default_rng(n)
    src = rng.integers(-1, n_slots + 1, n)
    dst = rng.permutation(n_slots)[:n] if n <= n_slots else rng.integers(0, n_slots, n)
    b = cache(n_slots, seed=n, big=n_slots <= 300)
    want = copy_ref(pages(b), src, dst)
    gdn.state_copy(b, dev_i32(src), dev_i32(dst))
    assert same(b, want)


def fork_ref(old, live, src):
    new, live, dst = [b.copy() for b in old], live.copy(), []
    free = [s for s in range(len(live)) if not live[s]]
    was = live.copy()
    for s in src:
        if not (s == -1 or (0 <= s < len(was) and was[s])) or not free:
            dst.append(-1)
            continue
        d = free.pop(0)
        dst.append(d)
        live[d] = 1
        for x, y in zip(old, new):
            y[d] = x[s] if s >= 0 else 0
    return new, live, dst


@pytest.mark.parametrize("n_slots,n,share", [(1, 1, 0.0), (7, 3, 0.4), (7, 9, 0.5), (64, 20, 0.9), (40, 13, 1.0),
                                             (2500, 1500, 0.3)])
def test_fork(n_slots, n, share):
    import gated_deltanet_recurrence_prefill_b200 as gdn
    rng = np.random.default_rng(n_slots + n)
    live = (rng.random(n_slots) < share).astype(np.int32) * rng.integers(1, 5, n_slots).astype(np.int32)
    src = rng.integers(-2, n_slots + 1, n)
    b = cache(n_slots, seed=n)[: 2 if n_slots > 100 else None]
    want, wlive, wdst = fork_ref(pages(b), live, src)
    dl = dev_i32(live)
    dst = gdn.state_fork(b, dl, dev_i32(src))
    assert dst.tolist() == wdst
    assert np.array_equal(dl.cpu().numpy() != 0, wlive != 0)
    assert same(b, want)
    gdn.state_free(dl, dst)                                # the -1 among them are ignored
    assert np.array_equal(dl.cpu().numpy() != 0, live != 0)


@pytest.mark.parametrize("n_slots,share", [(1, 0.0), (1, 1.0), (2, 0.5), (9, 0.5), (40, 0.0), (40, 1.0), (97, 0.3),
                                           (97, 0.8), (2100, 0.5)])
def test_compact(n_slots, share):
    import gated_deltanet_recurrence_prefill_b200 as gdn
    rng = np.random.default_rng(n_slots)
    live = (rng.random(n_slots) < share).astype(np.int32)
    b = cache(n_slots, seed=3)[: 2 if n_slots > 100 else None]
    old = pages(b)
    dl = dev_i32(live)
    moved = gdn.state_compact(b, dl).cpu().numpy()
    left = int(live.sum())
    assert np.array_equal(dl.cpu().numpy(), (np.arange(n_slots) < left).astype(np.int32))
    new = pages(b)
    assert sorted(moved[live != 0]) == list(range(left)) and (moved[live == 0] == -1).all()
    for s in np.nonzero(live)[0]:
        assert s >= left or moved[s] == s                  # a page already in front stays
        assert all(np.array_equal(x[moved[s]], y[s]) for x, y in zip(new, old))
    late = [moved[s] for s in np.nonzero(live)[0] if s >= left]
    assert late == sorted(late)


def test_free_ignores_slots_outside():
    import gated_deltanet_recurrence_prefill_b200 as gdn
    import torch
    guard = torch.ones(12, dtype=torch.int32, device="cuda")
    live = guard[4:8]
    gdn.state_free(live, dev_i32([-1, 4, 2, 100, 2]))
    assert guard.tolist() == [1] * 6 + [0] + [1] * 5
    gdn.state_free(live, dev_i32([]))


def test_pages_outside_the_lists_and_beyond_the_cache_stay():
    """Moves write only the named pages: the cache lies in a larger buffer with patterned margins."""
    import torch
    import gated_deltanet_recurrence_prefill_b200 as gdn
    raw = torch.full((4096 + 10 * 1040 + 4096,), 77, dtype=torch.uint8, device="cuda")
    page = raw[4096:4096 + 10 * 1040].view(10, 1040)
    page.copy_(torch.randint(0, 255, (10, 1040), dtype=torch.uint8, device="cuda"))
    want = copy_ref([page.cpu().numpy()], [3, 9], [5, 0])
    gdn.state_copy(page, dev_i32([3, 9]), dev_i32([5, 0]))
    assert same([page], want)
    live = dev_i32([1, 0, 1, 1, 0, 1, 1, 1, 1, 1])
    gdn.state_fork(page, live, dev_i32([-1, 9]))
    assert (raw[:4096] == 77).all() and (raw[-4096:] == 77).all()
    assert not page[1].any() and torch.equal(page[4], page[9])


def test_offsets_past_32_bits():
    """Pages whose byte offsets do not fit 32 bits."""
    import torch
    import gated_deltanet_recurrence_prefill_b200 as gdn
    b = torch.empty(5, 1 << 28, dtype=torch.float32, device="cuda")          # pages of 1 GiB
    for i in range(5):
        b[i] = i + 1
    gdn.state_copy(b, dev_i32([4, 0]), dev_i32([0, 4]))
    assert [float(b[i, 0]) for i in range(5)] == [5, 2, 3, 4, 1] and [float(b[i, -1]) for i in range(5)] == [5, 2, 3, 4, 1]
    live = dev_i32([0, 1, 0, 0, 1])
    moved = gdn.state_compact(b, live)
    assert moved.tolist() == [-1, 1, -1, -1, 0] and float(b[0, 12345678]) == 1
    assert gdn.state_fork(b, live, dev_i32([1, -1])).tolist() == [2, 3]
    assert float(b[2, -1]) == 2 and float(b[3].abs().max()) == 0


def test_captured_and_replayed():
    import torch
    import gated_deltanet_recurrence_prefill_b200 as gdn
    b = cache(9, seed=5)
    start = [x.clone() for x in b]
    live0 = dev_i32([1, 1, 0, 1, 1, 0, 1, 1, 0])
    live, src, dst, done, fresh = live0.clone(), dev_i32([0, 1, 3]), dev_i32([3, 0, 1]), dev_i32([1]), dev_i32([0, -1])

    def go():
        gdn.state_copy(b, src, dst)
        gdn.state_free(live, done)
        moved = gdn.state_compact(b, live)
        return moved, gdn.state_fork(b, live, fresh)
    first = go()
    want = [x.clone() for x in b]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = go()
    for _ in range(2):
        for x, y in zip(b, start):
            x.copy_(y)
        live.copy_(live0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(b, want))
        assert all(torch.equal(x, y) for x, y in zip(first, held))


def test_copies_of_few_and_many_pages_at_once():
    """Calls from several threads, whose kernels need different amounts of shared memory."""
    import threading
    import torch
    import gated_deltanet_recurrence_prefill_b200 as gdn
    rng = np.random.default_rng(3)
    sizes = (4, 700, 1024, 300)
    lists = [[rng.permutation(n) for _ in range(60)] for n in sizes]
    caches = [[torch.arange(n * 48, device="cuda", dtype=torch.int32).view(n, 48)] for n in sizes]
    want = [c[0].cpu().numpy() for c in caches]
    device = [[dev_i32(p) for p in l] for l in lists]
    places = [dev_i32(np.arange(n)) for n in sizes]
    streams = [torch.cuda.Stream() for _ in sizes]
    torch.cuda.synchronize()
    failed = []

    def run(k):
        try:
            for p in device[k]:
                gdn.state_copy(caches[k], p, places[k], stream=streams[k])
        except Exception as e:  # noqa: BLE001
            failed.append(e)
    threads = [threading.Thread(target=run, args=(k,)) for k in range(len(sizes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for k in range(len(sizes)):
        for p in lists[k]:
            want[k] = want[k][p]
        assert np.array_equal(caches[k][0].cpu().numpy(), want[k])
