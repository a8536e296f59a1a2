"""One workspace for linear attention calls of many sizes.  Nothing here reaches CUDA: the calls are refused for the
workspace's size (6) or, where that would do, for its alignment (3), which is checked after it."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def L():
    from gated_deltanet_recurrence_prefill_b200 import build, _lib
    build.build()
    return _lib.lib()


P, OFF = C.c_void_p(0x10000), C.c_void_p(0x20010)


def prefill(L, n, T, heads, ws_bytes):
    Hqk, Hv = heads
    return L.gdn_linear_prefill(P, P, P, 0, 0, 0, P, 1, P, n, T, Hqk, Hv, 128, 0.1, None, None, P, 1, OFF, ws_bytes, None)


def backward(L, n, T, heads, ws_bytes):
    Hqk, Hv = heads
    return L.gdn_linear_prefill_backward(P, P, P, 0, 0, 0, P, 1, P, n, T, Hqk, Hv, 128, 0.1, None, P, None, P, P, P, 1, P,
                                         None, OFF, ws_bytes, None)


@pytest.mark.parametrize("heads", [(1, 1), (4, 12), (16, 48), (16, 16)], ids=str)
@pytest.mark.parametrize("n,T", [(1, 1024), (4, 1088), (4, 1024), (16, 8192), (33, 9000), (64, 4096), (1, 65536), (2, 700000)])
def test_a_workspace_serves_all_smaller_calls(L, heads, n, T):
    lengths = sorted({max(1, T * i // 41) for i in range(42)} | {T - 1, T - 63, T - 64, T - 65, 1, 63, 64, 65, 960, 4096, 4097})
    for size, call in ((L.gdn_linear_prefill_workspace_size, prefill), (L.gdn_linear_prefill_backward_workspace_size, backward)):
        ws = size(n, T, *heads, 128)
        for n2 in sorted({1, 2, 3, n // 2, n - 1, n, 32, 33}):
            for T2 in lengths:
                if 0 < n2 <= n and T2 <= T:
                    assert call(L, n2, T2, heads, ws) == 3, (call.__name__, n2, T2)
                    # and the size asked for is always enough
                    assert call(L, n2, T2, heads, size(n2, T2, *heads, 128)) == 3


def test_a_workspace_without_the_least_is_refused(L):
    assert prefill(L, 4, 5000, (16, 48), 255) == 6
    assert prefill(L, 4, 5000, (16, 48), 256) == 3
    fixed = 256 + 2 * 5000 * 48 * 4 + 5000 * 16 * 512
    assert backward(L, 4, 5000, (16, 48), fixed) == 6
