"""The fp64 reference of linear attention (oracle/linear.py) against closed forms and differences, and the refusals
of the new entry points, which are checked on the host and need no GPU."""
import ctypes as C

import numpy as np
import pytest

from oracle import linear as ref


def case(seed, lengths, Hqk, Hv, d=8, per_head=False):
    rng = np.random.default_rng(seed)
    T = sum(lengths)
    n = lambda *s: rng.standard_normal(s)  # noqa: E731
    g = -rng.uniform(0.0, 1.5, Hv if per_head else (T, Hv))
    cu = np.concatenate([[0], np.cumsum(lengths)])
    return dict(q=n(T, Hqk, d), k=n(T, Hqk, d), v=n(T, Hv, d), g=g, cu_seqlens=cu, scale=0.37,
                initial_state=n(len(lengths), Hv, d, d)), n(T, Hv, d), n(len(lengths), Hv, d, d)


def test_reference_is_the_sum_over_earlier_tokens():
    a, _, _ = case(1, [5, 0, 7], 2, 4)
    o, fin, _ = ref.prefill(**a)
    q, k = ref._spread(a["q"], 4), ref._spread(a["k"], 4)
    for n in range(3):
        for t in range(a["cu_seqlens"][n], a["cu_seqlens"][n + 1]):
            G = lambda s: np.exp(a["g"][s + 1:t + 1].sum(0))  # noqa: B023, E731
            want = np.einsum("h,hij,hj->hi", G(a["cu_seqlens"][n] - 1), a["initial_state"][n], q[t])
            for s in range(a["cu_seqlens"][n], t + 1):
                want += (G(s) * (q[t] * k[s]).sum(-1))[:, None] * a["v"][s]
            np.testing.assert_allclose(o[t], a["scale"] * want, rtol=1e-10, atol=1e-12)
    np.testing.assert_array_equal(fin[1], a["initial_state"][1])


@pytest.mark.parametrize("per_head", [False, True])
def test_reference_gradients_against_differences(per_head):
    a, d_o, d_fin = case(2, [4, 0, 6], 2, 4, per_head=per_head)

    def loss(**kw):
        o, fin, _ = ref.prefill(**dict(a, **kw))
        return (o * d_o).sum() + (fin * d_fin).sum()

    grads = ref.prefill_backward(d_o=d_o, d_final_state=d_fin, **a)
    rng = np.random.default_rng(3)
    for name, gname in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("initial_state", "d_initial_state")):
        direction = rng.standard_normal(a[name].shape)
        h = 1e-5
        diff = (loss(**{name: a[name] + h * direction}) - loss(**{name: a[name] - h * direction})) / (2 * h)
        want = (grads[gname] * direction).sum()
        # a central difference is off by h^2 / 6 times the third derivative and by 64-bit rounding / h
        assert abs(diff - want) <= 1e-7 * max(1.0, abs(want)), name


def test_gradients_are_three_passes_of_the_operator():
    """dq is the operator on (d_o, v, k) with the state transposed; dk and dv are it backwards in time."""
    a, d_o, d_fin = case(4, [6, 5], 4, 4)
    grads = ref.prefill_backward(d_o=d_o, d_final_state=d_fin, **a)
    t = lambda s: s.transpose(0, 1, 3, 2)  # noqa: E731
    dq, _, _ = ref.prefill(d_o, a["v"], a["k"], a["g"], a["cu_seqlens"], a["scale"], t(a["initial_state"]))
    np.testing.assert_allclose(dq, grads["dq"], rtol=1e-10, atol=1e-12)
    # backwards in time the decay of a token acts behind it: shift the gates by one
    for n in range(2):
        s, e = a["cu_seqlens"][n], a["cu_seqlens"][n + 1]
        g = np.concatenate([a["g"][s + 1:e], np.zeros((1, 4))])[::-1]
        flip = lambda x: x[s:e][::-1]  # noqa: B023, E731
        cu = [0, e - s]
        dk, _, _ = ref.prefill(flip(a["v"]), flip(a["scale"] * d_o), flip(a["q"]), g, cu, 1.0, t(d_fin[n:n + 1]))
        dv, last, _ = ref.prefill(flip(a["k"]), flip(a["q"]), flip(a["scale"] * d_o), g, cu, 1.0, d_fin[n:n + 1])
        np.testing.assert_allclose(dk[::-1], grads["dk"][s:e], rtol=1e-10, atol=1e-12)
        np.testing.assert_allclose(dv[::-1], grads["dv"][s:e], rtol=1e-10, atol=1e-12)
        np.testing.assert_allclose(np.exp(a["g"][s])[:, None, None] * last[0], grads["d_initial_state"][n],
                                   rtol=1e-10, atol=1e-12)


# ---- refusals: nothing below reaches CUDA -------------------------------------------------------

@pytest.fixture(scope="module")
def L():
    from gated_deltanet_recurrence_prefill_b200 import build, _lib
    build.build()
    return _lib.lib()


FAKE = 0x10000


def p(x=FAKE):
    return C.c_void_p(x)


def test_linear_prefill_refuses(L):
    ws = L.gdn_linear_prefill_workspace_size(1, 64, 16, 48, 128)
    assert ws > 0 and ws % 256 == 0

    def call(q=p(), ldq=0, ldv=0, g=p(), per=1, cu=None, n=1, T=64, Hqk=16, Hv=48, d=128, o=p(), o16=1, w=p(0x20000), wb=ws):
        return L.gdn_linear_prefill(q, p(), p(), ldq, 0, ldv, g, per, cu, n, T, Hqk, Hv, d, 0.1, None, None, o, o16,
                                    w, wb, None)
    assert call(d=64) == 2 and call(Hv=40) == 2 and call(T=2 ** 31) == 2
    assert call(Hqk=0) == 1 and call(T=-1) == 1 and call(n=2) == 1 and call(q=None) == 1 and call(g=None) == 1
    assert call(per=2) == 1 and call(o16=-1) == 1
    assert call(ldq=16 * 128 - 8) == 1 and call(ldv=48 * 128 + 4) == 3
    assert call(o=p(FAKE + 8)) == 3 and call(cu=p(FAKE + 4)) == 3
    assert call(w=None) == 6 and call(wb=ws - 1) == 6 and call(w=p(0x20010)) == 3


def test_linear_backward_refuses(L):
    ws = L.gdn_linear_prefill_backward_workspace_size(1, 64, 16, 48, 128)
    assert ws > 0 and ws % 256 == 0

    def call(d_o=p(), dg=p(), per=1, d0=None, df=None, g16=1, T=64, d=128, w=p(0x20000), wb=ws):
        return L.gdn_linear_prefill_backward(p(), p(), p(), 0, 0, 0, p(), per, None, 1, T, 16, 48, d, 0.1, None, d_o,
                                             df, p(), p(), p(), g16, dg, d0, w, wb, None)
    assert call(d=96) == 2 and call(d_o=None) == 1 and call(dg=None) == 1 and call(g16=2) == 1
    assert call(dg=None, per=0, T=0) == 1
    assert call(d0=p(0x30000), df=p(0x30000)) == 1
    assert call(d_o=p(FAKE + 2)) == 3 and call(wb=ws - 1) == 6 and call(w=None) == 6


def test_linear_decode_refuses(L):
    def call(q=p(), state=p(), slot=None, n_seq=4, layers=2, Hv=48, d=128, n_slots=4, s16=0, o16=0):
        return L.gdn_linear_decode_step(q, p(), p(), p(), 1, slot, n_seq, layers, 16, Hv, d, 0.1, n_slots, state, s16,
                                        p(), o16, None)
    assert call(d=64) == 2 and call(Hv=47) == 2 and call(n_seq=2 ** 30) == 1 and call(slot=p(), n_seq=2 ** 30) == 2
    assert call(layers=0) == 1 and call(n_slots=3) == 1 and call(state=None) == 1 and call(s16=3) == 1
    assert call(q=p(FAKE + 4)) == 3
    assert call(q=None, n_seq=0) == 0


def test_state_pool_refuses(L):
    from gated_deltanet_recurrence_prefill_b200._lib import StateBuffer
    ok = (StateBuffer * 9)(*[StateBuffer(0x10000 * (i + 1), 64) for i in range(9)])
    odd = (StateBuffer * 1)(StateBuffer(0x10000, 40))
    off = (StateBuffer * 1)(StateBuffer(0x10008, 64))
    none = (StateBuffer * 1)(StateBuffer(None, 64))
    assert L.gdn_state_copy(ok, 9, 4, p(), p(), 1, None) == 2
    assert L.gdn_state_copy(ok, 1, 4, p(), p(), 1025, None) == 2
    assert L.gdn_state_copy(odd, 1, 4, p(), p(), 1, None) == 3
    assert L.gdn_state_copy(off, 1, 4, p(), p(), 1, None) == 3
    assert L.gdn_state_copy(none, 1, 4, p(), p(), 1, None) == 1
    assert L.gdn_state_copy(ok, 1, 0, p(), p(), 1, None) == 1
    assert L.gdn_state_copy(ok, 1, 4, None, p(), 1, None) == 1
    assert L.gdn_state_copy(ok, 1, 4, p(FAKE + 2), p(), 1, None) == 3
    assert L.gdn_state_copy(ok, 1, 4, p(), p(), 0, None) == 0
    twice = (StateBuffer * 2)(StateBuffer(0x10000, 64), StateBuffer(0x10080, 64))
    assert L.gdn_state_copy(twice, 2, 4, p(), p(), 1, None) == 1                             # they overlap
    assert L.gdn_state_copy(twice, 2, 2, p(), p(), 0, None) == 0
    ws = L.gdn_state_workspace_size(4)
    assert ws > 0
    assert L.gdn_state_fork(ok, 1, 4, p(), p(), p(), 2, p(0x20000), ws, None) == 1          # src is dst
    assert L.gdn_state_fork(ok, 1, 4, None, p(), p(0x11000), 2, p(0x20000), ws, None) == 1
    assert L.gdn_state_fork(ok, 1, 4, p(), p(), p(0x11000), 2, p(0x20000), ws - 1, None) == 6
    assert L.gdn_state_fork(ok, 1, 4, p(), p(), p(0x11000), 0, None, 0, None) == 0
    assert L.gdn_state_compact(ok, 1, 4, p(), None, p(0x20000), ws, None) == 1
    assert L.gdn_state_compact(ok, 1, 4, p(), p(0x11000), None, 0, None) == 6
    assert L.gdn_state_free(None, 4, p(), 1, None) == 1
    assert L.gdn_state_free(p(), 4, None, 1, None) == 1
    assert L.gdn_state_free(p(), 4, None, 0, None) == 0


def test_refuses_long_lists_and_outputs_in_place_of_inputs(L):
    from gated_deltanet_recurrence_prefill_b200._lib import StateBuffer
    b = (StateBuffer * 1)(StateBuffer(0x10000, 64))
    ws = L.gdn_state_workspace_size(4)
    a1, a2, w, most = p(0x11000), p(0x12000), p(0x20000), 2 ** 31 - 1
    assert L.gdn_state_fork(b, 1, 4, p(), a1, a2, most, w, ws, None) == 2
    assert L.gdn_state_fork(b, 1, 4, p(), a1, p(), 2, w, ws, None) == 1                     # dst is live
    assert L.gdn_state_compact(b, 1, 4, p(), p(), w, ws, None) == 1                         # moved is live
    assert L.gdn_state_free(p(), 4, a1, most, None) == 2
    assert L.gdn_state_free(p(), most, a1, 1, None) == 2
    ws = L.gdn_linear_prefill_backward_workspace_size(1, 64, 16, 48, 128)
    s0 = p(0x30000)
    assert L.gdn_linear_prefill_backward(p(), p(), p(), 0, 0, 0, p(), 1, None, 1, 64, 16, 48, 128, 0.1, s0, p(), None,
                                         p(), p(), p(), 1, p(), s0, w, ws, None) == 1       # d_initial is initial


def test_binding_refuses_host_tensors_and_shapes():
    import torch
    import gated_deltanet_recurrence_prefill_b200 as gdn
    q = torch.zeros(4, 1, 128, dtype=torch.bfloat16)
    g = torch.zeros(4, 2)
    v = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        gdn.linear_prefill(q, q, v, g)                                   # not on a GPU
    with pytest.raises(ValueError):
        gdn.linear_prefill(q, q[:3], v, g)
    with pytest.raises(TypeError):
        gdn.linear_prefill(q.float(), q, v, g)
    with pytest.raises(ValueError):
        gdn.linear_prefill(q.transpose(0, 1).contiguous().transpose(0, 1)[:, :, ::2], q, v, g)
    with pytest.raises(ValueError):
        gdn.state_copy([torch.zeros(3, 8), torch.zeros(4, 8)], torch.zeros(1, dtype=torch.int32),
                       torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        gdn.state_copy([torch.zeros(8, 3).t()], torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
