"""The bounds of tests/linear_bounds.py on emulated passes: float32 arithmetic is within them, one rounding to bf16 too
many is not."""
import numpy as np
import pytest

from oracle import linear as ref
from tests.linear_bounds import Exact, bf16, gradients, norm, walk
from tests.test_gpu_linear import LENGTHS, Case

CASES = [(lengths, gates) for lengths in LENGTHS + [[500, 40, 300]] for gates in ("mixed",)] + \
        [([150, 33, 320], gates) for gates in ("none", "strong", "reset")]


def case(lengths, gates, Hv=3, init=True):
    return Case(700, lengths, 1, Hv, gates=gates, init=init)


@pytest.mark.parametrize("lengths,gates", CASES, ids=str)
def test_bounds_tell_float32_from_bf16(lengths, gates):
    c = case(lengths, gates)
    e = Exact(c)
    fold = e.fold

    def taken(**how):
        dq, dk, dg = gradients(c, **how)
        return dict(dq=fold(dq.astype(np.float64)), dk=fold(dk.astype(np.float64)), dg=dg)
    e.check_exact_passes(taken(dtype=np.float32))
    both = taken(round_state=bf16, round_scores=bf16)
    with pytest.raises(AssertionError, match="dq"):
        e.check_exact_passes(both)
    for name in ("dq", "dk", "dg"):                                # each of them by itself
        if name == "dg" and c.T == 1:                              # (known at both ends of one token)
            continue
        with pytest.raises(AssertionError, match=name):
            e.check_exact_passes(dict(taken(), **{name: both[name]}))
    for name, args in (("o", dict(x=c.q, y=c.k, z=c.v, init=c.s0)),
                       ("dv", dict(x=c.k, y=c.q, z=c.do, init=c.dfin, backward=True))):
        run = lambda **how: walk(args["x"], args["y"], args["z"], c.gr, c.cu, c.scale, args.get("backward", False),  # noqa: B023, E731
                                 args["init"], **how)[0]
        once = run(round_state=bf16, dtype=np.float32)
        e.check_output_pass(once, name, False)
        e.check_output_pass(bf16(once), name, True)
        with pytest.raises(AssertionError, match=name):
            e.check_output_pass(bf16(once), name, False)
        state = e.o_state if name == "o" else e.dv_state
        want = e.o if name == "o" else e.dv
        if norm(want - state) > 0.6 * norm(want):                   # scores that make up most of it
            with pytest.raises(AssertionError, match=name):
                e.check_output_pass(run(round_state=bf16, round_scores=bf16, dtype=np.float32), name, False)


@pytest.mark.parametrize("lengths", [[1], [65, 0, 130]], ids=str)
def test_the_emulation_is_the_reference(lengths):
    c = case(lengths, "mixed")
    e = Exact(c)
    want = ref.prefill_backward(c.q, c.k, c.v, c.gr, c.cu, c.scale, c.do, c.s0, c.dfin)
    o = ref.prefill(c.q, c.k, c.v, c.gr, c.cu, c.scale, c.s0)[0]
    for got, x in ((e.o, o), (e.fold(e.dq), want["dq"]), (e.fold(e.dk), want["dk"]), (e.dv, want["dv"]), (e.dg, want["dg"])):
        np.testing.assert_allclose(got, x, rtol=1e-9, atol=1e-9 * np.abs(x).max())
