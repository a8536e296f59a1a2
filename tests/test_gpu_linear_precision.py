"""How precise linear attention is, in the norm over each output (tests/linear_bounds.py derives the bounds and
tests/test_linear_bounds.py shows what they tell apart): dq, dk, dg and the states are made in float32 throughout; o and
dv carry the rounding to bf16 of the state that the tokens meet, and no other before their own."""
import pytest

from tests.helpers import dev_bf16, dev_f32, dev_i32, host
from tests.linear_bounds import Exact
from tests.test_gpu_linear import LENGTHS, Case

pytestmark = pytest.mark.gpu

CASES = [(lengths, "mixed") for lengths in LENGTHS + [[500, 40, 300], [1500, 40, 900]]] + \
        [([150, 33, 320], gates) for gates in ("none", "strong", "reset")]


def run(c, dtype):
    import gated_deltanet_recurrence_prefill_b200 as gdn
    q, k, v, g = c.dev()
    opt = lambda x: None if x is None else dev_f32(x)  # noqa: E731
    cu = dev_i32(c.cu)
    o, _ = gdn.linear_prefill(q, k, v, g, cu_seqlens=cu, scale=c.scale, initial_state=opt(c.s0), o_dtype=dtype)
    r = gdn.linear_prefill_backward(q, k, v, g, dev_bf16(c.dob), d_final_state=opt(c.dfin), cu_seqlens=cu, scale=c.scale,
                                    initial_state=opt(c.s0), grad_dtype=dtype)
    return {n: host(x) for n, x in dict(r, o=o).items()}


@pytest.mark.parametrize("lengths,gates", CASES, ids=str)
@pytest.mark.parametrize("Hqk,Hv,init", [(2, 2, True), (1, 3, False), (1, 3, True)])
def test_precision(lengths, gates, Hqk, Hv, init):
    import torch
    c = Case(800, lengths, Hqk, Hv, gates=gates, init=init)
    e = Exact(c)
    r = run(c, torch.float32)
    e.check_exact_passes(r)
    for name in ("o", "dv"):
        e.check_output_pass(r[name], name, False)
    r = run(c, torch.bfloat16)
    for name in ("o", "dv"):
        e.check_output_pass(r[name], name, True)


def test_precision_where_the_passes_take_turns():
    """Enough heads and parts that dq and dk are launches of their own, and sequences in several parts."""
    import torch
    c = Case(801, [700, 333], 16, 32)
    e = Exact(c)
    r = run(c, torch.float32)
    e.check_exact_passes(r)
    for name in ("o", "dv"):
        e.check_output_pass(r[name], name, False)
