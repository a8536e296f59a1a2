"""Linear attention with a decay per head where a value that does not count must not show: infinities and NaN at other
tokens."""
import numpy as np
import pytest

from tests.helpers import dev_bf16, dev_f32, dev_i32
from tests.test_gpu_linear import Case

pytestmark = pytest.mark.gpu

D = 128


# ---- infinities and NaN -------------------------------------------------------------------------
# One bad value at one token.  It reaches the outputs that the formulas compute from it, which are then not finite, and
# none of the others, which are those of the same call without it.  (dg is exempt: a running sum over the sequence, it may
# be NaN throughout.)

LENGTHS = [150, 30, 70]


def outputs(c, q, k, v, g, d_o, dtype):
    import gated_deltanet_recurrence_prefill_b200 as gdn
    cu, s0, dfin = dev_i32(c.cu), dev_f32(c.s0), dev_f32(c.dfin)
    o, fin = gdn.linear_prefill(q, k, v, g, cu_seqlens=cu, scale=c.scale, initial_state=s0, o_dtype=dtype)
    r = gdn.linear_prefill_backward(q, k, v, g, d_o, d_final_state=dfin, cu_seqlens=cu, scale=c.scale,
                                    initial_state=s0, grad_dtype=dtype)
    out = dict(o=o, fin=fin, dq=r["dq"], dk=r["dk"], dv=r["dv"], d0=r["d_initial_state"])
    return {n: x.float().cpu().numpy() for n, x in out.items()}


@pytest.mark.parametrize("m", [0, 11, 63, 64, 100, 149, 160])
def test_a_nan_decay_reaches_what_depends_on_it_only(m):
    """g_m is in o_t and dq_t from t = m on, and in dk_t and dv_t in front of m."""
    import torch
    c = Case(400 + m, LENGTHS, 1, 2)
    q, k, v, g = c.dev()
    d_o = dev_bf16(c.dob)
    clean = outputs(c, q, k, v, g, d_o, torch.float32)
    hit = g.clone()
    hit[m, 1] = float("nan")
    got = outputs(c, q, k, v, hit, d_o, torch.float32)
    n = int(np.searchsorted(c.cu, m, "right")) - 1
    t0, t1 = int(c.cu[n]), int(c.cu[n + 1])
    on = {name: np.zeros(x.shape, bool) for name, x in got.items()}
    on["o"][m:t1, 1] = on["dq"][m:t1] = on["fin"][n, 1] = on["d0"][n, 1] = True
    on["dk"][t0:m] = on["dv"][t0:m, 1] = True
    for name in got:
        assert np.isnan(got[name][on[name]]).all(), name
        # sums of other decays start elsewhere: an exponent moves by 2^-20 at most, a part of a score by 2^-16
        a, b = got[name][~on[name]], clean[name][~on[name]]
        assert np.abs(a - b).max() <= 2.0 ** -14 * np.abs(b).max(), name
