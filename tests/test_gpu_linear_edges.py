"""Linear attention with a decay per head where a value that does not count must not show: infinities and NaN at other
tokens, decays far below those that matter, what a workspace held or was made for."""
import numpy as np
import pytest

from oracle import linear as ref
from tests.helpers import dev_bf16, dev_f32, dev_i32, host
from tests.test_gpu_linear import Case, check_backward, check_prefill, close

pytestmark = pytest.mark.gpu

D = 128


# ---- infinities and NaN -------------------------------------------------------------------------
# One bad value at one token.  It reaches the outputs that the formulas compute from it, which are then not finite, and
# none of the others, which are those of the same call without it: bit for bit, where nothing that they are made of has
# changed.  (dg is exempt: a running sum over the sequence, it may be NaN throughout.)

LENGTHS = [150, 30, 70]


def outputs(c, q, k, v, g, d_o, dtype):
    import gated_deltanet_recurrence_prefill_b200 as gdn
    cu, s0, dfin = dev_i32(c.cu), dev_f32(c.s0), dev_f32(c.dfin)
    o, fin = gdn.linear_prefill(q, k, v, g, cu_seqlens=cu, scale=c.scale, initial_state=s0, o_dtype=dtype)
    r = gdn.linear_prefill_backward(q, k, v, g, d_o, d_final_state=dfin, cu_seqlens=cu, scale=c.scale,
                                    initial_state=s0, grad_dtype=dtype)
    out = dict(o=o, fin=fin, dq=r["dq"], dk=r["dk"], dv=r["dv"], d0=r["d_initial_state"])
    return {n: x.float().cpu().numpy() for n, x in out.items()}


def reached(c, which, m, head, i, out):
    """{output: the elements that depend on the bad one}: token m of the sequence [t0, t1), value head `head` (its key
    head), element i."""
    n = int(np.searchsorted(c.cu, m, "right")) - 1
    t0, t1 = int(c.cu[n]), int(c.cu[n + 1])
    rep = c.Hv // c.Hqk
    kh = head // rep
    vh = slice(kh * rep, kh * rep + rep) if which in ("q", "k") else head         # the value heads that see it
    on = {name: np.zeros(x.shape, bool) for name, x in out.items()}
    now, later, earlier = slice(m, m + 1), slice(m, t1), slice(t0, m + 1)
    if which == "q":
        on["o"][now, vh] = True
        on["dk"][earlier, kh, i] = True
        on["dv"][earlier, vh] = True
        on["d0"][n, vh, :, i] = True
    elif which == "k":
        on["o"][later, vh] = True
        on["fin"][n, vh, :, i] = True
        on["dq"][later, kh, i] = True
        on["dv"][now, vh] = True
    elif which == "v":
        on["o"][later, vh, i] = True
        on["fin"][n, vh, i] = True
        on["dq"][later, kh] = True
        on["dk"][now, kh] = True
    elif which == "d_o":
        on["dq"][now, kh] = True
        on["dk"][earlier, kh] = True
        on["dv"][earlier, vh, i] = True
        on["d0"][n, vh, i] = True
    return on


# the token: the first and last of a chunk of a sequence, and some inside, whole chunks and cut ones
@pytest.mark.parametrize("m", [0, 11, 31, 63, 64, 100, 149, 150, 165, 179, 249])
@pytest.mark.parametrize("which", ["q", "k", "v", "d_o"])
@pytest.mark.parametrize("Hqk,Hv", [(2, 2), (1, 3)])
def test_one_bad_value_reaches_what_depends_on_it_only(which, m, Hqk, Hv):
    import torch
    c = Case(300 + m, LENGTHS, Hqk, Hv)
    q, k, v, g = c.dev()
    d_o = dev_bf16(c.dob)
    head, i = Hv - 1, (37 * m + 5) % D
    for bad, dtype in ((float("nan"), torch.bfloat16), (float("inf"), torch.float32), (-float("inf"), torch.bfloat16)):
        clean = outputs(c, q, k, v, g, d_o, dtype)
        x = dict(q=q, k=k, v=v, d_o=d_o)
        hit = x[which].clone()
        hit[m, head if which in ("v", "d_o") else head // (Hv // Hqk), i] = bad
        x[which] = hit
        got = outputs(c, x["q"], x["k"], x["v"], g, x["d_o"], dtype)
        on = reached(c, which, m, head, i, got)
        for name in got:
            assert not np.isfinite(got[name][on[name]]).any(), (name, bad)
            assert np.array_equal(got[name][~on[name]], clean[name][~on[name]]), (name, bad)


def test_many_bad_values():
    """Several tokens and elements of a chunk, both signs, at once: each element of o turns at its first one."""
    import gated_deltanet_recurrence_prefill_b200 as gdn
    c = Case(77, [200], 1, 1)
    q, k, v, g = c.dev()
    clean = gdn.linear_prefill(q, k, v, g, scale=c.scale, initial_state=dev_f32(c.s0))[0].float().cpu().numpy()
    rng = np.random.default_rng(4)
    first = np.full(D, 200)
    for _ in range(60):
        m, i = int(rng.integers(64, 200)), int(rng.integers(0, D))
        v[m, 0, i] = float(rng.choice([np.nan, np.inf, -np.inf]))
        first[i] = min(first[i], m)
    o = gdn.linear_prefill(q, k, v, g, scale=c.scale, initial_state=dev_f32(c.s0))[0].float().cpu().numpy()
    on = np.arange(200)[:, None] >= first
    assert not np.isfinite(o[:, 0][on]).any() and np.array_equal(o[:, 0][~on], clean[:, 0][~on])


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


# ---- decays ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("every", [2, 3, 7])
@pytest.mark.parametrize("reset", [-float("inf"), -104.0, -60.0])
def test_scores_between_resets(every, reset):
    """Many resets in a chunk take the sum of its log decays far away (64 / 2 of them to -4,800 in base 2, where float32
    numbers are 2^-11 apart), and the scores of the tokens between two of them, whose decays are ordinary, keep their
    digits: 2^-16 of each by their two bf16 parts, and as much again for the 128 products, the decay, the sum over the
    few tokens that count and the scale.  q and k are positive, so that a score is as large as its products'
    magnitudes.  One rounded exponent a token would be off by up to 2^-12 ln 2 twice, 3e-4 of a score.  (Behind the
    first chunk of a sequence the state's copy adds half a step of bf16, 2^-8, of what comes from the state: the
    magnitudes of the whole without those of the chunks by themselves.)"""
    import torch
    import gated_deltanet_recurrence_prefill_b200 as gdn
    c = Case(500 + every, [64, 50, 128], 2, 4, init=False)
    q, k, v, g = c.dev()
    q, k = q.abs(), k.abs()
    g[::every] = reset
    g[1::every] = -0.01 - g[1::every].abs() % 0.7
    o, _ = gdn.linear_prefill(q, k, v, g, cu_seqlens=dev_i32(c.cu), scale=c.scale, o_dtype=torch.float32)
    gr = np.maximum(host(g), -104.0)
    want = ref.prefill(host(q), host(k), c.v, gr, c.cu, c.scale)[0]
    m, _ = ref.sizes(host(q), host(k), c.v, gr, c.cu, c.scale)
    chunks = np.concatenate([np.arange(a, b, 64) for a, b in zip(c.cu[:-1], c.cu[1:])] + [c.cu[-1:]])
    alone, _ = ref.sizes(host(q), host(k), c.v, gr, chunks, c.scale)
    close(o, want, 2.0 ** -15 * m + 2.0 ** -8 * (m - alone) + 1e-30, "o")


# ---- workspaces -----------------------------------------------------------------------------------

def test_a_workspace_made_for_a_larger_call():
    """Every shorter call works in it, though one of its own might be larger, and it may hold anything."""
    import torch
    import gated_deltanet_recurrence_prefill_b200 as gdn
    Hqk, Hv, most = 1, 2, [300, 200, 1300, 61]
    back = gdn.lib().gdn_linear_prefill_backward_workspace_size
    size = max(gdn.linear_prefill_workspace_size(4, sum(most), Hqk, Hv), back(4, sum(most), Hqk, Hv, D))
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    for i, lengths in enumerate([most, [1088], [960, 1], [300, 0, 41, 2], [64], [1]]):
        check_with(Case(600 + i, lengths, Hqk, Hv), ws, ws)


@pytest.mark.parametrize("lengths", [[1100, 40, 300], [4200], [30] * 39 + [1500]], ids=["three", "one", "listed"])
def test_workspaces_smaller_than_the_fastest_plan_wants(lengths):
    """The least, and half of what is between it and the full size: other cuts, the same results up to rounding.  A byte
    less than the least is refused."""
    import torch
    import gated_deltanet_recurrence_prefill_b200 as gdn
    c = Case(620, lengths, 1, 2)
    n, T = len(lengths), sum(lengths)
    full = gdn.linear_prefill_workspace_size(n, T, 1, 2)
    most = gdn.lib().gdn_linear_prefill_backward_workspace_size(n, T, 1, 2, D)
    # what the gradients cannot do without: dot products, dk's or dq's sums, final states, and for parts of 4,096 tokens
    # their sums of dg, starting states and decays in both directions, and lists
    up = lambda x: -(-x // 256) * 256  # noqa: E731
    parts = n if T <= 4096 else T // 4096 + n
    split = T > 4096
    joints = 2 * up(parts * 2 * D * D * 4) + 2 * up(parts * 2 * 4) if split else 0
    lists = up((parts + T // 4096 + n + 1) * 4) if split and n > 32 else 0
    least = 256 + 2 * up(T * 2 * 4) + up(T * D * 4) + up(n * 2 * D * D * 4) + up(parts * 2 * 8) + joints + lists
    assert full > 256 and most > least
    for share in (0.0, 0.5):
        pre, back = (int(a + share * (b - a)) // 256 * 256 for a, b in ((256, full), (least, most)))
        check_with(c, torch.full((pre,), 255, dtype=torch.uint8, device="cuda"),
                   torch.full((back,), 255, dtype=torch.uint8, device="cuda"))
    q, k, v, g = c.dev()
    with pytest.raises(RuntimeError):
        gdn.linear_prefill_backward(q, k, v, g, dev_bf16(c.dob), cu_seqlens=dev_i32(c.cu),
                                    workspace=torch.empty(least - 1, dtype=torch.uint8, device="cuda"))


def check_with(c, ws_prefill, ws_backward):
    import gated_deltanet_recurrence_prefill_b200 as gdn
    q, k, v, g = c.dev()
    cu, s0 = dev_i32(c.cu), dev_f32(c.s0)
    o, fin = gdn.linear_prefill(q, k, v, g, cu_seqlens=cu, scale=c.scale, initial_state=s0, workspace=ws_prefill)
    check_prefill(c, o, fin, True)
    assert gdn.prefill_status(ws_prefill) == 0
    r = gdn.linear_prefill_backward(q, k, v, g, dev_bf16(c.dob), d_final_state=dev_f32(c.dfin), cu_seqlens=cu,
                                    scale=c.scale, initial_state=s0, workspace=ws_backward)
    check_backward(c, r, True)
    assert gdn.prefill_status(ws_backward) == 0
