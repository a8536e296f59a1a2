"""Linear attention with a decay per head on the GPU against the fp64 reference (oracle/linear.py).

Tolerances.  Half a step of bf16 is 2^-8 of a value, of float32 2^-24.
 * o, dq, dk, dv: the score matrix and the state the tokens meet are rounded to bf16 (2^-8 of the magnitudes m that
   they multiply, oracle.linear.sizes), the result once more when it is stored as bf16 (2^-8 of itself).  The float32
   part is far smaller: fp32 tolerance below, of the same m.
 * states, dg and the step: float32.  A sum of n terms is off by at most n 2^-24 of the sum of magnitudes, a decay
   by 2^-21 (argument and exponential) per chunk it is chained over, and the tensor cores may cut instead of round
   (2^-23); with n <= 64 + 8 chunks that is below (96 + 24 chunks) 2^-23 of the sum of magnitudes.
"""
import numpy as np
import pytest

from oracle import linear as ref
from tests.helpers import dev_bf16, dev_f32, dev_i32, host

pytestmark = pytest.mark.gpu

B16 = 2.0 ** -8
D = 128


def f32_tol(n_tokens):
    return (96 + 24 * (-(-n_tokens // 64))) * 2.0 ** -23


def bits(x):
    """float -> bf16 bit patterns, cut (exact values of their own)."""
    return (np.ascontiguousarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def wide(b):
    return (b.astype(np.uint32) << 16).view(np.float32)


class Case:
    def __init__(self, seed, lengths, Hqk, Hv, per_head=False, init=True, gates="mixed", tail=0):
        rng = np.random.default_rng(seed)
        self.T, self.Hqk, self.Hv, self.N = sum(lengths), Hqk, Hv, len(lengths)
        rows = self.T + tail
        self.rows = rows
        n = lambda *s: rng.standard_normal(s)  # noqa: E731
        unit = lambda x: x / np.sqrt((x * x).sum(-1, keepdims=True) + 1e-6)  # noqa: E731
        self.qb, self.kb = bits(unit(n(rows, Hqk, D))), bits(unit(n(rows, Hqk, D)))
        self.vb, self.dob = bits(n(rows, Hv, D)), bits(n(rows, Hv, D))
        shape = (Hv,) if per_head else (rows, Hv)
        g = -np.exp(rng.uniform(-7.8, -0.3, shape))
        if gates == "reset" and not per_head:
            g[rng.random(shape) < 0.1] = -np.inf
            g[rng.random(shape) < 0.1] = np.finfo(np.float32).min
        if gates == "none":
            g[:] = 0.0
        if gates == "strong":
            g = -np.exp(rng.uniform(0.0, 4.0, shape))
        self.g = g.astype(np.float32)
        self.cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
        self.scale = 0.11
        self.s0 = (0.5 * n(self.N, Hv, D, D)).astype(np.float32) if init else None
        self.dfin = (0.3 * n(self.N, Hv, D, D)).astype(np.float32) if init else None
        T = self.T
        self.q, self.k, self.v, self.do = (wide(x)[:T] for x in (self.qb, self.kb, self.vb, self.dob))
        self.gr = np.maximum(self.g if per_head else self.g[:T], -104.0)

    def dev(self, packed=False):
        q, k, v = dev_bf16(self.qb), dev_bf16(self.kb), dev_bf16(self.vb)
        if packed:
            import torch
            row = torch.cat([x.flatten(1) for x in (q, k, v)], 1)
            q, k, v = (x.unflatten(1, (-1, D)) for x in row.split([self.Hqk * D, self.Hqk * D, self.Hv * D], 1))
        return q, k, v, dev_f32(self.g)


def close(x, want, tol, name):
    x = host(x)
    assert np.isfinite(x).all(), name
    off = np.abs(x - want) - tol
    at = np.unravel_index(np.argmax(off), off.shape)
    assert off[at] <= 0, f"{name}{at}: {x[at]} against {want[at]}, off by {abs(x[at] - want[at])}, allowed {np.broadcast_to(tol, off.shape)[at]}"


def check_prefill(c, o, fin, o16):
    want, wfin, _ = ref.prefill(c.q, c.k, c.v, c.gr, c.cu, c.scale, c.s0)
    m, size = ref.sizes(c.q, c.k, c.v, c.gr, c.cu, c.scale, initial_state=c.s0)
    t32 = f32_tol(max(np.diff(c.cu)))
    if o is not None:
        close(o[:c.T], want, (B16 + t32) * m + (B16 * np.abs(want) if o16 else 0) + 1e-30, "o")
    if fin is not None:
        close(fin, wfin, t32 * size + 1e-30, "final_state")


LENGTHS = [
    [1], [2], [63], [64], [65], [128], [200],
    [1, 63, 64, 0, 65, 130],
    [0, 0, 3], [5, 0],
    [700],
    [129, 257, 1],
]


@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
@pytest.mark.parametrize("Hqk,Hv", [(1, 1), (2, 6)])
def test_prefill(lengths, Hqk, Hv):
    import torch
    import gated_deltanet_recurrence_prefill_b200 as gdn
    for i, (per_head, init, o16, packed) in enumerate([(False, True, True, False), (True, False, False, True)]):
        c = Case(100 + i, lengths, Hqk, Hv, per_head=per_head, init=init)
        q, k, v, g = c.dev(packed)
        o, fin = gdn.linear_prefill(q, k, v, g, cu_seqlens=dev_i32(c.cu), scale=c.scale,
                                    initial_state=None if c.s0 is None else dev_f32(c.s0),
                                    o_dtype=torch.bfloat16 if o16 else torch.float32)
        check_prefill(c, o, fin, o16)


@pytest.mark.parametrize("gates", ["none", "strong", "reset"])
def test_prefill_gates(gates):
    import gated_deltanet_recurrence_prefill_b200 as gdn
    c = Case(7, [150, 33, 320], 2, 4, gates=gates)
    q, k, v, g = c.dev()
    o, fin = gdn.linear_prefill(q, k, v, g, cu_seqlens=dev_i32(c.cu), scale=c.scale, initial_state=dev_f32(c.s0))
    check_prefill(c, o, fin, True)


def test_prefill_many_parts():
    """A length whose sequences are worked on in several parts."""
    import gated_deltanet_recurrence_prefill_b200 as gdn
    c = Case(8, [1500, 40, 900], 1, 2)
    q, k, v, g = c.dev()
    o, fin = gdn.linear_prefill(q, k, v, g, cu_seqlens=dev_i32(c.cu), scale=c.scale, initial_state=dev_f32(c.s0))
    check_prefill(c, o, fin, True)


def test_prefill_single_sequence_default_arguments_and_in_place_state():
    import gated_deltanet_recurrence_prefill_b200 as gdn
    c = Case(9, [333], 2, 2)
    c.scale = D ** -0.5
    q, k, v, g = c.dev()
    s = dev_f32(c.s0)
    o, fin = gdn.linear_prefill(q, k, v, g, initial_state=s, final_state=s)
    assert fin.data_ptr() == s.data_ptr()
    check_prefill(c, o, fin, True)
    o2, none = gdn.linear_prefill(q, k, v, g, initial_state=dev_f32(c.s0), want_final_state=False)
    assert none is None and (o2.view(dtype=o.dtype) == o).all()


def test_prefill_no_tokens():
    import torch
    import gated_deltanet_recurrence_prefill_b200 as gdn
    c = Case(10, [0, 0], 1, 2)
    q, k, v, g = c.dev()
    s = dev_f32(c.s0)
    o, fin = gdn.linear_prefill(q, k, v, g, cu_seqlens=dev_i32(c.cu), initial_state=s)
    assert o.shape[0] == 0 and torch.equal(fin, s)
    _, fin = gdn.linear_prefill(q, k, v, g, cu_seqlens=dev_i32(c.cu))
    assert not fin.any()


@pytest.mark.parametrize("lengths", [[70, 61, 3], [1], [64], [200]], ids=str)
def test_rows_behind_the_last_sequence(lengths):
    """Rows that no sequence owns are not read (they hold NaN) and their outputs stay."""
    import torch
    import gated_deltanet_recurrence_prefill_b200 as gdn
    c = Case(11, lengths, 1, 2, tail=37)
    q, k, v, g = c.dev()
    for x in (q, k, v, g):
        x[c.T:] = float("nan")
    o = torch.full((c.rows, 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    _, fin = gdn.linear_prefill(q, k, v, g, cu_seqlens=dev_i32(c.cu), scale=c.scale, initial_state=dev_f32(c.s0), o=o)
    check_prefill(c, o, fin, True)
    assert (o[c.T:] == 7.0).all()
    d_o = dev_bf16(c.dob)
    d_o[c.T:] = float("inf")
    out = {n: torch.full((c.rows, h, D), 7.0, dtype=torch.bfloat16, device="cuda") for n, h in (("dq", 1), ("dk", 1), ("dv", 2))}
    out["dg"] = torch.full((c.rows, 2), 7.0, device="cuda")
    r = gdn.linear_prefill_backward(q, k, v, g, d_o, d_final_state=dev_f32(c.dfin), cu_seqlens=dev_i32(c.cu),
                                    scale=c.scale, initial_state=dev_f32(c.s0), out=out)
    check_backward(c, r, True)
    for n in ("dq", "dk", "dv", "dg"):
        assert (r[n][c.T:] == 7.0).all()


def test_a_sequence_with_nan_leaves_its_neighbours():
    import gated_deltanet_recurrence_prefill_b200 as gdn
    c = Case(12, [70, 30, 90], 1, 1)
    q, k, v, g = c.dev()
    s0 = dev_f32(c.s0)
    cu = dev_i32(c.cu)
    o, fin = gdn.linear_prefill(q, k, v, g, cu_seqlens=cu, scale=c.scale, initial_state=s0)
    for x, bad in ((v, float("nan")), (k, float("inf")), (q, float("nan")), (g, float("nan"))):
        x[75:100] = bad
    o2, fin2 = gdn.linear_prefill(q, k, v, g, cu_seqlens=cu, scale=c.scale, initial_state=s0)
    keep = [i for i in range(190) if not 70 <= i < 100]
    assert (o2[keep] == o[keep]).all()
    assert (fin2[[0, 2]] == fin[[0, 2]]).all()
    assert fin2[1].isnan().any()


# ---- gradients ----------------------------------------------------------------------------------

def check_backward(c, r, g16):
    want = ref.prefill_backward(c.q, c.k, c.v, c.gr, c.cu, c.scale, c.do, c.s0, c.dfin)
    t32 = f32_tol(max(np.diff(c.cu)))
    t = lambda s: None if s is None else s.transpose(0, 1, 3, 2)  # noqa: E731
    rep = c.Hv // c.Hqk
    fold = lambda m: m.reshape(c.T, c.Hqk, rep, D).sum(2)  # noqa: E731
    mq, _ = ref.sizes(c.do, c.v, c.k, c.gr, c.cu, c.scale, initial_state=t(c.s0))
    mk, _ = ref.sizes(c.v, c.do, c.q, c.gr, c.cu, c.scale, True, t(c.dfin))
    mv, dsize = ref.sizes(c.k, c.q, c.do, c.gr, c.cu, c.scale, True, c.dfin)
    for name, m in (("dq", fold(mq)), ("dk", fold(mk)), ("dv", mv)):
        close(r[name][:c.T], want[name], (B16 + t32) * m + (B16 * np.abs(want[name]) if g16 else 0) + 1e-30, name)
    if r["d_initial_state"] is not None:
        close(r["d_initial_state"], want["d_initial_state"], t32 * dsize + 1e-30, "d_initial_state")
    # dg_t = <S_end, dS_end> + sum of q.dq - k.dk behind t: float32 errors of those sums of magnitudes
    spread = lambda x: np.repeat(np.abs(x), c.Hv // x.shape[1], 1)  # noqa: E731
    rq, ck = (spread(c.q) * mq).sum(-1), (spread(c.k) * mk).sum(-1)
    fin = ref.sizes(c.q, c.k, c.v, c.gr, c.cu, c.scale, initial_state=c.s0)[1]
    tol = np.zeros_like(rq)
    for n in range(c.N):
        s, e = c.cu[n], c.cu[n + 1]
        end = 0.0 if c.dfin is None else (fin[n] * np.abs(c.dfin[n])).sum((1, 2))
        tol[s:e] = end + np.cumsum((rq + ck)[s:e][::-1], 0)[::-1]
    if c.gr.ndim == 1:
        close(r["dg"], want["dg"], t32 * tol.sum(0) + 1e-30, "dg")
    else:
        wd = np.where(c.gr <= -104.0, 0.0, want["dg"])
        close(r["dg"][:c.T], wd, t32 * tol + 1e-30, "dg")


@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
@pytest.mark.parametrize("Hqk,Hv", [(2, 2), (1, 3)])
def test_backward(lengths, Hqk, Hv):
    import torch
    import gated_deltanet_recurrence_prefill_b200 as gdn
    for i, (per_head, init, g16, packed) in enumerate([(False, True, True, False), (True, False, False, True)]):
        c = Case(200 + i, lengths, Hqk, Hv, per_head=per_head, init=init)
        q, k, v, g = c.dev(packed)
        opt = lambda x: None if x is None else dev_f32(x)  # noqa: E731
        r = gdn.linear_prefill_backward(q, k, v, g, dev_bf16(c.dob), d_final_state=opt(c.dfin), cu_seqlens=dev_i32(c.cu),
                                        scale=c.scale, initial_state=opt(c.s0), want_d_initial=init,
                                        grad_dtype=torch.bfloat16 if g16 else torch.float32)
        assert r["dq"].dtype == (torch.bfloat16 if g16 else torch.float32)
        check_backward(c, r, g16)


@pytest.mark.parametrize("gates", ["none", "strong", "reset"])
def test_backward_gates(gates):
    import gated_deltanet_recurrence_prefill_b200 as gdn
    c = Case(13, [150, 33, 320], 2, 4, gates=gates)
    q, k, v, g = c.dev()
    r = gdn.linear_prefill_backward(q, k, v, g, dev_bf16(c.dob), d_final_state=dev_f32(c.dfin), cu_seqlens=dev_i32(c.cu),
                                    scale=c.scale, initial_state=dev_f32(c.s0))
    check_backward(c, r, True)


def test_backward_many_parts():
    import gated_deltanet_recurrence_prefill_b200 as gdn
    c = Case(14, [1500, 40, 900], 1, 2)
    q, k, v, g = c.dev()
    r = gdn.linear_prefill_backward(q, k, v, g, dev_bf16(c.dob), d_final_state=dev_f32(c.dfin), cu_seqlens=dev_i32(c.cu),
                                    scale=c.scale, initial_state=dev_f32(c.s0))
    check_backward(c, r, True)


def test_backward_of_no_tokens():
    import torch
    import gated_deltanet_recurrence_prefill_b200 as gdn
    c = Case(15, [0, 0], 1, 2, per_head=True)
    q, k, v, g = c.dev()
    dfin = dev_f32(c.dfin)
    r = gdn.linear_prefill_backward(q, k, v, g, dev_bf16(c.dob), d_final_state=dfin, cu_seqlens=dev_i32(c.cu),
                                    initial_state=dev_f32(c.s0))
    assert torch.equal(r["d_initial_state"], dfin) and not r["dg"].any()


def test_many_sequences():
    """More sequences than a warp finds its part among, long, short and empty ones: some in several parts."""
    import gated_deltanet_recurrence_prefill_b200 as gdn
    lengths = [(37 * i) % 11 for i in range(70)] + [1400] + [(13 * i) % 7 for i in range(40)] + [700, 0]
    c = Case(16, lengths, 1, 2)
    q, k, v, g = c.dev()
    cu, s0, dfin = dev_i32(c.cu), dev_f32(c.s0), dev_f32(c.dfin)
    o, fin = gdn.linear_prefill(q, k, v, g, cu_seqlens=cu, scale=c.scale, initial_state=s0)
    check_prefill(c, o, fin, True)
    r = gdn.linear_prefill_backward(q, k, v, g, dev_bf16(c.dob), d_final_state=dfin, cu_seqlens=cu, scale=c.scale,
                                    initial_state=s0)
    check_backward(c, r, True)


def test_rows_past_32_bits():
    """A sequence whose rows start past 2^32 bytes gives what it gives alone ."""
    import torch
    import gated_deltanet_recurrence_prefill_b200 as gdn
    Hv, n = 16, 1100
    T = (1 << 32) // (Hv * D * 2) + n
    gen = torch.Generator(device="cuda").manual_seed(3)
    v = torch.zeros(T, Hv, D, dtype=torch.bfloat16, device="cuda")
    q, k = (torch.zeros(T, 2, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = torch.full((T, Hv), -0.05, device="cuda")
    for x in (q, k, v):
        x[-n:] = torch.randn(n, *x.shape[1:], generator=gen, device="cuda").bfloat16()
    g[-n:] = -torch.rand(n, Hv, generator=gen, device="cuda")
    cu = dev_i32([0, T - n, T])
    o, fin = gdn.linear_prefill(q, k, v, g, cu_seqlens=cu)
    assert not o[:T - n].any() and not fin[0].any()
    small = [x[-n:].clone() for x in (q, k, v, g)]
    o1, fin1 = gdn.linear_prefill(*small)
    want, wfin, _ = ref.prefill(host(small[0]), host(small[1]), host(small[2]), host(small[3]), [0, n], D ** -0.5)
    m, size = ref.sizes(host(small[0]), host(small[1]), host(small[2]), host(small[3]), [0, n], D ** -0.5)
    for oo, ff in ((o[-n:], fin[1:]), (o1, fin1)):
        close(oo, want, (B16 + f32_tol(n)) * m + B16 * np.abs(want) + 1e-30, "o")
        close(ff, wfin, f32_tol(n) * size + 1e-30, "final_state")
    d_o = torch.zeros_like(v)
    d_o[-n:] = torch.randn(n, Hv, D, generator=gen, device="cuda").bfloat16()
    r = gdn.linear_prefill_backward(q, k, v, g, d_o, cu_seqlens=cu)
    r1 = gdn.linear_prefill_backward(*small, d_o[-n:].clone())
    for name in ("dq", "dk", "dv", "dg"):
        a, b = r[name][-n:].float(), r1[name].float()
        # the cuts may differ: the same to the rounding of the result and of what enters it
        assert (a - b).norm() <= 4 * B16 * b.norm(), name
        assert not r[name][:T - n].any(), name


# ---- one token ----------------------------------------------------------------------------------

@pytest.mark.parametrize("n_seq,layers,Hqk,Hv", [(1, 1, 1, 1), (1, 3, 2, 6), (5, 2, 2, 4), (40, 2, 4, 12), (9, 7, 16, 48)])
@pytest.mark.parametrize("s16", [False, True])
def test_decode(n_seq, layers, Hqk, Hv, s16):
    import torch
    import gated_deltanet_recurrence_prefill_b200 as gdn
    for per_unit, use_slot, o16 in ((True, True, False), (False, False, True)):
        rng = np.random.default_rng(n_seq + 10 * layers + s16)
        n = lambda *s: rng.standard_normal(s)  # noqa: E731
        U, slots = n_seq * layers, n_seq + 2
        qb, kb, vb = bits(n(U, Hqk, D)), bits(n(U, Hqk, D)), bits(n(U, Hv, D))
        g = -np.exp(rng.uniform(-8, 2, (U if per_unit else layers, Hv))).astype(np.float32)
        g[0, 0] = -np.inf
        S = n(slots * layers, Hv, D, D).astype(np.float32)
        Sb = bits(S) if s16 else None
        S = wide(Sb) if s16 else S
        slot = rng.permutation(slots)[:n_seq].astype(np.int32) if use_slot else None
        if use_slot and n_seq > 2:
            slot[1], slot[2] = -1, slots                     # rows without a sequence
        st = dev_bf16(Sb) if s16 else dev_f32(S)
        with np.errstate(all="ignore"):
            o, after = ref.decode(wide(qb), wide(kb), wide(vb), g, S, slot, n_seq, layers, 0.2)
            size, sizes = ref.decode(np.abs(wide(qb)), np.abs(wide(kb)), np.abs(wide(vb)), g, np.abs(S), slot, n_seq, layers, 0.2)
        got = gdn.linear_decode_step(dev_bf16(qb), dev_bf16(kb), dev_bf16(vb), dev_f32(g), st, n_seq, layers,
                                     slot=None if slot is None else dev_i32(slot), scale=0.2,
                                     o_dtype=torch.bfloat16 if o16 else None)
        # a dot product of 128 terms, an exponential and a product: (128 + 8) 2^-24 of the sum of magnitudes
        t32 = 136 * 2.0 ** -24
        close(got, o, t32 * size + (B16 * np.abs(o) if o16 else 0) + 1e-30, "o")
        close(st, after, t32 * sizes + (B16 * np.abs(after) if s16 else 0) + 1e-30, "state")
        if use_slot:
            idle = [s for s in range(slots) if s not in set(slot.tolist())]
            flat = host(st).reshape(slots, layers, Hv, D, D)[idle]
            assert np.array_equal(flat, S.reshape(slots, layers, Hv, D, D)[idle])


# ---- together, as they are used -----------------------------------------------------------------

def test_a_serving_run():
    """Prompts prefilled, their states put into a cache, one forked, tokens decoded, one sequence ended, the cache
    compacted, more tokens: every output equals the same tokens' in one long prefill."""
    import torch
    import gated_deltanet_recurrence_prefill_b200 as gdn
    lens, steps, Hqk, Hv = [90, 17, 130], 6, 2, 4
    c = Case(21, [n + steps for n in lens], Hqk, Hv, per_head=True, init=False)
    q, k, v, g = c.dev()
    whole, _ = gdn.linear_prefill(q, k, v, g, cu_seqlens=dev_i32(c.cu), scale=c.scale, o_dtype=torch.float32)
    want, _, _ = ref.prefill(c.q, c.k, c.v, c.gr, c.cu, c.scale)
    m, _ = ref.sizes(c.q, c.k, c.v, c.gr, c.cu, c.scale)
    rows = np.concatenate([np.arange(c.cu[i], c.cu[i] + n) for i, n in enumerate(lens)])
    at = torch.from_numpy(rows).cuda()
    cu = dev_i32(np.concatenate([[0], np.cumsum(lens)]))
    _, fin = gdn.linear_prefill(q[at], k[at], v[at], g, cu_seqlens=cu, scale=c.scale)
    cache = torch.full((8, 1, Hv, D, D), float("nan"), device="cuda")
    conv = torch.arange(8.0, device="cuda").view(8, 1, 1, 1).repeat(1, 1, 8, 3).contiguous()
    live = torch.zeros(8, dtype=torch.int32, device="cuda")
    slots = gdn.state_fork([cache, conv], live, dev_i32([-1, -1, -1]))
    assert slots.tolist() == [0, 1, 2] and not cache[:3].any() and not conv[:3].any()
    cache[slots.long(), 0] = fin
    twin = gdn.state_fork([cache, conv], live, slots[:1])                     # a second sample of sequence 0
    assert twin.tolist() == [3] and torch.equal(cache[3], cache[0])
    rows_of = {0: 0, 1: 1, 2: 2, 3: 0}
    place = {0: 0, 1: 1, 2: 2, 3: 3}
    for t in range(steps):
        if t == 3:                                                            # sequence 1 ends
            gdn.state_free(live, dev_i32([place.pop(1)]))
            moved = gdn.state_compact([cache, conv], live).tolist()
            place = {i: moved[s] for i, s in place.items()}
            assert sorted(place.values()) == [0, 1, 2] and live.tolist() == [1, 1, 1, 0, 0, 0, 0, 0]
        ids = sorted(place)
        tok = torch.tensor([c.cu[rows_of[i]] + lens[rows_of[i]] + t for i in ids], device="cuda")
        o = gdn.linear_decode_step(q[tok], k[tok], v[tok], g.view(1, -1), cache.view(8, Hv, D, D), len(ids), 1,
                                   slot=dev_i32([place[i] for i in ids]), scale=c.scale)
        tk = tok.cpu().numpy()
        close(o, want[tk], f32_tol(140) * 8 * m[tk] + 1e-30, "decoded o")
        close(whole[tok], want[tk], (B16 + f32_tol(140)) * m[tk], "prefilled o")


def test_front_end_prefill_and_norm_together():
    """The layer as it is used: convolution front end, linear attention, gated output norm, and back."""
    import torch
    import gated_deltanet_recurrence_prefill_b200 as gdn
    import synth
    fe = synth.make_frontend([100, 37], seed=7, init_state=True, Hqk=2, Hv=6)
    cu = dev_i32(fe.cu_seqlens)
    q, k, v = gdn.conv1d_silu(dev_bf16(fe.qkv), dev_f32(fe.conv_w), 2, 6, cu_seqlens=cu)
    T = q.shape[0]
    g = -torch.rand(T, 6, device="cuda")
    o, _ = gdn.linear_prefill(q, k, v, g, cu_seqlens=cu, o_dtype=torch.float32)
    z = torch.randn(T, 6, D, device="cuda").bfloat16()
    y = gdn.gated_norm(o, z, torch.ones(D, device="cuda"))
    want, _, _ = ref.prefill(host(q), host(k), host(v), host(g), fe.cu_seqlens, D ** -0.5)
    m, _ = ref.sizes(host(q), host(k), host(v), host(g), fe.cu_seqlens, D ** -0.5)
    close(o, want, (B16 + f32_tol(100)) * m, "o")
    assert torch.isfinite(y.float()).all()
    nb = gdn.gated_norm_backward(o, z, torch.ones(D, device="cuda"), torch.randn(T, 6, D, device="cuda"))
    r = gdn.linear_prefill_backward(q, k, v, g, nb["d_o"].bfloat16(), cu_seqlens=cu, grad_dtype=torch.float32)
    fb = gdn.conv1d_silu_backward(dev_bf16(fe.qkv), dev_f32(fe.conv_w), r["dq"], r["dk"], r["dv"], 2, 6, cu_seqlens=cu)
    assert all(torch.isfinite(fb[n]).all() for n in ("d_qkv", "d_conv_w"))
    grads = ref.prefill_backward(host(q), host(k), host(v), host(g), fe.cu_seqlens, D ** -0.5, host(nb["d_o"].bfloat16()))
    mv, _ = ref.sizes(host(k), host(q), host(nb["d_o"].bfloat16()), host(g), fe.cu_seqlens, D ** -0.5, True)
    close(r["dv"], grads["dv"], (B16 + f32_tol(100)) * mv + 1e-30, "dv")


# ---- streams, captures, repeats -----------------------------------------------------------------

def test_same_result_every_time_on_another_stream_and_replayed():
    import torch
    import gated_deltanet_recurrence_prefill_b200 as gdn
    c = Case(31, [500, 77], 2, 6)
    q, k, v, g = c.dev(True)
    cu, s0, dfin, d_o = dev_i32(c.cu), dev_f32(c.s0), dev_f32(c.dfin), dev_bf16(c.dob)

    def both(stream=None):
        o, fin = gdn.linear_prefill(q, k, v, g, cu_seqlens=cu, scale=c.scale, initial_state=s0, stream=stream)
        r = gdn.linear_prefill_backward(q, k, v, g, d_o, d_final_state=dfin, cu_seqlens=cu, scale=c.scale,
                                        initial_state=s0, stream=stream)
        return [o, fin] + [r[n] for n in ("dq", "dk", "dv", "dg", "d_initial_state")]
    first = both()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, both()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = both(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for x in held:
        x.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, held))


def test_two_calls_at_once():
    """Two streams at a time, each with its own workspace."""
    import torch
    import gated_deltanet_recurrence_prefill_b200 as gdn
    cases = [Case(41, [900, 33], 2, 4), Case(42, [64, 1200], 2, 4)]
    dev = [(c.dev(), dev_i32(c.cu), dev_f32(c.s0)) for c in cases]
    run = lambda d, s: gdn.linear_prefill(*d[0], cu_seqlens=d[1], initial_state=d[2], stream=s)  # noqa: E731
    alone = [run(d, None) for d in dev]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in dev]
    for _ in range(20):
        both = [run(d, s) for d, s in zip(dev, streams)]
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_decode_captured_and_replayed():
    import torch
    import gated_deltanet_recurrence_prefill_b200 as gdn
    gen = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q, k, v, g, S = r(6, 2, D).bfloat16(), r(6, 2, D).bfloat16(), r(6, 4, D).bfloat16(), -r(6, 4).abs(), r(8, 4, D, D)
    slot, start = dev_i32([3, -1, 0]), S.clone()
    o = gdn.linear_decode_step(q, k, v, g, S, 3, 2, slot=slot)
    want = S.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = gdn.linear_decode_step(q, k, v, g, S, 3, 2, slot=slot)
    S.copy_(start)
    held.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(S, want) and torch.equal(held, o) and not o[2:4].any()


def test_workspace_reports_no_timeout():
    import torch
    import gated_deltanet_recurrence_prefill_b200 as gdn
    c = Case(32, [300], 1, 1)
    q, k, v, g = c.dev()
    ws = torch.full((gdn.linear_prefill_workspace_size(1, 300, 1, 1),), 255, dtype=torch.uint8, device="cuda")
    gdn.linear_prefill(q, k, v, g, workspace=ws)
    assert gdn.prefill_status(ws) == 0


def test_scores_of_short_sequences():
    """Without a state in front only the scores matter: two bf16 parts keep 2^-16 of each (m); the 128 products of a
    score are added in float32, at most 128 x 2^-23 = 2^-16 of their magnitudes (m_abs), the decay, the sum over at most
    64 tokens and the scale less than as much again.  Scores rounded once to bf16 are off by up to 2^-9 of m."""
    import torch
    import gated_deltanet_recurrence_prefill_b200 as gdn
    c = Case(51, [1, 3, 17, 0, 64, 2], 2, 4, init=False)
    q, k, v, g = c.dev()
    o, _ = gdn.linear_prefill(q, k, v, g, cu_seqlens=dev_i32(c.cu), scale=c.scale, o_dtype=torch.float32)
    want = ref.prefill(c.q, c.k, c.v, c.gr, c.cu, c.scale)[0]
    m, _ = ref.sizes(c.q, c.k, c.v, c.gr, c.cu, c.scale)
    m_abs, _ = ref.sizes(*(np.abs(x) for x in (c.q, c.k, c.v)), c.gr, c.cu, c.scale)
    close(o, want, 2.0 ** -16 * m + 2.0 ** -15 * m_abs + 1e-30, "o")


def test_rows_but_no_tokens():
    """Sequences that are all empty, with rows behind them."""
    import torch
    import gated_deltanet_recurrence_prefill_b200 as gdn
    c = Case(52, [0, 0, 0], 1, 2, per_head=True, tail=150)
    q, k, v, g = c.dev()
    cu, s0, dfin = dev_i32(c.cu), dev_f32(c.s0), dev_f32(c.dfin)
    o = torch.full((150, 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    _, fin = gdn.linear_prefill(q, k, v, g, cu_seqlens=cu, initial_state=s0, o=o)
    assert torch.equal(fin, s0) and (o == 7.0).all()
    out = {n: torch.full((150, h, D), 7.0, device="cuda") for n, h in (("dq", 1), ("dk", 1), ("dv", 2))}
    r = gdn.linear_prefill_backward(q, k, v, g, dev_bf16(c.dob), d_final_state=dfin, cu_seqlens=cu, initial_state=s0,
                                    out=out)
    assert torch.equal(r["d_initial_state"], dfin) and not r["dg"].any()
    assert all((r[n] == 7.0).all() for n in ("dq", "dk", "dv"))


@pytest.mark.parametrize("lengths,Hqk,Hv", [([90], 2, 4), ([70, 0, 131, 64, 1], 16, 32)], ids=["together", "in turn"])
@pytest.mark.parametrize("g16", [True, False])
def test_backward_passes_together_and_in_turn(lengths, Hqk, Hv, g16):
    import torch
    import gated_deltanet_recurrence_prefill_b200 as gdn
    c = Case(53, lengths, Hqk, Hv)
    q, k, v, g = c.dev(True)
    r = gdn.linear_prefill_backward(q, k, v, g, dev_bf16(c.dob), d_final_state=dev_f32(c.dfin), cu_seqlens=dev_i32(c.cu),
                                    scale=c.scale, initial_state=dev_f32(c.s0),
                                    grad_dtype=torch.bfloat16 if g16 else torch.float32)
    check_backward(c, r, g16)


@pytest.mark.parametrize("lengths", [[300], [6000], [170] * 39 + [3000]], ids=["whole", "in parts", "listed"])
def test_one_workspace_for_call_after_call(lengths):
    """Calls that follow one another on a stream share a workspace, whatever it held; its error word ends clear."""
    import torch
    import gated_deltanet_recurrence_prefill_b200 as gdn
    cases = [Case(60 + i, lengths, 1, 2) for i in range(2)]
    size = max(gdn.linear_prefill_workspace_size(len(lengths), sum(lengths), 1, 2),
               gdn.lib().gdn_linear_prefill_backward_workspace_size(len(lengths), sum(lengths), 1, 2, D))
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    dev = [(c.dev(), dev_bf16(c.dob), dev_i32(c.cu), dev_f32(c.s0), dev_f32(c.dfin)) for c in cases]

    def run(d, workspace):
        o, fin = gdn.linear_prefill(*d[0], cu_seqlens=d[2], initial_state=d[3], workspace=workspace)
        r = gdn.linear_prefill_backward(*d[0], d[1], cu_seqlens=d[2], initial_state=d[3], d_final_state=d[4],
                                        workspace=workspace)
        return [o, fin] + [r[n] for n in ("dq", "dk", "dv", "dg", "d_initial_state")]
    alone = []
    for d in dev:
        alone.append(run(d, None))
        torch.cuda.synchronize()
    for _ in range(3):
        for got, want in zip([run(d, ws) for d in dev], alone):
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert gdn.prefill_status(ws) == 0
