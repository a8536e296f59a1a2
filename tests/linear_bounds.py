"""Bounds in norm for linear attention with a decay per head, and an emulation of its chunked passes to try them on.

Elementwise bounds by sums of magnitudes are many times larger than the errors are, since roundings are independent of
one another.  In the norm over a whole tensor they add as squares, and a part that is rounded once too often shows.

* steps(C) 2^-23 is what float32 leaves of a pass over C chunks: 2^-23 of a partial sum (the tensor cores may cut) for
  each addition that follows another: 8 for a score's 128 products, 12 for the products with it in three parts, 24 for
  those with the state, 3 each for a decay (exponent, exponential, product), one each for the scale, the sum of both
  and a value head; per chunk 12 + 3 + 3 + 2 for the state.  With up to 12 value heads: 8 + 12 + 24 + 3 + 3 + 2 + 12 = 64
  and 20 C.
* A rounding to bf16 is off by at most 2^-8 of the binade's foot, uniformly: in the mean 2^-8 / sqrt(3) of it, and of
  the values themselves, spread evenly over the binade's logarithm, sqrt(3 / (8 ln 2)) of that, 1.66e-3.  ROUNDED
  takes a tenth more.
"""
import numpy as np

from oracle import linear as ref

D = 128
ROUNDED = 1.1 * 2.0 ** -8 / np.sqrt(3.0) * np.sqrt(3.0 / (8.0 * np.log(2.0)))


def steps(cu):
    return (64 + 20 * -(-int(max(np.diff(cu))) // 64)) * 2.0 ** -23


def norm(x):
    return float(np.sqrt((np.asarray(x, np.float64) ** 2).sum()))


def bf16(x):
    """Rounded to bf16, to nearest and even, as float32."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return (((b + 0x7fff + ((b >> 16) & 1)) >> 16) << 16).astype(np.uint32).view(np.float32)


def walk(x, y, z, g, cu, scale, backward=False, init=None, round_state=None, round_scores=None, dtype=np.float64):
    """A pass in chunks of 64 (out_t = a_t A x_t + sum Gamma_ts (x_t . y_s) z_s) in `dtype`, with the state's copy and
    the scores rounded on the way if asked for: (out, the part of it that comes from the state, the last state)."""
    g = np.asarray(g, np.float64)
    x, y, z = (ref._spread(i, g.shape[-1]).astype(dtype) for i in (x, y, z))
    T, Hv = x.shape[:2]
    g = np.broadcast_to(g, (T, Hv))
    out, inter = np.zeros((T, Hv, D), dtype), np.zeros((T, Hv, D), dtype)
    last = np.zeros((len(cu) - 1, Hv, D, D), dtype)
    id_ = lambda a: a  # noqa: E731
    rs, rp = round_state or id_, round_scores or id_
    for n in range(len(cu) - 1):
        A = last[n] if init is None else np.asarray(init[n], dtype).copy()
        edges = [(s, min(s + 64, cu[n + 1])) for s in range(cu[n], cu[n + 1], 64)]
        for s, e in edges[::-1] if backward else edges:
            G = np.cumsum(g[s:e], 0)
            a, w = np.exp(G), np.exp(G[-1] - G)
            gam = np.exp(np.where(np.tri(e - s)[:, :, None] > 0, G[:, None] - G[None, :], -np.inf))
            if backward:
                a, w, gam = w * scale, a * scale, gam.transpose(1, 0, 2)
                inter[s:e] = (a / scale).astype(dtype)[..., None] * np.einsum("hij,thj->thi", rs(A), x[s:e])
            else:
                inter[s:e] = (a * scale).astype(dtype)[..., None] * np.einsum("hij,thj->thi", rs(A), x[s:e])
            p = rp(np.einsum("thd,shd->tsh", x[s:e], y[s:e]) * gam.astype(dtype))
            out[s:e] = inter[s:e] + dtype(scale) * np.einsum("tsh,shd->thd", p, z[s:e])
            A = np.exp(G[-1]).astype(dtype)[:, None, None] * A + np.einsum("sh,shi,shj->hij", w.astype(dtype), z[s:e], y[s:e])
        last[n] = A
    return out, inter, last


def transposed(s):
    return None if s is None else s.transpose(0, 1, 3, 2)


def gradients(c, **how):
    """dq and dk for each value head and dg (per token) by the passes behind them, as the kernels take them: dg as a
    running sum from the last token, tied down at the first."""
    dq, _, fin = walk(c.do, c.v, c.k, c.gr, c.cu, c.scale, init=transposed(c.s0), **how)
    dk, _, first = walk(c.v, c.do, c.q, c.gr, c.cu, c.scale, backward=True, init=transposed(c.dfin), **how)
    wide = lambda x: ref._spread(x, c.Hv)  # noqa: E731
    diff = (wide(c.q) * dq).sum(-1, dtype=np.float64) - (wide(c.k) * dk).sum(-1, dtype=np.float64)
    dg = np.zeros((c.T, c.Hv))
    decays = np.broadcast_to(c.gr, (c.T, c.Hv))
    for n in range(c.N):
        s, e = c.cu[n], c.cu[n + 1]
        if s == e:
            continue
        prod = lambda a, b: 0.0 if a is None or b is None else (np.float64(a[n]) * b[n]).sum((1, 2))  # noqa: B023, E731
        front = prod(transposed(c.s0), first)
        total = prod(fin, transposed(c.dfin)) + np.cumsum(diff[s:e][::-1], 0)[::-1]
        left = np.arange(e - s, 0, -1)[:, None]
        dg[s:e] = total - (total[0] - front) / (e - s) * left
    return dq, dk, np.where(decays <= -104.0, 0.0, dg)


class Exact:
    """What a Case's outputs are in 64 bits, and what their bounds are made of."""

    def __init__(self, c):
        self.c = c
        self.o, self.o_state, _ = walk(c.q, c.k, c.v, c.gr, c.cu, c.scale, init=c.s0)
        self.dq, self.dk, self.dg = gradients(c)
        self.dv, self.dv_state, _ = walk(c.k, c.q, c.do, c.gr, c.cu, c.scale, backward=True, init=c.dfin)

    def fold(self, x):
        return x.reshape(self.c.T, self.c.Hqk, -1, D).sum(2)

    def check_exact_passes(self, r):
        """dq, dk (float32) and dg: nothing is rounded to fewer than 32 bits on their way.  An error of dq_t is as likely
        in any direction: of q_t . dq_t it is sqrt(1 / 128) of |q_t| times its norm, four times that allowed; dg sums those
        behind a token, and <S, dS> behind them, 1 / 128 of the norms likewise."""
        c, eps = self.c, steps(self.c.cu)
        for name, want in (("dq", self.fold(self.dq)), ("dk", self.fold(self.dk))):
            off = norm(np.asarray(r[name], np.float64)[:c.T] - want)
            assert off <= eps * norm(want), f"{name}: off by {off / norm(want)} of its norm, allowed {eps}"
        if c.gr.ndim == 1:
            return
        each = lambda x: np.sqrt((ref._spread(x, c.Hv) ** 2).sum(-1))  # noqa: E731
        rho = (each(c.q) * each(self.dq)) ** 2 + (each(c.k) * each(self.dk)) ** 2
        total = 0.0
        for n in range(c.N):
            s, e = c.cu[n], c.cu[n + 1]
            total += (np.arange(1, e - s + 1)[:, None] * rho[s:e]).sum() * 16 / D
            if c.dfin is not None and e > s:
                fin = walk(c.q[s:e], c.k[s:e], c.v[s:e], c.gr[s:e], [0, e - s], c.scale, init=None if c.s0 is None else c.s0[n:n + 1])[2]
                total += (e - s) * ((fin[0] ** 2).sum((1, 2)) * (np.float64(c.dfin[n]) ** 2).sum((1, 2))).sum() * 16 / D ** 2
        allowed = eps * (np.sqrt(total) + norm(self.dg))
        off = norm(np.asarray(r["dg"], np.float64)[:c.T] - self.dg)
        assert off <= allowed, f"dg: off by {off}, allowed {allowed}, norm {norm(self.dg)}"

    def check_output_pass(self, got, name, stored16):
        """o or dv: the state's copy is rounded to bf16, the scores are kept to 2^-16, the result is stored."""
        want, state = (self.o, self.o_state) if name == "o" else (self.dv, self.dv_state)
        allowed = np.hypot(ROUNDED * norm(state), ROUNDED * norm(want) if stored16 else 0.0) + \
            (steps(self.c.cu) + 2.0 ** -16) * norm(want)
        off = norm(np.asarray(got, np.float64)[:self.c.T] - want)
        assert off <= allowed, f"{name}: off by {off / norm(want)} of its norm, allowed {allowed / norm(want)}"
