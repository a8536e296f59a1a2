"""fp64 reference of linear attention with a decay per head and of the state cache's page operations.

The recurrence is taken token by token from its definition,

    S_t = e^{g_t} S_{t-1} + v_t k_t^T,      o_t = scale * S_t q_t,

and its gradients from reverse-mode differentiation of those two lines, with none of the chunked algebra of the
kernels.  All arrays are numpy; q and k are [T, Hqk, d], v and o [T, Hv, d], g [T, Hv], states [N, Hv, d_v, d_k].
"""
import numpy as np


def _spread(x, Hv):
    return np.repeat(np.asarray(x, np.float64), Hv // x.shape[1], axis=1)


def _gates(g, T):
    g = np.asarray(g, np.float64)
    return np.broadcast_to(g, (T, g.shape[-1]))


def prefill(q, k, v, g, cu_seqlens, scale, initial_state=None):
    """(o, final_state, states): states[t] is S_t, for the gradients."""
    v = np.asarray(v, np.float64)
    T, Hv, d = v.shape
    q, k, g = _spread(q, Hv), _spread(k, Hv), _gates(g, T)
    N = len(cu_seqlens) - 1
    fin = np.zeros((N, Hv, d, d))
    o = np.zeros((T, Hv, d))
    states = np.zeros((T, Hv, d, d))
    for n in range(N):
        S = fin[n] if initial_state is None else np.asarray(initial_state[n], np.float64).copy()
        for t in range(cu_seqlens[n], cu_seqlens[n + 1]):
            S = np.exp(g[t])[:, None, None] * S + v[t][:, :, None] * k[t][:, None, :]
            o[t] = scale * np.einsum("hij,hj->hi", S, q[t])
            states[t] = S
        fin[n] = S
    return o, fin, states


def prefill_backward(q, k, v, g, cu_seqlens, scale, d_o, initial_state=None, d_final_state=None):
    """Gradients of sum(o * d_o) + sum(final_state * d_final_state)."""
    Hqk = q.shape[1]
    v = np.asarray(v, np.float64)
    T, Hv, d = v.shape
    _, _, states = prefill(q, k, v, g, cu_seqlens, scale, initial_state)
    qs, ks, gs = _spread(q, Hv), _spread(k, Hv), _gates(g, T)
    d_o = np.asarray(d_o, np.float64)
    N = len(cu_seqlens) - 1
    dq, dk, dv, dg = np.zeros((T, Hv, d)), np.zeros((T, Hv, d)), np.zeros((T, Hv, d)), np.zeros((T, Hv))
    first = np.zeros((N, Hv, d, d))
    for n in range(N):
        R = first[n] if d_final_state is None else np.asarray(d_final_state[n], np.float64).copy()
        for t in range(cu_seqlens[n + 1] - 1, cu_seqlens[n] - 1, -1):
            before = (states[t - 1] if t > cu_seqlens[n] else
                      np.zeros((Hv, d, d)) if initial_state is None else np.asarray(initial_state[n], np.float64))
            R = R + scale * d_o[t][:, :, None] * qs[t][:, None, :]
            dq[t] = scale * np.einsum("hij,hi->hj", states[t], d_o[t])
            dk[t] = np.einsum("hij,hi->hj", R, v[t])
            dv[t] = np.einsum("hij,hj->hi", R, ks[t])
            decay = np.exp(gs[t])[:, None, None]
            dg[t] = (decay * R * before).sum((1, 2))
            R = decay * R
        first[n] = R
    fold = lambda x: x.reshape(T, Hqk, Hv // Hqk, d).sum(2)  # noqa: E731
    return dict(dq=fold(dq), dk=fold(dk), dv=dv, dg=dg.sum(0) if np.ndim(g) == 1 else dg, d_initial_state=first)


def sizes(x, y, z, g, cu_seqlens, scale, backward=False, initial_state=None, chunk=64):
    """The sums of magnitudes that bound the rounding of a chunked pass.

    A pass computes out_t = a_t A x_t + sum_s Gamma_ts (x_t . y_s) z_s over the tokens s of t's chunk, A being the
    state at the chunk's edge.  Returns (m, fin): m[t] = the same sum with |A|, |x_t|, |x_t . y_s| and |z_s|, the
    magnitude that a relative error of A or of the scores acts on; fin = the state with |z| |y|^T in place of z y^T.
    backward: the pass that runs from the last token to the first (gradients of k and v)."""
    x, y, z = (np.asarray(i, np.float64) for i in (x, y, z))
    T, Hv, d = x.shape[0], np.shape(g)[-1], x.shape[2]
    x, y, z, g = _spread(x, Hv), _spread(y, Hv), _spread(z, Hv), _gates(g, T)
    N = len(cu_seqlens) - 1
    m, fin = np.zeros((T, Hv, d)), np.zeros((N, Hv, d, d))
    for n in range(N):
        A = fin[n] if initial_state is None else np.asarray(initial_state[n], np.float64).copy()
        size = np.abs(A)
        t0, t1 = cu_seqlens[n], cu_seqlens[n + 1]
        edges = [(s, min(s + chunk, t1)) for s in range(t0, t1, chunk)]
        for s, e in edges[::-1] if backward else edges:
            G = np.cumsum(g[s:e], 0)
            a, w = np.exp(G), np.exp(G[-1] - G)
            diff = G[:, None] - G[None, :]
            keep = np.tri(e - s)[:, :, None] > 0
            gam = np.exp(np.where(keep, diff, -np.inf))                    # [t, s, h]
            if backward:
                a, w, gam = w, a, gam.transpose(1, 0, 2)
            p = np.einsum("thd,shd->tsh", x[s:e], y[s:e]) * gam
            m[s:e] = np.einsum("tsh,shd->thd", np.abs(p), np.abs(z[s:e])) * abs(scale)
            m[s:e] += (1.0 if backward else abs(scale)) * a[..., None] * np.einsum("hij,thj->thi", np.abs(A), np.abs(x[s:e]))
            ws = w * (scale if backward else 1.0)
            total = np.exp(G[-1])[:, None, None]
            A = total * A + np.einsum("sh,shi,shj->hij", ws, z[s:e], y[s:e])
            size = total * size + np.einsum("sh,shi,shj->hij", np.abs(ws), np.abs(z[s:e]), np.abs(y[s:e]))
        fin[n] = size
    return m, fin


def decode(q, k, v, g, state, slot, n_seq, layers, scale):
    """One token: (o, state after); a slot outside the cache gives a zero row."""
    v = np.asarray(v, np.float64)
    Hv, d = v.shape[1:]
    q, k = _spread(q, Hv), _spread(k, Hv)
    S = np.array(state, np.float64).reshape(-1, layers, Hv, d, d)
    o = np.zeros((n_seq, layers, Hv, d))
    for n in range(n_seq):
        s = n if slot is None else int(slot[n])
        if not 0 <= s < S.shape[0]:
            continue
        for l in range(layers):
            u = n * layers + l
            decay = np.exp(np.asarray(g[u if len(g) == n_seq * layers else l], np.float64))
            S[s, l] = decay[:, None, None] * S[s, l] + v[u][:, :, None] * k[u][:, None, :]
            o[n, l] = scale * np.einsum("hij,hj->hi", S[s, l], q[u])
    return o.reshape(-1, Hv, d), S.reshape(np.shape(state))
