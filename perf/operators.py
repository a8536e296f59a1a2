"""Operators for serving and training recurrent layers, as cases that can be timed and compared.

Six kinds of case, each one pass through what a user calls:

  prefill   linear attention with a decay per head over packed prompts (chunked form)
  step      its recurrent form, one token for every running sequence, state updated in place
  backward  the gradients of the prefill
  copy      pages of a state cache copied at once (reordering of beams, among others)
  fork      new pages for new sequences, copied from a running one or zero, and given back
  turnover  finished sequences freed, the cache compacted, new sequences started

The recurrence, per value head with log decay g (one per head, or one per token and head):

    S_t = e^{g_t} S_{t-1} + v_t k_t^T,      o_t = scale * S_t q_t.

With `own` false, run() computes in plain torch operations; with `own` true it calls the package.
"""
import math

import torch

own = False

D = 128          # head width
CHUNK = 64       # tokens of a chunk in the plain form


# ---- cases ------------------------------------------------------------------------------------

def listed():
    return [
        # a handful of short prompts admitted together: one-token, odd and empty ones among them
        dict(name="prefill_ragged", kind="prefill", lengths="1,63,64,0,65,130", Hqk=16, Hv=48, gate="token",
             init=True, packed=False, scale=0.0),
        # one long document, fixed decays per head, q, k and v being views of one projection
        dict(name="prefill_long", kind="prefill", lengths="65536", Hqk=16, Hv=48, gate="head", init=False,
             packed=True, scale=0.0),
        # a small training batch of uneven documents, carried state and its gradient included
        dict(name="backward_ragged", kind="backward", lengths="130,1,64,77,0,300", Hqk=4, Hv=12, gate="head",
             init=True, packed=False, scale=0.0),
        # a training sequence at the layer's full width, decays from the token
        dict(name="backward_8k", kind="backward", lengths="8192", Hqk=16, Hv=48, gate="token", init=False,
             packed=True, scale=0.0),
        # one user's next token in a small model: latency
        dict(name="step_single", kind="step", n_seq=1, layers=4, Hqk=4, Hv=12, n_slots=2, state="float32",
             gate="token", scale=0.0),
        # a full decode batch, a few rows of it padding, states in bf16 at scattered slots
        dict(name="step_batch", kind="step", n_seq=64, layers=48, Hqk=16, Hv=48, n_slots=70, state="bfloat16",
             gate="head", scale=0.0),
        # four beams of a small model reordered
        dict(name="copy_beams_small", kind="copy", n=4, n_slots=6, layers=2, Hqk=4, Hv=12, state="bfloat16"),
        # the beams of a batch reordered in place: most pages are read and overwritten
        dict(name="copy_beams_batch", kind="copy", n=57, n_slots=64, layers=24, Hqk=16, Hv=48, state="float32"),
        # two samples continued from one prompt, and a third one from nothing
        dict(name="fork_few", kind="fork", n=3, n_slots=9, running=5, layers=2, Hqk=4, Hv=12, state="float32"),
        # a prompt's state handed to 32 samples
        dict(name="fork_samples", kind="fork", n=32, n_slots=48, running=13, layers=48, Hqk=16, Hv=48,
             state="bfloat16"),
        # one of a few sequences ends and another one begins
        dict(name="turnover_few", kind="turnover", n=2, n_slots=9, running=7, layers=2, Hqk=4, Hv=12,
             state="bfloat16"),
        # a quarter of a decode batch ends at once
        dict(name="turnover_batch", kind="turnover", n=21, n_slots=96, running=83, layers=24, Hqk=16, Hv=48,
             state="float32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lengths(rng, total, most):
    n = rng.randint(1, min(most, total))
    cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [total]))


def draw(rng):
    kind = rng.choice(["prefill", "step", "backward", "copy", "fork", "turnover"])
    Hqk, Hv = rng.choice([(1, 1), (2, 4), (4, 12), (8, 8), (8, 32), (16, 16), (16, 48)])
    state = rng.choice(["float32", "bfloat16"])
    scale = rng.choice([0.0, round(rng.uniform(0.02, 1.0), 3)])
    if kind in ("prefill", "backward"):
        total = _log_int(rng, 1, 60000 if kind == "prefill" else 7500)
        return dict(kind=kind, lengths=_lengths(rng, total, 9), Hqk=Hqk, Hv=Hv, gate=rng.choice(["token", "head"]),
                    init=rng.random() < 0.5, packed=rng.random() < 0.5, scale=scale)
    if kind == "step":
        n_seq, layers = _log_int(rng, 1, 64 if state == "bfloat16" else 32), _log_int(rng, 1, 48)
        return dict(kind=kind, n_seq=n_seq, layers=layers, Hqk=Hqk, Hv=Hv, n_slots=n_seq + rng.randint(0, 5),
                    state=state, gate=rng.choice(["token", "head"]), scale=scale)
    layers = _log_int(rng, 1, 24)
    if kind == "copy":
        n_slots = _log_int(rng, 2, 64)
        return dict(kind=kind, n=rng.randint(1, n_slots), n_slots=n_slots, layers=layers, Hqk=Hqk, Hv=Hv, state=state)
    running = _log_int(rng, 2, 70)
    if kind == "fork":
        n = rng.randint(1, min(20, running))
        return dict(kind=kind, n=n, n_slots=running + n + rng.randint(0, 2), running=running, layers=layers, Hqk=Hqk,
                    Hv=Hv, state=state)
    return dict(kind=kind, n=rng.randint(1, max(1, min(running // 2, 20))), n_slots=running + rng.randint(0, 13),
                running=running, layers=layers, Hqk=Hqk, Hv=Hv, state=state)


def _lens(case):
    return [int(x) for x in case["lengths"].split(",")]


def _scale(case):
    return case["scale"] if case["scale"] else D ** -0.5


def work(case):
    kind, Hqk, Hv = case["kind"], case["Hqk"], case["Hv"]
    if kind in ("prefill", "backward"):
        lens = _lens(case)
        T, n = sum(lens), len(lens)
        # pairs of a query and a key of the same chunk, and tokens that meet a carried state
        pairs = sum((x // CHUNK) * (CHUNK * (CHUNK + 1) // 2) + (x % CHUNK) * (x % CHUNK + 1) // 2 for x in lens)
        gate = 4 * Hv * (T if case["gate"] == "token" else 1)
        states = n * Hv * D * D * 4 * (2 if case["init"] else 1)
        if kind == "prefill":
            return {"bytes": 2 * T * D * (2 * Hqk + 2 * Hv) + gate + states + 4 * (n + 1),
                    "flops": Hv * (4 * D * pairs + 4 * D * D * T)}
        # S0 read and its gradient written, the final state's gradient read
        more = n * Hv * D * D * 4 * 3 if case["init"] else 0
        return {"bytes": 2 * T * D * (4 * Hqk + 3 * Hv) + 2 * gate + more + 4 * (n + 1),
                "flops": Hv * (10 * D * pairs + 10 * D * D * T)}
    el = 4 if case["state"] == "float32" else 2
    page = case["layers"] * Hv * D * D * el
    if kind == "step":
        live = sum(1 for s in _step_slots(case) if s >= 0)
        U = case["n_seq"] * case["layers"]
        return {"bytes": 2 * live * page + U * D * (2 * Hqk * 2 + Hv * 2 + Hv * 4)
                + 4 * Hv * (U if case["gate"] == "token" else case["layers"]) + 4 * case["n_seq"],
                "flops": 5 * D * D * Hv * live * case["layers"]}
    page += case["layers"] * (2 * Hqk + Hv) * D * 3 * 4            # the convolution's history
    if kind == "copy":
        src, dst = _copy_lists(case)
        moved = [(a, b) for a, b in zip(src, dst) if a != b]
        return {"bytes": page * (len(set(a for a, _ in moved)) + len(moved)) + 8 * case["n"], "flops": 0}
    _, src, done = _pool_lists(case)
    made = page * (len(src) + len(set(a for a in src if a >= 0)))
    if kind == "fork":
        return {"bytes": made + 8 * len(src), "flops": 0}
    left = case["running"] - case["n"]
    gaps = sum(1 for s in done if s < left)
    return {"bytes": made + 2 * gaps * page + 4 * case["n_slots"], "flops": 0}


# ---- inputs -----------------------------------------------------------------------------------

def _mix(*values):
    x = 1234567
    for v in values:
        x = (x * 1103515245 + int(v) * 40503 + 12345) % (1 << 31)
    return x


def _shuffled(n, key):
    order, x = list(range(n)), key
    for i in range(n - 1, 0, -1):
        x = _mix(x, i)
        j = x % (i + 1)
        order[i], order[j] = order[j], order[i]
    return order


def _step_slots(case):
    """The slot of each row of the batch; one row in sixteen is padding (-1)."""
    slots = _shuffled(case["n_slots"], 77 + case["n_seq"])[: case["n_seq"]]
    return [-1 if i % 16 == 15 else s for i, s in enumerate(slots)]


def _copy_lists(case):
    """Beams i <- parent(i): parents repeat, most pages are both read and overwritten."""
    slots = _shuffled(case["n_slots"], 5 + case["n"])[: case["n"]]
    src = [slots[_mix(i, case["n"]) % case["n"]] for i in range(case["n"])]
    return src, slots


def _pool_lists(case):
    """(the running slots, what each new page starts from (-1: zero), the slots that finish)."""
    running, n = case["running"], case["n"]
    if case["kind"] == "fork":
        live = sorted(_shuffled(case["n_slots"], 3)[:running])
        src = [-1 if i % 8 == 7 or (n <= 3 and i == n - 1) else live[_mix(i, n) % max(1, running // 4)] for i in range(n)]
        return live, src, []
    done = sorted(_shuffled(running, 9)[:n])
    src = [-1 if i % 4 else 0 for i in range(n)]
    return list(range(running)), src, done


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    Hqk, Hv, kind = case["Hqk"], case["Hv"], case["kind"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def gates(*shape):
        # log decays as layers have them: memories of two to a few thousand tokens, some tokens that reset
        x = -torch.exp(torch.rand(*shape, generator=gen, device=dev) * 7.5 - 7.8)
        if len(shape) > 1:
            x = torch.where(torch.rand(*shape, generator=gen, device=dev) < 0.002, torch.full_like(x, -30.0), x)
        return x

    def unit(x):
        return x / x.square().sum(-1, keepdim=True).sqrt().clamp_min(1e-6)

    if kind in ("prefill", "backward"):
        lens = _lens(case)
        T, n = sum(lens), len(lens)
        q, k = unit(normal(T, Hqk, D)).bfloat16(), unit(normal(T, Hqk, D)).bfloat16()
        v = (normal(T, Hv, D)).bfloat16()
        if case["packed"]:
            row = torch.cat([x.reshape(T, -1) for x in (q, k, v)], 1)
            q, k, v = (x.unflatten(1, (-1, D)) for x in row.split([Hqk * D, Hqk * D, Hv * D], 1))
        ends = [0]
        for x in lens:
            ends.append(ends[-1] + x)
        st = dict(kind=kind, q=q, k=k, v=v, g=gates(T, Hv) if case["gate"] == "token" else gates(Hv),
                  cu=torch.tensor(ends, dtype=torch.int32, device=dev), scale=_scale(case),
                  s0=0.5 * normal(n, Hv, D, D) if case["init"] else None)
        # where each token stands among whole chunks, for the plain form
        place, seq = [], []
        for i, x in enumerate(lens):
            nc = -(-x // CHUNK)
            place.append(len(seq) * CHUNK + torch.arange(x))
            seq += [i] * nc
        st["place"] = torch.cat(place).to(dev)
        st["seq"] = torch.tensor(seq, device=dev)
        if kind == "backward":
            st["d_o"] = normal(T, Hv, D).bfloat16()
            st["d_final"] = 0.3 * normal(n, Hv, D, D) if case["init"] else None
        return st
    dtype = getattr(torch, case["state"])
    layers, slots = case["layers"], case["n_slots"]
    state = torch.empty(slots, layers, Hv, D, D, dtype=dtype, device=dev)
    for i in range(slots):
        state[i] = 0.5 * normal(layers, Hv, D, D)
    if kind == "step":
        n = case["n_seq"]
        return dict(kind=kind, q=unit(normal(n * layers, Hqk, D)).bfloat16(), k=unit(normal(n * layers, Hqk, D)).bfloat16(),
                    v=normal(n * layers, Hv, D).bfloat16(), g=gates(*((n * layers, Hv) if case["gate"] == "token" else (layers, Hv))),
                    state=state.view(slots * layers, Hv, D, D), n_seq=n, layers=layers, scale=_scale(case),
                    slot=torch.tensor(_step_slots(case), dtype=torch.int32, device=dev))
    conv = normal(slots, layers, (2 * Hqk + Hv) * D, 3)
    st = dict(kind=kind, buffers=[state, conv])
    if kind == "copy":
        src, dst = _copy_lists(case)
        st["src"], st["dst"] = (torch.tensor(x, dtype=torch.int32, device=dev) for x in (src, dst))
        return st
    running, src, done = _pool_lists(case)
    st["live"] = torch.zeros(slots, dtype=torch.int32, device=dev)
    st["live"][torch.tensor(running, device=dev)] = 1
    st["src"] = torch.tensor(src, dtype=torch.int32, device=dev)
    st["done"] = torch.tensor(done, dtype=torch.int32, device=dev)
    return st


# ---- one pass ---------------------------------------------------------------------------------

def run(st):
    return {"prefill": _prefill, "backward": _backward, "step": _step, "copy": _copy, "fork": _fork,
            "turnover": _turnover}[st["kind"]](st)


def _prefill(st):
    if own:
        import gated_deltanet_recurrence_prefill_b200 as gdn
        o, s = gdn.linear_prefill(st["q"], st["k"], st["v"], st["g"], cu_seqlens=st["cu"], scale=st["scale"],
                                  initial_state=st["s0"], o_dtype=torch.bfloat16)
        return {"o": o, "final_state": s}
    c = _Chunks(st)
    start, end = c.states(c.outer(c.w, c.v, c.k), st["s0"])
    p = (c.q @ c.k.transpose(-1, -2)) * c.gamma
    o = st["scale"] * (p @ c.v + c.a[..., None] * (c.q @ start.transpose(-1, -2)))
    return {"o": c.back(o).bfloat16(), "final_state": end}


def _backward(st):
    if own:
        import gated_deltanet_recurrence_prefill_b200 as gdn
        r = gdn.linear_prefill_backward(st["q"], st["k"], st["v"], st["g"], st["d_o"], d_final_state=st["d_final"],
                                        cu_seqlens=st["cu"], scale=st["scale"], initial_state=st["s0"],
                                        want_d_initial=st["s0"] is not None)
        return {n: r[n] for n in ("dq", "dk", "dv", "dg", "d_initial_state")}
    c, scale = _Chunks(st), st["scale"]
    d_o = c.lay(st["d_o"])
    start, final = c.states(c.outer(c.w, c.v, c.k), st["s0"])
    d_end, d_first = c.states_back(scale * c.outer(c.a, d_o, c.q), st["d_final"])
    p = (c.q @ c.k.transpose(-1, -2)) * c.gamma * scale
    dp = (d_o @ c.v.transpose(-1, -2)) * c.gamma * scale
    dq = dp @ c.k + scale * c.a[..., None] * (d_o @ start)
    dk = dp.transpose(-1, -2) @ c.q + c.w[..., None] * (c.v @ d_end)
    dv = p.transpose(-1, -2) @ d_o + c.w[..., None] * (c.k @ d_end.transpose(-1, -2))
    # gradient of the decays: what passes the chunk's end, and what its tokens add, from the last one back
    after = c.after(start, c.outer(c.w, c.v, c.k))
    beyond = (after.double() * d_end.double()).sum((-1, -2))
    own_part = (c.q.double() * dq.double()).sum(-1) - (c.k.double() * dk.double()).sum(-1)
    dg = c.back((beyond[..., None] + own_part.flip(-1).cumsum(-1).flip(-1))[..., None])[..., 0]
    if st["g"].dim() == 1:
        dg = dg.sum(0)
    Hqk = st["q"].shape[1]

    def heads(x):
        x = c.back(x)
        return x.unflatten(1, (Hqk, -1)).sum(2).bfloat16()
    return {"dq": heads(dq), "dk": heads(dk), "dv": c.back(dv).bfloat16(), "dg": dg.float(),
            "d_initial_state": d_first if st["s0"] is not None else None}


class _Chunks:
    """q, k, v and the decays of packed sequences laid out in whole chunks [chunk, head, token, ...],
    products in 32 bits, sums of log decays in 64."""

    def __init__(self, st):
        self.place, self.seq, self.n_seq = st["place"], st["seq"], st["cu"].numel() - 1
        self.Hv = st["v"].shape[1]
        self.nc = self.seq.numel()
        self.q, self.k, self.v = self.lay(st["q"]), self.lay(st["k"]), self.lay(st["v"])
        T = st["q"].shape[0]
        g = st["g"] if st["g"].dim() == 2 else st["g"].expand(T, -1)
        total = self.lay(g[..., None]).double()[..., 0].cumsum(-1)                # within the chunk
        self.a = total.exp().float()
        self.w = (total[..., -1:] - total).exp().float()
        diff = total[..., :, None] - total[..., None, :]
        keep = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=g.device).tril()
        self.gamma = torch.where(keep, diff, -torch.inf).exp().float()
        self.whole = total[..., -1]                                              # [chunk, head]
        upto = self.whole.cumsum(0)
        before = upto - self.whole
        same = self.seq[:, None] == self.seq[None, :]
        earlier = same & torch.ones_like(same).tril(-1)
        # decay from the end of chunk j to the start of chunk c
        d = torch.where(earlier[..., None], before[:, None] - upto[None, :], -torch.inf).exp().float()
        self.between = d.permute(2, 0, 1)
        # decay from the start of its sequence to a chunk's start, and from a chunk's end to the sequence's end
        here = (torch.arange(self.n_seq, device=g.device)[:, None] == self.seq[None, :]).double()
        sums = here @ self.whole                                                 # [sequence, head]
        starts = torch.cat([torch.zeros_like(sums[:1]), sums.cumsum(0)[:-1]])
        self.since = (before - starts[self.seq]).exp().float()
        self.until = (starts[self.seq] + sums[self.seq] - upto).exp().float()
        self.all = sums.exp().float()
        self.here = here

    def lay(self, x):
        """[T, H, ...] -> [chunk, Hv, token, ...] in 32 bits, zeros where a chunk has no token."""
        y = x.new_zeros(self.nc * CHUNK, *x.shape[1:], dtype=torch.float32)
        y[self.place] = x.float()
        y = y.view(self.nc, CHUNK, *x.shape[1:]).transpose(1, 2)
        return y.repeat_interleave(self.Hv // y.shape[1], 1) if y.shape[1] != self.Hv else y

    def back(self, x):
        return x.transpose(1, 2).reshape(self.nc * CHUNK, self.Hv, -1)[self.place]

    @staticmethod
    def outer(w, x, y):
        return (w[..., None] * x).transpose(-1, -2) @ y

    def _mix(self, decay, local):
        y = decay @ local.transpose(0, 1).reshape(self.Hv, self.nc, -1)
        return y.view(self.Hv, self.nc, D, D).transpose(0, 1)

    def _sum(self, decay, local):
        w = self.here.float()[..., None] * decay                                 # [sequence, chunk, head]
        y = w.permute(2, 0, 1) @ local.transpose(0, 1).reshape(self.Hv, self.nc, -1)
        return y.view(self.Hv, self.n_seq, D, D).transpose(0, 1).contiguous()

    def states(self, local, s0):
        """(the state before each chunk, each sequence's last one) from each chunk's own sum."""
        start, end = self._mix(self.between, local), self._sum(self.until, local)
        if s0 is not None:
            start = start + self.since[..., None, None] * s0[self.seq]
            end = end + self.all[..., None, None] * s0
        return start, end

    def states_back(self, local, d_final):
        end, first = self._mix(self.between.transpose(-1, -2), local), self._sum(self.since, local)
        if d_final is not None:
            end = end + self.until[..., None, None] * d_final[self.seq]
            first = first + self.all[..., None, None] * d_final
        return end, first

    def after(self, start, local):
        return self.whole.exp().float()[..., None, None] * start + local


def _step(st):
    if own:
        import gated_deltanet_recurrence_prefill_b200 as gdn
        o = gdn.linear_decode_step(st["q"], st["k"], st["v"], st["g"], st["state"], st["n_seq"], st["layers"],
                                   slot=st["slot"], scale=st["scale"])
        return {"o": o, "state": st["state"]}
    n, layers, Hv = st["n_seq"], st["layers"], st["v"].shape[1]
    rep = Hv // st["q"].shape[1]
    state = st["state"].view(-1, layers, Hv, D, D)
    o = torch.zeros(n, layers, Hv, D, device=state.device)
    q, k = (st[x].view(n, layers, -1, D).repeat_interleave(rep, 2).float() for x in ("q", "k"))
    v = st["v"].view(n, layers, Hv, D).float()
    g = st["g"].view(-1, layers, Hv).expand(n, -1, -1)
    row = (st["slot"] >= 0).nonzero()[:, 0]
    slot = st["slot"][row].long()
    s = state[slot].float()
    s.mul_(g[row].exp()[..., None, None])
    s.addcmul_(v[row][..., None], k[row][..., None, :])
    o[row] = st["scale"] * (s @ q[row][..., None])[..., 0]
    state[slot] = s.to(state.dtype)
    return {"o": o.view(n * layers, Hv, D), "state": st["state"]}


def _copy(st):
    if own:
        import gated_deltanet_recurrence_prefill_b200 as gdn
        gdn.state_copy(st["buffers"], st["src"], st["dst"])
        return {"buffers": st["buffers"]}
    _move(st["buffers"], st["src"].long(), st["dst"].long())
    return {"buffers": st["buffers"]}


def _move(buffers, src, dst):
    for b in buffers:
        b[dst] = b[src]


def _fork(st):
    """New pages for `src`, then given back, as samples that end."""
    if own:
        import gated_deltanet_recurrence_prefill_b200 as gdn
        dst = gdn.state_fork(st["buffers"], st["live"], st["src"])
        gdn.state_free(st["live"], dst)
        return {"dst": dst, "live": st["live"], "buffers": st["buffers"]}
    dst = _begin(st)
    st["live"][dst.long()] = 0
    return {"dst": dst, "live": st["live"], "buffers": st["buffers"]}


def _begin(st):
    live, src = st["live"], st["src"]
    dst = torch.argsort(live, stable=True)[: src.numel()]          # the lowest free slots
    for b in st["buffers"]:
        b[dst] = b[src.clamp_min(0).long()] * (src >= 0).view(-1, *[1] * (b.dim() - 1)).to(b.dtype)
    live[dst] = 1
    return dst.int()


def _turnover(st):
    """Finished sequences freed, the running ones moved to the front, new ones begun behind them."""
    if own:
        import gated_deltanet_recurrence_prefill_b200 as gdn
        gdn.state_free(st["live"], st["done"])
        moved = gdn.state_compact(st["buffers"], st["live"])
        dst = gdn.state_fork(st["buffers"], st["live"], st["src"])
        return {"moved": moved, "dst": dst, "live": st["live"], "buffers": st["buffers"]}
    live = st["live"]
    live[st["done"].long()] = 0
    slots = torch.arange(live.numel(), device=live.device)
    left = live.sum()
    front = slots < left
    gaps = torch.nonzero(front & (live == 0))[:, 0]
    late = torch.nonzero(~front & (live != 0))[:, 0]
    _move(st["buffers"], late, gaps)
    moved = torch.where(live != 0, slots, -1)
    moved[late] = gaps
    live.copy_(front)
    return {"moved": moved.int(), "dst": _begin(st), "live": live, "buffers": st["buffers"]}


# ---- the same in 64 bits, from the definitions ---------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    kind = st["kind"]
    if kind in ("prefill", "backward"):
        if sum(_lens(case)) > 70000:
            return None
        return _exact_tokens(st)
    if kind == "step":
        return _exact_step(st)
    return _exact_pool(st)


def _exact_tokens(st):
    """Token by token, the sequences side by side, one after another of their tokens."""
    cu = st["cu"].tolist()
    n, Hv = len(cu) - 1, st["v"].shape[1]
    dev, scale = st["v"].device, st["scale"]
    rep = Hv // st["q"].shape[1]
    wide = {m: st[m].double().repeat_interleave(rep, 1) for m in ("q", "k")}
    v = st["v"].double()
    T = v.shape[0]
    decay = (st["g"] if st["g"].dim() == 2 else st["g"].expand(T, -1)).double().exp()
    back = st["kind"] == "backward"
    S = st["s0"].double().clone() if st["s0"] is not None else torch.zeros(n, Hv, D, D, dtype=torch.float64, device=dev)
    lens = [b - a for a, b in zip(cu, cu[1:])]
    # sequences by falling length, so that those still running are a prefix
    order = sorted(range(n), key=lambda i: -lens[i])
    S = S[order]
    base = torch.tensor([cu[i] for i in order], device=dev)
    o = torch.zeros(T, Hv, D, dtype=torch.float64, device=dev)
    dq = torch.zeros_like(o)
    d_o = st["d_o"].double() if back else None
    alive = [sum(1 for x in lens if x > t) for t in range(max(lens))]
    for t, m in enumerate(alive):
        at = base[:m] + t
        s = S[:m]
        s.mul_(decay[at][..., None, None]).addcmul_(v[at][..., None], wide["k"][at][..., None, :])
        if back:
            dq[at] = scale * torch.einsum("nhij,nhi->nhj", s, d_o[at])
        else:
            o[at] = scale * torch.einsum("nhij,nhj->nhi", s, wide["q"][at])
    undo = torch.tensor([order.index(i) for i in range(n)], device=dev)
    if not back:
        return {"o": o, "final_state": S[undo]}
    R = st["d_final"][order].double() if st["d_final"] is not None else torch.zeros_like(S)
    dk, dv, dg = torch.zeros_like(o), torch.zeros_like(o), torch.zeros(T, Hv, dtype=torch.float64, device=dev)
    # <S, dS> behind each token, carried from the last one back
    B = (S * R).sum((-1, -2))
    for t in range(max(lens) - 1, -1, -1):
        m = alive[t]
        at = base[:m] + t
        r, b = R[:m], B[:m]
        r.addcmul_(scale * d_o[at][..., None], wide["q"][at][..., None, :])
        b += (wide["q"][at] * dq[at]).sum(-1)
        dk[at] = torch.einsum("nhij,nhi->nhj", r, v[at])
        dv[at] = torch.einsum("nhij,nhj->nhi", r, wide["k"][at])
        b -= (dv[at] * v[at]).sum(-1)
        dg[at] = b
        r.mul_(decay[at][..., None, None])
    fold = lambda x: x.view(T, -1, rep, D).sum(2)  # noqa: E731
    return {"dq": fold(dq), "dk": fold(dk), "dv": dv, "dg": dg.sum(0) if st["g"].dim() == 1 else dg,
            "d_initial_state": R[undo] if st["s0"] is not None else None}


def _exact_step(st):
    n, layers, Hv = st["n_seq"], st["layers"], st["v"].shape[1]
    rep = Hv // st["q"].shape[1]
    state = st["state"].double() if st["state"].numel() < (1 << 27) else None
    o = torch.zeros(n * layers, Hv, D, dtype=torch.float64, device=st["q"].device)
    for i, slot in enumerate(st["slot"].tolist()):
        if slot < 0:
            continue
        u, p = slice(i * layers, (i + 1) * layers), slice(slot * layers, (slot + 1) * layers)
        q, k = (st[m][u].double().repeat_interleave(rep, 1) for m in ("q", "k"))
        decay = (st["g"][u] if st["g"].shape[0] == n * layers and n > 1 else st["g"][:layers]).double().exp()
        s = decay[..., None, None] * st["state"][p].double() + torch.einsum("lhi,lhj->lhij", st["v"][u].double(), k)
        o[u] = st["scale"] * torch.einsum("lhij,lhj->lhi", s, q)
        if state is not None:
            state[p] = s
    return {"o": o, "state": state}


def _exact_pool(st):
    """Page by page, in Python."""
    old = [b.double() if b.numel() < (1 << 27) else b for b in st["buffers"]]
    if any(b.dtype != torch.float64 for b in old):
        old = None
    if st["kind"] == "copy":
        if old is None:
            return None
        new = [b.clone() for b in old]
        for a, b in zip(st["src"].tolist(), st["dst"].tolist()):
            for x, y in zip(old, new):
                y[b] = x[a]
        return {"buffers": new}
    live, out = st["live"].tolist(), {}
    if st["kind"] == "turnover":
        for s in st["done"].tolist():
            live[s] = 0
        left = sum(live)
        out["moved"] = [s if live[s] else -1 for s in range(len(live))]
        gaps = [s for s in range(left) if not live[s]]
        for a, b in zip([s for s in range(left, len(live)) if live[s]], gaps):
            out["moved"][a] = b
            for x in old or []:
                x[b] = x[a]
        live = [1] * left + [0] * (len(live) - left)
    dst = [s for s in range(len(live)) if not live[s]][: st["src"].numel()]
    before = None if old is None else [b.clone() for b in old]
    for a, b in zip(st["src"].tolist(), dst):
        live[b] = 1
        for x, y in zip(before or [], old or []):
            y[b] = x[a] if a >= 0 else 0
    if st["kind"] == "fork":
        for s in dst:
            live[s] = 0
    whole = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    out = {m: whole(x) for m, x in out.items()}
    return dict(out, dst=whole(dst), live=whole(live), buffers=old)
