"""Workloads of the causal operators: packed causal softmax attention with
grouped heads (forward, training, single tokens against caches) and linear
attention with a decay for each head (prompts, training, single tokens).

``run`` computes one pass: in its plain form with elementary torch operations
in 32 bits, or, where ``own`` is true, by the calls a user makes of this
framework.  ``exact`` gives the same outputs in 64 bits, sequence by sequence.
"""

from __future__ import annotations

import math

import torch

own = False


# ------------------------------------------------------------------ cases

def _text(lengths):
    return " ".join(str(n) for n in lengths)


def _numbers(text):
    return [int(n) for n in text.split()]


def listed():
    return [
        # the smallest call: one short prompt, where latency counts
        dict(name="attn prompt 37", kind="attn", q="37", k="37", cap=0, Hq=12, Hkv=4, d=128),
        # an ordinary batch of prompts of mixed lengths, packed without padding
        dict(name="attn prompts packed", kind="attn",
             q=_text([1, 2048, 333, 7, 1024, 129, 1500, 64, 640, 255, 777, 1, 90, 512, 128, 1111]),
             k=_text([1, 2048, 333, 7, 1024, 129, 1500, 64, 640, 255, 777, 1, 90, 512, 128, 1111]),
             cap=0, Hq=16, Hkv=4, d=128),
        # one long prompt
        dict(name="attn prompt 16384", kind="attn", q="16384", k="16384", cap=0, Hq=12, Hkv=4,
             d=128),
        # a training step on packed documents, small heads, every head with its own keys
        dict(name="attn train packed d64", kind="attn_train",
             q=_text([700, 1, 1333, 256, 65, 2000, 31, 900]),
             k=_text([700, 1, 1333, 256, 65, 2000, 31, 900]), cap=0, Hq=8, Hkv=8, d=64),
        # a training step on long sequences with shared key heads
        dict(name="attn train 2x8192", kind="attn_train", q="8192 8192", k="8192 8192", cap=0,
             Hq=12, Hkv=4, d=128),
        # one generated token for each of many sequences, caches of a fixed capacity filled unevenly
        dict(name="attn tokens 48 caches", kind="attn", q=_text([1] * 48),
             k=_text([(i * 2654435761 >> 7) % 8192 + 1 for i in range(48)]), cap=8192, Hq=16,
             Hkv=4, d=128),
        # one generated token of one sequence
        dict(name="attn token 1 cache", kind="attn", q="1", k="4001", cap=4096, Hq=12, Hkv=4,
             d=128),
        # an ordinary batch of prompts through the decayed linear branch, states kept
        dict(name="decay prompts packed", kind="decay",
             q=_text([1, 2048, 333, 7, 1024, 129, 1500, 64, 640, 255, 777, 1]), H=12, d=128,
             start=False),
        # one long prompt that continues from a state
        dict(name="decay prompt 16384", kind="decay", q="16384", H=12, d=128, start=True),
        # a training step over packed sequences that continue from states
        dict(name="decay train packed", kind="decay_train",
             q=_text([4096, 1333, 1, 2500, 64, 190]), H=8, d=64, start=True),
        # one generated token for each of many sequences
        dict(name="decay tokens 192", kind="step", n=192, H=12, d=128),
        # one generated token of one sequence, where latency counts
        dict(name="decay token 1", kind="step", n=1, H=12, d=128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["attn", "attn", "attn_train", "attn_cache", "decay", "decay_train", "step"])
    d = rng.choice([64, 128])
    if kind == "step":
        return dict(kind="step", n=_log_int(rng, 1, 192), H=_log_int(rng, 1, 16), d=d)
    # the plain form works on padded score matrices: their number of entries is bounded
    most = {"attn": 16384 ** 2 * 12, "attn_train": 8192 ** 2 * 24, "decay": 16384 ** 2 * 12,
            "decay_train": 4096 ** 2 * 48}.get(kind, 0)
    if kind == "attn_cache":
        n, G, Hkv = _log_int(rng, 1, 48), rng.randint(1, 8), rng.randint(1, 4)
        cap = 8 * _log_int(rng, 8, 1024)
        q = [rng.choice([1, 1, 1, 2, 5])] * n
        k = [rng.randint(q[0], cap) for _ in range(n)]
        return dict(kind="attn", q=_text(q), k=_text(k), cap=cap, Hq=G * Hkv, Hkv=Hkv, d=d)
    Hkv = rng.randint(1, 8)
    G = rng.choice([1, 1, 2, 3, 4]) if kind.startswith("attn") else 1
    while G * Hkv > 16:
        G -= 1
    n = _log_int(rng, 1, 16)
    longest = _log_int(rng, 1, min(16384, int(math.sqrt(most / (n * G * Hkv * 1.01)))))
    q = [longest] + [_log_int(rng, 1, longest) for _ in range(n - 1)]
    rng.shuffle(q)
    if kind.startswith("decay"):
        return dict(kind=kind, q=_text(q), H=Hkv, d=d, start=rng.random() < 0.5)
    k = list(q)
    if kind == "attn" and rng.random() < 0.4:  # prompts that continue behind cached keys
        k = [a + rng.randint(0, max(1, longest // 2)) for a in q]
        q = [max(1, a * 2 // 3) for a in q]
    return dict(kind=kind, q=_text(q), k=_text(k), cap=0, Hq=G * Hkv, Hkv=Hkv, d=d)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, gain=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * gain).to(torch.bfloat16)


def _offsets(lengths):
    off = [0]
    for n in lengths:
        off.append(off[-1] + n)
    return off


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _decays(H):
    """Log-decays of the heads, from a memory of about 2 tokens to one of about 2000."""
    return torch.tensor([-math.exp(math.log(0.5) + (math.log(5e-4) - math.log(0.5)) * h /
                                   max(1, H - 1)) for h in range(H)],
                        dtype=torch.float32, device="cuda")


def _inputs(case, seed):
    g = _gen(seed)
    kind, d = case["kind"], case["d"]
    s = dict(case)
    if kind == "step":
        n, H = case["n"], case["H"]
        s["qv"], s["kv"], s["vv"] = (_normal(g, n, H, d) for _ in range(3))
        s["state"] = torch.randn(n, H, d, d, generator=g, device="cuda")
        s["log_decay"] = _decays(H)
        s["scale"] = d ** -0.5
        return s
    lq = _numbers(case["q"])
    s["lq"], s["scale"] = lq, d ** -0.5
    s["q_off"] = _int32(_offsets(lq))
    tq = sum(lq)
    if kind.startswith("attn"):
        lk, cap = _numbers(case["k"]), case["cap"]
        tk = cap * len(lk) if cap else sum(lk)
        s["lk"], s["tk"] = lk, tk
        s["k_off"] = _int32([cap * i for i in range(len(lk) + 1)] if cap else _offsets(lk))
        s["k_len"] = _int32(lk) if cap else None
        # queries with a gain: some rows look at few keys, as trained heads do
        s["qv"] = _normal(g, tq, case["Hq"], d, gain=2.0)
        s["kv"], s["vv"] = (_normal(g, tk, case["Hkv"], d) for _ in range(2))
        if kind == "attn_train":
            s["do"] = _normal(g, tq, case["Hq"], d)
        return s
    H = case["H"]
    s["qv"], s["kv"], s["vv"] = (_normal(g, tq, H, d) for _ in range(3))
    s["log_decay"] = _decays(H)
    n = len(lq)
    s["state0"] = (torch.randn(n, H, d, d, generator=g, device="cuda") if case["start"] else None)
    if kind == "decay_train":
        s["do"] = _normal(g, tq, H, d)
        s["d_state1"] = torch.randn(n, H, d, d, generator=g, device="cuda")
    return s


def _padding(lengths, starts, device="cuda"):
    """Row of every (sequence, position) of a padded batch, and the place of every packed row in it."""
    longest = max(lengths)
    n = torch.tensor(lengths, device=device)
    pos = torch.arange(longest, device=device)
    rows = torch.tensor(starts, device=device)[:, None] + torch.minimum(pos[None], n[:, None] - 1)
    seq = torch.repeat_interleave(torch.arange(len(lengths), device=device), n)
    at = torch.arange(sum(lengths), device=device) - torch.tensor(
        _offsets(lengths)[:-1], device=device)[seq]
    return rows, seq, at, n


def prepare(case, seed):
    s = _inputs(case, seed)
    if case["kind"] == "step":
        if own:
            import sparse_linear_attention_block_b200 as slab
            s["shape"] = slab.make_decay_shape(case["n"], case["n"], case["H"], case["d"],
                                               scale=s["scale"])
            s["buf"] = slab.DecayBuffers.allocate(s["shape"], state=False)
        return s
    lq = s["lq"]
    s["q_pad"] = _padding(lq, _offsets(lq)[:-1])
    if case["kind"].startswith("attn"):
        lk, cap = s["lk"], case["cap"]
        s["k_pad"] = _padding(lk, [cap * i for i in range(len(lk))] if cap else _offsets(lk)[:-1])
        if own:
            import sparse_linear_attention_block_b200 as slab
            s["shape"] = slab.make_causal_shape(len(lq), sum(lq), s["tk"], case["Hq"],
                                                case["Hkv"], case["d"], max_q=max(lq),
                                                scale=s["scale"])
            s["buf"] = slab.CausalBuffers.allocate(s["shape"],
                                                   backward=case["kind"] == "attn_train")
    elif own:
        import sparse_linear_attention_block_b200 as slab
        s["shape"] = slab.make_decay_shape(len(lq), sum(lq), case["H"], case["d"],
                                           scale=s["scale"])
        s["buf"] = slab.DecayBuffers.allocate(s["shape"], backward=case["kind"] == "decay_train")
    return s


# ------------------------------------------------------------------ plain forms

def _padded(x, rows):
    """Packed [rows, heads, d] to padded 32-bit [sequence, head, position, d]."""
    return x[rows].float().transpose(1, 2)


def _packed(x, seq, at):
    """Padded [sequence, head, position, ...] to packed rows [row, head, ...]."""
    return x[seq, :, at]


def _plain_attention(s):
    (rq, seq, at, nq), (rk, kseq, kat, nk) = s["q_pad"], s["k_pad"]
    Hkv, G, d = s["Hkv"], s["Hq"] // s["Hkv"], s["d"]
    q = _padded(s["qv"], rq).unflatten(1, (Hkv, G))
    k, v = (_padded(s[x], rk).unsqueeze(2) for x in ("kv", "vv"))
    a = torch.arange(rq.shape[1], device="cuda")
    b = torch.arange(rk.shape[1], device="cuda")
    seen = b[None, None] <= a[None, :, None] + (nk - nq)[:, None, None]
    seen &= (b[None] < nk[:, None])[:, None]
    seen = seen[:, None, None]
    w = (q @ k.transpose(-1, -2)).mul_(s["scale"]).masked_fill_(~seen, -math.inf)
    top = w.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    w = w.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    w /= torch.where(total == 0, 1.0, total)
    o = w @ v
    lse = _packed((top + total.log()).squeeze(-1).flatten(1, 2), seq, at).t().contiguous()
    out = _packed(o.flatten(1, 2), seq, at).to(torch.bfloat16)
    if s["kind"] == "attn":
        return [out, lse]
    # gradients; rows behind a sequence's end get no weight
    real = (a[None] < nq[:, None])[:, None, None, :, None]
    do = _padded(s["do"], rq).unflatten(1, (Hkv, G)) * real
    dv = (w.transpose(-1, -2) @ do).sum(2)
    slope = do @ v.transpose(-1, -2)
    slope -= (o * do).sum(-1, keepdim=True)
    slope *= w
    slope *= s["scale"]
    dq = slope @ k
    dk = (slope.transpose(-1, -2) @ q).sum(2)
    return [out, lse, _packed(dq.flatten(1, 2), seq, at).to(torch.bfloat16),
            _packed(dk, kseq, kat).to(torch.bfloat16), _packed(dv, kseq, kat).to(torch.bfloat16)]


def _plain_decay(s):
    rq, seq, at, n = s["q_pad"]
    g, scale = s["log_decay"], s["scale"]
    q, k, v = (_padded(s[x], rq) for x in ("qv", "kv", "vv"))
    t = torch.arange(rq.shape[1], device="cuda")
    real = (t[None] < n[:, None])[:, None, :, None].float()
    k, v = k * real, v * real
    ago = (t[:, None] - t[None]).float()
    w = torch.where(ago >= 0, (g[:, None, None] * ago.clamp(min=0)).exp(), 0.0)  # head, t, s
    since = (g[:, None] * (t + 1)).exp()[None, :, :, None]                       # from the start
    left = (n[:, None] - 1 - t[None]).clamp(min=0)                               # to the end
    until = (g[None, :, None] * left[:, None]).exp()[..., None] * real
    whole = (g[None] * n[:, None]).exp()[..., None, None]
    mix = (q @ k.transpose(-1, -2)).mul_(w)
    o = mix @ v
    state = (k * until).transpose(-1, -2) @ v
    if s["state0"] is not None:
        o += since * (q @ s["state0"])
        state = state + whole * s["state0"]
    out = _packed(o * scale, seq, at).to(torch.bfloat16)
    if s["kind"] == "decay":
        return [out, state]
    do = _padded(s["do"], rq) * real
    end = s["d_state1"]
    dv = scale * (mix.transpose(-1, -2) @ do) + until * (k @ end)
    slope = (do @ v.transpose(-1, -2)).mul_(w).mul_(scale)
    dq = slope @ k
    dk = slope.transpose(-1, -2) @ q + until * (v @ end.transpose(-1, -2))
    if s["state0"] is not None:
        dq += scale * since * (do @ s["state0"].transpose(-1, -2))
    start = scale * ((q * since).transpose(-1, -2) @ do) + whole * end
    return [out, state] + [_packed(x, seq, at).to(torch.bfloat16) for x in (dq, dk, dv)] + [start]


def _plain_step(s):
    q, k, v = (s[x].float() for x in ("qv", "kv", "vv"))
    s["state"].mul_(s["log_decay"].exp()[None, :, None, None])
    s["state"].add_(k[..., :, None] * v[..., None, :])
    o = (q[..., None, :] @ s["state"]).squeeze(-2) * s["scale"]
    return [o.to(torch.bfloat16), s["state"]]


# ------------------------------------------------------------------ this framework's calls

def _own(s):
    import sparse_linear_attention_block_b200 as slab
    b, kind = s["buf"], s["kind"]
    if kind.startswith("attn"):
        slab.sla_causal_forward(s["shape"], s["qv"], s["kv"], s["vv"], s["q_off"], s["k_off"],
                                s["k_len"], b.o, b.lse, b.workspace)
        if kind == "attn":
            return [b.o, b.lse]
        slab.sla_causal_backward(s["shape"], s["qv"], s["kv"], s["vv"], s["q_off"], s["k_off"],
                                 b.o, b.lse, s["do"], b.dq, b.dk, b.dv, b.workspace)
        return [b.o, b.lse, b.dq, b.dk, b.dv]
    if kind == "step":
        slab.sla_decay_step(s["shape"], s["qv"], s["kv"], s["vv"], s["log_decay"], s["state"],
                            s["state"], b.o)
        return [b.o, s["state"]]
    slab.sla_decay_forward(s["shape"], s["qv"], s["kv"], s["vv"], s["log_decay"], s["q_off"],
                           s["state0"], b.o, b.state, b.workspace)
    if kind == "decay":
        return [b.o, b.state]
    slab.sla_decay_backward(s["shape"], s["qv"], s["kv"], s["vv"], s["log_decay"], s["q_off"],
                            s["state0"], s["do"], s["d_state1"], b.dq, b.dk, b.dv, b.d_state,
                            b.workspace)
    return [b.o, b.state, b.dq, b.dk, b.dv, b.d_state]


def run(state):
    if own:
        return _own(state)
    if state["kind"] == "step":
        return _plain_step(state)
    return _plain_attention(state) if state["kind"].startswith("attn") else _plain_decay(state)


# ------------------------------------------------------------------ work and exact values

def work(case):
    d, kind = case["d"], case["kind"]
    if kind == "step":
        n, H = case["n"], case["H"]
        return {"bytes": n * H * (8 * d * d + 8 * d) + 4 * H, "flops": 5 * n * H * d * d}
    lq = _numbers(case["q"])
    t = sum(lq)
    if kind.startswith("attn"):
        Hq, Hkv, lk = case["Hq"], case["Hkv"], _numbers(case["k"])
        pairs = sum(sum(min(b, max(0, a + 1 + b - c)) for a in (0, c - 1)) / 2 * c if b >= c else
                    b * (b + 1) / 2 for c, b in zip(lq, lk))
        rows, keys = t * Hq, sum(lk) * Hkv
        if kind == "attn":
            return {"bytes": rows * (4 * d + 4) + keys * 4 * d, "flops": 4 * d * pairs * Hq}
        return {"bytes": rows * (8 * d + 4) + keys * 8 * d, "flops": 14 * d * pairs * Hq}
    H, n = case["H"], len(lq)
    states = n * H * d * d * 4
    some = states if case["start"] else 0
    if kind == "decay":
        return {"bytes": t * H * 8 * d + states + some, "flops": 4 * d * d * t * H}
    return {"bytes": t * H * 16 * d + 3 * states + some, "flops": 14 * d * d * t * H}


def _exact_attention(s):
    Hq, Hkv, d, scale = s["Hq"], s["Hkv"], s["d"], s["scale"]
    G, train = Hq // Hkv, s["kind"] == "attn_train"
    wide = dict(dtype=torch.float64, device="cuda")
    tq = sum(s["lq"])
    out, lse = torch.zeros(tq, Hq, d, **wide), torch.full((Hq, tq), -math.inf, **wide)
    dq = torch.zeros(tq, Hq, d, **wide) if train else None
    dk, dv = (torch.zeros(s["tk"], Hkv, d, **wide) if train else None for _ in range(2))
    first = s["k_off"].tolist()
    row = 0
    for i, (nq, nk) in enumerate(zip(s["lq"], s["lk"])):
        mine, keys = slice(row, row + nq), slice(first[i], first[i] + nk)
        row += nq
        hidden = torch.ones(nq, nk, dtype=torch.bool, device="cuda").triu(nk - nq + 1)
        for h in range(Hq):
            q, k, v = (x.double() for x in (s["qv"][mine, h], s["kv"][keys, h // G],
                                            s["vv"][keys, h // G]))
            z = (q @ k.T) * scale
            z[hidden] = -math.inf
            l = torch.logsumexp(z, -1)
            p = torch.exp(z - torch.where(l == -math.inf, 0.0, l)[:, None])
            del z
            out[mine, h], lse[h, mine] = p @ v, l
            if train:
                do = s["do"][mine, h].double()
                dv[keys, h // G] += p.T @ do
                ds = p * (do @ v.T - (out[mine, h] * do).sum(-1, keepdim=True)) * scale
                dq[mine, h] = ds @ k
                dk[keys, h // G] += ds.T @ q
    return [out, lse, dq, dk, dv] if train else [out, lse]


def _exact_decay(s):
    """The recurrence itself, in steps of up to 128 tokens."""
    H, d, scale, train = s["H"], s["d"], s["scale"], s["kind"] == "decay_train"
    wide = dict(dtype=torch.float64, device="cuda")
    t = sum(s["lq"])
    g = s["log_decay"].double()
    out = torch.zeros(t, H, d, **wide)
    grads = [torch.zeros(t, H, d, **wide) for _ in range(3)]
    ends, starts = [], []
    row = 0

    def step(i, j):
        c = j - i
        u = torch.arange(c, **wide)
        mix = torch.tril(torch.exp(g[:, None, None] * torch.tril(u[:, None] - u[None])))
        q, k, v = (s[x][i:j].double().transpose(0, 1) for x in ("qv", "kv", "vv"))
        fade = torch.exp(g[:, None] * u[None])[..., None]      # after u tokens
        back = fade.flip(1)                                    # c - 1 - u tokens before the end
        return c, mix, q, k, v, fade, back, torch.exp(g * c)[:, None, None]

    for i, n in enumerate(s["lq"]):
        cuts = [(a, min(row + n, a + 128)) for a in range(row, row + n, 128)]
        row += n
        S = torch.zeros(H, d, d, **wide) if s["state0"] is None else s["state0"][i].double()
        lam = torch.exp(g)[:, None, None]
        for a, b in cuts:
            c, mix, q, k, v, fade, back, whole = step(a, b)
            o = (mix * (q @ k.mT)) @ v + lam * fade * (q @ S)
            out[a:b] = (scale * o).transpose(0, 1)
            if train:
                do = s["do"][a:b].double().transpose(0, 1)
                dq = (mix * (do @ v.mT)) @ k + lam * fade * (do @ S.mT)
                grads[0][a:b] = (scale * dq).transpose(0, 1)
            S = whole * S + (k * back).mT @ v
        ends.append(S)
        if train:
            B = s["d_state1"][i].double()  # with respect to the state behind the step's tokens
            for a, b in reversed(cuts):
                c, mix, q, k, v, fade, back, whole = step(a, b)
                do = s["do"][a:b].double().transpose(0, 1) * scale
                grads[1][a:b] = ((mix * (do @ v.mT)).mT @ q + back * (v @ B.mT)).transpose(0, 1)
                grads[2][a:b] = ((mix * (q @ k.mT)).mT @ do + back * (k @ B)).transpose(0, 1)
                B = whole * B + (lam * fade * q).mT @ do
            starts.append(B)
    return [out, torch.stack(ends)] + (grads + [torch.stack(starts)] if train else [])


def exact(case, seed):
    s = _inputs(case, seed)
    if case["kind"] == "step":
        S = s["state"].double() * torch.exp(s["log_decay"].double())[None, :, None, None]
        S += torch.einsum("nhk,nhv->nhkv", s["kv"].double(), s["vv"].double())
        return [torch.einsum("nhk,nhkv->nhv", s["qv"].double(), S) * s["scale"], S]
    return _exact_attention(s) if case["kind"].startswith("attn") else _exact_decay(s)
