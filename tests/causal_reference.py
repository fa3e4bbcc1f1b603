"""The causal operators in 64 bits from their definitions, sequence by sequence,
with the companions that the tolerances need: for every output the sum of the
absolute values of its terms.

Tolerances.  u = 2^-8 is half a step of bf16 (relative).  The kernels round to
bf16 once at each output and once at the operands that they feed back into a
matrix product (the weights P, the slopes dS, the state read by a query), and
hold everything else in 32 bits.  So an output that is a sum of terms t_i with
one rounded factor each is off by at most u |sum t_i| + u sum |t_i|; a quarter
of u on top (2^-10) covers the 32-bit scores: they are off by at most
d 2^-23 scale sum |q k|, below 2^-11 for the values used here, which is the
relative error of exp of them, and the exponential's own 2^-20.
The bound on the whole tensor (2-norm) takes the roundings as independent, each
with a root mean square of at most u / sqrt(3): three of them give u.
"""

import math

import torch

U = 2.0 ** -8


def heads(x, rows, h):
    return x[rows, h].double()


def attention(q, k, v, seqs, scale, d_o=None):
    """seqs: [(q0, nq, k0, nk)].  Values, tolerances and which rows are written."""
    tq, Hq, d = q.shape
    tk, Hkv, _ = k.shape
    G = Hq // Hkv
    z = dict(dtype=torch.float64, device=q.device)
    r = dict(o=torch.zeros(tq, Hq, d, **z), lse=torch.full((Hq, tq), -math.inf, **z))
    t = dict(o=torch.zeros(tq, Hq, d, **z), lse=torch.zeros(Hq, tq, **z))
    for n, x in (("dq", q), ("dk", k), ("dv", v)):
        r[n], t[n] = torch.zeros(x.shape, **z), torch.zeros(x.shape, **z)
    slip = dict(dq=0.0, dk=0.0)
    used_q = torch.zeros(tq, dtype=torch.bool, device=q.device)
    used_k = torch.zeros(tk, dtype=torch.bool, device=q.device)
    for q0, nq, k0, nk in seqs:
        a, b = slice(q0, q0 + nq), slice(k0, k0 + nk)
        used_q[a] = True
        used_k[b] = True
        if nq == 0:
            continue
        seen = (torch.arange(nk, device=q.device)[None] <=
                torch.arange(nq, device=q.device)[:, None] + nk - nq)
        for h in range(Hq):
            Q, K, V = heads(q, a, h), heads(k, b, h // G), heads(v, b, h // G)
            s = torch.where(seen, Q @ K.T * scale, -math.inf)
            if nk:
                lse = torch.logsumexp(s, 1)
                mass = (Q.abs() @ K.abs().T).amax(1) * scale
            else:
                lse = torch.full((nq,), -math.inf, **z)
                mass = torch.zeros(nq, **z)
            p = torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[:, None])
            o = p @ V
            r["o"][a, h], r["lse"][h, a] = o, lse
            t["o"][a, h] = U * o.abs() + 1.25 * U * (p @ V.abs())
            t["lse"][h, a] = d * 2.0 ** -23 * mass + 2.0 ** -18
            if d_o is None:
                continue
            g = heads(d_o, a, h)
            dd = (t["o"][a, h] * g.abs()).sum(1, keepdim=True)  # o's own error in D
            ds = p * (g @ V.T - (o * g).sum(1, keepdim=True)) * scale
            ra = math.sqrt(2 / 3) * U * (o * g).norm(dim=1, keepdim=True) * scale
            slip["dq"] += float((ra * (p @ K)).square().sum())
            slip["dk"] += float(((ra * p).T.square() @ Q.square()).sum())
            off = 1.25 * U * ds.abs() + p * dd * scale
            r["dq"][a, h] = ds @ K
            t["dq"][a, h] = off @ K.abs()
            r["dk"][b, h // G] += ds.T @ Q
            t["dk"][b, h // G] += off.T @ Q.abs()
            r["dv"][b, h // G] += p.T @ g
            t["dv"][b, h // G] += 1.25 * U * (p.T @ g.abs())
    for n in ("dq", "dk", "dv"):
        t[n] += U * r[n].abs()
    norms = {n: U for n in ("o", "dv")}
    for n in ("dq", "dk"):
        norms[n] = U + 3 * math.sqrt(slip[n]) / max(float(r[n].norm()), 1e-30)
    r["norms"] = norms
    return r, t, used_q, used_k


def decay(q, k, v, log_decay, seqs, scale, state_in=None, d_o=None, d_state_out=None):
    """seqs: [(first row, rows)].  The recurrence as one masked product per sequence."""
    T, H, d = q.shape
    z = dict(dtype=torch.float64, device=q.device)
    g = log_decay.double()
    n = len(seqs)
    r, t = {}, {}
    for name, x in (("o", q), ("dq", q), ("dk", k), ("dv", v)):
        r[name], t[name] = torch.zeros(x.shape, **z), torch.zeros(x.shape, **z)
    for name in ("state", "d_state"):
        r[name], t[name] = torch.zeros(n, H, d, d, **z), torch.zeros(n, H, d, d, **z)

    def power(h, e):  # exp(g e), 1 at e = 0 also where g is -inf
        return torch.where(e == 0, 1.0, torch.exp(g[h] * torch.where(e == 0, 1.0, e)))

    for i, (row, m) in enumerate(seqs):
        at = slice(row, row + m)
        e = torch.arange(m, **z)
        for h in range(H):
            S0 = state_in[i, h].double() if state_in is not None else torch.zeros(d, d, **z)
            B = (d_state_out[i, h].double() if d_state_out is not None
                 else torch.zeros(d, d, **z))
            Q, K, V = heads(q, at, h), heads(k, at, h), heads(v, at, h)
            ago = e[:, None] - e[None]
            w = torch.where(ago >= 0, power(h, ago.clamp(min=0)), 0.0)
            since, until = power(h, e + 1)[:, None], power(h, m - 1 - e)[:, None]
            whole = power(h, torch.tensor(float(m), **z))

            def put(name, idx, value, terms, rounded=True):
                r[name][idx] = value
                t[name][idx] = (U * value.abs() + 1.25 * U * terms if rounded
                                else 2.0 ** -16 * terms)

            put("o", (at, h), scale * ((w * (Q @ K.T)) @ V + since * (Q @ S0)),
                scale * ((w * (Q.abs() @ K.abs().T)) @ V.abs() + since * (Q.abs() @ S0.abs())))
            put("state", (i, h), (K * until).T @ V + whole * S0,
                (K * until).abs().T @ V.abs() + whole * S0.abs(), False)
            if d_o is None:
                continue
            D = heads(d_o, at, h)
            a = w * (D @ V.T) * scale
            aa = w * (D.abs() @ V.abs().T) * scale
            put("dq", (at, h), a @ K + scale * since * (D @ S0.T),
                aa @ K.abs() + scale * since * (D.abs() @ S0.abs().T))
            put("dk", (at, h), a.T @ Q + until * (V @ B.T),
                aa.T @ Q.abs() + until * (V.abs() @ B.abs().T))
            put("dv", (at, h), scale * (w * (Q @ K.T)).T @ D + until * (K @ B),
                scale * (w * (Q.abs() @ K.abs().T)).T @ D.abs() + until * (K.abs() @ B.abs()))
            put("d_state", (i, h), scale * (Q * since).T @ D + whole * B,
                scale * (Q * since).abs().T @ D.abs() + whole * B.abs(), False)
    return r, t


def check(name, got, ref, tol, norm=None):
    """Every element within its tolerance, infinities equal, and the 2-norm."""
    got = got.double()
    fine = torch.isfinite(ref)
    assert torch.equal(got[~fine], ref[~fine]), f"{name}: infinities differ"
    assert torch.isfinite(got[fine]).all(), f"{name}: not finite"
    off = (got - ref)[fine].abs()
    # the smallest bf16 numbers have a fixed step
    bad = off > tol[fine] + 2.0 ** -120
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} outside, worst "
                           f"{float((off / (tol[fine] + 1e-30)).max()):.3g} of the tolerance")
    if norm is not None and fine.any():
        rel = float(off.norm() / ref[fine].norm().clamp(min=1e-30))
        assert rel <= norm, f"{name}: 2-norm of the error {rel:.3g} of the result's"
