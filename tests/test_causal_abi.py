"""Host-side checks of the causal entry points: sizes, refusals before anything
is launched, the binding's checks, and the 64-bit reference against central
differences.  No GPU."""

import ctypes
import math

import pytest
import torch

import causal_reference as ref
import sparse_linear_attention_block_b200 as slab
from sparse_linear_attention_block_b200 import build as slab_build

GOOD = 0x7f0000000000  # aligned, never dereferenced: every check fails first


@pytest.fixture(scope="module")
def L():
    slab_build.build()
    return slab.lib()


def causal(**kw):
    a = dict(n_seq=2, total_q=300, total_k=400, Hq=4, Hkv=2, d=64)
    a.update(kw)
    return slab.make_causal_shape(**a)


def decay(**kw):
    a = dict(n_seq=2, total=300, H=4, d=64)
    a.update(kw)
    return slab.make_decay_shape(**a)


def test_sizes(L):
    s = slab.sla_causal_query_sizes(causal())
    assert s.lse_bytes == 4 * 300 * 4 and s.workspace_bytes > 0
    s = slab.sla_decay_query_sizes(decay())
    assert s.state_bytes == 2 * 4 * 64 * 64 * 4 and s.workspace_bytes > 0


@pytest.mark.parametrize("kw,code", [
    (dict(n_seq=0), 1), (dict(total_q=0), 1), (dict(total_k=0), 1), (dict(Hq=3), 1),
    (dict(Hkv=0), 1), (dict(max_q=-1), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(d=96), 2), (dict(n_seq=2 ** 20 + 1), 2),
    (dict(total_q=2 ** 30), 2), (dict(Hq=2048, Hkv=1), 2),
    (dict(q=(256, 60)), 1),          # heads overlap
    (dict(q=(128, 64)), 1),          # rows overlap
    (dict(k=(128, 68)), 1),          # not a multiple of 8
    (dict(v=(0, 64)), 1),            # a broadcast tensor
    (dict(o=(256, 0)), 1),
    (dict(o=(2 ** 40, 64)), 1),
])
def test_causal_shapes_refused(L, kw, code):
    with pytest.raises(slab.SlaError) as e:
        slab.sla_causal_query_sizes(causal(**kw))
    assert e.value.status == code


@pytest.mark.parametrize("kw", [dict(q=(640, 64)), dict(q=(64, 300 * 64)), dict(k=(128, 64)),
                                dict(Hq=2, Hkv=2, q=(64, 64 * 300)), dict(o=(256, 64))])
def test_strides_accepted(L, kw):
    slab.sla_causal_query_sizes(causal(**kw))


@pytest.mark.parametrize("kw,code", [
    (dict(n_seq=0), 1), (dict(total=0), 1), (dict(H=0), 1), (dict(scale=float("nan")), 1),
    (dict(d=32), 2), (dict(total=2 ** 30), 2), (dict(H=1025), 2), (dict(q=(256, 60)), 1)])
def test_decay_shapes_refused(L, kw, code):
    with pytest.raises(slab.SlaError) as e:
        slab.sla_decay_query_sizes(decay(**kw))
    assert e.value.status == code


def test_null_misaligned_and_small_arguments_are_refused(L):
    def rejects(fn, shape, args, ws, optional=()):
        """args with every required one dropped and every pointer misaligned in turn."""
        byref = ctypes.byref(shape)
        tail = [ws, 16, None] if ws else [None]
        for i, x in enumerate(args):
            bad = list(args)
            if i not in optional:
                bad[i] = None
                assert fn(byref, *bad, *tail) == 1, i
            bad[i] = GOOD + 2
            assert fn(byref, *bad, *tail) == 1, i
        assert fn(None, *args, *tail) == 1
        if ws:
            assert fn(byref, *args, None, 1 << 40, None) == 1
            assert fn(byref, *args, GOOD + 512, 1 << 40, None) == 1
            assert fn(byref, *args, *tail) == 3  # the workspace is too small

    rejects(L.sla_causal_forward, causal(), [GOOD] * 8, GOOD, optional=(5,))
    rejects(L.sla_causal_backward, causal(), [GOOD] * 11, GOOD)
    rejects(L.sla_decay_forward, decay(), [GOOD] * 8, GOOD, optional=(5, 7))
    rejects(L.sla_decay_backward, decay(), [GOOD] * 12, GOOD, optional=(5, 7, 11))
    rejects(L.sla_decay_step, decay(n_seq=300), [GOOD] * 7, None)
    # a step has one row for each sequence
    assert L.sla_decay_step(ctypes.byref(decay()), *[GOOD] * 7, None) == 1


def test_the_binding_refuses_other_tensors(L):
    """Types, sizes, strides and devices, before the library is called."""
    s = causal()
    bf = torch.bfloat16
    q, k = torch.zeros(300, 4, 64, dtype=bf), torch.zeros(400, 2, 64, dtype=bf)

    def refused(q=q, k=k):
        with pytest.raises(slab.SlaError) as e:
            slab.sla_causal_forward(s, q, k, GOOD, GOOD, GOOD, None, GOOD, GOOD, GOOD)
        assert e.value.status == 1
        return str(e.value)

    assert "not on a CUDA device" in refused()
    assert "bfloat16" in refused(q=q.float())
    assert "shape" in refused(q=q[:299])
    assert "strides" in refused(q=torch.zeros(300, 4, 128, dtype=bf)[..., ::2])
    assert "strides" in refused(q=torch.zeros(4, 300, 64, dtype=bf).transpose(0, 1))


def test_reference_gradients_against_differences():
    torch.manual_seed(0)
    q, k, v, d_o = (torch.randn(14, h, 4, dtype=torch.float64) for h in (2, 1, 1, 2))
    seqs = [(0, 5, 0, 5), (5, 3, 5, 6), (8, 6, 11, 3)]
    r, _, _, _ = ref.attention(q, k, v, seqs, 0.7, d_o)
    for name, x in (("q", q), ("k", k), ("v", v)):
        dirn, vals = torch.randn_like(x), []
        for e in (1e-5, -1e-5):
            a = {"q": q, "k": k, "v": v}
            a[name] = x + e * dirn
            vals.append(float((ref.attention(a["q"], a["k"], a["v"], seqs, 0.7)[0]["o"] *
                               d_o).sum()))
        assert math.isclose((vals[0] - vals[1]) / 2e-5, float((r["d" + name] * dirn).sum()),
                            rel_tol=1e-6, abs_tol=1e-7)


def test_reference_decay_is_the_recurrence_and_its_gradients():
    torch.manual_seed(1)
    T, H, d = 13, 3, 4
    q, k, v, d_o = (torch.randn(T, H, d, dtype=torch.float64) for _ in range(4))
    g = torch.tensor([0.0, -0.3, -math.inf], dtype=torch.float64)
    seqs = [(1, 7), (8, 0), (8, 4)]
    s0, s1 = (torch.randn(3, H, d, d, dtype=torch.float64) for _ in range(2))
    r, _ = ref.decay(q, k, v, g, seqs, 0.5, s0, d_o, s1)
    for i, (row, n) in enumerate(seqs):
        for h in range(H):
            S = s0[i, h]
            for t in range(row, row + n):
                S = math.exp(g[h]) * S + torch.outer(k[t, h], v[t, h])
                assert torch.allclose(r["o"][t, h], 0.5 * q[t, h] @ S)
            assert torch.allclose(r["state"][i, h], S)
    for name, x, grad in (("q", q, "dq"), ("k", k, "dk"), ("v", v, "dv"), ("s", s0, "d_state")):
        dirn, vals = torch.randn_like(x), []
        for e in (1e-5, -1e-5):
            a = {"q": q, "k": k, "v": v, "s": s0}
            a[name] = x + e * dirn
            out, _ = ref.decay(a["q"], a["k"], a["v"], g, seqs, 0.5, a["s"])
            vals.append(float((out["o"] * d_o).sum() + (out["state"] * s1).sum()))
        assert math.isclose((vals[0] - vals[1]) / 2e-5, float((r[grad] * dirn).sum()),
                            rel_tol=1e-6, abs_tol=1e-7)
