"""Packed causal softmax attention with grouped heads on the GPU, against the
definition in 64 bits (causal_reference.py has the tolerances)."""

import math

import pytest
import torch

import causal_reference as ref
import sparse_linear_attention_block_b200 as slab

pytestmark = pytest.mark.gpu


def offsets(lengths, start=0):
    off = [start]
    for n in lengths:
        off.append(off[-1] + n)
    return off


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rand(g, *shape, gain=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * gain).to(torch.bfloat16)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


LAYOUTS = ("rows", "fused", "heads")


def tensors(g, layout, tq, tk, Hq, Hkv, d, gain=2.0):
    """q, k, v in one of the layouts that strides allow."""
    if layout == "fused" and tq == tk:  # slices of one projection, with a margin
        x = rand(g, tq, Hq + 2 * Hkv + 1, d)
        x[:, :Hq] *= gain
        return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:Hq + 2 * Hkv]
    if layout == "heads":
        return tuple(rand(g, h, n, d, gain=f).transpose(0, 1)
                     for h, n, f in ((Hq, tq, gain), (Hkv, tk, 1.0), (Hkv, tk, 1.0)))
    return rand(g, tq, Hq, d, gain=gain), rand(g, tk, Hkv, d), rand(g, tk, Hkv, d)


class Case:
    def __init__(self, lq, lk=None, Hq=2, Hkv=1, d=64, layout="rows", seed=0, lead=0, tail=0,
                 cap=0, max_q=0, scale=0.0, gain=2.0, backward=False):
        lk = lq if lk is None else lk
        g = gen(seed)
        self.lq, self.lk = lq, lk
        qo = offsets(lq, lead)
        tq = qo[-1] + tail
        if cap:
            ko, tk = [cap * i for i in range(len(lk))], cap * len(lk)
            self.k_len = i32(lk)
        else:
            ko, self.k_len = offsets(lk, lead), None
            tk = ko[-1] + tail
        tq, tk = max(tq, 1), max(tk, 1)
        self.q_off, self.k_off = i32(qo), i32(ko)
        self.seqs = [(qo[i], lq[i], ko[i], lk[i]) for i in range(len(lq))]
        self.q, self.k, self.v = tensors(g, layout, tq, tk, Hq, Hkv, d, gain)
        self.d_o = rand(g, tq, Hq, d)
        self.scale = scale or d ** -0.5
        self.shape = slab.make_causal_shape(len(lq), tq, tk, Hq, Hkv, d, max_q=max_q, scale=scale,
                                            q=self.q, k=self.k, v=self.v)
        self.buf = slab.CausalBuffers.allocate(self.shape, backward=backward)
        b = self.buf
        for t in (b.o, b.lse, b.dq, b.dk, b.dv):
            if t is not None:
                t.fill_(77.0)

    def forward(self):
        b = self.buf
        slab.sla_causal_forward(self.shape, self.q, self.k, self.v, self.q_off, self.k_off,
                                self.k_len, b.o, b.lse, b.workspace)

    def backward(self):
        b = self.buf
        slab.sla_causal_backward(self.shape, self.q, self.k, self.v, self.q_off, self.k_off, b.o,
                                 b.lse, self.d_o, b.dq, b.dk, b.dv, b.workspace)

    def check(self, backward=False):
        b = self.buf
        slab.sla_check(b.workspace)
        r, t, uq, uk = ref.attention(self.q, self.k, self.v, self.seqs, self.scale,
                                     self.d_o if backward else None)
        ref.check("o", b.o[uq], r["o"][uq], t["o"][uq], ref.U)
        ref.check("lse", b.lse[:, uq], r["lse"][:, uq], t["lse"][:, uq])
        # rows of no sequence are left as they were
        assert (b.o[~uq] == 77.0).all() and (b.lse[:, ~uq] == 77.0).all()
        if backward:
            for n, x, used in (("dq", b.dq, uq), ("dk", b.dk, uk), ("dv", b.dv, uk)):
                ref.check(n, x[used], r[n][used], t[n][used], r["norms"][n])
                assert (x[~used] == 77.0).all(), n


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lq", [[1], [37], [64], [127, 128, 129], [1, 0, 1, 5, 0, 63, 65],
                                [255, 256, 257], [300, 1, 513, 33], [1000]], ids=str)
def test_prompts(lq, d):
    c = Case(lq, Hq=4, Hkv=2, d=d, lead=3, tail=5, seed=len(lq))
    c.forward()
    c.check()


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (3, 3), (6, 2), (8, 2), (16, 1), (5, 5)])
def test_grouped_heads(Hq, Hkv):
    c = Case([200, 70, 131], Hq=Hq, Hkv=Hkv, d=128, seed=Hq, backward=True)
    c.forward()
    c.backward()
    c.check(backward=True)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("d", [64, 128])
def test_layouts(layout, d):
    c = Case([140, 3, 260], Hq=4, Hkv=2, d=d, layout=layout, lead=2, tail=9, seed=5, backward=True)
    assert c.buf.dq.stride() == c.q.stride() and c.buf.dk.stride() == c.k.stride()
    c.forward()
    c.backward()
    c.check(backward=True)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lq,lk", [
    ([1], [1]), ([1, 1, 1], [5, 129, 1000]), ([3, 1, 7], [700, 64, 7]), ([130], [390]),
    ([40, 64, 200], [41, 640, 201]),
    ([5, 200, 9], [2, 90, 0]),       # rows that see nothing, a sequence without keys
    ([0, 4], [10, 20]),              # keys that nobody sees
], ids=str)
def test_continued_and_empty_rows(lq, lk, d):
    c = Case(lq, lk, Hq=6, Hkv=2, d=d, lead=1, tail=4, seed=3, backward=True)
    c.forward()
    c.backward()
    c.check(backward=True)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (8, 2), (16, 1), (12, 4)])
@pytest.mark.parametrize("nq", [1, 2, 5, 16])
def test_tokens_against_caches(nq, Hq, Hkv, d):
    lk = [n for n in (nq, 17, 64, 65, 300, 1023, 1024) if n >= nq]
    c = Case([nq] * len(lk), lk, Hq=Hq, Hkv=Hkv, d=d, cap=1024, max_q=nq, seed=nq)
    for i, n in enumerate(lk):  # what lies behind a cache's length does not matter
        c.k[i * 1024 + n:(i + 1) * 1024] = math.nan
        c.v[i * 1024 + n:(i + 1) * 1024] = math.inf
    c.forward()
    c.check()


def test_one_long_cache():
    c = Case([1], [20000], Hq=4, Hkv=1, d=128, max_q=1, seed=1)
    c.forward()
    c.check()


def test_sequences_may_share_keys():
    c = Case([2, 2, 1], [300, 300, 200], Hq=4, Hkv=2, d=64, cap=512, max_q=2, seed=2)
    c.k_off.zero_()
    c.seqs = [(q0, n, 0, k) for q0, n, _, k in c.seqs]
    c.forward()
    c.check()


@pytest.mark.parametrize("d", [64, 128])
def test_foreign_rows_do_not_matter(d):
    """NaN and infinities in the rows around and between sequences."""
    c = Case([100, 30, 190], Hq=4, Hkv=2, d=d, lead=40, tail=40, seed=9, backward=True)
    c.seqs = [s for i, s in enumerate(c.seqs) if i != 1]
    for x, y in ((c.q, math.nan), (c.k, math.nan), (c.v, math.inf), (c.d_o, -math.inf)):
        x[:40] = y
        x[-40:] = y
    c.forward()
    c.backward()
    b = c.buf
    r, t, uq, uk = ref.attention(c.q, c.k, c.v, c.seqs, c.scale, c.d_o)
    ref.check("o", b.o[uq], r["o"][uq], t["o"][uq], ref.U)
    for n, x, used in (("dq", b.dq, uq), ("dk", b.dk, uk), ("dv", b.dv, uk)):
        ref.check(n, x[used], r[n][used], t[n][used], r["norms"][n])
    # the sequence in the middle again with its neighbours' values spoilt
    keep = b.o[140:170].clone(), b.dk[140:170].clone()
    for x, y in ((c.q, math.nan), (c.k, math.nan), (c.v, math.inf), (c.d_o, -math.inf)):
        x[:140] = y
        x[170:] = y
    c.forward()
    c.backward()
    assert torch.equal(b.o[140:170], keep[0]) and torch.equal(b.dk[140:170], keep[1])


@pytest.mark.parametrize("gain", [0.0, 40.0])
def test_flat_and_steep_rows(gain):
    """All scores equal, and scores of several hundred."""
    c = Case([260, 61], Hq=2, Hkv=1, d=64, gain=gain, seed=11, backward=True)
    c.forward()
    c.backward()
    # a score of s is off by 64 2^-23 scale sum|q k| < 2^-6 here (sum|q k| < 64 * 40 * 16): its
    # weight by as much, which replaces the 2^-10 of the ordinary bound
    b, r = c.buf, ref.attention(c.q, c.k, c.v, c.seqs, c.scale, c.d_o)
    f = 1.0 if gain == 0.0 else 8.0
    for n, x in (("o", b.o), ("dq", b.dq), ("dk", b.dk), ("dv", b.dv)):
        ref.check(n, x, r[0][n], f * r[1][n])
    ref.check("lse", b.lse, r[0]["lse"], r[1]["lse"])


def test_rising_scores():
    """Every key scores higher than all before it, so the running maximum moves all the time."""
    c = Case([600], Hq=1, Hkv=1, d=64, seed=4)
    c.k[:, 0, 0] = torch.arange(600, device="cuda").to(torch.bfloat16) / 4
    c.q[:, 0, 0] = 4.0
    c.forward()
    c.check()


@pytest.mark.parametrize("n", [1, 31, 32, 33, 200])
def test_many_sequences(n):
    """A CTA finds its tile by itself among up to 32 sequences, from a list beyond."""
    lq = [(i * 37) % 150 for i in range(n)]
    lk = [a + (i * 11) % 90 for i, a in enumerate(lq)]
    c = Case(lq, lk, Hq=2, Hkv=1, d=64, seed=n, lead=2, tail=3, backward=True)
    c.forward()
    c.backward()
    c.check(backward=True)


@pytest.mark.parametrize("lq", [[1, 1, 1], [2, 3, 2], [1, 2, 1, 5]], ids=str)
def test_gradients_of_very_short_sequences(lq):
    """Rows whose weight lies on one or two keys: the slopes nearly cancel.  A row that sees one key
    has no slope: D and dP agree to fp32 there (d 2^-23 sum|do v| scale |k| at most), where a D
    from the rounded output would leave 2^-9 of it."""
    c = Case(lq, Hq=2, Hkv=1, d=64, seed=18, backward=True)
    c.forward()
    c.backward()
    slab.sla_check(c.buf.workspace)
    r, _, _, _ = ref.attention(c.q, c.k, c.v, c.seqs, c.scale, c.d_o)
    first = [s[0] for s in c.seqs]
    for h in range(2):
        mass = (c.d_o[first, h].double().abs() * c.v[first, 0].double().abs()).sum(1, keepdim=True)
        limit = 4 * 64 * 2.0 ** -23 * mass * c.scale * c.k[first, 0].double().abs()
        assert (c.buf.dq[first, h].double().abs() <= limit + 2.0 ** -120).all()
    # the rest as a whole: the rounding of dq itself, and of dS for dk, a root mean square of
    # u / sqrt(3) each
    for n, x in (("dq", c.buf.dq), ("dk", c.buf.dk)):
        if float(r[n].norm()) > 1e-6:
            assert float((x.double() - r[n]).norm() / r[n].norm()) <= ref.U, n


def test_own_scale_and_max_q():
    c = Case([77, 130], Hq=2, Hkv=2, d=128, scale=0.03, max_q=130, seed=6)
    c.forward()
    c.check()


def test_bad_offsets_are_skipped_and_reported():
    c = Case([60, 50, 40], Hq=2, Hkv=1, d=64, seed=8, tail=10)
    good = c.q_off.clone()
    for bad in ([0, 60, 50, 150], [0, 60, 110, 10 ** 9], [-5, 60, 110, 150]):
        c.q_off.copy_(i32(bad))
        c.buf.o.fill_(77.0)
        c.buf.lse.fill_(77.0)
        c.forward()
        with pytest.raises(slab.SlaError) as e:
            slab.sla_check(c.buf.workspace)
        assert e.value.status == 6
    c.q_off.copy_(good)
    c.shape.max_q = 55  # shorter than the first sequence
    c.buf.o.fill_(77.0)
    c.buf.lse.fill_(77.0)
    c.forward()
    with pytest.raises(slab.SlaError):
        slab.sla_check(c.buf.workspace)
    assert (c.buf.o[:60] == 77.0).all()
    c.seqs = c.seqs[1:]
    c.check()


@pytest.mark.parametrize("n", [3, 40])
def test_offsets_that_fall_back_stay_in_bounds(n):
    """Every second sequence falls back to row 0, so the rest overlap and ask for more tiles than
    there are rows: what is written is written within the tensors, and it is reported."""
    c = Case([400] + [0] * (n - 1), Hq=2, Hkv=1, d=64, seed=8, tail=8, backward=True)
    bad = [0 if i % 2 == 0 else 400 for i in range(n + 1)]
    c.q_off.copy_(i32(bad))
    c.k_off.copy_(i32(bad))
    c.forward()
    c.backward()
    with pytest.raises(slab.SlaError) as e:
        slab.sla_check(c.buf.workspace)
    assert e.value.status == 6
    assert (c.buf.o[400:] == 77.0).all() and (c.buf.dk[400:] == 77.0).all()


def test_equal_inputs_give_equal_bits():
    c = Case([700, 129, 400], Hq=6, Hkv=2, d=128, seed=10, backward=True)
    c.forward()
    c.backward()
    b = c.buf
    first = [x.clone() for x in (b.o, b.lse, b.dq, b.dk, b.dv)]
    for _ in range(3):
        c.forward()
        c.backward()
        assert all(torch.equal(x, y) for x, y in zip(first, (b.o, b.lse, b.dq, b.dk, b.dv)))


def test_captured_and_replayed_with_other_lengths():
    c = Case([300, 40, 1], Hq=4, Hkv=2, d=128, seed=12, backward=True)
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.forward()
        c.backward()
    lengths = [41, 0, 299]
    off = offsets(lengths)
    c.q_off.copy_(i32(off))
    c.k_off.copy_(i32(off))
    c.seqs = [(off[i], n, off[i], n) for i, n in enumerate(lengths)]
    for t in (c.buf.o, c.buf.lse, c.buf.dq, c.buf.dk, c.buf.dv):
        t.fill_(77.0)
    graph.replay()
    c.check(backward=True)


def test_captured_tokens_replayed_with_longer_caches():
    """A token step captured once and replayed as the caches grow."""
    c = Case([1, 1, 1], [5, 100, 64], Hq=8, Hkv=2, d=128, cap=512, max_q=1, seed=13)
    c.forward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.forward()
    for lk in ([6, 101, 65], [512, 0, 300]):
        c.k_len.copy_(i32(lk))
        c.seqs = [(i, 1, 512 * i, n) for i, n in enumerate(lk)]
        c.buf.o.fill_(77.0)
        graph.replay()
        c.check()


def test_streams_given_by_the_caller():
    c = Case([200, 31], Hq=4, Hkv=2, d=64, seed=14)
    side = torch.cuda.Stream()
    b = c.buf
    for stream in (side, side.cuda_stream):
        b.o.fill_(77.0)
        side.wait_stream(torch.cuda.current_stream())
        slab.sla_causal_forward(c.shape, c.q, c.k, c.v, c.q_off, c.k_off, None, b.o, b.lse,
                                b.workspace, stream=stream)
        slab.sla_check(b.workspace, stream)
        c.check()


def test_shapes_follow_their_fields():
    """A shape that is changed after a call is checked and used as it is now."""
    c = Case([60, 20], Hq=2, Hkv=1, d=64, seed=15)
    c.forward()
    c.shape.softmax_scale = 0.05
    c.scale = 0.05
    c.forward()
    c.check()
    c.shape.total_q = 79
    with pytest.raises(slab.SlaError):
        c.forward()


def test_a_mixed_batch_of_prompts_and_tokens():
    """What a server runs in one call: whole prompts, a prompt that continues, generated tokens."""
    lq, lk = [150, 1, 1, 40, 1], [150, 700, 33, 300, 1]
    for max_q in (0, 150):
        c = Case(lq, lk, Hq=8, Hkv=2, d=128, cap=704, max_q=max_q, seed=16)
        c.forward()
        c.check()


def test_lengths_that_pass_the_work_lists_buckets():
    """A long key range in few rows: costs of more than 2048 tiles share buckets in the list."""
    n = 40
    lq, lk = [70] + [3] * (n - 1), [300000] + [50] * (n - 1)
    c = Case(lq, lk, Hq=1, Hkv=1, d=64, seed=17)
    c.forward()
    c.check()


def test_two_streams_at_once():
    cases = [Case([900, 300], Hq=4, Hkv=2, d=128, seed=20 + i, backward=True) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                c.forward()
                c.backward()
    torch.cuda.synchronize()
    for c in cases:
        c.check(backward=True)


def test_gradients_against_differences():
    """d/de of sum(o * d_o) along random directions, from the 64-bit forward."""
    c = Case([90, 41], Hq=4, Hkv=2, d=64, seed=30, backward=True)
    c.forward()
    c.backward()
    g = gen(31)
    for name, x, grad in (("q", c.q, c.buf.dq), ("k", c.k, c.buf.dk), ("v", c.v, c.buf.dv)):
        dirn = torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float64)
        eps, vals = 1e-4, []
        for sgn in (1, -1):
            args = {n: getattr(c, n).double() for n in "qkv"}
            args[name] = args[name] + sgn * eps * dirn
            o = ref.attention(args["q"], args["k"], args["v"], c.seqs, c.scale)[0]["o"]
            vals.append(float((o * c.d_o.double()).sum()))
        num = (vals[0] - vals[1]) / (2 * eps)
        got = float((grad.double() * dirn).sum())
        # the gradient's 2-norm error is at most U of its norm; along a direction the
        # independent roundings add up as a random walk, 6 standard deviations of the tensor's bound
        norm = ref.attention(c.q, c.k, c.v, c.seqs, c.scale, c.d_o)[0]["norms"]["d" + name]
        assert abs(got - num) <= 6 * norm * float(grad.double().norm()) + 1e-5, name


def test_a_large_tensor_beyond_32_bit_offsets():
    """Row offsets times strides past 2^31 elements: two sequences at both ends of a wide tensor."""
    rows, width = 70000, 32768
    x = torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda")  # 4.6 GB
    g = gen(40)
    d, H = 128, 2
    view = lambda c: x[:, c:c + H * d].unflatten(1, (H, d))
    q, k, v, o = (view(i * 1024) for i in range(4))
    for t in (q, k, v):
        t[:200] = rand(g, 200, H, d)
        t[-200:] = rand(g, 200, H, d)
    shape = slab.make_causal_shape(3, rows, rows, H, H, d, q=q, k=k, v=v, o=o)
    buf = slab.CausalBuffers.allocate(slab.make_causal_shape(3, rows, rows, H, H, d))
    q_off = i32([0, 150, rows - 170, rows])
    k_off = i32([0, 150, rows - 170, rows])
    k_len = i32([150, 0, 170])  # the sequence in the middle sees nothing
    slab.sla_causal_forward(shape, q, k, v, q_off, k_off, k_len, o, buf.lse, buf.workspace)
    slab.sla_check(buf.workspace)
    seqs = [(0, 150, 0, 150), (rows - 170, 170, rows - 170, 170)]
    for q0, n, _, _ in seqs:
        sl = slice(q0, q0 + n)
        r, t, _, _ = ref.attention(q[sl], k[sl], v[sl], [(0, n, 0, n)], d ** -0.5)
        ref.check("o", o[sl], r["o"], t["o"], ref.U)
