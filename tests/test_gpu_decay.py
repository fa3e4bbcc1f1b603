"""Linear attention with a decay for each head on the GPU, against the
definition in 64 bits (causal_reference.py has the tolerances)."""

import math

import pytest
import torch

import causal_reference as ref
import sparse_linear_attention_block_b200 as slab
from test_gpu_causal import gen, i32, offsets, rand

pytestmark = pytest.mark.gpu

DECAYS = [0.0, -1e-4, -0.02, -0.7, -9.0, -math.inf]


class Case:
    def __init__(self, lengths, H=3, d=64, start=True, end=True, layout="rows", seed=0, lead=0,
                 tail=0, log_decay=None, backward=False, scale=0.0):
        g = gen(seed)
        off = offsets(lengths, lead)
        T = max(1, off[-1] + tail)
        n = len(lengths)
        self.seqs = [(off[i], lengths[i]) for i in range(n)]
        self.off = i32(off)
        if layout == "fused":
            x = rand(g, T, 3 * H + 1, d)
            self.q, self.k, self.v = x[:, :H], x[:, H:2 * H], x[:, 2 * H:3 * H]
        elif layout == "heads":
            self.q, self.k, self.v = (rand(g, H, T, d).transpose(0, 1) for _ in range(3))
        else:
            self.q, self.k, self.v = (rand(g, T, H, d) for _ in range(3))
        self.d_o = rand(g, T, H, d)
        some = lambda: torch.randn(n, H, d, d, generator=g, device="cuda")
        self.s0 = some() if start else None
        self.s1 = some() if end else None
        if log_decay is None:
            log_decay = [DECAYS[(h + seed) % len(DECAYS)] for h in range(H)]
        self.g = torch.tensor(log_decay, dtype=torch.float32, device="cuda")
        self.scale = scale or d ** -0.5
        self.shape = slab.make_decay_shape(n, T, H, d, scale=scale, q=self.q, k=self.k, v=self.v)
        self.buf = slab.DecayBuffers.allocate(self.shape, backward=backward)
        b = self.buf
        self.used = torch.zeros(T, dtype=torch.bool, device="cuda")
        for a, m in self.seqs:
            self.used[a:a + m] = True
        for t in (b.o, b.state, b.dq, b.dk, b.dv, b.d_state):
            if t is not None:
                t.fill_(77.0)

    def forward(self):
        b = self.buf
        slab.sla_decay_forward(self.shape, self.q, self.k, self.v, self.g, self.off, self.s0, b.o,
                               b.state, b.workspace)

    def backward(self):
        b = self.buf
        slab.sla_decay_backward(self.shape, self.q, self.k, self.v, self.g, self.off, self.s0,
                                self.d_o, self.s1, b.dq, b.dk, b.dv, b.d_state, b.workspace)

    def check(self, backward=False, norm=ref.U):
        b = self.buf
        slab.sla_check(b.workspace)
        r, t = ref.decay(self.q, self.k, self.v, self.g, self.seqs, self.scale, self.s0,
                         self.d_o if backward else None, self.s1)
        names = (("o", b.o),) + ((("dq", b.dq), ("dk", b.dk), ("dv", b.dv)) if backward else ())
        for n, x in names:
            ref.check(n, x[self.used], r[n][self.used], t[n][self.used], norm)
            assert (x[~self.used] == 77.0).all(), n
        ref.check("state", b.state, r["state"], t["state"], 2.0 ** -18)
        if backward:
            ref.check("d_state", b.d_state, r["d_state"], t["d_state"], 2.0 ** -18)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths", [[1], [2], [63, 64, 65], [127, 128, 129], [1, 0, 5, 0],
                                     [300, 1, 513], [1500]], ids=str)
def test_prompts(lengths, d):
    for start in (False, True):
        c = Case(lengths, H=6, d=d, start=start, lead=3, tail=4, seed=len(lengths))
        c.forward()
        c.check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths", [[1], [2, 1, 0], [64, 128], [63, 129, 200], [700]], ids=str)
@pytest.mark.parametrize("start,end", [(True, True), (False, False), (False, True)])
def test_training(lengths, start, end, d):
    c = Case(lengths, H=6, d=d, start=start, end=end, lead=2, tail=3, seed=7, backward=True)
    c.forward()
    c.backward()
    c.check(backward=True)


@pytest.mark.parametrize("layout", ["rows", "fused", "heads"])
@pytest.mark.parametrize("d", [64, 128])
def test_layouts(layout, d):
    c = Case([140, 3, 260], H=4, d=d, layout=layout, lead=2, tail=9, seed=5, backward=True)
    c.forward()
    c.backward()
    c.check(backward=True)


def test_long_prompts_of_few_heads():
    """Few (sequence, head) pairs and many tokens: the work along a sequence is split."""
    c = Case([5000, 2500], H=2, d=128, seed=3, log_decay=[-1e-4, -0.01], backward=True)
    c.forward()
    c.backward()
    # 5000 tokens are 313 steps of 16 tokens: 313 2^-23 is below the 2^-14 used for the states here
    b = c.buf
    slab.sla_check(b.workspace)
    r, t = ref.decay(c.q, c.k, c.v, c.g, c.seqs, c.scale, c.s0, c.d_o, c.s1)
    for n in ("o", "dq", "dk", "dv"):
        ref.check(n, getattr(b, n), r[n], t[n], ref.U)
    ref.check("state", b.state, r["state"], 4 * t["state"], 2.0 ** -17)
    ref.check("d_state", b.d_state, r["d_state"], 4 * t["d_state"], 2.0 ** -17)


@pytest.mark.parametrize("n", [1, 32, 33, 150])
def test_many_sequences(n):
    """A CTA finds its piece by itself among up to 32 sequences, from a list beyond; some of the
    sequences are cut."""
    lengths = [(i * 53) % 90 for i in range(n)]
    lengths[n // 2] = 1300
    lengths[-1] = 700
    c = Case(lengths, H=2, d=64, seed=n, log_decay=[-0.003, -0.2], lead=1, tail=2, backward=True)
    c.forward()
    c.backward()
    c.check(backward=True)


@pytest.mark.parametrize("n", [3, 40])
def test_offsets_that_fall_back_stay_in_bounds(n):
    c = Case([1500] + [0] * (n - 1), H=2, d=64, seed=8, tail=8, log_decay=[-0.1, -0.2],
             backward=True)
    c.off.copy_(i32([0 if i % 2 == 0 else 1500 for i in range(n + 1)]))
    c.forward()
    c.backward()
    with pytest.raises(slab.SlaError) as e:
        slab.sla_check(c.buf.workspace)
    assert e.value.status == 6
    assert (c.buf.o[1500:] == 77.0).all() and (c.buf.dk[1500:] == 77.0).all()


def test_state_in_place_and_in_two_parts():
    """A prompt in two calls through one state buffer gives what one call gives."""
    c = Case([400, 90], H=2, d=64, seed=9, log_decay=[-0.01, -0.3])
    c.forward()
    whole = c.buf.state.clone()
    state = c.s0.clone()
    o = torch.full_like(c.buf.o, 77.0)
    first = i32([0, 250, 250])            # the first 250 tokens of sequence 0, none of sequence 1
    slab.sla_decay_forward(c.shape, c.q, c.k, c.v, c.g, first, state, o, state, c.buf.workspace)
    rest = i32([250, 400, 490])
    slab.sla_decay_forward(c.shape, c.q, c.k, c.v, c.g, rest, state, o, state, c.buf.workspace)
    slab.sla_check(c.buf.workspace)
    r, t = ref.decay(c.q, c.k, c.v, c.g, c.seqs, c.scale, c.s0)
    ref.check("o", o, r["o"], t["o"], ref.U)
    ref.check("state", state, r["state"], t["state"], 2.0 ** -18)
    ref.check("whole", whole, r["state"], t["state"], 2.0 ** -18)


def test_state_gradient_in_place():
    c = Case([130, 64], H=2, d=64, seed=10, backward=True)
    c.forward()
    given = c.s1.clone()
    b = c.buf
    c.backward()
    expected = [x.clone() for x in (b.dq, b.dk, b.dv, b.d_state)]
    slab.sla_decay_backward(c.shape, c.q, c.k, c.v, c.g, c.off, c.s0, c.d_o, given, b.dq, b.dk,
                            b.dv, given, b.workspace)
    for x, y in zip(expected, (b.dq, b.dk, b.dv, given)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,H", [(1, 1), (1, 12), (7, 3), (64, 5)])
def test_tokens(n, H, d):
    g = gen(n)
    q, k, v = (rand(g, n, H, d) for _ in range(3))
    s0 = torch.randn(n, H, d, d, generator=g, device="cuda")
    ld = torch.tensor([DECAYS[h % len(DECAYS)] for h in range(H)], device="cuda")
    shape = slab.make_decay_shape(n, n, H, d)
    o, s1 = torch.empty_like(q), torch.empty_like(s0)
    slab.sla_decay_step(shape, q, k, v, ld, s0, s1, o)
    r, t = ref.decay(q, k, v, ld, [(i, 1) for i in range(n)], d ** -0.5, s0)
    # nothing but the output is rounded to bf16 here; the state takes three 32-bit roundings
    ref.check("o", o, r["o"], ref.U * r["o"].abs() + 2.0 ** -16 * t["o"] / ref.U)
    ref.check("state", s1, r["state"], t["state"], 2.0 ** -21)
    again = s0.clone()
    slab.sla_decay_step(shape, q, k, v, ld, again, again, o)
    assert torch.equal(again, s1)


def test_tokens_of_strided_rows():
    g = gen(3)
    x = rand(g, 9, 3 * 4 + 2, 64)
    q, k, v = x[:, :4], x[:, 4:8], x[:, 8:12]
    s0 = torch.randn(9, 4, 64, 64, generator=g, device="cuda")
    ld = torch.tensor([-0.1, -0.2, -0.3, 0.0], device="cuda")
    shape = slab.make_decay_shape(9, 9, 4, 64, q=q, k=k, v=v)
    o, s1 = torch.empty(9, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.empty_like(s0)
    slab.sla_decay_step(shape, q, k, v, ld, s0, s1, o)
    r, t = ref.decay(q, k, v, ld, [(i, 1) for i in range(9)], 64 ** -0.5, s0)
    ref.check("o", o, r["o"], t["o"])
    ref.check("state", s1, r["state"], t["state"], 2.0 ** -21)


def test_prompt_then_tokens():
    """As a server uses them: the prompts in one call, then one token at a time, equal to the
    prompts with the tokens behind them."""
    H, d, lengths, more = 3, 64, [70, 1, 129], 4
    g = gen(21)
    T = sum(lengths) + more * len(lengths)
    q, k, v = (rand(g, T, H, d) for _ in range(3))
    ld = torch.tensor([-0.01, -0.2, 0.0], device="cuda")
    prompt, tokens, row = [], [], 0
    for n in lengths:
        prompt += range(row, row + n)
        tokens.append(range(row + n, row + n + more))
        row += n + more
    P = torch.tensor(prompt, device="cuda")
    shape = slab.make_decay_shape(3, len(prompt), H, d)
    buf = slab.DecayBuffers.allocate(shape)
    slab.sla_decay_forward(shape, q[P], k[P], v[P], ld, i32(offsets(lengths)), None, buf.o,
                           buf.state, buf.workspace)
    got = torch.empty_like(q)
    got[P] = buf.o
    one = slab.make_decay_shape(3, 3, H, d)
    o = torch.empty(3, H, d, dtype=torch.bfloat16, device="cuda")
    for j in range(more):
        at = torch.tensor([t[j] for t in tokens], device="cuda")
        slab.sla_decay_step(one, q[at], k[at], v[at], ld, buf.state, buf.state, o)
        got[at] = o
    slab.sla_check(buf.workspace)
    off = offsets([n + more for n in lengths])
    seqs = [(off[i], lengths[i] + more) for i in range(3)]
    r, t = ref.decay(q, k, v, ld, seqs, d ** -0.5)
    ref.check("o", got, r["o"], t["o"], ref.U)
    ref.check("state", buf.state, r["state"], t["state"], 2.0 ** -18)


def test_bad_decays_and_offsets_are_reported():
    c = Case([100, 50], H=2, d=64, seed=1, log_decay=[0.5, -0.1])
    c.forward()
    with pytest.raises(slab.SlaError) as e:
        slab.sla_check(c.buf.workspace)
    assert e.value.status == 6
    c.g.copy_(torch.tensor([0.0, -0.1]))  # what the bad value is taken as
    c.check()
    c.off.copy_(i32([0, 100, 90]))
    c.buf.state.fill_(77.0)
    c.forward()
    with pytest.raises(slab.SlaError):
        slab.sla_check(c.buf.workspace)
    assert (c.buf.state[1] == 77.0).all()


def test_foreign_rows_do_not_matter():
    c = Case([100, 190], H=2, d=128, lead=40, tail=40, seed=9, log_decay=[-0.01, 0.0],
             backward=True)
    for x, y in ((c.q, math.nan), (c.k, math.nan), (c.v, math.inf), (c.d_o, -math.inf)):
        x[:40] = y
        x[-40:] = y
    c.forward()
    c.backward()
    c.check(backward=True)
    b = c.buf
    keep = [x[40:140].clone() for x in (b.o, b.dq, b.dk, b.dv)]
    for x, y in ((c.q, math.nan), (c.k, math.nan), (c.v, math.inf), (c.d_o, -math.inf)):
        x[140:] = y
    c.forward()
    c.backward()
    for x, y in zip(keep, (b.o, b.dq, b.dk, b.dv)):
        assert torch.equal(x, y[40:140])


def test_equal_inputs_give_equal_bits():
    c = Case([3000, 129], H=2, d=128, seed=10, log_decay=[-0.01, -0.3], backward=True)
    c.forward()
    c.backward()
    b = c.buf
    first = [x.clone() for x in (b.o, b.state, b.dq, b.dk, b.dv, b.d_state)]
    for _ in range(3):
        c.forward()
        c.backward()
        assert all(torch.equal(x, y)
                   for x, y in zip(first, (b.o, b.state, b.dq, b.dk, b.dv, b.d_state)))


def test_captured_and_replayed_with_other_lengths():
    c = Case([300, 40, 1], H=2, d=64, seed=12, backward=True)
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.forward()
        c.backward()
    lengths = [41, 0, 299]
    off = offsets(lengths)
    c.off.copy_(i32(off))
    c.seqs = [(off[i], n) for i, n in enumerate(lengths)]
    c.used.zero_()
    c.used[:340] = True
    for t in (c.buf.o, c.buf.dq, c.buf.dk, c.buf.dv):
        t.fill_(77.0)
    graph.replay()
    c.check(backward=True)


def test_gradients_against_differences():
    c = Case([60, 33], H=2, d=64, seed=30, log_decay=[-0.05, -0.4], backward=True)
    c.forward()
    c.backward()
    g = gen(31)
    b = c.buf
    for name, grad in (("q", b.dq), ("k", b.dk), ("v", b.dv), ("s0", b.d_state)):
        x = getattr(c, name)
        dirn = torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float64)
        eps, vals = 1e-4, []
        for sgn in (1, -1):
            a = {n: getattr(c, n).double() for n in ("q", "k", "v", "s0")}
            a[name] = a[name] + sgn * eps * dirn
            r, _ = ref.decay(a["q"], a["k"], a["v"], c.g, c.seqs, c.scale, a["s0"])
            vals.append(float((r["o"] * c.d_o.double()).sum() +
                              (r["state"] * c.s1.double()).sum()))
        num = (vals[0] - vals[1]) / (2 * eps)
        got = float((grad.double() * dirn).sum())
        assert abs(got - num) <= 6 * ref.U * float(grad.double().norm()) + 1e-5, name


def test_attention_and_decay_in_one_layer():
    """The two causal branches of one layer share q, k, v and offsets: prompts, then a training
    step on their sum, then a token against the caches that the prompts left."""
    H, d, lengths = 2, 64, [90, 33, 150]
    c = Case(lengths, H=H, d=d, start=False, end=False, seed=40, log_decay=[-0.01, -0.2],
             backward=True)
    sh = slab.make_causal_shape(3, c.q.shape[0], c.k.shape[0], H, H, d)
    ab = slab.CausalBuffers.allocate(sh, backward=True)
    slab.sla_causal_forward(sh, c.q, c.k, c.v, c.off, c.off, None, ab.o, ab.lse, ab.workspace)
    c.forward()
    both = ab.o + c.buf.o
    slab.sla_causal_backward(sh, c.q, c.k, c.v, c.off, c.off, ab.o, ab.lse, c.d_o, ab.dq, ab.dk,
                             ab.dv, ab.workspace)
    c.backward()
    slab.sla_check(ab.workspace)
    c.check(backward=True)
    ra, ta, _, _ = ref.attention(c.q, c.k, c.v, [(a, n, a, n) for a, n in c.seqs], c.scale, c.d_o)
    rd, td = ref.decay(c.q, c.k, c.v, c.g, c.seqs, c.scale, None, c.d_o)
    total = ra["o"] + rd["o"]
    ref.check("sum", both, total, ta["o"] + td["o"] + ref.U * total.abs(), ref.U)
    for n in ("dq", "dk", "dv"):
        got = getattr(ab, n).double() + getattr(c.buf, n).double()
        ref.check(n, got, ra[n] + rd[n], ta[n] + td[n])
