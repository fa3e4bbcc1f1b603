"""Binding of the causal operators of ``include/sla.h``: packed causal softmax
attention with grouped heads and linear attention with a decay for each head.

As with the other entry points the caller owns every buffer and the C library
does the work; the functions here check the tensors against the shape (type,
sizes, strides, one device) and raise :class:`SlaError` before anything is
launched.  They run on the tensors' device, on its current stream unless one is
given.  Plain integers are taken as device pointers of the current device, as they are.

    shape = make_causal_shape(n_seq, total_q, total_k, Hq, Hkv, d)
    buf = CausalBuffers.allocate(shape, backward=True)
    sla_causal_forward(shape, q, k, v, q_off, k_off, None, buf.o, buf.lse, buf.workspace)
    sla_causal_backward(shape, q, k, v, q_off, k_off, buf.o, buf.lse, d_o,
                        buf.dq, buf.dk, buf.dv, buf.workspace)
"""

from __future__ import annotations

import ctypes
import dataclasses

import sparse_linear_attention_block_b200 as _slab

__all__ = ["Strides", "CausalShape", "CausalSizes", "DecayShape", "DecaySizes", "CausalBuffers",
           "DecayBuffers", "make_causal_shape", "make_decay_shape", "sla_causal_query_sizes",
           "sla_causal_forward", "sla_causal_backward", "sla_decay_query_sizes",
           "sla_decay_forward", "sla_decay_backward", "sla_decay_step"]


class Strides(ctypes.Structure):
    """sla_strides: elements from one row, and from one head, to the next."""
    _fields_ = [("row", ctypes.c_int64), ("head", ctypes.c_int64)]


class CausalShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("n_seq", "total_q", "total_k", "Hq", "Hkv", "d",
                                            "max_q")] + [
        ("softmax_scale", ctypes.c_float)] + [(n, Strides) for n in "qkvo"]


class CausalSizes(ctypes.Structure):
    _fields_ = [("lse_bytes", ctypes.c_size_t), ("workspace_bytes", ctypes.c_size_t)]


class DecayShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("n_seq", "total", "H", "d")] + [
        ("scale", ctypes.c_float)] + [(n, Strides) for n in "qkvo"]


class DecaySizes(ctypes.Structure):
    _fields_ = [("state_bytes", ctypes.c_size_t), ("workspace_bytes", ctypes.c_size_t)]


def declare(L):
    """Argument types of the causal entry points of the loaded library."""
    vp, sz, P = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER
    L.sla_causal_query_sizes.argtypes = [P(CausalShape), P(CausalSizes)]
    L.sla_causal_forward.argtypes = [P(CausalShape)] + [vp] * 9 + [sz, vp]
    L.sla_causal_backward.argtypes = [P(CausalShape)] + [vp] * 12 + [sz, vp]
    L.sla_decay_query_sizes.argtypes = [P(DecayShape), P(DecaySizes)]
    L.sla_decay_forward.argtypes = [P(DecayShape)] + [vp] * 9 + [sz, vp]
    L.sla_decay_backward.argtypes = [P(DecayShape)] + [vp] * 13 + [sz, vp]
    L.sla_decay_step.argtypes = [P(DecayShape)] + [vp] * 8
    for n in ("sla_causal_query_sizes", "sla_causal_forward", "sla_causal_backward",
              "sla_decay_query_sizes", "sla_decay_forward", "sla_decay_backward",
              "sla_decay_step"):
        getattr(L, n).restype = ctypes.c_int


def _strides(x) -> Strides:
    """(row, head) strides from None (contiguous), a pair, or a [rows, heads, d] tensor."""
    if x is None:
        return Strides(0, 0)
    if isinstance(x, (tuple, list)):
        return Strides(*x)
    return Strides(x.stride(0), x.stride(1))


def make_causal_shape(n_seq, total_q, total_k, Hq, Hkv, d, max_q=0, scale=0.0, q=None, k=None,
                      v=None, o=None) -> CausalShape:
    """q, k, v, o: strides of the tensors where they are not contiguous, as
    (row, head) pairs or as the tensors themselves."""
    return CausalShape(n_seq, total_q, total_k, Hq, Hkv, d, max_q, float(scale), _strides(q),
                       _strides(k), _strides(v), _strides(o))


def make_decay_shape(n_seq, total, H, d, scale=0.0, q=None, k=None, v=None, o=None) -> DecayShape:
    return DecayShape(n_seq, total, H, d, float(scale), _strides(q), _strides(k), _strides(v),
                      _strides(o))


def sla_causal_query_sizes(shape: CausalShape) -> CausalSizes:
    out = CausalSizes()
    _slab._check(_slab.lib().sla_causal_query_sizes(ctypes.byref(shape), ctypes.byref(out)),
                 "sla_causal_query_sizes")
    return out


def sla_decay_query_sizes(shape: DecayShape) -> DecaySizes:
    out = DecaySizes()
    _slab._check(_slab.lib().sla_decay_query_sizes(ctypes.byref(shape), ctypes.byref(out)),
                 "sla_decay_query_sizes")
    return out


class _Args:
    """Checks the tensors of one call and collects their addresses."""

    def __init__(self, what):
        self.what, self.device = what, None

    def refuse(self, name, why):
        raise _slab.SlaError(1, f"{self.what}: {name} {why}")

    def _on(self, t, name):
        device = t.device
        if device.type != "cuda":
            self.refuse(name, f"is on {device}, not on a CUDA device")
        if self.device is None:
            self.device = device
        elif device != self.device:
            self.refuse(name, f"is on {device}, others on {self.device}")
        return t.data_ptr()

    def rows(self, t, name, rows, heads, d, st):
        """A bf16 [rows, heads, d] tensor with the shape's strides."""
        if isinstance(t, int):
            return t
        import torch
        if t.dtype is not torch.bfloat16:
            self.refuse(name, f"is {t.dtype}, not torch.bfloat16")
        if t.shape != (rows, heads, d):
            self.refuse(name, f"has shape {tuple(t.shape)}, not {(rows, heads, d)}")
        r, h = (st.row, st.head) if st.row or st.head else (heads * d, d)
        a, b, c = t.stride()
        if (a != r and rows > 1) or (b != h and heads > 1) or c != 1:
            self.refuse(name, f"has strides {(a, b, c)}, the shape says {(r, h, 1)}")
        return self._on(t, name)

    def whole(self, t, name, dtype, numel, optional=False):
        """A contiguous tensor of at least `numel` elements."""
        if t is None:
            if not optional:
                self.refuse(name, "is required")
            return None
        if isinstance(t, int):
            return t
        if t.dtype is not dtype:
            self.refuse(name, f"is {t.dtype}, not {dtype}")
        if t.numel() < numel or not t.is_contiguous():
            self.refuse(name, f"is not contiguous with {numel} elements")
        return self._on(t, name)

    def call(self, fn, stream, *args):
        import torch
        if self.device is None:  # plain pointers only
            _slab._check(fn(*args, _slab._stream(stream)), self.what)
            return
        if stream is None:
            raw = torch.cuda.current_stream(self.device).cuda_stream
        else:
            device = getattr(stream, "device", None)
            if device is not None and device != self.device:
                self.refuse("stream", f"is on {device}, the tensors on {self.device}")
            raw = stream if isinstance(stream, int) else stream.cuda_stream
        if torch.cuda.current_device() == self.device.index:
            status = fn(*args, raw)
        else:
            with torch.cuda.device(self.device):
                status = fn(*args, raw)
        _slab._check(status, self.what)


def _qkv(a, s, q, k, v, rows_q, rows_k, Hq, Hkv, names="qkv"):
    return (a.rows(q, names[0], rows_q, Hq, s.d, s.q), a.rows(k, names[1], rows_k, Hkv, s.d, s.k),
            a.rows(v, names[2], rows_k, Hkv, s.d, s.v))


def _workspace(a, ws):
    import torch
    return a.whole(ws, "workspace", torch.uint8, 0), ws.numel()


def sla_causal_forward(shape: CausalShape, q, k, v, q_off, k_off, k_len, o, lse, workspace,
                       stream=None):
    """Causal attention of packed sequences; k_len (or None) as in sla.h."""
    import torch
    s, a = shape, _Args("sla_causal_forward")
    i32 = torch.int32
    ptrs = _qkv(a, s, q, k, v, s.total_q, s.total_k, s.Hq, s.Hkv)
    ptrs += (a.whole(q_off, "q_off", i32, s.n_seq + 1),
             a.whole(k_off, "k_off", i32, s.n_seq + (k_len is None)),
             a.whole(k_len, "k_len", i32, s.n_seq, optional=True),
             a.rows(o, "o", s.total_q, s.Hq, s.d, s.o),
             a.whole(lse, "lse", torch.float32, s.Hq * s.total_q))
    a.call(_slab.lib().sla_causal_forward, stream, ctypes.byref(s), *ptrs,
           *_workspace(a, workspace))


def sla_causal_backward(shape: CausalShape, q, k, v, q_off, k_off, o, lse, d_o, dq, dk, dv,
                        workspace, stream=None):
    """Gradients of sum(o * d_o); dq, dk, dv have the strides of q, k, v."""
    import torch
    s, a = shape, _Args("sla_causal_backward")
    i32 = torch.int32
    ptrs = _qkv(a, s, q, k, v, s.total_q, s.total_k, s.Hq, s.Hkv)
    ptrs += (a.whole(q_off, "q_off", i32, s.n_seq + 1), a.whole(k_off, "k_off", i32, s.n_seq + 1),
             a.rows(o, "o", s.total_q, s.Hq, s.d, s.o),
             a.whole(lse, "lse", torch.float32, s.Hq * s.total_q),
             a.rows(d_o, "d_o", s.total_q, s.Hq, s.d, s.o))
    ptrs += _qkv(a, s, dq, dk, dv, s.total_q, s.total_k, s.Hq, s.Hkv, ("dq", "dk", "dv"))
    a.call(_slab.lib().sla_causal_backward, stream, ctypes.byref(s), *ptrs,
           *_workspace(a, workspace))


def sla_decay_forward(shape: DecayShape, q, k, v, log_decay, off, state_in, o, state_out,
                      workspace, stream=None):
    """Decayed linear attention of packed sequences; state_in, state_out may be None."""
    import torch
    s, a = shape, _Args("sla_decay_forward")
    f32, n = torch.float32, s.n_seq * s.H * s.d * s.d
    ptrs = _qkv(a, s, q, k, v, s.total, s.total, s.H, s.H)
    ptrs += (a.whole(log_decay, "log_decay", f32, s.H), a.whole(off, "off", torch.int32,
                                                                s.n_seq + 1),
             a.whole(state_in, "state_in", f32, n, optional=True),
             a.rows(o, "o", s.total, s.H, s.d, s.o),
             a.whole(state_out, "state_out", f32, n, optional=True))
    a.call(_slab.lib().sla_decay_forward, stream, ctypes.byref(s), *ptrs,
           *_workspace(a, workspace))


def sla_decay_backward(shape: DecayShape, q, k, v, log_decay, off, state_in, d_o, d_state_out, dq,
                       dk, dv, d_state_in, workspace, stream=None):
    """Gradients of sum(o * d_o) + sum(state_out * d_state_out); the states and
    their gradients may be None."""
    import torch
    s, a = shape, _Args("sla_decay_backward")
    f32, n = torch.float32, s.n_seq * s.H * s.d * s.d
    ptrs = _qkv(a, s, q, k, v, s.total, s.total, s.H, s.H)
    ptrs += (a.whole(log_decay, "log_decay", f32, s.H), a.whole(off, "off", torch.int32,
                                                                s.n_seq + 1),
             a.whole(state_in, "state_in", f32, n, optional=True),
             a.rows(d_o, "d_o", s.total, s.H, s.d, s.o),
             a.whole(d_state_out, "d_state_out", f32, n, optional=True))
    ptrs += _qkv(a, s, dq, dk, dv, s.total, s.total, s.H, s.H, ("dq", "dk", "dv"))
    ptrs += (a.whole(d_state_in, "d_state_in", f32, n, optional=True),)
    a.call(_slab.lib().sla_decay_backward, stream, ctypes.byref(s), *ptrs,
           *_workspace(a, workspace))


def sla_decay_step(shape: DecayShape, q, k, v, log_decay, state_in, state_out, o, stream=None):
    """One token for each sequence; state_out may be state_in."""
    import torch
    s, a = shape, _Args("sla_decay_step")
    f32, n = torch.float32, s.n_seq * s.H * s.d * s.d
    ptrs = _qkv(a, s, q, k, v, s.total, s.total, s.H, s.H)
    ptrs += (a.whole(log_decay, "log_decay", f32, s.H), a.whole(state_in, "state_in", f32, n),
             a.whole(state_out, "state_out", f32, n), a.rows(o, "o", s.total, s.H, s.d, s.o))
    a.call(_slab.lib().sla_decay_step, stream, ctypes.byref(s), *ptrs)


def _allocate_workspace(nbytes, device, stream):
    """A 1024-byte aligned workspace with a cleared error word."""
    import torch
    ws = torch.empty(int(nbytes) + 1024, dtype=torch.uint8, device=device)
    off = (-ws.data_ptr()) % 1024
    ws = ws[off:off + int(nbytes)]
    with torch.cuda.device(ws.device):
        _slab.sla_workspace_init(ws, stream)
    return ws


def _like(st, rows, heads, d, device):
    """An uninitialised bf16 [rows, heads, d] tensor with the given strides."""
    import torch
    if not (st.row or st.head):
        return torch.empty(rows, heads, d, dtype=torch.bfloat16, device=device)
    size = (rows - 1) * st.row + (heads - 1) * st.head + d
    return torch.empty(size, dtype=torch.bfloat16, device=device).as_strided(
        (rows, heads, d), (st.row, st.head, 1))


@dataclasses.dataclass
class CausalBuffers:
    """Output buffers and the workspace of packed causal attention for one shape;
    the gradients are None unless ``backward``."""
    shape: CausalShape
    o: object
    lse: object
    dq: object
    dk: object
    dv: object
    workspace: object

    @classmethod
    def allocate(cls, shape: CausalShape, device="cuda", backward=False, stream=None):
        import torch
        s, sizes = shape, sla_causal_query_sizes(shape)
        grads = [_like(st, n, h, s.d, device) if backward else None
                 for st, n, h in ((s.q, s.total_q, s.Hq), (s.k, s.total_k, s.Hkv),
                                  (s.v, s.total_k, s.Hkv))]
        return cls(s, _like(s.o, s.total_q, s.Hq, s.d, device),
                   torch.empty(s.Hq, s.total_q, dtype=torch.float32, device=device), *grads,
                   _allocate_workspace(sizes.workspace_bytes, device, stream))


@dataclasses.dataclass
class DecayBuffers:
    """Output buffers and the workspace of the decayed linear attention for one
    shape; ``state`` is the state behind each sequence, ``d_state`` the gradient
    of the state before it."""
    shape: DecayShape
    o: object
    state: object
    dq: object
    dk: object
    dv: object
    d_state: object
    workspace: object

    @classmethod
    def allocate(cls, shape: DecayShape, device="cuda", state=True, backward=False, stream=None):
        import torch
        s, sizes = shape, sla_decay_query_sizes(shape)

        def states(wanted):
            return torch.empty(s.n_seq, s.H, s.d, s.d, dtype=torch.float32,
                               device=device) if wanted else None
        grads = [_like(st, s.total, s.H, s.d, device) if backward else None
                 for st in (s.q, s.k, s.v)]
        return cls(s, _like(s.o, s.total, s.H, s.d, device), states(state), *grads,
                   states(backward), _allocate_workspace(sizes.workspace_bytes, device, stream))
