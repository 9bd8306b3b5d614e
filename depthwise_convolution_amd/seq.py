"""Python binding of the sequence operators (``include/dwconv_seq.h``): the
causal depthwise convolution, the gated delta rule and the norms around a
block.

The functions carry the C ABI's names and only marshal arguments (GPU tensors
or raw device pointers as ints); the classes own a plan, check shapes, types,
devices and strides, and allocate outputs and workspaces with torch:

    conv = CausalDepthwiseConv1d(C=8192, K=4, dtype="bf16", act="silu")
    mixed = conv(x, w, bias, offsets=offsets)              # tokens x C
    q, k, v = mixed.split([Hk * Dk, Hk * Dk, Hv * Dv], 1)  # slices are taken as they are
    rule = GatedDeltaRule(Hk, Hv, Dk, Dv, "bf16")
    o = rule(q.unflatten(1, (Hk, Dk)), k.unflatten(1, (Hk, Dk)), v.unflatten(1, (Hv, Dv)),
             g, beta, offsets=offsets, state_out=state)
    norm = BlockNorm(Dv, "bf16", after="rms", before="none", gate_act="silu")
    z, _ = norm(o, gate=gate, w_after=w)

``offsets`` (int32, one more than there are sequences) cuts the tokens into
sequences; outputs of tokens behind the last one are left as they were (not
initialised where the call allocates them).  What a call allocates belongs to
``stream`` where one is given, else to torch's current stream of the tensors'
device.  A given stream does not wait for the current one: order them with
``wait_stream``.  The caller's tensors may be dropped after a call on a torch
stream; on a raw handle they have to live until the stream has passed the call.

Nothing is recorded for autograd; ``backward`` gives the gradients.  A tensor that
requires a gradient is refused while gradients are enabled: the outputs would carry
none.  Under ``torch.no_grad()`` and in an ``autograd.Function`` it is taken.
"""
import ctypes

import torch

from . import DwconvError, _dtype_code, _lib

__all__ = ["CausalDepthwiseConv1d", "GatedDeltaRule", "BlockNorm", "SEQ_ACTIVATIONS", "NORM_KINDS"]

SEQ_ACTIVATIONS = {"none": 0, "silu": 1, "sigmoid": 2}
NORM_KINDS = {"none": 0, "rms": 1, "layer": 2}
_TORCH = {0: torch.float32, 1: torch.float16, 2: torch.bfloat16}

_H, _I, _L, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
_OUT, _SIZE = ctypes.POINTER(ctypes.c_void_p), ctypes.POINTER(ctypes.c_size_t)
_QKV = [_H, _L, _H, _L, _H, _L, _H, _H]
_NORM = [_H, _I, _H, _H, _H, _I, _H, _H, _H, _H, _H]
_SIGNATURES = {
    "dwconv_causal_create": [_OUT, _I, _I, _I, _I],
    "dwconv_causal_destroy": [_H],
    "dwconv_causal_fwd": [_H, _H, _L, _H, _H, _H, _I, _I, _H, _H, _H, _L, _H],
    "dwconv_causal_step": [_H, _H, _L, _H, _H, _H, _H, _I, _I, _H, _L, _H],
    "dwconv_causal_bwd_workspace": [_H, _I, _SIZE],
    "dwconv_causal_bwd": [_H, _H, _L, _H, _H, _H, _I, _I, _H, _H, _L, _H, _H, _L, _H, _H, _H, _H, _H],
    "dwconv_delta_create": [_OUT, _I, _I, _I, _I, _I, _F, _I, _F],
    "dwconv_delta_destroy": [_H],
    "dwconv_delta_workspace": [_H, _I, _I, _I, _SIZE],
    "dwconv_delta_fwd": [_H] + _QKV + [_H, _I, _I, _H, _H, _H, _L, _H, _H],
    "dwconv_delta_step": [_H] + _QKV + [_H, _H, _I, _I, _H, _L, _H],
    "dwconv_delta_bwd": [_H] + _QKV + [_H, _I, _I, _H, _H, _L, _H, _H, _L, _H, _L, _H, _L, _H, _H, _H, _H, _H],
    "dwconv_norm_create": [_OUT, _I, _I, _I, _I, _I, _F],
    "dwconv_norm_destroy": [_H],
    "dwconv_norm_fwd": _NORM + [_H, _H, _H],
    "dwconv_norm_bwd_workspace": [_H, _I, _I, _SIZE],
    "dwconv_norm_bwd": _NORM + [_H] * 12,
}
for _name, _args in _SIGNATURES.items():
    getattr(_lib, _name).argtypes = _args
    getattr(_lib, _name).restype = _I
__all__ += list(_SIGNATURES)


def _p(t):
    if t is None or isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("tensors must live on the GPU")
    return t.data_ptr()


def _call(name, *args):
    rc = getattr(_lib, name)(*args)
    if rc != 0:
        raise DwconvError(rc, name)


_INT = 2 ** 31 - 1


def _n(name, v):
    """A count as the C ABI's int, which ctypes would silently cut to 32 bits."""
    if v > _INT or v < ~_INT:
        raise ValueError(f"{name}: {v} is more than the library counts ({_INT})")
    return v


def _create(name, *args):
    for v in args:
        if isinstance(v, int):
            _n(name, v)
    h = _H()
    _call(name, ctypes.byref(h), *args)
    return h.value


def _bytes(name, *args):
    n = ctypes.c_size_t()
    _call(name, *args, ctypes.byref(n))
    return n.value


def _code(table, v):
    if isinstance(v, str):
        if v not in table:
            raise ValueError(f"unknown choice {v!r}: one of {sorted(table)}")
        return table[v]
    return int(v)


# --- the C ABI's functions -------------------------------------------------
def dwconv_causal_create(C, K, dtype, act):
    """Plan of a causal depthwise convolution (an int); DwconvError on bad sizes."""
    return _create("dwconv_causal_create", C, K, _dtype_code(dtype), _code(SEQ_ACTIVATIONS, act))


def dwconv_causal_destroy(h):
    _lib.dwconv_causal_destroy(h)


def dwconv_causal_fwd(h, x, ldx, w, bias, offsets, seqs, tokens, state_in, state_out, y, ldy, stream):
    _call("dwconv_causal_fwd", h, _p(x), ldx, _p(w), _p(bias), _p(offsets), _n("seqs", seqs), _n("tokens", tokens),
          _p(state_in), _p(state_out), _p(y), ldy, stream)


def dwconv_causal_step(h, x, ldx, w, bias, state, slots, n_slots, rows, y, ldy, stream):
    _call("dwconv_causal_step", h, _p(x), ldx, _p(w), _p(bias), _p(state), _p(slots), _n("n_slots", n_slots),
          _n("rows", rows), _p(y), ldy, stream)


def dwconv_causal_bwd_workspace(h, tokens) -> int:
    return _bytes("dwconv_causal_bwd_workspace", h, _n("tokens", tokens))


def dwconv_causal_bwd(h, x, ldx, w, bias, offsets, seqs, tokens, state_in, dy, lddy, dstate_out, dx, lddx, dw, dbias,
                      dstate_in, workspace, stream):
    _call("dwconv_causal_bwd", h, _p(x), ldx, _p(w), _p(bias), _p(offsets), _n("seqs", seqs), _n("tokens", tokens),
          _p(state_in), _p(dy), lddy, _p(dstate_out), _p(dx), lddx, _p(dw), _p(dbias), _p(dstate_in), _p(workspace),
          stream)


def dwconv_delta_create(Hk, Hv, Dk, Dv, dtype, scale, normalize, eps):
    """Plan of a gated delta rule (an int); DwconvError on bad sizes."""
    return _create("dwconv_delta_create", Hk, Hv, Dk, Dv, _dtype_code(dtype), scale, int(normalize), eps)


def dwconv_delta_destroy(h):
    _lib.dwconv_delta_destroy(h)


def dwconv_delta_workspace(h, seqs, tokens, backward) -> int:
    return _bytes("dwconv_delta_workspace", h, _n("seqs", seqs), _n("tokens", tokens), int(backward))


def dwconv_delta_fwd(h, q, ldq, k, ldk, v, ldv, g, beta, offsets, seqs, tokens, state_in, state_out, o, ldo,
                     workspace, stream):
    _call("dwconv_delta_fwd", h, _p(q), ldq, _p(k), ldk, _p(v), ldv, _p(g), _p(beta), _p(offsets), _n("seqs", seqs),
          _n("tokens", tokens), _p(state_in), _p(state_out), _p(o), ldo, _p(workspace), stream)


def dwconv_delta_step(h, q, ldq, k, ldk, v, ldv, g, beta, state, slots, n_slots, rows, o, ldo, stream):
    _call("dwconv_delta_step", h, _p(q), ldq, _p(k), ldk, _p(v), ldv, _p(g), _p(beta), _p(state), _p(slots),
          _n("n_slots", n_slots), _n("rows", rows), _p(o), ldo, stream)


def dwconv_delta_bwd(h, q, ldq, k, ldk, v, ldv, g, beta, offsets, seqs, tokens, state_in, d_o, lddo, dstate_out, dq,
                     lddq, dk, lddk, dv, lddv, dg, dbeta, dstate_in, workspace, stream):
    _call("dwconv_delta_bwd", h, _p(q), ldq, _p(k), ldk, _p(v), ldv, _p(g), _p(beta), _p(offsets), _n("seqs", seqs),
          _n("tokens", tokens), _p(state_in), _p(d_o), lddo, _p(dstate_out), _p(dq), lddq, _p(dk), lddk, _p(dv), lddv,
          _p(dg), _p(dbeta), _p(dstate_in), _p(workspace), stream)


def dwconv_norm_create(D, dtype, after, before, gate_act, eps):
    """Plan of the norms around a block (an int); DwconvError on bad sizes."""
    return _create("dwconv_norm_create", D, _dtype_code(dtype), _code(NORM_KINDS, after), _code(NORM_KINDS, before),
                   _code(SEQ_ACTIVATIONS, gate_act), eps)


def dwconv_norm_destroy(p):
    _lib.dwconv_norm_destroy(p)


def dwconv_norm_fwd(p, rows, o, residual, gate, rows_per_gate, scale, w_after, b_after, w_before, b_before, h, y,
                    stream):
    _call("dwconv_norm_fwd", p, _n("rows", rows), _p(o), _p(residual), _p(gate), _n("rows_per_gate", rows_per_gate),
          _p(scale), _p(w_after), _p(b_after), _p(w_before), _p(b_before), _p(h), _p(y), stream)


def dwconv_norm_bwd_workspace(p, rows, rows_per_gate) -> int:
    return _bytes("dwconv_norm_bwd_workspace", p, _n("rows", rows), _n("rows_per_gate", rows_per_gate))


def dwconv_norm_bwd(p, rows, o, residual, gate, rows_per_gate, scale, w_after, b_after, w_before, b_before, dh, dy,
                    d_o, dresidual, dgate, dscale, dw_after, db_after, dw_before, db_before, workspace, stream):
    _call("dwconv_norm_bwd", p, _n("rows", rows), _p(o), _p(residual), _p(gate), _n("rows_per_gate", rows_per_gate),
          _p(scale), _p(w_after), _p(b_after), _p(w_before), _p(b_before), _p(dh), _p(dy), _p(d_o), _p(dresidual),
          _p(dgate), _p(dscale), _p(dw_after), _p(db_after), _p(dw_before), _p(db_before), _p(workspace), stream)


# --- plans with checks and allocation --------------------------------------
def _dense(name, t, shape, dtype, dev):
    """``t`` is a dense tensor of that shape and type on that device."""
    if t.shape != shape or t.dtype is not dtype or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous {dtype} tensor of shape {shape} on {dev} is needed, got "
                         f"{t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}")


def _tokens(name, t, shape, dtype, dev):
    """Token stride of ``t``, whose channels (heads x channels) are dense."""
    width = shape[1] if len(shape) == 2 else shape[1] * shape[2]
    ok = t.shape == shape and t.dtype is dtype and t.device == dev
    if ok and not t.is_contiguous():
        st = t.stride()
        ok = shape[-1] == 1 or st[-1] == 1
        if len(shape) == 3 and shape[1] > 1:
            ok = ok and st[1] == shape[2]
        if shape[0] > 1:
            ok = ok and st[0] >= width
        if ok and shape[0] > 1:
            return st[0]
    if not ok:
        raise ValueError(f"{name}: a {dtype} tensor of shape {shape} on {dev} with dense channels and a token stride "
                         f"of at least {width} is needed, got {t.dtype} {tuple(t.shape)} strides {t.stride()} on "
                         f"{t.device}")
    return width


def _sequences(offsets, dev):
    if offsets is None:
        return 1
    if offsets.dim() != 1 or offsets.numel() < 1:
        raise ValueError("offsets: one dimension, one value more than there are sequences")
    _dense("offsets", offsets, (offsets.numel(),), torch.int32, dev)
    return _n("offsets", offsets.numel() - 1)


def _slots(slots, rows, n_slots, dev):
    _n("state", n_slots)
    if slots is None:
        if rows > n_slots:
            raise ValueError(f"{rows} rows without slots need as many cache entries, got {n_slots}")
    else:
        _dense("slots", slots, (rows,), torch.int32, dev)


def _current_raw(index):
    return torch.cuda.current_stream(index).cuda_stream


# the same handle without a Stream object around it: 0.1 us instead of 2.8, a
# fifth of a one-token step's call
_current_raw = getattr(torch._C, "_cuda_getCurrentRawStream", _current_raw)


def _on(dev, stream, body, *tensors):
    """``body`` with the raw handle of ``stream`` (a torch stream, a raw handle,
    None: the current one), ``dev`` current and that stream the one torch
    allocates for.  ``tensors`` are the caller's: torch's allocator keeps their
    memory until a torch stream has passed the call.  (Not for a raw handle, whose
    stream may be gone by the time a tensor is freed.)"""
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                raise ValueError("the sequence operators record nothing for autograd, but a tensor requires a gradient: "
                                 "call them under torch.no_grad() (or in an autograd.Function) and use backward()")
    if stream is None and torch.cuda.current_device() == dev.index:
        return body(_current_raw(dev.index))
    keep = stream is not None and not isinstance(stream, (int, torch.cuda.ExternalStream))
    if keep and stream.device != dev:
        raise ValueError(f"stream: it belongs to {stream.device}, the tensors to {dev}")
    with torch.cuda.device(dev):
        if stream is None:
            return body(_current_raw(dev.index))
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, dev) if stream else torch.cuda.default_stream(dev)
        with torch.cuda.stream(stream):
            out = body(stream.cuda_stream)
        if keep:
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)
        return out


class _Plan:
    _destroy = None
    handle = None

    def close(self):
        if self.handle:
            getattr(_lib, self._destroy)(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _device(self, name, t):
        if not self.handle:
            raise ValueError("the plan is closed")
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{name}: a GPU tensor is needed")
        return t.device


def _workspace(ws, need, dev):
    if ws is None:
        return torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    if ws.device != dev or not ws.is_contiguous() or ws.numel() * ws.element_size() < need:
        raise ValueError(f"workspace: {need} contiguous bytes on {dev} are needed")
    return ws


class CausalDepthwiseConv1d(_Plan):
    """y[t] = act(bias + sum_k w[k] ext[t + k]) over packed sequences, ext =
    [state_in; x].  x, y: tokens x C; w: K x C; bias: C float32 or None; states:
    sequences x (K-1) x C in x's type.  ``act``: "silu" or "none"."""

    _destroy = "dwconv_causal_destroy"

    def __init__(self, C, K, dtype="bf16", act="silu"):
        code = _dtype_code(dtype)
        self.handle = dwconv_causal_create(C, K, code, act)
        self.C, self.K, self.dtype = C, K, _TORCH[code]

    def _common(self, x, w, bias, offsets, state_in):
        dev, dt = self._device("x", x), self.dtype
        if x.dim() != 2:
            raise ValueError("x: tokens x channels")
        n, seqs = _n("x", x.shape[0]), _sequences(offsets, dev)
        _dense("w", w, (self.K, self.C), dt, dev)
        if bias is not None:
            _dense("bias", bias, (self.C,), torch.float32, dev)
        if state_in is not None:
            _dense("state_in", state_in, (seqs, self.K - 1, self.C), dt, dev)
        return dev, dt, n, seqs, _tokens("x", x, (n, self.C), dt, dev)

    def __call__(self, x, w, bias=None, offsets=None, state_in=None, state_out=None, y=None, stream=None):
        """Returns y; ``state_out``, where given, gets the last K-1 rows of
        every sequence's ext."""
        dev, dt, n, seqs, ldx = self._common(x, w, bias, offsets, state_in)
        if state_out is not None:
            _dense("state_out", state_out, (seqs, self.K - 1, self.C), dt, dev)

        def body(raw):
            nonlocal y
            if y is None:
                y = torch.empty((n, self.C), dtype=dt, device=dev)
            dwconv_causal_fwd(self.handle, x, ldx, w, bias, offsets, seqs, n, state_in, state_out, y,
                              _tokens("y", y, (n, self.C), dt, dev), raw)
            return y

        return _on(dev, stream, body, x, w, bias, offsets, state_in, state_out, y)

    def step(self, x, w, bias, state, slots=None, y=None, stream=None):
        """One token for each row of x; ``state`` (cache entries x (K-1) x C) is
        shifted in place.  Row i has entry slots[i] (None: entry i); a slot
        outside the cache skips the row, its y stays as it was."""
        dev, dt, n, _, ldx = self._common(x, w, bias, None, None)
        entries = state.shape[0]
        _dense("state", state, (entries, self.K - 1, self.C), dt, dev)
        _slots(slots, n, entries, dev)

        def body(raw):
            nonlocal y
            if y is None:
                y = torch.empty((n, self.C), dtype=dt, device=dev)
            dwconv_causal_step(self.handle, x, ldx, w, bias, state, slots, entries, n, y,
                               _tokens("y", y, (n, self.C), dt, dev), raw)
            return y

        return _on(dev, stream, body, x, w, bias, state, slots, y)

    def backward(self, x, w, dy, bias=None, offsets=None, state_in=None, dstate_out=None, dx=None, dw=None,
                 dbias=None, dstate_in=None, workspace=None, stream=None):
        """(dx, dw, dbias, dstate_in) for the output gradient dy and, where
        given, the gradient dstate_out of the final states.  dw and dbias are
        float32; dbias is None without a bias, dstate_in without a state."""
        dev, dt, n, seqs, ldx = self._common(x, w, bias, offsets, state_in)
        lddy = _tokens("dy", dy, (n, self.C), dt, dev)
        states = (seqs, self.K - 1, self.C)
        if dstate_out is not None:
            _dense("dstate_out", dstate_out, states, dt, dev)

        def body(raw):
            nonlocal dx, dw, dbias, dstate_in
            ws = _workspace(workspace, dwconv_causal_bwd_workspace(self.handle, n), dev)
            if dx is None:
                dx = torch.empty((n, self.C), dtype=dt, device=dev)
            if dw is None:
                dw = torch.empty((self.K, self.C), dtype=torch.float32, device=dev)
            if dbias is None and bias is not None:
                dbias = torch.empty(self.C, dtype=torch.float32, device=dev)
            if dstate_in is None and state_in is not None:
                dstate_in = torch.empty(states, dtype=dt, device=dev)
            _dense("dw", dw, (self.K, self.C), torch.float32, dev)
            if dbias is not None:
                _dense("dbias", dbias, (self.C,), torch.float32, dev)
            if dstate_in is not None:
                _dense("dstate_in", dstate_in, states, dt, dev)
            dwconv_causal_bwd(self.handle, x, ldx, w, bias, offsets, seqs, n, state_in, dy, lddy, dstate_out, dx,
                              _tokens("dx", dx, (n, self.C), dt, dev), dw, dbias, dstate_in, ws, raw)
            return dx, dw, dbias, dstate_in

        return _on(dev, stream, body, x, w, bias, offsets, state_in, dy, dstate_out, dx, dw, dbias, dstate_in, workspace)


class GatedDeltaRule(_Plan):
    """S_t = e^g S + k (beta (v - e^g S^T k))^T, o = S_t^T q, for Hv value heads
    that share Hk key heads.  q, k: tokens x Hk x Dk; v, o: tokens x Hv x Dv; g,
    beta: tokens x Hv float32; states: sequences x Hv x Dk x Dv float32.
    ``scale`` multiplies q (None: 1 / sqrt(Dk)); ``normalize`` divides q and k
    by their lengths first."""

    _destroy = "dwconv_delta_destroy"

    def __init__(self, Hk, Hv, Dk, Dv, dtype="bf16", scale=None, normalize=True, eps=1e-6):
        code = _dtype_code(dtype)
        if scale is None:
            scale = Dk ** -0.5 if Dk > 0 else 1.0
        self.handle = dwconv_delta_create(Hk, Hv, Dk, Dv, code, scale, normalize, eps)
        self.Hk, self.Hv, self.Dk, self.Dv, self.dtype = Hk, Hv, Dk, Dv, _TORCH[code]

    def _common(self, q, k, v, g, beta):
        dev, dt = self._device("q", q), self.dtype
        n = _n("q", q.shape[0])
        lds = (_tokens("q", q, (n, self.Hk, self.Dk), dt, dev), _tokens("k", k, (n, self.Hk, self.Dk), dt, dev),
               _tokens("v", v, (n, self.Hv, self.Dv), dt, dev))
        _dense("g", g, (n, self.Hv), torch.float32, dev)
        _dense("beta", beta, (n, self.Hv), torch.float32, dev)
        return dev, dt, n, lds

    def __call__(self, q, k, v, g, beta, offsets=None, state_in=None, state_out=None, o=None, workspace=None,
                 stream=None):
        """Returns o; ``state_out``, where given, gets every sequence's last
        state (it may be state_in itself)."""
        dev, dt, n, (ldq, ldk, ldv) = self._common(q, k, v, g, beta)
        seqs = _sequences(offsets, dev)
        states = (seqs, self.Hv, self.Dk, self.Dv)
        for name, t in (("state_in", state_in), ("state_out", state_out)):
            if t is not None:
                _dense(name, t, states, torch.float32, dev)

        def body(raw):
            nonlocal o
            ws = _workspace(workspace, dwconv_delta_workspace(self.handle, seqs, n, False), dev)
            if o is None:
                o = torch.empty((n, self.Hv, self.Dv), dtype=dt, device=dev)
            dwconv_delta_fwd(self.handle, q, ldq, k, ldk, v, ldv, g, beta, offsets, seqs, n, state_in, state_out, o,
                             _tokens("o", o, (n, self.Hv, self.Dv), dt, dev), ws, raw)
            return o

        return _on(dev, stream, body, q, k, v, g, beta, offsets, state_in, state_out, o, workspace)

    def step(self, q, k, v, g, beta, state, slots=None, o=None, stream=None):
        """One token for each row; ``state`` (cache entries x Hv x Dk x Dv) is
        updated in place.  Slots as for CausalDepthwiseConv1d.step."""
        dev, dt, n, (ldq, ldk, ldv) = self._common(q, k, v, g, beta)
        entries = state.shape[0]
        _dense("state", state, (entries, self.Hv, self.Dk, self.Dv), torch.float32, dev)
        _slots(slots, n, entries, dev)

        def body(raw):
            nonlocal o
            if o is None:
                o = torch.empty((n, self.Hv, self.Dv), dtype=dt, device=dev)
            dwconv_delta_step(self.handle, q, ldq, k, ldk, v, ldv, g, beta, state, slots, entries, n, o,
                              _tokens("o", o, (n, self.Hv, self.Dv), dt, dev), raw)
            return o

        return _on(dev, stream, body, q, k, v, g, beta, state, slots, o)

    def backward(self, q, k, v, g, beta, do, offsets=None, state_in=None, dstate_out=None, dq=None, dk=None, dv=None,
                 dg=None, dbeta=None, dstate_in=None, workspace=None, stream=None):
        """(dq, dk, dv, dg, dbeta, dstate_in) for the output gradient do and,
        where given, the gradient dstate_out of the final states; dstate_in is
        None without a state."""
        dev, dt, n, (ldq, ldk, ldv) = self._common(q, k, v, g, beta)
        seqs = _sequences(offsets, dev)
        states = (seqs, self.Hv, self.Dk, self.Dv)
        keys, values = (n, self.Hk, self.Dk), (n, self.Hv, self.Dv)
        lddo = _tokens("do", do, values, dt, dev)
        for name, t in (("state_in", state_in), ("dstate_out", dstate_out)):
            if t is not None:
                _dense(name, t, states, torch.float32, dev)

        def body(raw):
            nonlocal dq, dk, dv, dg, dbeta, dstate_in
            ws = _workspace(workspace, dwconv_delta_workspace(self.handle, seqs, n, True), dev)
            if dq is None:
                dq = torch.empty(keys, dtype=dt, device=dev)
            if dk is None:
                dk = torch.empty(keys, dtype=dt, device=dev)
            if dv is None:
                dv = torch.empty(values, dtype=dt, device=dev)
            if dg is None:
                dg = torch.empty((n, self.Hv), dtype=torch.float32, device=dev)
            if dbeta is None:
                dbeta = torch.empty((n, self.Hv), dtype=torch.float32, device=dev)
            if dstate_in is None and state_in is not None:
                dstate_in = torch.empty(states, dtype=torch.float32, device=dev)
            _dense("dg", dg, (n, self.Hv), torch.float32, dev)
            _dense("dbeta", dbeta, (n, self.Hv), torch.float32, dev)
            if dstate_in is not None:
                _dense("dstate_in", dstate_in, states, torch.float32, dev)
            dwconv_delta_bwd(self.handle, q, ldq, k, ldk, v, ldv, g, beta, offsets, seqs, n, state_in, do, lddo,
                             dstate_out, dq, _tokens("dq", dq, keys, dt, dev), dk, _tokens("dk", dk, keys, dt, dev),
                             dv, _tokens("dv", dv, values, dt, dev), dg, dbeta, dstate_in, ws, raw)
            return dq, dk, dv, dg, dbeta, dstate_in

        return _on(dev, stream, body, q, k, v, g, beta, do, offsets, state_in, dstate_out, dq, dk, dv, dg, dbeta,
                   dstate_in, workspace)


class BlockNorm(_Plan):
    """h = residual + scale * N_after(o) * act(gate) and y = N_before(h), rows of
    D channels.  ``after``, ``before``: "rms", "layer" or "none"; ``gate_act``:
    "silu", "sigmoid" or "none".  A gate row serves ``rows_per_gate`` rows.  scale
    and the norms' weights and biases are D float32 values."""

    _destroy = "dwconv_norm_destroy"

    def __init__(self, D, dtype="bf16", after="rms", before="rms", gate_act="silu", eps=1e-6):
        code = _dtype_code(dtype)
        self.handle = dwconv_norm_create(D, code, after, before, gate_act, eps)
        self.D, self.dtype = D, _TORCH[code]
        self.after, self.before = _code(NORM_KINDS, after), _code(NORM_KINDS, before)

    def _common(self, o, residual, gate, scale, w_after, b_after, w_before, b_before, per):
        dev, D = self._device("o", o), self.D
        if o.dim() < 1 or o.shape[-1] != D:
            raise ValueError(f"o: rows of {D} channels")
        shape = tuple(o.shape)
        _dense("o", o, shape, self.dtype, dev)
        rows = _n("o", o.numel() // D)
        if residual is not None:
            _dense("residual", residual, shape, self.dtype, dev)
        if _n("rows_per_gate", per) < 1:
            raise ValueError("rows_per_gate: at least 1")
        if gate is not None:
            if gate.numel() != -(-rows // per) * D:
                raise ValueError(f"gate: {-(-rows // per)} rows of {D} channels, got {tuple(gate.shape)}")
            _dense("gate", gate, tuple(gate.shape), self.dtype, dev)
        else:
            per = 1
        for name, t in (("scale", scale), ("w_after", w_after), ("b_after", b_after), ("w_before", w_before),
                        ("b_before", b_before)):
            if t is not None:
                _dense(name, t, (D,), torch.float32, dev)
        return dev, rows, per

    def __call__(self, o, residual=None, gate=None, scale=None, w_after=None, b_after=None, w_before=None,
                 b_before=None, rows_per_gate=1, h=None, y=None, stream=None):
        """Returns (h, y); y is None where ``before`` is "none" (a given one is not
        written)."""
        dev, rows, per = self._common(o, residual, gate, scale, w_after, b_after, w_before, b_before, rows_per_gate)

        def body(raw):
            nonlocal h, y
            if h is None:
                h = torch.empty_like(o)
            if y is None and self.before:
                y = torch.empty_like(o)
            _dense("h", h, tuple(o.shape), self.dtype, dev)
            if y is not None:
                _dense("y", y, tuple(o.shape), self.dtype, dev)
            dwconv_norm_fwd(self.handle, rows, o, residual, gate, per, scale, w_after, b_after, w_before, b_before, h,
                            y, raw)
            return h, y if self.before else None

        return _on(dev, stream, body, o, residual, gate, scale, w_after, b_after, w_before, b_before, h, y)

    def backward(self, o, dh=None, dy=None, residual=None, gate=None, scale=None, w_after=None, b_after=None,
                 w_before=None, b_before=None, rows_per_gate=1, workspace=None, stream=None):
        """Gradients of (o, residual, gate, scale, w_after, b_after, w_before,
        b_before) for those of h and y; None for what was not given or has no
        part in the plan."""
        dev, rows, per = self._common(o, residual, gate, scale, w_after, b_after, w_before, b_before, rows_per_gate)
        for name, t in (("dh", dh), ("dy", dy)):
            if t is not None:
                _dense(name, t, tuple(o.shape), self.dtype, dev)

        def body(raw):
            ws = _workspace(workspace, dwconv_norm_bwd_workspace(self.handle, rows, per), dev)
            like = [o, residual, gate, scale, w_after if self.after else None,
                    b_after if self.after == 2 else None, w_before if self.before else None,
                    b_before if self.before == 2 else None]
            grads = [None if t is None else torch.empty_like(t) for t in like]
            dwconv_norm_bwd(self.handle, rows, o, residual, gate, per, scale, w_after, b_after, w_before, b_before, dh,
                            dy, *grads, ws, raw)
            return tuple(grads)

        return _on(dev, stream, body, o, dh, dy, residual, gate, scale, w_after, b_after, w_before, b_before, workspace)
