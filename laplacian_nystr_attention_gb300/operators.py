"""The operators beside the attention, as objects over torch tensors: ``GatedScan``,
``ResidualNorm`` and ``GradClip``, each one plan of the C ABI in include/lapl_ops.h.

Like ``LaplacianNystromAttention`` they check their arguments and use PyTorch only to allocate
device memory and to pick the stream.  A plan belongs to the device that is current when it is
made; its calls take tensors of that device and are refused while another one is current.  Calls
run on torch's current stream unless one is given, which must already be ordered after whatever
wrote the inputs.  Workspaces are allocated per call, so calls captured into several graphs share
nothing.
"""
from __future__ import annotations

import ctypes

from . import _lib
from ._lib import (LAPL_BF16, LAPL_F32, LAPL_F8E4M3, LAPL_GATE_DECAY, LAPL_GATE_SIGMOID,
                   LAPL_SCAN_CHUNK)

_DTYPES = {"f32": LAPL_F32, "bf16": LAPL_BF16, "f8": LAPL_F8E4M3}
_GATES = {"decay": LAPL_GATE_DECAY, "sigmoid": LAPL_GATE_SIGMOID}
#: The largest fp32 value, and so the largest norm to clip to.
FLOAT_MAX = 3.4028234663852886e38


def make_scan_config(sequences, tokens, channels, gate="sigmoid", reverse=0, in_dtype="f32",
                     out_dtype="f32", grad_dtype="f32", x_stride=0,
                     g_stride=0) -> _lib.lapl_scan_config:
    """gate: "decay" or "sigmoid" or the lapl_gate integer; x_stride, g_stride: elements from one
    token to the next (0: channels)."""
    return _lib.lapl_scan_config(int(sequences), int(tokens), int(channels),
                                 _GATES.get(gate, gate), int(reverse),
                                 _DTYPES.get(in_dtype, in_dtype),
                                 _DTYPES.get(out_dtype, out_dtype),
                                 _DTYPES.get(grad_dtype, grad_dtype), int(x_stride), int(g_stride))


def make_norm_config(batch, heads, tokens, head_dim, eps=1e-6, x_dtype="f32", res_dtype="f32",
                     out_dtype="f32", grad_dtype="f32", scale_group=0) -> _lib.lapl_norm_config:
    """out_dtype: "f32", "bf16" or "f8" (e4m3 with scales)."""
    return _lib.lapl_norm_config(int(batch), int(heads), int(tokens), int(head_dim), float(eps),
                                 _DTYPES.get(x_dtype, x_dtype), _DTYPES.get(res_dtype, res_dtype),
                                 _DTYPES.get(out_dtype, out_dtype),
                                 _DTYPES.get(grad_dtype, grad_dtype), int(scale_group))


def _torch_dtype(code):
    """None for what is no dtype: the library refuses such a configuration."""
    import torch
    return {LAPL_F32: torch.float32, LAPL_BF16: torch.bfloat16,
            LAPL_F8E4M3: torch.float8_e4m3fn}.get(code)


class _Layout:
    """What an argument has to be: type, shape, and the strides of contiguous rows, `rows` elements
    apart where given."""

    __slots__ = ("name", "dtype", "shape", "strides", "rows")

    def __init__(self, name, dtype, shape, rows=0):
        self.name, self.dtype, self.shape = name, dtype, tuple(shape)
        self.rows = rows or self.shape[-1]
        self.strides = self.strides_of(self.shape)

    def strides_of(self, shape):
        strides, step = [1], self.rows
        for n in reversed(shape[1:-1]):
            strides.append(step)
            step *= n
        if len(shape) > 1:
            strides.append(step)
        return tuple(reversed(strides))


class _Plan:
    """A handle, its device, and what the three operators' calls have in common."""

    _destroy = None
    _index = -1

    def _open(self, handle):
        import torch
        self.handle = handle
        self._empty = torch.empty
        self._raw_stream = torch._C._cuda_getCurrentRawStream   # the address alone, at 1/30 the time
        self._index = torch.cuda.current_device()
        self.device = torch.device("cuda", self._index)

    def _check(self, t, want):
        """t's address, if it is what `want` says; ValueError otherwise."""
        if (t.dtype is not want.dtype or t.shape != want.shape or t.stride() != want.strides
                or t.get_device() != self._index):
            self._check_closely(t, want)
        return t.data_ptr()

    def _check_closely(self, t, want):
        """The same for tensors with size-1 dimensions, whose strides say nothing, and with more
        leading dimensions, and the messages."""
        shape = want.shape
        if len(shape) == 3 and t.dim() > 3:      # [B, H, N, d] for [S, N, C] with B H = S
            lead = 1
            for n in t.shape[:-2]:
                lead *= n
            if lead == shape[0]:
                shape = tuple(t.shape[:-2]) + shape[1:]
        if t.dtype is not want.dtype:
            raise ValueError(f"{want.name}: expected {want.dtype}, got {t.dtype}")
        if t.get_device() != self._index:
            raise ValueError(f"{want.name}: expected a tensor on {self.device}, got {t.device}")
        if t.shape != shape:
            raise ValueError(f"{want.name}: expected shape {shape}, got {tuple(t.shape)}")
        strides = want.strides_of(shape)
        if t.numel() and any(n != 1 and a != b for n, a, b in zip(shape, t.stride(), strides)):
            raise ValueError(f"{want.name}: expected strides {strides}, got {t.stride()}")

    def _on(self, stream, tensors):
        """A context in which the call's stream is current; tensors that the call uses on a stream
        that is not theirs are kept for it."""
        import torch
        if stream.device != self.device:
            raise ValueError(f"stream: expected one of {self.device}, got {stream.device}")
        if stream != torch.cuda.current_stream(self.device):
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)
        return torch.cuda.stream(stream)

    def close(self):
        if getattr(self, "handle", None) is not None:
            type(self)._destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class GatedScan(_Plan):
    """h_i = a_i h_{i-1} + x_i ("decay": a = g) or + (1 - a_i) x_i ("sigmoid": a = sigmoid(g)) over
    the tokens of each sequence, for every channel.

    Long sequences wait for one another's parts on the GPU, each wait bounded to a second; results
    of a call whose wait gave up are undefined, and check_device_errors() is what tells."""

    _destroy = staticmethod(_lib.lapl_scan_destroy)

    def __init__(self, cfg: _lib.lapl_scan_config):
        self._open(_lib.lapl_scan_create(cfg))
        self._layouts(cfg)

    def _layouts(self, c):
        import torch
        self.cfg = c
        tokens = (c.sequences, c.tokens, c.channels)
        self.state_shape = (c.sequences, c.channels)
        self.states_shape = (c.sequences, -(-c.tokens // LAPL_SCAN_CHUNK), c.channels)
        i, g = _torch_dtype(c.in_dtype), _torch_dtype(c.grad_dtype)
        self._x = _Layout("x", i, tokens, c.x_stride)
        self._g = _Layout("g", i, tokens, c.g_stride)
        self._out = _Layout("out", _torch_dtype(c.out_dtype), tokens)
        self._dout = _Layout("dout", g, tokens)
        self._dx = _Layout("dx", g, tokens, c.x_stride)
        self._dg = _Layout("dg", g, tokens, c.g_stride)
        self._lengths = _Layout("lengths", torch.int32, (c.sequences,))
        self._states = _Layout("states", torch.float32, self.states_shape)
        self._state = {name: _Layout(name, torch.float32, self.state_shape)
                       for name in ("h0", "final", "dfinal", "dh0")}

    def forward(self, x, g, h0=None, lengths=None, out=None, states=None, final=None, stream=None):
        """h, the state after every token.  x, g: [S, N, C] or [B, H, N, d] with B H = S; h0, final:
        fp32 [S, C] (final is written; it may be h0); lengths: int32 [S]; states: fp32
        ``states_shape``, written for backward()."""
        if stream is not None:
            with self._on(stream, (x, g, h0, lengths, out, states, final)):
                return self.forward(x, g, h0, lengths, out, states, final)
        at_x = self._check(x, self._x)
        if out is None:
            out = self._empty(x.shape, dtype=self._out.dtype, device=self.device)
            at_out = out.data_ptr()
        else:
            at_out = self._check(out, self._out)
        _lib.lapl_scan_forward(
            self.handle, at_x, self._check(g, self._g),
            None if h0 is None else self._check(h0, self._state["h0"]),
            None if lengths is None else self._check(lengths, self._lengths), at_out,
            None if states is None else self._check(states, self._states),
            None if final is None else self._check(final, self._state["final"]),
            self._raw_stream(self._index))
        return out

    __call__ = forward

    def backward(self, x, g, states, dout, dfinal=None, lengths=None, grads=None, stream=None):
        """(dx, dg, dh0) for a loss with dLoss/dout = dout and dLoss/dfinal = dfinal.  states: what
        forward() wrote for the same x, g, h0 and lengths.  grads: optional dict with preallocated
        "dx", "dg" (grad_dtype, rows apart as x's and g's) and "dh0" (fp32 [S, C]; may be
        dfinal)."""
        if stream is not None:
            with self._on(stream, (x, g, states, dout, dfinal, lengths, *(grads or {}).values())):
                return self.backward(x, g, states, dout, dfinal, lengths, grads)
        get = (grads or {}).get
        dx, dg, dh0 = get("dx"), get("dg"), get("dh0")
        at_x, at_g = self._check(x, self._x), self._check(g, self._g)
        dx, at_dx = self._like(dx, self._dx, x)
        dg, at_dg = self._like(dg, self._dg, g)
        if dh0 is None:
            dh0 = self._empty(self.state_shape, dtype=self._states.dtype, device=self.device)
            at_dh0 = dh0.data_ptr()
        else:
            at_dh0 = self._check(dh0, self._state["dh0"])
        _lib.lapl_scan_backward(
            self.handle, at_x, at_g, self._check(states, self._states),
            None if lengths is None else self._check(lengths, self._lengths),
            self._check(dout, self._dout),
            None if dfinal is None else self._check(dfinal, self._state["dfinal"]),
            at_dx, at_dg, at_dh0, self._raw_stream(self._index))
        return dx, dg, dh0

    def check_device_errors(self, stream=None):
        """Raises LaplAttnError if a wait on this device has given up since the last time it was
        asked; waits for the stream's work so far (not while it is captured)."""
        if stream is not None:
            with self._on(stream, ()):
                return self.check_device_errors()
        _lib.lapl_scan_device_errors(self.handle, self._raw_stream(self._index))

    def _like(self, grad, want, like):
        """A gradient and its address: the one given, checked, or a new one in rows as like's."""
        if grad is not None:
            return grad, self._check(grad, want)
        if want.rows == want.shape[-1]:
            grad = self._empty(like.shape, dtype=want.dtype, device=self.device)
        else:
            grad = self._empty((*like.shape[:-1], want.rows), dtype=want.dtype,
                               device=self.device)[..., :want.shape[-1]]
        return grad, grad.data_ptr()


class ResidualNorm(_Plan):
    """s = x + residual, y = s / sqrt(mean(s^2) + eps) * weight over the H d values of each token,
    x as the attention writes it, [B, H, N, d]."""

    _destroy = staticmethod(_lib.lapl_norm_destroy)

    def __init__(self, cfg: _lib.lapl_norm_config):
        self._open(_lib.lapl_norm_create(cfg))
        self._layouts(cfg)
        self.workspace_bytes = _lib.lapl_norm_workspace_size(self.handle)
        self._workspace_floats = self.workspace_bytes // 4

    def _layouts(self, c):
        import torch
        self.cfg = c
        self.f8 = c.out_dtype == LAPL_F8E4M3
        self.width = c.heads * c.head_dim
        self.rows_shape = (c.batch, c.tokens, self.width)
        self.scales_shape = (c.batch, c.tokens, self.width // (c.scale_group or self.width))
        heads = (c.batch, c.heads, c.tokens, c.head_dim)
        res, g = _torch_dtype(c.res_dtype), _torch_dtype(c.grad_dtype)
        self._x = _Layout("x", _torch_dtype(c.x_dtype), heads)
        self._dx = _Layout("dx", g, heads)
        self._x_row = _Layout("x", _torch_dtype(c.x_dtype), self.rows_shape)
        self._dx_row = _Layout("dx", g, self.rows_shape)
        self._weight = _Layout("weight", torch.float32, (self.width,))
        self._dweight = _Layout("dweight", torch.float32, (self.width,))
        self._residual = _Layout("residual", res, self.rows_shape)
        self._sum = _Layout("sum", res, self.rows_shape)
        self._rstd = _Layout("rstd", torch.float32, self.rows_shape[:2])
        self._out = _Layout("out", _torch_dtype(c.out_dtype), self.rows_shape)
        self._scales = _Layout("scales", torch.float32, self.scales_shape)
        self._dy = _Layout("dy", g, self.rows_shape)
        self._dsum = _Layout("dsum", g, self.rows_shape)
        self._dres = _Layout("dres", g, self.rows_shape)

    def _by_head(self, t, want, want_row):
        return self._check(t, want_row if self.cfg.heads == 1 and t.dim() == 3 else want)

    def forward(self, x, weight=None, residual=None, sum=None, rstd=None, out=None, scales=None,
                stream=None):
        """y, or (y, scales) for 8-bit outputs.  x: [B, H, N, d] (or [B, N, d] with one head);
        weight: fp32 [W]; residual, sum: [B, N, W] (sum is written; it may be residual); rstd: fp32
        [B, N], written for backward(); scales: fp32 [B, N, groups of a row]."""
        if stream is not None:
            with self._on(stream, (x, weight, residual, sum, rstd, out, scales)):
                return self.forward(x, weight, residual, sum, rstd, out, scales)
        if scales is not None and not self.f8:
            raise ValueError("scales: only for 8-bit outputs")
        if out is None:
            out = self._empty(self.rows_shape, dtype=self._out.dtype, device=self.device)
            at_out = out.data_ptr()
        else:
            at_out = self._check(out, self._out)
        if scales is None and self.f8:
            scales = self._empty(self.scales_shape, dtype=self._scales.dtype, device=self.device)
        _lib.lapl_norm_forward(
            self.handle, self._by_head(x, self._x, self._x_row),
            None if residual is None else self._check(residual, self._residual),
            None if weight is None else self._check(weight, self._weight),
            None if sum is None else self._check(sum, self._sum),
            None if rstd is None else self._check(rstd, self._rstd), at_out,
            None if scales is None else self._check(scales, self._scales),
            self._raw_stream(self._index))
        return (out, scales) if self.f8 else out

    __call__ = forward

    def backward(self, sum, rstd, weight, dy, dsum=None, grads=None, stream=None):
        """(dx, dres, dweight) for a loss with dLoss/dy = dy and dLoss/dsum = dsum from sum's other
        uses.  sum, rstd: what forward() wrote (without a residual and with one head, sum may be x
        itself).  grads: optional dict with preallocated "dx" ([B, H, N, d], the dout that the
        attention's backward takes), "dres" ([B, N, W]; may be dsum) and "dweight" (fp32 [W]), or
        None for one that is not wanted."""
        if stream is not None:
            with self._on(stream, (sum, rstd, weight, dy, dsum, *(grads or {}).values())):
                return self.backward(sum, rstd, weight, dy, dsum, grads)
        grads = grads or {}
        dx, at_dx = self._wanted(grads, self._dx)
        dres, at_dres = self._wanted(grads, self._dres)
        dweight, at_dweight = self._wanted(grads, self._dweight)
        workspace = None
        if dweight is not None:
            workspace = self._empty(self._workspace_floats, dtype=self._rstd.dtype,
                                    device=self.device)
        _lib.lapl_norm_backward(
            self.handle, self._check(sum, self._sum), self._check(rstd, self._rstd),
            None if weight is None else self._check(weight, self._weight),
            self._check(dy, self._dy), None if dsum is None else self._check(dsum, self._dsum),
            at_dx, at_dres, at_dweight,
            None if workspace is None else workspace.data_ptr(), self.workspace_bytes,
            self._raw_stream(self._index))
        return dx, dres, dweight

    def _wanted(self, grads, want):
        """A gradient and its address: the one given, checked, or a new one; None for None."""
        if want.name not in grads:
            t = self._empty(want.shape, dtype=want.dtype, device=self.device)
            return t, t.data_ptr()
        t = grads[want.name]
        if t is None:
            return None, None
        return t, self._by_head(t, want, self._dx_row) if want is self._dx else self._check(t, want)


class GradClip(_Plan):
    """The global norm of a list of gradients, and clipping to a largest norm.

    counts: values of each tensor; dtypes: "f32" or "bf16" (or the lapl_dtype integer) for each."""

    _destroy = staticmethod(_lib.lapl_clip_destroy)

    def __init__(self, counts, dtypes):
        self.counts = [int(n) for n in counts]
        self.dtypes = [_DTYPES.get(t, t) for t in dtypes]
        if len(self.counts) != len(self.dtypes):
            raise ValueError(f"{len(self.counts)} counts and {len(self.dtypes)} dtypes")
        self._torch_dtypes = [_torch_dtype(t) for t in self.dtypes]
        n = len(self.counts)
        room = max(n, 1)
        self._open(_lib.lapl_clip_create(_lib.lapl_clip_config(
            n, (ctypes.c_longlong * room)(*self.counts), (ctypes.c_int * room)(*self.dtypes))))
        self.workspace_bytes = _lib.lapl_clip_workspace_size(self.handle)
        self._workspace_floats = self.workspace_bytes // 4
        self._float = _torch_dtype(LAPL_F32)
        self._devices = [self._index] * n

    @classmethod
    def like(cls, tensors):
        """A plan for these tensors' sizes and types."""
        import torch
        names = {torch.float32: "f32", torch.bfloat16: "bf16"}
        for t in tensors:
            if t.dtype not in names:
                raise ValueError(f"expected float32 or bfloat16 tensors, got {t.dtype}")
        return cls([t.numel() for t in tensors], [names[t.dtype] for t in tensors])

    def _list(self, tensors, name):
        """The tensors' addresses, if they are the plan's."""
        if len(tensors) != len(self.counts):
            raise ValueError(f"{name}: expected {len(self.counts)} tensors, got {len(tensors)}")
        if ([t.dtype for t in tensors] != self._torch_dtypes
                or [t.numel() for t in tensors] != self.counts
                or [t.get_device() for t in tensors] != self._devices
                or not all([t.is_contiguous() for t in tensors])):
            for t, n, dtype in zip(tensors, self.counts, self._torch_dtypes):
                if (t.dtype is not dtype or t.numel() != n or t.get_device() != self._index
                        or not t.is_contiguous()):
                    raise ValueError(f"{name}: expected a contiguous {dtype} tensor of {n} values "
                                     f"on {self.device}, got {t.dtype} {tuple(t.shape)} with "
                                     f"strides {t.stride()} on {t.device}")
        return [t.data_ptr() for t in tensors]

    def _room(self):
        """The norm's place, and a workspace."""
        return (self._empty((), dtype=self._float, device=self.device),
                self._empty(self._workspace_floats, dtype=self._float, device=self.device))

    def norm(self, grads, stream=None):
        """The global norm, a device scalar."""
        if stream is not None:
            with self._on(stream, grads):
                return self.norm(grads)
        at = self._list(grads, "grads")
        norm, ws = self._room()
        _lib.lapl_clip_norm(self.handle, at, norm.data_ptr(), ws.data_ptr(), self.workspace_bytes,
                            self._raw_stream(self._index))
        return norm

    def clip(self, grads, max_norm, outs=None, stream=None):
        """Scales the gradients to a global norm of at most max_norm, in place or into ``outs``;
        returns the norm before that, a device scalar.  A norm that is not finite changes no
        value."""
        if stream is not None:
            with self._on(stream, [*grads, *(outs or [])]):
                return self.clip(grads, max_norm, outs)
        at = self._list(grads, "grads")
        to = None if outs is None else self._list(outs, "outs")
        norm, ws = self._room()
        _lib.lapl_clip_apply(self.handle, at, to, max_norm, norm.data_ptr(), ws.data_ptr(),
                             self.workspace_bytes, self._raw_stream(self._index))
        return norm
