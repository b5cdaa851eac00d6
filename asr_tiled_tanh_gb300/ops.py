"""Python binding of include/rnnt_ops.h: the operators around the loss.

    LabelEmbedding   hL from the labels, and the table's gradient from dhL
    FrameNorm        hA from the encoder's frames (group norm + activation, channels last,
                     ragged lengths), and the frames' gradient from dhA
    Orthogonalizer   the orthogonalised update of a weight matrix (Newton-Schulz products)

Argument checks and marshalling only; each class owns the workspace, saved state and status
word of one problem size, as ``Rnnt`` does for the loss.  A call works on the current stream
unless one is given, writes into the tensor it is handed or into a new one (of that stream's
memory), and returns it.  An object's own buffers are made on the stream that is current then.
Calls of one object share its buffers and must not overlap on the GPU: use one object per
stream.  An object belongs to one GPU: its tensors live there, and it is the current device
when a call is made.
"""
from __future__ import annotations

import ctypes

import torch

from .binding import RNNT_BF16, RNNT_F32, RnntError, _check, load

_DTYPES = {"f32": (RNNT_F32, torch.float32), "bf16": (RNNT_BF16, torch.bfloat16)}
_ACTS = {"none": 0, "silu": 1, "relu": 2}


class RnntEmbedDims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("U1", ctypes.c_int), ("V", ctypes.c_int),
                ("D", ctypes.c_int), ("blank", ctypes.c_int), ("sos", ctypes.c_int),
                ("table_dtype", ctypes.c_int), ("row_dtype", ctypes.c_int),
                ("scale", ctypes.c_float), ("ld_table", ctypes.c_longlong),
                ("ld_rows", ctypes.c_longlong)]


class RnntNormDims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("C", ctypes.c_int),
                ("G", ctypes.c_int), ("act", ctypes.c_int), ("dtype", ctypes.c_int),
                ("eps", ctypes.c_float), ("x_frame", ctypes.c_longlong),
                ("x_batch", ctypes.c_longlong), ("y_frame", ctypes.c_longlong),
                ("y_batch", ctypes.c_longlong)]


class RnntOrthDims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int), ("cols", ctypes.c_int), ("batch", ctypes.c_int),
                ("in_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int), ("steps", ctypes.c_int),
                ("eps", ctypes.c_float), ("in_ld", ctypes.c_longlong),
                ("in_batch", ctypes.c_longlong), ("out_ld", ctypes.c_longlong),
                ("out_batch", ctypes.c_longlong)]


# Handle of a device's current stream.  (torch.cuda.current_stream builds a Stream object, 3.8 us
# of a 10 us call; this is what its own compiled code takes.)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


_current_device = torch.cuda.current_device


def _dtype(name):
    try:
        return _DTYPES[name]
    except KeyError:
        raise ValueError(f"dtype {name!r}: one of {sorted(_DTYPES)}") from None


def _dims(struct, *values):
    """The C struct of these values; whole numbers that its fields cannot hold are refused."""
    d = struct(*values)
    for (name, _), v in zip(struct._fields_, values):
        if isinstance(v, int) and getattr(d, name) != v and not isinstance(getattr(d, name), float):
            raise ValueError(f"{name} = {v}: out of range")
    return d


def _strides(given, rows, width):
    """(batch, row) strides of rows of `width` elements; None or 0: dense, as in C."""
    batch, row = given or (0, 0)
    row = row or width
    return batch or rows * row, row


class _Op:
    """Status word and workspace of one problem size."""

    def __init__(self, ws_bytes, what, device):
        if ws_bytes == 0:
            raise RnntError(1, what)
        self.device = device
        self.ws = torch.empty(ws_bytes, dtype=torch.uint8, device=device)
        self.ws_bytes = ws_bytes
        self.status_word = torch.zeros(1, dtype=torch.int32, device=device)
        self._args = (self.ws.data_ptr(), ws_bytes, self.status_word.data_ptr())
        self._index = self.ws.device.index

    def _ptr(self, t, name, dtype, layout):
        """Data pointer of a tensor of the plan's GPU that has exactly this type and layout."""
        shape, strides = layout
        if t.dtype is not dtype or t.shape != shape or t.get_device() != self._index:
            raise ValueError(f"{name}: a tensor of {dtype} {tuple(shape)} on {self.ws.device} is "
                             f"needed, got {t.dtype} {tuple(t.shape)} on {t.device}")
        if t.stride() != strides:
            # (the stride of a dimension of length 1 is never used)
            if any(n > 1 and a != b for n, a, b in zip(shape, t.stride(), strides)):
                raise ValueError(f"{name}: strides {strides} are needed, got {t.stride()}")
        return t.data_ptr()

    def _stream(self, stream):
        """Handle of the stream to work on: the one given, else the device's current one."""
        # (a launch goes to the current device, wherever its pointers and stream belong)
        if _current_device() != self._index:
            raise ValueError(f"the plan is of {self.ws.device}, the current device is "
                             f"cuda:{_current_device()}")
        if stream is None:
            return _raw_stream(self._index)
        return stream if isinstance(stream, int) else stream.cuda_stream

    def _empty(self, layout, dtype, stream):
        """A new tensor for a call on `stream` to write."""
        shape, strides = layout
        if stream is None:
            return torch.empty_strided(shape, strides, dtype=dtype, device=self.device)
        # (memory is ordered on the stream it was asked for: from the current one's it could
        # be a block that the current stream still uses)
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=self.ws.device)
        with torch.cuda.stream(stream):
            return torch.empty_strided(shape, strides, dtype=dtype, device=self.device)

    def status(self, stream=None):
        """(status code, raw word) of every call so far; synchronizes the stream."""
        w = ctypes.c_int32(0)
        code = load().rnnt_ops_status(self.status_word.data_ptr(), self._stream(stream),
                                      ctypes.byref(w))
        return code, int(w.value)


class LabelEmbedding(_Op):
    """hL[b,u] = scale * E[id(b,u)] for u <= U_len[b], else 0 (id(b,0) = blank with sos).

    B, U1, V, D: samples, label positions, labels, width.  dtype: of the table; out_dtype: of
    the rows and of their gradient.  ld_table, ld_rows: row strides in elements (0: D).
    """

    def __init__(self, B, U1, V, D, dtype="bf16", out_dtype="bf16", scale=1.0, sos=True, blank=0,
                 ld_table=0, ld_rows=0, device="cuda"):
        tcode, self._tt = _dtype(dtype)
        rcode, self._rt = _dtype(out_dtype)
        self.dims = _dims(RnntEmbedDims, B, U1, V, D, blank, int(sos), tcode, rcode, scale,
                          ld_table, ld_rows)
        self._d = ctypes.byref(self.dims)
        lib = load()
        super().__init__(lib.rnnt_embed_workspace_bytes(self._d), "LabelEmbedding(dims)", device)
        self._fwd, self._bwd = lib.rnnt_embed_fwd, lib.rnnt_embed_bwd
        lt, lr = ld_table or D, ld_rows or D
        self._ids = ((B, U1), (U1, 1))
        self._len = ((B,), (1,))
        self._table = ((V, D), (lt, 1))
        self._rows = ((B, U1, D), (U1 * lr, lr, 1))

    def _in(self, ids, U_len):
        return (self._ptr(ids, "ids", torch.int32, self._ids),
                None if U_len is None else self._ptr(U_len, "U_len", torch.int32, self._len))

    def fwd(self, table, ids, U_len=None, out=None, stream=None):
        """The rows [B,U1,D] of ids [B,U1] int32; U_len [B] int32 or None (every row)."""
        if out is None:
            out = self._empty(self._rows, self._rt, stream)
        i, u = self._in(ids, U_len)
        _check(self._fwd(self._d, i, u, self._ptr(table, "table", self._tt, self._table),
                         self._ptr(out, "out", self._rt, self._rows), self._args[2],
                         self._stream(stream)), "rnnt_embed_fwd")
        return out

    def bwd(self, dout, ids, U_len=None, dtable=None, stream=None):
        """The table's gradient [V,D] fp32 from the rows' gradient."""
        if dtable is None:
            dtable = self._empty(self._table, torch.float32, stream)
        i, u = self._in(ids, U_len)
        _check(self._bwd(self._d, i, u, self._ptr(dout, "dout", self._rt, self._rows),
                         self._ptr(dtable, "dtable", torch.float32, self._table), *self._args,
                         self._stream(stream)), "rnnt_embed_bwd")
        return dtable


class FrameNorm(_Op):
    """y = act(gamma * xh + beta), xh the group norm of x [B,T,C] over the frames t < T_len[b].

    x_strides, y_strides: (batch, frame) strides in elements of x and dx, and of y and dy
    (None, or 0 for either: dense).  fwd keeps the statistics that bwd reads.
    """

    def __init__(self, B, T, C, G, act="silu", dtype="bf16", eps=1e-5, x_strides=None,
                 y_strides=None, device="cuda"):
        code, self._t = _dtype(dtype)
        if act not in _ACTS:
            raise ValueError(f"act {act!r}: one of {sorted(_ACTS)}")
        xs, ys = _strides(x_strides, T, C), _strides(y_strides, T, C)
        self.dims = _dims(RnntNormDims, B, T, C, G, _ACTS[act], code, eps, xs[1], xs[0], ys[1],
                          ys[0])
        self._d = ctypes.byref(self.dims)
        lib = load()
        super().__init__(lib.rnnt_norm_workspace_bytes(self._d), "FrameNorm(dims)", device)
        self.saved = torch.empty(lib.rnnt_norm_saved_bytes(self._d), dtype=torch.uint8,
                                 device=device)
        self._saved = self.saved.data_ptr()
        self._fwd, self._bwd = lib.rnnt_norm_fwd, lib.rnnt_norm_bwd
        self._x = ((B, T, C), (xs[0], xs[1], 1))
        self._y = ((B, T, C), (ys[0], ys[1], 1))
        self._c = ((C,), (1,))
        self._len = ((B,), (1,))

    def _params(self, gamma, beta, T_len):
        f = torch.float32
        return (None if gamma is None else self._ptr(gamma, "gamma", f, self._c),
                None if beta is None else self._ptr(beta, "beta", f, self._c),
                None if T_len is None else self._ptr(T_len, "T_len", torch.int32, self._len))

    def fwd(self, x, gamma=None, beta=None, T_len=None, y=None, stream=None):
        """y [B,T,C]; gamma, beta [C] fp32 or None; T_len [B] int32 or None (every frame)."""
        if y is None:
            y = self._empty(self._y, self._t, stream)
        _check(self._fwd(self._d, self._ptr(x, "x", self._t, self._x),
                         *self._params(gamma, beta, T_len), self._ptr(y, "y", self._t, self._y),
                         self._saved, *self._args, self._stream(stream)), "rnnt_norm_fwd")
        return y

    def bwd(self, x, dy, gamma=None, beta=None, T_len=None, dx=None, dgamma=None, dbeta=None,
            stream=None):
        """(dx, dgamma, dbeta) for the x and T_len of the last fwd."""
        if dx is None:
            dx = self._empty(self._x, self._t, stream)
        f = torch.float32
        if dgamma is None:
            dgamma = self._empty(self._c, f, stream)
        if dbeta is None:
            dbeta = self._empty(self._c, f, stream)
        pg, pb = (self._ptr(dgamma, "dgamma", f, self._c), self._ptr(dbeta, "dbeta", f, self._c))
        _check(self._bwd(self._d, self._ptr(x, "x", self._t, self._x),
                         self._ptr(dy, "dy", self._t, self._y), *self._params(gamma, beta, T_len),
                         self._saved, self._ptr(dx, "dx", self._t, self._x), pg, pb, *self._args,
                         self._stream(stream)), "rnnt_norm_bwd")
        return dx, dgamma, dbeta


class Orthogonalizer(_Op):
    """O = the Newton-Schulz iterate of G / |G|_F after `steps` steps (see include/rnnt_ops.h).

    G [batch,rows,cols], or [rows,cols] with batch = 1.  in_strides, out_strides: (batch, row)
    strides in elements (None, or 0 for either: dense).
    """

    def __init__(self, rows, cols, batch=1, dtype="f32", out_dtype="bf16", steps=5, eps=1e-7,
                 in_strides=None, out_strides=None, device="cuda"):
        icode, self._it = _dtype(dtype)
        ocode, self._ot = _dtype(out_dtype)
        i, o = _strides(in_strides, rows, cols), _strides(out_strides, rows, cols)
        self.dims = _dims(RnntOrthDims, rows, cols, batch, icode, ocode, steps, eps, i[1], i[0],
                          o[1], o[0])
        self._d = ctypes.byref(self.dims)
        lib = load()
        super().__init__(lib.rnnt_orth_workspace_bytes(self._d), "Orthogonalizer(dims)", device)
        self._run = lib.rnnt_orth
        self._in = ((batch, rows, cols), (i[0], i[1], 1))
        self._out = ((batch, rows, cols), (o[0], o[1], 1))

    def run(self, G, out=None, stream=None):
        flat = G.dim() == 2
        if out is None:
            out = self._empty(self._out, self._ot, stream)
            out = out[0] if flat and self.dims.batch == 1 else out
        o = out[None] if out.dim() == 2 else out
        _check(self._run(self._d, self._ptr(G[None] if flat else G, "G", self._it, self._in),
                         self._ptr(o, "out", self._ot, self._out), *self._args,
                         self._stream(stream)), "rnnt_orth")
        return out


class RnntTestingOrth(ctypes.Structure):
    """What rnnt_orth runs for a size (include/rnnt_testing.h)."""
    _fields_ = [("thin", ctypes.c_int), ("exact", ctypes.c_int), ("splits", ctypes.c_int),
                ("bn", ctypes.c_int * 3), ("units", ctypes.c_int * 3), ("halved", ctypes.c_int),
                ("blocks", ctypes.c_int)]


def rnnt_testing_orth_plan(dims) -> RnntTestingOrth:
    out = RnntTestingOrth()
    _check(load().rnnt_testing_orth_plan(ctypes.byref(dims), ctypes.byref(out)),
           "rnnt_testing_orth_plan")
    return out
