"""Python binding of include/rnnt_ops.h: the operators around the loss.

    LabelEmbedding   hL from the labels, and the table's gradient from dhL
    FrameNorm        hA from the encoder's frames (group norm + activation, channels last,
                     ragged lengths), and the frames' gradient from dhA
    LayerNorm        layer norm of frames or label rows, each by itself, and its gradients
    Orthogonalizer   the orthogonalised update of a weight matrix (Newton-Schulz products)
    GradClip         the norm of all gradients together, and their clipping
    AdamW            the AdamW update of many tensors, with the clipping's scale

Argument checks and marshalling only; each class owns the workspace, saved state and status
word of one problem size, as ``Rnnt`` does for the loss.  A call works on the current stream
unless one is given, writes into the tensor it is handed or into a new one (of that stream's
memory), and returns it.  An object's own buffers are made on the stream that is current then.
Calls of one object share its buffers and must not overlap on the GPU: use one object per
stream.  An object belongs to one GPU: its tensors live there, and it is the current device
when a call is made.  What a call writes of the tensors that it is handed counts as written for
autograd: a graph that still holds their old values refuses its backward pass, as it does after an
in-place operation of torch.
"""
from __future__ import annotations

import array
import copy
import ctypes
import functools
import importlib.util
import itertools
import operator
import os

import torch

from . import build as _build
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


class RnntLnDims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("C", ctypes.c_int),
                ("label_rows", ctypes.c_int), ("x_dtype", ctypes.c_int),
                ("y_dtype", ctypes.c_int), ("eps", ctypes.c_float),
                ("x_frame", ctypes.c_longlong), ("x_batch", ctypes.c_longlong),
                ("y_frame", ctypes.c_longlong), ("y_batch", ctypes.c_longlong)]


class RnntGradList(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int), ("count", ctypes.POINTER(ctypes.c_longlong)),
                ("dtype", ctypes.POINTER(ctypes.c_int))]


class RnntAdamwOpts(ctypes.Structure):
    _fields_ = [("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_float),
                ("lr", ctypes.c_float), ("decay", ctypes.c_float),
                ("decays", ctypes.POINTER(ctypes.c_float))]


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


@functools.lru_cache(None)
def _helper():
    """The functions of csrc/lists.cpp, or None where it was not built."""
    path = _build.lists_path()
    if not os.path.exists(path):
        return None
    spec = importlib.util.spec_from_file_location("rnnt_lists", path)
    try:
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
    except ImportError:  # (another build of torch under the same version)
        return None
    return module


class _Want:
    """What a tensor has to be: type, shape and strides (words: for csrc/lists.cpp)."""
    _CODES = {torch.float32: 0, torch.bfloat16: 1, torch.int32: 2}

    def __init__(self, dtype, shape, strides):
        self.dtype, self.layout = dtype, (shape, strides)
        self._words = array.array("q", [self._CODES[dtype], len(shape), *shape, *strides])
        self.at = self._words.buffer_info()[0]


def _signed(t):
    """Whether the tensor's memory has the other sign (a view that torch negates at its use)."""
    return isinstance(t, torch.Tensor) and t.is_neg()


def _dense(shape):
    """Strides of a dense tensor."""
    return torch.empty(shape, device="meta").stride()


class _Op:
    """Status word and workspace of one problem size."""

    def __init__(self, ws_bytes, what, device, works=True):
        # (0 bytes: invalid; works: whether a call takes the workspace)
        if ws_bytes == 0:
            raise RnntError(1, what)
        self.device = device
        self.ws = torch.empty(ws_bytes * works, dtype=torch.uint8, device=device)
        self.ws_bytes = ws_bytes
        self.status_word = torch.zeros(1, dtype=torch.int32, device=device)
        self._args = (self.ws.data_ptr(), ws_bytes, self.status_word.data_ptr())
        self._index = self.ws.device.index
        self._fast = _helper() if self.ws.is_cuda else None

    def _pointer(self, t, name, want, written=False):
        """_ptr of what is wanted (0.1 us where it is that, 0.5 by _ptr); counts what is written."""
        if self._fast is not None:
            p = self._fast.pointer(t, want.at, self._index, written)
            if p is not None:
                return p
        p = self._ptr(t, name, want.dtype, want.layout)
        if written:
            self._wrote(t)
        return p

    def _new(self, want, stream):
        """_empty of what is wanted."""
        if stream is None and self._fast is not None:
            return self._fast.empty(want.at, self._index)
        return self._empty(want.layout, want.dtype, stream)

    def _ptr(self, t, name, dtype, layout):
        """Data pointer of a tensor of the plan's GPU that has exactly this type and layout."""
        shape, strides = layout
        if (t.dtype is not dtype or t.shape != shape or t.get_device() != self._index
                or _signed(t)):
            raise ValueError(f"{name}: a tensor of {dtype} {tuple(shape)} on {self.ws.device} is "
                             f"needed, got {t.dtype} {tuple(t.shape)} on {t.device}"
                             + " with its sign left to do" * _signed(t))
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

    def _wrote(self, *ts):
        """Count these tensors, or lists of them, as written (0.15 us with csrc/lists.cpp)."""
        if self._fast is not None:
            return self._fast.wrote(*ts)
        flat = itertools.chain.from_iterable(t if type(t) is list else (t,) for t in ts)
        torch.autograd.graph.increment_version([t for t in flat if isinstance(t, torch.Tensor)])

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
        given = out
        if out is None:
            out = self._empty(self._rows, self._rt, stream)
        i, u = self._in(ids, U_len)
        _check(self._fwd(self._d, i, u, self._ptr(table, "table", self._tt, self._table),
                         self._ptr(out, "out", self._rt, self._rows), self._args[2],
                         self._stream(stream)), "rnnt_embed_fwd")
        self._wrote(given)
        return out

    def bwd(self, dout, ids, U_len=None, dtable=None, stream=None):
        """The table's gradient [V,D] fp32 from the rows' gradient."""
        given = dtable
        if dtable is None:
            dtable = self._empty(self._table, torch.float32, stream)
        i, u = self._in(ids, U_len)
        _check(self._bwd(self._d, i, u, self._ptr(dout, "dout", self._rt, self._rows),
                         self._ptr(dtable, "dtable", torch.float32, self._table), *self._args,
                         self._stream(stream)), "rnnt_embed_bwd")
        self._wrote(given)
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
        given = y
        if y is None:
            y = self._empty(self._y, self._t, stream)
        _check(self._fwd(self._d, self._ptr(x, "x", self._t, self._x),
                         *self._params(gamma, beta, T_len), self._ptr(y, "y", self._t, self._y),
                         self._saved, *self._args, self._stream(stream)), "rnnt_norm_fwd")
        self._wrote(given)
        return y

    def bwd(self, x, dy, gamma=None, beta=None, T_len=None, dx=None, dgamma=None, dbeta=None,
            stream=None):
        """(dx, dgamma, dbeta) for the x and T_len of the last fwd."""
        given = dx, dgamma, dbeta
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
        self._wrote(*given)
        return dx, dgamma, dbeta


class LayerNorm(_Op):
    """y = gamma * xh + beta, xh a row of x [B,T,C] less its mean, over its deviation.

    Rows t < lengths[b] exist, or with label_rows (the rows of LabelEmbedding) rows
    u <= lengths[b]; the others' y and dx are 0.  dtype: of x and dx; out_dtype: of y and dy
    (None: dtype).  x_strides, y_strides: (batch, frame) strides in elements of x and dx, and of
    y and dy (None, or 0 for either: dense).  fwd keeps the statistics that bwd reads.
    """

    def __init__(self, B, T, C, dtype="bf16", out_dtype=None, eps=1e-5, label_rows=False,
                 x_strides=None, y_strides=None, device="cuda"):
        xcode, xt = _dtype(dtype)
        ycode, yt = _dtype(dtype if out_dtype is None else out_dtype)
        xs, ys = _strides(x_strides, T, C), _strides(y_strides, T, C)
        self.dims = _dims(RnntLnDims, B, T, C, int(label_rows), xcode, ycode, eps, xs[1], xs[0],
                          ys[1], ys[0])
        self._d = ctypes.byref(self.dims)
        lib = load()
        super().__init__(lib.rnnt_ln_workspace_bytes(self._d), "LayerNorm(dims)", device)
        self.saved = torch.empty(lib.rnnt_ln_saved_bytes(self._d), dtype=torch.uint8,
                                 device=device)
        self._saved = self.saved.data_ptr()
        self._fwd, self._bwd = lib.rnnt_ln_fwd, lib.rnnt_ln_bwd
        self._x = _Want(xt, (B, T, C), (xs[0], xs[1], 1))
        self._y = _Want(yt, (B, T, C), (ys[0], ys[1], 1))
        self._c = _Want(torch.float32, (C,), (1,))
        self._len = _Want(torch.int32, (B,), (1,))

    def _opt(self, t, name, want):
        return None if t is None else self._pointer(t, name, want)

    def fwd(self, x, gamma=None, beta=None, lengths=None, y=None, stream=None):
        """y [B,T,C]; gamma, beta [C] fp32 or None; lengths [B] int32 or None (every row)."""
        if y is None:
            y = self._new(self._y, stream)
        _check(self._fwd(self._d, self._pointer(x, "x", self._x),
                         self._opt(gamma, "gamma", self._c), self._opt(beta, "beta", self._c),
                         self._opt(lengths, "lengths", self._len),
                         self._pointer(y, "y", self._y, True), self._saved, self._args[2],
                         self._stream(stream)), "rnnt_ln_fwd")
        return y

    def bwd(self, x, dy, gamma=None, lengths=None, dx=None, dgamma=None, dbeta=None, stream=None):
        """(dx, dgamma, dbeta) for the x and lengths of the last fwd."""
        if dx is None:
            dx = self._new(self._x, stream)
        if dgamma is None:
            dgamma = self._new(self._c, stream)
        if dbeta is None:
            dbeta = self._new(self._c, stream)
        _check(self._bwd(self._d, self._pointer(x, "x", self._x), self._pointer(dy, "dy", self._y),
                         self._opt(gamma, "gamma", self._c),
                         self._opt(lengths, "lengths", self._len), self._saved,
                         self._pointer(dx, "dx", self._x, True),
                         self._pointer(dgamma, "dgamma", self._c, True),
                         self._pointer(dbeta, "dbeta", self._c, True), *self._args,
                         self._stream(stream)), "rnnt_ln_bwd")
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
        given = out
        if out is None:
            out = self._empty(self._out, self._ot, stream)
            out = out[0] if flat and self.dims.batch == 1 else out
        o = out[None] if out.dim() == 2 else out
        _check(self._run(self._d, self._ptr(G[None] if flat else G, "G", self._it, self._in),
                         self._ptr(o, "out", self._ot, self._out), *self._args,
                         self._stream(stream)), "rnnt_orth")
        self._wrote(given)
        return out


def _listed(ts):
    return ts if type(ts) is list else list(ts)


_PAIR = _Want(torch.float32, (2,), (1,))
_ONE = _Want(torch.float32, (1,), (1,))


class _Kind:
    """What a list's tensors have to be: their types and shapes."""

    def __init__(self, name, types, shapes):
        self.name, self.types = name, types
        words = []
        for t, k in zip(types, shapes):
            words += [int(t is torch.bfloat16), len(k), *k]
        self._words = array.array("q", words)
        self.at = self._words.buffer_info()[0]

    def called(self, name):
        """The same of another list."""
        other = copy.copy(self)
        other.name = name
        return other


class _ListOp(_Op):
    """An operator on a list of dense tensors of fixed shapes."""

    def __init__(self, shapes, dtype, what, device, works=True):
        self._shapes = [torch.Size(k) for k in shapes]
        self._n = n = len(self._shapes)
        names = [dtype] * n if isinstance(dtype, str) else list(dtype)
        if len(names) != n:
            raise ValueError(f"{len(names)} dtypes for {n} tensors")
        codes = [_dtype(k) for k in names]
        self._count = (ctypes.c_longlong * n)(*[k.numel() for k in self._shapes])
        self._codes = (ctypes.c_int * n)(*[c for c, _ in codes])
        self.list = RnntGradList(n, self._count, self._codes)
        self._l = ctypes.byref(self.list)
        self._grads = self._kind("grads", [t for _, t in codes])
        self._take_list = _helper() and _helper().take
        super().__init__(load().rnnt_clip_workspace_bytes(self._l), what, device, works)

    def _kind(self, name, types):
        return _Kind(name, types, self._shapes)

    def _take(self, lists, kinds, layouts):
        """The data pointers of lists (a tuple), one list after another: an array, and its address
        for the C side.  layouts: the kinds' addresses."""
        n = self._n
        a = array.array("Q", bytes(8 * n * len(lists)))
        at = a.buffer_info()[0]
        if self._take_list is None:
            for k, (ts, kind) in enumerate(zip(lists, kinds)):
                if not self._fits(ts, kind):
                    self._refuse(ts, kind)
                a[k * n:(k + 1) * n] = array.array("Q", [t.data_ptr() for t in ts])
        else:
            bad = self._take_list(lists, layouts, n, self._index, at)
            if bad >= 0:
                self._refuse(lists[bad], kinds[bad])
        return a, at

    def _fits(self, ts, kind):
        return len(ts) == self._n and all(
            t.shape == k and t.dtype is d and t.get_device() == self._index and t.is_contiguous()
            and not _signed(t) for t, k, d in zip(ts, self._shapes, kind.types))

    def _refuse(self, ts, kind):
        if len(ts) != self._n:
            raise ValueError(f"{kind.name}: {len(ts)} tensors, the plan has {self._n}")
        for i, (t, k, d) in enumerate(zip(ts, self._shapes, kind.types)):
            if not (t.shape == k and t.dtype is d and t.get_device() == self._index
                    and t.is_contiguous()):
                raise ValueError(f"{kind.name}[{i}]: a dense tensor of {d} {tuple(k)} on "
                                 f"{self.ws.device} is needed, got {t.dtype} {tuple(t.shape)} of "
                                 f"strides {t.stride()} on {t.device}")
        raise ValueError(f"{kind.name}: dense CUDA tensors of resolved sign are needed")


class GradClip(_ListOp):
    """norm = the 2-norm of all gradients together; scale = min(1, max_norm / (norm + eps)).

    shapes: of the tensors, in the order of every call's list.  dtype: the gradients' ("f32" or
    "bf16"), one for all or a list.  Results are fp32 [2] tensors (norm, scale).
    """

    def __init__(self, shapes, max_norm=1.0, dtype="f32", eps=1e-6, device="cuda"):
        super().__init__(shapes, dtype, "GradClip(shapes)", device)
        self.max_norm, self.eps = float(max_norm), float(eps)
        if not self.max_norm >= 0 or not 0 <= self.eps < float("inf") or not (
                self.max_norm or self.eps):
            raise ValueError(f"max_norm {max_norm}, eps {eps}: not negative, not both 0")
        self._kinds = self._grads, self._grads.called("into")
        self._layouts = tuple(k.at for k in self._kinds)
        self._clip = load().rnnt_clip

    def _call(self, grads, into, out, stream):
        if out is None:
            out = self._new(_PAIR, stream)
        lists = [_listed(grads)]
        if into is not None and into is not grads:
            lists.append(_listed(into))
        held, g = self._take(tuple(lists), self._kinds, self._layouts)
        w = None if into is None else g + 8 * self._n * (len(lists) - 1)
        _check(self._clip(self._l, g, w, self.max_norm, self.eps,
                          self._pointer(out, "out", _PAIR, True), self._args[0],
                          self.ws_bytes, self._stream(stream)), "rnnt_clip")
        if into is not None:
            self._wrote(lists[-1])
        return out

    def norm(self, grads, out=None, stream=None):
        """(norm, scale) alone, as AdamW.step takes it; the gradients stay as they are."""
        return self._call(grads, None, out, stream)

    def clip(self, grads, into=None, out=None, stream=None):
        """The same, and the gradients times the scale, in place or into other tensors."""
        return self._call(grads, grads if into is None else into, out, stream)


class AdamW(_ListOp):
    """The AdamW update of a list of fp32 tensors (see include/rnnt_ops.h).

    shapes: of the tensors, in the order of every call's lists.  grad_dtype: "f32" or "bf16", one
    for all or a list.  weight_decay: one number for all or a list.  m, v: lists of fp32 tensors
    to keep the moments in (None: new ones, zeros); steps: updates they have taken.
    """

    def __init__(self, shapes, grad_dtype="f32", betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01,
                 m=None, v=None, steps=0, device="cuda"):
        super().__init__(shapes, grad_dtype, "AdamW(shapes)", device, works=False)
        n = len(self._shapes)
        if not (0 <= betas[0] < 1 and 0 <= betas[1] < 1 and 0 <= eps < float("inf")):
            raise ValueError(f"betas {betas}, eps {eps}: out of range")
        if not 0 <= steps < (1 << 31) - 1:
            raise ValueError(f"steps = {steps}: out of range")
        one = isinstance(weight_decay, (int, float))
        if not one and len(weight_decay) != n:
            raise ValueError(f"{len(weight_decay)} weight decays for {n} tensors")
        self._decays = None if one else (ctypes.c_float * n)(*weight_decay)
        self.opts = RnntAdamwOpts(betas[0], betas[1], eps, 0.0, weight_decay if one else 0.0,
                                  self._decays)
        self._o = ctypes.byref(self.opts)
        params = self._kind("params", [torch.float32] * n)
        self._kinds = (params, self._grads, params.called("m"), params.called("v"),
                       self._kind("low", [torch.bfloat16] * n))
        self._layouts = tuple(k.at for k in self._kinds)
        new = lambda: [torch.zeros(k, device=device) for k in self._shapes]  # noqa: E731
        self._moments = tuple(list(new() if k is None else k) for k in (m, v))
        self._counts = torch.tensor([int(steps), 0], dtype=torch.int32, device=device)
        self._steps = self._counts.data_ptr()
        self._run = load().rnnt_adamw

    @property
    def m(self):
        """The first moments (to resume: copy into them)."""
        return tuple(self._moments[0])

    @property
    def v(self):
        """The second moments."""
        return tuple(self._moments[1])

    @property
    def steps(self):
        """int32 [2] on the device: the updates taken so far, and a word of the library's."""
        return self._counts

    def step(self, params, grads, lr, clip=None, low=None, stream=None):
        """One update of params in place.

        lr: a number, or a device fp32 tensor of one element (a captured call reads it again at
        every replay); clip: GradClip's (norm, scale); low: tensors for the bf16 copies of params,
        an entry or all of them None.
        """
        if isinstance(lr, torch.Tensor):
            lr = self._pointer(lr.reshape(1), "lr", _ONE)
        else:
            self.opts.lr, lr = float(lr), None
        params = _listed(params)
        lists, held_l, w = (params, _listed(grads), *self._moments), None, None
        if low is not None:
            low = _listed(low)
            if any(map(operator.is_, low, itertools.repeat(None))):
                held_l, w = self._some(low)
            else:
                lists = *lists, low
        held, p = self._take(lists, self._kinds, self._layouts)
        size = 8 * self._n
        if len(lists) == 5:
            w = p + 4 * size
        c = None if clip is None else self._pointer(clip, "clip", _PAIR)
        _check(self._run(self._l, self._o, p, p + size, p + 2 * size, p + 3 * size, w, lr, c,
                         self._steps, self._stream(stream)), "rnnt_adamw")
        self._wrote(params, *self._moments, low)

    def _some(self, low):
        """The pointers of copies that only some tensors have."""
        if len(low) != self._n:
            raise ValueError(f"low: {len(low)} tensors, the plan has {self._n}")
        a = array.array("Q", [0 if t is None else self._ptr(
            t, f"low[{i}]", torch.bfloat16, (k, _dense(k))) for i, (t, k) in
            enumerate(zip(low, self._shapes))])
        return a, a.buffer_info()[0]


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
