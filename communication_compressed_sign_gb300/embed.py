"""ctypes binding of the input-layer operators (the C ABI in
include/lioncub_embed.h) and their torch-tensor wrappers.

:class:`TokenEmbedding` is the embedding lookup with scaling (and position
rows, and dropout) with its gradient by sorted tokens; :func:`dropout` and
:func:`dropout_backward` draw their mask from a counter-based generator
(:class:`Drop`) and never store it.  As in :mod:`.lioncub`, the functions
named ``lioncub_*`` keep the C names and raise :class:`LionCubError` with the
library's message; the wrappers check tensors, pass their pointers through and
allocate results with torch.  Results are not part of torch's autograd graph:
gradients come from the backward functions, called by hand (or from a
torch.autograd.Function of the caller's), and tensors that require a gradient
are refused while torch records one.
"""
from __future__ import annotations

import ctypes
import struct
from typing import NamedTuple

from . import lioncub
from .lioncub import ERR_STATE, OK, LionCubError

ROWS_BF16, ROWS_F32 = 0, 1
INDEX_I64, INDEX_I32 = 0, 1
MAX_VOCAB, MAX_DIM, MAX_TOKENS = 1 << 20, 1 << 16, 1 << 30
STATUS_INDEX = 8

# Every symbol include/lioncub_embed.h declares, for load checks.
EXPORTED = (
    "lioncub_embed_create", "lioncub_embed_forward", "lioncub_embed_backward", "lioncub_embed_status",
    "lioncub_embed_last_error", "lioncub_embed_destroy", "lioncub_dropout_forward", "lioncub_dropout_backward",
)


class Rows(ctypes.Structure):
    """lioncub_rows: a matrix whose row i starts stride * i elements after data."""
    _fields_ = [("data", ctypes.c_void_p), ("stride", ctypes.c_int64), ("type", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class TokenBatch(ctypes.Structure):
    """lioncub_token_batch: the places of a batch."""
    _fields_ = [("tokens", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("seq_len", ctypes.c_int64), ("first_position", ctypes.c_int64), ("index_type", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class DropSpec(ctypes.Structure):
    """lioncub_drop."""
    _fields_ = [("seed", ctypes.c_uint64), ("stream", ctypes.c_uint64), ("p", ctypes.c_float),
                ("reserved", ctypes.c_uint32)]


# The same three as bytes: a packed struct costs a third of a ctypes one, and a
# small call is bound by what the host does.
_pack_rows = struct.Struct("@Pqii").pack
_pack_batch = struct.Struct("@PPqqqii").pack
_pack_drop = struct.Struct("@QQfI").pack


class Drop(NamedTuple):
    """Dropout with probability p (to the nearest 1/65536), drawn from stream
    number `stream` of `seed`; give each (step, worker, layer) its own."""
    p: float
    seed: int
    stream: int = 0


_lib = None


def load() -> ctypes.CDLL:
    """The library with this header's functions declared (raises if it is missing)."""
    global _lib
    if _lib is None:
        L = lioncub.load()
        vp, i64 = ctypes.c_void_p, ctypes.c_int64
        rows = batch = drop = vp  # a struct's address: byref() of one, or its bytes
        L.lioncub_embed_create.argtypes = [ctypes.POINTER(vp), i64, i64, i64, i64, ctypes.c_float]
        L.lioncub_embed_forward.argtypes = [vp, batch, rows, rows, rows, drop, vp]
        L.lioncub_embed_backward.argtypes = [vp, batch, rows, rows, rows, rows, rows, drop, vp]
        L.lioncub_embed_status.argtypes = [vp, vp, vp]
        L.lioncub_embed_last_error.argtypes = [vp]
        L.lioncub_embed_destroy.argtypes = [vp]
        L.lioncub_embed_destroy.restype = None
        L.lioncub_dropout_forward.argtypes = [i64, i64, rows, rows, rows, drop, vp]
        L.lioncub_dropout_backward.argtypes = [i64, i64, rows, rows, drop, vp]
        for name in EXPORTED:
            if name != "lioncub_embed_destroy":
                getattr(L, name).restype = ctypes.c_int
        L.lioncub_embed_last_error.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _check(rc: int, h) -> None:
    if rc != OK:
        L = load()
        msg = L.lioncub_embed_last_error(h).decode() or L.lioncub_strerror(rc).decode()
        raise LionCubError(rc, msg)


def lioncub_embed_create(vocab: int, dim: int, positions: int, max_tokens: int, scale: float) -> int:
    h = ctypes.c_void_p()
    _check(load().lioncub_embed_create(ctypes.byref(h), vocab, dim, positions, max_tokens, scale), None)
    return h.value


def lioncub_embed_forward(h: int, batch, table, pos_table, out, drop, stream: int = 0) -> None:
    """batch, table, ...: structs as bytes or ctypes.byref(), None for NULL (likewise below)."""
    rc = (_lib or load()).lioncub_embed_forward(h, batch, table, pos_table, out, drop, stream or None)
    if rc:
        _check(rc, h)


def lioncub_embed_backward(h: int, batch, dout, base, grad, pos_base, pos_grad, drop, stream: int = 0) -> None:
    rc = (_lib or load()).lioncub_embed_backward(h, batch, dout, base, grad, pos_base, pos_grad, drop, stream or None)
    if rc:
        _check(rc, h)


def lioncub_embed_status(h: int, dst_ptr: int, stream: int = 0) -> None:
    _check(load().lioncub_embed_status(h, dst_ptr, stream or None), h)


def lioncub_embed_destroy(h: int) -> None:
    if h:
        load().lioncub_embed_destroy(h)


def lioncub_dropout_forward(rows: int, cols: int, x, residual, out, drop, stream: int = 0) -> None:
    rc = (_lib or load()).lioncub_dropout_forward(rows, cols, x, residual, out, drop, stream or None)
    if rc:
        _check(rc, None)


def lioncub_dropout_backward(rows: int, cols: int, dout, dx, drop, stream: int = 0) -> None:
    rc = (_lib or load()).lioncub_dropout_backward(rows, cols, dout, dx, drop, stream or None)
    if rc:
        _check(rc, None)


# ---- torch tensors -------------------------------------------------------------

# What the wrappers use of torch, looked up at their first call.
_torch = None
_row_types = _index_types = _raw_stream = _device = None


def _use_torch():
    global _torch, _row_types, _index_types, _raw_stream, _device
    import torch
    _row_types = {torch.bfloat16: ROWS_BF16, torch.float32: ROWS_F32}
    _index_types = {torch.int64: INDEX_I64, torch.int32: INDEX_I32}
    # the current stream's handle, without the Stream object that torch.cuda.current_stream() makes
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda device: torch.cuda.current_stream(device).cuda_stream)
    _device = torch.cuda.current_device
    _torch = torch


def _rows(t, name, nrows, cols, device):
    """A tensor (..., cols) of nrows rows on CUDA device number `device` as a
    packed Rows; a view, never a copy."""
    kind = _row_types.get(t.dtype)
    if kind is None or t.get_device() != device:
        raise ValueError(f"{name} must be a bfloat16 or float32 tensor on cuda:{device}")
    if t.requires_grad and _torch.is_grad_enabled():
        raise ValueError(f"{name} requires a gradient, but results are not part of torch's graph: "
                         "call under torch.no_grad() or pass a detached tensor")
    if not t.dim() or t.size(-1) != cols or t.numel() != nrows * cols:
        raise ValueError(f"{name} must have {nrows} rows of {cols} columns (got {tuple(t.shape)})")
    if t.is_contiguous():
        return _pack_rows(t.data_ptr(), cols, kind, 0)
    try:
        t = t.view(-1, cols)  # rows a fixed distance apart
    except RuntimeError:
        raise ValueError(f"{name}: its rows do not lie a fixed distance apart") from None
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: the columns of a row must be contiguous")
    return _pack_rows(t.data_ptr(), t.stride(0) if nrows > 1 else cols, kind, 0)


def _drop_spec(drop):
    if drop is None:
        return None
    p, seed, stream = drop
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"p must be in [0, 1] (got {p})")
    return _pack_drop(seed & 0xffffffffffffffff, stream & 0xffffffffffffffff, p, 0)


def _empty(shape, dtype, device, stream):
    """A result allocated for the stream that writes it."""
    if stream is None:
        return _torch.empty(shape, dtype=dtype, device=device)
    with _torch.cuda.stream(stream):
        return _torch.empty(shape, dtype=dtype, device=device)


class TokenEmbedding:
    """The embedding lookup drop(scale * table[token] + pos_table[position])
    of `vocab` token rows and `positions` position rows (0: none) of `dim`
    columns, and its gradient, for batches of at most max_tokens places.

    Tensors are CUDA tensors on the device that was current at construction:
    tokens int64 or int32, tables, activations and gradients bfloat16 or
    float32 with contiguous columns.  A negative token is an empty place.  The
    tables may be views of the flat parameter vector and the gradients views
    of a worker's flat gradient vector.  `stream` defaults to torch's current
    stream; calls to :meth:`backward` of one layer must be ordered.  The layer
    keeps the gradient's workspace, whose size goes by max_tokens, from
    construction on.
    """

    def __init__(self, vocab, dim, max_tokens, *, positions=0, scale=1.0):
        if _torch is None:
            _use_torch()
        self.vocab, self.dim, self.max_tokens = int(vocab), int(dim), int(max_tokens)
        self.positions, self.scale = int(positions), float(scale)
        self.h = None
        self.h = lioncub_embed_create(self.vocab, self.dim, self.positions, self.max_tokens, self.scale)
        self.device = _torch.device("cuda", _device())
        self._index = self.device.index

    def _batch(self, tokens, positions, seq_len, first_position):
        if not self.h:
            raise LionCubError(ERR_STATE, "the layer is closed")
        kind = _index_types.get(tokens.dtype)
        if kind is None or tokens.get_device() != self._index or not tokens.is_contiguous():
            raise ValueError(f"tokens must be a contiguous int64 or int32 tensor on {self.device}")
        n, at = tokens.numel(), 0
        if positions is not None:
            if (positions.dtype != tokens.dtype or positions.get_device() != self._index
                    or not positions.is_contiguous() or positions.numel() != n):
                raise ValueError("positions must be a contiguous tensor of tokens' type, size and device")
            at = positions.data_ptr()
        if seq_len is None:
            seq_len = max(1, tokens.size(-1)) if tokens.dim() else 1
        return n, _pack_batch(tokens.data_ptr(), at, n, seq_len, first_position, kind, 0)

    def forward(self, tokens, table, pos_table=None, *, positions=None, seq_len=None, first_position=0, drop=None,
                out=None, out_dtype=None, stream=None):
        """Rows for `tokens` (any shape): a tensor tokens.shape + (dim,), or `out`.

        table: (vocab, dim); pos_table: (positions, dim) of table's type, read
        at `positions` (tokens' shape and type) or, without them, at
        first_position + the place's index in its sequence of seq_len (the
        last dimension of tokens).  out_dtype: bfloat16 (default) or float32.
        """
        n, batch = self._batch(tokens, positions, seq_len, first_position)
        D, dev = self.dim, self._index
        # the tensors stay referenced until the launch, so that no result is allocated in an argument's memory
        rows = _rows(table, "table", self.vocab, D, dev)
        pos = None if pos_table is None else _rows(pos_table, "pos_table", self.positions, D, dev)
        if out is None:
            out = _empty((*tokens.shape, D), out_dtype or _torch.bfloat16, self.device, stream)
        lioncub_embed_forward(self.h, batch, rows, pos, _rows(out, "out", n, D, dev), _drop_spec(drop),
                              _raw_stream(dev) if stream is None else stream.cuda_stream)
        return out

    def backward(self, tokens, dout, grad, *, pos_grad=None, base=None, pos_base=None, positions=None, seq_len=None,
                 first_position=0, drop=None, stream=None):
        """Writes grad (vocab, dim) and, when given, pos_grad (positions, dim)
        from dout (tokens.shape + (dim,)), with the forward call's places and
        drop.  base / pos_base are added; passing grad itself as base adds in
        place and touches only the rows of the batch's tokens."""
        n, batch = self._batch(tokens, positions, seq_len, first_position)
        D, dev = self.dim, self._index
        g = _rows(grad, "grad", self.vocab, D, dev)
        b = None if base is None else _rows(base, "base", self.vocab, D, dev)
        pg = None if pos_grad is None else _rows(pos_grad, "pos_grad", self.positions, D, dev)
        pb = None if pos_base is None else _rows(pos_base, "pos_base", self.positions, D, dev)
        lioncub_embed_backward(self.h, batch, _rows(dout, "dout", n, D, dev), b, g, pb, pg, _drop_spec(drop),
                               _raw_stream(dev) if stream is None else stream.cuda_stream)
        return grad

    def status(self) -> int:
        """The status word (LIONCUB_STATUS_* and STATUS_INDEX bits; 0: all is well) after the calls
        before it on torch's current stream.  Synchronizes."""
        if not self.h:
            raise LionCubError(ERR_STATE, "the layer is closed")
        word = _torch.zeros(1, dtype=_torch.int32, device=self.device)
        lioncub_embed_status(self.h, word.data_ptr(), _raw_stream(self._index))
        return int(word.item())

    def close(self):
        if self.h:
            lioncub_embed_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _matrix(x, name):
    """(rows, cols, device number) of a tensor on the current CUDA device."""
    if _torch is None:
        _use_torch()
    dev = x.get_device()
    if dev < 0 or dev != _device():
        raise ValueError(f"{name} must be on the current CUDA device")
    if not x.dim():
        raise ValueError(f"{name} must have at least one dimension")
    cols = x.size(-1)
    return x.numel() // cols if cols else 0, cols, dev


def dropout(x, drop: Drop, *, residual=None, out=None, stream=None):
    """drop(x), plus `residual` (of the result's type) when given.  out: where
    to write (x itself, or the residual itself, is allowed); default a new
    tensor of residual's type, or x's."""
    rows, cols, dev = _matrix(x, "x")
    if out is None:
        out = _empty(x.shape, (x if residual is None else residual).dtype, x.device, stream)
    r = None if residual is None else _rows(residual, "residual", rows, cols, dev)
    lioncub_dropout_forward(rows, cols, _rows(x, "x", rows, cols, dev), r, _rows(out, "out", rows, cols, dev),
                            _drop_spec(drop), _raw_stream(dev) if stream is None else stream.cuda_stream)
    return out


def dropout_backward(dout, drop: Drop, *, out=None, stream=None):
    """The gradient of :func:`dropout` with respect to x, from the gradient of
    its result, with the same drop; out may be dout itself."""
    rows, cols, dev = _matrix(dout, "dout")
    if out is None:
        out = _empty(dout.shape, dout.dtype, dout.device, stream)
    lioncub_dropout_backward(rows, cols, _rows(dout, "dout", rows, cols, dev), _rows(out, "out", rows, cols, dev),
                             _drop_spec(drop), _raw_stream(dev) if stream is None else stream.cuda_stream)
    return out
