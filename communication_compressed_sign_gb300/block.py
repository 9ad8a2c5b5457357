"""ctypes binding of the block operators (the C ABI in include/lioncub_block.h)
and their torch-tensor wrappers.

:class:`RmsNorm` is the root-mean-square norm with the residual's addition and
its gradient, :class:`Packed` a matrix in 8 bits with scales (:func:`pack8`,
:func:`unpack8`), :func:`activation` and :func:`activation_backward` a SiLU or
GELU, gated or not, and :class:`Rotary` rotary positions.  A norm and an
activation can leave what their backward pass needs in 8 bits.  As in
:mod:`.embed`, results are not part of torch's autograd graph and gradients come
from the backward functions, called by hand: tensors that require a gradient while
torch records one, or have a forward-mode tangent, are refused.  A result that is a
lazy clone gets memory of its own first, by a copy on torch's current stream.
:func:`load` gives the library with the C functions declared.
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple

from . import embed
from .embed import _empty
from .lioncub import ERR_STATE, OK, LionCubError

CODES_INT8, CODES_E4M3 = 0, 1
SILU, GELU = 0, 1
SCALING_NONE, SCALING_LINEAR, SCALING_BASE, SCALING_PARTS = range(4)
NORM_MAX_DIM, ROTARY_MAX_DIM = 16384, 1024

# Every symbol include/lioncub_block.h declares, for load checks.
EXPORTED = (
    "lioncub_rms_norm_create", "lioncub_rms_norm_forward", "lioncub_rms_norm_backward", "lioncub_rms_norm_status",
    "lioncub_rms_norm_destroy", "lioncub_pack8", "lioncub_unpack8", "lioncub_activation_forward",
    "lioncub_activation_backward", "lioncub_rotary_frequencies", "lioncub_rotary_create", "lioncub_rotary_apply",
    "lioncub_rotary_destroy", "lioncub_block_last_error",
)


class PackedRows(ctypes.Structure):
    """lioncub_packed: a matrix in 8 bits."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("stride", ctypes.c_int64),
                ("scale_stride", ctypes.c_int64), ("group", ctypes.c_int32), ("format", ctypes.c_int32)]


class Heads(ctypes.Structure):
    """lioncub_heads."""
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64), ("place_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("heads", ctypes.c_int32), ("type", ctypes.c_int32)]


class Sequences(ctypes.Structure):
    """lioncub_sequences."""
    _fields_ = [("positions", ctypes.c_void_p), ("batch", ctypes.c_int64), ("seq_len", ctypes.c_int64),
                ("first_position", ctypes.c_int64), ("index_type", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class ScalingSpec(ctypes.Structure):
    """lioncub_rotary_scaling."""
    _fields_ = [("factor", ctypes.c_double), ("length", ctypes.c_double), ("low", ctypes.c_double), ("high", ctypes.c_double),
                ("kind", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_lib = None


def load() -> ctypes.CDLL:
    """The library with this header's functions declared (raises if it is missing)."""
    global _lib
    if _lib is None:
        L = embed.load()
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        L.lioncub_rms_norm_create.argtypes = [ctypes.POINTER(vp), i64, ctypes.c_float]
        L.lioncub_rms_norm_forward.argtypes = [vp, i64] + [vp] * 9
        L.lioncub_rms_norm_backward.argtypes = [vp, i64] + [vp] * 11
        L.lioncub_rms_norm_status.argtypes = [vp, vp, vp]
        L.lioncub_pack8.argtypes = L.lioncub_unpack8.argtypes = [i64, i64, vp, vp, vp]
        L.lioncub_activation_forward.argtypes = [i64, i64, i32] + [vp] * 6
        L.lioncub_activation_backward.argtypes = [i64, i64, i32] + [vp] * 9
        L.lioncub_rotary_frequencies.argtypes = [i64, ctypes.c_double, vp, vp]
        L.lioncub_rotary_create.argtypes = [ctypes.POINTER(vp), i64, i64, vp, ctypes.c_float, i32]
        L.lioncub_rotary_apply.argtypes = [vp] * 6 + [i32, vp]
        for name in EXPORTED:
            getattr(L, name).restype = i32
        for name in ("lioncub_rms_norm_destroy", "lioncub_rotary_destroy"):
            getattr(L, name).argtypes = [vp]
            getattr(L, name).restype = None
        L.lioncub_block_last_error.argtypes = []
        L.lioncub_block_last_error.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _check(rc: int) -> None:
    if rc != OK:
        L = load()
        raise LionCubError(rc, L.lioncub_block_last_error().decode() or L.lioncub_strerror(rc).decode())


def lioncub_rms_norm_create(dim: int, eps: float) -> int:
    h = ctypes.c_void_p()
    _check(load().lioncub_rms_norm_create(ctypes.byref(h), dim, eps))
    return h.value


def lioncub_rms_norm_status(h: int, dst_ptr: int, stream: int = 0) -> None:
    _check(load().lioncub_rms_norm_status(h, dst_ptr, stream or None))


def lioncub_rms_norm_destroy(h: int) -> None:
    if h:
        load().lioncub_rms_norm_destroy(h)


def lioncub_rotary_frequencies(rotary_dim: int, base: float, scaling=None) -> list[float]:
    out = (ctypes.c_double * max(1, min(rotary_dim, ROTARY_MAX_DIM) // 2))()
    _check(load().lioncub_rotary_frequencies(rotary_dim, base, None if scaling is None else ctypes.byref(scaling), out))
    return list(out)


def lioncub_rotary_create(head_dim: int, rotary_dim: int, frequencies, magnitude: float, interleaved: bool) -> int:
    h = ctypes.c_void_p()
    table = (ctypes.c_double * len(frequencies))(*frequencies)
    _check(load().lioncub_rotary_create(ctypes.byref(h), head_dim, rotary_dim, table, magnitude, int(interleaved)))
    return h.value


def lioncub_rotary_destroy(h: int) -> None:
    if h:
        load().lioncub_rotary_destroy(h)


# ---- torch tensors -------------------------------------------------------------
#
# The module _tensors reads what a call needs from the tensors and calls the library.

_torch = None
_tensors = None
_device = None


def _use_torch():
    global _torch, _tensors, _device
    embed._use_torch()
    import torch
    try:
        from . import _tensors as module
    except ImportError as e:
        raise RuntimeError("the _tensors module is missing or does not fit this torch: run "
                           "python -m communication_compressed_sign_gb300.build") from e
    L = load()
    module.bind(*(ctypes.cast(getattr(L, f"lioncub_{name}"), ctypes.c_void_p).value for name in (
        "rms_norm_forward", "rms_norm_backward", "pack8", "unpack8", "activation_forward", "activation_backward", "rotary_apply")))
    # the current device's number, without what torch.cuda.current_device() does before
    _device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _tensors, _torch = module, torch


def _raw(dev, stream):
    return embed._raw_stream(dev) if stream is None else stream.cuda_stream


class Packed:
    """A matrix in 8 bits: codes (..., cols), int8 or float8_e4m3fn, and fp32
    scales (..., groups), one for each `group` columns of a row (32, 64, 128 or
    256; 0: one for the whole row).  A code stands for code * scale.  Both may
    be views whose rows lie a fixed distance apart."""

    __slots__ = ("codes", "scales", "group")

    def __init__(self, codes, scales, group=128):
        self.codes, self.scales, self.group = codes, scales, int(group)

    @classmethod
    def empty(cls, shape, group=128, dtype=None, device=None, stream=None):
        """One to be written, of `shape`; dtype int8 (default) or float8_e4m3fn."""
        if _torch is None:
            _use_torch()
        dtype = _torch.int8 if dtype is None else dtype
        device = _torch.device("cuda", embed._device()) if device is None else device
        cols = shape[-1]
        groups = -(-cols // group) if group else 1
        return cls(_empty(tuple(shape), dtype, device, stream), _empty((*shape[:-1], groups), _torch.float32, device, stream), group)

    @property
    def shape(self):
        return self.codes.shape

    def __repr__(self):
        return f"Packed({tuple(self.codes.shape)}, {self.codes.dtype}, group={self.group})"


class RmsNorm:
    """The root-mean-square norm of rows of `dim` columns,
    h * rstd * weight with h = x + residual and rstd = 1 / sqrt(mean(h^2) + eps),
    and its gradient.

    Tensors are CUDA tensors on the device that was current at construction,
    bfloat16 or float32 in any mixture, with contiguous columns.  `stream`
    defaults to torch's current stream; calls to :meth:`backward` of one norm must
    be ordered, since they share its workspace.
    """

    def __init__(self, dim, eps=1e-5):
        if _torch is None:
            _use_torch()
        self.dim, self.eps = int(dim), float(eps)
        self.h = 0
        self.h = lioncub_rms_norm_create(self.dim, self.eps)
        self.device = _torch.device("cuda", embed._device())
        self._index = self.device.index

    def forward(self, x, weight=None, *, residual=None, summed=None, saved=None, rstd=None, out=None, out_dtype=None, stream=None):
        """The normed rows of x (..., dim) + residual: `out`, a tensor or a
        :class:`Packed` to be written, by default a new tensor of out_dtype (x's
        type).  Written too, where they are given: summed = x + residual (x or
        the residual itself is allowed), saved (a Packed) the same in 8 bits,
        and rstd (float32, one a row); the backward pass needs rstd and one of
        the two."""
        if not self.h:
            raise LionCubError(ERR_STATE, "the norm is closed")
        if out is None:
            out = _empty(x.shape, out_dtype or x.dtype, self.device, stream)
        rc = _tensors.rms_norm_forward(self.h, self.dim, self._index, x, residual, weight, summed, saved, rstd, out,
                                       _raw(self._index, stream))
        if rc:
            _check(rc)
        return out

    def backward(self, dout, saved, rstd, weight=None, *, residual_grad=None, out=None, out_dtype=None, weight_grad=None,
                 weight_base=None, again=None, stream=None):
        """The gradient of x, which is the residual's too, from dout and what the
        forward call left: `saved`, its summed (or x) or its saved Packed, and rstd.
        residual_grad is added: what reaches the sum by another way.  weight_grad
        (dim,) is written where it is given, weight_base added to it (weight_grad
        itself adds in place); again receives the normed rows once more."""
        if not self.h:
            raise LionCubError(ERR_STATE, "the norm is closed")
        if out is None:
            out = _empty(dout.shape, out_dtype or dout.dtype, self.device, stream)
        rc = _tensors.rms_norm_backward(self.h, self.dim, self._index, dout, saved, rstd, weight, residual_grad, out, weight_base,
                                        weight_grad, again, _raw(self._index, stream))
        if rc:
            _check(rc)
        return out

    def status(self) -> int:
        """The status word (0: all is well) after the calls before it on torch's
        current stream.  Synchronizes."""
        if not self.h:
            raise LionCubError(ERR_STATE, "the norm is closed")
        word = _torch.zeros(1, dtype=_torch.int32, device=self.device)
        lioncub_rms_norm_status(self.h, word.data_ptr(), embed._raw_stream(self._index))
        return int(word.item())

    def close(self):
        if self.h:
            lioncub_rms_norm_destroy(self.h)
            self.h = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def pack8(x, *, group=128, dtype=None, out=None, stream=None) -> Packed:
    """x in 8 bits: `out`, or a new Packed of `group` and dtype (int8 by default)."""
    if _torch is None:
        _use_torch()
    dev = _device()
    if out is None:
        out = Packed.empty(x.shape, group, dtype, x.device, stream)
    rc = _tensors.pack8(dev, x, out, _raw(dev, stream))
    if rc:
        _check(rc)
    return out


def unpack8(x: Packed, *, out=None, out_dtype=None, stream=None):
    """What a Packed stands for: `out`, or a new tensor of out_dtype (bfloat16 by default)."""
    if _torch is None:
        _use_torch()
    dev, codes = _device(), x.codes
    if out is None:
        out = _empty(codes.shape, out_dtype or _torch.bfloat16, codes.device, stream)
    rc = _tensors.unpack8(dev, codes, x, out, _raw(dev, stream))
    if rc:
        _check(rc)
    return out


_kinds = {"silu": SILU, "gelu": GELU}


def _kind(kind):
    try:
        return _kinds[kind]
    except KeyError:
        raise ValueError(f"kind must be silu or gelu (got {kind!r})") from None


def activation(x, up=None, *, kind="gelu", out=None, saved=None, saved_up=None, stream=None):
    """f(x), times `up` where it is given; kind: "silu" or "gelu" (by the
    hyperbolic tangent).  out: where to write (x itself is allowed); saved and
    saved_up (Packed, groups of columns) receive x and up in 8 bits."""
    if _torch is None:
        _use_torch()
    dev = _device()
    if out is None:
        out = _empty(x.shape, x.dtype, x.device, stream)
    rc = _tensors.activation_forward(dev, _kind(kind), x, up, out, saved, saved_up, _raw(dev, stream))
    if rc:
        _check(rc)
    return out


def activation_backward(dout, x, up=None, *, kind="gelu", dx=None, dup=None, again=None, stream=None):
    """The gradient of :func:`activation` with respect to x, or with `up` the
    pair of both, from dout; x and up as tensors or as the Packed that the
    forward call saved.  dx, dup: where to write; again, where it is given,
    receives the forward call's result once more."""
    if _torch is None:
        _use_torch()
    dev = _device()
    if dx is None:
        dx = _empty(dout.shape, dout.dtype, dout.device, stream)
    if up is not None and dup is None:
        dup = _empty(dout.shape, dout.dtype, dout.device, stream)
    rc = _tensors.activation_backward(dev, _kind(kind), dout, x, up, dx, dup, again, _raw(dev, stream))
    if rc:
        _check(rc)
    return dx if up is None else (dx, dup)


class RotaryScaling(NamedTuple):
    """How frequencies are scaled for contexts `factor` times those trained on.

    kind: "linear" divides all of them; "base" raises the base, so that the
    slowest pair is divided by about `factor` and the fastest not at all; "parts"
    keeps the pairs that turn `high` times or more within `length` positions,
    divides those that turn `low` times or less, and interpolates between.
    magnitude multiplies rotated queries and keys (None: 0.1 ln(factor) + 1 for
    "parts", else 1)."""
    kind: str
    factor: float
    length: float = 0.0
    low: float = 1.0
    high: float = 32.0
    magnitude: float | None = None


_scalings = {"linear": SCALING_LINEAR, "base": SCALING_BASE, "parts": SCALING_PARTS}


class Rotary:
    """Rotary positions over the first rotary_dim (default all) columns of heads
    of head_dim.  Pair k turns by position * base^(-2 k / rotary_dim), scaled as
    `scaling` says, or by position * frequencies[k] where those are given; a pair
    is columns (k, k + rotary_dim / 2), or (2 k, 2 k + 1) when interleaved.

    Tensors are bfloat16 or float32 CUDA tensors on the device that was current
    at construction, of shape (batch, places, heads, head_dim) or (places, heads,
    head_dim) in any strides with contiguous columns: views of a fused product,
    or of a (batch, heads, places, head_dim) tensor by transpose(1, 2), need no
    copy.  Queries and keys may have different numbers of heads.
    """

    def __init__(self, head_dim, *, rotary_dim=None, base=10000.0, interleaved=False, scaling=None, frequencies=None,
                 magnitude=None):
        if _torch is None:
            _use_torch()
        self.head_dim = int(head_dim)
        self.rotary_dim = self.head_dim if rotary_dim is None else int(rotary_dim)
        self.interleaved = bool(interleaved)
        if frequencies is None:
            spec = None
            if scaling is not None:
                if scaling.kind not in _scalings:
                    raise ValueError(f"scaling must be linear, base or parts (got {scaling.kind!r})")
                spec = ScalingSpec(scaling.factor, scaling.length, scaling.low, scaling.high, _scalings[scaling.kind], 0)
            frequencies = lioncub_rotary_frequencies(self.rotary_dim, base, spec)
        elif scaling is not None:
            raise ValueError("frequencies are given as they are: scaling has no use")
        if len(frequencies) != self.rotary_dim // 2:
            raise ValueError(f"{self.rotary_dim // 2} frequencies are needed (got {len(frequencies)})")
        if magnitude is None:
            magnitude = 1.0
            if scaling is not None:
                magnitude = scaling.magnitude
                if magnitude is None:
                    magnitude = 0.1 * math.log(scaling.factor) + 1.0 if scaling.kind == "parts" else 1.0
        self.frequencies, self.magnitude = tuple(float(f) for f in frequencies), float(magnitude)
        self.h = 0
        self.h = lioncub_rotary_create(self.head_dim, self.rotary_dim, self.frequencies, self.magnitude, self.interleaved)
        self.device = _torch.device("cuda", embed._device())
        self._index = self.device.index

    def _apply(self, q, k, positions, first_position, q_out, k_out, stream, inverse):
        if not self.h:
            raise LionCubError(ERR_STATE, "the rotary positions are closed")
        if k is None and k_out is not None:
            raise ValueError("k_out without k")
        if q_out is None:
            q_out = _empty(q.shape, q.dtype, self.device, stream)
        if k is not None and k_out is None:
            k_out = _empty(k.shape, k.dtype, self.device, stream)
        rc = _tensors.rotary_apply(self.h, self.head_dim, self._index, q, q_out, k, k_out, positions, first_position, inverse,
                                   _raw(self._index, stream))
        if rc:
            _check(rc)
        return q_out if k is None else (q_out, k_out)

    def forward(self, q, k=None, *, positions=None, first_position=0, q_out=None, k_out=None, stream=None):
        """q, or the pair of q and k, rotated: new tensors, or q_out and k_out (q
        and k themselves are allowed).  positions: (batch, places), int64 or
        int32; without them a place's is first_position + its index."""
        return self._apply(q, k, positions, first_position, q_out, k_out, stream, 0)

    def backward(self, dq, dk=None, *, positions=None, first_position=0, q_out=None, k_out=None, stream=None):
        """The gradients of what :meth:`forward` took, from those of its results:
        the rotation by the negative angle."""
        return self._apply(dq, dk, positions, first_position, q_out, k_out, stream, 1)

    def close(self):
        if self.h:
            lioncub_rotary_destroy(self.h)
            self.h = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
