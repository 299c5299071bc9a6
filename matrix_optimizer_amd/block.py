"""ctypes binding of libmuon's row operators (include/muon_block.h): the norm,
dropout and expert routing that a decoder block runs between the matrices that
muon_step updates.

As in binding.py: argument marshalling only, on device memory the caller owns
(outputs included), on the current stream of the tensors' device or the given
hipStream_t; a missing library raises, there is no fallback.  Shapes, types
and devices are checked here, since the C ABI sees only addresses; values,
strides, alignment and overlap are checked there (MuonError).  Matrices are
[rows, cols] tensors whose last dimension is contiguous; any row stride.  With
a stream given, the caller orders it against the tensors' own use and keeps
them until it has run the call.
"""
from __future__ import annotations

import ctypes as C
import struct
from dataclasses import dataclass
from typing import Optional

import torch

from . import binding as B

MUON_ROW_F32, MUON_ROW_BF16, MUON_ROW_E4M3, MUON_ROW_E5M2 = range(4)
MUON_SCORE_SOFTMAX, MUON_SCORE_SIGMOID = 0, 1
MAX_EXPERTS, MAX_TOP_K = 1024, 32

EXPORTED = ["muon_block_abi_version", "muon_dropout", "muon_norm_forward", "muon_norm_backward",
            "muon_norm_workspace_bytes", "muon_route_forward", "muon_route_backward", "muon_route_order",
            "muon_route_order_workspace_bytes", "muon_route_balance"]

_SCORES = {"softmax": MUON_SCORE_SOFTMAX, "sigmoid": MUON_SCORE_SIGMOID}
_DTYPES = {torch.float32: B.MUON_F32, torch.bfloat16: B.MUON_BF16}
_ROW_DTYPES = {torch.float32: MUON_ROW_F32, torch.bfloat16: MUON_ROW_BF16, torch.float8_e4m3fn: MUON_ROW_E4M3,
               torch.float8_e5m2: MUON_ROW_E5M2}


class muon_dropout_spec(C.Structure):
    _fields_ = [("p", C.c_double), ("seed", C.c_uint64), ("offset", C.c_uint64), ("seed_device", C.c_void_p)]


class muon_norm_args(C.Structure):
    _fields_ = [("rows", C.c_int64), ("cols", C.c_int64), ("x", C.c_void_p), ("x_stride", C.c_int64),
                ("residual", C.c_void_p), ("residual_stride", C.c_int64), ("h", C.c_void_p), ("h_stride", C.c_int64),
                ("y", C.c_void_p), ("y_stride", C.c_int64), ("weight", C.c_void_p), ("scales", C.c_void_p),
                ("scales_stride", C.c_int64), ("rstd", C.c_void_p), ("dropout", C.c_void_p),
                ("dtype", C.c_int32), ("weight_dtype", C.c_int32), ("y_dtype", C.c_int32), ("group", C.c_int32),
                ("eps", C.c_float)]


class muon_norm_grad_args(C.Structure):
    _fields_ = [("rows", C.c_int64), ("cols", C.c_int64), ("dy", C.c_void_p), ("dy_stride", C.c_int64),
                ("h", C.c_void_p), ("h_stride", C.c_int64), ("dh", C.c_void_p), ("dh_stride", C.c_int64),
                ("dresidual", C.c_void_p), ("dresidual_stride", C.c_int64), ("dx", C.c_void_p),
                ("dx_stride", C.c_int64), ("rstd", C.c_void_p), ("weight", C.c_void_p), ("dweight", C.c_void_p),
                ("dropout", C.c_void_p), ("dtype", C.c_int32), ("weight_dtype", C.c_int32)]


class muon_route_spec(C.Structure):
    _fields_ = [("score", C.c_int32), ("top_k", C.c_int32), ("groups", C.c_int32), ("top_groups", C.c_int32),
                ("group_top", C.c_int32), ("renormalise", C.c_int32), ("scale", C.c_float)]


class muon_route_args(C.Structure):
    _fields_ = [("rows", C.c_int64), ("num_experts", C.c_int64), ("logits", C.c_void_p), ("logits_stride", C.c_int64),
                ("bias", C.c_void_p), ("token_mask", C.c_void_p), ("experts", C.c_void_p), ("weights", C.c_void_p),
                ("scores", C.c_void_p), ("dtype", C.c_int32)]


class muon_route_grad_args(C.Structure):
    _fields_ = [("rows", C.c_int64), ("num_experts", C.c_int64), ("logits", C.c_void_p), ("logits_stride", C.c_int64),
                ("experts", C.c_void_p), ("weights", C.c_void_p), ("dweights", C.c_void_p), ("dscores", C.c_void_p),
                ("dlogits", C.c_void_p), ("dlogits_stride", C.c_int64), ("dtype", C.c_int32)]


def _packer(cls):
    """The C struct as bytes from its fields in order: half the time of making a ctypes object."""
    codes = {C.c_int64: "q", C.c_uint64: "Q", C.c_void_p: "P", C.c_int32: "i", C.c_float: "f", C.c_double: "d"}
    fields = "".join(codes[t] for _, t in cls._fields_)
    s = struct.Struct("@" + fields + ("0q" if set(fields) & set("qQPd") else ""))
    assert s.size == C.sizeof(cls)
    return s.pack


_pack_norm, _pack_norm_grad = _packer(muon_norm_args), _packer(muon_norm_grad_args)
_pack_spec, _pack_route, _pack_route_grad = map(_packer, (muon_route_spec, muon_route_args, muon_route_grad_args))

_lib = None


def lib():
    """libmuon.so with the row operators' prototypes set."""
    global _lib
    if _lib is not None:
        return _lib
    L = B.lib()
    P, I64, I32, F = C.c_void_p, C.c_int64, C.c_int32, C.c_float
    sig = {"muon_block_abi_version": [], "muon_dropout": [I64, I64, P, I64, P, I64, I32, P, P],
           "muon_norm_forward": [P, P], "muon_norm_backward": [P, P, C.c_size_t, P],
           "muon_norm_workspace_bytes": [I64, I64, C.POINTER(C.c_size_t)], "muon_route_forward": [P, P, P],
           "muon_route_backward": [P, P, P], "muon_route_order": [I64, I64, P, P, P, P, P, P, C.c_size_t, P],
           "muon_route_order_workspace_bytes": [I64, I64, C.POINTER(C.c_size_t)],
           "muon_route_balance": [I64, P, P, P, F, P]}
    for name, args in sig.items():
        f = getattr(L, name)
        f.restype, f.argtypes = C.c_int32, args
    _lib = L
    return L


def muon_block_abi_version() -> int:
    return lib().muon_block_abi_version()


@dataclass
class Dropout:
    """Dropout of probability p, its mask given by (seed, offset) alone (muon_dropout_spec): the backward
    pass takes the forward's values.  `device`: an int64 or uint64 device tensor [seed, offset] read in
    their place when the kernels run, for captured graphs."""
    p: float
    seed: int = 0
    offset: int = 0
    device: Optional[torch.Tensor] = None

    def to_c(self):
        dev = None
        if self.device is not None:
            if self.device.dtype not in (torch.int64, torch.uint64) or self.device.numel() != 2 \
                    or not self.device.is_contiguous() or not self.device.is_cuda:
                raise ValueError("Dropout.device: a contiguous device tensor of two 64-bit integers")
            dev = self.device.data_ptr()
        return muon_dropout_spec(self.p, self.seed & 0xFFFFFFFFFFFFFFFF, self.offset & 0xFFFFFFFFFFFFFFFF, dev)


@dataclass
class Route:
    """How rows choose their experts (muon_route_spec)."""
    top_k: int
    score: str = "softmax"     # or "sigmoid"
    groups: int = 1
    top_groups: int = 1
    group_top: int = 2         # a group's value: the sum of its 1 or 2 best
    renormalise: bool = True
    scale: float = 1.0

    def to_c(self):
        """muon_route_spec as bytes."""
        if self.score not in _SCORES:
            raise ValueError(f"Route.score: 'softmax' or 'sigmoid', got {self.score!r}")
        return _pack_spec(_SCORES[self.score], self.top_k, self.groups, self.top_groups, self.group_top,
                          bool(self.renormalise), self.scale)


# The raw stream of a device's current stream; a Stream object costs 2 us to make.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


class _Call:
    """Checks one call's tensors against its first, a [rows, cols] matrix, whose shape, type and device the
    others share unless they say otherwise.  Small calls are bound by this code: few steps, no formatting
    before something is wrong."""
    __slots__ = ("where", "shape", "dtype", "index")

    def __init__(self, where: str, first):
        self.where, self.shape, self.dtype, self.index = where, first.shape, first.dtype, first.get_device()

    def rows(self):
        """(rows, cols, dtype code) of the first tensor."""
        if len(self.shape) != 2:
            raise ValueError(f"{self.where}: [rows, cols] is needed, got {list(self.shape)}")
        if self.dtype not in _DTYPES:
            raise TypeError(f"{self.where}: unsupported dtype {self.dtype}")
        self.on_device()
        return self.shape[0], self.shape[1], _DTYPES[self.dtype]

    def on_device(self):
        if self.index < 0:
            raise ValueError(f"{self.where}: device tensors are needed")

    def wrong(self, name, t, shape, dtypes):
        if t.shape != shape:
            raise ValueError(f"{self.where}: {name} must be {list(shape)}, got {list(t.shape)}")
        if t.dtype not in dtypes:
            raise ValueError(f"{self.where}: {name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
        if t.get_device() != self.index:
            raise ValueError(f"{self.where}: {name} is on {t.device}, not on device {self.index}")
        raise ValueError(f"{self.where}: {name} must be contiguous{' along its rows' if t.dim() == 2 else ''}")

    def matrix(self, name, t, dtype=None):
        """(address, row stride) of a matrix like the first, (0, 0) for None.  The stride of a single row is
        not read."""
        if t is None:
            return 0, 0
        if t.shape != self.shape or t.dtype is not (dtype or self.dtype) or t.get_device() != self.index:
            self.wrong(name, t, self.shape, (dtype or self.dtype,))
        s0, s1 = t.stride()
        if s1 != 1 and self.shape[1] > 1:
            self.wrong(name, t, self.shape, (t.dtype,))
        return t.data_ptr(), s0

    def flat(self, name, t, shape, dtypes):
        """Address of a contiguous tensor of one of `dtypes`, 0 for None."""
        if t is None:
            return 0
        if t.shape != shape or t.dtype not in dtypes or t.get_device() != self.index or not t.is_contiguous():
            self.wrong(name, t, shape, dtypes)
        return t.data_ptr()

    def workspace(self, t):
        if t is None:
            return None, 0
        if t.get_device() != self.index or not t.is_contiguous():
            raise ValueError(f"{self.where}: workspace must be a contiguous tensor on device {self.index}")
        return t.data_ptr(), t.numel() * t.element_size()

    def dropout(self, d):
        """(what keeps the C struct alive, its address)."""
        if d is None:
            return None, 0
        if d.device is not None and d.device.get_device() != self.index:
            raise ValueError(f"{self.where}: Dropout.device is on {d.device.device}, not on device {self.index}")
        c = d.to_c()
        return c, C.addressof(c)

    def run(self, fn, *args, stream):
        index = self.index
        if stream is None:
            stream = _raw_stream(index)
        if index != _current_device():
            with torch.cuda.device(index):
                st = fn(*args, stream)
        else:
            st = fn(*args, stream)
        if st != B.MUON_OK:
            raise B.MuonError(st, self.where)


_F32 = (torch.float32,)
_I32 = (torch.int32,)
_WEIGHT = (torch.float32, torch.bfloat16)
_BYTE = (torch.uint8, torch.bool)


def muon_dropout(x, y, dropout: Dropout, stream=None) -> None:
    """y = D(x); y may be x.  The backward pass is the same call on the gradient."""
    c = _Call("muon_dropout", x)
    rows, cols, dt = c.rows()
    keep, spec = c.dropout(dropout)
    c.run(lib().muon_dropout, rows, cols, *c.matrix("x", x), *c.matrix("y", y), dt, spec, stream=stream)


def muon_norm_forward(x, y, residual=None, h=None, weight=None, rstd=None, scales=None, group: int = 0,
                      eps: float = 1e-6, dropout: Optional[Dropout] = None, stream=None) -> None:
    """z = residual + D(x); h = z; y = z rstd weight (muon_norm_forward).  x, residual, h: one type (fp32 or
    bf16); y: fp32, bf16, float8_e4m3fn or float8_e5m2, the latter two with scales [rows, groups] fp32 (groups
    of `group` columns, 0 = the row).  h may be x or residual."""
    c = _Call("muon_norm_forward", x)
    rows, cols, dt = c.rows()
    if y.dtype not in _ROW_DTYPES:
        raise TypeError(f"muon_norm_forward: unsupported dtype {y.dtype}")
    keep, spec = c.dropout(dropout)
    groups = 0
    if scales is not None:
        groups = -(-cols // group) if group > 0 else 1
    a = _pack_norm(rows, cols, *c.matrix("x", x), *c.matrix("residual", residual), *c.matrix("h", h),
                   *c.matrix("y", y, y.dtype), c.flat("weight", weight, (cols,), _WEIGHT),
                   c.flat("scales", scales, (rows, groups), _F32), groups, c.flat("rstd", rstd, (rows,), _F32),
                   spec, dt, 0 if weight is None else _DTYPES[weight.dtype], _ROW_DTYPES[y.dtype], group, eps)
    c.run(lib().muon_norm_forward, a, stream=stream)


def norm_workspace_bytes(rows: int, cols: int) -> int:
    out = C.c_size_t()
    B._check(lib().muon_norm_workspace_bytes(rows, cols, C.byref(out)), "muon_norm_workspace_bytes")
    return out.value


def muon_norm_backward(dy, h, rstd, weight=None, dh=None, dresidual=None, dx=None, dweight=None, workspace=None,
                       dropout: Optional[Dropout] = None, stream=None) -> None:
    """The gradients of muon_norm_forward from its h and rstd: dresidual = dz, dx = D(dz), dweight (fp32, with
    a uint8 workspace of norm_workspace_bytes).  dh: the gradient arriving on the residual stream; dresidual
    may be dh."""
    c = _Call("muon_norm_backward", dy)
    rows, cols, dt = c.rows()
    keep, spec = c.dropout(dropout)
    a = _pack_norm_grad(rows, cols, *c.matrix("dy", dy), *c.matrix("h", h), *c.matrix("dh", dh),
                        *c.matrix("dresidual", dresidual), *c.matrix("dx", dx),
                        c.flat("rstd", rstd, (rows,), _F32), c.flat("weight", weight, (cols,), _WEIGHT),
                        c.flat("dweight", dweight, (cols,), _F32), spec, dt,
                        0 if weight is None else _DTYPES[weight.dtype])
    c.run(lib().muon_norm_backward, a, *c.workspace(workspace), stream=stream)


def muon_route_forward(route: Route, logits, experts, weights, bias=None, token_mask=None, scores=None,
                       stream=None) -> None:
    """experts [rows, top_k] int32 and weights fp32 of each row's logits [rows, E] (fp32 or bf16).  bias: fp32
    [E], moves the choice only; token_mask: bool or uint8 [rows], rows of 0 choose nothing (-1); scores: fp32
    [rows, E], optional output."""
    c = _Call("muon_route_forward", logits)
    rows, n, dt = c.rows()
    pairs = (rows, route.top_k)
    a = _pack_route(rows, n, *c.matrix("logits", logits), c.flat("bias", bias, (n,), _F32),
                    c.flat("token_mask", token_mask, (rows,), _BYTE), c.flat("experts", experts, pairs, _I32),
                    c.flat("weights", weights, pairs, _F32), c.flat("scores", scores, (rows, n), _F32), dt)
    c.run(lib().muon_route_forward, route.to_c(), a, stream=stream)


def muon_route_backward(route: Route, logits, experts, weights, dweights, dlogits, dscores=None, stream=None) -> None:
    """dlogits (logits' type, all written) from dweights, and dscores where the scores were used."""
    c = _Call("muon_route_backward", logits)
    rows, n, dt = c.rows()
    pairs = (rows, route.top_k)
    a = _pack_route_grad(rows, n, *c.matrix("logits", logits), c.flat("experts", experts, pairs, _I32),
                         c.flat("weights", weights, pairs, _F32), c.flat("dweights", dweights, pairs, _F32),
                         c.flat("dscores", dscores, (rows, n), _F32), *c.matrix("dlogits", dlogits), dt)
    c.run(lib().muon_route_backward, route.to_c(), a, stream=stream)


def route_order_workspace_bytes(num_pairs: int, num_experts: int) -> int:
    out = C.c_size_t()
    B._check(lib().muon_route_order_workspace_bytes(num_pairs, num_experts, C.byref(out)),
             "muon_route_order_workspace_bytes")
    return out.value


def muon_route_order(experts, counts, offsets, order, position, workspace, stream=None) -> None:
    """The pairs of `experts` (int32, any shape) grouped by expert: counts [E], offsets [E + 1], order [pairs],
    position (experts' shape), all int32; workspace: uint8 of route_order_workspace_bytes."""
    c = _Call("muon_route_order", experts)
    c.on_device()
    n, pairs = counts.numel(), experts.numel()
    c.run(lib().muon_route_order, pairs, n, c.flat("experts", experts, c.shape, _I32),
          c.flat("counts", counts, (n,), _I32), c.flat("offsets", offsets, (n + 1,), _I32),
          c.flat("order", order, (pairs,), _I32), c.flat("position", position, c.shape, _I32),
          *c.workspace(workspace), stream=stream)


def muon_route_balance(counts, bias, out, rate: float, stream=None) -> None:
    """out = bias + rate sign(mean(counts) - counts); out may be bias."""
    c = _Call("muon_route_balance", counts)
    c.on_device()
    n = counts.numel()
    c.run(lib().muon_route_balance, n, c.flat("counts", counts, (n,), _I32), c.flat("bias", bias, (n,), _F32),
          c.flat("out", out, (n,), _F32), rate, stream=stream)
