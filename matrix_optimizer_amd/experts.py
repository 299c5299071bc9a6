"""ctypes binding of libmuon's expert operators (include/muon_experts.h): what the
routed pairs of a decoder block go through between muon_route_order and the
residual stream, on the expert tensors that muon_step updates.

As in block.py: argument marshalling only, on device memory the caller owns
(outputs included), on the current stream of the tensors' device or the given
hipStream_t; shapes, types and devices are checked here (ValueError,
TypeError), values, strides, alignment and overlap in the C ABI (MuonError).
Matrices' last dimension is contiguous; any row stride.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import binding as B
from .block import _DTYPES, _F32, _I32, _ROW_DTYPES, _Call, _packer

EXPORTED = ["muon_experts_abi_version", "muon_expert_gather", "muon_expert_combine", "muon_expert_combine_backward",
            "muon_gate_forward", "muon_gate_backward", "muon_quantise_blocks", "muon_expert_product",
            "muon_expert_weight_grad", "muon_expert_weight_grad_workspace_bytes"]
BLOCK = 128     # columns that share a scale, and rows too in a matrix

_EIGHT = (torch.float8_e4m3fn, torch.float8_e5m2)
_BF16 = (torch.bfloat16,)
_I64, _P, _INT = C.c_int64, C.c_void_p, C.c_int32


def _fields(text):
    """'a:q b:P' as ctypes fields."""
    kinds = {"q": _I64, "P": _P, "i": _INT}
    return [(n, kinds[k]) for n, k in (f.split(":") for f in text.split())]


class muon_gather_args(C.Structure):
    _fields_ = _fields("rows:q cols:q top_k:q x:P x_stride:q out:P out_stride:q scales:P scales_stride:q out_scales:P "
                       "out_scales_stride:q groups:q order:P dtype:i")


class muon_combine_args(C.Structure):
    _fields_ = _fields("rows:q cols:q top_k:q places:q position:P weights:P y:P y_stride:q base:P base_stride:q out:P "
                       "out_stride:q dtype:i out_dtype:i")


class muon_combine_grad_args(C.Structure):
    _fields_ = _fields("rows:q cols:q top_k:q places:q position:P weights:P dout:P dout_stride:q y:P y_stride:q dy:P "
                       "dy_stride:q dy8:P dy8_stride:q scales:P scales_stride:q dweights:P dtype:i dy8_dtype:i")


class muon_gate_args(C.Structure):
    _fields_ = _fields("rows:q cols:q a:P a_stride:q y:P y_stride:q y8:P y8_stride:q scales:P scales_stride:q used:P "
                       "dtype:i y8_dtype:i")


class muon_gate_grad_args(C.Structure):
    _fields_ = _fields("rows:q cols:q a:P a_stride:q dy:P dy_stride:q da:P da_stride:q da8:P da8_stride:q scales:P "
                       "scales_stride:q used:P dtype:i da8_dtype:i")


class muon_quantise_args(C.Structure):
    _fields_ = _fields("batch:q rows:q cols:q x:P x_stride:q x_matrix:q q:P q_stride:q q_matrix:q scales:P qt:P "
                       "qt_stride:q qt_matrix:q scales_t:P dtype:i q_dtype:i")


class muon_product_args(C.Structure):
    _fields_ = _fields("rows:q n:q k:q num_experts:q a:P a_stride:q a_scales:P a_scales_stride:q w:P w_stride:q "
                       "w_matrix:q w_scales:P offsets:P out:P out_stride:q a_dtype:i w_dtype:i out_dtype:i")


class muon_weight_grad_args(C.Structure):
    _fields_ = _fields("rows:q n:q k:q num_experts:q dy:P dy_stride:q x:P x_stride:q offsets:P dw:P dw_stride:q "
                       "dw_matrix:q dw_dtype:i")


_pack_gather, _pack_combine, _pack_combine_grad = map(_packer, (muon_gather_args, muon_combine_args,
                                                                muon_combine_grad_args))
_pack_gate, _pack_gate_grad, _pack_quantise = map(_packer, (muon_gate_args, muon_gate_grad_args, muon_quantise_args))
_pack_product, _pack_weight_grad = _packer(muon_product_args), _packer(muon_weight_grad_args)

_lib = None


def lib():
    """libmuon.so with the expert operators' prototypes set."""
    global _lib
    if _lib is not None:
        return _lib
    L = B.lib()
    size = C.POINTER(C.c_size_t)
    sig = {n: [_P, _P] for n in EXPORTED[1:8]}
    sig.update({"muon_experts_abi_version": [], "muon_expert_weight_grad": [_P, _P, C.c_size_t, _P],
                "muon_expert_weight_grad_workspace_bytes": [_I64, _I64, _I64, _I64, size]})
    for name, args in sig.items():
        f = getattr(L, name)
        f.restype, f.argtypes = C.c_int32, args
    _lib = L
    return L


def muon_experts_abi_version() -> int:
    return lib().muon_experts_abi_version()


class _Experts(_Call):
    """_Call with matrices, and stacks of them, of shapes of their own."""
    __slots__ = ()

    def rows_of(self, name, t, shape, dtypes):
        """(address, row stride) of a matrix [rows, cols] of one of `dtypes`, (0, 0) for None."""
        if t is None:
            return 0, 0
        if t.shape != shape or t.dtype not in dtypes or t.get_device() != self.index:
            self.wrong(name, t, shape, dtypes)
        s0, s1 = t.stride()
        if s1 != 1 and shape[1] > 1 and shape[0] > 0:
            self.wrong(name, t, shape, dtypes)
        return t.data_ptr(), s0

    def matrix(self, name, t):
        return self.rows_of(name, t, self.shape, (self.dtype,))

    def stack(self, name, t, shape, dtypes):
        """(address, row stride, matrix stride) of matrices [batch, rows, cols], (0, 0, 0) for None."""
        if t is None:
            return 0, 0, 0
        if t.shape != shape or t.dtype not in dtypes or t.get_device() != self.index:
            self.wrong(name, t, shape, dtypes)
        s0, s1, s2 = t.stride()
        if s2 != 1 and shape[2] > 1 and t.numel() > 0:
            raise ValueError(f"{self.where}: {name} must be contiguous along its rows")
        return t.data_ptr(), s1, s0

    def dims(self, name, t, n):
        if t.dim() != n:
            raise ValueError(f"{self.where}: {name} must have {n} dimensions, got {list(t.shape)}")

    def eight(self, name, t, scales):
        """An 8-bit output and its scales come together."""
        if (t is None) != (scales is None):
            raise ValueError(f"{self.where}: {name} and its scales are given together")
        return 0 if t is None else _ROW_DTYPES.get(t.dtype, -1)


def _groups(cols):
    return -(-cols // BLOCK)


def muon_expert_gather(order, x, out, scales=None, out_scales=None, stream=None) -> None:
    """out[i] = x[order[i] // top_k] for order [rows * top_k] of muon_route_order; scales [rows, groups] fp32 go
    with the rows to out_scales.  x, out: fp32, bf16 or 8 bits.  Places without a pair are left as they are."""
    c = _Experts("muon_expert_gather", x)
    c.on_device()
    c.dims("x", x, 2)
    rows, cols = x.shape
    pairs = order.numel()
    if x.dtype not in _ROW_DTYPES:
        raise TypeError(f"muon_expert_gather: unsupported dtype {x.dtype}")
    if pairs % rows if rows else pairs:
        raise ValueError(f"muon_expert_gather: order must hold a whole number of pairs a row, got {pairs} for {rows} rows")
    if (scales is None) != (out_scales is None):
        raise ValueError("muon_expert_gather: scales and out_scales are given together")
    groups = 0
    if scales is not None:
        c.dims("scales", scales, 2)
        groups = scales.shape[1]
    a = _pack_gather(rows, cols, pairs // rows if rows else 1, *c.matrix("x", x), *c.rows_of("out", out, (pairs, cols), (x.dtype,)),
                     *c.rows_of("scales", scales, (rows, groups), _F32),
                     *c.rows_of("out_scales", out_scales, (pairs, groups), _F32), groups,
                     c.flat("order", order, order.shape, _I32), _ROW_DTYPES[x.dtype])
    c.run(lib().muon_expert_gather, a, stream=stream)


def muon_expert_combine(position, y, out, weights=None, base=None, stream=None) -> None:
    """out = base + sum over slots of weights y[position], position [rows, top_k] int32 of muon_route_order,
    weights fp32 (None: ones, the gradient of the gather); out (fp32 or bf16) may be base."""
    c = _Experts("muon_expert_combine", y)
    places, cols, dt = c.rows()
    c.dims("position", position, 2)
    rows, k = position.shape
    if out.dtype not in _DTYPES:
        raise TypeError(f"muon_expert_combine: unsupported dtype {out.dtype}")
    a = _pack_combine(rows, cols, k, places, c.flat("position", position, position.shape, _I32),
                      c.flat("weights", weights, position.shape, _F32), *c.matrix("y", y),
                      *c.rows_of("base", base, (rows, cols), (out.dtype,)),
                      *c.rows_of("out", out, (rows, cols), (out.dtype,)), dt, _DTYPES[out.dtype])
    c.run(lib().muon_expert_combine, a, stream=stream)


def muon_expert_combine_backward(position, dout, y=None, weights=None, dy=None, dweights=None, dy8=None, scales=None,
                                 stream=None) -> None:
    """dy[position] = weights dout, in dout's type and / or in 8 bits (dy8 with scales), and dweights [rows, top_k]
    = <dout, y[position]> (needs y)."""
    c = _Experts("muon_expert_combine_backward", dout)
    rows, cols, dt = c.rows()
    c.dims("position", position, 2)
    if dweights is not None and y is None:
        raise ValueError("muon_expert_combine_backward: dweights needs y")
    e = c.eight("dy8", dy8, scales)
    places = next((t.shape[0] for t in (y, dy, dy8) if t is not None), 0)
    of = (places, cols)
    a = _pack_combine_grad(rows, cols, position.shape[1], places,
                           c.flat("position", position, (rows, position.shape[1]), _I32),
                           c.flat("weights", weights, position.shape, _F32), *c.matrix("dout", dout),
                           *c.rows_of("y", y, of, (dout.dtype,)), *c.rows_of("dy", dy, of, (dout.dtype,)),
                           *c.rows_of("dy8", dy8, of, _EIGHT), *c.rows_of("scales", scales, (places, _groups(cols)), _F32),
                           c.flat("dweights", dweights, position.shape, _F32), dt, e)
    c.run(lib().muon_expert_combine_backward, a, stream=stream)


def _halves(c, a):
    rows, wide, dt = c.rows()
    if wide % 2:
        raise ValueError(f"{c.where}: a must be [rows, 2 cols], got {list(a.shape)}")
    return rows, wide // 2, dt


def muon_gate_forward(a, y=None, y8=None, scales=None, used=None, stream=None) -> None:
    """y = g sigmoid(g) u of a = [g | u] [rows, 2 cols], in a's type (y) and / or in 8 bits (y8 with scales).
    used: an int32 device tensor [1], rows from there on are left alone."""
    c = _Experts("muon_gate_forward", a)
    rows, cols, dt = _halves(c, a)
    e = c.eight("y8", y8, scales)
    args = _pack_gate(rows, cols, *c.matrix("a", a), *c.rows_of("y", y, (rows, cols), (a.dtype,)),
                      *c.rows_of("y8", y8, (rows, cols), _EIGHT),
                      *c.rows_of("scales", scales, (rows, _groups(cols)), _F32), c.flat("used", used, (1,), _I32), dt, e)
    c.run(lib().muon_gate_forward, args, stream=stream)


def muon_gate_backward(a, dy, da=None, da8=None, scales=None, used=None, stream=None) -> None:
    """da = [dg | du] of muon_gate_forward from dy, in a's type and / or in 8 bits (da8 with scales
    [rows, 2 cols / 128]; cols a multiple of 128)."""
    c = _Experts("muon_gate_backward", a)
    rows, cols, dt = _halves(c, a)
    e = c.eight("da8", da8, scales)
    args = _pack_gate_grad(rows, cols, *c.matrix("a", a), *c.rows_of("dy", dy, (rows, cols), (a.dtype,)),
                           *c.matrix("da", da), *c.rows_of("da8", da8, (rows, 2 * cols), _EIGHT),
                           *c.rows_of("scales", scales, (rows, _groups(2 * cols)), _F32),
                           c.flat("used", used, (1,), _I32), dt, e)
    c.run(lib().muon_gate_backward, args, stream=stream)


def muon_quantise_blocks(x, q=None, scales=None, qt=None, scales_t=None, stream=None) -> None:
    """Matrices x [batch, rows, cols] (or [rows, cols]; fp32 or bf16) in 8 bits with a scale for each 128 x 128 block: q
    like x with scales [batch, rows / 128, cols / 128] (rounded up), and / or transposed, qt with scales_t."""
    c = _Experts("muon_quantise_blocks", x)
    c.on_device()
    if x.dim() == 2:
        x, q, scales, qt, scales_t = (None if t is None else t.unsqueeze(0) for t in (x, q, scales, qt, scales_t))
    c.dims("x", x, 3)
    batch, rows, cols = x.shape
    if x.dtype not in _DTYPES:
        raise TypeError(f"muon_quantise_blocks: unsupported dtype {x.dtype}")
    e, et = c.eight("q", q, scales), c.eight("qt", qt, scales_t)
    if q is not None and qt is not None and q.dtype != qt.dtype:
        raise ValueError("muon_quantise_blocks: q and qt must have one dtype")
    rb, cb = _groups(rows), _groups(cols)
    a = _pack_quantise(batch, rows, cols, *c.stack("x", x, x.shape, (x.dtype,)), *c.stack("q", q, x.shape, _EIGHT),
                       c.flat("scales", scales, (batch, rb, cb), _F32),
                       *c.stack("qt", qt, (batch, cols, rows), _EIGHT),
                       c.flat("scales_t", scales_t, (batch, cb, rb), _F32), _DTYPES[x.dtype], e or et)
    c.run(lib().muon_quantise_blocks, a, stream=stream)


def muon_expert_product(a, a_scales, w, w_scales, out, offsets=None, stream=None) -> None:
    """out[i] = a[i] w[e]^T for the rows i of each expert e: a [rows, k] in 8 bits with a_scales [rows, k / 128]
    (rounded up), w [experts, n, k] (or [n, k]) in 8 bits with w_scales [experts, n / 128, k / 128], out [rows, n] fp32 or
    bf16, offsets int32 [experts + 1] of muon_route_order (None: one expert, all rows)."""
    c = _Experts("muon_expert_product", a)
    c.on_device()
    c.dims("a", a, 2)
    if w.dim() == 2:
        w, w_scales = w.unsqueeze(0), w_scales.unsqueeze(0)
    c.dims("w", w, 3)
    rows, k = a.shape
    experts, n = w.shape[:2]
    if out.dtype not in _DTYPES:
        raise TypeError(f"muon_expert_product: unsupported dtype {out.dtype}")
    args = _pack_product(rows, n, k, experts, *c.rows_of("a", a, (rows, k), _EIGHT),
                         *c.rows_of("a_scales", a_scales, (rows, _groups(k)), _F32),
                         *c.stack("w", w, (experts, n, k), _EIGHT),
                         c.flat("w_scales", w_scales, (experts, _groups(n), _groups(k)), _F32),
                         c.flat("offsets", offsets, (experts + 1,), _I32),
                         *c.rows_of("out", out, (rows, n), (out.dtype,)), _ROW_DTYPES[a.dtype], _ROW_DTYPES[w.dtype],
                         _DTYPES[out.dtype])
    c.run(lib().muon_expert_product, args, stream=stream)


def expert_weight_grad_workspace_bytes(rows: int, num_experts: int, n: int, k: int) -> int:
    out = C.c_size_t()
    B._check(lib().muon_expert_weight_grad_workspace_bytes(rows, num_experts, n, k, C.byref(out)),
             "muon_expert_weight_grad_workspace_bytes")
    return out.value


def muon_expert_weight_grad(dy, x, dw, offsets=None, workspace=None, stream=None) -> None:
    """dw[e] = dy_e^T x_e over the rows of each expert: dy [rows, n] and x [rows, k] bf16, dw [experts, n, k] (or
    [n, k]) fp32 or bf16, all of it written; offsets as in muon_expert_product; workspace: uint8 of
    expert_weight_grad_workspace_bytes."""
    c = _Experts("muon_expert_weight_grad", dy)
    c.on_device()
    c.dims("dy", dy, 2)
    c.dims("x", x, 2)
    if dw.dim() == 2:
        dw = dw.unsqueeze(0)
    c.dims("dw", dw, 3)
    rows, n = dy.shape
    experts, k = dw.shape[0], x.shape[1]
    if dw.dtype not in _DTYPES:
        raise TypeError(f"muon_expert_weight_grad: unsupported dtype {dw.dtype}")
    args = _pack_weight_grad(rows, n, k, experts, *c.rows_of("dy", dy, (rows, n), _BF16),
                             *c.rows_of("x", x, (rows, k), _BF16), c.flat("offsets", offsets, (experts + 1,), _I32),
                             *c.stack("dw", dw, (experts, n, k), (dw.dtype,)), _DTYPES[dw.dtype])
    c.run(lib().muon_expert_weight_grad, args, *c.workspace(workspace), stream=stream)
