"""C ABI and binding of the expert operators on the CPU: every declared symbol
is exported and every argument error is caught before anything is launched.
Host buffers stand in for device pointers, so the fake-pointer tests run only
where no GPU is visible."""
import ctypes as C
import os
import re

import numpy as np
import pytest
import torch

from matrix_optimizer_amd import binding as B
from matrix_optimizer_amd import experts as X

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED = B.MUON_OK, B.MUON_ERR_INVALID_ARG, B.MUON_ERR_UNSUPPORTED
SMALL, HIP = B.MUON_ERR_WORKSPACE_TOO_SMALL, B.MUON_ERR_HIP


def test_library_exports_every_declared_symbol():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "muon_experts.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(muon_[a-z_]+)\s*\(", src))
    assert names == set(X.EXPORTED)
    for n in names:
        assert hasattr(X.lib(), n), n
    assert X.muon_experts_abi_version() == 1


def test_structs_have_the_headers_fields():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "muon_experts.h")).read(), flags=re.S)
    for body, name in re.findall(r"typedef struct \{(.*?)\} (muon_\w+);", src, flags=re.S):
        fields = []
        for decl in filter(None, (d.strip() for d in body.split(";"))):
            kind, names = re.match(r"((?:const )?\w+\*?)\s+(.*)", decl, flags=re.S).groups()
            for n in names.split(","):
                c = C.c_void_p if "*" in kind else {"int64_t": C.c_int64, "int32_t": C.c_int32}[kind]
                fields.append((n.strip(), c))
        assert fields == getattr(X, name)._fields_, name


@pytest.fixture
def mem():
    if torch.cuda.device_count() > 0:
        pytest.skip("fake-pointer validation tests run only where no GPU is visible")
    raw = np.full(1 << 20, 0x5A, np.uint8)
    base = (raw.ctypes.data + 255) & ~255
    yield lambda i: base + i * 32768     # disjoint 32 KiB slots
    assert np.all(raw == 0x5A)


def _caller(fn, struct, **defaults):
    def call(**over):
        return getattr(X.lib(), fn)(C.byref(struct(**{**defaults, **over})), None)
    return call


def _refused(call, cases, status=INVALID):
    for bad in cases:
        assert call(**bad) == status, bad


def test_gather_refusals(mem):
    call = _caller("muon_expert_gather", X.muon_gather_args, rows=4, cols=64, top_k=2, x=mem(0), x_stride=64, out=mem(1),
                   out_stride=64, scales=mem(2), scales_stride=1, out_scales=mem(3), out_scales_stride=1, groups=1,
                   order=mem(4), dtype=2)
    _refused(call, (dict(rows=-1), dict(cols=0), dict(top_k=0), dict(x=None), dict(out=None), dict(order=None),
                    dict(out_scales=None), dict(scales=None), dict(groups=0), dict(dtype=4), dict(dtype=-1),
                    dict(x_stride=63), dict(out_stride=0), dict(scales_stride=0), dict(out_scales=mem(3) + 2),
                    dict(order=mem(4) + 1), dict(out=mem(0)), dict(out=mem(4)), dict(out_scales=mem(2)),
                    dict(out_scales=mem(1) + 4), dict(dtype=1, x=mem(0) + 1), dict(dtype=0, out=mem(1) + 2),
                    dict(scales=None, out_scales=None)))
    _refused(call, (dict(rows=1 << 31), dict(rows=1 << 20, top_k=1 << 11), dict(top_k=1 << 31),
                    dict(cols=1 << 31, x_stride=1 << 31, out_stride=1 << 31)), UNSUPPORTED)
    assert X.lib().muon_expert_gather(None, None) == INVALID
    assert call(rows=0, x=None, out=None) == OK
    assert call() == call(scales=None, out_scales=None, groups=0) == HIP    # complete: there is no device


def test_combine_refusals(mem):
    call = _caller("muon_expert_combine", X.muon_combine_args, rows=4, cols=64, top_k=2, places=8, position=mem(0),
                   weights=mem(1), y=mem(2), y_stride=64, base=mem(3), base_stride=64, out=mem(4), out_stride=64,
                   dtype=1, out_dtype=1)
    _refused(call, (dict(rows=-1), dict(cols=0), dict(top_k=0), dict(places=-1), dict(position=None), dict(y=None),
                    dict(out=None), dict(dtype=2), dict(out_dtype=3), dict(y_stride=63), dict(base_stride=1),
                    dict(out_stride=-64), dict(weights=mem(1) + 2), dict(position=mem(0) + 2), dict(out=mem(2)),
                    dict(out=mem(0)), dict(out=mem(1)), dict(out=mem(3), out_stride=65), dict(out=mem(3) + 2),
                    dict(out_dtype=0, out=mem(4) + 2)))
    _refused(call, (dict(top_k=33), dict(rows=1 << 31), dict(places=1 << 31), dict(rows=1 << 28, top_k=16)), UNSUPPORTED)
    assert X.lib().muon_expert_combine(None, None) == INVALID
    assert call(rows=0, y=None) == OK
    assert call() == call(out=mem(3)) == call(weights=None, base=None) == call(places=0, y=None) == HIP


def test_combine_backward_refusals(mem):
    call = _caller("muon_expert_combine_backward", X.muon_combine_grad_args, rows=4, cols=200, top_k=2, places=8,
                   position=mem(0), weights=mem(1), dout=mem(2), dout_stride=200, y=mem(3), y_stride=200, dy=mem(4),
                   dy_stride=200, dy8=mem(5), dy8_stride=200, scales=mem(6), scales_stride=2, dweights=mem(7), dtype=1,
                   dy8_dtype=2)
    _refused(call, (dict(rows=-1), dict(cols=0), dict(top_k=0), dict(places=-1), dict(position=None), dict(dout=None),
                    dict(y=None), dict(scales=None), dict(dy8=None), dict(dtype=2), dict(dy8_dtype=1), dict(dy8_dtype=4),
                    dict(scales_stride=1), dict(dy=mem(2)), dict(dy=mem(3)), dict(dy8=mem(4)), dict(scales=mem(5) + 4),
                    dict(dweights=mem(1)), dict(dweights=mem(7) + 1), dict(dy8=mem(0)), dict(dy_stride=199),
                    dict(dy=None, dy8=None, scales=None, dweights=None)))
    _refused(call, (dict(top_k=33), dict(rows=1 << 31)), UNSUPPORTED)
    assert call(rows=0, dout=None) == OK
    assert call() == call(dweights=None, y=None) == call(dy=None, dy8=None, scales=None) == HIP
    assert call(places=0, y=None, dy=None, dy8=None, scales=None) == HIP


def test_gate_refusals(mem):
    call = _caller("muon_gate_forward", X.muon_gate_args, rows=4, cols=200, a=mem(0), a_stride=400, y=mem(1), y_stride=200,
                   y8=mem(2), y8_stride=200, scales=mem(3), scales_stride=2, used=mem(4), dtype=1, y8_dtype=3)
    _refused(call, (dict(rows=-1), dict(cols=0), dict(a=None), dict(a_stride=399), dict(y_stride=199), dict(y8_stride=1),
                    dict(scales=None), dict(y8=None), dict(scales_stride=1), dict(dtype=2), dict(y8_dtype=0),
                    dict(used=mem(4) + 2), dict(used=mem(1)), dict(y=mem(0)), dict(y=mem(0) + 400), dict(y8=mem(1)),
                    dict(scales=mem(2)), dict(y=None, y8=None, scales=None)))
    _refused(call, (dict(rows=1 << 31), dict(cols=1 << 30, a_stride=1 << 31)), UNSUPPORTED)
    assert call(rows=0, a=None) == OK
    assert call() == call(y=None) == call(y8=None, scales=None) == call(used=None) == HIP


def test_gate_backward_refusals(mem):
    call = _caller("muon_gate_backward", X.muon_gate_grad_args, rows=4, cols=256, a=mem(0), a_stride=512, dy=mem(1),
                   dy_stride=256, da=mem(2), da_stride=512, da8=mem(3), da8_stride=512, scales=mem(4), scales_stride=4,
                   used=mem(5), dtype=1, da8_dtype=2)
    _refused(call, (dict(rows=-1), dict(cols=0), dict(a=None), dict(dy=None), dict(a_stride=511), dict(dy_stride=255),
                    dict(da_stride=511), dict(da8_stride=511), dict(scales_stride=3), dict(scales=None), dict(da8=None),
                    dict(da=mem(0)), dict(da8=mem(1)), dict(scales=mem(2)), dict(dtype=2), dict(da8_dtype=1),
                    dict(used=mem(3)), dict(da=None, da8=None, scales=None)))
    _refused(call, (dict(rows=1 << 31), dict(cols=200), dict(cols=1 << 30)), UNSUPPORTED)
    assert call(rows=0, a=None) == OK
    assert call() == call(cols=200, da8=None, scales=None) == call(da=None) == HIP


def test_quantise_refusals(mem):
    call = _caller("muon_quantise_blocks", X.muon_quantise_args, batch=2, rows=30, cols=64, x=mem(0), x_stride=64,
                   x_matrix=1920, q=mem(1), q_stride=64, q_matrix=1920, scales=mem(2), qt=mem(3), qt_stride=30,
                   qt_matrix=1920, scales_t=mem(4), dtype=1, q_dtype=2)
    _refused(call, (dict(batch=-1), dict(rows=-1), dict(cols=0), dict(x=None), dict(scales=None), dict(scales_t=None),
                    dict(q=None), dict(qt=None), dict(x_stride=63), dict(q_stride=63), dict(qt_stride=29),
                    dict(q_matrix=1919), dict(qt_matrix=0), dict(x_matrix=-1), dict(dtype=2), dict(q_dtype=1),
                    dict(q=mem(0)), dict(qt=mem(1)), dict(scales_t=mem(2)), dict(scales=mem(1) + 1920 + 4),
                    dict(x=mem(0) + 1), dict(q=None, qt=None, scales=None, scales_t=None), dict(x_matrix=1 << 62)))
    _refused(call, (dict(batch=1 << 31), dict(rows=1 << 31), dict(batch=1 << 20, rows=1 << 20, cols=1 << 20)), UNSUPPORTED)
    assert call(rows=0, x=None) == call(batch=0, x=None) == OK
    assert call() == call(q=None, scales=None) == call(qt=None, scales_t=None) == HIP
    assert call(batch=1, x_matrix=0, q_matrix=0, qt_matrix=0) == HIP
    # matrices that interleave: x's and q's columns of one wider buffer
    assert call(dtype=1, x=mem(5), x_stride=128, x_matrix=30 * 128, q=mem(5) + 128, q_stride=256, q_matrix=30 * 256) == HIP


def test_product_refusals(mem):
    call = _caller("muon_expert_product", X.muon_product_args, rows=6, n=130, k=140, num_experts=2, a=mem(0), a_stride=140,
                   a_scales=mem(1), a_scales_stride=2, w=mem(2), w_stride=140, w_matrix=130 * 140, w_scales=mem(4),
                   offsets=mem(5), out=mem(6), out_stride=130, a_dtype=2, w_dtype=3, out_dtype=1)
    _refused(call, (dict(rows=-1), dict(n=0), dict(k=0), dict(num_experts=0), dict(a=None), dict(a_scales=None),
                    dict(w=None), dict(w_scales=None), dict(offsets=None), dict(out=None), dict(a_stride=139),
                    dict(a_scales_stride=1), dict(w_stride=139), dict(w_matrix=18199), dict(out_stride=129),
                    dict(a_dtype=1), dict(w_dtype=0), dict(out_dtype=2), dict(out=mem(0)), dict(out=mem(2) + 40),
                    dict(out=mem(6) + 1), dict(out=mem(5)), dict(a_scales=mem(1) + 2), dict(w_scales=mem(4) + 1),
                    dict(offsets=mem(5) + 2), dict(out=mem(4))))
    _refused(call, (dict(rows=1 << 31), dict(n=1 << 31), dict(k=1 << 31), dict(num_experts=1025),
                    dict(num_experts=1024, n=1 << 30, k=1 << 30)), UNSUPPORTED)
    assert call(rows=0, a=None) == OK
    _refused(call, (dict(rows=(1 << 31) - 1, n=(1 << 31) - 1, k=1, w_stride=1, num_experts=1),), UNSUPPORTED)   # too many tiles
    assert call() == call(num_experts=1, offsets=None, w_matrix=0) == HIP


def test_weight_grad_refusals(mem):
    defaults = dict(rows=6, n=30, k=40, num_experts=2, dy=mem(0), dy_stride=30, x=mem(1), x_stride=40, offsets=mem(2),
                    dw=mem(3), dw_stride=40, dw_matrix=1200, dw_dtype=0)

    def call(ws=mem(4), wsb=1 << 14, **over):
        return X.lib().muon_expert_weight_grad(C.byref(X.muon_weight_grad_args(**{**defaults, **over})), ws, wsb, None)

    _refused(call, (dict(rows=-1), dict(n=0), dict(k=0), dict(num_experts=0), dict(dy=None), dict(x=None),
                    dict(offsets=None), dict(dw=None), dict(dy_stride=29), dict(x_stride=39), dict(dw_stride=39),
                    dict(dw_matrix=1199), dict(dw_dtype=2), dict(dw=mem(0)), dict(dw=mem(1) + 4), dict(dw=mem(2)),
                    dict(dy=mem(0) + 1), dict(dw=mem(3) + 2)))
    _refused(call, (dict(rows=1 << 31), dict(n=1 << 31), dict(num_experts=1025)), UNSUPPORTED)
    assert call() == call(num_experts=1, offsets=None) == HIP
    assert call(rows=0, dy=None, x=None, offsets=None, num_experts=1) == HIP    # zeros are still written
    out = C.c_size_t(7)
    f = X.lib().muon_expert_weight_grad_workspace_bytes
    assert f(-1, 1, 1, 1, C.byref(out)) == f(1, 0, 1, 1, C.byref(out)) == f(1, 1, 0, 1, C.byref(out)) == INVALID
    assert f(1, 1, 1, 0, C.byref(out)) == f(1, 1, 1, 1, None) == INVALID
    assert f(1 << 31, 1, 1, 1, C.byref(out)) == f(1, 1025, 1, 1, C.byref(out)) == UNSUPPORTED
    assert out.value == 7
    for args in ((0, 1, 1, 1), (100000, 1, 64, 64), (50000, 64, 7168, 2048), (100000, 3, 300, 200)):
        need = X.expert_weight_grad_workspace_bytes(*args)
        assert need % 256 == 0
        if need:
            rows, e, n, k = args
            sizes = dict(rows=rows, num_experts=e, n=n, k=k, dy_stride=n, x_stride=k, dw_stride=k, dw_matrix=n * k)
            assert call(wsb=need - 1, **sizes) == SMALL
            far = 1 << 46     # addresses apart: nothing is read before the launch
            sizes.update(dy=far, x=2 * far, dw=3 * far)
            assert call(ws=4 * far + 16, wsb=need, **sizes) == call(ws=None, wsb=need, **sizes) == INVALID
            assert call(ws=3 * far, wsb=need, **sizes) == INVALID


def test_binding_refuses_what_does_not_fit():
    x, y = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16)
    order, pos = torch.zeros(8, dtype=torch.int32), torch.zeros(4, 2, dtype=torch.int32)
    e = torch.zeros(4, 64, dtype=torch.float8_e4m3fn)
    for call in (lambda: X.muon_expert_gather(order, x, y), lambda: X.muon_expert_combine(pos, y, x),
                 lambda: X.muon_expert_combine_backward(pos, x, dy=y), lambda: X.muon_gate_forward(x, y=x),
                 lambda: X.muon_gate_backward(x, x, da=x), lambda: X.muon_quantise_blocks(x, e, torch.zeros(1, 1)),
                 lambda: X.muon_expert_product(e, torch.zeros(4, 1), e, torch.zeros(1, 1), x),
                 lambda: X.muon_expert_weight_grad(x, x, torch.zeros(64, 64))):
        with pytest.raises(ValueError):     # host tensors
            call()


class _OnDevice(torch.Tensor):
    """A host tensor that says it is on device 0, for the checks of shapes and types."""
    def get_device(self):
        return 0


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(_OnDevice)


def test_binding_checks_shapes_and_types():
    if torch.cuda.device_count() > 0:
        pytest.skip("stand-in tensors only where no GPU is visible")
    f8, f32, i32 = torch.float8_e4m3fn, torch.float32, torch.int32
    x, y, order, pos = _t(4, 64), _t(8, 64), _t(8, dtype=i32), _t(4, 2, dtype=i32)
    e, s = _t(4, 64, dtype=f8), _t(4, 1, dtype=f32)
    w, ws = _t(3, 40, 64, dtype=f8), _t(3, 1, 1, dtype=f32)
    bad = [
        lambda: X.muon_expert_gather(_t(7, dtype=i32), x, y), lambda: X.muon_expert_gather(order, x, _t(7, 64)),
        lambda: X.muon_expert_gather(order, x, _t(8, 64, dtype=f32)), lambda: X.muon_expert_gather(order, x, y, scales=s),
        lambda: X.muon_expert_gather(order, x, y, scales=s, out_scales=_t(8, 2, dtype=f32)),
        lambda: X.muon_expert_gather(order.long(), x, y), lambda: X.muon_expert_gather(order, x[0], y),
        lambda: X.muon_expert_gather(order, _t(64, 4).t(), y),
        lambda: X.muon_expert_combine(pos, y, _t(5, 64)), lambda: X.muon_expert_combine(pos, y, x, weights=_t(4, 2)),
        lambda: X.muon_expert_combine(pos, y, x, base=_t(4, 64, dtype=f32)), lambda: X.muon_expert_combine(order, y, x),
        lambda: X.muon_expert_combine_backward(pos, x, dweights=_t(4, 2, dtype=f32)),
        lambda: X.muon_expert_combine_backward(pos, x, dy8=_t(8, 64, dtype=f8)),
        lambda: X.muon_expert_combine_backward(pos, x, y=y, dy=_t(7, 64)),
        lambda: X.muon_expert_combine_backward(_t(5, 2, dtype=i32), x, dy=y),
        lambda: X.muon_gate_forward(_t(4, 63), y=_t(4, 31)), lambda: X.muon_gate_forward(x, y=x),
        lambda: X.muon_gate_forward(x, y8=_t(4, 32, dtype=f8)), lambda: X.muon_gate_forward(x, y=_t(4, 32), used=order),
        lambda: X.muon_gate_backward(x, x, da=x), lambda: X.muon_gate_backward(x, _t(4, 32), da=_t(4, 32)),
        lambda: X.muon_quantise_blocks(x, q=e), lambda: X.muon_quantise_blocks(x, q=e, scales=_t(2, 1, dtype=f32)),
        lambda: X.muon_quantise_blocks(x, q=e, scales=_t(1, 1, dtype=f32), qt=_t(64, 4, dtype=torch.float8_e5m2),
                                       scales_t=_t(1, 1, dtype=f32)),
        lambda: X.muon_quantise_blocks(_t(4), q=e, scales=s),
        lambda: X.muon_expert_product(e, s, w, ws, _t(4, 41), _t(4, dtype=i32)),
        lambda: X.muon_expert_product(e, s, w, ws, _t(4, 40), _t(3, dtype=i32)),
        lambda: X.muon_expert_product(e, s, w, _t(3, 2, 1, dtype=f32), _t(4, 40), _t(4, dtype=i32)),
        lambda: X.muon_expert_product(x, s, w, ws, _t(4, 40), _t(4, dtype=i32)),
        lambda: X.muon_expert_product(e, _t(4, 2, dtype=f32), w, ws, _t(4, 40), _t(4, dtype=i32)),
        lambda: X.muon_expert_weight_grad(x, _t(5, 32), _t(3, 64, 32), _t(4, dtype=i32)),
        lambda: X.muon_expert_weight_grad(x, _t(4, 32), _t(3, 32, 64), _t(4, dtype=i32)),
        lambda: X.muon_expert_weight_grad(x, _t(4, 32, dtype=f32), _t(3, 64, 32), _t(4, dtype=i32)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print(i)
    for call in (lambda: X.muon_expert_gather(order, x.double(), y), lambda: X.muon_expert_combine(pos, y, x.half()),
                 lambda: X.muon_gate_forward(x.half(), y=x), lambda: X.muon_quantise_blocks(x.half(), q=e, scales=s),
                 lambda: X.muon_expert_product(e, s, w, ws, _t(4, 40, dtype=torch.float16), _t(4, dtype=i32)),
                 lambda: X.muon_expert_weight_grad(x, x, _t(64, 64, dtype=torch.float16))):
        with pytest.raises(TypeError):
            call()


def test_matrices_neither_repeat_nor_interleave(mem):
    """(rows - 1) * stride + columns is the least distance of a call's matrices, inputs' too."""
    call = _caller("muon_quantise_blocks", X.muon_quantise_args, batch=2, rows=30, cols=64, x=mem(0), x_stride=70,
                   x_matrix=29 * 70 + 64, q=mem(1), q_stride=70, q_matrix=29 * 70 + 64, scales=mem(2), dtype=1, q_dtype=2)
    assert call() == HIP
    _refused(call, (dict(x_matrix=0), dict(x_matrix=29 * 70 + 63), dict(x_stride=140, x_matrix=70),
                    dict(q_matrix=29 * 70 + 63), dict(q_stride=140, q_matrix=70)))
