"""C ABI of the row operators on the CPU: every declared symbol is exported
and every argument error is caught before anything is launched.  Host buffers
stand in for device pointers, so these run only where no GPU is visible."""
import ctypes as C
import os
import re

import numpy as np
import pytest
import torch

from matrix_optimizer_amd import binding as B
from matrix_optimizer_amd import block as K

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, SMALL = B.MUON_ERR_INVALID_ARG, B.MUON_ERR_UNSUPPORTED, B.MUON_ERR_WORKSPACE_TOO_SMALL


def test_library_exports_every_declared_symbol():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "muon_block.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(muon_[a-z_]+)\s*\(", src))
    assert names == set(K.EXPORTED)
    for n in names:
        assert hasattr(K.lib(), n), n
    assert K.muon_block_abi_version() == 1


@pytest.fixture
def mem():
    if torch.cuda.device_count() > 0:
        pytest.skip("fake-pointer validation tests run only where no GPU is visible")
    raw = np.full(1 << 20, 0x5A, np.uint8)
    base = (raw.ctypes.data + 255) & ~255
    yield lambda i: base + i * 16384     # disjoint 16 KiB slots
    assert np.all(raw == 0x5A)


def _norm(mem, **over):
    a = K.muon_norm_args(rows=4, cols=64, x=mem(0), x_stride=64, residual=mem(1), residual_stride=64, h=mem(2),
                         h_stride=64, y=mem(3), y_stride=64, weight=mem(4), rstd=mem(5), dtype=1, weight_dtype=0,
                         y_dtype=1, group=0, eps=1e-6)
    drop = over.pop("drop", None)
    for k, v in over.items():
        setattr(a, k, v)
    if drop is not None:
        a.dropout = C.addressof(drop)
    return K.lib().muon_norm_forward(C.byref(a), None)


def test_norm_forward_refusals(mem):
    for bad in (dict(rows=-1), dict(cols=0), dict(x=None), dict(y=None), dict(x=mem(0) + 1), dict(dtype=2),
                dict(dtype=-1), dict(weight_dtype=7), dict(y_dtype=4), dict(y_dtype=-1), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(x_stride=63), dict(residual_stride=0),
                dict(h_stride=-64), dict(y_stride=1), dict(x_stride=1 << 62), dict(group=32), dict(scales=mem(6)),
                dict(y_dtype=2), dict(y_dtype=2, scales=mem(6), scales_stride=0, group=32),
                dict(y_dtype=2, scales=mem(6), scales_stride=1, group=32),     # two groups a row
                dict(y_dtype=2, scales=mem(6), scales_stride=2, group=16),
                dict(y_dtype=2, scales=mem(6) + 2, scales_stride=2, group=32),
                dict(rstd=mem(5) + 2), dict(weight=mem(4) + 2),
                dict(y=mem(0)), dict(y=mem(1)), dict(y=mem(2)), dict(h=mem(0) + 2), dict(h=mem(0), h_stride=65),
                dict(rstd=mem(3)), dict(weight=mem(3)), dict(y=mem(0) + 3 * 128 + 126),
                dict(drop=K.muon_dropout_spec(-0.1, 0, 0, None)), dict(drop=K.muon_dropout_spec(1.5, 0, 0, None)),
                dict(drop=K.muon_dropout_spec(float("nan"), 0, 0, None)),
                dict(drop=K.muon_dropout_spec(0.1, 0, 0, mem(7) + 4)),
                dict(drop=K.muon_dropout_spec(0.1, 0, 0, mem(3)))):
        assert _norm(mem, **bad) == INVALID, bad
    assert _norm(mem, rows=1 << 31) == UNSUPPORTED
    assert _norm(mem, cols=1 << 31, x_stride=1 << 31) == UNSUPPORTED
    assert K.lib().muon_norm_forward(None, None) == INVALID
    assert _norm(mem, rows=0, x=None, y=None) == B.MUON_OK


def test_interleaved_rows_are_no_overlap(mem):
    """Column ranges of one wider buffer interleave; a range that runs into another is refused."""
    L = K.lib()
    spec = K.muon_dropout_spec(0.5, 1, 1, None)

    def call(xo, yo, rows=4, cols=64, xs=128, ys=128):
        return L.muon_dropout(rows, cols, mem(0) + xo, xs, mem(0) + yo, ys, 1, C.byref(spec), None)

    assert call(0, 126) == INVALID            # one element into x's columns
    assert call(0, 130) == INVALID            # y's last column is the next row's first of x
    assert call(130, 0) == INVALID
    assert call(0, 256 * 2 + 64) == INVALID   # two rows down, half into
    assert call(0, 0, ys=192) == INVALID      # same base, another stride
    assert call(0, 2, rows=1) == INVALID
    # allowed layouts reach the launch, which fails here: there is no device
    assert call(0, 128) == B.MUON_ERR_HIP
    assert call(0, 0) == B.MUON_ERR_HIP


def _grad(mem, ws=None, wsb=None, **over):
    a = K.muon_norm_grad_args(rows=4, cols=64, dy=mem(0), dy_stride=64, h=mem(1), h_stride=64, dh=mem(2), dh_stride=64,
                              dresidual=mem(3), dresidual_stride=64, dx=mem(4), dx_stride=64, rstd=mem(5),
                              weight=mem(6), dweight=mem(7), dtype=0, weight_dtype=0)
    for k, v in over.items():
        setattr(a, k, v)
    need = K.norm_workspace_bytes(4, 64)
    return K.lib().muon_norm_backward(C.byref(a), mem(8) if ws is None else ws, need if wsb is None else wsb, None)


def test_norm_backward_refusals(mem):
    for bad in (dict(rows=-1), dict(cols=0), dict(dy=None), dict(h=None), dict(rstd=None), dict(dtype=3),
                dict(weight_dtype=2), dict(dy_stride=1), dict(dresidual=mem(0)), dict(dresidual=mem(1)),
                dict(dx=mem(3)), dict(dresidual=mem(2), dresidual_stride=65), dict(dx=mem(2)), dict(dweight=mem(0)),
                dict(dweight=mem(7) + 1), dict(dweight=mem(8)), dict(dresidual=None, dx=None, dweight=None)):
        assert _grad(mem, **bad) == INVALID, bad
    assert _grad(mem, wsb=K.norm_workspace_bytes(4, 64) - 1) == SMALL
    assert _grad(mem, ws=mem(8) + 16) == INVALID
    assert _grad(mem, ws=0) == INVALID
    assert _grad(mem, rows=0, dweight=None, wsb=0) == B.MUON_OK
    out = C.c_size_t(7)
    assert K.lib().muon_norm_workspace_bytes(-1, 4, C.byref(out)) == INVALID
    assert K.lib().muon_norm_workspace_bytes(4, 0, C.byref(out)) == INVALID
    assert K.lib().muon_norm_workspace_bytes(4, 4, None) == INVALID
    assert K.lib().muon_norm_workspace_bytes(1 << 31, 4, C.byref(out)) == UNSUPPORTED
    assert out.value == 7
    for rows, cols in ((0, 1), (1, 1), (100000, 8192), (5, 100000)):
        assert K.norm_workspace_bytes(rows, cols) % 256 == 0


def test_dropout_refusals(mem):
    L, ok = K.lib(), K.muon_dropout_spec(0.5, 1, 1, None)
    call = lambda rows=4, cols=64, x=mem(0), y=mem(1), dt=0, spec=ok: L.muon_dropout(  # noqa: E731
        rows, cols, x, 64, y, 64, dt, C.byref(spec) if spec else None, None)
    assert call(rows=-1) == call(cols=0) == call(x=None) == call(y=None) == call(dt=2) == call(spec=None) == INVALID
    assert call(x=mem(0) + 2) == INVALID and call(y=mem(0) + 4) == INVALID
    assert call(spec=K.muon_dropout_spec(2.0, 1, 1, None)) == INVALID
    assert call(rows=1 << 31) == UNSUPPORTED
    assert call(rows=0) == B.MUON_OK


def test_dropout_seed_apart_from_the_output(mem):
    """{seed, offset} on the device may be neither inside y nor inside an x that is y, as in the norm's calls."""
    L = K.lib()

    def call(seed, y=mem(1)):
        spec = K.muon_dropout_spec(0.5, 1, 1, seed)
        return L.muon_dropout(4, 64, mem(0), 64, y, 64, 0, C.byref(spec), None)

    assert call(mem(1)) == call(mem(1) + 1016) == call(mem(1) - 8) == call(mem(0) + 8, mem(0)) == INVALID
    assert call(mem(1) + 4) == INVALID                                  # not 8-byte aligned
    # apart, or inside an input: these reach the launch, which fails here
    assert call(mem(1) + 1024) == call(mem(1) - 16) == call(mem(0)) == B.MUON_ERR_HIP


def _route(mem, spec=None, **over):
    s = K.muon_route_spec(1, 4, 4, 2, 2, 1, 1.0)
    for k, v in (spec or {}).items():
        setattr(s, k, v)
    a = K.muon_route_args(rows=8, num_experts=16, logits=mem(0), logits_stride=16, bias=mem(1), token_mask=mem(2),
                          experts=mem(3), weights=mem(4), scores=mem(5), dtype=1)
    for k, v in over.items():
        setattr(a, k, v)
    return K.lib().muon_route_forward(C.byref(s), C.byref(a), None)


def test_route_forward_refusals(mem):
    for bad in (dict(score=2), dict(score=-1), dict(top_k=0), dict(top_k=9), dict(top_k=17), dict(groups=0),
                dict(groups=3), dict(groups=-4), dict(top_groups=0), dict(top_groups=5), dict(group_top=0),
                dict(group_top=3), dict(renormalise=2), dict(scale=0.0), dict(scale=float("inf")),
                dict(scale=float("nan")), dict(scale=-1.0)):
        assert _route(mem, bad) == INVALID, bad
    for bad in (dict(rows=-1), dict(num_experts=0), dict(logits=None), dict(experts=None), dict(weights=None),
                dict(logits=mem(0) + 1), dict(logits_stride=15), dict(dtype=2), dict(bias=mem(1) + 2),
                dict(experts=mem(0)), dict(weights=mem(3) + 64), dict(scores=mem(4)), dict(experts=mem(2)),
                dict(weights=mem(1))):
        assert _route(mem, **bad) == INVALID, bad
    assert _route(mem, dict(groups=1, top_groups=1), num_experts=1025, logits_stride=1025) == UNSUPPORTED
    assert _route(mem, dict(groups=1, top_groups=1, top_k=33), num_experts=64, logits_stride=64) == UNSUPPORTED
    assert _route(mem, rows=1 << 31) == UNSUPPORTED
    assert _route(mem, rows=0, logits=None) == B.MUON_OK
    assert K.lib().muon_route_forward(None, None, None) == INVALID


def test_route_backward_refusals(mem):
    def call(spec=None, **over):
        s = K.muon_route_spec(0, 4, 0, 0, 0, 1, 1.0)     # groups are not read
        for k, v in (spec or {}).items():
            setattr(s, k, v)
        a = K.muon_route_grad_args(rows=8, num_experts=16, logits=mem(0), logits_stride=16, experts=mem(1),
                                   weights=mem(2), dweights=mem(3), dscores=mem(4), dlogits=mem(5), dlogits_stride=16,
                                   dtype=0)
        for k, v in over.items():
            setattr(a, k, v)
        return K.lib().muon_route_backward(C.byref(s), C.byref(a), None)

    for bad in (dict(score=2), dict(top_k=0), dict(top_k=17), dict(renormalise=-1), dict(scale=0.0)):
        assert call(bad) == INVALID, bad
    for bad in (dict(logits=None), dict(experts=None), dict(weights=None), dict(dweights=None), dict(dlogits=None),
                dict(dlogits=mem(0)), dict(dlogits=mem(4)), dict(dlogits_stride=8), dict(logits_stride=8),
                dict(dscores=mem(4) + 1), dict(dtype=2), dict(rows=-3)):
        assert call(**bad) == INVALID, bad
    assert call(num_experts=2000, logits_stride=2000, dlogits_stride=2000) == UNSUPPORTED
    assert call(rows=0, logits=None) == B.MUON_OK


def test_order_and_balance_refusals(mem):
    L = K.lib()
    need = K.route_order_workspace_bytes(100, 16)

    def order(n=100, e=16, x=mem(0), c=mem(1), o=mem(2), d=mem(3), p=mem(4), w=mem(5), wb=need):
        return L.muon_route_order(n, e, x, c, o, d, p, w, wb, None)

    assert order(n=-1) == order(e=0) == order(x=None) == order(c=None) == order(o=None) == order(d=None) == INVALID
    assert order(p=None) == order(w=None) == order(w=mem(5) + 16) == order(x=mem(0) + 2) == order(p=mem(3)) == INVALID
    assert order(o=mem(1) + 60) == order(d=mem(0)) == INVALID
    assert order(wb=need - 1) == SMALL
    assert order(n=(1 << 31) - 1) == order(e=1025) == UNSUPPORTED
    # no pairs: no workspace, and nothing but counts and offsets (the launch fails here, there is no device)
    assert K.route_order_workspace_bytes(0, 16) == 0
    assert order(n=0, x=None, d=None, p=None, w=None, wb=0) == B.MUON_ERR_HIP
    assert order(n=0, c=None) == INVALID
    bal = lambda n=16, c=mem(0), b=mem(1), o=mem(2), r=0.1: L.muon_route_balance(n, c, b, o, r, None)  # noqa: E731
    assert bal(n=0) == bal(c=None) == bal(b=None) == bal(o=None) == bal(r=float("nan")) == bal(o=mem(0)) == INVALID
    assert bal(o=mem(1) + 4) == INVALID
    assert bal(n=1025) == UNSUPPORTED


def test_order_largest_number_of_pairs():
    """num_pairs < 2^31 - 2^16."""
    L, out, most = K.lib(), C.c_size_t(7), (1 << 31) - (1 << 16)
    assert L.muon_route_order_workspace_bytes(most, 256, C.byref(out)) == UNSUPPORTED and out.value == 7
    assert L.muon_route_order_workspace_bytes(most - 1, 256, C.byref(out)) == B.MUON_OK and out.value > 7


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError):
        K.muon_dropout(x, x, K.Dropout(0.1))
    with pytest.raises(ValueError):
        K.muon_dropout(torch.zeros(8), x, K.Dropout(0.1))
    with pytest.raises(TypeError):
        K.muon_dropout(x.double(), x, K.Dropout(0.1))
    with pytest.raises(ValueError):
        K.Route(2, score="other").to_c()
    with pytest.raises(ValueError):
        K.Dropout(0.1, device=torch.zeros(2, dtype=torch.int64)).to_c()
