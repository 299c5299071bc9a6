"""The norm and dropout of muon_block.h on the GPU against the float64 oracle.

Tolerances, set from the arithmetic: an output of type t is one rounding
(eps(t) / 2 relative: bf16 2^-8, fp32 2^-24, e4m3 2^-4, e5m2 2^-3, and half a
subnormal step near zero) off the fp32 value, and that value is off the exact
one by the fp32 operations before it.  A row's sum of n squares, formed by at
least 256 lanes and added in a tree, takes at most n / 256 + 16 roundings in a
row; a handful follow.  SLACK(n) = (n / 256 + 32) 2^-24 relative to the terms'
magnitudes covers them.
"""
import numpy as np
import pytest
import torch

from matrix_optimizer_amd import binding as B
from matrix_optimizer_amd import block as K
from oracle import block_oracle as O

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -4, "e5m2": 2.0 ** -3}
SUB = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "e4m3": 2.0 ** -10, "e5m2": 2.0 ** -17}   # half a subnormal step
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    K.lib()


def slack(n):
    return (n / 256 + 32) * 2.0 ** -24


def f64(t):
    return None if t is None else t.detach().to(torch.float64).cpu().numpy()


def rows(rng, r, c, kind, scale=1.0, pad=0, shift=0):
    """Normal values [r, c] of a type; pad / shift: as columns shift.. of a buffer `pad` columns wider."""
    full = torch.from_numpy(rng.standard_normal((r, c + pad)).astype(np.float32) * np.float32(scale)).cuda().to(T[kind])
    return full[:, shift:shift + c]


def out(r, c, kind, pad=0, shift=0):
    """An output inside a buffer filled with 7, to show that nothing else is written."""
    full = torch.full((r, c + pad), 7.0, device="cuda").to(T[kind])
    return full, full[:, shift:shift + c]


def check_padding(full, c, shift):
    f = full.float()
    assert bool((f[:, :shift] == 7).all()) and bool((f[:, shift + c:] == 7).all())


def close(got, ref, kind, terms, n, what):
    """|got - ref| within a rounding of ref and the fp32 slack relative to `terms`."""
    bound = HALF[kind] * np.abs(ref) * (1 + 2.0 ** -8) + SUB[kind] + slack(n) * terms
    err = np.abs(got - ref)
    assert np.all(err <= bound), f"{what}: {np.max(err / bound):.3g} of the bound"


SHAPES = [(1, 1), (2, 7), (1, 8), (3, 9), (5, 64), (4, 129), (3, 1000), (2, 2048), (7, 2051), (2, 4096), (3, 8200),
          (1, 16384), (2, 16392), (1, 40001), (300, 256), (1100, 72)]


def run_forward(rng, r, c, kind, ykind, group=0, residual=True, weight="f32", drop=None, pad=0, shift=0, inplace=""):
    x = rows(rng, r, c, kind, 1.0, pad, shift)
    res = rows(rng, r, c, kind, 2.0, pad, shift) if residual else None
    w = rows(rng, 1, c, weight, 0.2).reshape(-1) + 1 if weight else None
    xv, rv = f64(x), f64(res)
    if inplace:
        hfull, h = None, {"x": x, "residual": res}[inplace]
    else:
        hfull, h = out(r, c, kind, pad, shift)
    yfull, y = out(r, c, ykind, pad, shift)
    rstd = torch.zeros(r, device="cuda")
    g = group or c
    scales = torch.zeros(r, -(-c // g), device="cuda") if ykind in O.FMAX else None
    d = K.Dropout(*drop) if drop else None
    K.muon_norm_forward(x, y, residual=res, h=h, weight=w, rstd=rstd, scales=scales, group=group, eps=EPS, dropout=d)
    torch.cuda.synchronize()
    z, ref_rstd, ref_y = O.norm_forward(xv, rv, f64(w), EPS, drop)
    terms = np.abs(z) + (0 if rv is None else np.abs(rv)) + np.abs(xv)
    close(f64(h), z, kind, terms, 1, "h")
    close(f64(rstd), ref_rstd, "f32", np.abs(ref_rstd), c, "rstd")
    yt = np.abs(ref_y) + terms * ref_rstd[:, None] * (1 if w is None else np.abs(f64(w))) * 2.0 ** -1
    if scales is None:
        close(f64(y), ref_y, ykind, yt, c, "y")
    else:
        s = O.scales_of(ref_y, ykind, group)
        big = O.scales_of(yt, ykind, group)
        close(f64(scales), s, "f32", big + s, c, "scales")
        per = np.repeat(f64(scales), g, axis=1)[:, :c]
        close(f64(y), ref_y / per, ykind, yt / per, c, "y / scale")
    for full in (hfull, yfull):
        if full is not None:
            check_padding(full, c, shift)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("r,c", SHAPES)
def test_norm_forward_shapes(r, c, kind):
    run_forward(np.random.default_rng(r * 100003 + c), r, c, kind, kind)


@pytest.mark.parametrize("r,c", SHAPES)
def test_norm_forward_8bit_row_scale(r, c):
    run_forward(np.random.default_rng(c), r, c, "bf16", "e4m3")


@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("ykind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("r,c", [(3, 1), (3, 31), (2, 129), (4, 1000), (2, 4096), (2, 5000), (1, 33000)])
def test_norm_forward_8bit_groups(r, c, ykind, group):
    run_forward(np.random.default_rng(group + c), r, c, "bf16" if c % 2 else "f32", ykind, group)


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("weight", [None, "f32", "bf16"])
@pytest.mark.parametrize("drop", [None, (0.1, 3, 1 << 40), (1.0, 5, 6), (0.0, 1, 1)])
def test_norm_forward_options(residual, weight, drop):
    run_forward(np.random.default_rng(4), 5, 777, "bf16", "f32", residual=residual, weight=weight, drop=drop)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("ykind", ["bf16", "e4m3"])
@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 8), (9, 3), (1, 1)])
def test_norm_forward_strides_and_alignment(kind, ykind, pad, shift):
    for r, c in ((5, 512), (3, 2049), (2, 17000)):
        run_forward(np.random.default_rng(5), r, c, kind, ykind, pad=pad, shift=shift, drop=(0.3, 9, 9))


@pytest.mark.parametrize("inplace", ["x", "residual"])
@pytest.mark.parametrize("c", [100, 4096, 40000])
@pytest.mark.parametrize("ykind", ["bf16", "e4m3"])
def test_norm_forward_in_place(inplace, c, ykind):
    run_forward(np.random.default_rng(6), 4, c, "bf16", ykind, inplace=inplace, drop=(0.2, 1, 2))


@pytest.mark.parametrize("c", [64, 5000, 40000])
def test_norm_forward_special_values(c):
    """Zero rows, NaN and infinity stay in their own row; an 8-bit NaN does not enter the group's maximum."""
    x = torch.ones(5, c, device="cuda")
    x[0] = 0
    x[1, 3] = float("nan")
    x[2, 5] = float("inf")
    x[3] = 1e-30
    y = torch.empty_like(x)
    K.muon_norm_forward(x, y, eps=EPS)
    assert bool((y[0] == 0).all()) and bool(y[1].isnan().all())
    assert bool(y[2, 5].isnan()) and bool((y[2, 6:] == 0).all())
    assert torch.allclose(y[3], torch.full_like(y[3], 1e-27), rtol=1e-5, atol=0)
    assert torch.allclose(y[4], torch.ones_like(y[4]), rtol=1e-5)
    for kind in ("e4m3", "e5m2"):
        q = torch.empty(5, c, device="cuda", dtype=T[kind])
        s = torch.empty(5, -(-c // 32), device="cuda")
        w = torch.ones(c, device="cuda")
        w[9] = float("nan")
        K.muon_norm_forward(x, q, weight=w, scales=s, group=32, eps=EPS)
        assert bool((s[0] == 1).all()) and bool((q[0].float()[torch.arange(c) != 9] == 0).all())
        assert bool(q[4].float()[9].isnan()) and int(q[4].float().isnan().sum()) == 1
        assert torch.allclose(s[4] * O.FMAX[kind], torch.ones_like(s[4]), rtol=1e-5)
        assert bool(q[1].float().isnan().all())


def test_norm_forward_tiny_scale():
    """y below 2^-126 FMAX keeps a normal scale."""
    x = torch.ones(1, 64, device="cuda")
    w = torch.full((64,), 1e-37, device="cuda")
    y, s = torch.empty(1, 64, device="cuda", dtype=T["e4m3"]), torch.empty(1, 1, device="cuda")
    K.muon_norm_forward(x, y, weight=w, scales=s, eps=0.0)
    assert s.item() == 2.0 ** -126
    close(f64(y), np.full((1, 64), float(w[0]) / 2.0 ** -126), "e4m3", 1e-37 / 2.0 ** -126, 64, "y")


EDGES = [63, 65, 127, 128, 255, 257, 511, 512, 513, 1023, 1024, 1025, 4095, 4097, 8192, 8193, 16383, 16385]


@pytest.mark.parametrize("c", EDGES)
def test_norm_widths_where_the_layout_changes(c):
    """Widths beside those at which a row goes to more lanes, to a workgroup, to more chunks a lane, to passes."""
    for r in (1, 5, 70):
        run_forward(np.random.default_rng(c), r, c, "bf16", "e4m3", 128, drop=(0.1, 1, c))
        run_forward(np.random.default_rng(c), r, c, "f32", "bf16", weight="bf16")
        run_backward(np.random.default_rng(c), r, c, "bf16", drop=(0.1, 1, c))
        run_backward(np.random.default_rng(c), r, c, "f32", stream=False)


def run_backward(rng, r, c, kind, weight="f32", stream=True, drop=None, pad=0, shift=0, dx=True, dr=True, inplace=False):
    h, dy = rows(rng, r, c, kind, 2.0, pad, shift), rows(rng, r, c, kind, 0.1, pad, shift)
    dh = rows(rng, r, c, kind, 0.1, pad, shift) if stream else None
    w = rows(rng, 1, c, weight, 0.2).reshape(-1) + 1 if weight else None
    rstd = torch.from_numpy((1 / np.sqrt((f64(h) ** 2).mean(1) + EPS)).astype(np.float32)).cuda()
    dhv = f64(dh)
    rfull, res = (None, dh) if inplace else out(r, c, kind, pad, shift) if dr else (None, None)
    xfull, dxt = out(r, c, kind, pad, shift) if dx else (None, None)
    dwt = torch.full((c,), 7.0, device="cuda")
    ws = torch.empty(max(K.norm_workspace_bytes(r, c), 256), dtype=torch.uint8, device="cuda")
    K.muon_norm_backward(dy, h, rstd, weight=w, dh=dh, dresidual=res, dx=dxt, dweight=dwt, workspace=ws,
                         dropout=K.Dropout(*drop) if drop else None)
    torch.cuda.synchronize()
    dz, dxr, dwr = O.norm_backward(f64(dy), f64(h), f64(rstd), f64(w), dhv, drop)
    xh = np.abs(f64(h) * f64(rstd)[:, None])
    g = np.abs(f64(dy)) * (1 if w is None else np.abs(f64(w)))
    terms = f64(rstd)[:, None] * (g + xh * (g * xh).mean(1, keepdims=True)) + (0 if dhv is None else np.abs(dhv))
    if res is not None:
        close(f64(res), dz, kind, terms, c, "dresidual")
    if dxt is not None:
        up = 1.0 if not drop or drop[0] == 1 else 1 / (1 - drop[0])
        close(f64(dxt), dxr, kind, terms * up * 1.01, c, "dx")
    # dweight: a column's sum over the rows, at most rows / 64 + 600 roundings in a row
    t = (np.abs(f64(dy)) * xh).sum(0)
    assert np.all(np.abs(f64(dwt) - dwr) <= (r / 64 + 600) * 2.0 ** -24 * t + 1e-30), "dweight"
    for full in (rfull, xfull):
        if full is not None:
            check_padding(full, c, shift)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("r,c", SHAPES)
def test_norm_backward_shapes(r, c, kind):
    run_backward(np.random.default_rng(r + c), r, c, kind)


@pytest.mark.parametrize("stream", [True, False])
@pytest.mark.parametrize("weight", [None, "f32", "bf16"])
@pytest.mark.parametrize("drop", [None, (0.1, 3, 1 << 40), (1.0, 5, 6)])
def test_norm_backward_options(stream, weight, drop):
    run_backward(np.random.default_rng(7), 6, 777, "bf16", weight, stream, drop)


@pytest.mark.parametrize("dx,dr", [(True, False), (False, True), (False, False)])
def test_norm_backward_outputs(dx, dr):
    run_backward(np.random.default_rng(8), 9, 1500, "f32", dx=dx, dr=dr)
    run_backward(np.random.default_rng(8), 9, 1500, "bf16", stream=True, inplace=True, dx=dx)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("pad,shift", [(8, 8), (9, 3), (1, 1)])
def test_norm_backward_strides_and_alignment(kind, pad, shift):
    for r, c in ((5, 512), (3, 2049), (2, 17000)):
        run_backward(np.random.default_rng(9), r, c, kind, pad=pad, shift=shift, drop=(0.3, 9, 9))


@pytest.mark.parametrize("r,c", [(5000, 64), (3000, 1000), (2500, 4096)])
def test_norm_backward_many_rows(r, c):
    run_backward(np.random.default_rng(10), r, c, "bf16", drop=(0.1, 2, 3))


def test_norm_backward_against_differences():
    """The gradient of the forward call itself, by differences of its fp32 outputs summed in 64 bits."""
    rng = np.random.default_rng(11)
    r, c, eps = 2, 24, 2e-2
    x, res = rows(rng, r, c, "f32"), rows(rng, r, c, "f32")
    w, dy, dh = rows(rng, 1, c, "f32").reshape(-1), rows(rng, r, c, "f32"), rows(rng, r, c, "f32")
    drop = K.Dropout(0.25, 77, 3)

    def forward(x, res, w):
        h, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(r, device="cuda")
        K.muon_norm_forward(x, y, residual=res, h=h, weight=w, rstd=rstd, eps=EPS, dropout=drop)
        return h, y, rstd

    def loss(*v):
        h, y, _ = forward(*v)
        return float((y.double() * dy.double()).sum() + (h.double() * dh.double()).sum())

    h, _, rstd = forward(x, res, w)
    dx, dr, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(c, device="cuda")
    ws = torch.empty(max(K.norm_workspace_bytes(r, c), 256), dtype=torch.uint8, device="cuda")
    K.muon_norm_backward(dy, h, rstd, weight=w, dh=dh, dresidual=dr, dx=dx, dweight=dw, workspace=ws, dropout=drop)
    # differences: eps^2 / 6 of a third derivative of order 10 at unit-scale values, and 2^-24 of each of the
    # ~100 terms over 2 eps: 10 * 4e-4 / 6 + 100 * 6e-8 / 4e-2 < 1e-3
    for base, grad in ((x, dx), (res, dr), (w, dw)):
        for i in range(0, base.numel(), 5):
            v = [t.clone() for t in (x, res, w)]
            k = [j for j, t in enumerate((x, res, w)) if t is base][0]
            v[k].view(-1)[i] += eps
            hi = loss(*v)
            v[k].view(-1)[i] -= 2 * eps
            assert abs((hi - loss(*v)) / (2 * eps) - float(grad.view(-1)[i])) < 1e-3, (k, i)


# ---- dropout --------------------------------------------------------------
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("r,c,pad,shift", [(1, 1, 0, 0), (3, 7, 0, 0), (5, 8, 0, 0), (33, 1001, 9, 3), (2, 40000, 8, 8),
                                           (700, 64, 0, 0), (1, 300000, 0, 0)])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
def test_dropout(kind, r, c, pad, shift, p):
    rng = np.random.default_rng(c)
    x = rows(rng, r, c, kind, 1.0, pad, shift)
    full, y = out(r, c, kind, pad, shift)
    seed, off = 0xFEDCBA9876543210, (3 << 33) + 1
    K.muon_dropout(x, y, K.Dropout(p, seed, off))
    ref = O.dropout(f64(x), p, seed, off)
    got = f64(y)
    assert np.array_equal(got == 0, (ref == 0))
    assert np.all(np.abs(got - ref) <= HALF[kind] * np.abs(ref) * (1 + 2.0 ** -8) + 2.0 ** -24 * np.abs(ref))
    check_padding(full, c, shift)
    want = y.clone()
    K.muon_dropout(x, x, K.Dropout(p, seed, off))   # in place
    assert torch.equal(x, want)


def test_dropout_drops_nan_and_infinity():
    x = torch.full((4, 4096), float("nan"), device="cuda")
    x[1] = float("inf")
    y = torch.empty_like(x)
    K.muon_dropout(x, y, K.Dropout(0.5, 1, 2))
    keep = torch.from_numpy(O.keep_mask(4, 4096, 0.5, 1, 2)).cuda()
    assert bool((y[~keep] == 0).all()) and bool((~y[keep].isfinite()).all())


def test_far_rows():
    """Offsets past 2^31 elements: the last rows of a matrix of more than 2^31 elements."""
    r, c = 70000, 32768
    x = torch.empty(r, c, dtype=torch.bfloat16, device="cuda").normal_()
    y = torch.empty_like(x)
    d = (0.1, 11, 12)
    K.muon_dropout(x, y, K.Dropout(*d))
    keep = O.keep_mask(r, 16, *d)[-3:]
    got = f64(y[-3:, :16])
    assert np.array_equal(got != 0, keep & (f64(x[-3:, :16]) != 0))
    del y
    rstd = torch.empty(r, device="cuda")
    yn = torch.empty_like(x)
    K.muon_norm_forward(x, yn, rstd=rstd, eps=EPS)
    _, ref, yr = O.norm_forward(f64(x[-2:]), eps=EPS)
    close(f64(rstd[-2:]), ref, "f32", ref, c, "rstd")
    close(f64(yn[-2:]), yr, "bf16", np.abs(yr), c, "y")


# ---- streams, graphs, empty inputs ------------------------------------------
def test_zero_rows():
    e = torch.empty(0, 64, device="cuda")
    K.muon_dropout(e, e, K.Dropout(0.5))
    K.muon_norm_forward(e, e.clone(), eps=EPS)
    dw = torch.full((64,), 7.0, device="cuda")
    K.muon_norm_backward(e, e, torch.empty(0, device="cuda"), dresidual=e.clone(), dweight=dw)
    assert bool((dw == 0).all())


def test_refusals_leave_outputs():
    x = torch.randn(4, 64, device="cuda")
    y = torch.full_like(x, 7.0)
    for bad in (dict(p=1.5), dict(p=-1.0)):
        with pytest.raises(B.MuonError) as e:
            K.muon_dropout(x, y, K.Dropout(**bad))
        assert e.value.status == B.MUON_ERR_INVALID_ARG
    with pytest.raises(B.MuonError):
        K.muon_norm_forward(x, y, eps=-1.0)
    with pytest.raises(ValueError):
        K.muon_norm_forward(x, y[:2])
    with pytest.raises(ValueError):
        K.muon_norm_forward(x, y, residual=x.bfloat16())
    with pytest.raises(ValueError):
        K.muon_norm_forward(x.t(), y.t())
    with pytest.raises(ValueError):
        K.muon_norm_forward(x, y, weight=torch.ones(64))
    torch.cuda.synchronize()
    assert bool((y == 7).all())


def test_side_stream_and_reproducible():
    x, res = torch.randn(600, 1000, device="cuda"), torch.randn(600, 1000, device="cuda")
    s = torch.cuda.Stream()
    got = []
    for k in range(3):
        h, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(600, device="cuda")
        dr, dw = torch.empty_like(x), torch.empty(1000, device="cuda")
        ws = torch.empty(K.norm_workspace_bytes(600, 1000), dtype=torch.uint8, device="cuda")
        st = None
        if k == 1:
            s.wait_stream(torch.cuda.current_stream())
            st = s.cuda_stream
        K.muon_norm_forward(x, y, residual=res, h=h, rstd=rstd, eps=EPS, stream=st)
        K.muon_norm_backward(y, h, rstd, dresidual=dr, dweight=dw, workspace=ws, stream=st)
        if k == 1:
            torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        got.append((h, y, rstd, dr, dw))
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


def test_graph_replays_with_device_seed():
    """Captured once, replayed with new inputs and new seeds in the device tensor, eager work in between."""
    r, c = 37, 1500
    x, w = torch.randn(r, c, device="cuda"), torch.randn(c, device="cuda")
    seed = torch.tensor([1, 2], dtype=torch.int64, device="cuda")
    h, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(r, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty(c, device="cuda")
    ws = torch.empty(K.norm_workspace_bytes(r, c), dtype=torch.uint8, device="cuda")

    def step(d):
        K.muon_norm_forward(x, y, h=h, weight=w, rstd=rstd, eps=EPS, dropout=d)
        K.muon_norm_backward(y, h, rstd, weight=w, dx=dx, dweight=dw, workspace=ws, dropout=d)

    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        step(K.Dropout(0.2, device=seed))
    torch.cuda.current_stream().wait_stream(side)
    for k in range(4):
        x.normal_()
        seed.copy_(torch.tensor([100 + k, k << 40]))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (h, y, rstd, dx, dw)]
        for t in (h, y, rstd, dx, dw):
            t.zero_()
        step(K.Dropout(0.2, 100 + k, k << 40))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (h, y, rstd, dx, dw))), k


@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("ykind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("r,c", [(60000, 64), (4000, 1024), (1000, 4096), (200, 20000), (5001, 777)])
def test_norm_8bit_is_the_rounded_quotient(r, c, ykind, group):
    """The scale is max |y| times 1 / FMAX and the stored value y / scale as fp32 divides, rounded to 8 bits:
    equal bit for bit to the fp32 output of the same call divided on the host."""
    rng = np.random.default_rng(r + group)
    x, res = rows(rng, r, c, "bf16"), rows(rng, r, c, "bf16", 2.0)
    x[0, :16], res[0, :16] = -0.0, -0.0
    w = rows(rng, 1, c, "f32", 0.2).reshape(-1) + 1
    y, q = torch.empty(r, c, device="cuda"), torch.empty(r, c, device="cuda", dtype=T[ykind])
    g = group or c
    n = -(-c // g)
    s = torch.empty(r, n, device="cuda")
    K.muon_norm_forward(x, y, residual=res, weight=w, eps=EPS)
    K.muon_norm_forward(x, q, residual=res, weight=w, scales=s, group=group, eps=EPS)
    y, q, s = y.cpu(), q.cpu(), s.cpu()
    parts = torch.nn.functional.pad(y, (0, n * g - c)).reshape(r, n, g)
    scale = parts.abs().amax(2) * torch.tensor(1 / O.FMAX[ykind])
    assert torch.equal(s, scale)
    ref = (parts / scale[:, :, None]).reshape(r, n * g)[:, :c].clamp(-O.FMAX[ykind], O.FMAX[ykind]).to(T[ykind])
    off = q.view(torch.uint8) != ref.view(torch.uint8)
    assert int(off.sum()) == 0, f"{int(off.sum())} of {off.numel()}"


@pytest.mark.parametrize("ykind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("c", [64, 5000, 20000])
@pytest.mark.parametrize("group", [0, 32])
def test_norm_8bit_infinity(ykind, c, group):
    """An infinite y makes its group's scale infinite, itself a NaN and the rest of the group zeros."""
    x, w = torch.ones(3, c, device="cuda"), torch.ones(c, device="cuda")
    w[37] = float("inf")
    g = group or c
    q, s = torch.empty(3, c, device="cuda", dtype=T[ykind]), torch.empty(3, -(-c // g), device="cuda")
    K.muon_norm_forward(x, q, weight=w, scales=s, group=group, eps=EPS)
    q, k = q.float().cpu(), 37 // g
    assert bool(s[:, k].isinf().all()) and int(s.isinf().sum()) == 3
    inside = torch.arange(c) // g == k
    assert bool(q[:, 37].isnan().all()) and int(q.isnan().sum()) == 3
    assert bool((q[:, inside & (torch.arange(c) != 37)] == 0).all())
    assert bool((q[:, ~inside] == O.FMAX[ykind]).all())
