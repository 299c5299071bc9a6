"""Gather, combine, gate and block quantisation of muon_experts.h on the GPU
against the float64 oracle.

Tolerances, set from the arithmetic: an output of type t is one rounding
(HALF[t] relative, half a subnormal step near zero) off the fp32 value, and
that is off the exact one by the fp32 operations before it, each 2^-24
relative to its result (U).  An 8-bit value times its stored scale is a
rounding off v, with two roundings more for the quotient.
"""
import numpy as np
import pytest
import torch

from matrix_optimizer_amd import binding as B
from matrix_optimizer_amd import experts as X
from oracle import block_oracle as RO
from oracle import experts_oracle as O

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -4, "e5m2": 2.0 ** -3}
SUB = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "e4m3": 2.0 ** -10, "e5m2": 2.0 ** -17}   # half a subnormal step
U = 2.0 ** -24
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    X.lib()


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


def untouched(full, c, shift, rows_left=()):
    f = full.float()
    assert bool((f[:, :shift] == 7).all()) and bool((f[:, shift + c:] == 7).all())
    assert bool((f[list(rows_left)] == 7).all())


def close(got, ref, kind, slack, what):
    """Within a rounding of ref and the given absolute slack; equal where ref is not finite."""
    fine = np.isfinite(ref)
    assert np.array_equal(got[~fine], ref[~fine], equal_nan=True), what
    bound = HALF[kind] * (np.abs(ref) + slack) + SUB[kind] + slack
    err = np.abs(got - ref)[fine]
    assert np.all(err <= bound[fine]), f"{what}: {np.max(err / bound[fine]):.3g} of the bound"


def close8(q, scales, ref, kind, slack, what, block_rows=1, ref_scales=None):
    """8-bit values with their scales against the values ref; `slack` absolute, of the fp32 values before."""
    want = O.row_scales(ref, kind) if ref_scales is None else ref_scales
    big = O.row_scales(np.abs(ref) + slack, kind) if ref_scales is None else want
    assert np.all(np.abs(scales - want) <= (big - want) + 4 * U * want), what
    s = O.expand(scales, ref.shape[0], ref.shape[1], block_rows)
    assert np.all(np.abs(q * s - ref) <= (HALF[kind] * (1 + 4 * U) + 4 * U) * (np.abs(ref) + slack) + slack + SUB[kind] * s), what


def routed(rng, t, k, e, missing=0.1):
    """Distinct experts a row, some rows without: experts, order, position of the pairs."""
    idx = np.stack([rng.permutation(e)[:k] for _ in range(t)]).reshape(t, k).astype(np.int32)
    idx[rng.random(t) < missing] = -1
    _, offsets, order, position = RO.route_order(idx, e)
    return offsets, order.astype(np.int32), position.reshape(t, k).astype(np.int32)


def dev(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda().to(dtype) if dtype else torch.from_numpy(np.ascontiguousarray(a)).cuda()


WIDTHS = [1, 7, 8, 9, 15, 16, 17, 31, 64, 127, 128, 129, 500, 1000, 2051, 4096, 7168, 8200, 16392]


# ---- gather -------------------------------------------------------------------
@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3", "e5m2"])
@pytest.mark.parametrize("c", WIDTHS)
def test_gather(kind, c):
    rng = np.random.default_rng(c)
    t, k, e = (3, 2, 5) if c > 4000 else (23, 3, 7)
    _, order, _ = routed(rng, t, k, e)
    for pad, shift in ((0, 0), (5, 3)):
        x, groups = rows(rng, t, c, kind, 1.0, pad, shift), -(-c // 128)
        full, o = out(t * k, c, kind, pad, shift)
        eight = kind in O.FMAX
        s = rows(rng, t, groups, "f32", 1.0, pad, shift) if eight else None
        sfull, so = out(t * k, groups, "f32", pad, shift) if eight else (None, None)
        X.muon_expert_gather(dev(order), x, o, scales=s, out_scales=so)
        left = [i for i in range(t * k) if order[i] < 0]
        untouched(full, c, shift, left)
        want = O.gather(order, x.float().cpu().numpy(), k)
        got = o.float().cpu().numpy()
        for i, row in want.items():
            assert np.array_equal(got[i], row), (i, c)
        if eight:
            untouched(sfull, groups, shift, left)
            for i, row in O.gather(order, s.cpu().numpy(), k).items():
                assert np.array_equal(so[i].cpu().numpy(), row)


def test_gather_keeps_bits_and_ignores_bad_order():
    """NaN payloads and every byte pass unchanged; entries outside the pairs count as none."""
    x = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(4, 3).view(torch.float8_e4m3fn)
    o = torch.zeros(8, 768, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    order = torch.tensor([7, -1, 8, 0, 2**31 - 1, -2**31, 3, 3], dtype=torch.int32, device="cuda")
    X.muon_expert_gather(order, x, o)
    got = o.view(torch.uint8)
    for i, p in enumerate(order.tolist()):
        want = x.view(torch.uint8)[p // 2] if 0 <= p < 8 else torch.zeros_like(got[i])
        assert torch.equal(got[i], want), i


def test_gather_more_rows_than_the_grid():
    t, k = 700_000, 2
    x = torch.arange(t, dtype=torch.float32, device="cuda").reshape(t, 1) * 2
    order = torch.randperm(t * k, device="cuda").to(torch.int32)
    o = torch.zeros(t * k, 1, device="cuda")
    X.muon_expert_gather(order, x, o)
    assert torch.equal(o[:, 0], (order // k).float() * 2)


def test_gather_large_offsets():
    """Rows beyond 2^31 bytes of the buffer, to such rows."""
    x = torch.zeros(70_000, 40_000, dtype=torch.uint8, device="cuda")
    x[:, 0] = torch.arange(70_000, device="cuda") % 251
    x[:, -1] = torch.arange(70_000, device="cuda") % 241
    order = torch.arange(70_000 - 1, -1, -1, dtype=torch.int32, device="cuda")
    o = torch.zeros_like(x)
    X.muon_expert_gather(order, x.view(torch.float8_e5m2), o.view(torch.float8_e5m2))
    assert torch.equal(o[:, 0], x[:, 0].flip(0)) and torch.equal(o[:, -1], x[:, -1].flip(0))


# ---- combine ------------------------------------------------------------------
def combine_case(rng, t, k, e, c, kind, okind, weights, base, pad=0, shift=0, inplace=False):
    _, _, position = routed(rng, t, k, e, 0.2)
    y = rows(rng, t * k, c, kind, 1.0, pad, shift)
    w = rng.standard_normal((t, k)).astype(np.float32) if weights else None
    bs = rows(rng, t, c, okind, 2.0, pad, shift) if base else None
    bv = f64(bs)
    full, o = out(t, c, okind, pad, shift)
    if inplace:
        o = bs
    X.muon_expert_combine(dev(position), y, o, weights=None if w is None else dev(w), base=bs)
    ref, size = O.combine(position, f64(y), w, bv)
    close(f64(o), ref, okind, (k + 1) * U * size, "combine")
    if not inplace:
        untouched(full, c, shift)


@pytest.mark.parametrize("kind,okind", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("c", WIDTHS)
def test_combine_widths(c, kind, okind):
    rng = np.random.default_rng(c)
    combine_case(rng, 5, 3, 6, c, kind, okind, True, True)
    combine_case(rng, 3, 2, 6, c, kind, okind, False, False, 5, 3)


@pytest.mark.parametrize("k", [1, 2, 4, 5, 8, 9, 31, 32])
def test_combine_slots(k):
    rng = np.random.default_rng(k)
    combine_case(rng, 40, k, 40, 72, "bf16", "bf16", True, False)
    combine_case(rng, 9, k, 32, 300, "f32", "f32", False, True, inplace=True)


@pytest.mark.parametrize("t", [1, 2, 255, 1000, 5000])
def test_combine_rows(t):
    combine_case(np.random.default_rng(t), t, 4, 16, 136, "bf16", "bf16", True, True, 3, 1)


def test_combine_masked_places_are_not_read():
    """NaN in places that no slot names, and rows without a place: base alone, or zeros."""
    y = torch.full((6, 20), NAN, device="cuda")
    y[2] = 1.5
    position = torch.tensor([[-1, 2], [-1, -1], [6, -2**31], [2**31 - 1, -1]], dtype=torch.int32, device="cuda")
    w = torch.full((4, 2), 2.0, device="cuda")
    w[1:] = NAN
    o = torch.full((4, 20), 9.0, device="cuda")
    X.muon_expert_combine(position, y, o, weights=w)
    assert torch.equal(o[0], torch.full((20,), 3.0, device="cuda")) and bool((o[1:] == 0).all())
    base = torch.full((4, 20), -4.0, device="cuda")
    X.muon_expert_combine(position, y, o, weights=w, base=base)
    assert bool((o[1:] == -4).all()) and bool((o[0] == -1).all())
    X.muon_expert_combine(position, torch.empty(0, 20, device="cuda"), o, weights=w, base=base)
    assert bool((o == -4).all())
    # infinities follow the formula
    y[2, 0] = INF
    X.muon_expert_combine(position, y, o, weights=torch.zeros(4, 2, device="cuda"))
    assert bool(torch.isnan(o[0, 0])) and bool((o[0, 1:] == 0).all())


def test_combine_is_the_gradient_of_gather():
    rng = np.random.default_rng(5)
    _, order, position = routed(rng, 30, 3, 8)
    x, g = rows(rng, 30, 40, "f32"), rows(rng, 90, 40, "f32")
    o = torch.zeros(90, 40, device="cuda")
    X.muon_expert_gather(dev(order), x, o)
    dx = torch.empty(30, 40, device="cuda")
    X.muon_expert_combine(dev(position), g, dx)
    left, right = float((o.double() * g.double()).sum()), float((x.double() * dx.double()).sum())
    size = float((o.double() * g.double()).abs().sum())
    assert abs(left - right) <= 4 * U * size


# ---- combine's gradients --------------------------------------------------------
def combine_backward_case(rng, t, k, e, c, kind, eight=None, weights=True, dy=True, dweights=True, pad=0, shift=0):
    _, order, position = routed(rng, t, k, e, 0.2)
    n = t * k
    dout, y = rows(rng, t, c, kind, 0.01, pad, shift), rows(rng, n, c, kind, 1.0, pad, shift)
    w = rng.standard_normal((t, k)).astype(np.float32) if weights else None
    dfull, d = out(n, c, kind, pad, shift) if dy else (None, None)
    efull, d8 = out(n, c, eight, pad, shift) if eight else (None, None)
    sfull, s = out(n, -(-c // 128), "f32", pad, shift) if eight else (None, None)
    dw = torch.full((t, k), 7.0, device="cuda") if dweights else None
    X.muon_expert_combine_backward(dev(position), dout, y=y if dweights else None, weights=None if w is None else dev(w),
                                   dy=d, dweights=dw, dy8=d8, scales=s)
    ref, rdw, size = O.combine_backward(position, f64(dout), f64(y), w)
    at, left = sorted(ref), [i for i in range(n) if i not in ref]
    want = np.array([ref[i] for i in at]).reshape(len(at), c)
    if dy:
        untouched(dfull, c, shift, left)
        close(f64(d)[at], want, kind, U * np.abs(want), "dy")
    if eight:
        untouched(efull, c, shift, left)
        untouched(sfull, -(-c // 128), shift, left)
        close8(f64(d8)[at], f64(s)[at], want, eight, U * np.abs(want), "dy8")
    if dweights:
        # a lane adds at most c / 64 + 8 products in a row, then a tree of the lanes
        close(f64(dw), rdw, "f32", (c / 64 + 20) * U * size, "dweights")


@pytest.mark.parametrize("kind,eight", [("bf16", "e4m3"), ("f32", "e5m2"), ("bf16", None), ("bf16", "e5m2"), ("f32", "e4m3")])
@pytest.mark.parametrize("c", WIDTHS)
def test_combine_backward_widths(c, kind, eight):
    rng = np.random.default_rng(c)
    combine_backward_case(rng, 5, 3, 6, c, kind, eight)
    combine_backward_case(rng, 3, 2, 6, c, kind, eight, pad=5, shift=3)


@pytest.mark.parametrize("k", [1, 2, 3, 8, 9, 32])
def test_combine_backward_slots_and_parts(k):
    rng = np.random.default_rng(k)
    for c in (72, 1100):
        combine_backward_case(rng, 9, k, 40, c, "bf16", "e4m3", weights=False)
        combine_backward_case(rng, 9, k, 40, c, "bf16", "e4m3", dy=False, dweights=False)
        combine_backward_case(rng, 9, k, 40, c, "f32", None, dweights=False)
        combine_backward_case(rng, 9, k, 40, c, "f32", None, dy=False)


@pytest.mark.parametrize("t", [1, 2, 257, 3000])
def test_combine_backward_rows(t):
    combine_backward_case(np.random.default_rng(t), t, 4, 16, 136, "bf16", "e4m3")


def test_combine_backward_against_differences():
    """The gradient of sum(out * dout) by central differences of the oracle's forward pass in 64 bits."""
    rng = np.random.default_rng(11)
    _, _, position = routed(rng, 6, 2, 4)
    y, w, d = rng.standard_normal((12, 10)), rng.standard_normal((6, 2)).astype(np.float32), rng.standard_normal((6, 10))
    y, d = y.astype(np.float32), d.astype(np.float32)
    dy, dw = torch.zeros(12, 10, device="cuda"), torch.zeros(6, 2, device="cuda")
    X.muon_expert_combine_backward(dev(position), dev(d), y=dev(y), weights=dev(w), dy=dy, dweights=dw)
    loss = lambda yy, ww: float((O.combine(position, yy, ww)[0] * d).sum())   # noqa: E731
    h = 2.0 ** -10   # the loss is bilinear: central differences are exact but for rounding
    for arr, got in ((y, f64(dy)), (w, f64(dw))):
        for at in np.ndindex(arr.shape):
            up, down = arr.astype(np.float64), arr.astype(np.float64)
            up[at] += h
            down[at] -= h
            args = lambda v: (v, w) if arr is y else (y.astype(np.float64), v)   # noqa: E731
            diff = (loss(*args(up)) - loss(*args(down))) / (2 * h)
            assert abs(got[at] - diff) <= 1e-5 * (1 + abs(diff)), at


def test_combine_backward_special_values():
    """Infinities, NaN and zero weights: the scale takes no NaN, an infinity makes it infinite."""
    d = torch.ones(4, 130, device="cuda")
    d[0, 0], d[1, 0], d[2] = NAN, INF, 0
    position = torch.arange(4, dtype=torch.int32, device="cuda").reshape(4, 1)
    w = torch.tensor([[1.0], [2.0], [3.0], [NAN]], device="cuda")
    d8, s = torch.zeros(4, 130, device="cuda").to(T["e4m3"]), torch.zeros(4, 2, device="cuda")
    X.muon_expert_combine_backward(position, d, weights=w, dy8=d8, scales=s)
    q, one = d8.float(), np.float32(1) / np.float32(448)
    assert bool(torch.isnan(q[0, 0])) and bool((q[0, 1:] == 448).all()) and np.array_equal(s[0].cpu().numpy(), [one, one])
    assert bool(torch.isnan(q[1, 0])) and bool((q[1, 1:128] == 0).all()) and s[1, 0] == INF and bool((q[1, 128:] == 448).all())
    assert bool((q[2] == 0).all()) and bool((s[2] == 1).all())
    assert bool(torch.isnan(q[3]).all()) and bool((s[3] == 1).all())
    w[:] = 0   # 0 * inf is NaN, the others 0: no maximum
    X.muon_expert_combine_backward(position, d, weights=w, dy8=d8, scales=s)
    q = d8.float()
    assert bool(torch.isnan(q[1, 0])) and bool((q[1, 1:] == 0).all()) and bool((s == 1).all())


# ---- gate ---------------------------------------------------------------------
# the exponential and the quotient are within two roundings each, with the sum and the products before y eight in all
GATE = 8 * U


def gate_case(rng, r, c, kind, eight=None, y=True, pad=0, shift=0, used=None, scale=2.0):
    a = rows(rng, r, 2 * c, kind, scale, pad, shift)
    n = r if used is None else min(max(used, 0), r)
    yfull, yo = out(r, c, kind, pad, shift) if y else (None, None)
    efull, y8 = out(r, c, eight, pad, shift) if eight else (None, None)
    sfull, s = out(r, -(-c // 128), "f32", pad, shift) if eight else (None, None)
    u = None if used is None else torch.tensor([used], dtype=torch.int32, device="cuda")
    X.muon_gate_forward(a, y=yo, y8=y8, scales=s, used=u)
    ref = O.gate(f64(a))[:n]
    left = range(n, r)
    if y:
        untouched(yfull, c, shift, left)
        close(f64(yo)[:n], ref, kind, GATE * np.abs(ref), "y")
    if eight:
        untouched(efull, c, shift, left)
        untouched(sfull, -(-c // 128), shift, left)
        close8(f64(y8)[:n], f64(s)[:n], ref, eight, GATE * np.abs(ref), "y8")


@pytest.mark.parametrize("kind,eight", [("bf16", "e4m3"), ("f32", "e5m2"), ("f32", None), ("f32", "e4m3")])
@pytest.mark.parametrize("c", WIDTHS)
def test_gate_widths(c, kind, eight):
    rng = np.random.default_rng(c)
    gate_case(rng, 5, c, kind, eight)
    gate_case(rng, 3, c, kind, eight, pad=5, shift=3)


@pytest.mark.parametrize("r", [1, 2, 255, 3000])
def test_gate_rows(r):
    rng = np.random.default_rng(r)
    gate_case(rng, r, 200, "bf16", "e4m3", used=r - 1)
    gate_case(rng, r, 128, "bf16", "e5m2", y=False)
    for used in (-5, 0, r, r + 7):
        gate_case(rng, r, 40, "f32", "e4m3", used=used)


def gate_backward_case(rng, r, c, kind, eight=None, da=True, pad=0, shift=0, used=None):
    a, dy = rows(rng, r, 2 * c, kind, 2.0, pad, shift), rows(rng, r, c, kind, 0.01, pad, shift)
    n = r if used is None else min(max(used, 0), r)
    dfull, d = out(r, 2 * c, kind, pad, shift) if da else (None, None)
    efull, d8 = out(r, 2 * c, eight, pad, shift) if eight else (None, None)
    sfull, s = out(r, 2 * c // 128, "f32", pad, shift) if eight else (None, None)
    u = None if used is None else torch.tensor([used], dtype=torch.int32, device="cuda")
    X.muon_gate_backward(a, dy, da=d, da8=d8, scales=s, used=u)
    ref, size = (v[:n] for v in O.gate_backward(f64(a), f64(dy)))
    left = range(n, r)
    if da:
        untouched(dfull, 2 * c, shift, left)
        close(f64(d)[:n], ref, kind, 12 * U * size, "da")
    if eight:
        untouched(efull, 2 * c, shift, left)
        untouched(sfull, 2 * c // 128, shift, left)
        close8(f64(d8)[:n], f64(s)[:n], ref, eight, 12 * U * size, "da8")


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("c", WIDTHS)
def test_gate_backward_widths(c, kind):
    rng = np.random.default_rng(c)
    for pad, shift in ((0, 0), (5, 3)):
        gate_backward_case(rng, 3, c, kind, None, pad=pad, shift=shift)
        if c % 128 == 0:
            gate_backward_case(rng, 3, c, kind, "e4m3", pad=pad, shift=shift)
            gate_backward_case(rng, 3, c, kind, "e5m2", da=False, pad=pad, shift=shift)


@pytest.mark.parametrize("r", [1, 2, 255, 3000])
def test_gate_backward_rows(r):
    rng = np.random.default_rng(r)
    for used in (None, r - 1, 0, r + 7):
        gate_backward_case(rng, r, 128, "bf16", "e4m3", used=used)


def test_gate_backward_against_differences():
    rng = np.random.default_rng(3)
    a, dy = rng.standard_normal((3, 20)).astype(np.float32), rng.standard_normal((3, 10)).astype(np.float32)
    da = torch.zeros(3, 20, device="cuda")
    X.muon_gate_backward(dev(a), dev(dy), da=da)
    h, got = 2.0 ** -13, f64(da)
    for at in np.ndindex(a.shape):
        up, down = a.astype(np.float64), a.astype(np.float64)
        up[at] += h
        down[at] -= h
        diff = ((O.gate(up) - O.gate(down)) * dy).sum() / (2 * h)
        assert abs(got[at] - diff) <= 1e-5 * (1 + abs(diff)), at   # h^2 / 6 times a third derivative below 1


def test_gate_far_values():
    """Gates far from zero keep their digits; rows not in use may hold anything; infinities follow the formula."""
    g = np.array([-1e4, -100.0, -88.0, -80.0, -20.0, -1e-30, 0.0, 1e-30, 20.0, 80.0, 100.0, 1e4, 3e38], np.float32)
    a = np.stack([np.concatenate([g, np.full(13, 1.0, np.float32)])] * 2)
    a[1] = np.nan
    y, da = torch.zeros(2, 13, device="cuda"), torch.zeros(2, 26, device="cuda")
    used = torch.ones(1, dtype=torch.int32, device="cuda")
    X.muon_gate_forward(dev(a), y=y, used=used)
    ref = O.gate(a[:1].astype(np.float64))
    tiny = 2.0 ** -126 * (1 + np.abs(g))     # the exponential's subnormal results lose digits
    close(f64(y)[:1], ref, "f32", GATE * np.abs(ref) + tiny, "y")
    X.muon_gate_backward(dev(a), torch.ones(2, 13, device="cuda"), da=da, used=used)
    ref, size = O.gate_backward(a[:1].astype(np.float64), np.ones((1, 13)))
    close(f64(da)[:1], ref, "f32", 12 * U * size + np.concatenate([tiny, tiny]), "da")
    assert bool((y[1] == 0).all()) and bool((da[1] == 0).all())
    b = torch.tensor([[INF, NAN, 1.0, 2.0, 3.0, NAN]], device="cuda")
    o = torch.zeros(1, 3, device="cuda")
    X.muon_gate_forward(b, y=o)
    assert o[0, 0] == INF and bool(torch.isnan(o[0, 1:]).all())


# ---- quantise -----------------------------------------------------------------
def quantise_case(rng, b, r, c, kind, eight, q=True, qt=True, pad=0, shift=0, scale=0.02):
    full = torch.from_numpy(rng.standard_normal((b, r + 2, c + pad)).astype(np.float32) * np.float32(scale)).cuda().to(T[kind])
    x = full[:, 1:r + 1, shift:shift + c]
    seven = lambda *s: torch.full(s, 7.0, device="cuda")   # noqa: E731
    rb, cb = -(-r // 128), -(-c // 128)
    qf, tf = seven(b, r + 2, c + pad).to(T[eight]), seven(b, c + 2, r + pad).to(T[eight])
    qv, tv = qf[:, 1:r + 1, shift:shift + c], tf[:, 1:c + 1, shift:shift + r]
    s, st = seven(b, rb, cb), seven(b, cb, rb)
    X.muon_quantise_blocks(x, q=qv if q else None, scales=s if q else None, qt=tv if qt else None,
                           scales_t=st if qt else None)
    for i in range(b):
        ref = f64(x[i])
        want = O.block_scales(ref, eight)
        for on, got, sc in ((q, f64(qv[i]), f64(s[i])), (qt, f64(tv[i]).T, f64(st[i]).T)):
            if on:
                assert np.array_equal(sc, want)
                close8(got, sc, ref, eight, 0.0, "q", 128, want)
    for f, h, w, on in ((qf, r, c, q), (tf, c, r, qt)):
        edge = f.float().clone()
        if on:
            edge[:, 1:h + 1, shift:shift + w] = 7
        assert bool((edge == 7).all())


@pytest.mark.parametrize("kind,eight", [("bf16", "e4m3"), ("f32", "e5m2"), ("bf16", "e5m2"), ("f32", "e4m3")])
@pytest.mark.parametrize("r,c", [(1, 1), (1, 300), (300, 1), (7, 9), (64, 64), (127, 129), (128, 128), (129, 127), (130, 500),
                                 (256, 384), (257, 1003)])
def test_quantise_shapes(r, c, kind, eight):
    rng = np.random.default_rng(r * 1000 + c)
    quantise_case(rng, 2, r, c, kind, eight)
    quantise_case(rng, 1, r, c, kind, eight, pad=5, shift=3)
    quantise_case(rng, 3, r, c, kind, eight, qt=False)
    quantise_case(rng, 3, r, c, kind, eight, q=False, pad=8, shift=8)


def test_quantise_plain_matrix_and_special_values():
    x = torch.ones(200, 150, device="cuda")
    x[0, 0], x[130, 0], x[0, 140], x[140, 140] = NAN, INF, -2, 2.0 ** -140
    x[128:, 128:] = 0
    x[140, 140] = 2.0 ** -140
    q, s = torch.zeros(200, 150, device="cuda").to(T["e4m3"]), torch.zeros(2, 2, device="cuda")
    X.muon_quantise_blocks(x, q, s)
    v, one = q.float(), float(np.float32(1) / np.float32(448))
    assert bool(torch.isnan(v[0, 0])) and v[0, 1] == 448 and s[0, 0] == one
    assert s[1, 0] == INF and bool(torch.isnan(v[130, 0])) and bool((v[128:, :128].nan_to_num(0) == 0).all())
    assert s[0, 1] == float(np.float32(2) / np.float32(448)) and v[0, 140] == -448 and v[1, 141] == 224
    assert s[1, 1] == 2.0 ** -126 and v[140, 140] == 0    # 2^-14 of a scale: below half the smallest value
    x.zero_()
    X.muon_quantise_blocks(x, q, s)
    assert bool((s == 1).all()) and bool((q.float() == 0).all())


def test_quantise_ties_to_even():
    """Values halfway between two 8-bit ones, whole scale: to the even one."""
    for kind, top in (("e4m3", 448.0), ("e5m2", 57344.0)):
        grid = torch.arange(0, 0x7C if kind == "e5m2" else 0x7F, dtype=torch.uint8).view(T[kind]).float()
        mid = (grid[1:] + grid[:-1]) / 2
        x = torch.zeros(2, 128)
        x[0, :grid.numel()], x[1, :mid.numel()] = grid, mid
        x[:, 127] = top
        q, s = torch.zeros(2, 128, device="cuda").to(T[kind]), torch.zeros(1, 1, device="cuda")
        X.muon_quantise_blocks(x.cuda(), q, s)
        assert s.item() == 1
        assert np.array_equal(f64(q), O.round8(f64(x), kind)), kind
