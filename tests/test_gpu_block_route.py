"""Expert routing, the order of the pairs and the balance update on the GPU
against the float64 oracle.

The choice is exact: experts, counts, order and position are compared whole.
Weights and scores are fp32 results of a few fp32 or fp64 operations and a sum
of at most 1024 positive terms: 2^-24 for the stored rounding, and for an fp32
exp, quotient and sum (16 per lane and a tree) at most 32 roundings, 2^-19
relative together.  dlogits in type t: eps(t) / 2 relative plus 2^-19 of the
terms that add up to it.
"""
import numpy as np
import pytest
import torch

from matrix_optimizer_amd import binding as B
from matrix_optimizer_amd import block as K
from oracle import block_oracle as O

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
REL = 2.0 ** -19


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    K.lib()


def f64(t):
    return None if t is None else t.detach().to(torch.float64).cpu().numpy()


def logits_of(rng, t, e, kind, scale=1.5, pad=0, shift=0):
    full = torch.from_numpy((rng.standard_normal((t, e + pad)) * scale).astype(np.float32)).cuda().to(T[kind])
    return full[:, shift:shift + e]


def run(logits, route, bias=None, mask=None, scores=True):
    t, e = logits.shape
    idx = torch.full((t, route.top_k), 99, dtype=torch.int32, device="cuda")
    w = torch.full((t, route.top_k), 7.0, device="cuda")
    s = torch.full((t, e), 7.0, device="cuda") if scores else None
    K.muon_route_forward(route, logits, idx, w, bias=bias, token_mask=mask, scores=s)
    torch.cuda.synchronize()
    return idx, w, s


def check(logits, route, bias=None, mask=None):
    idx, w, s = run(logits, route, bias, mask)
    ri, rw, rs = O.route_forward(f64(logits), None if mask is None else mask.cpu().numpy(), top_k=route.top_k,
                                 score=route.score, bias=f64(bias), groups=route.groups, top_groups=route.top_groups,
                                 group_top=route.group_top, renormalise=route.renormalise, scale=route.scale)
    assert np.array_equal(idx.cpu().numpy(), ri)
    assert np.all(np.abs(f64(w) - rw) <= REL * rw + 1e-38)
    assert np.all(np.abs(f64(s) - rs) <= REL * rs + 1e-38)
    i2, w2, _ = run(logits, route, bias, mask, scores=False)
    assert torch.equal(idx, i2) and torch.equal(w, w2)
    return idx, w


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,k", [(1, 1), (2, 1), (3, 3), (8, 2), (17, 5), (32, 32), (60, 4), (64, 6), (100, 7), (128, 8),
                                 (160, 6), (200, 32), (256, 8), (257, 9), (384, 8), (512, 10), (700, 3), (1024, 32)])
def test_route_sizes(e, k, score):
    rng = np.random.default_rng(e)
    for kind in ("bf16", "f32"):
        for renorm in (True, False):
            check(logits_of(rng, 33, e, kind), K.Route(k, score, renormalise=renorm, scale=1.25))
        bias = torch.from_numpy((rng.standard_normal(e) * 0.05).astype(np.float32)).cuda()
        check(logits_of(rng, 33, e, kind), K.Route(k, score), bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,k,g,tg,gt", [(8, 2, 2, 1, 2), (8, 2, 8, 4, 2), (60, 4, 12, 3, 1), (64, 6, 8, 3, 2),
                                         (96, 4, 3, 2, 2), (256, 8, 8, 4, 2), (256, 8, 16, 1, 1), (1024, 8, 32, 5, 2),
                                         (1000, 20, 100, 7, 2), (512, 3, 512, 3, 2), (1024, 8, 1024, 512, 2), (21, 21, 7, 7, 2)])
@pytest.mark.parametrize("biased", [True, False])
def test_route_groups(e, k, g, tg, gt, score, biased):
    rng = np.random.default_rng(e + g)
    bias = torch.from_numpy((rng.standard_normal(e) * 0.1).astype(np.float32)).cuda() if biased else None
    check(logits_of(rng, 40, e, "f32"), K.Route(k, score, g, tg, gt), bias)
    check(logits_of(rng, 40, e, "bf16", pad=5, shift=3), K.Route(k, score, g, tg, gt, renormalise=False), bias)


@pytest.mark.parametrize("t", [1, 2, 3, 5, 16, 17, 63, 257, 5000])
def test_route_rows(t):
    rng = np.random.default_rng(t)
    check(logits_of(rng, t, 64, "bf16"), K.Route(6, "sigmoid"))
    check(logits_of(rng, t, 256, "f32"), K.Route(8, "softmax", 8, 4))


@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 8), (9, 3), (1, 1)])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_route_strides_and_alignment(pad, shift, kind):
    rng = np.random.default_rng(3)
    for e in (24, 64, 250, 256):
        check(logits_of(rng, 21, e, kind, pad=pad, shift=shift), K.Route(4, "softmax", renormalise=False))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [True, False])
def test_route_near_ties(score, biased):
    """Scores closer than fp32 resolves, or equal: decided in 64 bits, equal ones by the index."""
    rng = np.random.default_rng(12)
    e, t = 64, 400
    base = rng.standard_normal((t, 1)) * 0.5
    near = base + rng.integers(-3, 4, (t, e)) * 2.0 ** -23
    l = torch.from_numpy(near.astype(np.float32)).cuda()
    bias = torch.from_numpy((rng.integers(-2, 3, e) * 2.0 ** -25).astype(np.float32)).cuda() if biased else None
    check(l, K.Route(5, score), bias)
    check(l, K.Route(5, score, 8, 3), bias)
    check(torch.zeros(5, e, device="cuda"), K.Route(7, score), bias)
    check(torch.zeros(5, e, device="cuda"), K.Route(7, score, 8, 3), bias)
    # bf16 logits repeat a lot
    check(logits_of(rng, 300, 256, "bf16", 0.02), K.Route(8, score, 8, 4), None)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_masks_and_extremes(score, groups, renorm):
    rng = np.random.default_rng(5)
    e, k = 16, 4
    l = logits_of(rng, 12, e, "f32")
    l[0] = float("-inf")                        # nothing open
    l[1, 1:] = float("-inf")                    # one open
    l[2, 3] = float("nan")
    l[3] = torch.finfo(torch.float32).min       # the type's lowest value is no closed expert
    l[4, ::2] = torch.finfo(torch.float32).min
    l[5, 7] = float("inf")
    l[6] = float("inf")
    l[7] = float("nan")
    l[8] = -90.0                                # a sigmoid below fp32's smallest normal value
    l[9] = 90.0
    l[10, :12] = float("-inf")                  # one group open
    for mask in (None, torch.tensor([1, 1, 1, 0, 1, 1, 0, 1, 1, 1, 1, 0], dtype=torch.uint8, device="cuda")):
        for bias in (None, torch.linspace(-0.1, 0.1, e, device="cuda")):
            check(l, K.Route(k, score, groups, max(1, groups // 2), renormalise=renorm), bias, mask)
    check(l.bfloat16(), K.Route(k, score, groups, groups, renormalise=renorm), None, mask.bool())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e", [30, 64, 256, 1024])
def test_route_wide_values(score, e):
    """Logits and biases spread far wider than their usual range, the chosen ones far below the largest too."""
    rng = np.random.default_rng(e)
    for scale in (40.0, 1e4, 1e30):
        l = logits_of(rng, 25, e, "f32", scale)
        check(l, K.Route(7, score))
        check(l, K.Route(7, score, 2, 1))
    l = torch.zeros(9, e, device="cuda")
    l[:, ::3] = torch.arange(l[:, ::3].shape[1], device="cuda") * -7.0 - 100.0
    l[:, 1::3] = float("-inf")
    l[3:, 2::3] = -3e4
    check(l, K.Route(10, score))
    for wide in (3.0, 1e6):
        bias = torch.from_numpy((rng.standard_normal(e) * wide).astype(np.float32)).cuda()
        check(logits_of(rng, 25, e, "f32"), K.Route(7, score), bias)
        check(logits_of(rng, 25, e, "bf16"), K.Route(7, score, 2, 1), bias)


def choose(l, bias, route):
    """The experts of route's rule for many rows without closed experts, in 64 bits."""
    t, e = l.shape
    if route.score == "sigmoid":
        s = 1 / (1 + np.exp(-l))
    else:
        s = np.exp(l - l.max(1, keepdims=True))
        s = s / s.sum(1, keepdims=True)
    rank = s + bias
    n = e // route.groups
    best = -np.sort(-rank.reshape(t, route.groups, n), axis=2)[:, :, :route.group_top]
    out = np.argsort(-best.sum(2), axis=1, kind="stable")[:, route.top_groups:]
    hidden = np.zeros((t, route.groups), bool)
    np.put_along_axis(hidden, out, True, 1)
    rank = np.where(np.repeat(hidden, n, axis=1), -np.inf, rank)
    return np.argsort(-rank, axis=1, kind="stable")[:, :route.top_k]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("far", [10.0, 1e3, 1e5, 1e6])
@pytest.mark.parametrize("n,g,tg", [(2, 2, 1), (5, 6, 2), (8, 4, 1), (16, 8, 3), (64, 4, 2), (128, 8, 3)])
def test_route_groups_whose_biases_cancel(n, g, tg, far, score):
    """A group's value is a small sum of large terms where its two best have biases of opposite sign: the rounding
    of the terms, not of the sum, decides how near two groups may be."""
    rng = np.random.default_rng(n * g)
    t = 20000 if n * g <= 32 else 2000
    bias = np.full((g, n), -2 * far, np.float32)
    bias[0::2, :2] = far, -far
    bias[1::2, :2] = 0
    bias = bias.reshape(-1)
    # scores of a group's two best so near those of the next that fp32 sums of this size do not tell them apart
    l = rng.standard_normal((t, g * n)).astype(np.float32) * np.float32(0.5)
    if score == "softmax":
        l.reshape(t, g, n)[:, :, :2] += 4
    route = K.Route(2, score, g, tg, 2)
    idx = run(torch.from_numpy(l).cuda(), route, torch.from_numpy(bias).cuda(), scores=False)[0]
    wrong = (idx.cpu().numpy() != choose(l.astype(np.float64), bias.astype(np.float64), route)).any(1)
    assert not wrong.any(), f"{int(wrong.sum())} of {t} rows"


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,k,g", [(8, 4, 1), (30, 6, 1), (64, 6, 8), (256, 8, 8), (256, 8, 1), (1024, 32, 4)])
def test_route_bias_not_finite(e, k, g, score):
    """A bias that is NaN or infinite chooses no expert twice and none that there is not, also where equal values
    are put in order in 64 bits; rows of other calls are not concerned."""
    for far in (float("nan"), float("inf"), -float("inf")):
        for every in (1, 2, 3):
            bias = torch.zeros(e, device="cuda")
            bias[::every] = far
            for l in (torch.zeros(33, e, device="cuda"), torch.randn(33, e, device="cuda").bfloat16()):
                idx, w, _ = run(l, K.Route(k, score, g, max(1, g // 2)), bias, scores=False)
                got = idx.cpu().numpy()
                assert got.min() >= -1 and got.max() < e
                for row in got:
                    on = row[row >= 0]
                    assert len(set(on)) == len(on)
                w = w.cpu().numpy()
                assert np.isfinite(w).all() and (w >= 0).all() and (w[got < 0] == 0).all()


@pytest.mark.parametrize("low", [(-60, -69, -92, -104), (-69, -100, -100, -75), (-60, -104, -110, -140),
                                 (-80, -81, -95, -170), (-40, -90, -100, -130), (-3, -90, -101, -120)])
def test_route_weights_of_widely_spread_small_scores(low):
    """Renormalised weights hold where the smaller chosen scores are below fp32's normal range and their ratios to
    the others are not."""
    l = torch.tensor([low], dtype=torch.float32, device="cuda").repeat(5, 1)
    l += torch.arange(5, device="cuda")[:, None] * 0.37
    check(l, K.Route(4, "sigmoid", scale=2.5))
    check(l.bfloat16(), K.Route(4, "sigmoid"))
    # chosen far below the largest score: by a bias, and by the groups
    for e in (16, 64, 256):
        wide = torch.zeros(5, e, device="cuda")
        wide[:, 1:] = -200.0
        wide[:, 4:8] = l
        bias = torch.zeros(e, device="cuda")
        bias[4:8] = 3.0
        for score in ("softmax", "sigmoid"):
            check(wide, K.Route(4, score, scale=0.5), bias)
            check(wide, K.Route(4, score, e // 4, 1, 1), bias)


# ---- backward ---------------------------------------------------------------
def check_backward(logits, route, idx, w, dscores=False, rng=None, pad=0, shift=0):
    t, e = logits.shape
    kind = "bf16" if logits.dtype == torch.bfloat16 else "f32"
    dw = torch.from_numpy(rng.standard_normal((t, route.top_k)).astype(np.float32)).cuda()
    ds = torch.from_numpy(rng.standard_normal((t, e)).astype(np.float32)).cuda() if dscores else None
    full = torch.full((t, e + pad), 7.0, device="cuda").to(logits.dtype)
    dl = full[:, shift:shift + e]
    K.muon_route_backward(route, logits, idx, w, dw, dl, dscores=ds)
    torch.cuda.synchronize()
    i, wv = idx.cpu().numpy().astype(np.int64), f64(w)
    ref = O.route_backward(f64(logits), i, wv, f64(dw), route.score, route.renormalise, route.scale, f64(ds))
    on = i >= 0
    a = np.where(on, wv * np.abs(f64(dw)), 0)
    terms = np.zeros((t, e))
    lead = a + (wv / route.scale * a.sum(1, keepdims=True) if route.renormalise else 0)
    np.add.at(terms, (np.arange(t)[:, None], np.maximum(i, 0)), np.where(on, lead, 0))
    s = np.array([np.exp(O.log_scores(np.where(np.isnan(r), -np.inf, np.minimum(r, 3.4028234e38)), route.score))
                  for r in f64(logits)])
    if route.score == "softmax" and not route.renormalise:
        terms += s * a.sum(1, keepdims=True)
    if dscores:
        terms += s * (np.abs(f64(ds)) + (s * np.abs(f64(ds))).sum(1, keepdims=True))
    got = f64(dl)
    assert np.all(np.abs(got - ref) <= HALF[kind] * np.abs(ref) * (1 + 2.0 ** -8) + REL * terms + 1e-37)
    assert np.all(got[~on.any(1)] == 0)
    f = full.float()
    assert bool((f[:, :shift] == 7).all()) and bool((f[:, shift + e:] == 7).all())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dscores", [True, False])
@pytest.mark.parametrize("e,k", [(1, 1), (3, 3), (8, 2), (17, 5), (64, 6), (100, 7), (256, 8), (257, 32), (1024, 32)])
def test_route_backward(e, k, score, renorm, dscores):
    rng = np.random.default_rng(e + k)
    for kind in ("bf16", "f32"):
        route = K.Route(k, score, renormalise=renorm, scale=2.5)
        l = logits_of(rng, 37, e, kind)
        idx, w, _ = run(l, route)
        check_backward(l, route, idx, w, dscores, rng)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_masks(score, renorm):
    rng = np.random.default_rng(9)
    l = logits_of(rng, 9, 16, "f32", pad=9, shift=3)
    l[0] = float("-inf")
    l[1, 1:] = float("-inf")
    l[2, 3] = float("nan")
    l[3, ::2] = float("-inf")
    l[4] = -90.0
    l[5] = 90.0
    mask = torch.tensor([1, 1, 1, 1, 1, 1, 0, 1, 0], dtype=torch.uint8, device="cuda")
    route = K.Route(4, score, renormalise=renorm, scale=0.5)
    idx, w, _ = run(l, route, None, mask)
    for ds in (False, True):
        check_backward(l, route, idx, w, ds, rng, pad=9, shift=3)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("e,k", [(8, 2), (64, 6), (256, 8), (1000, 10)])
def test_route_backward_sigmoid_small_scores(e, k, renorm, kind):
    """dscores s (1 - s) of experts whose scores are small keeps its leading digits: logits from -60 to 10, and
    no term of the other experts in the bound."""
    rng = np.random.default_rng(e)
    l = torch.from_numpy(rng.uniform(-60, 10, (40, e)).astype(np.float32)).cuda().to(T[kind])
    l[0], l[1] = -40.0, -8.0
    route = K.Route(k, "sigmoid", renormalise=renorm, scale=2.5)
    idx, w, _ = run(l, route)
    dw = torch.from_numpy(rng.standard_normal((40, k)).astype(np.float32)).cuda()
    ds = torch.from_numpy(rng.standard_normal((40, e)).astype(np.float32)).cuda()
    dl = torch.empty_like(l)
    K.muon_route_backward(route, l, idx, w, dw, dl, dscores=ds)
    i, wv = idx.cpu().numpy().astype(np.int64), f64(w)
    ref = O.route_backward(f64(l), i, wv, f64(dw), "sigmoid", renorm, 2.5, f64(ds))
    lead = wv * np.abs(f64(dw))
    lead = lead + (wv / 2.5 * lead.sum(1, keepdims=True) if renorm else 0)
    s = 1 / (1 + np.exp(-f64(l)))
    terms = s * (1 - s) * np.abs(f64(ds))
    np.add.at(terms, (np.arange(40)[:, None], i), lead)
    assert np.all(np.abs(f64(dl) - ref) <= HALF[kind] * np.abs(ref) * (1 + 2.0 ** -8) + REL * terms)


@pytest.mark.parametrize("t", [1, 5, 64, 3000])
def test_route_backward_rows(t):
    rng = np.random.default_rng(t)
    route = K.Route(6, "sigmoid", scale=2.5)
    l = logits_of(rng, t, 64, "bf16")
    idx, w, _ = run(l, route)
    check_backward(l, route, idx, w, True, rng)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_backward_against_differences(score):
    """Differences of the forward call's own fp32 weights and scores."""
    rng = np.random.default_rng(21)
    route = K.Route(3, score, renormalise=True, scale=1.5)
    l = logits_of(rng, 3, 12, "f32")
    dw = torch.from_numpy(rng.standard_normal((3, 3)).astype(np.float32)).cuda()
    ds = torch.from_numpy(rng.standard_normal((3, 12)).astype(np.float32)).cuda()
    idx, w, _ = run(l, route)
    g = torch.empty_like(l)
    K.muon_route_backward(route, l, idx, w, dw, g, dscores=ds)

    def loss(v):
        i, w2, s2 = run(v, route)
        # the choice may change under the difference: take the weights of the first choice only where it stays
        return torch.equal(i, idx), float((w2.double() * dw.double()).sum() + (s2.double() * ds.double()).sum())

    seen = 0
    eps = 1e-2   # third derivatives of order 5: 5 eps^2 / 6 < 1e-4; 50 terms' 2^-24 over 2 eps: 1.5e-4
    for i in range(l.numel()):
        hi, lo = l.clone(), l.clone()
        hi.view(-1)[i] += eps
        lo.view(-1)[i] -= eps
        (a, fa), (b, fb) = loss(hi), loss(lo)
        if a and b:
            seen += 1
            assert abs((fa - fb) / (2 * eps) - float(g.view(-1)[i])) < 1e-3
    assert seen > 24


# ---- order, balance -----------------------------------------------------------
def check_order(experts, e):
    n = experts.numel()
    counts = torch.full((e,), 77, dtype=torch.int32, device="cuda")
    offsets = torch.full((e + 1,), 77, dtype=torch.int32, device="cuda")
    order = torch.full((n,), 77, dtype=torch.int32, device="cuda")
    pos = torch.full_like(experts, 77)
    ws = torch.empty(max(K.route_order_workspace_bytes(n, e), 256), dtype=torch.uint8, device="cuda").fill_(0x5A)
    K.muon_route_order(experts, counts, offsets, order, pos, ws)
    torch.cuda.synchronize()
    flat = experts.reshape(-1).cpu().numpy().astype(np.int64)
    key = np.where((flat < 0) | (flat >= e), e, flat)
    by = np.argsort(key, kind="stable")
    rc = np.bincount(key, minlength=e + 1)[:e]
    ro = np.concatenate([[0], np.cumsum(rc)])
    rp = np.empty(n, np.int64)
    rp[by] = np.arange(n)
    assert np.array_equal(counts.cpu().numpy(), rc) and np.array_equal(offsets.cpu().numpy(), ro)
    assert np.array_equal(order.cpu().numpy(), np.where(np.arange(n) < ro[e], by, -1))
    assert np.array_equal(pos.reshape(-1).cpu().numpy(), np.where(key == e, -1, rp))


@pytest.mark.parametrize("e", [1, 2, 8, 60, 64, 255, 256, 1024])
@pytest.mark.parametrize("n,k", [(1, 1), (7, 3), (16, 6), (64, 1), (1000, 8), (1023, 8), (1024, 8), (1025, 8),
                                 (4096, 1), (4097, 1), (5000, 4), (40000, 6)])
def test_order(n, k, e):
    rng = np.random.default_rng(n + e)
    idx = rng.integers(-1, e, (n, k)).astype(np.int32)
    check_order(torch.from_numpy(idx).cuda(), e)


def test_order_lopsided():
    rng = np.random.default_rng(0)
    for e in (3, 256):
        check_order(torch.zeros(20000, 1, dtype=torch.int32, device="cuda"), e)          # one expert takes all
        check_order(torch.full((9000, 2), e - 1, dtype=torch.int32, device="cuda"), e)
        check_order(torch.full((3000, 3), -1, dtype=torch.int32, device="cuda"), e)      # none at all
        far = rng.integers(-5, e + 5, 10000).astype(np.int32)                            # entries out of range
        far[::7], far[3::11] = 2 ** 31 - 1, -2 ** 31
        check_order(torch.from_numpy(far).cuda(), e)
        check_order(torch.empty(0, 4, dtype=torch.int32, device="cuda"), e)


@pytest.mark.parametrize("n", [200000, 1100000])
def test_order_large(n):
    """More rounds than tiles: tiles of one and of several rounds."""
    idx = torch.randint(-1, 256, (n, 8), dtype=torch.int32, device="cuda",
                        generator=torch.Generator(device="cuda").manual_seed(3))
    check_order(idx, 256)


def test_order_matches_oracle():
    idx = np.random.default_rng(1).integers(-1, 9, (50, 3)).astype(np.int32)
    t = torch.from_numpy(idx).cuda()
    counts, offsets = torch.empty(8, dtype=torch.int32, device="cuda"), torch.empty(9, dtype=torch.int32, device="cuda")
    order, pos = torch.empty(150, dtype=torch.int32, device="cuda"), torch.empty_like(t)
    ws = torch.empty(K.route_order_workspace_bytes(150, 8), dtype=torch.uint8, device="cuda")
    K.muon_route_order(t, counts, offsets, order, pos, ws)
    for got, ref in zip((counts, offsets, order, pos), O.route_order(idx, 8)):
        assert np.array_equal(got.cpu().numpy(), ref)


@pytest.mark.parametrize("e", [1, 3, 64, 1000, 1024])
def test_balance(e):
    rng = np.random.default_rng(e)
    counts = rng.integers(0, 2 ** 31 - 1, e).astype(np.int32)      # sums past 32 bits
    counts[: e // 3] = counts.astype(np.int64).sum() // e
    bias = rng.standard_normal(e).astype(np.float32)
    c, b = torch.from_numpy(counts).cuda(), torch.from_numpy(bias).cuda()
    out = torch.empty_like(b)
    rate = float(np.float32(0.001))
    K.muon_route_balance(c, b, out, rate)
    ref = O.route_balance(counts, bias.astype(np.float64), rate)
    assert np.all(np.abs(f64(out) - ref) <= 2.0 ** -24 * np.abs(ref))
    K.muon_route_balance(c, b, b, rate)
    assert torch.equal(b, out)
    same = torch.full((e,), 5, dtype=torch.int32, device="cuda")
    K.muon_route_balance(same, out, b, rate)
    assert torch.equal(b, out)


# ---- streams, graphs, refusals --------------------------------------------------
def test_zero_rows():
    l = torch.empty(0, 8, device="cuda")
    K.muon_route_forward(K.Route(2), l, torch.empty(0, 2, dtype=torch.int32, device="cuda"),
                         torch.empty(0, 2, device="cuda"))
    K.muon_route_backward(K.Route(2), l, torch.empty(0, 2, dtype=torch.int32, device="cuda"),
                          torch.empty(0, 2, device="cuda"), torch.empty(0, 2, device="cuda"), torch.empty_like(l))


def test_refusals_leave_outputs():
    l = torch.randn(4, 8, device="cuda")
    idx, w = torch.full((4, 2), 7, dtype=torch.int32, device="cuda"), torch.full((4, 2), 7.0, device="cuda")
    for bad in (K.Route(2, groups=3), K.Route(2, groups=4, top_groups=5), K.Route(2, scale=0.0), K.Route(2, group_top=3)):
        with pytest.raises(B.MuonError) as e:
            K.muon_route_forward(bad, l, idx, w)
        assert e.value.status == B.MUON_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        K.muon_route_forward(K.Route(3), l, idx, w)
    with pytest.raises(ValueError):
        K.muon_route_forward(K.Route(2), l, idx.long(), w)
    with pytest.raises(B.MuonError) as e:
        K.muon_route_order(idx, idx.new_empty(8), idx.new_empty(9), idx.new_empty(8), torch.empty_like(idx),
                           torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == B.MUON_ERR_WORKSPACE_TOO_SMALL
    torch.cuda.synchronize()
    assert bool((idx == 7).all()) and bool((w == 7).all())


def test_graph_replays_match_eager():
    t, e = 500, 64
    route = K.Route(6, "sigmoid", 8, 4, scale=2.0)
    l, bias = torch.empty(t, e, device="cuda"), torch.zeros(e, device="cuda")
    idx, w = torch.empty(t, 6, dtype=torch.int32, device="cuda"), torch.empty(t, 6, device="cuda")
    dw, dl = torch.randn(t, 6, device="cuda"), torch.empty(t, e, device="cuda")
    counts, offsets = idx.new_empty(e), idx.new_empty(e + 1)
    order, pos = idx.new_empty(t * 6), torch.empty_like(idx)
    ws = torch.empty(K.route_order_workspace_bytes(t * 6, e), dtype=torch.uint8, device="cuda")
    new = torch.empty_like(bias)
    outs = (idx, w, dl, counts, offsets, order, pos, new)

    def step():
        K.muon_route_forward(route, l, idx, w, bias=bias)
        K.muon_route_backward(route, l, idx, w, dw, dl)
        K.muon_route_order(idx, counts, offsets, order, pos, ws)
        K.muon_route_balance(counts, bias, new, 0.01)

    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    for k in range(4):
        l.normal_()
        bias.normal_(0, 0.05)
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in outs]
        for v in outs:
            v.zero_()
        ws.fill_(0x77)
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, outs)), k
