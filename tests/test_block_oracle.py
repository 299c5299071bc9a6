"""The row operators' oracle pinned on the CPU: published Philox vectors, the
mask's statistics, gradients against differences, and the routing rules on
hand-made rows."""
import numpy as np
import pytest

from oracle import block_oracle as O


@pytest.mark.parametrize("ctr,key,out", [
    # known answers of philox4x32-10 published with the generator
    ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
])
def test_philox_known_answers(ctr, key, out):
    assert tuple(int(v) for v in O.philox4x32(ctr, key)) == out


def test_keep_mask_rate_and_independence():
    m = O.keep_mask(400, 1000, 0.1, 7, 9)
    n = m.size
    assert abs(m.mean() - (1 - 6554 / 65536)) < 5 * np.sqrt(0.09 / n)   # five standard deviations
    assert not np.array_equal(m, O.keep_mask(400, 1000, 0.1, 8, 9))
    assert not np.array_equal(m, O.keep_mask(400, 1000, 0.1, 7, 10))
    assert np.array_equal(m[:50, :77], O.keep_mask(50, 77, 0.1, 7, 9))   # a smaller matrix: the same corner
    assert O.keep_mask(4, 9, 0.0, 1, 1).all() and not O.keep_mask(4, 9, 1.0, 1, 1).any()


def _difference(f, x, i, eps=1e-6):
    a, b = x.copy(), x.copy()
    a.flat[i] += eps
    b.flat[i] -= eps
    return (f(a) - f(b)) / (2 * eps)


@pytest.mark.parametrize("drop", [None, (0.3, 5, 6)])
def test_norm_gradient_against_differences(drop):
    rng = np.random.default_rng(0)
    x, r = rng.standard_normal((3, 13)), rng.standard_normal((3, 13))
    w, dy, dh = rng.standard_normal(13), rng.standard_normal((3, 13)), rng.standard_normal((3, 13))

    def loss(x, r, w):
        z, _, y = O.norm_forward(x, r, w, 1e-3, drop)
        return (y * dy).sum() + (z * dh).sum()

    z, rstd, _ = O.norm_forward(x, r, w, 1e-3, drop)
    dz, dx, dw = O.norm_backward(dy, z, rstd, w, dh, drop)
    for i in range(39):
        assert abs(_difference(lambda v: loss(v, r, w), x, i) - dx.flat[i]) < 1e-7
        assert abs(_difference(lambda v: loss(x, v, w), r, i) - dz.flat[i]) < 1e-7
    for i in range(13):
        assert abs(_difference(lambda v: loss(x, r, v), w, i) - dw[i]) < 1e-7


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
@pytest.mark.parametrize("aux", [True, False])
def test_route_gradient_against_differences(score, renormalise, aux):
    rng = np.random.default_rng(1)
    l = rng.standard_normal((4, 9)) * 2
    l[1, 3] = -np.inf
    kw = dict(top_k=3, score=score, renormalise=renormalise, scale=1.7)
    mask = np.array([1, 1, 0, 1])
    dw, ds = rng.standard_normal((4, 3)), rng.standard_normal((4, 9))
    idx, w, _ = O.route_forward(l, mask, **kw)
    g = O.route_backward(l, idx, w, dw, score, renormalise, 1.7, ds if aux else None)

    def loss(v):
        i2, w2, s2 = O.route_forward(v, mask, **kw)
        assert np.array_equal(i2, idx)
        return (w2 * dw).sum() + ((s2 * ds).sum() if aux else 0)

    for i in range(l.size):
        if np.isfinite(l.flat[i]):
            assert abs(_difference(loss, l, i) - g.flat[i]) < 1e-7
        else:
            assert g.flat[i] == 0


def test_route_rules():
    # ties to the lowest index, bias moves the choice and not the weight
    idx, w, s = O.route_row(np.array([1.0, 2.0, 2.0, 0.0]), 2, "softmax", renormalise=False)
    assert list(idx) == [1, 2] and np.allclose(w, s[[1, 2]])
    idx, w, _ = O.route_row(np.zeros(4), 2, "sigmoid", bias=np.array([0, 0, 0.5, 0.1]))
    assert list(idx) == [2, 3] and np.allclose(w, 0.5)
    # groups: the sum of the two best decides, the best single expert's group may lose
    l = np.array([5.0, -9, -9, -9, 1, 1, -9, -9])
    assert list(O.route_row(l, 2, "sigmoid", groups=2, top_groups=1)[0]) == [4, 5]
    assert list(O.route_row(l, 2, "sigmoid", groups=2, top_groups=1, group_top=1)[0]) == [0, 1]
    # closed experts, an empty row, scores that underflow
    idx, w, _ = O.route_row(np.array([-np.inf, 3.0, np.nan]), 2, "softmax")
    assert list(idx) == [1, -1] and list(w) == [1, 0]
    assert list(O.route_row(np.full(3, -np.inf), 2, "sigmoid")[0]) == [-1, -1]
    assert np.allclose(O.route_row(np.array([-1e30, -1e30]), 2, "sigmoid")[1], 0.5)


def test_order_and_balance_rules():
    counts, offsets, order, pos = O.route_order(np.array([[2, 0], [-1, 2], [0, 9]]), 3)
    assert list(counts) == [2, 0, 2] and list(offsets) == [0, 2, 2, 4]
    assert list(order) == [1, 4, 0, 3, -1, -1] and pos.tolist() == [[2, 0], [-1, 3], [1, -1]]
    assert np.allclose(O.route_balance([4, 2, 0], [0, 0, 0.5], 0.1), [-0.1, 0, 0.6])
