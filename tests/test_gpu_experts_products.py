"""The experts' 8-bit products and weight gradients of muon_experts.h on the GPU
against the float64 oracle, the whole path of routed pairs, streams and graphs.

Tolerances, set from the arithmetic: products of 8-bit and of bf16 values are
exact in fp32; a sum of n of them, in whatever order, takes at most n
additions, each off by at most a unit in the last place of the sum of
magnitudes (2^-23, as the matrix instruction may cut instead of rounding), and
the scales' product and its application two roundings more.  With bf16 outputs
each product may besides lose 2^-13 of the largest of the eight that it is
added with (a power of two not above it, subnormal factors counted as the
smallest normal one): seven of eight do, 7 2^-13 of the sum of magnitudes.
The output is one rounding of its type.
"""
import numpy as np
import pytest
import torch

from matrix_optimizer_amd import binding as B
from matrix_optimizer_amd import block as K
from matrix_optimizer_amd import experts as X
from oracle import experts_oracle as O
from tests.test_gpu_experts_rows import HALF, SUB, T, U, dev, f64, out, rows, untouched

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    X.lib()


def within(got, ref, kind, slack, what):
    bound = HALF[kind] * (np.abs(ref) + slack) + SUB[kind] + slack
    err = np.abs(got - ref)
    assert np.all(err <= bound), f"{what}: {np.nanmax(err / bound):.3g} of the bound"


CUT = 7 * 2.0 ** -13


def product_slack(size, k, okind):
    return ((min(k, 128) + -(-k // 128) + 4) * 2 * U + (CUT if okind == "bf16" else 0)) * size


def eight(rng, shape, kind, pad=0, shift=0):
    """Values of an 8-bit type over its whole finite range, few of them large, as columns of a wider buffer."""
    v = rng.standard_normal(shape[:-1] + (shape[-1] + pad,)) * np.exp(1.5 * rng.standard_normal(shape[:-1] + (1,)))
    v = np.clip(v * 8, -O.FMAX[kind], O.FMAX[kind])
    return torch.from_numpy(v.astype(np.float32)).cuda().to(T[kind])[..., shift:shift + shape[-1]]


def scales(rng, *shape, pad=0, shift=0):
    full = np.exp(rng.standard_normal(shape[:-1] + (shape[-1] + pad,)) - 4).astype(np.float32)
    return torch.from_numpy(full).cuda()[..., shift:shift + shape[-1]]


def product_case(rng, counts, n, k, fa="e4m3", fw="e4m3", okind="bf16", tail=0, pad=0, shift=0):
    e = len(counts)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    r = int(offsets[-1]) + tail
    kb, nb = -(-k // 128), -(-n // 128)
    a, as_ = eight(rng, (r, k), fa, pad, shift), scales(rng, r, kb, pad=pad, shift=shift)
    if tail:     # rows that no expert has: NaN must not spread
        a[-tail:] = float("nan")
        as_[-tail:] = float("nan")
    w, ws = eight(rng, (e, n, k), fw, pad, shift), scales(rng, e, nb, kb)
    full, o = out(r, n, okind, pad, shift)
    X.muon_expert_product(a, as_, w, ws, o, offsets=dev(offsets))
    ref, size = O.product(np.nan_to_num(f64(a)), np.nan_to_num(f64(as_)), f64(w), f64(ws), offsets, (fa, fw))
    live = int(offsets[-1])
    untouched(full, n, shift, range(live, r))
    within(f64(o)[:live], ref[:live], okind, product_slack(size[:live], k, okind), "product")


@pytest.mark.parametrize("n,k", [(1, 1), (1, 128), (16, 15), (17, 16), (64, 127), (128, 128), (130, 129), (200, 144),
                                 (256, 256), (129, 1000), (300, 513), (512, 1024), (48, 2064)])
def test_product_sizes(n, k):
    rng = np.random.default_rng(n * 10007 + k)
    product_case(rng, [5, 0, 130, 1], n, k)
    product_case(rng, [3, 200], n, k, okind="f32", tail=9, pad=5, shift=3)
    product_case(rng, [2, 1, 0, 1], n, k, okind="f32", tail=2, pad=16, shift=16)


@pytest.mark.parametrize("fa,fw", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("okind", ["bf16", "f32"])
def test_product_types(fa, fw, okind):
    rng = np.random.default_rng(5)
    product_case(rng, [40, 3], 144, 272, fa, fw, okind)
    product_case(rng, [300, 260], 272, 400, fa, fw, okind, tail=3)
    product_case(rng, [1], 33, 130, fa, fw, okind)


@pytest.mark.parametrize("counts", [[1], [2], [15], [16], [17], [31], [33], [63, 64, 65], [127], [128], [129], [255, 257],
                                    [0, 0, 5, 0], [0] * 70 + [3] + [0] * 70 + [200], [1] * 100, [700], [385, 1, 640]])
def test_product_runs(counts):
    rng = np.random.default_rng(sum(counts) * 1000 + len(counts))
    product_case(rng, counts, 272, 256)
    product_case(rng, counts, 128, 528, okind="f32", tail=5)


@pytest.mark.parametrize("okind", ["bf16", "f32"])
@pytest.mark.parametrize("k", [4096, 4133, 7168])
@pytest.mark.parametrize("rows", [1, 16, 33, 64])
def test_product_of_few_rows_by_eight_waves(rows, k, okind):
    """One matrix with few columns and long rows: eight waves share the blocks of k."""
    rng = np.random.default_rng(rows * 10007 + k)
    product_case(rng, [rows], 40, k, okind=okind)
    product_case(rng, [rows - 1, 1], 35, k, "e5m2", "e4m3", okind, tail=2, pad=5, shift=3)


@pytest.mark.parametrize("counts,n,k,okind", [
    ([600] + [0] * 8 + [2], 96, 4224, "f32"), ([0] * 4 + [300] + [0] * 3 + [290, 1], 48, 4100, "f32"),                # eight waves
    ([0] * 60 + [300] + [0] * 60 + [600, 3, 0, 65], 272, 1040, "bf16"), ([700] + [1] * 20, 80, 1024, "f32"),    # four
    ([0] * 60 + [257] + [0] * 70 + [513], 272, 256, "bf16"), ([1, 640, 0, 320] + [0] * 12, 64, 384, "f32")])    # one
def test_product_of_long_runs_among_few_rows(counts, n, k, okind):
    """Few rows an expert in the mean, but runs of several times 256: the workgroups of a run take several turns."""
    rng = np.random.default_rng(sum(counts) + k)
    product_case(rng, counts, n, k, okind=okind, tail=3)


@pytest.mark.parametrize("counts,n,k", [([600] + [0] * 14 + [3], 64, 1040), ([600] + [0] * 8 + [2], 96, 4224),
                                        ([1, 640, 0, 320] + [0] * 12, 64, 384), ([40, 0, 513], 4200, 272)])
def test_product_of_long_runs_to_bf16(counts, n, k):
    """The same to bf16: waves in groups of four, of eight and single, and runs that go to tiles."""
    rng = np.random.default_rng(sum(counts) + n + k)
    product_case(rng, counts, n, k, tail=3)


def test_product_one_expert_without_offsets():
    rng = np.random.default_rng(8)
    a, as_, w, ws = eight(rng, (37, 200), "e4m3"), scales(rng, 37, 2), eight(rng, (150, 200), "e4m3"), scales(rng, 2, 2)
    o, p = torch.zeros(37, 150, device="cuda"), torch.zeros(37, 150, device="cuda")
    X.muon_expert_product(a, as_, w, ws, o)
    X.muon_expert_product(a, as_, w, ws, p, offsets=torch.tensor([0, 37], dtype=torch.int32, device="cuda"))
    assert torch.equal(o, p)
    ref, size = O.product(f64(a), f64(as_), f64(w)[None], f64(ws)[None], [0, 37])
    within(f64(o), ref, "f32", 150 * U * size, "product")


def test_product_all_experts_and_bad_offsets():
    """1024 experts; offsets outside the rows are taken to their nearer end, backward runs are empty."""
    rng = np.random.default_rng(9)
    product_case(rng, list(rng.integers(0, 3, 1024)), 20, 32)
    for offsets in ([-7, 3, 9, 1 << 30], [5, 2, 40, 20], [0, 0, 0, -2**31], [64, 64, 64, 64]):
        a, as_ = eight(rng, (40, 48), "e4m3"), scales(rng, 40, 1)
        w, ws = eight(rng, (3, 24, 48), "e4m3"), scales(rng, 3, 1, 1)
        full, o = out(40, 24, "f32")
        X.muon_expert_product(a, as_, w, ws, o, offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"))
        ref, size = O.product(f64(a), f64(as_), f64(w), f64(ws), offsets)
        live = ~np.isnan(ref[:, 0])
        untouched(full, 24, 0, np.nonzero(~live)[0].tolist())
        within(f64(o)[live], ref[live], "f32", 60 * U * size[live], offsets)


def test_product_special_values_stay_in_their_rows():
    rng = np.random.default_rng(10)
    a, as_ = eight(rng, (300, 256), "e5m2"), scales(rng, 300, 2)
    w, ws = eight(rng, (1, 272, 256), "e4m3"), scales(rng, 1, 3, 2)
    want = torch.zeros(300, 272, device="cuda")
    X.muon_expert_product(a, as_, w, ws, want)
    a[7, 200], as_[9, 1], w[0, 33, 5] = float("nan"), float("inf"), float("nan")
    o = torch.zeros(300, 272, device="cuda")
    X.muon_expert_product(a, as_, w, ws, o)
    assert bool(torch.isnan(o[7]).all()) and bool(torch.isnan(o[:, 33]).all()) and bool((~torch.isfinite(o[9])).all())
    keep = torch.ones(300, 272, dtype=torch.bool, device="cuda")
    keep[7], keep[9], keep[:, 33] = False, False, False
    assert torch.equal(o[keep], want[keep])


def test_product_input_gradient_by_transposed_matrices():
    """dx = dy w by the same call on the transposed 8-bit copy of the matrices."""
    rng = np.random.default_rng(12)
    e, n, k = 3, 200, 144
    x = torch.from_numpy(rng.standard_normal((e, n, k)).astype(np.float32)).cuda()
    q = lambda *s: torch.zeros(*s, device="cuda").to(T["e4m3"])   # noqa: E731
    w, ws, wt, wst = q(e, n, k), torch.zeros(e, 2, 2, device="cuda"), q(e, k, n), torch.zeros(e, 2, 2, device="cuda")
    X.muon_quantise_blocks(x, w, ws, wt, wst)
    counts = [30, 0, 21]
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    dy, dys = eight(rng, (51, n), "e5m2"), scales(rng, 51, 2)
    dx = torch.zeros(51, k, device="cuda")
    X.muon_expert_product(dy, dys, wt, wst, dx, offsets=dev(offsets))
    dyv = f64(dy) * O.expand(f64(dys), 51, n)
    for i, (lo, hi) in enumerate(O.runs(offsets, 51)):
        wv = f64(w[i]) * O.expand(f64(ws[i]), n, k, 128)
        within(f64(dx)[lo:hi], dyv[lo:hi] @ wv, "f32", 140 * 2 * U * (np.abs(dyv[lo:hi]) @ np.abs(wv)), "dx")


# ---- weight gradients -------------------------------------------------------------
def weight_grad_case(rng, counts, n, k, okind="bf16", tail=0, pad=0, shift=0, guard=None):
    e = len(counts)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    r = int(offsets[-1]) + tail
    dy, x = rows(rng, r, n, "bf16", 0.01, pad, shift), rows(rng, r, k, "bf16", 1.0, pad, shift)
    if tail:
        dy[-tail:] = float("nan")
        x[-tail:] = float("inf")
    full = torch.full((e, n + 1, k + pad), 7.0, device="cuda").to(T[okind])
    dw = full[:, :n, shift:shift + k]
    ws = torch.full((max(X.expert_weight_grad_workspace_bytes(r, e, n, k), 256),), 0xFF, dtype=torch.uint8, device="cuda")
    X.muon_expert_weight_grad(dy, x, dw, offsets=dev(offsets), workspace=ws)
    live = int(offsets[-1])
    ref, size = O.weight_grad(f64(dy)[:live], f64(x)[:live], offsets, e)
    within(f64(dw), ref, okind, (max(counts) + 16) * 2 * U * size, "dw")
    edge = full.float().clone()
    edge[:, :n, shift:shift + k] = 7
    assert bool((edge == 7).all())


@pytest.mark.parametrize("n,k", [(1, 1), (1, 130), (130, 1), (7, 9), (32, 64), (64, 33), (127, 129), (128, 128), (200, 136),
                                 (256, 256), (257, 264), (520, 300)])
def test_weight_grad_sizes(n, k):
    rng = np.random.default_rng(n * 1009 + k)
    weight_grad_case(rng, [5, 0, 70, 1], n, k)
    weight_grad_case(rng, [33, 64], n, k, "f32", tail=9, pad=5, shift=3)
    weight_grad_case(rng, [100, 2], n, k, "f32", pad=8, shift=8)


@pytest.mark.parametrize("counts", [[0], [1], [15], [16], [17], [31, 32, 33], [63, 64, 65], [128], [500], [0, 3, 0, 0],
                                    [0] * 70 + [3] + [0] * 70, [2000]])
def test_weight_grad_runs(counts):
    rng = np.random.default_rng(sum(counts) * 1000 + len(counts))
    weight_grad_case(rng, counts, 40, 72)
    weight_grad_case(rng, counts, 144, 80, "f32", tail=70)


def test_weight_grad_plain_matrix_no_rows_bad_offsets():
    rng = np.random.default_rng(3)
    dy, x = rows(rng, 90, 20, "bf16"), rows(rng, 90, 30, "bf16")
    ws = torch.empty(max(256, X.expert_weight_grad_workspace_bytes(90, 3, 20, 30)), dtype=torch.uint8, device="cuda")
    dw = torch.full((20, 30), 7.0, device="cuda")
    X.muon_expert_weight_grad(dy, x, dw, workspace=ws)
    ref, size = O.weight_grad(f64(dy), f64(x), [0, 90], 1)
    within(f64(dw)[None], ref, "f32", 110 * 2 * U * size, "dw")
    X.muon_expert_weight_grad(dy[:0], x[:0], dw, workspace=ws)
    assert bool((dw == 0).all())
    dw = torch.full((3, 20, 30), 7.0, device="cuda")
    X.muon_expert_weight_grad(dy[:0], x[:0], dw, offsets=torch.zeros(4, dtype=torch.int32, device="cuda"), workspace=ws)
    assert bool((dw == 0).all())
    for offsets in ([-7, 3, 9, 1 << 30], [5, 2, 40, 20], [0, 0, 0, -2**31]):
        X.muon_expert_weight_grad(dy, x, dw, offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"), workspace=ws)
        ref, size = O.weight_grad(f64(dy), f64(x), offsets, 3)
        within(f64(dw), ref, "f32", 110 * 2 * U * size, offsets)


def test_weight_grad_against_differences():
    """The gradient of sum(dy * (x w^T)) by central differences; the loss is linear in w."""
    rng = np.random.default_rng(4)
    dy, x = rows(rng, 12, 5, "bf16"), rows(rng, 12, 6, "bf16")
    offsets = [0, 4, 4, 12]
    dw = torch.zeros(3, 5, 6, device="cuda")
    X.muon_expert_weight_grad(dy, x, dw, offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"),
                              workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
    w, d, xv, got = rng.standard_normal((3, 5, 6)), f64(dy), f64(x), f64(dw)
    loss = lambda v: sum((d[lo:hi] * (xv[lo:hi] @ v[e].T)).sum() for e, (lo, hi) in enumerate(O.runs(offsets, 12)))  # noqa: E731
    for at in np.ndindex(w.shape):
        up, down = w.copy(), w.copy()
        up[at] += 0.5
        down[at] -= 0.5
        assert abs(got[at] - (loss(up) - loss(down))) <= 1e-5 * (1 + abs(got[at])), at


# ---- the whole path ---------------------------------------------------------------
class Path:
    """A routed layer in 8 bits, forward and backward, in buffers of its own: norm, routing, order, gather, product,
    gate, product, combine, and back to the gradients of everything that is learned."""

    def __init__(self, rows=70, hidden=256, inner=128, experts=8, top_k=2, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.T, self.H, self.F, self.E, self.k = rows, hidden, inner, experts, top_k
        randn = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
        self.x, self.dout = randn(rows, hidden).bfloat16(), (randn(rows, hidden) * 0.01).bfloat16()
        self.w1 = (randn(experts, 2 * inner, hidden) * hidden ** -0.5).bfloat16()
        self.w2 = (randn(experts, hidden, inner) * inner ** -0.5).bfloat16()
        self.logits = randn(rows, experts)
        P = self.P = rows * top_k
        b = self.b = {}
        bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")   # noqa: E731
        f32 = lambda *s: torch.zeros(*s, device="cuda")                        # noqa: E731
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")     # noqa: E731
        f8 = lambda *s: torch.zeros(*s, device="cuda").to(T["e4m3"])           # noqa: E731
        up = lambda v: -(-v // 128)                                            # noqa: E731
        H, F, E = hidden, inner, experts
        for name, w in (("w1", self.w1), ("w2", self.w2)):
            e, n, m = w.shape
            b[name], b[name + "s"] = f8(e, n, m), f32(e, up(n), up(m))
            b[name + "t"], b[name + "ts"] = f8(e, m, n), f32(e, up(m), up(n))
        b.update(y8=f8(rows, H), y8s=f32(rows, up(H)), y=bf(rows, H), idx=i32(rows, top_k), wt=f32(rows, top_k),
                 counts=i32(E), offsets=i32(E + 1), order=i32(P), pos=i32(rows, top_k), g8=f8(P, H), g8s=f32(P, up(H)),
                 gy=bf(P, H), a=bf(P, 2 * F), m=bf(P, F), m8=f8(P, F), m8s=f32(P, up(F)), o=bf(P, H), out=bf(rows, H),
                 do=bf(P, H), do8=f8(P, H), do8s=f32(P, up(H)), dwt=f32(rows, top_k), dm=bf(P, F), da=bf(P, 2 * F),
                 da8=f8(P, 2 * F), da8s=f32(P, up(2 * F)), dg=bf(P, H), dy=bf(rows, H), dw1=f32(E, 2 * F, H),
                 dw2=f32(E, H, F), rstd=f32(rows))
        need = max(K.route_order_workspace_bytes(P, E), X.expert_weight_grad_workspace_bytes(P, E, 2 * F, H),
                   X.expert_weight_grad_workspace_bytes(P, E, H, F), 256)
        self.ws = torch.zeros(need, dtype=torch.uint8, device="cuda")

    def __call__(self):
        b = self.b
        used = b["offsets"][-1:]
        for name, w in (("w1", self.w1), ("w2", self.w2)):
            X.muon_quantise_blocks(w, b[name], b[name + "s"], b[name + "t"], b[name + "ts"])
        K.muon_norm_forward(self.x, b["y8"], scales=b["y8s"], group=128, rstd=b["rstd"])
        K.muon_norm_forward(self.x, b["y"])
        K.muon_route_forward(K.Route(self.k), self.logits, b["idx"], b["wt"])
        K.muon_route_order(b["idx"], b["counts"], b["offsets"], b["order"], b["pos"], self.ws)
        X.muon_expert_gather(b["order"], b["y8"], b["g8"], scales=b["y8s"], out_scales=b["g8s"])
        X.muon_expert_gather(b["order"], b["y"], b["gy"])
        X.muon_expert_product(b["g8"], b["g8s"], b["w1"], b["w1s"], b["a"], offsets=b["offsets"])
        X.muon_gate_forward(b["a"], y=b["m"], y8=b["m8"], scales=b["m8s"], used=used)
        X.muon_expert_product(b["m8"], b["m8s"], b["w2"], b["w2s"], b["o"], offsets=b["offsets"])
        X.muon_expert_combine(b["pos"], b["o"], b["out"], weights=b["wt"], base=self.x)
        X.muon_expert_combine_backward(b["pos"], self.dout, y=b["o"], weights=b["wt"], dy=b["do"], dweights=b["dwt"],
                                       dy8=b["do8"], scales=b["do8s"])
        X.muon_expert_weight_grad(b["do"], b["m"], b["dw2"], offsets=b["offsets"], workspace=self.ws)
        X.muon_expert_product(b["do8"], b["do8s"], b["w2t"], b["w2ts"], b["dm"], offsets=b["offsets"])
        X.muon_gate_backward(b["a"], b["dm"], da=b["da"], da8=b["da8"], scales=b["da8s"], used=used)
        X.muon_expert_weight_grad(b["da"], b["gy"], b["dw1"], offsets=b["offsets"], workspace=self.ws)
        X.muon_expert_product(b["da8"], b["da8s"], b["w1t"], b["w1ts"], b["dg"], offsets=b["offsets"])
        X.muon_expert_combine(b["pos"], b["dg"], b["dy"])
        return {n: b[n].clone() for n in ("out", "dwt", "dw1", "dw2", "dy", "o", "a")}


def test_path_against_autograd():
    """The layer's output and gradients against autograd in 64 bits with the bf16 weights and the same routing.  An 8-bit
    rounding is 2^-4 at most, 2^-4 / sqrt(3) about in the mean; a product of two such operands is sqrt(2) times that off
    in norm, 5 %, and the worst gradient passes six 8-bit roundings (norm, two matrices, gate, two gradients) and their
    transposed copies: sqrt(6) 3.6 % = 9 % and their bf16 stores 1 %; 15 % covers it."""
    p = Path()
    got = p()
    torch.cuda.synchronize()
    d = lambda t: t.detach().double().cpu().requires_grad_()   # noqa: E731
    x = p.x.double().cpu()
    yn = (x / torch.sqrt(x.square().mean(1, keepdim=True) + 1e-6)).requires_grad_()
    w1, w2, wt = d(p.w1), d(p.w2), d(p.b["wt"])
    idx = p.b["idx"].long().cpu()
    a = torch.einsum("th,tkfh->tkf", yn, w1[idx])
    g, u = a[..., :p.F], a[..., p.F:]
    o = torch.einsum("tkf,tkhf->tkh", g * torch.sigmoid(g) * u, w2[idx])
    ref = x + (wt[:, :, None] * o).sum(1)
    (ref * p.dout.double().cpu()).sum().backward()
    branch = (ref - x).detach()
    off = lambda v, r: float((v.double().cpu() - r).norm() / r.norm())   # noqa: E731
    assert off(got["out"].double().cpu() - x, branch) < 0.15
    for name, want in (("dwt", wt.grad), ("dw1", w1.grad), ("dw2", w2.grad), ("dy", yn.grad)):
        assert off(got[name], want) < 0.15, (name, off(got[name], want))


def test_path_on_another_stream_and_twice_is_the_same():
    p = Path(rows=300, seed=1)
    first = p()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        second = p()
    side.synchronize()
    for n in first:
        assert torch.equal(first[n], second[n]), n


def test_path_replayed_from_a_graph():
    """Captured once, replayed on new inputs with eager work in between; each replay equals the eager run."""
    p, eager = Path(rows=130, seed=2), Path(rows=130, seed=2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        p()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        res = p()
    g = torch.Generator(device="cuda").manual_seed(7)
    for i in range(4):
        p.x.copy_(torch.randn(p.x.shape, generator=g, device="cuda"))
        p.logits.copy_(torch.randn(p.logits.shape, generator=g, device="cuda"))
        eager.x.copy_(p.x)
        eager.logits.copy_(p.logits)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = eager()
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(res[n], want[n]), (i, n)


def test_two_paths_at_once():
    a, b = Path(rows=200, seed=3), Path(rows=150, seed=4)
    wa, wb = a(), b()
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(s):
        ga = a()
    with torch.cuda.stream(t):
        gb = b()
    torch.cuda.synchronize()
    for want, got in ((wa, ga), (wb, gb)):
        for n in want:
            assert torch.equal(want[n], got[n]), n


def test_refused_calls_touch_nothing():
    o = torch.full((8, 64), 7.0, device="cuda")
    y = torch.ones(8, 64, device="cuda")
    pos = torch.zeros(8, 1, dtype=torch.int32, device="cuda")
    with pytest.raises(B.MuonError):
        X.muon_expert_combine(pos, o, o)                       # out is y
    with pytest.raises(ValueError):
        X.muon_expert_combine(pos.cpu(), y, o)
    with pytest.raises(B.MuonError):
        X.muon_expert_combine(torch.zeros(8, 33, dtype=torch.int32, device="cuda"), y, o)
    q = torch.zeros(8, 128, device="cuda").to(T["e4m3"])
    with pytest.raises(B.MuonError):                           # halves of 64 columns share a group
        X.muon_gate_backward(torch.ones(8, 128, device="cuda"), y, da8=q, scales=torch.ones(8, 1, device="cuda"))
    torch.cuda.synchronize()
    assert bool((o == 7).all())
