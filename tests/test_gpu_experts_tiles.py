"""Products and weight gradients of more tiles than there are workgroups on the
GPU: each workgroup goes from tile to tile, over runs of every length, against
products in 64 bits on the same device.  Tolerances as in
test_gpu_experts_products.py; sums of magnitudes are taken in 64 bits too.
"""
import numpy as np
import pytest
import torch

from matrix_optimizer_amd import experts as X
from tests.test_gpu_experts_products import CUT
from tests.test_gpu_experts_rows import HALF, SUB, T, U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    X.lib()


def within(got, ref, kind, slack, what):
    bound = HALF[kind] * (ref.abs() + slack) + SUB[kind] + slack
    worst = ((got.double() - ref).abs() / bound).nan_to_num(nan=float("inf")).max().item()
    assert worst <= 1, f"{what}: {worst:.3g} of the bound"


def offsets_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def dequantised(q, scales, rows_too=False):
    """8-bit values times their scales in 64 bits, subnormal values lifted for the magnitudes."""
    s = scales.double()
    s = s.repeat_interleave(128, -1)[..., :q.shape[-1]]
    if rows_too:
        s = s.repeat_interleave(128, -2)[..., :q.shape[-2], :]
    v = q.double()
    low = 2.0 ** -6 if q.dtype == torch.float8_e4m3fn else 2.0 ** -14
    return v * s, torch.where(v == 0, 0.0, v.abs().clamp(min=low)) * s


@pytest.mark.parametrize("n,k,okind", [(8200, 272, "bf16"), (8200, 144, "bf16"), (8192, 640, "bf16"), (8203, 1040, "bf16"),
                                       (8200, 272, "f32"), (8200, 273, "bf16")])
@pytest.mark.parametrize("counts", [[700, 0, 385, 1, 640], [64, 128, 192, 256, 257, 65, 300, 33], [2000], [513] * 4])
def test_products_of_many_tiles(counts, n, k, okind):
    g = torch.Generator(device="cuda").manual_seed(sum(counts) + n + k)
    e, offsets = len(counts), offsets_of(counts)
    live = int(offsets[-1])
    r = live + 3
    eight = lambda *s: (torch.randn(*s, generator=g, device="cuda") * 30).to(T["e4m3"])                # noqa: E731
    scales = lambda *s: torch.exp(torch.randn(*s, generator=g, device="cuda") - 3)                     # noqa: E731
    a, as_ = eight(r, k), scales(r, -(-k // 128))
    w, ws = eight(e, n, k), scales(e, -(-n // 128), -(-k // 128))
    a[live:] = float("nan")
    out = torch.full((r, n), 7.0, device="cuda").to(T[okind])
    X.muon_expert_product(a, as_, w, ws, out, offsets=torch.from_numpy(offsets).cuda())
    assert bool((out[live:] == 7).all())
    av, am = dequantised(a[:live], as_[:live])
    for i, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        wv, wm = dequantised(w[i], ws[i], True)
        slack = ((128 + -(-k // 128) + 4) * 2 * U + (CUT if okind == "bf16" else 0)) * (am[lo:hi] @ wm.T)
        if hi > lo:
            within(out[lo:hi], av[lo:hi] @ wv.T, okind, slack, (i, n, k))


@pytest.mark.parametrize("n,k,okind", [(2056, 2048, "bf16"), (2048, 2056, "f32"), (2056, 2056, "bf16"), (2051, 1027, "bf16")])
@pytest.mark.parametrize("counts", [[0, 1, 63, 64, 65, 200, 130, 7], [0] * 8, [300] * 4 + [1] * 4])
def test_weight_gradients_of_many_tiles(counts, n, k, okind):
    g = torch.Generator(device="cuda").manual_seed(sum(counts) + n + k)
    e, offsets = len(counts), offsets_of(counts)
    live = int(offsets[-1])
    r = live + 70
    dy = (torch.randn(r, n, generator=g, device="cuda") * 0.01).bfloat16()
    x = torch.randn(r, k, generator=g, device="cuda").bfloat16()
    dy[live:], x[live:] = float("nan"), float("inf")
    dw = torch.full((e, n, k), 7.0, device="cuda").to(T[okind])
    ws = torch.full((max(256, X.expert_weight_grad_workspace_bytes(r, e, n, k)),), 0xFF, dtype=torch.uint8, device="cuda")
    X.muon_expert_weight_grad(dy, x, dw, offsets=torch.from_numpy(offsets).cuda(), workspace=ws)
    for i, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        d, v = dy[lo:hi].double(), x[lo:hi].double()
        within(dw[i], d.T @ v, okind, (hi - lo + 16) * 2 * U * (d.abs().T @ v.abs()), i)


@pytest.mark.parametrize("n,k", [(40, 72), (33, 21), (256, 512), (300, 200)])
@pytest.mark.parametrize("counts", [[9000], [5000, 0, 4000], [20000, 1, 3, 700]])
def test_weight_gradients_of_split_rows(counts, n, k):
    """Few tiles, so that the rows go to several workgroups and their parts are joined."""
    g = torch.Generator(device="cuda").manual_seed(sum(counts) + n)
    e, offsets = len(counts), offsets_of(counts)
    r = int(offsets[-1])
    assert X.expert_weight_grad_workspace_bytes(r, e, n, k) > 0
    dy, x = (torch.randn(r, c, generator=g, device="cuda").bfloat16() for c in (n, k))
    for okind in ("f32", "bf16"):
        dw = torch.full((e, n, k), 7.0, device="cuda").to(T[okind])
        ws = torch.full((X.expert_weight_grad_workspace_bytes(r, e, n, k),), 0xFF, dtype=torch.uint8, device="cuda")
        X.muon_expert_weight_grad(dy, x, dw, offsets=torch.from_numpy(offsets).cuda(), workspace=ws)
        for i, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
            d, v = dy[lo:hi].double(), x[lo:hi].double()
            within(dw[i], d.T @ v, okind, (hi - lo + 64) * 2 * U * (d.abs().T @ v.abs()), i)


@pytest.mark.parametrize("n,k,okind", [(1001, 707, "bf16"), (1001, 712, "f32"), (1000, 715, "bf16"), (333, 2049, "f32")])
@pytest.mark.parametrize("pad,shift", [(0, 0), (5, 3)])
def test_weight_gradients_of_odd_widths(n, k, okind, pad, shift):
    """Widths that are no whole pieces, with work enough that the rows are copied to such first."""
    counts = [5000, 0, 2100, 1]
    g = torch.Generator(device="cuda").manual_seed(n + k)
    offsets = offsets_of(counts)
    live = int(offsets[-1])
    r = live + 70
    need = X.expert_weight_grad_workspace_bytes(r, 4, n, k)
    assert need >= 2 * r * (n + k)
    dy, x = (torch.randn(r, c + pad, generator=g, device="cuda").bfloat16()[:, shift:shift + c] for c in (n, k))
    dy[live:], x[live:] = float("nan"), float("inf")
    full = torch.full((4, n + 1, k + pad), 7.0, device="cuda").to(T[okind])
    dw = full[:, :n, shift:shift + k]
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    X.muon_expert_weight_grad(dy, x, dw, offsets=torch.from_numpy(offsets).cuda(), workspace=ws[:need])
    for i, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        d, v = dy[lo:hi].double(), x[lo:hi].double()
        within(dw[i], d.T @ v, okind, (hi - lo + 64) * 2 * U * (d.abs().T @ v.abs()), i)
    edge = full.float().clone()
    edge[:, :n, shift:shift + k] = 7
    assert bool((edge == 7).all()) and bool((ws[need:] == 0xFF).all())


@pytest.mark.parametrize("n,k", [(1001, 1003), (1001, 712), (1000, 1005)])
def test_weight_gradients_of_odd_widths_leave_rows_without_a_run(n, k):
    """Rows behind the last run are not copied either: the copies' places for them in the workspace keep what they
    held.  16 experts are enough tiles, so that the workspace holds the copies alone: dy's, then x's."""
    counts = [90] * 15 + [113]
    offsets = offsets_of(counts)
    live = int(offsets[-1])
    r = live + 301
    g = torch.Generator(device="cuda").manual_seed(n + k)
    wide = [-(-c // 8) * 8 for c in (n, k)]
    need = X.expert_weight_grad_workspace_bytes(r, 16, n, k)
    assert need == -(-2 * r * sum(wide) // 256) * 256
    dy, x = (torch.randn(r, c, generator=g, device="cuda").bfloat16() for c in (n, k))
    dw = torch.full((16, n, k), 7.0, device="cuda")
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    X.muon_expert_weight_grad(dy, x, dw, offsets=torch.from_numpy(offsets).cuda(), workspace=ws)
    at = 0
    for c, of in zip(wide, (dy, x)):
        rows = ws[at:at + 2 * r * c].view(r, 2 * c)
        copied = rows[:live].view(torch.bfloat16)[:, :of.shape[1]]
        assert torch.equal(copied, of[:live]) and bool((rows[live:] == 0xFF).all())
        at += 2 * r * c
    for i, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        d, v = dy[lo:hi].double(), x[lo:hi].double()
        within(dw[i], d.T @ v, "f32", (hi - lo + 16) * 2 * U * (d.abs().T @ v.abs()), i)


def test_weight_gradients_of_odd_widths_and_bad_offsets():
    """Runs out of order and offsets outside the rows: the copies reach to the end of the furthest run."""
    n, k, r = 1001, 1003, 1500
    g = torch.Generator(device="cuda").manual_seed(3)
    dy, x = (torch.randn(r, c, generator=g, device="cuda").bfloat16() for c in (n, k))
    ws = torch.full((X.expert_weight_grad_workspace_bytes(r, 3, n, k),), 0xFF, dtype=torch.uint8, device="cuda")
    assert ws.numel() >= 2 * r * (n + k)
    for offsets in ([700, 1400, 30, 200], [-7, 600, 600, 1 << 30], [0, 0, 0, -2**31], [1499, 1500, 1500, 3]):
        dw = torch.full((3, n, k), 7.0, device="cuda")
        X.muon_expert_weight_grad(dy, x, dw, offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"), workspace=ws)
        at = [min(max(v, 0), r) for v in offsets]
        for i, (lo, hi) in enumerate(zip(at, at[1:])):
            d, v = dy[lo:max(lo, hi)].double(), x[lo:max(lo, hi)].double()
            within(dw[i], d.T @ v, "f32", (max(hi - lo, 0) + 64) * 2 * U * (d.abs().T @ v.abs()), (offsets, i))


def test_products_repeat_bitwise():
    """The same call twice, with other work on the card in between: the same bits."""
    g = torch.Generator(device="cuda").manual_seed(1)
    counts = [900, 3, 450, 0, 647]
    offsets = torch.from_numpy(offsets_of(counts)).cuda()
    eight = lambda *s: (torch.randn(*s, generator=g, device="cuda") * 30).to(T["e4m3"])   # noqa: E731
    a, w = eight(2000, 1152), eight(5, 6144, 1152)
    as_, ws = torch.rand(2000, 9, generator=g, device="cuda"), torch.rand(5, 48, 9, generator=g, device="cuda")
    first = torch.zeros(2000, 6144, dtype=torch.bfloat16, device="cuda")
    second = torch.zeros_like(first)
    X.muon_expert_product(a, as_, w, ws, first, offsets=offsets)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        z = torch.randn(4096, 4096, device="cuda") @ torch.randn(4096, 4096, device="cuda")
    X.muon_expert_product(a, as_, w, ws, second, offsets=offsets)
    torch.cuda.synchronize()
    assert torch.equal(first, second) and bool(torch.isfinite(z).all())
