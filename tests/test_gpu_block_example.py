"""examples/moe_block.py: its gradients against autograd of the same block in
float64 on the CPU, with the same choice of experts and the same dropout mask,
and its loss over a few steps with the Muon, bias and norm updates."""
import numpy as np
import pytest
import torch

from examples import moe_block as X
from oracle import block_oracle as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def test_gradients_match_autograd():
    """bf16 stores on the way (y, the inner product, the experts' outputs and their gradients) leave each
    gradient a few roundings of 2^-9 (root mean square) off: 3 % in norm covers ten of them in a row."""
    b = X.MoEBlock(hidden=64, inner=96, experts=8, top_k=2, groups=2, top_groups=1, p=0.2, seed=3)
    b.bias.copy_(torch.linspace(-0.05, 0.05, 8))
    g = torch.Generator(device="cuda").manual_seed(4)
    x, r = (torch.randn(50, 64, generator=g, device="cuda").bfloat16() for _ in range(2))
    target = torch.randn(50, 64, generator=g, device="cuda")
    loss, dx, dr = b.forward_backward(x, r, target, step=7)
    torch.cuda.synchronize()

    d = lambda t: t.detach().double().cpu().requires_grad_()   # noqa: E731
    xs, rs, R, W1, W2, gain = map(d, (x, r, b.R, b.W1, b.W2, b.gain))
    keep = torch.from_numpy(O.keep_mask(50, 64, 0.2, 3, 7))
    h = rs + torch.where(keep, xs * (65536 / (65536 - O.threshold(0.2))), 0.0)
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-6) * gain
    logits = y @ R.t()
    # the choice itself, from the logits the block saw
    seen = (b.rooms[50]["y"] @ b.R.t()).double().cpu().numpy()
    idx, _, _ = O.route_forward(seen, top_k=2, score="sigmoid", bias=b.bias.double().cpu().numpy(), groups=2,
                                top_groups=1)
    assert np.array_equal(b.rooms[50]["idx"].cpu().numpy(), idx)
    at = torch.from_numpy(idx)
    s = torch.sigmoid(logits).gather(1, at)
    w = s / s.sum(1, keepdim=True)
    o = torch.einsum("tkf,tkhf->tkh", torch.relu(torch.einsum("th,tkfh->tkf", y, W1[at])), W2[at])
    ref = ((h + (w[:, :, None] * o).sum(1)) - target.double().cpu()).square().mean()
    ref.backward()
    assert abs(loss.item() - ref.item()) < 0.03 * ref.item()
    for name, got, want in (("dx", dx, xs), ("dr", dr, rs), ("dR", b.dR, R), ("dW1", b.dW1, W1), ("dW2", b.dW2, W2),
                            ("dgain", b.dgain, gain)):
        off = (got.double().cpu() - want.grad).norm() / want.grad.norm()
        assert off < 0.03, (name, float(off))


def test_update_uses_the_last_call():
    """Steps of several row counts in turn: the bias follows the counts of the step before each update."""
    b = X.MoEBlock(hidden=64, inner=96, experts=8, top_k=2, groups=2, top_groups=1, seed=3)
    g = torch.Generator(device="cuda").manual_seed(5)
    for step, rows in enumerate((50, 37, 120, 50)):
        x, r = (torch.randn(rows, 64, generator=g, device="cuda").bfloat16() for _ in range(2))
        b.forward_backward(x, r, torch.randn(rows, 64, generator=g, device="cuda"), step)
        counts, before = b.rooms[rows]["counts"].cpu().numpy(), b.bias.double().cpu().numpy()
        assert counts.sum() == rows * 2
        b.update(rate=0.125)
        assert np.array_equal(b.bias.double().cpu().numpy(), O.route_balance(counts, before, 0.125)), step


def test_steps_lower_the_loss():
    losses = X.main(["--steps", "12", "--rows", "512"])
    assert all(np.isfinite(losses)) and losses[-1] < 0.8 * losses[0]
