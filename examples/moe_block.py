"""Training steps of one decoder block with routed experts on libmuon: the row
operators (matrix_optimizer_amd.block) around the matrices that muon_step
updates.

    python -m examples.moe_block [--steps N] [--rows T]

A step, for a branch output x and the residual stream r:

    h, y     norm of r + dropout(x)                 muon_norm_forward
    experts  top_k of E by sigmoid(y R^T) + bias    muon_route_forward
    order    the (row, slot) pairs by expert        muon_route_order
    o_e      relu(y_e W1_e^T) W2_e^T per expert     library products
    out      h + sum over slots of weight o_e

and back from a squared error: muon_route_backward, muon_norm_backward.  The
router R and the expert tensors W1, W2 go through Muon (BatchedMuon), the
balance bias through muon_route_balance, the norm's weight is plain gradient
descent.  Everything is bf16 on the device but the bias and the norm's weight.
"""
from __future__ import annotations

import argparse

import torch

from matrix_optimizer_amd import binding as B
from matrix_optimizer_amd import block as K


class MoEBlock:
    def __init__(self, hidden=256, inner=512, experts=16, top_k=4, groups=4, top_groups=2, p=0.1, seed=0, lr=0.02):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.H, self.F, self.E, self.k, self.p, self.seed = hidden, inner, experts, top_k, p, seed
        self.route = K.Route(top_k, "sigmoid", groups, top_groups, renormalise=True, scale=1.0)
        # R [E, H], W1 [E, F, H], W2 [E, H, F] live in Muon's batch buffers
        self.muon = B.BatchedMuon([(experts, hidden), (experts, inner, hidden), (experts, hidden, inner)], torch.bfloat16,
                                  B.HParams(lr=lr, weight_decay=0.0))
        self.R, self.W1, self.W2 = (self._view(i, self.muon.params) for i in range(3))
        self.dR, self.dW1, self.dW2 = (self._view(i, self.muon.grads) for i in range(3))
        for w in (self.R, self.W1, self.W2):
            w.copy_(torch.randn(w.shape, generator=g, device="cuda") * w.shape[-1] ** -0.5)
        self.gain = torch.ones(hidden, device="cuda")
        self.dgain = torch.empty_like(self.gain)
        self.bias = torch.zeros(experts, device="cuda")
        self.rooms, self.last = {}, None

    def _view(self, i, buffers):
        """Parameter i inside the batch buffers (its matrices are one run of one batch here)."""
        for b in self.muon.plan.batches:
            for param, first, count, offset in b.segments:
                if param == i:
                    m = buffers[b.index].view(-1, b.M, b.N)[offset // (b.M * b.N):][:count]
                    return m if len(self.muon.plan.shapes[i]) == 3 else m[0]
        raise KeyError(i)

    def _room(self, rows):
        """Buffers for `rows` rows, kept from step to step."""
        if rows not in self.rooms:
            T, H, E, k = rows, self.H, self.E, self.k
            bf = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")   # noqa: E731
            f32 = lambda *s: torch.empty(*s, device="cuda")                        # noqa: E731
            i32 = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")     # noqa: E731
            ws = max(K.norm_workspace_bytes(T, H), K.route_order_workspace_bytes(T * k, E), 256)
            self.rooms[rows] = dict(h=bf(T, H), y=bf(T, H), rstd=f32(T), dr=bf(T, H), dx=bf(T, H), idx=i32(T, k), w=f32(T, k),
                                    dlogits=bf(T, E), counts=i32(E), offsets=i32(E + 1), order=i32(T * k), place=i32(T, k),
                                    ws=torch.empty(ws, dtype=torch.uint8, device="cuda"))
        return self.rooms[rows]

    def forward_backward(self, x, residual, target, step=0):
        """(loss, dx, dresidual); the parameters' gradients are left in dR, dW1, dW2, dgain."""
        T, k = x.shape[0], self.k
        m = self.last = self._room(T)
        drop = K.Dropout(self.p, self.seed, step)
        K.muon_norm_forward(x, m["y"], residual=residual, h=m["h"], weight=self.gain, rstd=m["rstd"], dropout=drop)
        logits = m["y"] @ self.R.t()
        K.muon_route_forward(self.route, logits, m["idx"], m["w"], bias=self.bias)
        K.muon_route_order(m["idx"], m["counts"], m["offsets"], m["order"], m["place"], m["ws"])
        off = m["offsets"].tolist()
        token = m["order"][:off[-1]].long() // k
        ye = m["y"][token]
        inner = torch.empty(off[-1], self.F, dtype=x.dtype, device="cuda")
        o = torch.empty_like(ye)
        for e in range(self.E):
            s = slice(off[e], off[e + 1])
            inner[s] = torch.relu(ye[s] @ self.W1[e].t())
            o[s] = inner[s] @ self.W2[e].t()
        slots = o[m["place"].long()].float()                       # [T, k, H]: every row has its k experts here
        out = m["h"].float() + (slots * m["w"][:, :, None]).sum(1)
        err = out - target
        loss = err.square().mean()

        dout = err * (2 / err.numel())
        dw = (slots * dout[:, None, :]).sum(2)
        do = torch.empty_like(o)
        do[m["place"].long().reshape(-1)] = (m["w"][:, :, None] * dout[:, None, :]).reshape(T * k, -1).to(o.dtype)
        dye = torch.empty_like(ye)
        for e in range(self.E):
            s = slice(off[e], off[e + 1])
            self.dW2[e] = do[s].t() @ inner[s]
            di = (do[s] @ self.W2[e]) * (inner[s] > 0)
            self.dW1[e] = di.t() @ ye[s]
            dye[s] = di @ self.W1[e]
        K.muon_route_backward(self.route, logits, m["idx"], m["w"], dw, m["dlogits"])
        self.dR.copy_(m["dlogits"].t() @ m["y"])
        dy = (dye[m["place"].long()].float().sum(1) + (m["dlogits"] @ self.R).float()).to(x.dtype)
        K.muon_norm_backward(dy, m["h"], m["rstd"], weight=self.gain, dh=dout.to(x.dtype), dresidual=m["dr"], dx=m["dx"],
                             dweight=self.dgain, workspace=m["ws"], dropout=drop)
        return loss, m["dx"], m["dr"]

    def update(self, rate=1e-3, gain_lr=0.1):
        self.muon.step()
        self.gain.add_(self.dgain, alpha=-gain_lr)
        K.muon_route_balance(self.last["counts"], self.bias, self.bias, rate)   # of the last forward_backward


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--rows", type=int, default=2048)
    a = ap.parse_args(argv)
    block = MoEBlock()
    g = torch.Generator(device="cuda").manual_seed(1)
    data = lambda: torch.randn(a.rows, block.H, generator=g, device="cuda")   # noqa: E731
    x, r = data().bfloat16(), data().bfloat16()
    target = r.float() + torch.tanh(data() * 0.1 + x.float().roll(1, 1))
    losses = []
    for step in range(a.steps):
        loss, _, _ = block.forward_backward(x, r, target, step)
        block.update()
        losses.append(float(loss))
        counts = block.rooms[a.rows]["counts"]
        print(f"step {step:3d}  loss {losses[-1]:.4f}  busiest expert {int(counts.max())} of {a.rows * block.k} pairs")
    return losses


if __name__ == "__main__":
    main()
