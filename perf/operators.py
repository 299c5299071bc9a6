"""Cases of the row operators of a decoder block with routed experts: root-mean-square norm with the
residual's addition (forward with 8-bit outputs, backward), dropout from a counter-based generator,
routing to experts (forward, backward) and the order of the routed pairs with the balance update.

``run`` computes a case in elementary torch operations, or through matrix_optimizer_amd.block where
``own`` is true; ``exact`` gives the floating outputs in 64 bits.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
BYTES = {"f32": 4, "bf16": 2, "e4m3": 1, "e5m2": 1}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
EPS = 1e-6
RATE = 1e-3          # step of the balance bias
U32 = 0xFFFFFFFF


def listed():
    return [
        # one new token's row between two layers of a served model: latency alone
        dict(name="norm_one_token", op="norm_forward", rows=1, cols=4096, type="bf16", out="bf16", group=0,
             residual=True, weight="bf16", p=0.0, wide=False),
        # a prompt's rows before an 8-bit product: scales per 128 columns; the MLP width of the large matrices
        dict(name="norm_prompt_e4m3", op="norm_forward", rows=4096, cols=8192, type="bf16", out="e4m3", group=128,
             residual=True, weight="bf16", p=0.0, wide=False),
        # a training step's rows: the branch's dropout, the residual stream kept for the backward pass
        dict(name="norm_train_dropout", op="norm_forward", rows=16384, cols=4096, type="bf16", out="bf16", group=0,
             residual=True, weight="f32", p=0.1, wide=False),
        # the same step's backward pass
        dict(name="norm_train_backward", op="norm_backward", rows=16384, cols=4096, type="bf16", weight="f32",
             p=0.1, stream=True, wide=False),
        # the check precision, an odd width inside a wider buffer: no row but the first is aligned
        dict(name="norm_odd_backward", op="norm_backward", rows=777, cols=2051, type="f32", weight="f32", p=0.0,
             stream=False, wide=True),
        # dropout over one large activation
        dict(name="dropout_large", op="dropout", rows=8192, cols=28672, type="bf16", p=0.1, wide=False),
        # dropout over a few odd fp32 rows
        dict(name="dropout_odd", op="dropout", rows=129, cols=1001, type="f32", p=0.5, wide=True),
        # a training step's routing: sigmoid scores, a balance bias, 4 of 8 groups, padding tokens
        dict(name="route_train_groups", op="route_forward", rows=32768, experts=256, k=8, groups=8, top_groups=4,
             type="bf16", score="sigmoid", bias=True, renormalise=True, padding=0.03, closed=0.0, scores=False),
        # a served batch's routing, 64 experts as in the expert workload
        dict(name="route_served", op="route_forward", rows=16, experts=64, k=6, groups=1, top_groups=1,
             type="f32", score="softmax", bias=False, renormalise=False, padding=0.0, closed=0.0, scores=False),
        # the gradient of the router's logits, with that of the scores (an auxiliary loss reads them)
        dict(name="route_train_backward", op="route_backward", rows=32768, experts=64, k=6, type="bf16",
             score="softmax", renormalise=True, padding=0.03, dscores=True),
        # the pairs of a training step in the experts' order, and the balance bias after it
        dict(name="order_train", op="route_order", rows=131072, experts=256, k=8, padding=0.03),
        # the pairs of a served batch
        dict(name="order_served", op="route_order", rows=16, experts=64, k=6, padding=0.0),
    ]


def _spread(rng, lo, hi):
    """A size between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    n = _spread(rng, lo, hi)
    return n if rng.random() < 0.4 else max(lo, n // 64 * 64)


def draw(rng):
    op = rng.choice(["norm_forward", "norm_forward", "norm_backward", "dropout", "route_forward", "route_forward",
                     "route_backward", "route_order"])
    if op in ("norm_forward", "norm_backward"):
        cols = _width(rng, 64, 16384)
        kind = rng.choice(["bf16", "bf16", "f32"])
        rows = min(_spread(rng, 1, 16384), (160 << 20) // (BYTES[kind] * cols))
        case = dict(op=op, rows=rows, cols=cols, type=kind,
                    weight=rng.choice(["f32", "bf16", "none"]), p=rng.choice([0.0, 0.0, 0.1, 0.25]),
                    wide=rng.random() < 0.3)
        if op == "norm_forward":
            out = rng.choice([case["type"], "bf16", "e4m3", "e4m3", "e5m2"])
            return dict(case, out=out, group=rng.choice([0, 32, 64, 128]) if out in LARGEST else 0,
                        residual=rng.random() < 0.7)
        return dict(case, stream=rng.random() < 0.7)
    if op == "dropout":
        cols = _width(rng, 16, 32768)
        kind = rng.choice(["bf16", "f32"])
        rows = min(_spread(rng, 1, 65536), (1 << 28) // (BYTES[kind] * cols))
        return dict(op=op, rows=rows, cols=cols, type=kind, p=rng.choice([0.05, 0.1, 0.3, 0.5]),
                    wide=rng.random() < 0.3)
    experts = rng.choice([8, 16, 24, 32, 40, 64, 96, 128, 160, 256, 384, 512])
    k = rng.randint(1, min(10, experts // 2))
    rows = min(_spread(rng, 1, 65536), (1 << 23) // experts)
    padding = rng.choice([0.0, 0.05])
    if op == "route_order":
        return dict(op=op, rows=rows, experts=experts, k=k, padding=padding)
    case = dict(op=op, rows=rows, experts=experts, k=k, type=rng.choice(["bf16", "f32"]),
                score=rng.choice(["softmax", "sigmoid"]), renormalise=rng.random() < 0.6, padding=padding)
    if op == "route_backward":
        return dict(case, dscores=rng.random() < 0.5)
    groups = rng.choice([1, 1, 4, 8])
    if experts // groups < 2:
        groups = 1
    fewest = -(-k // (experts // groups))
    return dict(case, groups=groups, top_groups=rng.randint(fewest, max(fewest, groups // 2)),
                bias=rng.random() < 0.6, closed=rng.choice([0.0, 0.1]), scores=rng.random() < 0.3)


def _rows_of(gen, rows, cols, dtype, wide, scale=1.0):
    """Normal values [rows, cols]; `wide`: as columns 3.. of a buffer 8 columns wider and one more."""
    if not wide:
        return (torch.randn(rows, cols, generator=gen, device="cuda") * scale).to(dtype)
    full = (torch.randn(rows, cols + 9, generator=gen, device="cuda") * scale).to(dtype)
    return full[:, 3:3 + cols]


def _logits_of(gen, case):
    t, e = case["rows"], case["experts"]
    l = torch.randn(t, e, generator=gen, device="cuda") * 1.5 + torch.randn(e, generator=gen, device="cuda") * 0.5
    return l.to(TYPES[case["type"]])


def _choice_of(gen, case):
    """Expert indices [rows, k] as a router gives them: distinct in a row, some experts busier; -1 in padding rows."""
    t, e, k = case["rows"], case["experts"], case["k"]
    l = torch.randn(t, e, generator=gen, device="cuda") + torch.randn(e, generator=gen, device="cuda") * 0.7
    idx = torch.topk(l, k, dim=1).indices.to(torch.int32)
    idx[torch.rand(t, generator=gen, device="cuda") < case["padding"]] = -1
    return idx


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dev, op = "cuda", case["op"]
    st = {"case": case}
    if op in ("norm_forward", "norm_backward", "dropout"):
        t, h, dt = case["rows"], case["cols"], TYPES[case["type"]]
        st["seed"], st["offset"] = int(seed) * 2654435761 + 12345, int(seed) % 1000 + (5 << 32)
        if op == "dropout":
            st["x"] = _rows_of(gen, t, h, dt, case["wide"])
            st["y"] = torch.empty(t, h, dtype=dt, device=dev)
            return st
        st["w"] = None
        if case["weight"] != "none":
            st["w"] = (1 + 0.1 * torch.randn(h, generator=gen, device=dev)).to(TYPES[case["weight"]])
        if op == "norm_forward":
            out = TYPES[case["out"]]
            st["x"] = _rows_of(gen, t, h, dt, case["wide"], 0.7)
            st["r"] = None
            if case["residual"]:   # a residual stream: a few columns much larger than the others
                st["r"] = _rows_of(gen, t, h, dt, case["wide"], 2.0)
                st["r"][:, :: max(1, h // 5)] *= 8
            st["y"] = torch.empty(t, h, dtype=out, device=dev)
            st["h"] = torch.empty(t, h, dtype=dt, device=dev) if case["residual"] or case["p"] > 0 else None
            st["rstd"] = torch.empty(t, dtype=torch.float32, device=dev)
            st["scales"] = None
            if case["out"] in LARGEST:
                g = case["group"] or h
                st["scales"] = torch.empty(t, -(-h // g), dtype=torch.float32, device=dev)
            return st
        st["h"] = _rows_of(gen, t, h, dt, case["wide"], 2.0)
        st["rstd"] = torch.rsqrt(st["h"].double().square().mean(1) + EPS).float()
        st["dy"] = _rows_of(gen, t, h, dt, case["wide"], 1e-2)
        st["dh"] = _rows_of(gen, t, h, dt, False, 1e-2) if case["stream"] else None
        st["dr"] = torch.empty(t, h, dtype=dt, device=dev)
        st["dx"] = torch.empty(t, h, dtype=dt, device=dev) if case["p"] > 0 else None
        st["dw"] = torch.empty(h, dtype=torch.float32, device=dev) if st["w"] is not None else None
        return st
    t, e, k = case["rows"], case["experts"], case["k"]
    if op == "route_order":
        st["idx"] = _choice_of(gen, case)
        st["bias"] = torch.randn(e, generator=gen, device=dev) * 0.05
        st["counts"] = torch.empty(e, dtype=torch.int32, device=dev)
        st["offsets"] = torch.empty(e + 1, dtype=torch.int32, device=dev)
        st["order"] = torch.empty(t * k, dtype=torch.int32, device=dev)
        st["position"] = torch.empty(t, k, dtype=torch.int32, device=dev)
        st["new_bias"] = torch.empty(e, dtype=torch.float32, device=dev)
        return st
    st["logits"] = _logits_of(gen, case)
    if op == "route_forward":
        if case["closed"] > 0:
            st["logits"].masked_fill_(torch.rand(t, e, generator=gen, device=dev) < case["closed"], -math.inf)
        st["bias"] = torch.randn(e, generator=gen, device=dev) * 0.05 if case["bias"] else None
        st["keep"] = torch.rand(t, generator=gen, device=dev) >= case["padding"] if case["padding"] > 0 else None
        st["idx"] = torch.empty(t, k, dtype=torch.int32, device=dev)
        st["weights"] = torch.empty(t, k, dtype=torch.float32, device=dev)
        st["scores"] = torch.empty(t, e, dtype=torch.float32, device=dev) if case["scores"] else None
        return st
    # the backward pass has the forward's choice and weights in hand
    l = st["logits"].double()
    st["idx"] = torch.topk(l, k, dim=1).indices.to(torch.int32)
    s = torch.softmax(l, 1) if case["score"] == "softmax" else torch.sigmoid(l)
    w = s.gather(1, st["idx"].long())
    if case["renormalise"]:
        w = w / w.sum(1, keepdim=True)
    pad = torch.rand(t, generator=gen, device=dev) < case["padding"]
    st["idx"][pad] = -1
    st["weights"] = (2.5 * w).float().masked_fill(pad[:, None], 0)
    st["dweights"] = torch.randn(t, k, generator=gen, device=dev) * 1e-2
    st["dscores"] = torch.randn(t, e, generator=gen, device=dev) * 1e-3 if case["dscores"] else None
    st["dlogits"] = torch.empty(t, e, dtype=TYPES[case["type"]], device=dev)
    return st


# ---- the plain forms --------------------------------------------------------

def _philox_round(c0, c1, c2, c3, k0, k1):
    a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57        # 64-bit wrapping products of 32-bit words
    return (((b >> 32) & U32) ^ c1 ^ k0, b & U32, ((a >> 32) & U32) ^ c3 ^ k1, a & U32)


def _keep(rows, cols, p, seed, offset):
    """Philox4x32-10 of (column / 8, row, offset) keyed by the seed: eight 16-bit numbers a block, kept from p 2^16 on."""
    blocks = (cols + 7) // 8
    c0 = torch.arange(blocks, device="cuda", dtype=torch.int64)[None, :].expand(rows, blocks)
    c1 = torch.arange(rows, device="cuda", dtype=torch.int64)[:, None].expand(rows, blocks)
    c2, c3 = torch.full_like(c0, offset & U32), torch.full_like(c0, (offset >> 32) & U32)
    k0, k1 = seed & U32, (seed >> 32) & U32
    d0, d1 = 0x9E3779B9, 0xBB67AE85
    c = _philox_round(c0, c1, c2, c3, k0, k1)
    c = _philox_round(*c, (k0 + d0) & U32, (k1 + d1) & U32)
    c = _philox_round(*c, (k0 + 2 * d0) & U32, (k1 + 2 * d1) & U32)
    c = _philox_round(*c, (k0 + 3 * d0) & U32, (k1 + 3 * d1) & U32)
    c = _philox_round(*c, (k0 + 4 * d0) & U32, (k1 + 4 * d1) & U32)
    c = _philox_round(*c, (k0 + 5 * d0) & U32, (k1 + 5 * d1) & U32)
    c = _philox_round(*c, (k0 + 6 * d0) & U32, (k1 + 6 * d1) & U32)
    c = _philox_round(*c, (k0 + 7 * d0) & U32, (k1 + 7 * d1) & U32)
    c = _philox_round(*c, (k0 + 8 * d0) & U32, (k1 + 8 * d1) & U32)
    c = _philox_round(*c, (k0 + 9 * d0) & U32, (k1 + 9 * d1) & U32)
    c = torch.stack(c, 2)
    numbers = torch.stack((c & 0xFFFF, c >> 16), 3).reshape(rows, blocks * 8)[:, :cols]
    return numbers >= int(p * 65536 + 0.5)


def _dropped(x, case, st):
    if case["p"] == 0:
        return x
    keep = _keep(case["rows"], case["cols"], case["p"], st["seed"] & (2**64 - 1), st["offset"])
    return torch.where(keep, x * (65536.0 / (65536 - int(case["p"] * 65536 + 0.5))), 0.0)


def _plain_norm_forward(case, st):
    z = _dropped(st["x"].float(), case, st)
    if st["r"] is not None:
        z = z + st["r"].float()
    rstd = 1 / torch.sqrt((z * z).mean(1) + EPS)
    y = z * rstd[:, None]
    if st["w"] is not None:
        y = y * st["w"].float()
    out = {"rstd": rstd, "h": z.to(st["x"].dtype) if st["h"] is not None else None}
    if st["scales"] is None:
        return dict(out, y=y.to(TYPES[case["out"]]))
    g, top = case["group"] or case["cols"], LARGEST[case["out"]]
    n = -(-case["cols"] // g)
    parts = torch.nn.functional.pad(y, (0, n * g - case["cols"])).reshape(case["rows"], n, g)
    most = parts.abs().amax(2)
    scales = torch.where(most > 0, torch.clamp(most / top, min=2.0**-126), 1.0)
    q = torch.clamp(parts / scales[:, :, None], -top, top).reshape(case["rows"], n * g)[:, : case["cols"]]
    return dict(out, y=q.to(TYPES[case["out"]]), scales=scales)


def _plain_norm_backward(case, st):
    dy, rstd = st["dy"].float(), st["rstd"][:, None]
    xhat = st["h"].float() * rstd
    g = dy * st["w"].float() if st["w"] is not None else dy
    dz = rstd * (g - xhat * (g * xhat).mean(1, keepdim=True))
    if st["dh"] is not None:
        dz = dz + st["dh"].float()
    return {"dr": dz.to(st["h"].dtype),
            "dx": _dropped(dz, case, st).to(st["h"].dtype) if st["dx"] is not None else None,
            "dw": (dy * xhat).sum(0) if st["w"] is not None else None}


def _plain_scores(l, score):
    """Scores in 64 bits; 0 where an expert is closed (a logit of -inf)."""
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    most = l.amax(1, keepdim=True)
    e = torch.exp(l - torch.where(most == -math.inf, 0.0, most))
    total = e.sum(1, keepdim=True)
    return e / torch.where(total > 0, total, 1.0)


def _plain_route_forward(case, st):
    t, e, k, n = case["rows"], case["experts"], case["k"], case["groups"]
    l = st["logits"].double()                 # 64 bits: the order of near scores decides who is chosen
    open_ = l > -math.inf
    s = torch.where(open_, _plain_scores(l, case["score"]), 0.0)
    rank = s + st["bias"].double() if st["bias"] is not None else l
    rank = torch.where(open_, rank, -math.inf)
    if n > 1:
        by = torch.where(open_, s + st["bias"].double() if st["bias"] is not None else s, -math.inf)
        two = torch.sort(by.reshape(t, n, e // n), dim=2, descending=True, stable=True).values[:, :, :2]
        of_group = two[:, :, 0] + torch.where(two[:, :, 1] > -math.inf, two[:, :, 1], 0.0)
        best = torch.sort(of_group, dim=1, descending=True, stable=True).indices[:, : case["top_groups"]]
        kept = torch.zeros(t, n, dtype=torch.bool, device=l.device).scatter_(1, best, True)
        rank = torch.where(kept.repeat_interleave(e // n, 1), rank, -math.inf)
    got = torch.sort(rank, dim=1, descending=True, stable=True)
    idx = got.indices[:, :k]
    valid = got.values[:, :k] > -math.inf
    if st["keep"] is not None:
        valid = valid & st["keep"][:, None]
        s = torch.where(st["keep"][:, None], s, 0.0)
    w = torch.where(valid, s.gather(1, idx), 0.0)
    if case["renormalise"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    return {"idx": torch.where(valid, idx, -1).to(torch.int32), "weights": (w * 2.5).float(),
            "scores": s.float() if st["scores"] is not None else None}


def _plain_route_backward(case, st):
    l = st["logits"].float()
    chosen = st["idx"] >= 0
    row = chosen[:, :1]
    idx = st["idx"].clamp(min=0).long()
    a = torch.where(chosen, st["weights"] * st["dweights"], 0.0)
    if case["renormalise"]:
        a = a - st["weights"] / 2.5 * a.sum(1, keepdim=True)
    d = torch.zeros_like(l).scatter_add_(1, idx, torch.where(chosen, a, 0.0))
    if case["score"] == "sigmoid":
        s = 1 / (1 + torch.exp(-l))
        d = d * (1 - s)
        if st["dscores"] is not None:
            d = d + st["dscores"] * s * (1 - s)
    else:
        s = torch.exp(l - l.amax(1, keepdim=True))
        s = s / s.sum(1, keepdim=True)
        if not case["renormalise"]:
            d = d - s * a.sum(1, keepdim=True)
        if st["dscores"] is not None:
            d = d + s * (st["dscores"] - (s * st["dscores"]).sum(1, keepdim=True))
    return {"dlogits": torch.where(row, d, 0.0).to(st["logits"].dtype)}


def _plain_route_order(case, st):
    e, flat = case["experts"], st["idx"].reshape(-1)
    n = flat.numel()
    key = torch.where(flat < 0, e, flat)
    got = torch.sort(key, stable=True)
    offsets = torch.searchsorted(got.values.contiguous(), torch.arange(e + 1, dtype=torch.int32, device="cuda"))
    places = torch.arange(n, device="cuda")
    position = torch.empty_like(places).scatter_(0, got.indices, places)
    counts = offsets[1:] - offsets[:-1]
    new = st["bias"] + RATE * torch.sign(counts.sum() - counts * e).float()
    return {"counts": counts.to(torch.int32), "offsets": offsets.to(torch.int32), "new_bias": new,
            "order": torch.where(places < offsets[e], got.indices, -1).to(torch.int32),
            "position": torch.where(flat < 0, -1, position).to(torch.int32).reshape(st["idx"].shape)}


# ---- the framework's operators ----------------------------------------------

def _room(st, need):
    """A workspace, kept beside the buffers that it serves."""
    if "room" not in st:
        st["room"] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    return st["room"]


def _own_norm_forward(K, case, st):
    drop = K.Dropout(case["p"], st["seed"], st["offset"]) if case["p"] > 0 else None
    K.muon_norm_forward(st["x"], st["y"], residual=st["r"], h=st["h"], weight=st["w"], rstd=st["rstd"],
                        scales=st["scales"], group=case["group"], eps=EPS, dropout=drop)
    return {"rstd": st["rstd"], "h": st["h"], "y": st["y"], "scales": st["scales"]}


def _own_norm_backward(K, case, st):
    drop = K.Dropout(case["p"], st["seed"], st["offset"]) if case["p"] > 0 else None
    room = _room(st, K.norm_workspace_bytes(case["rows"], case["cols"])) if st["dw"] is not None else None
    K.muon_norm_backward(st["dy"], st["h"], st["rstd"], weight=st["w"], dh=st["dh"], dresidual=st["dr"], dx=st["dx"],
                         dweight=st["dw"], workspace=room, dropout=drop)
    return {"dr": st["dr"], "dx": st["dx"], "dw": st["dw"]}


def _own_dropout(K, case, st):
    K.muon_dropout(st["x"], st["y"], K.Dropout(case["p"], st["seed"], st["offset"]))
    return {"y": st["y"]}


def _own_route_forward(K, case, st):
    spec = K.Route(top_k=case["k"], score=case["score"], groups=case["groups"], top_groups=case["top_groups"],
                   group_top=2, renormalise=case["renormalise"], scale=2.5)
    K.muon_route_forward(spec, st["logits"], st["idx"], st["weights"], bias=st["bias"], token_mask=st["keep"],
                         scores=st["scores"])
    return {"idx": st["idx"], "weights": st["weights"], "scores": st["scores"]}


def _own_route_backward(K, case, st):
    spec = K.Route(top_k=case["k"], score=case["score"], renormalise=case["renormalise"], scale=2.5)
    K.muon_route_backward(spec, st["logits"], st["idx"], st["weights"], st["dweights"], st["dlogits"],
                          dscores=st["dscores"])
    return {"dlogits": st["dlogits"]}


def _own_route_order(K, case, st):
    room = _room(st, K.route_order_workspace_bytes(case["rows"] * case["k"], case["experts"]))
    K.muon_route_order(st["idx"], st["counts"], st["offsets"], st["order"], st["position"], room)
    K.muon_route_balance(st["counts"], st["bias"], st["new_bias"], RATE)
    return {"counts": st["counts"], "offsets": st["offsets"], "order": st["order"], "position": st["position"],
            "new_bias": st["new_bias"]}


def run(state):
    case = state["case"]
    if own:
        from matrix_optimizer_amd import block as K
        return {"norm_forward": _own_norm_forward, "norm_backward": _own_norm_backward, "dropout": _own_dropout,
                "route_forward": _own_route_forward, "route_backward": _own_route_backward,
                "route_order": _own_route_order}[case["op"]](K, case, state)
    if case["op"] == "dropout":
        return {"y": _dropped(state["x"].float(), case, state).to(state["x"].dtype)}
    return {"norm_forward": _plain_norm_forward, "norm_backward": _plain_norm_backward,
            "route_forward": _plain_route_forward, "route_backward": _plain_route_backward,
            "route_order": _plain_route_order}[case["op"]](case, state)


def work(case):
    op = case["op"]
    if op in ("norm_forward", "norm_backward", "dropout"):
        t, h, b = case["rows"], case["cols"], BYTES[case["type"]]
        n = t * h
        if op == "dropout":
            return {"bytes": 2 * n * b, "flops": n}
        w = 0 if case["weight"] == "none" else h * BYTES[case["weight"]]
        if op == "norm_forward":
            stored = 1 if case["residual"] or case["p"] > 0 else 0
            scales = t * -(-h // (case["group"] or h)) * 4 if case["out"] in LARGEST else 0
            return {"bytes": n * b * (1 + case["residual"] + stored) + n * BYTES[case["out"]] + w + 4 * t + scales,
                    "flops": 6 * n}
        return {"bytes": n * b * (3 + case["stream"] + (case["p"] > 0)) + 4 * t + w + (4 * h if w else 0),
                "flops": 10 * n}
    t, e, k = case["rows"], case["experts"], case["k"]
    if op == "route_forward":
        return {"bytes": t * e * (BYTES[case["type"]] + 4 * case["scores"]) + 8 * t * k + 4 * e * case["bias"]
                + (t if case["padding"] > 0 else 0), "flops": t * e * 4}
    if op == "route_backward":
        read = case["score"] == "softmax" and not case["renormalise"] or case["dscores"] or case["score"] == "sigmoid"
        return {"bytes": t * e * (BYTES[case["type"]] * (1 + read) + 4 * case["dscores"]) + 12 * t * k,
                "flops": t * e * 4}
    return {"bytes": 12 * t * k + 4 * (4 * e + 1), "flops": t * k}


# ---- the definitions in 64 bits ---------------------------------------------

def _exact_keep(rows, cols, p, seed, offset):
    """The same generator by its definition, on the host in unsigned 64-bit integers."""
    blocks = (cols + 7) // 8
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    ctr = [np.broadcast_to(np.arange(blocks, dtype=np.uint64)[None, :], (rows, blocks)),
           np.broadcast_to(np.arange(rows, dtype=np.uint64)[:, None], (rows, blocks)),
           np.uint64(offset & 0xFFFFFFFF), np.uint64((offset >> 32) & 0xFFFFFFFF)]
    key = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    for _ in range(10):
        one, two = ctr[0] * np.uint64(0xD2511F53), ctr[2] * np.uint64(0xCD9E8D57)
        ctr = [(two >> half) ^ ctr[1] ^ np.uint64(key[0]), two & low, (one >> half) ^ ctr[3] ^ np.uint64(key[1]),
               one & low]
        key = [(key[0] + 0x9E3779B9) & 0xFFFFFFFF, (key[1] + 0xBB67AE85) & 0xFFFFFFFF]
    words = np.empty((rows, blocks, 8), dtype=np.uint16)
    for j in range(4):
        words[:, :, 2 * j] = (ctr[j] & np.uint64(0xFFFF)).astype(np.uint16)
        words[:, :, 2 * j + 1] = (ctr[j] >> np.uint64(16)).astype(np.uint16)
    least = math.floor(p * 65536 + 0.5)
    return torch.from_numpy(words.reshape(rows, -1)[:, :cols] >= least).cuda(), 65536 / (65536 - least)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    wide = lambda v: None if v is None else v.to(torch.float64)  # noqa: E731
    if op in ("norm_forward", "norm_backward", "dropout"):
        drop = lambda v: v  # noqa: E731
        if case["p"] > 0:
            keep, up = _exact_keep(case["rows"], case["cols"], case["p"], st["seed"] & (2**64 - 1), st["offset"])
            drop = lambda v: (v * up).masked_fill_(~keep, 0)  # noqa: E731
        if op == "dropout":
            return {"y": drop(wide(st["x"]))}
        w = wide(st["w"]) if st["w"] is not None else torch.ones(case["cols"], dtype=torch.float64, device="cuda")
        if op == "norm_forward":
            z = drop(wide(st["x"]))
            z = z if st["r"] is None else z + wide(st["r"])
            size = (z.square().sum(1) / case["cols"] + EPS).sqrt()
            y = z / size[:, None] * w
            out = {"rstd": 1 / size, "h": z if st["h"] is not None else None, "y": y}
            if st["scales"] is not None:
                g = case["group"] or case["cols"]
                n = -(-case["cols"] // g)
                most = torch.zeros(case["rows"], n * g, dtype=torch.float64, device="cuda")
                most[:, : case["cols"]] = y.abs()
                out["scales"] = most.reshape(case["rows"], n, g).amax(2) / LARGEST[case["out"]]
                out["y"] = y / out["scales"].repeat_interleave(g, 1)[:, : case["cols"]]
            return out
        h, dy, r = wide(st["h"]), wide(st["dy"]), wide(st["rstd"])[:, None]
        dot = (dy * w * h).sum(1, keepdim=True) / case["cols"]
        dz = r * dy * w - h * r**3 * dot
        dz = dz if st["dh"] is None else dz + wide(st["dh"])
        return {"dr": dz, "dx": drop(dz.clone()) if st["dx"] is not None else None,
                "dw": (dy * (h * r)).sum(0) if st["dw"] is not None else None}
    if op == "route_order":
        idx = st["idx"].cpu().numpy().reshape(-1)
        counts = np.bincount(idx[idx >= 0], minlength=case["experts"]).astype(np.int64)
        step = np.sign(counts.sum() - counts * case["experts"])
        return {"counts": None, "offsets": None, "order": None, "position": None,
                "new_bias": st["bias"].cpu().numpy().astype(np.float64) + RATE * step}
    l = st["logits"].double().cpu().numpy()
    t, e, k = case["rows"], case["experts"], case["k"]
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        if case["score"] == "sigmoid":
            s = 1 / (1 + np.exp(-l))
        else:
            s = np.exp(l - l.max(1, keepdims=True))
            s = s / s.sum(1, keepdims=True)
    if op == "route_forward":
        shut = np.isneginf(l)
        s = np.where(shut, 0, s)
        bias = st["bias"].double().cpu().numpy() if st["bias"] is not None else np.zeros(e)
        order_by = np.where(shut, -np.inf, s + bias if st["bias"] is not None else l)
        n = case["groups"]
        if n > 1:
            two = -np.sort(-np.where(shut, -np.inf, s + bias).reshape(t, n, -1), axis=2)[:, :, :2]
            of = np.where(np.isneginf(two), 0, two).sum(2)
            of[np.isneginf(two[:, :, 0])] = -np.inf
            left_out = np.argsort(-of, axis=1, kind="stable")[:, case["top_groups"]:]
            hidden = np.zeros((t, n), dtype=bool)
            np.put_along_axis(hidden, left_out, True, 1)
            order_by = np.where(np.repeat(hidden, e // n, axis=1), -np.inf, order_by)
        idx = np.argsort(-order_by, axis=1, kind="stable")[:, :k]
        fine = ~np.isneginf(np.take_along_axis(order_by, idx, 1))
        if st["keep"] is not None:
            live = st["keep"].cpu().numpy()[:, None]
            fine, s = fine & live, np.where(live, s, 0)
        w = np.where(fine, np.take_along_axis(s, idx, 1), 0)
        if case["renormalise"]:
            total = w.sum(1, keepdims=True)
            w = w / np.where(total > 0, total, 1)
        return {"idx": None, "weights": 2.5 * w, "scores": s if st["scores"] is not None else None}
    # d loss / d score of the loss sum(weights dweights) + sum(scores dscores), then through the scores
    idx = st["idx"].cpu().numpy().astype(np.int64)
    fine, at = idx >= 0, np.maximum(idx, 0)
    g = np.where(fine, st["dweights"].double().cpu().numpy(), 0)
    w = st["weights"].double().cpu().numpy() / 2.5
    chosen = np.where(fine, np.take_along_axis(s, at, 1), 1)
    if case["renormalise"]:   # weights = 2.5 s / total with total = s / w
        by = 2.5 * (g - (g * w).sum(1, keepdims=True)) * np.where(fine, w / chosen, 0)
    else:
        by = 2.5 * g
    ds = np.zeros((t, e))
    np.add.at(ds, (np.arange(t)[:, None], at), np.where(fine, by, 0))
    if st["dscores"] is not None:
        ds = ds + st["dscores"].double().cpu().numpy()
    d = s * (1 - s) * ds if case["score"] == "sigmoid" else s * (ds - (s * ds).sum(1, keepdims=True))
    return {"dlogits": np.where(fine[:, :1], d, 0)}
