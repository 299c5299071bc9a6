"""Cases of the operators that routed pairs go through between the router and the residual stream: rows
gathered into the experts' order and combined back (with the gradient), the gated activation (forward,
backward), weights quantised in blocks of 128 x 128, the experts' 8-bit product with a scale for each block
of 128, and the gradient of the experts' weights.

``run`` computes a case in elementary torch operations, or through matrix_optimizer_amd.experts where
``own`` is true; ``exact`` gives the floating outputs in 64 bits.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
BYTES = {"f32": 4, "bf16": 2, "e4m3": 1, "e5m2": 1}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
LEAST = 2.0**-126    # of a scale
BLOCK = 128


def listed():
    return [
        # a training step's normed rows, in 8 bits with their scales, to the experts that they were routed to
        dict(name="gather_train_e4m3", op="gather", rows=8192, k=6, experts=64, cols=7168, type="e4m3", padding=0.03),
        # a served batch's results back to their rows, onto the residual stream: latency alone
        dict(name="combine_served", op="combine", rows=16, k=6, experts=64, cols=7168, type="bf16", out="bf16",
             weights=True, base=True, padding=0.0),
        # a training step's gradient of the same: rows for both products behind it, and the routing weights'
        dict(name="combine_train_backward", op="combine_backward", rows=8192, k=6, experts=64, cols=7168, type="bf16",
             eight="e4m3", padding=0.03),
        # the activation between a training step's two products, kept for the backward pass and in 8 bits
        dict(name="gate_train", op="gate", rows=49152, cols=2048, type="bf16", eight="e4m3", tail=0.03),
        # its gradient in the check precision at an odd width
        dict(name="gate_odd_backward", op="gate_backward", rows=2001, cols=1371, type="f32", eight="none", tail=0.03),
        # an owner's expert matrices after their update, in 8 bits for the forward and the backward product
        dict(name="quantise_experts", op="quantise", batch=16, rows=2048, cols=7168, type="bf16", eight="e4m3", both=True),
        # matrices of odd sizes in the check precision: blocks that end early in both directions
        dict(name="quantise_odd", op="quantise", batch=3, rows=1001, cols=777, type="f32", eight="e5m2", both=False),
        # a served batch: one or two rows an expert, the weights' bytes are what counts
        dict(name="product_served", op="product", rows=96, experts=64, active=50, n=4096, k=7168, a="e4m3", w="e4m3",
             out="bf16", tail=0.0),
        # a training step's gate and up product
        dict(name="product_train", op="product", rows=49152, experts=64, active=64, n=4096, k=7168, a="e4m3", w="e4m3",
             out="bf16", tail=0.03),
        # an input gradient of odd widths and ragged groups, some of them empty
        dict(name="product_odd_gradient", op="product", rows=3001, experts=16, active=13, n=1371, k=2051, a="e5m2",
             w="e4m3", out="f32", tail=0.03),
        # the down projections' gradient for the optimizer
        dict(name="weight_grad_train", op="weight_grad", rows=49152, experts=64, active=64, n=7168, k=2048, out="bf16",
             tail=0.03),
        # odd widths, experts without rows
        dict(name="weight_grad_odd", op="weight_grad", rows=777, experts=8, active=6, n=1001, k=515, out="f32",
             tail=0.03),
    ]


def _spread(rng, lo, hi):
    """A size between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    n = _spread(rng, lo, hi)
    return n if rng.random() < 0.3 else max(lo, n // 128 * 128)


def draw(rng):
    op = rng.choice(["gather", "combine", "combine", "combine_backward", "gate", "gate_backward", "quantise", "product",
                     "product", "product", "weight_grad", "weight_grad"])
    if op in ("gather", "combine", "combine_backward"):
        experts = rng.choice([8, 16, 64, 128, 256])
        k = rng.randint(1, 8)
        cols = _width(rng, 64, 8192)
        rows = min(_spread(rng, 1, 16384), 350_000_000 // (k * cols))
        case = dict(op=op, rows=rows, k=k, experts=experts, cols=cols, padding=rng.choice([0.0, 0.05]))
        if op == "gather":
            return dict(case, type=rng.choice(["e4m3", "e5m2", "bf16", "bf16"]))
        case["type"] = rng.choice(["bf16", "bf16", "f32"])
        if op == "combine":
            return dict(case, out=rng.choice([case["type"], "f32"]), weights=rng.random() < 0.7, base=rng.random() < 0.5)
        return dict(case, eight=rng.choice(["none", "e4m3", "e5m2"]))
    tail = rng.choice([0.0, 0.05])
    if op in ("gate", "gate_backward"):
        cols = _width(rng, 128, 14336)
        case = dict(op=op, rows=min(_spread(rng, 1, 65536), 100_000_000 // cols), cols=cols,
                    type=rng.choice(["bf16", "bf16", "f32"]), tail=tail)
        whole = op == "gate" or cols % BLOCK == 0
        return dict(case, eight=rng.choice(["none", "e4m3", "e5m2"]) if whole else "none")
    if op == "quantise":
        rows, cols = _width(rng, 64, 8192), _width(rng, 64, 8192)
        return dict(op=op, batch=min(_spread(rng, 1, 64), max(1, 230_000_000 // (rows * cols))), rows=rows, cols=cols,
                    type=rng.choice(["bf16", "bf16", "f32"]), eight=rng.choice(["e4m3", "e4m3", "e5m2"]),
                    both=rng.random() < 0.6)
    experts = rng.choice([1, 4, 8, 16, 32, 64, 128])
    rows = _spread(rng, 1, 49152)
    most = min(experts, _rows_used(dict(rows=rows, tail=tail)))
    active = rng.randint((most + 1) // 2, most)
    n, k = _width(rng, 64, 8192), _width(rng, 64, 8192)
    largest = 1_800_000_000 if op == "product" else 600_000_000
    while experts * n * k > largest or rows * n * k > 1.4e12:
        n, k = max(64, n // 2), max(64, k // 2)
    case = dict(op=op, rows=rows, experts=experts, active=active, n=n, k=k, out=rng.choice(["bf16", "bf16", "f32"]),
                tail=tail)
    if op == "product":
        case.update(a=rng.choice(["e4m3", "e4m3", "e5m2"]), w="e4m3")
    return case


# ---- inputs -----------------------------------------------------------------

def _normal(gen, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def _routed(gen, case):
    """What the router and the pairs' order give: order [pairs], position [rows, k], weights [rows, k]."""
    t, e, k = case["rows"], case["experts"], case["k"]
    l = torch.randn(t, e, generator=gen, device="cuda") + torch.randn(e, generator=gen, device="cuda") * 0.7
    top = torch.topk(l, k, dim=1)
    weights = torch.softmax(top.values, 1)
    idx = top.indices
    pad = torch.rand(t, generator=gen, device="cuda") < case["padding"]
    idx[pad] = e
    weights[pad] = 0
    flat = idx.reshape(-1)
    got = torch.sort(flat, stable=True)
    places = torch.arange(t * k, device="cuda")
    used = got.values < e
    order = torch.where(used, got.indices, -1).to(torch.int32)
    position = torch.empty_like(places).scatter_(0, got.indices, torch.where(used, places, -1))
    return order, position.to(torch.int32).reshape(t, k), weights


def _rows_used(case):
    return case["rows"] - int(case["rows"] * case["tail"])


def _groups(gen, case):
    """Offsets of the experts' rows: `active` experts with one row at least, some of them busier."""
    e, active, total = case["experts"], case["active"], _rows_used(case)
    which = torch.randperm(e, generator=gen, device="cuda")[:active]
    p = torch.exp(0.7 * torch.randn(active, generator=gen, device="cuda"))
    # the rows after each expert's first one, cut at random places
    cut = torch.floor(torch.cumsum(p / p.sum(), 0) * (total - active) + 0.5).long()
    cut[-1] = total - active
    counts = torch.zeros(e, dtype=torch.int64, device="cuda")
    counts[which] = 1 + torch.diff(cut, prepend=torch.zeros(1, dtype=torch.int64, device="cuda"))
    offsets = torch.zeros(e + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    return offsets.to(torch.int32), offsets.tolist()


def _scales(most, kind):
    """most / LARGEST, an fp32 quotient (a division by a plain number would multiply by its reciprocal)."""
    return torch.where(most > 0, torch.clamp(most / torch.full_like(most, LARGEST[kind]), min=LEAST), 1.0)


def _eight_rows(x, kind):
    """Rows in 8 bits, a scale for each 128 columns."""
    rows, cols = x.shape
    n = -(-cols // BLOCK)
    parts = torch.nn.functional.pad(x, (0, n * BLOCK - cols)).reshape(rows, n, BLOCK)
    most = parts.abs().amax(2)
    scales = _scales(most, kind)
    q = torch.clamp(parts / scales[:, :, None], -LARGEST[kind], LARGEST[kind]).reshape(rows, n * BLOCK)[:, :cols]
    return q.to(TYPES[kind]).contiguous(), scales


def _eight_blocks(x, kind):
    """A matrix in 8 bits, a scale for each 128 x 128 block."""
    rows, cols = x.shape
    m, n = -(-rows // BLOCK), -(-cols // BLOCK)
    parts = torch.nn.functional.pad(x, (0, n * BLOCK - cols, 0, m * BLOCK - rows)).reshape(m, BLOCK, n, BLOCK)
    most = parts.abs().amax(3).amax(1)
    scales = _scales(most, kind)
    q = torch.clamp(parts / scales[:, None, :, None], -LARGEST[kind], LARGEST[kind])
    return q.reshape(m * BLOCK, n * BLOCK)[:rows, :cols].to(TYPES[kind]).contiguous(), scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dev, op = "cuda", case["op"]
    st = {"case": case}
    if op in ("gather", "combine", "combine_backward"):
        t, k, h = case["rows"], case["k"], case["cols"]
        p, n = t * k, -(-h // BLOCK)
        st["order"], st["position"], st["weights"] = _routed(gen, case)
        if op == "gather":
            x = _normal(gen, t, h)
            if case["type"] in LARGEST:
                st["x"], st["x_scales"] = _eight_rows(x, case["type"])
                st["out_scales"] = torch.zeros(p, n, device=dev)
            else:
                st["x"], st["x_scales"], st["out_scales"] = x.to(TYPES[case["type"]]), None, None
            st["out"] = torch.zeros(p, h, device=dev).to(TYPES[case["type"]])
            return st
        dt = TYPES[case["type"]]
        st["y"] = _normal(gen, p, h, dtype=dt)
        if op == "combine":
            if not case["weights"]:
                st["weights"] = None
            st["base"] = _normal(gen, t, h, scale=2.0, dtype=TYPES[case["out"]]) if case["base"] else None
            st["out"] = torch.empty(t, h, dtype=TYPES[case["out"]], device=dev)
            return st
        st["dout"] = _normal(gen, t, h, scale=1e-2, dtype=dt)
        st["dy"] = torch.zeros(p, h, dtype=dt, device=dev)
        st["dweights"] = torch.empty(t, k, device=dev)
        st["dy8"], st["scales"] = None, None
        if case["eight"] in LARGEST:
            st["dy8"], st["scales"] = torch.zeros(p, h, device=dev).to(TYPES[case["eight"]]), torch.zeros(p, n, device=dev)
        return st
    if op in ("gate", "gate_backward"):
        p, f, dt = case["rows"], case["cols"], TYPES[case["type"]]
        st["used"] = torch.tensor([_rows_used(case)], dtype=torch.int32, device=dev)
        st["a"] = _normal(gen, p, 2 * f, scale=1.5, dtype=dt)
        width = f
        if op == "gate":
            st["y"] = torch.zeros(p, f, dtype=dt, device=dev)
        else:
            width = 2 * f
            st["dy"] = _normal(gen, p, f, scale=1e-2, dtype=dt)
            st["da"] = torch.zeros(p, 2 * f, dtype=dt, device=dev)
        st["eight"], st["scales"] = None, None
        if case["eight"] in LARGEST:
            st["eight"] = torch.zeros(p, width, device=dev).to(TYPES[case["eight"]])
            st["scales"] = torch.zeros(p, -(-width // BLOCK), device=dev)
        return st
    if op == "quantise":
        b, m, n = case["batch"], case["rows"], case["cols"]
        kind = TYPES[case["eight"]]
        st["x"] = _normal(gen, b, m, n, scale=0.02, dtype=TYPES[case["type"]])
        mb, nb = -(-m // BLOCK), -(-n // BLOCK)
        st["q"], st["scales"] = torch.empty(b, m, n, dtype=kind, device=dev), torch.empty(b, mb, nb, device=dev)
        st["qt"], st["scales_t"] = None, None
        if case["both"]:
            st["qt"], st["scales_t"] = torch.empty(b, n, m, dtype=kind, device=dev), torch.empty(b, nb, mb, device=dev)
        return st
    p, e, n, k = case["rows"], case["experts"], case["n"], case["k"]
    st["offsets"], st["bounds"] = _groups(gen, case)
    if op == "product":
        st["a"], st["a_scales"] = _eight_rows(_normal(gen, p, k), case["a"])
        st["w"] = torch.empty(e, n, k, dtype=TYPES[case["w"]], device=dev)
        st["w_scales"] = torch.empty(e, -(-n // BLOCK), -(-k // BLOCK), device=dev)
        for i in range(e):
            st["w"][i], st["w_scales"][i] = _eight_blocks(_normal(gen, n, k, scale=0.02), case["w"])
        st["out"] = torch.zeros(p, n, dtype=TYPES[case["out"]], device=dev)
        return st
    st["dy"] = _normal(gen, p, n, scale=1e-2, dtype=torch.bfloat16)
    st["x"] = _normal(gen, p, k, dtype=torch.bfloat16)
    st["dw"] = torch.empty(e, n, k, dtype=TYPES[case["out"]], device=dev)
    return st


# ---- the plain forms --------------------------------------------------------

def _plain_gather(case, st):
    order = st["order"].long()
    used = (order >= 0)[:, None]
    at = order.clamp(min=0) // case["k"]
    out = {"out": torch.where(used, st["x"].float()[at], 0.0).to(st["x"].dtype), "scales": None}
    if st["x_scales"] is not None:
        out["scales"] = torch.where(used, st["x_scales"][at], 0.0)
    return out


def _plain_combine(case, st):
    position = st["position"].long()
    total = st["base"].float() if st["base"] is not None else torch.zeros(case["rows"], case["cols"], device="cuda")
    for j in range(case["k"]):
        at = position[:, j]
        term = st["y"][at.clamp(min=0)].float()
        if st["weights"] is not None:
            term = term * st["weights"][:, j, None]
        total = total + torch.where((at >= 0)[:, None], term, 0.0)
    return {"out": total.to(TYPES[case["out"]])}


def _plain_eight(v, used, kind):
    """Rows of fp32 values in 8 bits with their scales; zeros where not used."""
    q, scales = _eight_rows(v, kind)
    return torch.where(used, q.float(), 0.0).to(q.dtype), torch.where(used, scales, 0.0)


def _plain_combine_backward(case, st):
    order, position = st["order"].long(), st["position"].long()
    dout = st["dout"].float()
    used = (order >= 0)[:, None]
    pair = order.clamp(min=0)
    v = st["weights"].reshape(-1)[pair][:, None] * dout[pair // case["k"]]
    out = {"dy": torch.where(used, v, 0.0).to(st["dout"].dtype), "dy8": None, "scales": None}
    if st["dy8"] is not None:
        out["dy8"], out["scales"] = _plain_eight(v, used, case["eight"])
    dots = [(dout * st["y"][position[:, j].clamp(min=0)].float()).sum(1) for j in range(case["k"])]
    out["dweights"] = torch.where(position >= 0, torch.stack(dots, 1), 0.0)
    return out


def _plain_gate(case, st):
    f = case["cols"]
    g, u = st["a"][:, :f].float(), st["a"][:, f:].float()
    v = g / (1 + torch.exp(-g)) * u
    used = (torch.arange(case["rows"], device="cuda") < st["used"])[:, None]
    out = {"y": torch.where(used, v, 0.0).to(st["a"].dtype), "eight": None, "scales": None}
    if st["eight"] is not None:
        out["eight"], out["scales"] = _plain_eight(v, used, case["eight"])
    return out


def _plain_gate_backward(case, st):
    f = case["cols"]
    g, u, dy = st["a"][:, :f].float(), st["a"][:, f:].float(), st["dy"].float()
    s = 1 / (1 + torch.exp(-g))
    v = torch.cat((dy * u * s * (1 + g * (1 - s)), dy * g * s), 1)
    used = (torch.arange(case["rows"], device="cuda") < st["used"])[:, None]
    out = {"da": torch.where(used, v, 0.0).to(st["a"].dtype), "eight": None, "scales": None}
    if st["eight"] is not None:
        out["eight"], out["scales"] = _plain_eight(v, used, case["eight"])
    return out


def _plain_quantise(case, st):
    b, m, n = case["batch"], case["rows"], case["cols"]
    mb, nb = -(-m // BLOCK), -(-n // BLOCK)
    x = torch.nn.functional.pad(st["x"].float(), (0, nb * BLOCK - n, 0, mb * BLOCK - m)).reshape(b, mb, BLOCK, nb, BLOCK)
    top = LARGEST[case["eight"]]
    most = x.abs().amax(4).amax(2)
    scales = _scales(most, case["eight"])
    q = torch.clamp(x / scales[:, :, None, :, None], -top, top).reshape(b, mb * BLOCK, nb * BLOCK)[:, :m, :n]
    q = q.to(TYPES[case["eight"]])
    both = st["qt"] is not None
    return {"q": q.contiguous(), "scales": scales, "qt": q.transpose(1, 2).contiguous() if both else None,
            "scales_t": scales.transpose(1, 2).contiguous() if both else None}


def _plain_product(case, st):
    p, n, k = case["rows"], case["n"], case["k"]
    rows = st["a"].float() * st["a_scales"].repeat_interleave(BLOCK, 1)[:, :k]
    out = torch.zeros(p, n, dtype=TYPES[case["out"]], device="cuda")
    for e in range(case["experts"]):
        lo, hi = st["bounds"][e], st["bounds"][e + 1]
        if lo == hi:
            continue
        s = st["w_scales"][e].repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]
        out[lo:hi] = (rows[lo:hi] @ (st["w"][e].float() * s).t()).to(out.dtype)
    return {"out": out}


def _plain_weight_grad(case, st):
    out = torch.empty_like(st["dw"])
    for e in range(case["experts"]):
        lo, hi = st["bounds"][e], st["bounds"][e + 1]
        if lo == hi:
            out[e] = 0
        else:
            out[e] = (st["dy"][lo:hi].float().t() @ st["x"][lo:hi].float()).to(out.dtype)
    return {"dw": out}


# ---- the framework's operators ----------------------------------------------

def _own_gather(X, case, st):
    X.muon_expert_gather(st["order"], st["x"], st["out"], scales=st["x_scales"], out_scales=st["out_scales"])
    return {"out": st["out"], "scales": st["out_scales"]}


def _own_combine(X, case, st):
    X.muon_expert_combine(st["position"], st["y"], st["out"], weights=st["weights"], base=st["base"])
    return {"out": st["out"]}


def _own_combine_backward(X, case, st):
    X.muon_expert_combine_backward(st["position"], st["dout"], y=st["y"], weights=st["weights"], dy=st["dy"],
                                   dweights=st["dweights"], dy8=st["dy8"], scales=st["scales"])
    return {"dy": st["dy"], "dy8": st["dy8"], "scales": st["scales"], "dweights": st["dweights"]}


def _own_gate(X, case, st):
    X.muon_gate_forward(st["a"], y=st["y"], y8=st["eight"], scales=st["scales"], used=st["used"])
    return {"y": st["y"], "eight": st["eight"], "scales": st["scales"]}


def _own_gate_backward(X, case, st):
    X.muon_gate_backward(st["a"], st["dy"], da=st["da"], da8=st["eight"], scales=st["scales"], used=st["used"])
    return {"da": st["da"], "eight": st["eight"], "scales": st["scales"]}


def _own_quantise(X, case, st):
    X.muon_quantise_blocks(st["x"], st["q"], st["scales"], qt=st["qt"], scales_t=st["scales_t"])
    return {"q": st["q"], "scales": st["scales"], "qt": st["qt"], "scales_t": st["scales_t"]}


def _own_product(X, case, st):
    X.muon_expert_product(st["a"], st["a_scales"], st["w"], st["w_scales"], st["out"], offsets=st["offsets"])
    return {"out": st["out"]}


def _own_weight_grad(X, case, st):
    if "room" not in st:   # a workspace, kept beside the buffers that it serves
        need = X.expert_weight_grad_workspace_bytes(case["rows"], case["experts"], case["n"], case["k"])
        st["room"] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    X.muon_expert_weight_grad(st["dy"], st["x"], st["dw"], offsets=st["offsets"], workspace=st["room"])
    return {"dw": st["dw"]}


def run(state):
    case = state["case"]
    if own:
        from matrix_optimizer_amd import experts as X
        return {"gather": _own_gather, "combine": _own_combine, "combine_backward": _own_combine_backward,
                "gate": _own_gate, "gate_backward": _own_gate_backward, "quantise": _own_quantise,
                "product": _own_product, "weight_grad": _own_weight_grad}[case["op"]](X, case, state)
    return {"gather": _plain_gather, "combine": _plain_combine, "combine_backward": _plain_combine_backward,
            "gate": _plain_gate, "gate_backward": _plain_gate_backward, "quantise": _plain_quantise,
            "product": _plain_product, "weight_grad": _plain_weight_grad}[case["op"]](case, state)


def work(case):
    op = case["op"]
    if op in ("gather", "combine", "combine_backward"):
        t, k, h, b = case["rows"], case["k"], case["cols"], BYTES[case["type"]]
        n = -(-h // BLOCK)
        if op == "gather":
            row = h * b + (4 * n if case["type"] in LARGEST else 0)
            return {"bytes": (t + t * k) * row + 4 * t * k, "flops": t * k * h}
        if op == "combine":
            return {"bytes": t * k * h * b + t * h * BYTES[case["out"]] * (1 + case["base"]) + 4 * t * k
                    + (4 * t * k if case["weights"] else 0), "flops": 2 * t * k * h}
        eight = h + 4 * n if case["eight"] in LARGEST else 0
        return {"bytes": t * h * b + t * k * (2 * h * b + eight) + 12 * t * k, "flops": 3 * t * k * h}
    if op in ("gate", "gate_backward"):
        p, f, b = _rows_used(case), case["cols"], BYTES[case["type"]]
        width = f if op == "gate" else 2 * f
        eight = width + 4 * -(-width // BLOCK) if case["eight"] in LARGEST else 0
        return {"bytes": p * (2 * f * b + (f if op == "gate" else 3 * f) * b + eight), "flops": 8 * p * f}
    if op == "quantise":
        m, n = case["rows"], case["cols"]
        blocks = -(-m // BLOCK) * -(-n // BLOCK)
        return {"bytes": case["batch"] * (m * n * BYTES[case["type"]] + (1 + case["both"]) * (m * n + 4 * blocks)),
                "flops": 2 * case["batch"] * m * n}
    p, e, n, k = _rows_used(case), case["experts"], case["n"], case["k"]
    if op == "product":
        nb, kb = -(-n // BLOCK), -(-k // BLOCK)
        return {"bytes": p * (k + 4 * kb) + case["active"] * (n * k + 4 * nb * kb) + p * n * BYTES[case["out"]] + 4 * e,
                "flops": 2 * p * n * k}
    return {"bytes": 2 * p * (n + k) + e * n * k * BYTES[case["out"]] + 4 * e, "flops": 2 * p * n * k}


# ---- the definitions in 64 bits ---------------------------------------------

def _wide(v):
    return v.to(torch.float64)


def _narrow(v):
    return v.to(torch.float32)


def _exact_rounded(v, kind):
    """The nearest values of an 8-bit format with `digits` fraction bits and exponents from `low` on, ties to even."""
    digits, low = (3, -6) if kind == "e4m3" else (2, -14)
    step = torch.exp2(torch.frexp(v).exponent.double().sub_(1).clamp_(min=low).sub_(digits))
    return torch.round(v / step).mul_(step).clamp_(-LARGEST[kind], LARGEST[kind])


def _exact_scaled(v, kind):
    """v / scale as stored and the scale, a group of 128 columns at a time."""
    q, scales = torch.empty_like(v), []
    for c in range(0, v.shape[1], BLOCK):
        most = v[:, c:c + BLOCK].abs().max(1).values
        s = _wide(_narrow((most / LARGEST[kind]).clamp_min(LEAST)))   # a scale is held in 32 bits
        s = torch.where(most == 0, torch.ones_like(s), s)
        q[:, c:c + BLOCK] = v[:, c:c + BLOCK] / s[:, None]
        scales.append(s)
    return _exact_rounded(q, kind), torch.stack(scales, 1)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("gather", "combine", "combine_backward"):
        t, k, h = case["rows"], case["k"], case["cols"]
        # the pairs that have a place, by their slots
        slot = torch.nonzero(st["position"].reshape(-1) >= 0).squeeze(1)
        place, row = st["position"].reshape(-1)[slot].long(), slot // k
        empty = lambda *s: torch.zeros(*s, dtype=torch.float64, device="cuda")  # noqa: E731
        if op == "gather":
            out = empty(t * k, h)
            out[place] = _wide(st["x"])[row]
            scales = None
            if st["x_scales"] is not None:
                scales = empty(t * k, st["x_scales"].shape[1])
                scales[place] = _wide(st["x_scales"])[row]
            return {"out": out, "scales": scales}
        if op == "combine":
            out = _wide(st["base"]).clone() if st["base"] is not None else empty(t, h)
            w = _wide(st["weights"]).reshape(-1)[slot] if st["weights"] is not None else torch.ones_like(_wide(slot))
            out.index_add_(0, row, _wide(st["y"])[place] * w[:, None])
            return {"out": out}
        d = _wide(st["dout"])[row]
        dw = empty(t * k)
        dw[slot] = (d * _wide(st["y"])[place]).sum(1)
        d *= _wide(st["weights"]).reshape(-1)[slot][:, None]
        out = {"dy": empty(t * k, h), "dy8": None, "scales": None, "dweights": dw.reshape(t, k)}
        out["dy"][place] = d
        if st["dy8"] is not None:
            out["dy8"], out["scales"] = empty(t * k, h), empty(t * k, st["scales"].shape[1])
            out["dy8"][place], out["scales"][place] = _exact_scaled(d, case["eight"])
        return out
    if op in ("gate", "gate_backward"):
        f, used = case["cols"], _rows_used(case)
        g, u = _wide(st["a"][:, :f]), _wide(st["a"][:, f:])
        s = torch.sigmoid(g)
        if op == "gate":
            v, name = g * s * u, "y"
        else:
            dy, name = _wide(st["dy"]), "da"
            v = torch.empty(case["rows"], 2 * f, dtype=torch.float64, device="cuda")
            v[:, :f] = dy * u * (s + g * s * torch.sigmoid(-g))
            v[:, f:] = dy * (g * s)
        v[used:] = 0
        out = {name: v, "eight": None, "scales": None}
        if st["eight"] is not None:
            out["eight"], out["scales"] = _exact_scaled(v, case["eight"])
            out["scales"][used:] = 0
        return out
    if op == "quantise":
        b, m, n = case["batch"], case["rows"], case["cols"]
        mb, nb = -(-m // BLOCK), -(-n // BLOCK)
        q, scales = _wide(st["x"]), torch.empty(b, mb, nb, dtype=torch.float64, device="cuda")
        for i in range(mb):
            for j in range(nb):
                part = q[:, i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK]
                most = part.abs().amax((1, 2))
                s = _wide(_narrow((most / LARGEST[case["eight"]]).clamp_min(LEAST).masked_fill(most == 0, 1)))
                part /= s[:, None, None]
                scales[:, i, j] = s
        for i in range(b):
            q[i] = _exact_rounded(q[i], case["eight"])
        both = case["both"]
        return {"q": q, "scales": scales, "qt": q.mT.contiguous() if both else None,
                "scales_t": scales.mT.contiguous() if both else None}
    if op == "product":
        out = torch.zeros(case["rows"], case["n"], dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            rows = slice(st["bounds"][e], st["bounds"][e + 1])
            if rows.start == rows.stop:
                continue
            a, w = _wide(st["a"][rows]), _wide(st["w"][e])
            for j, c in enumerate(range(0, case["k"], BLOCK)):
                a[:, c:c + BLOCK] *= _wide(st["a_scales"][rows, j])[:, None]
                for i, r in enumerate(range(0, case["n"], BLOCK)):
                    w[r:r + BLOCK, c:c + BLOCK] *= _wide(st["w_scales"][e, i, j])
            out[rows] = a @ w.mT
        return {"out": out}
    dw = torch.zeros(case["experts"], case["n"], case["k"], dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        rows = slice(st["bounds"][e], st["bounds"][e + 1])
        if rows.start < rows.stop:
            dw[e] = _wide(st["dy"][rows]).mT @ _wide(st["x"][rows])
    return {"dw": dw}
