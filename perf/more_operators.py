"""Cases of the routing to experts and of the experts' BF16 product (bias, activation, residual), forward and backward.

`own` False: plain torch in 32 bits (the order of choices in 64, since whole numbers come of it); True: the
library's calls on the same state.  `exact` gives the definition's values in 64 bits.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # one small batch of the smallest routing shape: launches are the cost
        dict(name="route_tiny", op="route", n=128, e=16, k=4, groups=4, keep=2, by="max", score="softmax", bias=False, renorm=True,
             dtype="f32", mask=0.0, train=False),
        # a decode batch, plain top-8 of 256 with a bias for balance
        dict(name="route_decode", op="route", n=128, e=256, k=8, groups=1, keep=1, by="max", score="sigmoid", bias=True, renorm=True,
             dtype="f32", mask=0.0, train=False),
        # a prefill batch: top-4 of 8 groups, top-8 of 256 experts, a few experts out of service, padded rows
        dict(name="route_prefill", op="route", n=4096, e=256, k=8, groups=8, keep=4, by="top2", score="sigmoid", bias=True, renorm=True,
             dtype="f32", mask=0.05, train=False),
        # the skewed batch in training: choices, weights and the gradient of the logits
        dict(name="route_skewed_train", op="route", n=16384, e=256, k=8, groups=8, keep=4, by="max", score="sigmoid", bias=False,
             renorm=True, dtype="f32", mask=0.0, train=True),
        # a training step's tokens, weights as the softmax gives them, so that every logit has a gradient
        dict(name="route_train", op="route", n=65536, e=256, k=8, groups=1, keep=1, by="max", score="softmax", bias=False, renorm=False,
             dtype="bf16", mask=0.0, train=True),
        # the smallest routing shape's product
        dict(name="product_tiny", op="product", rows=512, e=16, k=256, f=512, act="relu", bias=True, residual=False, zipf=0.0,
             padded=False, train=False),
        # one token through one dense layer and onto the residual stream
        dict(name="product_one_token", op="product", rows=1, e=1, k=7168, f=4096, act="none", bias=True, residual=True, zipf=0.0,
             padded=False, train=False),
        # a decode batch through all experts' gated first layer: the weights' bytes are the cost
        dict(name="product_decode", op="product", rows=1024, e=256, k=7168, f=4096, act="swiglu", bias=False, residual=False, zipf=0.0,
             padded=True, train=False),
        # a prefill batch through all experts' gated first layer
        dict(name="product_prefill", op="product", rows=32768, e=256, k=7168, f=4096, act="swiglu", bias=False, residual=False, zipf=0.0,
             padded=False, train=False),
        # a large batch with a skewed expert load through the experts' second layer
        dict(name="product_skewed", op="product", rows=131072, e=256, k=2048, f=7168, act="none", bias=True, residual=False, zipf=1.1,
             padded=False, train=False),
        # training: the gated first layer of the experts that one GPU holds, forward and backward
        dict(name="product_train", op="product", rows=32768, e=32, k=7168, f=4096, act="swiglu", bias=False, residual=False, zipf=1.1,
             padded=False, train=True),
        # training: a dense layer (an expert that every token passes) with all of the epilogue, forward and backward
        dict(name="product_dense_train", op="product", rows=8192, e=1, k=2048, f=7168, act="gelu", bias=True, residual=True, zipf=0.0,
             padded=False, train=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    if rng.random() < 0.45:
        e = _log(rng, 1, 512)
        groups = rng.choice([1] + [g for g in range(1, min(e, 32) + 1) if e % g == 0])
        return dict(op="route", n=_log(rng, 1, min(65536, 16777216 // e)), e=e, k=rng.randint(1, min(e, 16)), groups=groups,
                    keep=rng.randint((groups + 1) // 2, groups), by=rng.choice(["max", "top2"]), score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, renorm=rng.random() < 0.6, dtype=rng.choice(["f32", "bf16", "f16"]),
                    mask=rng.choice([0.0, 0.05, 0.5]), train=rng.random() < 0.5)
    train = rng.random() < 0.4
    act = rng.choice(["none", "relu", "gelu", "silu", "swiglu", "swiglu"])
    k = 8 * _log(rng, 1, 896)
    f = _log(rng, 1, 7168)
    if act == "swiglu":
        f = 2 * -(-f // 2)
    e = _log(rng, 1, min(256, (32 if train else 256) * 4096 * 7168 // (f * k)))
    most = int(1.9e12 / (2 * f * k)) if train else int(3.8e12 / (2 * f * k))
    return dict(op="product", rows=_log(rng, 1, max(1, min(most, 131072 if k <= 2048 else 32768))), e=e, k=k, f=f, act=act,
                bias=rng.random() < 0.5, residual=rng.random() < 0.3, zipf=rng.choice([0.0, 1.1]), padded=rng.random() < 0.3, train=train)


# ---- plain forms -------------------------------------------------------------------------------


def _route(st):
    c, x = st["case"], st["logits"]
    n, e, k, groups = c["n"], c["e"], c["k"], c["groups"]
    wide = x.double()                                      # neighbours in the order may be nearer than 32 bits tell
    dead = torch.isneginf(wide)
    if c["score"] == "softmax":
        s = torch.exp(wide - wide.amax(dim=1, keepdim=True).clamp(min=-1e300))
        s = s / s.sum(dim=1, keepdim=True).clamp(min=1e-300)
    else:
        s = 1 / (1 + torch.exp(-wide))
    choice = wide if st["bias"] is None else torch.where(dead, -torch.inf, s + st["bias"].double())
    if groups > 1:
        if c["by"] == "top2":
            v = torch.where(dead, -torch.inf, s if st["bias"] is None else choice).reshape(n, groups, -1)
            top = torch.sort(v, dim=2, descending=True).values[:, :, :2]
            top[:, :, 1:] = torch.where(torch.isneginf(top[:, :, 1:]), 0, top[:, :, 1:])
            value = top.sum(dim=2)
        else:
            value = choice.reshape(n, groups, -1).amax(dim=2)
        best = torch.sort(value, dim=1, descending=True, stable=True).indices[:, : c["keep"]]
        kept = torch.zeros((n, groups), dtype=torch.bool, device=x.device).scatter_(1, best, True)
        choice = torch.where(kept.repeat_interleave(e // groups, dim=1), choice, -torch.inf)
    value, idx = torch.sort(choice, dim=1, descending=True, stable=True)
    there, idx = ~torch.isneginf(value[:, :k]), idx[:, :k]
    l = torch.where(there, x.gather(1, idx).float(), -torch.inf)
    if c["score"] == "sigmoid":
        w = 1 / (1 + torch.exp(-l))
    else:
        top = (l if c["renorm"] else x.float()).amax(dim=1, keepdim=True).clamp(min=-1e38)
        w = torch.exp(l - top)
        if not c["renorm"]:
            w = w / torch.exp(x.float() - top).sum(dim=1, keepdim=True).clamp(min=1e-30)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True).clamp(min=1e-30)
    w = w * c["scale"]
    out = {"idx": torch.where(there, idx, -1).int(), "weights": w}
    if not c["train"]:
        return out
    part = w / c["scale"]
    g = torch.where(there, st["g"], 0) * c["scale"]
    dot = (g * part).sum(dim=1, keepdim=True)
    if c["score"] == "sigmoid":
        v = part * (1 / (1 + torch.exp(l))) * (g - dot if c["renorm"] else g)
    else:
        v = part * (g - dot)
    grad = torch.zeros((n, e + 1), device=x.device)        # a column more, for slots without an expert
    if c["score"] == "softmax" and not c["renorm"]:
        p = torch.exp(x.float() - top)
        grad[:, :e] = -dot * p / p.sum(dim=1, keepdim=True).clamp(min=1e-30)
    grad.scatter_(1, torch.where(there, idx, e), v)
    return dict(out, grad=grad[:, :e].to(x.dtype))


def _activate(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "swiglu":
        gate, up = z.chunk(2, dim=1)
        return gate / (1 + torch.exp(-gate)) * up
    return z


def _slope(z, g, act):
    """The gradient of z from the activation's, g."""
    if act == "relu":
        return torch.where(z > 0, g, 0)
    if act == "gelu":
        return g * (0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return g * s * (1 + z * (1 - s))
    if act == "swiglu":
        gate, up = z.chunk(2, dim=1)
        s = 1 / (1 + torch.exp(-gate))
        return torch.cat((g * up * s * (1 + gate * (1 - s)), g * gate * s), dim=1)
    return g


def _product(st):
    """Expert by expert, since their rows are ragged."""
    c = st["case"]
    y = torch.zeros_like(st["y"])
    if c["train"]:
        da = torch.zeros_like(st["a"])
        dw = torch.zeros_like(st["w"])
        db = torch.zeros_like(st["w"][:, :, 0])
    for i, (r0, r1) in enumerate(st["spans"]):
        if r1 <= r0:
            continue
        a, w = st["a"][r0:r1].float(), st["w"][i].float()
        z = a @ w.T
        if c["bias"]:
            z = z + st["bias"][i].float()
        v = _activate(z, c["act"])
        if c["residual"]:
            v = v + st["residual"][r0:r1].float()
        y[r0:r1] = v.bfloat16()
        if c["train"]:
            dz = _slope(z, st["g"][r0:r1].float(), c["act"])
            da[r0:r1] = (dz @ w).bfloat16()
            dw[i] = (dz.T @ a).bfloat16()
            db[i] = dz.sum(dim=0).bfloat16()
    if not c["train"]:
        return y
    return {"y": y, "grad_a": da, "grad_w": dw, **({"grad_bias": db} if c["bias"] else {})}


# ---- inputs ------------------------------------------------------------------------------------


def _prepare_route(c, gen, dev):
    n, e = c["n"], c["e"]
    logits = torch.randn((n, e), generator=gen, device=dev)
    logits -= 0.3 * 1.1 * torch.log(1 + torch.randperm(e, generator=gen, device=dev).float())
    if c["mask"]:   # experts that a token may not take, and padding at the end
        logits[torch.rand((n, e), generator=gen, device=dev) < c["mask"]] = -torch.inf
        logits[n - int(0.05 * n):] = -torch.inf
    # a bias that balancing has moved in steps of a thousandth
    bias = torch.round(50 * torch.randn(e, generator=gen, device=dev)) / 1000 if c["bias"] else None
    st = dict(logits=logits.to(DTYPES[c["dtype"]]), bias=bias)
    if c["train"]:
        st["g"] = torch.randn((n, c["k"]), generator=gen, device=dev)
    return st


def _capacity(rows, e):
    """Rows a padded expert has room for, fixed before the counts are known."""
    return min(rows, 8 + 2 * -(-rows // e))


def _prepare_product(c, gen, dev):
    rows, e, k, f = c["rows"], c["e"], c["k"], c["f"]
    w = torch.ones(e, device=dev)
    if c["zipf"]:
        w = (1 + torch.randperm(e, generator=gen, device=dev).float()) ** (-0.3 * c["zipf"])
    ids = torch.multinomial(w, rows, replacement=True, generator=gen)
    count = torch.bincount(ids, minlength=e)
    off = torch.zeros(e + 1, dtype=torch.int32, device=dev)
    off[1:] = count.cumsum(0)
    count, ends, cap = count.tolist(), off.tolist(), 0
    spans = [(ends[i], ends[i + 1]) for i in range(e)]
    if c["padded"]:
        cap = _capacity(rows, e)
        spans = [(i * cap, i * cap + min(cap, count[i])) for i in range(e)]
        rows = e * cap

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16).mul_(scale)

    out = f // 2 if c["act"] == "swiglu" else f
    st = dict(a=normal(rows, k), w=normal(e, f, k, scale=k ** -0.5), off=off, cap=cap, spans=spans,
              bias=normal(e, f, scale=0.1) if c["bias"] else None, residual=normal(rows, out) if c["residual"] else None,
              y=torch.zeros((rows, out), dtype=torch.bfloat16, device=dev))
    if c["train"]:
        st.update(g=normal(rows, out), grad_a=torch.zeros((rows, k), dtype=torch.bfloat16, device=dev))
    return st


def prepare(case, seed):
    case = dict(case, scale=2.5)
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    return dict((_prepare_route if case["op"] == "route" else _prepare_product)(case, gen, dev), case=case)


# ---- one pass ----------------------------------------------------------------------------------


def _run_own(st):
    import combine_get_layout_02_b200 as cgl

    c = st["case"]
    if c["op"] == "route":
        how = dict(score=c["score"], renormalize=c["renorm"], scale=c["scale"])
        r = cgl.route(st["logits"], c["k"], bias=st["bias"], num_groups=c["groups"], topk_groups=c["keep"], group_score=c["by"], **how)
        out = {"idx": r.topk_idx, "weights": r.topk_weights}
        return dict(out, grad=cgl.route_backward(st["g"], st["logits"], r.topk_idx, **how)) if c["train"] else out
    where = (st["off"], st["cap"])
    how = dict(bias=st["bias"], activation=c["act"], residual=st["residual"], y=st["y"])
    if not c["train"]:
        return cgl.matmul_bf16(st["a"], st["w"], *where, **how)
    z = None
    if c["act"] == "none":
        y = cgl.matmul_bf16(st["a"], st["w"], *where, **how)
    else:
        y, z = cgl.matmul_bf16(st["a"], st["w"], *where, with_preact=True, **how)
    d = cgl.matmul_bf16_backward(st["g"], st["a"], st["w"], *where, activation=c["act"], preact=z, want_bias=c["bias"], grad_a=st["grad_a"])
    return {"y": y, "grad_a": d.grad_a, "grad_w": d.grad_w, **({"grad_bias": d.grad_bias} if c["bias"] else {})}


def run(state):
    if own:
        return _run_own(state)
    return _route(state) if state["case"]["op"] == "route" else _product(state)


def work(case):
    c = case
    if c["op"] == "route":   # logits once, choices and weights once; in training their gradient in and the logits' out
        row = c["n"] * c["e"] * BYTES[c["dtype"]]
        b = row + 8 * c["n"] * c["k"] + (4 * c["e"] if c["bias"] else 0)
        if c["train"]:
            b += row + 4 * c["n"] * c["k"]
        return {"bytes": b, "flops": 8 * c["n"] * c["e"]}
    r, f, k = c["rows"], c["f"], c["k"]
    out = f // 2 if c["act"] == "swiglu" else f
    e = c["e"] * (1 - (1 - 1 / c["e"]) ** r)   # experts that have a row
    b = 2 * (r * k + e * f * k + r * out * (2 if c["residual"] else 1) + (e * f if c["bias"] else 0))
    if c["train"]:            # the output's gradient in; the gradients of rows, weights and bias out
        b += 2 * (r * out + r * k + c["e"] * f * k + (c["e"] * f if c["bias"] else 0))
    return {"bytes": b, "flops": 2 * r * f * k * (3 if c["train"] else 1)}


# ---- the definition in 64 bits -----------------------------------------------------------------


def _route64(st):
    """By repeated maxima: the best groups one by one, then the best experts one by one."""
    c = st["case"]
    l = st["logits"].double()
    n, e = l.shape
    open_ = l > -torch.inf
    if c["score"] == "softmax":
        s = torch.nan_to_num(torch.softmax(l, dim=1), nan=0.0)
    else:
        s = torch.sigmoid(l)
    choice = l.clone() if st["bias"] is None else s + st["bias"].double()
    choice[~open_] = -torch.inf
    rows = torch.arange(n, device=l.device)
    if c["groups"] > 1:
        per = e // c["groups"]
        v = (choice if st["bias"] is not None or c["by"] == "max" else torch.where(open_, s, -torch.inf)).view(n, c["groups"], per)
        value = v.max(dim=2).values
        if c["by"] == "top2" and per > 1:
            first = v.argmax(dim=2, keepdim=True)
            second = v.scatter(2, first, -torch.inf).max(dim=2).values
            value = value + torch.where(second > -torch.inf, second, 0.0)
        allowed = torch.zeros((n, c["groups"]), dtype=torch.bool, device=l.device)
        for _ in range(c["keep"]):
            best = (value == value.max(dim=1, keepdim=True).values).int().argmax(dim=1)   # the first of equals
            allowed[rows, best] |= value[rows, best] > -torch.inf
            value[rows, best] = -torch.inf
        choice[~allowed.repeat_interleave(per, dim=1)] = -torch.inf
    ids = []
    for _ in range(c["k"]):
        top = choice.max(dim=1, keepdim=True).values
        best = (choice == top).int().argmax(dim=1)
        ids.append(torch.where(top[:, 0] > -torch.inf, best, -1))
        choice[rows, best] = -torch.inf
    idx = torch.stack(ids, dim=1)
    # weights as a dense [n, e] matrix over the picked experts
    picked = torch.zeros((n, e + 1), dtype=torch.bool, device=l.device)
    picked[rows[:, None], torch.where(idx >= 0, idx, e)] = True
    picked = picked[:, :e]
    share = torch.where(picked, s, 0.0)
    if c["renorm"]:
        if c["score"] == "softmax":
            share = torch.nan_to_num(torch.softmax(torch.where(picked, l, -torch.inf), dim=1), nan=0.0)
        else:
            share = share / share.sum(dim=1, keepdim=True).clamp(min=1e-300)
    at = idx.clamp(min=0)
    out = {"idx": idx.int(), "weights": c["scale"] * torch.where(idx >= 0, share.gather(1, at), 0.0)}
    if not c["train"]:
        return out
    g = torch.zeros((n, e + 1), dtype=torch.float64, device=l.device)
    g[rows[:, None], torch.where(idx >= 0, idx, e)] = c["scale"] * st["g"].double()
    g = g[:, :e]
    dot = (g * share).sum(dim=1, keepdim=True)
    if c["score"] == "softmax":
        grad = (share if c["renorm"] else s) * (g - dot)
    elif c["renorm"]:
        grad = share * torch.sigmoid(-l) * (g - dot)
    else:
        grad = share * torch.sigmoid(-l) * g
    return dict(out, grad=torch.where(open_, grad, 0.0))


def _product64(st):
    c = st["case"]
    dev, act = st["a"].device, c["act"]
    y = torch.zeros(st["y"].shape, dtype=torch.float64, device=dev)
    if c["train"]:
        da = torch.zeros(st["a"].shape, dtype=torch.float64, device=dev)
        dw = torch.zeros(st["w"].shape, dtype=torch.float64, device=dev)
        db = torch.zeros(st["w"].shape[:2], dtype=torch.float64, device=dev)
    for i, (r0, r1) in enumerate(st["spans"]):
        if r1 <= r0:
            continue
        rows, weight = st["a"][r0:r1].double(), st["w"][i].double()
        z = torch.mm(rows, weight.t())
        if c["bias"]:
            z += st["bias"][i].double()
        half = z.shape[1] // 2
        if act == "swiglu":
            s = torch.sigmoid(z[:, :half])
            y[r0:r1] = z[:, :half] * s * z[:, half:]
        elif act == "silu":
            s = torch.sigmoid(z)
            y[r0:r1] = z * s
        elif act == "gelu":
            s = 0.5 * torch.special.erfc(-z / math.sqrt(2))
            y[r0:r1] = z * s
        else:
            y[r0:r1] = z.clamp(min=0) if act == "relu" else z
        if c["residual"]:
            y[r0:r1] += st["residual"][r0:r1].double()
        if not c["train"]:
            continue
        g = st["g"][r0:r1].double()
        if act == "swiglu":
            dgate = s + z[:, :half] * s * (1 - s)
            d = torch.cat((g * z[:, half:] * dgate, g * z[:, :half] * s), dim=1)
        elif act == "silu":
            d = g * (s + z * s * (1 - s))
        elif act == "gelu":
            d = g * (s + z * torch.exp(-z * z / 2) * (2 * math.pi) ** -0.5)
        else:
            d = g * (z > 0) if act == "relu" else g
        da[r0:r1] = torch.mm(d, weight)
        dw[i] = torch.mm(d.t(), rows)
        db[i] = d.sum(0)
    if not c["train"]:
        return y
    out = {"y": y, "grad_a": da, "grad_w": dw}
    if c["bias"]:
        out["grad_bias"] = db
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return _route64(st) if st["case"]["op"] == "route" else _product64(st)
