"""Cases of the balance loss, the MXFP4 rows (quantise, dequantise, dispatch) and the experts' MXFP4 product.

`own` False: plain torch in 32 bits; True: the library's calls on the same state.  `exact` gives the
definition's values in 64 bits.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # one small batch of the smallest routing shape: launches are the cost
        dict(name="balance_tiny", op="balance", n=128, e=16, k=4, s=1, score="softmax", dtype="f32", pad=0.0, fused=True),
        # a prefill batch of 256 experts, sigmoid scores, loss and gradient in one call
        dict(name="balance_prefill", op="balance", n=4096, e=256, k=8, s=1, score="sigmoid", dtype="f32", pad=0.0, fused=True),
        # a training step's tokens, loss per sequence, padded tails, forward and backward as two calls
        dict(name="balance_train", op="balance", n=65536, e=256, k=8, s=16, score="softmax", dtype="bf16", pad=0.1, fused=False),
        # a decode batch's activations
        dict(name="rows_decode", op="rows", n=128, h=7168, dtype="bf16"),
        # a group of experts' weights from their 32-bit master copy
        dict(name="rows_weights", op="rows", n=16384, h=7168, dtype="f32"),
        # decode: padded receive rows, 128 tokens
        dict(name="dispatch_decode", op="dispatch", n=128, h=7168, e=256, k=8, padded=True, skip=0.0),
        # prefill: compact receive rows
        dict(name="dispatch_prefill", op="dispatch", n=4096, h=7168, e=256, k=8, padded=False, skip=0.0),
        # the smallest routing shape's product
        dict(name="product_tiny", op="product", rows=512, e=16, k=256, f=512, zipf=0.0, padded=False),
        # one token through one dense layer: a matrix-vector product
        dict(name="product_one_token", op="product", rows=1, e=1, k=7168, f=4096, zipf=0.0, padded=False),
        # a decode batch through all experts' first layer: the weights' bytes are the cost
        dict(name="product_decode", op="product", rows=1024, e=256, k=7168, f=4096, zipf=0.0, padded=True),
        # a prefill batch through all experts' first layer
        dict(name="product_prefill", op="product", rows=32768, e=256, k=7168, f=4096, zipf=0.0, padded=False),
        # a large batch with a skewed expert load through the experts' second layer
        dict(name="product_skewed", op="product", rows=131072, e=256, k=2048, f=7168, zipf=1.1, padded=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["balance", "rows", "dispatch", "product", "product"])
    if op == "balance":
        s = rng.choice([1, 1, 2, 3, 8, 16])
        e = _log(rng, 1, 512)
        n = s * _log(rng, 1, max(1, min(65536, 16777216 // e) // s))
        return dict(op=op, n=n, e=e, k=rng.randint(1, min(e, 8)), s=s, score=rng.choice(["softmax", "sigmoid"]),
                    dtype=rng.choice(["f32", "bf16", "f16"]), pad=rng.choice([0.0, 0.1, 0.5]), fused=rng.random() < 0.5)
    if op == "rows":
        h = 32 * _log(rng, 1, 256)
        return dict(op=op, n=_log(rng, 1, min(131072, 16384 * 7168 // h)), h=h, dtype=rng.choice(["f32", "bf16", "f16"]))
    if op == "dispatch":
        h = 32 * _log(rng, 1, 256)
        e = _log(rng, 1, 256)
        k = rng.randint(1, min(e, 8))
        return dict(op=op, n=_log(rng, 1, min(16384, 4096 * 7168 * 8 // (h * k))), h=h, e=e, k=k,
                    padded=rng.random() < 0.3, skip=rng.choice([0.0, 0.0, 0.2]))
    k = 32 * _log(rng, 1, 224)
    f = _log(rng, 1, 7168)
    e = _log(rng, 1, min(256, 256 * 4096 * 7168 // (f * k)))
    return dict(op=op, rows=_log(rng, 1, 131072 if k <= 2048 else 32768), e=e, k=k, f=f, zipf=rng.choice([0.0, 1.1]),
                padded=rng.random() < 0.3)


# ---- plain forms -------------------------------------------------------------------------------


def _quantize(x):
    """Rows [n, h] -> (e2m1 values in 32 bits [n, h/32, 32], scales 2^e in 32 bits [n, h/32, 1])."""
    v = x.float().reshape(x.shape[0], -1, 32)
    m, ex = torch.frexp(v.abs().amax(dim=2, keepdim=True))
    e = torch.where(m > 0.75, ex - 2, ex - 3).clamp_(min=-127)   # 6 * 2^e >= m * 2^ex
    v = torch.ldexp(v, -e)
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = torch.copysign(torch.round(a / step) * step, v)
    return q, e


def _pack(q, e):
    """The same as bytes: codes [n, h/2] (low half first) and scale bytes [n, h/32]."""
    a = q.abs()
    c = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    c = (c + 8 * torch.signbit(q)).to(torch.uint8).reshape(q.shape[0], -1, 2)
    return c[:, :, 0] | (c[:, :, 1] << 4), (e + 127).to(torch.uint8).reshape(q.shape[0], -1)


def _values(codes, scales):
    """Bytes -> the values they stand for, in 32 bits."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    pairs = torch.stack((grid.repeat(16), grid.repeat_interleave(16)), dim=1)   # a byte's two values, low half first
    v = pairs[codes.int()].reshape(*scales.shape, 32)
    return torch.ldexp(v, scales.int().unsqueeze(-1) - 127).flatten(-2)


def _balance(st):
    c, idx = st["case"], st["idx"]
    n, e, k, s = c["n"], c["e"], c["k"], c["s"]
    ok = (idx >= 0) & (idx < e)
    seq = torch.arange(n, device=idx.device) // (n // s)
    slot = torch.where(ok, idx + seq[:, None] * e, s * e)
    counts = torch.bincount(slot.flatten(), minlength=s * e + 1)[: s * e].reshape(s, e)
    there = ok.any(dim=1)
    t = there.reshape(s, -1).sum(dim=1, keepdim=True)
    total = counts.sum(dim=1, keepdim=True)
    unit = c["alpha"] / (s * k * t.clamp(min=1).double() ** 2)
    mean = (unit * total).float()[seq]                                # [n, 1]
    w = (unit * (e * counts - total)).float()[seq]                    # [n, e], less its mean
    x = st["logits"].float()
    if c["score"] == "softmax":
        p = torch.exp(x - x.amax(dim=1, keepdim=True))
        gate = 1.0
    else:
        p = 1 / (1 + torch.exp(-x))
        gate = 1 / (1 + torch.exp(x))
    p = p / p.sum(dim=1, keepdim=True)
    dot = (p * w).sum(dim=1, keepdim=True)
    loss = torch.where(there[:, None], mean + dot, 0).double().sum().float().reshape(1)
    grad = torch.where(there[:, None], st["g"] * p * (w - dot) * gate, 0)
    return {"loss": loss, "counts": counts.int(), "grad": grad.to(st["logits"].dtype)}


def _dispatch(st):
    c = st["case"]
    q, e = _quantize(st["x"])
    v = torch.ldexp(q, e).reshape(c["n"], c["h"]).bfloat16()
    out = torch.zeros((st["rows"], c["h"]), dtype=torch.bfloat16, device=v.device)
    to = st["dst"].flatten()
    keep = to >= 0
    out[to[keep].long()] = v.repeat_interleave(c["k"], dim=0)[keep]
    return out


def _product(st):
    y = torch.zeros_like(st["y"])
    for i, (r0, r1) in enumerate(st["spans"]):
        if r1 > r0:
            y[r0:r1] = (_values(st["a"][r0:r1], st["sa"][r0:r1]) @ _values(st["w"][i], st["sw"][i]).T).bfloat16()
    return y


# ---- inputs ------------------------------------------------------------------------------------


def _route(n, e, k, gen, zipf=0.0):
    """Top-k ids of noisy scores, no expert twice for a token."""
    score = torch.randn((n, e), generator=gen, device="cuda")
    if zipf:
        score -= 0.3 * zipf * torch.log(1 + torch.randperm(e, generator=gen, device="cuda").float())
    return score, torch.topk(score, k, dim=1).indices.int()


def _capacity(copies, e):
    """Rows a padded expert has room for, fixed before the counts are known; copies past it are dropped."""
    return min(copies, 8 + 2 * -(-copies // e))


def _mx_rows(n, h, gen, dev):
    """MXFP4 rows of normal values, made in pieces."""
    codes = torch.empty((n, h // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((n, h // 32), dtype=torch.uint8, device=dev)
    step = max(1, (1 << 27) // h)
    for r in range(0, n, step):
        x = torch.randn((min(step, n - r), h), generator=gen, device=dev)
        codes[r:r + step], scales[r:r + step] = _pack(*_quantize(x))
    return codes, scales


def _prepare_balance(c, gen, dev):
    n, e, k, s = c["n"], c["e"], c["k"], c["s"]
    logits, idx = _route(n, e, k, gen, 1.1)
    if c["pad"]:   # the ends of the sequences are padding; a few single slots carry no copy
        t = n // s
        length = t - (torch.rand(s, generator=gen, device=dev) * 2 * c["pad"] * t).int()
        idx.view(s, t, k)[torch.arange(t, device=dev)[None, :] >= length[:, None]] = -1
        idx[torch.rand((n, k), generator=gen, device=dev) < 0.01] = -1
    dt = DTYPES[c["dtype"]]
    # gradients of the mean over tokens are tiny: in f16 they come with a loss scale
    g = 2.0 ** round(math.log2(n * e)) if c["dtype"] == "f16" else 0.5
    return dict(logits=logits.to(dt), idx=idx, g=torch.full((1,), g, device=dev))


def _prepare_rows(c, gen, dev):
    x = torch.randn((c["n"], c["h"]), generator=gen, device=dev)
    x[torch.rand(c["n"], generator=gen, device=dev) < 0.01] *= 100
    return dict(x=x.to(DTYPES[c["dtype"]]))


def _prepare_dispatch(c, gen, dev):
    n, h, e, k = c["n"], c["h"], c["e"], c["k"]
    st = _prepare_rows(dict(n=n, h=h, dtype="bf16"), gen, dev)
    ids = _route(n, e, k, gen)[1].flatten()
    if c["skip"]:
        ids[torch.rand(n * k, generator=gen, device=dev) < c["skip"]] = -1
    order = torch.argsort(torch.where(ids >= 0, ids, e), stable=True)
    place = torch.empty(n * k, dtype=torch.int64, device=dev)
    place[order] = torch.arange(n * k, device=dev)
    rows = n * k
    if c["padded"]:
        count = torch.bincount(ids[ids >= 0], minlength=e)
        cap = _capacity(rows, e)
        first = count.cumsum(0) - count
        at = ids.clamp(min=0).long()
        place = place - first[at]
        ids = torch.where(place < cap, ids, -1)
        place = at * cap + place
        rows = e * cap
    dst = torch.where(ids >= 0, place, -1).int().reshape(n, k)
    st.update(dst=dst, rows=rows, codes=torch.zeros((rows, h // 2), dtype=torch.uint8, device=dev),
              scales=torch.zeros((rows, h // 32), dtype=torch.uint8, device=dev),
              scratch=torch.zeros(2, dtype=torch.int64, device=dev))
    return st


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
    a, sa = _mx_rows(rows, k, gen, dev)
    wq, sw = _mx_rows(e * f, k, gen, dev)
    return dict(a=a, sa=sa, w=wq.view(e, f, -1), sw=sw.view(e, f, -1), off=off, cap=cap, spans=spans,
                y=torch.zeros((rows, f), dtype=torch.bfloat16, device=dev))


def prepare(case, seed):
    case = dict(case, alpha=0.01)
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    make = {"balance": _prepare_balance, "rows": _prepare_rows, "dispatch": _prepare_dispatch, "product": _prepare_product}
    return dict(make[case["op"]](case, gen, dev), case=case)


# ---- one pass ----------------------------------------------------------------------------------


def _run_own(st):
    import combine_get_layout_02_b200 as cgl

    c = st["case"]
    if c["op"] == "balance":
        how = dict(num_sequences=c["s"], alpha=c["alpha"], score=c["score"])
        if c["fused"]:
            b = cgl.balance_loss(st["logits"], st["idx"], grad_loss=st["g"], **how)
            return {"loss": b.loss, "counts": b.counts, "grad": b.grad_logits}
        b = cgl.balance_loss(st["logits"], st["idx"], **how)
        grad = cgl.balance_loss_backward(st["g"], st["logits"], st["idx"], b.counts, b.num_routed, **how)
        return {"loss": b.loss, "counts": b.counts, "grad": grad}
    if c["op"] == "rows":
        codes, scales = cgl.quantize_mxfp4(st["x"])
        return cgl.dequantize_mxfp4(codes, scales, dtype=st["x"].dtype)
    if c["op"] == "dispatch":
        cgl.dispatch_mxfp4(st["x"], st["dst"], st["rows"], recv_x=st["codes"], recv_scale=st["scales"], scratch=st["scratch"])
        return cgl.dequantize_mxfp4(st["codes"], st["scales"])
    return cgl.matmul_mxfp4(st["a"], st["sa"], st["w"], st["sw"], st["off"], st["cap"], y=st["y"])


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "balance":
        return _balance(state)
    if op == "rows":
        q, e = _quantize(state["x"])
        return torch.ldexp(q, e).reshape(state["x"].shape).to(state["x"].dtype)
    return _dispatch(state) if op == "dispatch" else _product(state)


def work(case):
    c = case
    if c["op"] == "balance":   # logits and ids once, gradient, counts and loss once
        b = 2 * c["n"] * c["e"] * BYTES[c["dtype"]] + 4 * c["n"] * c["k"] + 4 * c["s"] * c["e"] + 4
        return {"bytes": b, "flops": 12 * c["n"] * c["e"]}
    if c["op"] == "rows":      # values in, codes and scales out; codes and scales in, values out
        return {"bytes": c["n"] * c["h"] * 2 * (BYTES[c["dtype"]] + 17 / 32), "flops": 4 * c["n"] * c["h"]}
    if c["op"] == "dispatch":  # values and rows' places in, k rows out; the rows in, their values out
        n = c["n"] * c["k"] * c["h"] * (1 - c["skip"])
        return {"bytes": 2 * c["n"] * c["h"] + 4 * c["n"] * c["k"] + n * (2 * 17 / 32 + 2), "flops": 4 * n}
    r, f, k = c["rows"], c["f"], c["k"]
    e = c["e"] * (1 - (1 - 1 / c["e"]) ** r)   # experts that have a row
    return {"bytes": (r * k + e * f * k) * 17 / 32 + 2 * r * f, "flops": 2 * r * f * k}


# ---- the definition in 64 bits -----------------------------------------------------------------


def _mx64(x):
    """What MXFP4 holds of x, block by block: scale by comparison with powers of two, codes by the borders between them."""
    b = x.double().reshape(-1, 32)
    top = b.abs().max(dim=1, keepdim=True).values
    e = torch.floor(torch.log2(top.clamp(min=2.0 ** -140) / 6)) - 1
    for _ in range(3):
        e = torch.where(6 * torch.exp2(e) < top, e + 1, e)
    s = torch.exp2(e.clamp(min=-127))
    a = b.abs() / s
    q = torch.zeros_like(a)
    # value gained on passing a border; a tie goes to the neighbour with the even code
    for border, gain, tie_up in ((0.25, 0.5, False), (0.75, 0.5, True), (1.25, 0.5, False), (1.75, 0.5, True),
                                 (2.5, 1.0, False), (3.5, 1.0, True), (5.0, 2.0, False)):
        q += gain * ((a >= border) if tie_up else (a > border))
    return (torch.sign(b) * q * s).reshape(x.shape)


def _decoded64(codes, scales):
    c = torch.stack((codes & 15, codes >> 4), dim=2).reshape(codes.shape[0], -1).long()
    mantissa, exponent = (c & 1).double(), ((c >> 1) & 3).double()
    v = torch.where(exponent == 0, mantissa / 2, (1 + mantissa / 2) * torch.exp2(exponent - 1))
    v = torch.where(c > 7, -v, v)
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, dim=1)


def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    if c["op"] == "rows":
        return _mx64(st["x"])
    if c["op"] == "dispatch":
        out = torch.zeros((st["rows"], c["h"]), dtype=torch.float64, device=st["x"].device)
        v = _mx64(st["x"])
        for j in range(c["k"]):
            to = st["dst"][:, j].long()
            out[to[to >= 0]] = v[to >= 0]
        return out
    if c["op"] == "product":
        y = torch.zeros(st["y"].shape, dtype=torch.float64, device=st["y"].device)
        for i, (r0, r1) in enumerate(st["spans"]):
            if r1 > r0:
                y[r0:r1] = torch.mm(_decoded64(st["a"][r0:r1], st["sa"][r0:r1]), _decoded64(st["w"][i], st["sw"][i]).t())
        return y
    l = st["logits"].double().reshape(c["s"], -1, c["e"])
    idx = st["idx"].long().reshape(c["s"], -1, c["k"])
    loss, counts, grads = 0.0, [], []
    for i in range(c["s"]):
        ids = idx[i][(idx[i] >= 0) & (idx[i] < c["e"])]
        here = ((idx[i] >= 0) & (idx[i] < c["e"])).sum(1) > 0
        t = max(1, int(here.sum()))
        count = torch.zeros(c["e"], dtype=torch.float64, device=l.device).index_add_(0, ids, torch.ones_like(ids, dtype=torch.float64))
        unit = c["alpha"] / c["s"] / (c["k"] * t) / t
        weight = unit * c["e"] * count
        tilt = unit * (c["e"] * count - count.sum())   # the weight less its mean: exactly 0 where all counts are equal
        if c["score"] == "softmax":
            p = torch.softmax(l[i], dim=1)
            slope = p
        else:
            sig = torch.sigmoid(l[i])
            p = sig / sig.sum(1, keepdim=True)
            slope = p * torch.sigmoid(-l[i])
        p = p * here[:, None]
        loss = loss + (p * weight).sum()
        centred = tilt - (p * tilt).sum(1, keepdim=True)
        grads.append(st["g"].double() * slope * centred * here[:, None])
        counts.append(count.int())
    return {"loss": loss.reshape(1), "counts": torch.stack(counts), "grad": torch.cat(grads)}
