"""Cases that measure what stands between the residual stream and the expert-parallel dispatch, and back.

Each case is one operator as a training or serving program calls it: the root-mean-square norm in front of an expert
layer (with the residual's addition and rows of 8 bits for the exchange) and its gradient, the widening of 8-bit rows
that an exchange delivered, the routing of tokens to experts and its gradient, and the dropout with which a layer's
output goes back to the residual stream.  With ``own`` false, ``run`` computes them from elementary torch operations;
with ``own`` true it calls the library.
"""
import math

import torch

own = False

DEV = "cuda"
GROUP = 128  # columns that share a scale in a row of 8 bits
E4M3_MOST = 448.0
LEAST_SCALE = 2.0 ** -100


# ------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decoding token in front of a 4096-wide expert layer: residual added, norm for the router and the experts
        dict(name="norm token", op="norm", rows=1, width=4096, dtype="bfloat16", wdtype="bfloat16", residual=True, y=True,
             wire=False, pad=0),
        # the expert-parallel workload's tokens, 8 ranks x 4096 of 2048: the norm for the router beside its 8-bit rows for
        # the dispatch
        dict(name="norm micro-batch", op="norm", rows=32768, width=2048, dtype="bfloat16", wdtype="float32", residual=True,
             y=True, wire=True, pad=0),
        # a ragged batch of a small model in 32 bits, gradients into a float32 weight gradient
        dict(name="norm grad ragged", op="norm_grad", rows=509, width=1408, dtype="float32", dwdtype="float32", two=False,
             dres=True),
        # the backward pass at the expert-parallel workload's size: gradients from the router and from the experts, and the
        # one that comes down the residual stream
        dict(name="norm grad", op="norm_grad", rows=32768, width=2048, dtype="bfloat16", dwdtype="bfloat16", two=True,
             dres=True),
        # 8-bit rows of a decoding step's dispatch, 8 ranks x 16 tokens, top-6 of 64 experts
        dict(name="widen decode", op="widen", k=8, experts=8, rows=96, width=2048),
        # and of a training step's: 8 x 4096 tokens
        dict(name="widen", op="widen", k=8, experts=8, rows=24576, width=2048),
        # routing of a decoding step: 8 x 16 tokens, softmax, top-6 of 64 experts
        dict(name="route decode", op="route", tokens=128, experts=64, topk=6, dtype="bfloat16", score="softmax", bias=False,
             groups=1, top_groups=1, renormalise=True, scale=1.0),
        # routing of a training step over many experts: sigmoid scores, a bias for balance, 4 of 8 groups, top-8 of 256
        dict(name="route groups", op="route", tokens=32768, experts=256, topk=8, dtype="float32", score="sigmoid", bias=True,
             groups=8, top_groups=4, renormalise=True, scale=2.5),
        # gradient of a small batch's routing whose gates are the softmax's own
        dict(name="route grad small", op="route_grad", tokens=509, experts=64, topk=6, dtype="bfloat16", score="softmax",
             renormalise=False, scale=1.0),
        # gradient of a training step's routing
        dict(name="route grad", op="route_grad", tokens=32768, experts=256, topk=8, dtype="float32", score="sigmoid",
             renormalise=True, scale=2.5),
        # dropout of a small, odd tensor in 32 bits
        dict(name="dropout small", op="dropout", rows=33, width=1001, dtype="float32", p=0.1, residual=False, pad=0),
        # dropout of a layer's output on its way back to the residual stream, 4 micro-batches of 8192 tokens
        dict(name="dropout residual", op="dropout", rows=32768, width=4096, dtype="bfloat16", p=0.1, residual=True, pad=0),
    ]


_COST_CAP = None


def _cost(c):
    return work(c)["bytes"]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A row width: a multiple of 64 mostly, of 8 often, and now and then any number."""
    n, kind = _log_int(rng, lo, hi), rng.random()
    step = 64 if kind < 0.5 else 8 if kind < 0.85 else 1
    return max(step, n // step * step)


def draw(rng):
    global _COST_CAP
    if _COST_CAP is None:
        _COST_CAP = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["norm", "norm", "norm_grad", "widen", "route", "route", "route_grad", "dropout"])
        dtype = rng.choice(["bfloat16", "bfloat16", "float32"])
        c = dict(op=op)
        if op == "norm":
            y = rng.random() < 0.8
            c.update(rows=_log_int(rng, 1, 65536), width=_width(rng, 64, 8192), dtype=dtype,
                     wdtype=rng.choice(["bfloat16", "float32"]), residual=rng.random() < 0.7, y=y,
                     wire=not y or rng.random() < 0.4, pad=rng.choice([0, 0, 8, 64]))
        elif op == "norm_grad":
            c.update(rows=_log_int(rng, 1, 65536), width=_width(rng, 64, 8192), dtype=dtype,
                     dwdtype=rng.choice(["bfloat16", "float32"]), two=rng.random() < 0.5, dres=rng.random() < 0.7)
        elif op == "widen":
            c.update(k=rng.choice([1, 2, 4, 8, 16]), experts=rng.choice([1, 2, 4, 8, 16]), rows=_log_int(rng, 1, 24576),
                     width=_width(rng, 64, 8192))
        elif op in ("route", "route_grad"):
            groups = rng.choice([1, 1, 2, 4, 8])
            experts = groups * rng.choice([4, 5, 8, 16, 20, 32, 64]) if rng.random() < 0.8 else rng.randint(4, 512)
            groups = groups if experts % groups == 0 else 1
            top_groups = rng.randint(1, groups)
            topk = rng.randint(1, min(12, experts // groups * top_groups))
            c.update(tokens=_log_int(rng, 1, 65536), experts=experts, topk=topk, dtype=dtype,
                     score=rng.choice(["softmax", "sigmoid"]), renormalise=topk > 1 and rng.random() < 0.6,
                     scale=rng.choice([1.0, 2.5]))
            if op == "route":
                c.update(bias=rng.random() < 0.5, groups=groups, top_groups=top_groups)
        else:
            c.update(rows=_log_int(rng, 1, 65536), width=_width(rng, 64, 8192), dtype=dtype,
                     p=rng.choice([0.0, 0.05, 0.1, 0.3, 0.5]), residual=rng.random() < 0.6, pad=rng.choice([0, 0, 8, 64]))
        if _cost(c) <= _COST_CAP:
            return c


# ------------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 29)


def _dt(name):
    return torch.bfloat16 if name == "bfloat16" else torch.float32


def _normal(g, *shape, dtype=torch.bfloat16, sigma=1.0, mean=0.0):
    """N(mean, sigma), drawn in pieces so that the 32-bit draw of a large tensor does not fill the card."""
    n = math.prod(shape)
    out = torch.empty(n, dtype=dtype, device=DEV)
    for at in range(0, n, 1 << 27):
        m = min(1 << 27, n - at)
        out[at: at + m] = torch.randn(m, generator=g, device=DEV) * sigma + mean
    return out.view(shape)


def _rows(g, rows, width, pad, dtype, sigma=1.0):
    """Rows of a buffer that is `pad` values wider."""
    return _normal(g, rows, width + pad, dtype=dtype, sigma=sigma)[:, :width]


def _wire_bytes(width):
    """Bytes of a row of 8 bits: values, from the next multiple of 16 on one 32-bit scale for each 128 of them, and up to a
    multiple of 16; and where the scales start."""
    at = -(-width // 16) * 16
    return at + -(-(-(-width // GROUP) * 4) // 16) * 16, at


def _wire_views(wire, width):
    at = _wire_bytes(width)[1]
    return (wire[:, :width].view(torch.float8_e4m3fn),
            wire[:, at: at + -(-width // GROUP) * 4].view(torch.float32))


def _routing(c, g):
    """Logits as a router gives them: a token's own, and experts that are liked more than others."""
    liked = torch.randn(c["experts"], generator=g, device=DEV) * 0.5
    return (torch.randn(c["tokens"], c["experts"], generator=g, device=DEV) + liked).to(_dt(c["dtype"]))


def _came(c):
    """Rows that an exchange delivered: a receive buffer has room for more."""
    return c["rows"] - c["rows"] // 4


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(case=c)
    op = c["op"]
    if op == "norm":
        n, w, dt = c["rows"], c["width"], _dt(c["dtype"])
        s["x"] = _rows(g, n, w, c["pad"], dt)
        s["r"] = _rows(g, n, w, c["pad"], dt, sigma=4.0) if c["residual"] else None
        s["w"] = _normal(g, w, dtype=_dt(c["wdtype"]), sigma=0.2, mean=1.0)
        if own:
            s["h"] = torch.empty(n, w, dtype=dt, device=DEV) if c["residual"] else None
            s["y"] = torch.empty(n, w, dtype=dt, device=DEV) if c["y"] else None
            s["wire"] = torch.empty(n, _wire_bytes(w)[0], dtype=torch.uint8, device=DEV) if c["wire"] else None
    elif op == "norm_grad":
        n, w, dt = c["rows"], c["width"], _dt(c["dtype"])
        s["dy"] = _normal(g, n, w, dtype=dt, sigma=1e-2)
        s["dy2"] = _normal(g, n, w, dtype=dt, sigma=1e-3) if c["two"] else None
        s["h"] = _normal(g, n, w, dtype=dt, sigma=4.0)
        s["dres"] = _normal(g, n, w, dtype=dt, sigma=1e-2) if c["dres"] else None
        s["w"] = _normal(g, w, dtype=torch.float32, sigma=0.2, mean=1.0)
        if own:
            from collective_communication_schedules_gb300 import hoc
            s["dx"] = torch.empty(n, w, dtype=dt, device=DEV)
            s["dw"] = torch.empty(w, dtype=_dt(c["dwdtype"]), device=DEV)
            s["ws"] = torch.empty(hoc.rms_norm_workspace(n, w), dtype=torch.int32, device=DEV)
    elif op == "widen":
        k, w = c["k"], c["width"]
        # pairs of every (rank, source, expert): some experts get several times what others do
        share = torch.rand(k, k * c["experts"], generator=g, device=DEV) ** 2 + 0.05
        pairs = torch.multinomial(share, _came(c), replacement=True, generator=g)
        counts = torch.zeros_like(share, dtype=torch.int64).scatter_add_(1, pairs, torch.ones_like(pairs))
        s["seg"] = torch.zeros(k, k * c["experts"] + 1, dtype=torch.int64, device=DEV)
        s["seg"][:, 1:] = counts.cumsum(1)
        bytes_, at = _wire_bytes(w)
        s["wire"] = []
        for _ in range(k):
            buf = torch.zeros(c["rows"], bytes_, dtype=torch.uint8, device=DEV)
            q, scale = _wire_views(buf, w)
            q.copy_((torch.randn(c["rows"], w, generator=g, device=DEV) * 120).clamp(-E4M3_MOST, E4M3_MOST))
            scale.copy_(torch.rand(scale.shape, generator=g, device=DEV) * 0.01 + 1e-3)
            s["wire"].append(buf)
        if own:
            s["y"] = [torch.zeros(c["rows"], w, dtype=torch.bfloat16, device=DEV) for _ in range(k)]
    elif op == "route":
        s["logits"] = _routing(c, g)
        # steps of 0.001 up or down, as a balancing rule leaves them
        s["bias"] = torch.randint(-40, 41, (c["experts"],), generator=g, device=DEV) * 0.001 if c["bias"] else None
        if own:
            n = c["tokens"] * c["topk"]
            s["ids"] = torch.empty(n, dtype=torch.int32, device=DEV)
            s["gate"] = torch.empty(n, device=DEV)
    elif op == "route_grad":
        s["logits"] = _routing(c, g)
        s["ids"] = s["logits"].double().sort(dim=1, descending=True, stable=True).indices[:, :c["topk"]].int().reshape(-1)
        s["dgate"] = torch.randn(c["tokens"] * c["topk"], generator=g, device=DEV) * 1e-2
        if own:
            s["dlogits"] = torch.empty_like(s["logits"])
    else:
        n, w, dt = c["rows"], c["width"], _dt(c["dtype"])
        s["x"] = _rows(g, n, w, c["pad"], dt)
        s["r"] = _rows(g, n, w, c["pad"], dt, sigma=4.0) if c["residual"] else None
        # the generator's key and the number of the call
        s["seed"] = torch.tensor([int(seed) * 0x9E3779B9 + 12345, int(seed) % 1000 + (1 << 33)], dtype=torch.int64, device=DEV)
        if own:
            s["y"] = torch.empty(n, w, dtype=dt, device=DEV)
    return s


# ------------------------------------------------------------------------------------------------- the plain form
EPS = 1e-6


def _plain_norm(s):
    c = s["case"]
    w, dt = c["width"], _dt(c["dtype"])
    h = s["x"] if s["r"] is None else (s["x"].float() + s["r"].float()).to(dt)
    f = h.float()
    y = f * torch.rsqrt((f * f).mean(1, keepdim=True) + EPS) * s["w"].float()
    out = dict(h=h if s["r"] is not None else None, y=y.to(dt) if c["y"] else None)
    if c["wire"]:
        groups = -(-w // GROUP)
        v = torch.zeros(c["rows"], groups * GROUP, device=DEV)
        v[:, :w] = y
        v = v.view(c["rows"], groups, GROUP)
        scale = (v.abs().amax(2) / E4M3_MOST).clamp(min=LEAST_SCALE)
        out["q"] = (v / scale[:, :, None]).view(c["rows"], -1)[:, :w].clamp(-E4M3_MOST, E4M3_MOST).to(torch.float8_e4m3fn)
        out["scale"] = scale
    return out


def _plain_norm_grad(s):
    c = s["case"]
    h = s["h"].float()
    d = s["dy"].float() + (s["dy2"].float() if c["two"] else 0)
    rr = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    g = d * s["w"]
    dx = rr * (g - h * (rr * rr * (g * h).mean(1, keepdim=True)))
    if c["dres"]:
        dx = dx + s["dres"].float()
    dw = (d * h * rr).sum(0)
    return dict(dx=dx.to(s["dy"].dtype), dw=dw.to(_dt(c["dwdtype"])))


def _plain_widen(s):
    c = s["case"]
    w = c["width"]
    ys = []
    n = _came(c)
    for wire in s["wire"]:
        q, scale = _wire_views(wire[:n], w)
        y = torch.zeros(c["rows"], w, dtype=torch.bfloat16, device=DEV)
        y[:n] = q.float() * scale.repeat_interleave(GROUP, dim=1)[:, :w]
        ys.append(y)
    return dict(y=ys)


def _scores(score, z):
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    e = torch.exp(z - z.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_route(s):
    """Scores in 64 bits: which of two near ones is larger decides."""
    c = s["case"]
    t, e = s["logits"].shape
    score = _scores(c["score"], s["logits"].double())
    key = score if s["bias"] is None else score + s["bias"].double()
    if c["groups"] > 1:
        per = e // c["groups"]
        of_group = key.view(t, c["groups"], per).sort(dim=2, descending=True).values[:, :, :2].sum(2)
        best = of_group.sort(dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        keep = torch.zeros(t, c["groups"], dtype=torch.bool, device=DEV).scatter_(1, best, True)
        key = torch.where(keep.repeat_interleave(per, dim=1), key, torch.full_like(key, -math.inf))
    ids = key.sort(dim=1, descending=True, stable=True).indices[:, :c["topk"]]
    gate = score.gather(1, ids)
    if c["renormalise"]:
        gate = gate / gate.sum(1, keepdim=True)
    return dict(ids=ids.int().reshape(-1), gate=(gate * c["scale"]).float().reshape(-1))


def _plain_route_grad(s):
    c = s["case"]
    ids = s["ids"].view(c["tokens"], c["topk"]).long()
    dg = s["dgate"].view(c["tokens"], c["topk"]) * c["scale"]
    z = s["logits"].float()
    score = _scores(c["score"], z)
    chosen = score.gather(1, ids)
    if c["renormalise"]:
        total = chosen.sum(1, keepdim=True)
        u = chosen / total
        ds = (dg - (dg * u).sum(1, keepdim=True)) / total
    else:
        ds = dg
    if c["score"] == "sigmoid":
        dz = torch.zeros_like(z).scatter_(1, ids, ds * chosen * (1 - chosen))
    elif c["renormalise"]:  # a softmax over the chosen ones
        dz = torch.zeros_like(z).scatter_(1, ids, ds * chosen)
    else:
        dz = torch.zeros_like(z).scatter_(1, ids, ds)
        dz = score * (dz - (ds * chosen).sum(1, keepdim=True))
    return dict(dlogits=dz.to(s["logits"].dtype))


_M32 = 0xFFFFFFFF


def _mul_hi_lo(m, v):
    """High and low words of the 64-bit product of two 32-bit numbers held in int64."""
    t, u = v * (m & 0xFFFF), v * (m >> 16)
    return (u + (t >> 16)) >> 16, (t + ((u & 0xFFFF) << 16)) & _M32


def _uniform16(n, seed):
    """16 random bits for each of n elements: Philox4x32-10 (Salmon et al., 2011) under the key seed[0], of the counter
    (element / 8, seed[1]); its four words give eight elements their bits, the low half of a word first."""
    g = torch.arange(-(-n // 8), dtype=torch.int64, device=DEV)
    key, call = seed[0], seed[1]
    c0, c1 = g & _M32, g >> 32
    c2, c3 = (call & _M32).expand_as(g), ((call >> 32) & _M32).expand_as(g)
    k0, k1 = key & _M32, (key >> 32) & _M32
    for _ in range(10):
        h0, l0 = _mul_hi_lo(0xD2511F53, c0)
        h1, l1 = _mul_hi_lo(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & _M32, (k1 + 0xBB67AE85) & _M32
    words = torch.stack([c0, c1, c2, c3], dim=1)
    return torch.stack([words & 0xFFFF, words >> 16], dim=2).view(-1)[:n]


def _threshold(p):
    return min(65535, int(p * 65536 + 0.5))


def _plain_dropout(s):
    c = s["case"]
    t = _threshold(c["p"])
    x = s["x"].float()
    keep = (_uniform16(x.numel(), s["seed"]) >= t).view(x.shape)
    y = torch.where(keep, x * (65536 / (65536 - t)), torch.zeros_like(x))
    if s["r"] is not None:
        y = y + s["r"].float()
    return dict(y=y.to(s["x"].dtype))


def _plain(s):
    return dict(norm=_plain_norm, norm_grad=_plain_norm_grad, widen=_plain_widen, route=_plain_route,
                route_grad=_plain_route_grad, dropout=_plain_dropout)[s["case"]["op"]](s)


# ------------------------------------------------------------------------------------------------- one pass
def run(state):
    s = state
    if not own:
        return _plain(s)
    from collective_communication_schedules_gb300 import hoc
    c = s["case"]
    op = c["op"]
    if op == "norm":
        hoc.rms_norm(s["x"], s["w"], s["y"], eps=EPS, residual=s["r"], h=s["h"], wire=s["wire"])
        out = dict(h=s["h"], y=s["y"])
        if c["wire"]:
            out["q"], out["scale"] = hoc.wire8_views(s["wire"], c["width"])
        return out
    if op == "norm_grad":
        hoc.rms_norm_grad(s["dy"], s["h"], s["w"], s["dx"], eps=EPS, dy2=s["dy2"], dres=s["dres"], dw=s["dw"],
                          workspace=s["ws"])
        return dict(dx=s["dx"], dw=s["dw"])
    if op == "widen":
        hoc.expert_widen(s["wire"], s["seg"], s["y"])
        return dict(y=s["y"])
    if op == "route":
        hoc.ep_route(s["logits"], s["ids"], s["gate"], score=c["score"], bias=s["bias"], groups=c["groups"],
                     top_groups=c["top_groups"], renormalise=c["renormalise"], scale=c["scale"])
        return dict(ids=s["ids"], gate=s["gate"])
    if op == "route_grad":
        hoc.ep_route_grad(s["logits"], s["ids"], s["dgate"], s["dlogits"], score=c["score"],
                          renormalise=c["renormalise"], scale=c["scale"])
        return dict(dlogits=s["dlogits"])
    hoc.dropout(s["x"], s["y"], c["p"], s["seed"], residual=s["r"])
    return dict(y=s["y"])


# ------------------------------------------------------------------------------------------------- the least work
def work(case):
    """Bytes of every input read once and every output written once, and the operations on them."""
    c = case
    op = c["op"]
    b = 2 if c.get("dtype") == "bfloat16" else 4
    if op == "norm":
        n, w = c["rows"], c["width"]
        rows = b * (1 + 2 * c["residual"] + c["y"]) * w + (w + 4 * -(-w // GROUP) if c["wire"] else 0)
        return dict(bytes=n * rows + w * (2 if c["wdtype"] == "bfloat16" else 4), flops=(5 + 3 * c["wire"]) * n * w)
    if op == "norm_grad":
        n, w = c["rows"], c["width"]
        dw = 2 if c["dwdtype"] == "bfloat16" else 4
        return dict(bytes=n * w * b * (3 + c["two"] + c["dres"]) + w * (4 + dw), flops=10 * n * w)
    if op == "widen":
        n, w = c["k"] * _came(c), c["width"]
        return dict(bytes=n * (w + 4 * -(-w // GROUP) + 2 * w), flops=n * w)
    if op == "route":
        n, e = c["tokens"], c["experts"]
        return dict(bytes=n * (b * e + 8 * c["topk"]) + 4 * e * c["bias"], flops=n * (6 * e + c["topk"] * e))
    if op == "route_grad":
        n, e = c["tokens"], c["experts"]
        return dict(bytes=n * (2 * b * e + 8 * c["topk"]), flops=8 * n * e)
    n = c["rows"] * c["width"]
    return dict(bytes=n * b * (2 + c["residual"]), flops=3 * n)


# ------------------------------------------------------------------------------------------------- 64 bits
def _exact_bits(n, seed):
    """The generator's 16-bit numbers once more: 32-bit words in 16-bit halves, products from their four parts."""
    key, call = int(seed[0]) & (2 ** 64 - 1), int(seed[1]) & (2 ** 64 - 1)
    g = torch.arange((n + 7) // 8, dtype=torch.int64, device=DEV)

    def product(m, v):
        ml, mh, vl, vh = m % 65536, m // 65536, v.remainder(65536), v.div(65536, rounding_mode="floor")
        low, mid, high = ml * vl, ml * vh + mh * vl, mh * vh
        mid = mid + low.div(65536, rounding_mode="floor")
        return high + mid.div(65536, rounding_mode="floor"), mid.remainder(65536) * 65536 + low.remainder(65536)

    x = [g.remainder(2 ** 32), g.div(2 ** 32, rounding_mode="floor"), torch.full_like(g, call % 2 ** 32),
         torch.full_like(g, call // 2 ** 32)]
    for i in range(10):
        ka = (key % 2 ** 32 + i * 0x9E3779B9) % 2 ** 32
        kb = (key // 2 ** 32 + i * 0xBB67AE85) % 2 ** 32
        (ha, la), (hb, lb) = product(0xD2511F53, x[0]), product(0xCD9E8D57, x[2])
        x = [hb.bitwise_xor(x[1]).bitwise_xor(ka), lb, ha.bitwise_xor(x[3]).bitwise_xor(kb), la]
    bits = torch.empty(g.numel(), 8, dtype=torch.int32, device=DEV)
    for i, v in enumerate(x):
        bits[:, 2 * i] = v.remainder(65536)
        bits[:, 2 * i + 1] = v.div(65536, rounding_mode="floor")
    return bits.flatten()[:n]


def exact(case, seed):
    """The operators' definitions in 64 bits, on inputs made as run's are."""
    global own
    c, was = case, own
    own = False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op, f64 = c["op"], torch.float64
    if op == "norm":
        w = c["width"]
        h = s["x"].to(f64)
        if c["residual"]:
            h = h + s["r"].to(f64)
        stream = h
        if c["residual"]:  # the norm is of the sum as it is stored
            h = h.to(_dt(c["dtype"])).to(f64)
        y = torch.einsum("rc,r,c->rc", h, 1 / torch.sqrt(torch.einsum("rc,rc->r", h, h) / w + EPS), s["w"].to(f64))
        out = dict(h=stream if c["residual"] else None, y=y if c["y"] else None)
        if c["wire"]:
            parts = y.split(GROUP, dim=1)
            scale = torch.stack([p.abs().max(1).values for p in parts], 1) / E4M3_MOST
            out["scale"] = torch.maximum(scale, torch.full_like(scale, LEAST_SCALE))
            out["q"] = torch.cat([p / out["scale"][:, i: i + 1] for i, p in enumerate(parts)], 1)
        return out
    if op == "norm_grad":
        h = s["h"].to(f64)
        d = s["dy"].to(f64)
        if c["two"]:
            d = d + s["dy2"].to(f64)
        size = (h.square().sum(1) / c["width"] + EPS).sqrt()
        unit = h / size[:, None]
        dw = torch.einsum("rc,rc->c", d, unit)
        g = d * s["w"].to(f64)
        dx = (g - unit * torch.einsum("rc,rc->r", g, unit)[:, None] / c["width"]) / size[:, None]
        if c["dres"]:
            dx = dx + s["dres"].to(f64)
        return dict(dx=dx, dw=dw)
    if op == "widen":
        ys, n = [], _came(c)
        for wire in s["wire"]:
            q, scale = _wire_views(wire, c["width"])
            y = torch.zeros(c["rows"], c["width"], dtype=f64, device=DEV)
            for i, part in enumerate(y.split(GROUP, dim=1)):
                part[:n] = q[:n, i * GROUP: i * GROUP + part.shape[1]].to(f64) * scale[:n, i: i + 1].to(f64)
            ys.append(y)
        return dict(y=ys)
    if op in ("route", "route_grad"):
        z = s["logits"].to(f64).requires_grad_(op == "route_grad")
        score = torch.sigmoid(z) if c["score"] == "sigmoid" else torch.softmax(z, 1)
        if op == "route_grad":
            ids = s["ids"].view(c["tokens"], -1).long()
            chosen = torch.gather(score, 1, ids)
            gate = chosen / chosen.sum(1, keepdim=True) if c["renormalise"] else chosen
            return dict(dlogits=torch.autograd.grad(c["scale"] * gate, z, s["dgate"].to(f64).view_as(gate))[0])
        key = score + (s["bias"].to(f64) if c["bias"] else 0)
        order = torch.arange(c["experts"], device=DEV)
        if c["groups"] > 1:
            per = c["experts"] // c["groups"]
            strength = torch.stack([v.topk(min(2, per), 1).values.sum(1) for v in key.split(per, 1)], 1)
            least = strength.topk(c["top_groups"], 1).values[:, -1:]
            key = key.masked_fill((strength < least)[:, order // per], -math.inf)
        gate, ids = [], []
        for _ in range(c["topk"]):
            best = key.max(1, keepdim=True).values
            ids.append(torch.where(key == best, order, c["experts"]).min(1).values)
            gate.append(score[torch.arange(c["tokens"], device=DEV), ids[-1]])
            key = key.scatter(1, ids[-1][:, None], -math.inf)
        gate = torch.stack(gate, 1)
        if c["renormalise"]:
            gate = gate / gate.sum(1, keepdim=True)
        return dict(ids=torch.stack(ids, 1).int().flatten(), gate=c["scale"] * gate.flatten())
    t = int(math.floor(c["p"] * 65536 + 0.5))
    y = s["x"].to(f64) * (65536 / (65536 - t))
    y[(_exact_bits(y.numel(), s["seed"]) < t).view(y.shape)] = 0
    return dict(y=y + s["r"].to(f64) if c["residual"] else y)
