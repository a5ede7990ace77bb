"""Cases that measure the expert layer's, the linear layer's and the gradient operators.

Each case is one operator as a training or serving program calls it: the products of an expert layer between
dispatch and combine (forward, data gradient, weight gradient), the linear layer beside it (forward with its
epilogue, gradients), the gradient of the gate-weighted combine, and the clipping of gradients by their global norm.
With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits; with ``own`` true it calls the
library.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step of an expert layer: 8 ranks x 16 tokens, top-6 of 64 experts, the gated up projection
        dict(name="expert_mm decode", op="expert_mm", k=8, tokens=16, topk=6, experts=64, inp=2048, out=1280,
             act="swiglu", bias=False, train=False),
        # the expert-parallel workload's training step: 8 x 4096 tokens of 2048, top-6 of 64 experts drawn from
        # Zipf(1.1); the gated up projection, its pre-activation kept for the backward pass
        dict(name="expert_mm up", op="expert_mm", k=8, tokens=4096, topk=6, experts=64, inp=2048, out=1280,
             act="swiglu", bias=False, train=True),
        # few wide experts (top-2 of 8, 4096-wide rows), an odd token count, a down projection with its bias
        dict(name="expert_mm down", op="expert_mm", k=4, tokens=509, topk=2, experts=8, inp=1024, out=4096,
             act="none", bias=True, train=False),
        # data gradient of the down projection, through the gated activation below it
        dict(name="expert_dgrad", op="expert_dgrad", k=8, tokens=2048, topk=6, experts=64, inp=1280, out=2048,
             act="swiglu"),
        # weight gradient of the up projection
        dict(name="expert_wgrad", op="expert_wgrad", k=8, tokens=4096, topk=6, experts=64, inp=2048, out=2560,
             bias=False),
        # a pipeline stage's linear layer while decoding: one token of 4096
        dict(name="linear token", op="linear", rows=1, inp=4096, out=4096, act="silu", bias=True, residual=True,
             pad=0, train=False),
        # the same layer on a micro-batch of 4096 tokens, with everything its epilogue can do
        dict(name="linear micro-batch", op="linear", rows=4096, inp=4096, out=4096, act="gelu", bias=True,
             residual=True, pad=0, train=True),
        # gradients of a linear layer on an odd number of rows: input, weight and bias
        dict(name="linear grad", op="linear_grad", rows=2047, inp=2048, out=1408, bias=True),
        # a small model's gradients: 48 tensors of uneven sizes, at odd places of their bucket
        dict(name="clip small", op="clip", tensors=48, elems=1_500_001, dtype="float32", sigma=1e-2),
        # the data-parallel gradient stream: 32 buckets of 13,107,200 bf16 values
        dict(name="clip buckets", op="clip", tensors=32, elems=32 * 13_107_200, dtype="bfloat16", sigma=1e-3),
        # the backward pass of the expert-parallel combine at a small batch, top-2 of 8 experts
        dict(name="combine grad small", op="combine_grad", k=2, tokens=33, topk=2, experts=8, hidden=4096),
        # and at the expert-parallel workload's size
        dict(name="combine grad", op="combine_grad", k=8, tokens=4096, topk=6, experts=64, hidden=2048),
    ]


_COST_CAP = None


def _cost(c):
    w = work(c)
    return max(w["bytes"] / 6.7e12, w["flops"] / 2e15)


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A row width: a multiple of 64 mostly, of 8 often, and now and then any number."""
    n, kind = _log_int(rng, lo, hi), rng.random()
    step = 64 if kind < 0.5 else 8 if kind < 0.9 else 1
    return max(step, n // step * step)


def _draw_routed(rng):
    k = rng.choice([1, 2, 4, 8, 16])
    experts = k * rng.choice([1, 2, 3, 4, 8, 16])
    return dict(k=k, tokens=_log_int(rng, 1, 4096), topk=min(experts, rng.randint(1, 8)), experts=experts)


def draw(rng):
    global _COST_CAP
    if _COST_CAP is None:
        _COST_CAP = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["expert_mm", "expert_mm", "expert_dgrad", "expert_wgrad", "linear", "linear", "linear_grad",
                         "clip", "clip", "combine_grad"])
        c = dict(op=op)
        if op.startswith("expert"):
            c.update(_draw_routed(rng), inp=_width(rng, 256, 4096), out=_width(rng, 256, 4096))
        if op == "expert_mm":
            c.update(act=rng.choice(["none", "relu", "gelu", "silu", "swiglu", "swiglu"]), bias=rng.random() < 0.4,
                     train=rng.random() < 0.5)
        elif op == "expert_dgrad":
            c.update(act=rng.choice(["none", "gelu", "silu", "swiglu", "swiglu"]))
        elif op == "expert_wgrad":
            c.update(bias=rng.random() < 0.4)
        elif op == "linear":
            c.update(rows=_log_int(rng, 1, 8192), inp=_width(rng, 256, 7168), out=_width(rng, 256, 7168),
                     act=rng.choice(["none", "relu", "gelu", "silu", "swiglu"]), bias=rng.random() < 0.6,
                     residual=rng.random() < 0.6, pad=rng.choice([0, 0, 8, 64]), train=rng.random() < 0.5)
        elif op == "linear_grad":
            c.update(rows=_log_int(rng, 1, 8192), inp=_width(rng, 256, 7168), out=_width(rng, 256, 7168),
                     bias=rng.random() < 0.6)
        elif op == "clip":
            tensors = _log_int(rng, 1, 300)
            c.update(tensors=tensors, elems=max(tensors, _log_int(rng, 1000, 400_000_000)),
                     dtype=rng.choice(["float32", "bfloat16"]), sigma=rng.choice([1e-5, 1e-3, 1e-2, 1.0]))
        else:
            c.update(_draw_routed(rng), hidden=_width(rng, 512, 7168))
        if _cost(c) <= _COST_CAP and 3072 not in c.values():
            return c


# ------------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 17)


def _normal(g, *shape, sigma=1.0):
    """N(0, sigma) as bf16, drawn in pieces so that the 32-bit draw of a large tensor does not fill the card."""
    n = math.prod(shape)
    out = torch.empty(n, dtype=torch.bfloat16, device=DEV)
    for at in range(0, n, 1 << 27):
        m = min(1 << 27, n - at)
        out[at: at + m] = torch.randn(m, generator=g, device=DEV) * sigma
    return out.view(shape)


def _zipf(experts, s=1.1):
    w = [(e + 1.0) ** -s for e in range(experts)]
    return [v / sum(w) for v in w]


def _choose(c, g):
    """Expert ids [k, tokens, topk], distinct for a token, drawn from Zipf(1.1), and how many pairs each source has for
    each expert [k, experts]."""
    k, experts = c["k"], c["experts"]
    logp = torch.tensor(_zipf(experts), device=DEV).log()
    noise = torch.rand(k, c["tokens"], experts, generator=g, device=DEV).clamp_(1e-20, 1 - 1e-7)
    ids = (logp - (-noise.log()).log()).topk(c["topk"], dim=-1).indices
    counts = torch.zeros(k, experts, dtype=torch.int64, device=DEV)
    counts.scatter_add_(1, ids.reshape(k, -1), torch.ones_like(ids.reshape(k, -1)))
    return ids.to(torch.int32), counts


def _route(c, g):
    """Expert ids and counts of one batch; row ranges [k, k * G + 1] of the receive layout (rank by rank: source, then
    expert), on the device and as host lists; and the rows each receive buffer has room for: what an earlier batch
    sent, with slack, so that it is the same for every batch."""
    k, per = c["k"], c["experts"] // c["k"]
    _, earlier = _choose(c, _gen(12345))
    room = [int(1.05 * n + 7 * n ** 0.5 + 24) for n in earlier.view(k, k, per).sum((0, 2)).tolist()]
    ids, counts = _choose(c, g)
    seg = torch.zeros(k, k * per + 1, dtype=torch.int64, device=DEV)
    seg[:, 1:] = counts.view(k, k, per).permute(1, 0, 2).reshape(k, -1).cumsum(1)  # [rank, source, expert]
    ranges = [[min(v, n) for v in r] for r, n in zip(seg.tolist(), room)]
    return ids, counts, seg, ranges, room


def _gated(c):
    return 2 if c.get("act") == "swiglu" else 1


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(case=c)
    op = c["op"]
    if op.startswith("expert"):
        k, per = c["k"], c["experts"] // c["k"]
        _, _, s["seg"], s["ranges"], rows = _route(c, g)
        inp, out, mul = c["inp"], c["out"], _gated(c)
        buf = lambda width: [torch.zeros(n, width, dtype=torch.bfloat16, device=DEV) for n in rows]  # noqa: E731
        if op == "expert_mm":
            s["x"] = [_normal(g, n, inp) for n in rows]
            s["w"] = [_normal(g, per, mul * out, inp, sigma=inp ** -0.5) for _ in range(k)]
            s["b"] = [_normal(g, per, mul * out, sigma=0.5) for _ in range(k)] if c["bias"] else None
            if own:
                s["y"], s["pre"] = buf(out), buf(mul * out) if c["train"] else None
        elif op == "expert_dgrad":
            s["dy"] = [_normal(g, n, out, sigma=1e-2) for n in rows]
            s["w"] = [_normal(g, per, out, inp, sigma=inp ** -0.5) for _ in range(k)]
            s["pre"] = [_normal(g, n, mul * inp) for n in rows] if c["act"] != "none" else None
            if own:
                s["dx"] = buf(mul * inp)
        else:
            s["x"] = [_normal(g, n, inp) for n in rows]
            s["dy"] = [_normal(g, n, out, sigma=1e-2) for n in rows]
            if own:
                s["dw"] = [torch.empty(per, out, inp, dtype=torch.bfloat16, device=DEV) for _ in range(k)]
                s["db"] = [torch.empty(per, out, dtype=torch.bfloat16, device=DEV) for _ in range(k)] if c["bias"] else None
    elif op == "linear":
        n, inp, out, mul = c["rows"], c["inp"], c["out"], _gated(c)
        s["x"] = _normal(g, n, inp + c["pad"])[:, :inp]  # rows of a wider buffer where pad > 0
        s["w"] = _normal(g, mul * out, inp, sigma=inp ** -0.5)
        s["b"] = _normal(g, mul * out, sigma=0.5) if c["bias"] else None
        s["r"] = _normal(g, n, out) if c["residual"] else None
        if own:
            s["y"] = torch.empty(n, out, dtype=torch.bfloat16, device=DEV)
            s["pre"] = torch.empty(n, mul * out, dtype=torch.bfloat16, device=DEV) if c["train"] else None
    elif op == "linear_grad":
        n, inp, out = c["rows"], c["inp"], c["out"]
        s["x"], s["dy"] = _normal(g, n, inp), _normal(g, n, out, sigma=1e-2)
        s["w"] = _normal(g, out, inp, sigma=inp ** -0.5)
        if own:
            s["dx"], s["dw"] = torch.empty_like(s["x"]), torch.empty_like(s["w"])
            s["db"] = torch.empty(out, dtype=torch.bfloat16, device=DEV) if c["bias"] else None
    elif op == "clip":
        dt = torch.bfloat16 if c["dtype"] == "bfloat16" else torch.float32
        cuts = _cuts(c, seed)
        s["flat"] = _normal(g, c["elems"], sigma=c["sigma"]) if dt == torch.bfloat16 else torch.randn(
            c["elems"], generator=g, device=DEV) * c["sigma"]
        s["grads"] = [s["flat"][a:b] for a, b in zip(cuts, cuts[1:])]
        s["max_norm"] = 1.0
        s["out"] = torch.empty_like(s["flat"])
        s["outs"] = [s["out"][a:b] for a, b in zip(cuts, cuts[1:])]
        if own:
            from collective_communication_schedules_gb300 import hoc
            s["norm"] = torch.empty(1, device=DEV)
            s["src"], s["dst"] = hoc.TensorList(s["grads"]), hoc.TensorList(s["outs"])
            s["ws"] = torch.empty(hoc.grad_workspace(s["src"]), dtype=torch.int32, device=DEV)
    else:
        k, t, j, per = c["k"], c["tokens"], c["topk"], c["experts"] // c["k"]
        ids, counts, _, s["ranges"], room = _route(c, g)
        s["ids"] = [v.reshape(-1).contiguous() for v in ids]
        order = [torch.sort(v, stable=True).indices for v in s["ids"]]
        s["pos"] = [torch.empty_like(v).scatter_(0, o, torch.arange(t * j, dtype=torch.int32, device=DEV))
                    for v, o in zip(s["ids"], order)]
        s["counts"] = counts.view(k, k, per).sum(2) * c["hidden"]  # [source, rank], in elements
        s["rows"] = [_normal(g, n, c["hidden"]) for n in room]
        s["dy"] = [_normal(g, t, c["hidden"], sigma=1e-2) for _ in range(k)]
        s["gate"] = [torch.rand(t * j, generator=g, device=DEV) for _ in range(k)]
        if own:
            s["drows"] = [torch.zeros_like(v) for v in s["rows"]]
            s["dgate"] = [torch.empty_like(v) for v in s["gate"]]
    if own:
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return s


def _cuts(c, seed):
    """Places where the flat buffer is cut into the case's tensors: uneven, at any element."""
    n, m = c["tensors"], c["elems"]
    if m % n == 0 and m // n >= 1 << 20:
        return [i * (m // n) for i in range(n + 1)]
    import random
    rng = random.Random(int(seed))
    return [0] + sorted(rng.randint(0, m) for _ in range(n - 1)) + [m]


# ------------------------------------------------------------------------------------------------- the plain form
def _act(name, z):
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "swiglu":
        a, b = z.chunk(2, dim=-1)
        return a / (1 + torch.exp(-a)) * b
    return z


def _act_grad(name, z, d):
    """The gradient for the pre-activation z of an activation whose output's gradient is d."""
    if name == "relu":
        return torch.where(z > 0, d, torch.zeros_like(d))
    if name == "gelu":
        q = math.sqrt(2 / math.pi)
        th = torch.tanh(q * (z + 0.044715 * z * z * z))
        return d * (0.5 * (1 + th) + 0.5 * z * (1 - th * th) * q * (1 + 3 * 0.044715 * z * z))
    if name == "silu":
        sg = 1 / (1 + torch.exp(-z))
        return d * sg * (1 + z * (1 - sg))
    if name == "swiglu":
        a, b = z.chunk(2, dim=-1)
        sg = 1 / (1 + torch.exp(-a))
        return torch.cat([d * b * sg * (1 + a * (1 - sg)), d * a * sg], dim=-1)
    return d


def _expert_slices(s):
    """(rank, expert, the expert's row ranges in the rank's buffer, one for each source that sent it rows)."""
    k, per = s["case"]["k"], s["case"]["experts"] // s["case"]["k"]
    for d in range(k):
        r = s["ranges"][d]
        for e in range(per):
            at = [(r[a * per + e], r[a * per + e + 1]) for a in range(k)]
            yield d, e, [(lo, hi) for lo, hi in at if hi > lo]


def _rows_of(t, at):
    return torch.cat([t[lo:hi] for lo, hi in at]).float()


def _put_rows(t, at, v):
    for part, (lo, hi) in zip(v.split([hi - lo for lo, hi in at]), at):
        t[lo:hi] = part.to(t.dtype)


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "expert_mm":
        y = [torch.zeros(x.shape[0], c["out"], dtype=x.dtype, device=DEV) for x in s["x"]]
        pre = [torch.zeros(x.shape[0], _gated(c) * c["out"], dtype=x.dtype, device=DEV) for x in s["x"]] if c["train"] else None
        for d, e, at in _expert_slices(s):
            if at:
                z = _rows_of(s["x"][d], at) @ s["w"][d][e].float().t()
                if s["b"] is not None:
                    z = z + s["b"][d][e].float()
                if pre is not None:
                    _put_rows(pre[d], at, z)
                _put_rows(y[d], at, _act(c["act"], z))
        return dict(y=y, pre=pre)
    if op == "expert_dgrad":
        dx = [torch.zeros(v.shape[0], _gated(c) * c["inp"], dtype=v.dtype, device=DEV) for v in s["dy"]]
        for d, e, at in _expert_slices(s):
            if at:
                v = _rows_of(s["dy"][d], at) @ s["w"][d][e].float()
                if s["pre"] is not None:
                    v = _act_grad(c["act"], _rows_of(s["pre"][d], at), v)
                _put_rows(dx[d], at, v)
        return dict(dx=dx)
    if op == "expert_wgrad":
        k, per = c["k"], c["experts"] // c["k"]
        dw = [torch.zeros(per, c["out"], c["inp"], dtype=torch.bfloat16, device=DEV) for _ in range(k)]
        db = [torch.zeros(per, c["out"], dtype=torch.bfloat16, device=DEV) for _ in range(k)] if c["bias"] else None
        for d, e, at in _expert_slices(s):
            if at:
                v = _rows_of(s["dy"][d], at)
                dw[d][e] = (v.t() @ _rows_of(s["x"][d], at)).to(torch.bfloat16)
                if db is not None:
                    db[d][e] = v.sum(0).to(torch.bfloat16)
        return dict(dw=dw, db=db)
    if op == "linear":
        z = s["x"].float() @ s["w"].float().t()
        if s["b"] is not None:
            z = z + s["b"].float()
        y = _act(c["act"], z)
        if s["r"] is not None:
            y = y + s["r"].float()
        return dict(y=y.to(torch.bfloat16), pre=z.to(torch.bfloat16) if c["train"] else None)
    if op == "linear_grad":
        x, dy = s["x"].float(), s["dy"].float()
        return dict(dx=(dy @ s["w"].float()).to(torch.bfloat16), dw=(dy.t() @ x).to(torch.bfloat16),
                    db=dy.sum(0).to(torch.bfloat16) if c["bias"] else None)
    if op == "clip":
        total = torch.zeros(1, device=DEV)
        for v in s["grads"]:
            f = v.float()
            total = total + (f * f).sum()
        norm = total.sqrt()
        coef = torch.where(norm + 1e-6 > s["max_norm"], s["max_norm"] / (norm + 1e-6), torch.ones_like(norm))
        for v, o in zip(s["grads"], s["outs"]):
            o[:] = (v.float() * coef).to(o.dtype)
        return dict(norm=norm, out=s["out"])
    k, t, j = c["k"], c["tokens"], c["topk"]
    drows = [torch.zeros_like(v) for v in s["rows"]]
    dgate = []
    places = _places(s)
    for a in range(k):
        dg = torch.zeros(t * j, device=DEV)
        token = torch.arange(t * j, device=DEV) // j
        for d in range(k):
            pairs, row = places[a][d]
            v = s["dy"][a][token[pairs]].float()
            drows[d][row] = (v * s["gate"][a][pairs, None]).to(torch.bfloat16)
            dg[pairs] = (v * s["rows"][d][row].float()).sum(-1)
        dgate.append(dg)
    return dict(drows=drows, dgate=dgate)


def _places(s):
    """places[a][d]: the pairs of source a that went to rank d, and their rows in rank d's buffer."""
    c = s["case"]
    k, per = c["k"], c["experts"] // c["k"]
    first = [[0] * k for _ in range(k)]  # first packed row of source a that is bound for rank d
    for a in range(k):
        n = 0
        for d in range(k):
            first[a][d] = n
            n += s["ranges"][d][(a + 1) * per] - s["ranges"][d][a * per]
    out = []
    for a in range(k):
        order = torch.argsort(s["pos"][a])
        out.append([])
        for d in range(k):
            lo, hi = s["ranges"][d][a * per], s["ranges"][d][(a + 1) * per]
            pairs = order[first[a][d]: first[a][d] + hi - lo]
            out[a].append((pairs, torch.arange(lo, hi, device=DEV)))
    return out


# ------------------------------------------------------------------------------------------------- one pass
def run(state):
    s = state
    if not own:
        return _plain(s)
    from collective_communication_schedules_gb300 import hoc
    c = s["case"]
    op = c["op"]
    if op == "expert_mm":
        hoc.expert_mm(s["x"], s["w"], s["seg"], s["y"], bias=s["b"], act=c["act"], pre=s["pre"], status=s["status"])
        return dict(y=s["y"], pre=s["pre"])
    if op == "expert_dgrad":
        hoc.expert_mm_dgrad(s["dy"], s["w"], s["seg"], s["dx"], act=c["act"], pre=s["pre"], status=s["status"])
        return dict(dx=s["dx"])
    if op == "expert_wgrad":
        hoc.expert_mm_wgrad(s["dy"], s["x"], s["seg"], s["dw"], db=s["db"], status=s["status"])
        return dict(dw=s["dw"], db=s["db"])
    if op == "linear":
        hoc.linear(s["x"], s["w"], s["y"], bias=s["b"], act=c["act"], pre=s["pre"], residual=s["r"], status=s["status"])
        return dict(y=s["y"], pre=s["pre"])
    if op == "linear_grad":
        hoc.linear_dgrad(s["dy"], s["w"], s["dx"], status=s["status"])
        hoc.linear_wgrad(s["dy"], s["x"], s["dw"], db=s["db"], status=s["status"])
        return dict(dx=s["dx"], dw=s["dw"], db=s["db"])
    if op == "clip":
        hoc.grad_clip(s["src"], s["dst"], s["max_norm"], s["norm"], s["ws"])
        return dict(norm=s["norm"], out=s["out"])
    hoc.ep_combine_grad(s["dy"], s["rows"], [v.numel() for v in s["rows"]], s["ids"], s["pos"], s["counts"], s["gate"],
                        c["tokens"], c["topk"], c["hidden"], c["experts"], s["drows"], s["dgate"], s["status"])
    return dict(drows=s["drows"], dgate=s["dgate"])


# ------------------------------------------------------------------------------------------------- the least work
def work(case):
    """Bytes of every input read once and every output written once, and the products' operations."""
    c = case
    op = c["op"]
    if op.startswith("expert"):
        n = c["k"] * c["tokens"] * c["topk"]
        mul, inp, out = _gated(c), c["inp"], c["out"]
        touched = sum(1 - (1 - p) ** n for p in _zipf(c["experts"]))  # experts that get a row
        if op == "expert_mm":
            w = mul * out * inp
            rows = inp + out + (mul * out if c["train"] else 0)
        elif op == "expert_dgrad":
            w = out * inp
            rows = out + mul * inp * (2 if c["act"] != "none" else 1)
        else:
            w, rows, touched = out * inp, inp + out, c["experts"]
        return dict(bytes=int(2 * (n * rows + touched * w)), flops=2 * n * w)
    if op == "linear":
        n, inp, out, mul = c["rows"], c["inp"], c["out"], _gated(c)
        rows = inp + out * (1 + c["residual"]) + (mul * out if c["train"] else 0)
        return dict(bytes=2 * (n * rows + mul * out * inp), flops=2 * n * mul * out * inp)
    if op == "linear_grad":
        n, inp, out = c["rows"], c["inp"], c["out"]
        return dict(bytes=2 * (n * (2 * inp + out) + 2 * out * inp), flops=4 * n * out * inp)
    if op == "clip":
        return dict(bytes=2 * c["elems"] * (2 if c["dtype"] == "bfloat16" else 4), flops=3 * c["elems"])
    n = c["k"] * c["tokens"]
    return dict(bytes=2 * n * c["hidden"] * (2 * c["topk"] + 1) + 16 * n * c["topk"], flops=3 * n * c["topk"] * c["hidden"])


# ------------------------------------------------------------------------------------------------- 64 bits
def _exact_act(name, z):
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))  # (1 + tanh v) / 2 = 1 / (1 + exp(-2v))
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "swiglu":
        half = z.shape[-1] // 2
        return z[..., :half] * torch.sigmoid(z[..., :half]) * z[..., half:]
    return z


def exact(case, seed):
    """The operators' definitions in 64 bits, on inputs made as run's are. Activation gradients by automatic
    differentiation of the definition."""
    global own
    c, was = case, own
    own = False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op, f64 = c["op"], torch.float64
    if op.startswith("expert"):
        k, per = c["k"], c["experts"] // c["k"]
        ends = torch.tensor(s["ranges"])
        index = []  # rows of every (rank, expert)
        for d in range(k):
            length = (ends[d, 1:] - ends[d, :-1])
            expert = torch.arange(k * per).remainder(per).repeat_interleave(length)  # of every row that is routed
            index.append([torch.nonzero(expert == e).flatten().to(DEV) for e in range(per)])
        if op == "expert_wgrad":
            dw = [torch.stack([s["dy"][d][i].to(f64).t() @ s["x"][d][i].to(f64) for i in index[d]]) for d in range(k)]
            db = [torch.stack([s["dy"][d][i].to(f64).sum(0) for i in index[d]]) for d in range(k)] if c["bias"] else None
            return dict(dw=dw, db=db)
        one, two = [], []
        for d in range(k):
            src = s["x"][d] if op == "expert_mm" else s["dy"][d]
            width = _gated(c) * (c["out"] if op == "expert_mm" else c["inp"])
            z = torch.zeros(src.shape[0], width if op == "expert_mm" else c["inp"], dtype=f64, device=DEV)
            for e, i in enumerate(index[d]):
                if i.numel():
                    w = s["w"][d][e].to(f64)
                    z[i] = src[i].to(f64) @ (w.t() if op == "expert_mm" else w)
                    if op == "expert_mm" and s["b"] is not None:
                        z[i] += s["b"][d][e].to(f64)
            if op == "expert_mm":
                one.append(_exact_act(c["act"], z))
                two.append(z)
            else:
                one.append(_exact_act_grad(c["act"], s["pre"][d], z) if s["pre"] is not None else z)
        if op == "expert_dgrad":
            return dict(dx=one)
        return dict(y=one, pre=two if c["train"] else None)
    if op == "linear":
        z = s["x"].to(f64) @ s["w"].to(f64).t() + (s["b"].to(f64) if c["bias"] else 0)
        y = _exact_act(c["act"], z) + (s["r"].to(f64) if c["residual"] else 0)
        return dict(y=y, pre=z if c["train"] else None)
    if op == "linear_grad":
        dy = s["dy"].to(f64)
        return dict(dx=dy @ s["w"].to(f64), dw=dy.t() @ s["x"].to(f64), db=dy.sum(0) if c["bias"] else None)
    if op == "clip":
        norm = torch.linalg.vector_norm(s["flat"].to(f64)).reshape(1)
        return dict(norm=norm, out=s["flat"].to(f64) * torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0))
    k, t, j, h = c["k"], c["tokens"], c["topk"], c["hidden"]
    per = c["experts"] // k
    drows = [torch.zeros(v.shape, dtype=f64, device=DEV) for v in s["rows"]]
    dgate = []
    for a in range(k):
        rank, pos = s["ids"][a].long() // per, s["pos"][a].long()
        mine = torch.tensor([s["ranges"][d][(a + 1) * per] - s["ranges"][d][a * per] for d in range(k)])
        base = torch.tensor([s["ranges"][d][a * per] for d in range(k)]) - (mine.cumsum(0) - mine)
        row = pos + base.to(DEV)[rank]
        dg = torch.empty(t, j, dtype=f64, device=DEV)
        dy = s["dy"][a].to(f64)
        for slot in range(j):
            pick = torch.arange(t, device=DEV) * j + slot
            for d in range(k):
                m = torch.nonzero(rank[pick] == d).flatten()
                if m.numel():
                    at = row[pick[m]]
                    drows[d][at] = dy[m] * s["gate"][a][pick[m]].to(f64)[:, None]
                    dg[m, slot] = torch.einsum("rh,rh->r", dy[m], s["rows"][d][at].to(f64))
        dgate.append(dg.reshape(-1))
    return dict(drows=drows, dgate=dgate)


def _exact_act_grad(name, pre, d):
    out = []
    for z, v in zip(pre.split(16384), d.split(16384)):
        z = z.to(torch.float64).requires_grad_()
        y = _exact_act(name, z)
        out.append(torch.autograd.grad(y, z, v)[0])
    return torch.cat(out) if out else pre.to(torch.float64)
