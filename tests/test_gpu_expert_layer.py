"""The expert layer end to end: dispatch, gated products, combine, the whole backward pass and clipping, against the
same layer in 64 bits.

Bounds: every array that is handed on is rounded to bf16 (unit roundoff u = 2^-8), which changes it by at most u in
norm; a product with a random matrix keeps a relative change within a factor of 3 of itself (norm of the matrix
against its mean gain).  Results are therefore within 3 u times the number of roundings before them: y 4 (pre, h, out
and y, with pre exact in the forward pass), gradients up to 6."""
import pytest
import torch

from collective_communication_schedules_gb300 import hoc
from collective_communication_schedules_gb300.expert_layer import ExpertLayer

pytestmark = pytest.mark.gpu
DEV, BF, U = "cuda", torch.bfloat16, 2.0 ** -8


def problem(k, tokens, topk, hidden, ffn, experts, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = lambda *s, sigma=1.0: (torch.randn(*s, generator=g, device=DEV) * sigma).to(BF)  # noqa: E731
    per = experts // k
    return dict(
        ids=[torch.rand(tokens, experts, generator=g, device=DEV).topk(topk, 1).indices.to(torch.int32).flatten().contiguous()
             for _ in range(k)],
        x=[n(tokens, hidden) for _ in range(k)], dy=[n(tokens, hidden) for _ in range(k)],
        gate=[torch.rand(tokens * topk, generator=g, device=DEV) for _ in range(k)],
        w_up=[n(per, 2 * ffn, hidden, sigma=hidden ** -0.5) for _ in range(k)],
        w_down=[n(per, hidden, ffn, sigma=ffn ** -0.5) for _ in range(k)])


def in_64_bits(p, experts):
    """The layer and its gradients by automatic differentiation."""
    leaf = lambda ts: [t.double().requires_grad_() for t in ts]  # noqa: E731
    x, gate, up, down = leaf(p["x"]), leaf(p["gate"]), leaf(p["w_up"]), leaf(p["w_down"])
    per = up[0].shape[0]
    loss, ys = 0, []
    for s in range(len(x)):
        tokens = x[s].shape[0]
        topk = p["ids"][s].numel() // tokens
        ids = p["ids"][s].view(tokens, topk)
        y = torch.zeros_like(x[s])
        for e in range(experts):
            t, j = torch.nonzero(ids == e, as_tuple=True)
            a, b = (x[s][t] @ up[e // per][e % per].t()).chunk(2, 1)
            o = (a * torch.sigmoid(a) * b) @ down[e // per][e % per].t()
            y = y.index_add(0, t, o * gate[s][t * topk + j][:, None])
        ys.append(y)
        loss = loss + (y * p["dy"][s].double()).sum()
    loss.backward()
    return ys, x, gate, up, down


def near(got, want, roundings, what):
    got, want = torch.cat([t.double().flatten() for t in got]), torch.cat([t.double().flatten() for t in want])
    off = float((got - want).detach().norm() / want.detach().norm())
    assert off <= 3 * U * roundings, f"{what}: off by {off:.3g}"


@pytest.mark.parametrize("k,tokens,topk,hidden,ffn,experts", [
    (1, 5, 1, 64, 32, 2), (2, 100, 2, 128, 64, 8), (4, 77, 3, 264, 176, 16), (8, 33, 6, 72, 48, 64), (2, 40, 2, 50, 30, 4),
])
def test_layer_and_gradients(k, tokens, topk, hidden, ffn, experts):
    p = problem(k, tokens, topk, hidden, ffn, experts, seed=k)
    layer = ExpertLayer(k, tokens, topk, hidden, ffn, experts)
    new = lambda ts, dtype=None: [torch.empty_like(t, dtype=dtype or t.dtype) for t in ts]  # noqa: E731
    y, dx, dgate = new(p["x"]), new(p["x"]), new(p["gate"])
    dup, ddown = new(p["w_up"], torch.float32), new(p["w_down"], torch.float32)
    layer.forward(p["x"], p["ids"], p["gate"], p["w_up"], p["w_down"], y)
    layer.backward(p["dy"], p["ids"], p["gate"], p["w_up"], p["w_down"], dx, dgate, dup, ddown)
    torch.cuda.synchronize()
    assert layer.status.item() == 0
    ys, x, gate, up, down = in_64_bits(p, experts)
    near(y, ys, 4, "y")
    near(dx, [t.grad for t in x], 6, "dx")
    near(dgate, [t.grad for t in gate], 4, "dgate")
    near(dup, [t.grad for t in up], 6, "dw_up")
    near(ddown, [t.grad for t in down], 5, "dw_down")
    first = [t.clone() for t in dup + ddown]
    layer.backward(p["dy"], p["ids"], p["gate"], p["w_up"], p["w_down"], dx, dgate, dup, ddown, accumulate=True)
    for a, b in zip(first, dup + ddown):
        assert torch.equal(2 * a, b)
    # clip what the step made, over all ranks' weights
    norm = torch.empty(1, device=DEV)
    with hoc.TensorList(dup + ddown) as grads:
        ws = torch.empty(hoc.grad_workspace(grads), dtype=torch.int32, device=DEV)
        hoc.grad_clip(grads, grads, 1.0, norm, ws)
        want = float(torch.cat([2 * t.double().flatten() for t in first]).norm())
        assert abs(norm.item() - want) <= 1e-5 * want
        after = float(torch.cat([t.double().flatten() for t in dup + ddown]).norm())
        assert abs(after - min(1.0, want)) <= 1e-4


def test_layer_in_a_graph_follows_its_inputs():
    k, tokens, topk, hidden, ffn, experts = 2, 64, 2, 128, 64, 8
    p, q = problem(k, tokens, topk, hidden, ffn, experts, 1), problem(k, tokens, topk, hidden, ffn, experts, 2)
    layer = ExpertLayer(k, tokens, topk, hidden, ffn, experts)
    y = [torch.empty_like(t) for t in p["x"]]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    args = (p["x"], p["ids"], p["gate"], p["w_up"], p["w_down"], y)
    with torch.cuda.stream(s):
        layer.forward(*args)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        layer.forward(*args)
    for name in ("x", "ids", "gate"):
        for a, b in zip(p[name], q[name]):
            a.copy_(b)
    g.replay()
    torch.cuda.synchronize()
    again = [torch.empty_like(t) for t in y]
    layer.forward(q["x"], q["ids"], q["gate"], p["w_up"], p["w_down"], again)
    for a, b in zip(y, again):
        assert torch.equal(a, b)


def test_a_receive_buffer_that_is_too_small():
    """Rows past the capacity are dropped by the dispatch (status bit 0) and by everything after it."""
    k, tokens, topk, hidden, ffn, experts = 2, 64, 2, 64, 32, 4
    p = problem(k, tokens, topk, hidden, ffn, experts, 3)
    layer = ExpertLayer(k, tokens, topk, hidden, ffn, experts, capacity=50)
    y, dx, dgate = ([torch.empty_like(t) for t in p[n]] for n in ("x", "x", "gate"))
    dup, ddown = ([torch.empty_like(t) for t in p[n]] for n in ("w_up", "w_down"))
    layer.forward(p["x"], p["ids"], p["gate"], p["w_up"], p["w_down"], y)
    torch.cuda.synchronize()
    assert layer.status.item() & 1
    layer.backward(p["dy"], p["ids"], p["gate"], p["w_up"], p["w_down"], dx, dgate, dup, ddown)
    torch.cuda.synchronize()
    assert layer.status.item() & 4 == 0
    for t in y + dx + dgate + dup + ddown:
        assert bool(torch.isfinite(t).all())


@pytest.mark.parametrize("k,tokens,topk,experts,names", [(2, 40, 2, 2, "one"), (4, 30, 3, 4, "any"), (2, 25, 4, 4, "one")])
def test_tokens_that_name_an_expert_twice(k, tokens, topk, experts, names):
    """Nothing forbids it: every pair is a row of its own, and by default there is room for all of them at any rank."""
    hidden, ffn = 64, 32
    p = problem(k, tokens, topk, hidden, ffn, experts, 5)
    g = torch.Generator(device=DEV).manual_seed(9)
    p["ids"] = [torch.ones(tokens * topk, dtype=torch.int32, device=DEV) if names == "one" else
                torch.randint(0, experts, (tokens * topk,), generator=g, device=DEV, dtype=torch.int32) for _ in range(k)]
    layer = ExpertLayer(k, tokens, topk, hidden, ffn, experts)
    y, dx, dgate = ([torch.empty_like(t) for t in p[n]] for n in ("x", "x", "gate"))
    dup, ddown = ([torch.empty_like(t) for t in p[n]] for n in ("w_up", "w_down"))
    layer.forward(p["x"], p["ids"], p["gate"], p["w_up"], p["w_down"], y)
    layer.backward(p["dy"], p["ids"], p["gate"], p["w_up"], p["w_down"], dx, dgate, dup, ddown)
    torch.cuda.synchronize()
    assert layer.status.item() == 0
    ys, x, gate, up, down = in_64_bits(p, experts)
    near(y, ys, 4, "y")
    near(dx, [t.grad for t in x], 6, "dx")
    near(dgate, [t.grad for t in gate], 4, "dgate")
    near(dup, [t.grad for t in up], 7, "dw_up")  # (weight gradients are rounded to bf16 here: one more than above)
    near(ddown, [t.grad for t in down], 6, "dw_down")


def each_near(got, want, bound, what):
    """Every row of `got` (every expert's matrix) is near `want`'s, by that row's own norm; rows of zeros are exact."""
    for s, (a, b) in enumerate(zip(got, want)):
        a, b = a.double().flatten(1), b.detach().double().flatten(1)
        off, size = (a - b).norm(dim=1), b.norm(dim=1)
        bad = off > bound * size
        assert not bool(bad.any()), f"{what}: row {int(bad.nonzero()[0])} of rank {s} is off by {float((off / size)[bad].max()):.3g}"


@pytest.mark.parametrize("k,tokens,topk,hidden,ffn,experts", [
    (1, 5, 1, 64, 32, 2), (2, 100, 2, 128, 64, 8), (4, 77, 3, 264, 176, 16), (8, 33, 6, 72, 48, 64), (2, 40, 2, 50, 30, 4),
])
def test_every_token_and_every_expert(k, tokens, topk, hidden, ffn, experts):
    """The bounds of the whole arrays hold row by row too, twice as wide where a row is one token (50 to 264 values; an
    expert's matrix has thousands), so that one missing pair or one row from a neighbour's range is seen: a pair is at
    least 1 / sqrt(topk) of its token on average.  dgate is <o, dy>: o is off by at most 9 u of its norm (three roundings)
    in a direction that has nothing to do with dy, which leaves 9 u |o| |dy| / sqrt(hidden) on average; 6 times that."""
    p = problem(k, tokens, topk, hidden, ffn, experts, seed=20 + k)
    layer = ExpertLayer(k, tokens, topk, hidden, ffn, experts)
    y, dx, dgate = ([torch.empty_like(t) for t in p[n]] for n in ("x", "x", "gate"))
    dup, ddown = ([torch.empty_like(t, dtype=torch.float32) for t in p[n]] for n in ("w_up", "w_down"))
    layer.forward(p["x"], p["ids"], p["gate"], p["w_up"], p["w_down"], y)
    layer.backward(p["dy"], p["ids"], p["gate"], p["w_up"], p["w_down"], dx, dgate, dup, ddown)
    torch.cuda.synchronize()
    assert layer.status.item() == 0
    ys, x, gate, up, down = in_64_bits(p, experts)
    each_near(y, ys, 2 * 3 * 4 * U, "y")
    each_near(dx, [t.grad for t in x], 2 * 3 * 6 * U, "dx")
    each_near(dup, [t.grad for t in up], 3 * 6 * U, "dw_up")
    each_near(ddown, [t.grad for t in down], 3 * 5 * U, "dw_down")
    w_up, w_down = torch.cat(p["w_up"]).double(), torch.cat(p["w_down"]).double()
    for s in range(k):
        e, t = p["ids"][s].long(), torch.arange(tokens * topk, device=DEV) // topk
        a, b = torch.einsum("nfh,nh->nf", w_up[e], p["x"][s].double()[t]).chunk(2, 1)
        o = torch.einsum("nhf,nf->nh", w_down[e], a * torch.sigmoid(a) * b)
        scale = o.norm(dim=1) * p["dy"][s].double()[t].norm(dim=1) / hidden ** 0.5
        bad = (dgate[s].double() - gate[s].grad).abs() > 6 * 9 * U * scale
        assert not bool(bad.any()), f"dgate of pair {int(bad.nonzero()[0])} of source {s}"


def test_a_layer_is_used_at_once_on_a_stream_of_its_own():
    """What the constructor fills is there when it returns, whatever the stream that it was made on is doing."""
    k, tokens, topk, hidden, ffn, experts = 2, 64, 2, 128, 64, 8
    p = problem(k, tokens, topk, hidden, ffn, experts, 6)
    new = lambda n: [torch.empty_like(t) for t in p[n]]  # noqa: E731
    y, dx, dgate, dup, ddown = (new(n) for n in ("x", "x", "gate", "w_up", "w_down"))
    side = torch.cuda.Stream()
    before = ExpertLayer(k, tokens, topk, hidden, ffn, experts)  # memory for the second, with something in it
    before.forward(p["x"], p["ids"], p["gate"], p["w_up"], p["w_down"], y)  # (a kernel's first launch may wait)
    before.backward(p["dy"], p["ids"], p["gate"], p["w_up"], p["w_down"], dx, dgate, dup, ddown)
    before.status.fill_(7)
    before.ones[0].fill_(7.0)
    del before
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # cycles: about a tenth of a second
    layer = ExpertLayer(k, tokens, topk, hidden, ffn, experts)
    layer.forward(p["x"], p["ids"], p["gate"], p["w_up"], p["w_down"], y, stream=side)
    layer.backward(p["dy"], p["ids"], p["gate"], p["w_up"], p["w_down"], dx, dgate, dup, ddown, stream=side)
    side.synchronize()
    got = [t.clone() for t in y + dx + dgate + dup + ddown]
    torch.cuda.synchronize()
    assert layer.status.item() == 0
    layer.forward(p["x"], p["ids"], p["gate"], p["w_up"], p["w_down"], y)
    layer.backward(p["dy"], p["ids"], p["gate"], p["w_up"], p["w_down"], dx, dgate, dup, ddown)
    for a, b in zip(got, y + dx + dgate + dup + ddown):
        assert torch.equal(a, b)
