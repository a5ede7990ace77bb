"""The expert block end to end: norm, routing, dispatch (in bf16 and in rows of 8 bits), experts, combine, dropout and the whole
backward pass, against the same block in 64 bits.

Bounds: as for the expert layer (test_gpu_expert_layer.py), every array that is handed on is rounded to bf16 (u = 2^-8), and a
product with a random matrix keeps a relative change within a factor of 3 of itself.  h, n, the logits, pre, h of the experts,
their output and the combine's are rounded before y; the gates depend on the logits, whose rounding changes them by as much.
With rows of 8 bits the reference takes the tokens as they went through the exchange, and the gradient passes them by."""
import pytest
import torch

from collective_communication_schedules_gb300 import hoc
from collective_communication_schedules_gb300.expert_block import ExpertBlock
from tests import block_ref as ref

pytestmark = pytest.mark.gpu
DEV, BF, U, F64 = "cuda", torch.bfloat16, 2.0 ** -8, torch.float64


def problem(k, tokens, hidden, ffn, experts, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = lambda *s, sigma=1.0: (torch.randn(*s, generator=g, device=DEV) * sigma).to(BF)  # noqa: E731
    per = experts // k
    return dict(x=n(k * tokens, hidden), residual=n(k * tokens, hidden), dy=n(k * tokens, hidden),
                norm=(torch.randn(hidden, generator=g, device=DEV) * 0.2 + 1), router=n(experts, hidden, sigma=2 * hidden ** -0.5),
                w_up=[n(per, 2 * ffn, hidden, sigma=hidden ** -0.5) for _ in range(k)],
                w_down=[n(per, hidden, ffn, sigma=ffn ** -0.5) for _ in range(k)],
                bias=torch.randn(experts, generator=g, device=DEV) * 0.05,
                seed=torch.tensor([seed * 1000 + 1, 7], dtype=torch.int64, device=DEV))


def in_64_bits(p, block, ids, residual, sent=None):
    """The block on the ids that it chose; sent: what the tokens were when they got to the experts."""
    leaf = lambda t: t.to(F64).requires_grad_()  # noqa: E731
    x, norm, router = leaf(p["x"]), leaf(p["norm"]), leaf(p["router"])
    up, down = leaf(torch.cat(p["w_up"])), leaf(torch.cat(p["w_down"]))
    h = x + p["residual"].to(F64) if residual else x
    n = h / (h.square().mean(1, keepdim=True) + block.eps).sqrt() * norm
    z = n @ router.t()
    gate = ref.gates(z.cpu(), ids.cpu(), **block.routing).to(DEV)
    if sent is not None:
        n = n + (sent - n).detach()
    out = torch.zeros_like(h)
    for j in range(ids.shape[1]):
        for e in range(router.shape[0]):
            t = torch.nonzero(ids[:, j] == e).flatten()
            a, b = (n[t] @ up[e].t()).chunk(2, 1)
            out = out.index_add(0, t, (a * torch.sigmoid(a) * b) @ down[e].t() * gate[t, j, None])
    if block.drop:
        t = int(block.drop * 65536 + 0.5)
        keep = ref.philox_bits(out.numel(), p["seed"].tolist()).view(out.shape).to(DEV) >= t
        out = out * keep * (65536 / (65536 - t))
    y = h + out
    (y * p["dy"].to(F64)).sum().backward()
    return y, out, x, norm, router, up, down


def near(got, want, roundings, what):
    off = float((got.to(F64) - want).detach().norm() / want.detach().norm())
    assert off <= 3 * U * roundings, f"{what}: off by {off:.3g}"


def outputs(p):
    new = lambda t, dtype=None: torch.empty_like(t, dtype=dtype or t.dtype)  # noqa: E731
    return dict(y=new(p["x"]), dx=new(p["x"]), dnorm=new(p["norm"]), drouter=new(p["router"], torch.float32),
                dup=[new(t, torch.float32) for t in p["w_up"]], ddown=[new(t, torch.float32) for t in p["w_down"]])


def step(block, p, o, residual=True, bias=True, accumulate=False, stream=None):
    block.forward(p["x"], p["norm"], p["router"], p["w_up"], p["w_down"], o["y"], residual=p["residual"] if residual else None,
                  bias=p["bias"] if bias else None, seed=p["seed"], stream=stream)
    block.backward(p["dy"], p["norm"], p["router"], p["w_up"], p["w_down"], o["dx"], o["dnorm"], o["drouter"], o["dup"], o["ddown"],
                   seed=p["seed"], accumulate=accumulate, stream=stream)


CASES = [
    (1, 5, 1, 64, 32, 4, dict(renormalise=False)),
    (2, 100, 2, 128, 64, 8, dict(score="sigmoid", scale=2.5, drop=0.1)),
    (4, 60, 3, 264, 176, 16, dict(groups=4, top_groups=2, wire8=True)),
    (8, 33, 6, 128, 48, 64, dict(score="sigmoid", groups=8, top_groups=4, drop=0.25, wire8=True)),
]


@pytest.mark.parametrize("k,tokens,topk,hidden,ffn,experts,options", CASES)
@pytest.mark.parametrize("residual", [True, False])
def test_block_and_gradients(k, tokens, topk, hidden, ffn, experts, options, residual):
    p = problem(k, tokens, hidden, ffn, experts, seed=k)
    block = ExpertBlock(k, tokens, topk, hidden, ffn, experts, **options)
    o = outputs(p)
    step(block, p, o, residual)
    torch.cuda.synchronize()
    assert block.status.item() == 0
    ids = block.ids.view(k * tokens, topk)
    want_ids, _ = ref.route(block.logits.cpu(), topk, block.routing["score"], p["bias"].cpu(), block.choice["groups"],
                            block.choice["top_groups"] or block.choice["groups"])
    assert torch.equal(ids.cpu(), want_ids)
    sent = None
    if block.wire is not None:
        q, scale = hoc.wire8_views(block.wire, hidden)
        sent = (q.to(torch.float32) * scale.repeat_interleave(128, 1)[:, :hidden]).to(BF).to(F64)
        near(sent, block.n.to(F64), 8 / 3, "rows of 8 bits")  # half a step of e4m3 is 2^-4 of a value: 16 u at most, less on average
    y, out, x, norm, router, up, down = in_64_bits(p, block, ids, residual, sent)
    near(o["y"], y, 6, "y")
    h = p["x"].to(F64) + p["residual"].to(F64) if residual else p["x"].to(F64)
    off = float((o["y"].to(F64) - h - out).detach().norm())  # the block's own part, beside the roundings of h and y
    assert off <= 3 * U * 7 * float(out.detach().norm()) + 2 * U * float(y.detach().norm())
    near(o["dx"], x.grad, 8, "dx")
    near(o["dnorm"], norm.grad, 10, "dnorm")
    near(torch.cat(o["dup"]), up.grad, 8, "dw_up")
    near(torch.cat(o["ddown"]), down.grad, 7, "dw_down")
    if topk > 1 or not block.routing["renormalise"]:
        near(o["drouter"], router.grad, 12, "drouter")  # (differences of gate gradients)
    first = [o["dnorm"].clone(), o["drouter"].clone()] + [t.clone() for t in o["dup"] + o["ddown"]]
    block.backward(p["dy"], p["norm"], p["router"], p["w_up"], p["w_down"], o["dx"], o["dnorm"], o["drouter"], o["dup"], o["ddown"],
                   seed=p["seed"], accumulate=True)
    for a, b in zip(first, [o["dnorm"], o["drouter"]] + o["dup"] + o["ddown"]):
        assert torch.equal(2 * a, b)


def test_block_in_a_graph_on_a_stream_of_its_own():
    """A captured step follows its inputs: tokens, seed, bias."""
    k, tokens, topk, hidden, ffn, experts = 2, 64, 2, 128, 64, 8
    p, q = problem(k, tokens, hidden, ffn, experts, 1), problem(k, tokens, hidden, ffn, experts, 2)
    block = ExpertBlock(k, tokens, topk, hidden, ffn, experts, score="sigmoid", drop=0.2, wire8=True)
    o = outputs(p)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(block, p, o)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step(block, p, o)
    for name in ("x", "residual", "dy", "bias", "seed"):
        p[name].copy_(q[name])
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    again = outputs(p)
    step(block, p, again)
    for name in ("y", "dx", "dnorm", "drouter"):
        assert torch.equal(o[name], again[name]), name
    for a, b in zip(o["dup"] + o["ddown"], again["dup"] + again["ddown"]):
        assert torch.equal(a, b)


def test_two_blocks_at_once_on_two_streams():
    """Blocks share nothing: their captured steps run side by side and give what they give alone."""
    k, tokens, topk, hidden, ffn, experts = 2, 300, 2, 256, 128, 8
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    ps = [problem(k, tokens, hidden, ffn, experts, 3 + i) for i in range(2)]
    blocks = [ExpertBlock(k, tokens, topk, hidden, ffn, experts, drop=0.1) for _ in range(2)]
    alone = [outputs(p) for p in ps]
    for b, p, o in zip(blocks, ps, alone):
        step(b, p, o)
    torch.cuda.synchronize()
    both, graphs = [outputs(p) for p in ps], []
    for b, p, o, s in zip(blocks, ps, both, streams):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            step(b, p, o)
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for a, o in zip(alone, both):
        for name in ("y", "dx", "dnorm", "drouter"):
            assert torch.equal(a[name], o[name]), name


def test_tokens_without_an_expert_pass_by():
    """A bias that closes all experts but one for top-2: half of the slots are dropped, and the block still adds up."""
    k, tokens, hidden, ffn, experts = 2, 40, 128, 64, 4
    p = problem(k, tokens, hidden, ffn, experts, 5)
    p["bias"][:] = -float("inf")
    p["bias"][2] = 0.0
    block = ExpertBlock(k, tokens, 2, hidden, ffn, experts, renormalise=False)
    o = outputs(p)
    step(block, p, o)
    torch.cuda.synchronize()
    assert block.status.item() == 0
    ids = block.ids.view(-1, 2)
    assert bool((ids[:, 0] == 2).all()) and bool((ids[:, 1] == -1).all())
    y, out, x, norm, router, up, down = in_64_bits(p, block, ids, True)
    near(o["y"], y, 6, "y")
    near(o["dx"], x.grad, 8, "dx")
    near(torch.cat(o["dup"]), up.grad, 8, "dw_up")
    p["bias"][2] = -float("inf")  # and none at all
    step(block, p, o)
    torch.cuda.synchronize()
    assert bool((block.ids == -1).all())
    h = (p["x"].float() + p["residual"].float()).to(BF)
    assert torch.equal(o["y"], h) and torch.equal(o["dx"], p["dy"]) and bool((o["drouter"] == 0).all())


def test_block_of_no_tokens():
    p = problem(2, 0, 64, 32, 4, 1)
    block = ExpertBlock(2, 0, 2, 64, 32, 4, drop=0.1, wire8=True)
    o = outputs(p)
    step(block, p, o)
    torch.cuda.synchronize()
    assert block.status.item() == 0
    for t in [o["dnorm"], o["drouter"]] + o["dup"] + o["ddown"]:
        assert bool((t == 0).all())


def test_block_refuses():
    with pytest.raises(ValueError):
        ExpertBlock(2, 8, 1, 64, 32, 3)
    block = ExpertBlock(1, 8, 1, 64, 32, 2, drop=0.5)
    p = problem(1, 8, 64, 32, 2, 1)
    o = outputs(p)
    with pytest.raises(ValueError):
        block.forward(p["x"], p["norm"], p["router"], p["w_up"], p["w_down"], o["y"])
    with pytest.raises(ValueError):
        block.layer.__class__(1, 8, 1, 64, 32, 2, wire8=True).forward([p["x"]], [block.ids], [block.gate], p["w_up"], p["w_down"],
                                                                      [o["y"]])
