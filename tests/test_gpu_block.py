"""The operators around the dispatch on the GPU, against their formulas in 64 bits.

Bounds.  A rounding to a type is off by half a step of it, eps / 2 of the value.  The norm's mean square is a sum of at most
32 terms a thread, then 10 levels of a tree, in binary32: 43 * 2^-24 of itself, half of that in the square root's reciprocal
(which is off by 2 units, 4 * 2^-24), two products: NORM = 2^-19 is above all of it.  The gradient's mean of d w h is off by
(45 + 3) * 2^-24 of the sum of its terms' sizes, so an element of dx by 2^-18 of what block_ref.norm_grad gives as its terms."""
import math

import pytest
import torch

from collective_communication_schedules_gb300 import hoc
from tests import block_ref as ref

pytestmark = pytest.mark.gpu
DEV, BF, F32, F64 = "cuda", torch.bfloat16, torch.float32, torch.float64
NORM = 2.0 ** -19


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def rows_of(g, rows, width, dtype, pad=0, offset=0, sigma=1.0):
    """Rows of a wider buffer, `offset` elements behind its start; and the buffer."""
    flat = (torch.randn(rows * (width + pad) + offset + 8, generator=g, device=DEV) * sigma).to(dtype)
    return flat[offset: offset + rows * (width + pad)].view(rows, width + pad)[:, :width], flat


class Out:
    """An output of `rows` rows inside a buffer of 7s; check() sees that nothing else was written."""

    def __init__(self, rows, width, dtype, pad=0, offset=0):
        self.flat = torch.full((rows * (width + pad) + offset + 8,), 7, device=DEV).to(dtype)
        self.t = self.flat[offset: offset + rows * (width + pad)].view(rows, width + pad)[:, :width]
        self.rows, self.width, self.pad, self.offset = rows, width, pad, offset

    def check(self):
        mine = torch.zeros_like(self.flat, dtype=torch.bool)
        mine[self.offset: self.offset + self.rows * (self.width + self.pad)].view(self.rows, self.width + self.pad)[:, :self.width] = True
        assert bool((self.flat[~mine] == 7).all()), "written outside the rows"


def within(got, want, bound, what):
    off = (got.to(F64).cpu() - want.cpu()).abs()
    bad = ~(off <= bound.cpu())
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((off / bound.cpu().clamp(min=1e-300))[bad].max()):.3g} of the bound"


SHAPES = [  # rows, width, pad, offset
    (1, 1, 0, 0), (1, 8, 0, 0), (3, 7, 0, 0), (5, 64, 0, 0), (9, 256, 0, 0), (17, 264, 0, 0), (2, 1001, 0, 0), (33, 1024, 8, 0),
    (4, 1408, 0, 8), (7, 2048, 0, 0), (300, 2048, 64, 0), (6, 4096, 0, 0), (5, 4096, 1, 0), (3, 5560, 0, 1), (2, 8192, 0, 0),
    (2, 9000, 0, 0), (3, 16384, 0, 0), (1, 32768, 0, 0), (2, 32767, 0, 0), (1500, 40, 0, 0), (2600, 129, 3, 0), (1, 4097, 5, 3),
]


@pytest.mark.parametrize("dtype,wdtype", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("rows,width,pad,offset", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm(rows, width, pad, offset, dtype, wdtype, residual):
    g = gen(rows * 7 + width)
    x, _ = rows_of(g, rows, width, dtype, pad, offset)
    r = rows_of(g, rows, width, dtype, pad, offset, sigma=3.0)[0] if residual else None
    w = (torch.randn(width, generator=g, device=DEV) * 0.3 + 1).to(wdtype)
    h, y = Out(rows, width, dtype, pad, offset), Out(rows, width, dtype, pad, offset)
    wire = torch.full((rows, hoc.wire8_bytes(width)), 77, dtype=torch.uint8, device=DEV)
    hoc.rms_norm(x, w, y.t, eps=1e-5, residual=r, h=h.t if residual else None, wire=wire)
    torch.cuda.synchronize()
    wh, wy = ref.norm(x.cpu(), None if r is None else r.cpu(), w.cpu(), 1e-5)
    if residual:
        assert torch.equal(h.t.cpu(), wh)
        h.check()
    y.check()
    within(y.t, wy, (ref.half_step(dtype) + NORM) * wy.abs(), "y")
    check_wire(wire, wy, width)
    only = torch.full_like(wire, 77)
    hoc.rms_norm(x, w, None, eps=1e-5, residual=r, wire=only)
    assert torch.equal(wire, only)
    y2 = torch.empty_like(y.t)
    hoc.rms_norm(x, w, y2, eps=1e-5, residual=r)
    assert torch.equal(y.t, y2)


def check_wire(wire, wy, width):
    """Scales are off by the norm's error and two roundings; a value by half a step of e4m3, 2^-4 of it or, below the smallest
    normal number 2^-6, 2^-10."""
    q, scale = hoc.wire8_views(wire, width)
    groups = scale.shape[1]
    wide = torch.zeros(wy.shape[0], groups * 128, dtype=F64)
    wide[:, :width] = wy
    want = (wide.view(wy.shape[0], groups, 128).abs().amax(2) / 448).clamp(min=2.0 ** -100)
    within(scale, want, want * 2 * NORM, "scale")
    s = scale.cpu().to(F64).repeat_interleave(128, 1)[:, :width]
    within(q.to(F32).to(F64).cpu() * s, wy, torch.maximum((2.0 ** -4 + 2 * NORM) * wy.abs(), s * 2.0 ** -10 + 2 * NORM * wy.abs()), "q")
    n, at = hoc.wire8_bytes(width), -(-width // 16) * 16
    rest = [c for c in range(n) if width <= c < at or c >= at + 4 * groups]
    assert bool((wire[:, rest] == 77).all()), "bytes that hold nothing were written"


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("width", [64, 1001, 2048])
def test_norm_in_place(dtype, width):
    g = gen(3)
    x, r = rows_of(g, 50, width, dtype)[0], rows_of(g, 50, width, dtype)[0]
    w = torch.ones(width, device=DEV)
    h, y = torch.empty_like(x), torch.empty_like(x)
    hoc.rms_norm(x, w, y, eps=1e-6, residual=r, h=h)
    a, b = x.clone(), r.clone()
    hoc.rms_norm(a, w, a, eps=1e-6, residual=b, h=b)  # y into x, h into the residual
    assert torch.equal(a, y) and torch.equal(b, h)
    a, out = x.clone(), torch.empty_like(x)
    hoc.rms_norm(a, w, out, eps=1e-6, residual=r, h=a)
    assert torch.equal(a, h) and torch.equal(out, y)
    b = r.clone()
    hoc.rms_norm(x, w, b, eps=1e-6, residual=b)
    assert torch.equal(b, y)


def test_norm_of_rows_that_are_not_ordinary():
    """Zeros, a row of tiny values, infinities and NaN: each row for itself."""
    width = 256
    x = torch.randn(6, width, generator=gen(1), device=DEV)
    x[1] = 0
    x[2] *= 1e-30
    x[3, 5] = float("inf")
    x[4, 130] = float("nan")
    w = torch.ones(width, device=DEV)
    for t in (x, x.to(BF)):
        y = torch.empty_like(t)
        wire = torch.zeros(6, hoc.wire8_bytes(width), dtype=torch.uint8, device=DEV)
        hoc.rms_norm(t, w, y, eps=1e-6, wire=wire)
        q, scale = hoc.wire8_views(wire, width)
        assert bool((y[1] == 0).all()) and bool((q[1].float() == 0).all()) and bool((scale[1] == 2.0 ** -100).all())
        want = t.double() / (t.double().square().mean(1, keepdim=True) + 1e-6).sqrt()
        for row in (0, 2, 5):
            within(y[row], want[row], (ref.half_step(t.dtype) + NORM) * want[row].abs() + 1e-45, f"row {row}")
        assert bool(y[3, 5].isnan()) and bool((y[3, :5] == 0).all())
        assert bool(y[4].isnan().all()) and bool(q[4].float().isnan().all())
        assert bool(torch.isfinite(scale).all())


GRAD_SHAPES = [
    (1, 1, 0, 0), (1, 8, 0, 0), (3, 7, 0, 0), (5, 64, 0, 0), (64, 256, 0, 0), (2, 1001, 0, 0), (33, 1024, 8, 0), (509, 1408, 0, 0),
    (7, 2048, 0, 0), (2500, 2048, 0, 0), (6, 4096, 0, 0), (5, 4096, 1, 0), (3, 5560, 0, 1), (700, 8192, 0, 0), (2, 9000, 0, 0),
    (3, 16384, 0, 0), (1, 32768, 0, 0), (2, 32767, 0, 0), (3000, 40, 0, 0), (2600, 129, 3, 0),
]


@pytest.mark.parametrize("dtype,wdtype,dwdtype", [(BF, F32, F32), (BF, BF, BF), (F32, F32, F32), (F32, BF, BF)])
@pytest.mark.parametrize("rows,width,pad,offset", GRAD_SHAPES)
@pytest.mark.parametrize("two,stream", [(False, False), (True, True), (False, True)])
def test_norm_gradient(rows, width, pad, offset, dtype, wdtype, dwdtype, two, stream):
    g = gen(rows + width)
    dy, h = (rows_of(g, rows, width, dtype, pad, offset)[0] for _ in range(2))
    dy2 = rows_of(g, rows, width, dtype, pad, offset)[0] if two else None
    dres = rows_of(g, rows, width, dtype, pad, offset)[0] if stream else None
    w = (torch.randn(width, generator=g, device=DEV) * 0.3 + 1).to(wdtype)
    dx, dw = Out(rows, width, dtype, pad, offset), Out(1, width, dwdtype)
    dwt = dw.t.view(-1)
    ws = torch.full((hoc.rms_norm_workspace(rows, width),), -1, dtype=torch.int32, device=DEV)
    hoc.rms_norm_grad(dy, h, w, dx.t, eps=1e-5, dy2=dy2, dres=dres, dw=dwt, workspace=ws)
    torch.cuda.synchronize()
    cpu = lambda t: None if t is None else t.cpu()  # noqa: E731
    want, terms, ww, wterms = ref.norm_grad(dy.cpu(), cpu(dy2), h.cpu(), w.cpu(), 1e-5, cpu(dres))
    dx.check()
    dw.check()
    within(dx.t, want, ref.half_step(dtype) * want.abs() + 2.0 ** -18 * terms, "dx")
    # a CTA's rows one after the other (152 CTAs at least, where there are rows for them), then its like, in order
    adds = 64 + math.ceil(rows / 152) + 32
    within(dwt, ww, ref.half_step(dwdtype) * ww.abs() + adds * 2.0 ** -24 * wterms + 1e-30, "dw")
    # added to what is there, and without a weight gradient
    first = dwt.to(F64)
    again = torch.empty_like(dx.t)
    hoc.rms_norm_grad(dy, h, w, again, eps=1e-5, dy2=dy2, dres=dres, dw=dwt, accumulate=True, workspace=ws)
    within(dwt, 2 * first.cpu(), 2 * (ref.half_step(dwdtype) * 2 + 2.0 ** -23) * first.abs().cpu() + 1e-30, "dw added")
    assert torch.equal(again, dx.t)
    again = torch.empty_like(dx.t)
    hoc.rms_norm_grad(dy, h, w, again, eps=1e-5, dy2=dy2, dres=dres)
    assert torch.equal(again, dx.t)


@pytest.mark.parametrize("width", [64, 1001, 2048, 16384])
def test_norm_gradient_in_place(width):
    g = gen(4)
    dy, dy2, h, dres = (rows_of(g, 400, width, BF)[0] for _ in range(4))
    w = torch.ones(width, device=DEV)
    ws = torch.empty(hoc.rms_norm_workspace(400, width), dtype=torch.int32, device=DEV)
    dx, dw = torch.empty_like(dy), torch.empty(width, device=DEV)
    hoc.rms_norm_grad(dy, h, w, dx, eps=1e-6, dy2=dy2, dres=dres, dw=dw, workspace=ws)
    for name in ("dy", "dy2", "h", "dres"):
        t = dict(dy=dy, dy2=dy2, h=h, dres=dres)
        t[name] = t[name].clone()
        dw2 = torch.empty_like(dw)
        hoc.rms_norm_grad(t["dy"], t["h"], w, t[name], eps=1e-6, dy2=t["dy2"], dres=t["dres"], dw=dw2, workspace=ws)
        assert torch.equal(t[name], dx) and torch.equal(dw2, dw), name


def test_norm_gradient_by_differences():
    """<y, dy> changes by <dx, step> along a step of x, and by <dw, step> along one of the weight."""
    rows, width, eps = 20, 192, 1e-3
    g = gen(9)
    x, dy, step = (torch.randn(rows, width, generator=g, device=DEV) for _ in range(3))
    w, wstep = torch.rand(width, generator=g, device=DEV) + 0.5, torch.randn(width, generator=g, device=DEV)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ws = torch.empty(hoc.rms_norm_workspace(rows, width), dtype=torch.int32, device=DEV)
    hoc.rms_norm_grad(dy, x, w, dx, eps=eps, dw=dw, workspace=ws)
    f = lambda a, b: float((ref.norm(a.double().cpu(), None, b.double().cpu(), eps)[1] * dy.double().cpu()).sum())  # noqa: E731
    d = 1e-5
    for slope, grad, s in ((lambda t: f(x.double() + t * step.double(), w.double()), dx, step),
                           (lambda t: f(x.double(), w.double() + t * wstep.double()), dw, wstep)):
        want = (slope(d) - slope(-d)) / (2 * d)
        got = float((grad.double() * s.double()).sum())
        # differences are off by d^2 times third derivatives (of order 1 a value) and by 64-bit noise over d
        assert abs(got - want) <= 1e-5 * float((grad.double() * s.double()).abs().sum())


def test_no_rows_leave_a_weight_gradient_of_zeros():
    x = torch.empty(0, 128, dtype=BF, device=DEV)
    w, dw = torch.ones(128, device=DEV), torch.full((128,), 5.0, device=DEV)
    ws = torch.empty(hoc.rms_norm_workspace(0, 128), dtype=torch.int32, device=DEV)
    hoc.rms_norm(x, w, x, eps=1e-6)
    hoc.rms_norm_grad(x, x, w, x, eps=1e-6, dw=dw, accumulate=True, workspace=ws)
    assert bool((dw == 5).all())
    hoc.rms_norm_grad(x, x, w, x, eps=1e-6, dw=dw, workspace=ws)
    assert bool((dw == 0).all())


# ------------------------------------------------------------------------------------------------- rows of 8 bits
@pytest.mark.parametrize("width", [1, 7, 64, 72, 128, 129, 1001, 2048, 4096])
@pytest.mark.parametrize("caps,counts", [
    ([5], [[2, 1]]), ([5], [[0, 0]]), ([4, 0, 9], [[1, 3], [0, 0], [5, 9]]), ([300] * 4, [[100, 50], [0, 1], [299, 1], [0, 0]]),
    ([0, 0], [[3, 3], [0, 0]]), ([50] * 16, [[i, i] for i in range(16)]),
])
def test_widen(width, caps, counts):
    g = gen(width)
    k, n = len(caps), hoc.wire8_bytes(width)
    wire = [torch.randint(0, 256, (c, n), generator=g, device=DEV, dtype=torch.uint8) for c in caps]
    for t in wire:
        q, scale = hoc.wire8_views(t, width)
        q.view(torch.uint8)[q.float().isnan()] = 0
        scale.copy_(torch.rand(scale.shape, generator=g, device=DEV) * 2.0 ** torch.randint(-20, 20, scale.shape, generator=g, device=DEV))
    seg = torch.zeros(k, 3, dtype=torch.int64, device=DEV)
    seg[:, 1:] = torch.tensor(counts, device=DEV).cumsum(1)
    ys = [Out(c, width, BF) for c in caps]
    hoc.expert_widen(wire, seg, [o.t for o in ys])
    torch.cuda.synchronize()
    for d in range(k):
        rows = min(caps[d], sum(counts[d]))
        q, scale = hoc.wire8_views(wire[d], width)
        want = (q[:rows].double() * scale[:rows].double().repeat_interleave(128, 1)[:, :width]).float().to(BF)  # exact, then rounded once
        assert torch.equal(ys[d].t[:rows], want)
        assert bool((ys[d].t[rows:] == 7).all()), "rows behind the last were written"
        ys[d].check()


@pytest.mark.parametrize("k,caps", [(1, [4]), (3, [5, 0, 9]), (16, [2] * 16), (2, [0, 0])])
def test_widen_turns_the_counts_of_its_rows(k, caps):
    """Counts in elements of the rows that were moved become counts in elements of y."""
    width = 200
    n = hoc.wire8_bytes(width)
    wire = [torch.zeros(c, n, dtype=torch.uint8, device=DEV) for c in caps]
    rows = torch.arange(k * k, device=DEV).view(k, k) * 1000003
    counts = rows * (n // 2)
    hoc.expert_widen(wire, torch.zeros(k, 2, dtype=torch.int64, device=DEV), [torch.empty(c, width, dtype=BF, device=DEV) for c in caps],
                     counts=counts)
    assert torch.equal(counts, rows * width)


def test_widen_of_every_8_bit_value():
    wire = torch.zeros(1, hoc.wire8_bytes(256), dtype=torch.uint8, device=DEV)
    wire[0, :256] = torch.arange(256, device=DEV).to(torch.uint8)
    q, scale = hoc.wire8_views(wire, 256)
    scale.fill_(1.0)
    y = torch.empty(1, 256, dtype=BF, device=DEV)
    hoc.expert_widen([wire], torch.tensor([[0, 1]], device=DEV), [y])
    want = q.float().to(BF)
    assert torch.equal(y.isnan(), want.isnan()) and torch.equal(y[~want.isnan()], want[~want.isnan()])


# ------------------------------------------------------------------------------------------------- routing
def route(z, topk, **kw):
    tokens = z.shape[0]
    ids, gate = Out(1, tokens * topk, torch.int32), Out(1, tokens * topk, F32)
    hoc.ep_route(z, ids.t.view(-1), gate.t.view(-1), **kw)
    torch.cuda.synchronize()
    ids.check()
    gate.check()
    return ids.t.view(tokens, topk).cpu(), gate.t.view(tokens, topk).cpu()


def gate_bound(z, want, scale):
    """exp is off by 2 units and by its argument's rounding, the sums by up to 37 additions, quotient and products by one each:
    (64 + the range of the logits) * 2^-24; a sigmoid's exponent needs no rounding."""
    fin = z.double().cpu()
    fin = torch.where(torch.isfinite(fin), fin, torch.zeros_like(fin))
    return (64 + 2 * fin.abs().amax(1, keepdim=True)) * 2.0 ** -24 * want.abs() + 1e-37


def check_route(z, topk, bias=None, score="softmax", groups=1, top_groups=1, renormalise=False, scale=1.0):
    got = route(z, topk, bias=bias, score=score, groups=groups, top_groups=top_groups, renormalise=renormalise, scale=scale)
    want = ref.route(z.cpu(), topk, score, None if bias is None else bias.cpu(), groups, top_groups, renormalise, scale)
    bad = (got[0] != want[0]).any(1)
    assert not bool(bad.any()), f"{int(bad.sum())} tokens, first {int(bad.nonzero()[0])}: {got[0][bad][0]} for {want[0][bad][0]}"
    within(got[1], want[1], gate_bound(z, want[1], scale), "gate")
    return got


ROUTES = [  # tokens, experts, topk, groups, top_groups
    (1, 1, 1, 1, 1), (5, 2, 2, 1, 1), (7, 8, 3, 4, 2), (130, 64, 6, 1, 1), (33, 60, 4, 4, 3), (40, 160, 6, 8, 3), (50, 256, 8, 8, 4),
    (9, 128, 8, 1, 1), (20, 40, 5, 8, 4), (11, 512, 10, 8, 2), (6, 1024, 31, 1, 1), (6, 1000, 12, 4, 4), (13, 32, 31, 1, 1),
    (8, 31, 31, 1, 1), (12, 96, 2, 32, 5), (15, 33, 7, 11, 4), (4, 1024, 9, 16, 3), (3000, 64, 2, 1, 1), (2, 385, 12, 5, 1), (10, 64, 8, 32, 4),
]


@pytest.mark.parametrize("tokens,experts,topk,groups,top_groups", ROUTES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("biased,renormalise", [(False, False), (True, True), (False, True), (True, False)])
def test_route(tokens, experts, topk, groups, top_groups, score, dtype, biased, renormalise):
    g = gen(experts + topk)
    z = rows_of(g, tokens, experts, dtype, pad=3 if experts % 3 else 0, sigma=1.5)[0]
    bias = torch.randint(-40, 41, (experts,), generator=g, device=DEV) * 0.01 if biased else None
    check_route(z, topk, bias, score, groups, top_groups, renormalise, 2.5)


@pytest.mark.parametrize("experts,topk,groups,top_groups", [(64, 6, 1, 1), (256, 8, 8, 4), (100, 5, 1, 1), (40, 4, 5, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_keys_that_32_bits_cannot_tell_apart(experts, topk, groups, top_groups, score):
    """A bias that undoes the scores: all keys of a token lie within the rounding of a binary32 number, and 64 bits decide."""
    g = gen(experts)
    one = torch.randn(1, experts, generator=g, device=DEV)
    s = ref.scores(one.cpu(), score)
    bias = (0.9 - s).float()[0].to(DEV)
    assert (s + bias.cpu().double()).float().unique().numel() < experts / 4
    check_route(one.repeat(40, 1), topk, bias, score, groups, top_groups)
    z = one + torch.randn(300, experts, generator=g, device=DEV) * 1e-6  # and some of them near each other
    check_route(z, topk, bias, score, groups, top_groups, True)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top_groups,biased", [(1, 1, False), (1, 1, True), (8, 4, True), (8, 3, False)])
def test_equal_keys_go_to_the_lowest_expert(score, groups, top_groups, biased):
    g = gen(5)
    z = torch.randint(-2, 3, (200, 64), generator=g, device=DEV).float() * 0.5
    z[0] = 0
    z[1, ::2] = -0.0  # both zeros are one
    bias = torch.randint(-1, 2, (64,), generator=g, device=DEV) * 0.25 if biased else None
    check_route(z, 6, bias, score, groups, top_groups)
    check_route(z.to(BF), 6, bias, score, groups, top_groups)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top_groups", [(1, 1), (4, 2)])
@pytest.mark.parametrize("biased,renormalise", [(False, False), (True, True), (False, True), (True, False)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_masked_logits(score, groups, top_groups, biased, renormalise, dtype):
    """-inf and NaN are never chosen, also where nothing else is left; a row of nothing gets ids of -1 and gates of 0."""
    g = gen(6)
    z = torch.randn(40, 32, generator=g, device=DEV)
    z[0] = -math.inf
    z[1] = math.nan
    z[2] = -math.inf
    z[2, 17] = 0.5
    z[3] = math.nan
    z[3, [3, 9, 30]] = torch.tensor([1.0, 2.0, -1.0], device=DEV)
    z[4, 8:] = -math.inf
    z[5, ::2] = math.nan
    z[6] = torch.finfo(dtype).min
    z[7, 1:] = torch.finfo(dtype).min
    z[8] = 80.0
    z[9] = -80.0
    z[10, 20:] = -math.inf
    bias = torch.randn(32, generator=g, device=DEV) * 0.1 if biased else None
    if biased:
        bias[4] = -math.inf
        bias[5] = math.nan
    ids, gate = check_route(z.to(dtype), 6, bias, score, groups, top_groups, renormalise, 1.5)
    assert bool((ids[0] == -1).all()) and bool((gate[0] == 0).all())
    assert ids[2].tolist() == [17, -1, -1, -1, -1, -1]


def test_infinite_logits():
    z = torch.randn(4, 16, generator=gen(7), device=DEV)
    z[0, 5] = math.inf
    z[1, [3, 11]] = math.inf
    for renormalise in (False, True):
        for score in ("softmax", "sigmoid"):
            check_route(z, 4, None, score, renormalise=renormalise)


def test_far_logits_keep_their_gates():
    """Sigmoids that all underflow still have gates that add up to the scale."""
    z = torch.tensor([[-120.0, -121.0, -119.5, -300.0], [-90.0, 50.0, -91.0, 3.0], [100.0, 101.0, 102.0, -5.0]], device=DEV)
    for score in ("softmax", "sigmoid"):
        check_route(z, 3, None, score, renormalise=True, scale=2.0)


def grad_reference(z, ids, dgate, score, renormalise, scale):
    """dlogits by automatic differentiation of the gates' definition, masked experts apart; and the sizes of its terms."""
    zz = z.detach().to(F64).cpu()
    masked = ~(zz > -math.inf)
    zz = torch.where(masked, torch.full_like(zz, -1e4), zz).requires_grad_()  # far enough to have no share
    ok = (ids >= 0) & (ids < z.shape[1])
    ok &= ~masked.gather(1, ids.long().clamp(0, z.shape[1] - 1))
    use = torch.where(ok, ids, torch.full_like(ids, -1))
    dg = torch.where(ok, dgate.to(F64), torch.zeros((), dtype=F64))
    gate = ref.gates(zz, use, score, renormalise, scale)
    grad = torch.autograd.grad((gate * dg).sum(), zz)[0]
    return torch.where(masked, torch.zeros_like(grad), grad), masked


@pytest.mark.parametrize("tokens,experts,topk", [(1, 1, 1), (5, 2, 2), (130, 64, 6), (33, 60, 4), (40, 160, 6), (50, 256, 8), (6, 1024, 31),
                                                 (6, 1000, 12), (2000, 8, 2), (9, 385, 5)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("renormalise", [False, True])
def test_route_gradient(tokens, experts, topk, score, dtype, renormalise):
    g = gen(experts)
    z = rows_of(g, tokens, experts, dtype, pad=3 if experts % 3 else 0)[0]
    if experts > 8:
        z[0, 4:] = -math.inf
        z[1] = -math.inf
        z[2, 1] = math.nan
    ids, gate = route(z, topk, score=score, renormalise=renormalise, scale=2.5)
    dgate = torch.randn(tokens, topk, generator=g, device=DEV)
    dgate[(ids < 0).to(DEV)] = math.nan  # what lies behind a dropped slot is not looked at
    out = Out(tokens, experts, dtype, pad=5)
    hoc.ep_route_grad(z, ids.to(DEV).view(-1), dgate.view(-1), out.t, score=score, renormalise=renormalise, scale=2.5)
    torch.cuda.synchronize()
    out.check()
    want, masked = grad_reference(z, ids, dgate.cpu(), score, renormalise, 2.5)
    # an element is its score times a difference of terms that are at most the largest dgate: 64 + range roundings of those
    s = ref.scores(z.cpu(), score)
    share = s / s.gather(1, ids.long().clamp(min=0)).masked_fill(ids < 0, 0).sum(1, keepdim=True).clamp(min=1e-30) if renormalise else s
    most = dgate.cpu().double().nan_to_num(0.0).abs().amax(1, keepdim=True)
    within(out.t, want, ref.half_step(dtype) * want.abs() + 100 * 2.0 ** -24 * 2.5 * 2 * most * share + 1e-30, "dlogits")
    assert bool((out.t[masked.to(DEV)] == 0).all())
    same = z.clone()  # in place
    hoc.ep_route_grad(same, ids.to(DEV).view(-1), dgate.view(-1), same, score=score, renormalise=renormalise, scale=2.5)
    assert torch.equal(same, out.t)


def test_route_gradient_of_ids_that_repeat_or_lie_outside():
    """A dispatch takes any ids; a gate's slot counts for what it names."""
    g = gen(11)
    z = torch.randn(30, 16, generator=g, device=DEV)
    ids = torch.randint(0, 16, (30, 5), generator=g, device=DEV, dtype=torch.int32)
    ids[:, 3] = ids[:, 1]
    ids[4, 0], ids[5, 2], ids[6] = -7, 16, -1
    dgate = torch.randn(30, 5, generator=g, device=DEV)
    for score in ("softmax", "sigmoid"):
        for renormalise in (False, True):
            out = torch.full_like(z, 9.0)
            hoc.ep_route_grad(z, ids.view(-1), dgate.view(-1), out, score=score, renormalise=renormalise)
            want, _ = grad_reference(z, torch.where(ids < 16, ids, -1).cpu(), dgate.cpu(), score, renormalise, 1.0)
            within(out, want, 200 * 2.0 ** -24 * torch.full_like(want, float(dgate.abs().max()) * 2), "dlogits")


def test_equal_gate_gradients_cancel_where_gates_add_up():
    z = torch.randn(100, 64, generator=gen(12), device=DEV)
    for score in ("softmax", "sigmoid"):
        ids, _ = route(z, 6, score=score, renormalise=True)
        out = torch.empty_like(z)
        hoc.ep_route_grad(z, ids.to(DEV).view(-1), torch.full((600,), 0.37, device=DEV), out, score=score, renormalise=True)
        assert bool((out == 0).all())


# ------------------------------------------------------------------------------------------------- dropout
def seed_of(key, call):
    return torch.tensor([key, call], dtype=torch.int64, device=DEV)


def check_dropout(x, y, residual, p, key, call):
    t = min(65535, int(p * 65536 + 0.5))
    keep = (ref.philox_bits(x.numel(), (key, call)) >= t).view(x.shape)
    want = torch.where(keep, x.cpu().double() * (65536 / (65536 - t)), torch.zeros((), dtype=F64))
    # the factor and the product are rounded to 32 bits before the sum
    bound = 3 * 2.0 ** -24 * want.abs()
    if residual is not None:
        want = want + residual.cpu().double()
    within(y, want, (ref.half_step(x.dtype) + 2.0 ** -24) * want.abs() + bound, "y")
    return keep


@pytest.mark.parametrize("rows,width,pad,offset", [(1, 1, 0, 0), (3, 5, 0, 0), (7, 8, 0, 0), (33, 1001, 0, 0), (40, 264, 8, 0), (5, 64, 3, 1),
                                                   (300, 2048, 0, 0), (2, 4096, 0, 8), (1, 100003, 0, 0)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("p,residual", [(0.0, False), (0.1, True), (0.5, False), (0.99999, True), (1e-6, False)])
def test_dropout(rows, width, pad, offset, dtype, p, residual):
    g = gen(rows + width)
    x = rows_of(g, rows, width, dtype, pad, offset)[0]
    r = rows_of(g, rows, width, dtype, pad, offset)[0] if residual else None
    y = Out(rows, width, dtype, pad, offset)
    key, call = -(2 ** 62) + 12345, 2 ** 40 + 7
    hoc.dropout(x, y.t, p, seed_of(key, call), residual=r)
    torch.cuda.synchronize()
    y.check()
    check_dropout(x, y.t, r, p, key, call)
    a = x.clone()
    hoc.dropout(a, a, p, seed_of(key, call), residual=r)  # in place, and in rows that lie together: the same mask
    assert torch.equal(a, y.t)
    if residual:
        b = r.clone()
        hoc.dropout(x, b, p, seed_of(key, call), residual=b)
        assert torch.equal(b, y.t)


def test_dropout_drops_what_it_says_and_draws_anew():
    """Counts within five standard deviations; another key or call is another mask, and the two are independent."""
    n = 1 << 22
    x, y, z = torch.ones(n, device=DEV), torch.empty(n, device=DEV), torch.empty(n, device=DEV)
    for p in (0.05, 0.5, 0.9):
        q = int(p * 65536 + 0.5) / 65536
        hoc.dropout(x, y, p, seed_of(1, 1))
        for other in (seed_of(1, 2), seed_of(2, 1)):
            hoc.dropout(x, z, p, other)
            a, b = y == 0, z == 0
            assert abs(int(a.sum()) - n * q) <= 5 * (n * q * (1 - q)) ** 0.5
            both = int((a & b).sum())
            assert abs(both - n * q * q) <= 5 * (n * q * q) ** 0.5
        near = int((a[1:] & a[:-1]).sum())  # neighbours
        assert abs(near - n * q * q) <= 5 * (n * 3 * q * q) ** 0.5


def test_dropout_of_any_shape_is_that_of_the_flat_one():
    x = torch.randn(3, 5, 7, 11, generator=gen(2), device=DEV)
    a, b = torch.empty_like(x), torch.empty(x.numel(), device=DEV)
    hoc.dropout(x, a, 0.3, seed_of(5, 5))
    hoc.dropout(x.view(-1), b, 0.3, seed_of(5, 5))
    assert torch.equal(a.view(-1), b)


def test_dropout_keeps_infinities_of_dropped_elements_out():
    x = torch.full((4096,), math.inf, device=DEV)
    y = torch.empty_like(x)
    hoc.dropout(x, y, 0.5, seed_of(3, 4))
    assert not bool(y.isnan().any()) and bool((y == 0).any()) and bool((y == math.inf).any())


# ------------------------------------------------------------------------------------------------- graphs and streams
def calls():
    """Every operator on small inputs: (inputs that may change, call, outputs)."""
    g = gen(21)
    x, r, dy = (torch.randn(70, 320, generator=g, device=DEV).to(BF) for _ in range(3))
    w = torch.rand(320, generator=g, device=DEV)
    h, y, dx, d = (torch.empty_like(x) for _ in range(4))
    wire = torch.zeros(70, hoc.wire8_bytes(320), dtype=torch.uint8, device=DEV)
    dw = torch.empty(320, device=DEV)
    ws = torch.empty(hoc.rms_norm_workspace(70, 320), dtype=torch.int32, device=DEV)
    wide = torch.zeros(70, 320, dtype=BF, device=DEV)
    seg = torch.tensor([[0, 30, 70]], device=DEV)
    z, bias = torch.randn(70, 64, generator=g, device=DEV), torch.randn(64, generator=g, device=DEV) * 0.1
    ids, gate = torch.empty(420, dtype=torch.int32, device=DEV), torch.empty(420, device=DEV)
    dgate, dz = torch.randn(420, generator=g, device=DEV), torch.empty_like(z)
    seed = seed_of(77, 1)

    def call(stream=None):
        hoc.rms_norm(x, w, y, eps=1e-6, residual=r, h=h, wire=wire, stream=stream)
        hoc.expert_widen([wire], seg, [wide], stream=stream)
        hoc.ep_route(z, ids, gate, score="sigmoid", bias=bias, groups=8, top_groups=4, renormalise=True, stream=stream)
        hoc.ep_route_grad(z, ids, dgate, dz, score="sigmoid", renormalise=True, stream=stream)
        hoc.dropout(dy, d, 0.2, seed, stream=stream)
        hoc.rms_norm_grad(d, h, w, dx, eps=1e-6, dres=dy, dw=dw, workspace=ws, stream=stream)
    return (x, r, dy, z, dgate, seed, seg), call, (h, y, wire, wide, ids, gate, dz, d, dx, dw)


def test_captured_calls_follow_their_inputs():
    ins, call, outs = calls()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call(s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call(s)
    for seed in (1, 2):
        r = gen(seed)
        for t in ins[:5]:
            t.copy_(torch.randn(t.shape, generator=r, device=DEV))
        ins[5][1] = seed
        ins[6][0, 2] = 40 + seed
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        call()
        torch.cuda.synchronize()
        for a, b in zip(got, outs):
            assert torch.equal(a, b)


def test_calls_on_a_stream_of_their_own_wait_for_what_is_queued_there():
    ins, call, outs = calls()
    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    kept = [t.clone() for t in ins]
    s = torch.cuda.Stream()
    for t in ins[:5]:
        t.zero_()
    for t in outs:
        t.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(50_000_000)
        for t, k in zip(ins, kept):
            t.copy_(k)
    call(s)
    with torch.cuda.stream(s):
        got = [t.clone() for t in outs]
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_same_bits_every_time():
    g = gen(31)
    dy, h = (torch.randn(5000, 1024, generator=g, device=DEV).to(BF) for _ in range(2))
    w = torch.ones(1024, device=DEV)
    ws = torch.empty(hoc.rms_norm_workspace(5000, 1024), dtype=torch.int32, device=DEV)
    dx, dw = torch.empty_like(dy), torch.empty(10, 1024, device=DEV)
    for i in range(10):
        hoc.rms_norm_grad(dy, h, w, dx, eps=1e-6, dw=dw[i], workspace=ws)
    assert bool((dw == dw[0]).all())


# ------------------------------------------------------------------------------------------------- offsets past 32 bits
FAR = (70_001, 32_768)  # 2.3e9 elements


def far(pad=0):
    """Rows of zeros but for the last two, whose elements lie past 2^31."""
    t = torch.zeros(FAR[0], FAR[1] + pad, dtype=BF, device=DEV)[:, :FAR[1]]
    t[-2:] = torch.randn(2, FAR[1], generator=gen(40 + pad), device=DEV)
    return t


@pytest.mark.parametrize("pad", [0, 8, 1])
def test_norm_past_2_to_the_31(pad):
    x, w = far(pad), torch.rand(FAR[1], device=DEV) + 0.5
    y = torch.full_like(x, 7.0)
    hoc.rms_norm(x, w, y, eps=1e-6)
    _, want = ref.norm(x[-2:].cpu(), None, w.cpu(), 1e-6)
    within(y[-2:], want, (ref.half_step(BF) + NORM) * want.abs(), "y")
    assert bool((y[:-2] == 0).all())
    del y
    dx, dw = torch.empty_like(x), torch.empty(FAR[1], device=DEV)
    ws = torch.empty(hoc.rms_norm_workspace(*FAR), dtype=torch.int32, device=DEV)
    hoc.rms_norm_grad(x, x, w, dx, eps=1e-6, dw=dw, workspace=ws)
    wx, terms, ww, wterms = ref.norm_grad(x[-2:].cpu(), None, x[-2:].cpu(), w.cpu(), 1e-6, None)
    within(dx[-2:], wx, ref.half_step(BF) * wx.abs() + 2.0 ** -18 * terms, "dx")
    within(dw, ww, 200 * 2.0 ** -24 * wterms + 1e-30, "dw")  # two terms that are not zero
    assert bool((dx[:-2] == 0).all())


@pytest.mark.parametrize("pad", [0, 8, 1])
def test_dropout_past_2_to_the_31(pad):
    x = far(pad)
    seed = (3, 4)
    hoc.dropout(x, x, 0.25, seed_of(*seed), residual=None)
    want = far(pad)[-2:].cpu().double()
    keep = ref.philox_bits(2 * FAR[1], seed, (FAR[0] - 2) * FAR[1]).view(2, -1) >= 16384
    want = torch.where(keep, want * 65536 / 49152, torch.zeros((), dtype=F64))
    within(x[-2:], want, (ref.half_step(BF) + 2.0 ** -23) * want.abs(), "y")
    assert bool((x[:-2] == 0).all())


def test_routing_of_rows_that_lie_far_apart():
    wide = torch.zeros(40_000, 65_536, device=DEV)
    z = wide[:, :64]
    z.copy_(torch.randn(40_000, 64, generator=gen(44), device=DEV))
    together = z.clone()
    ids, gate, ids2, gate2 = (torch.empty(240_000, dtype=t, device=DEV) for t in (torch.int32, F32) * 2)
    hoc.ep_route(z, ids, gate, renormalise=True)
    hoc.ep_route(together, ids2, gate2, renormalise=True)
    assert torch.equal(ids, ids2) and torch.equal(gate, gate2)
    dgate = torch.randn(240_000, generator=gen(45), device=DEV)
    want = torch.empty_like(together)
    for renormalise in (True, False):
        hoc.ep_route_grad(together, ids, dgate, want, renormalise=renormalise)
        z.copy_(together)
        hoc.ep_route_grad(z, ids, dgate, z, renormalise=renormalise)
        assert torch.equal(z, want)


def test_widen_past_2_to_the_31():
    rows, width = 1_100_000, 2048
    wire = torch.zeros(rows, hoc.wire8_bytes(width), dtype=torch.uint8, device=DEV)
    q, scale = hoc.wire8_views(wire, width)
    q[-1] = torch.randn(width, generator=gen(46), device=DEV).to(q.dtype)
    scale[-1] = 0.5
    y = torch.full((rows, width), 7.0, dtype=BF, device=DEV)
    hoc.expert_widen([wire], torch.tensor([[0, 5, rows]], device=DEV), [y])
    assert torch.equal(y[-1], (q[-1].float() * 0.5).to(BF)) and bool((y[:-1] == 0).all())


def test_the_binding_refuses_bad_shapes():
    x = torch.zeros(4, 64, device=DEV)
    w = torch.ones(64, device=DEV)
    with pytest.raises(ValueError):
        hoc.rms_norm(x, w[:8], x, eps=1e-6)
    with pytest.raises(ValueError):
        hoc.rms_norm(x, w, x.t(), eps=1e-6)
    with pytest.raises(TypeError):
        hoc.rms_norm(x, w, x.to(BF), eps=1e-6)
    with pytest.raises(ValueError):
        hoc.rms_norm(x.t(), w[:4], x.t().clone(), eps=1e-6)
    with pytest.raises(ValueError):
        hoc.rms_norm(x, w, eps=1e-6, wire=torch.zeros(4, 64, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        hoc.rms_norm_grad(x, x, w, x.clone(), eps=1e-6, dw=w.clone())
    with pytest.raises(hoc.HocError):
        hoc.rms_norm_grad(x, x, w, x.clone(), eps=1e-6, dw=w.clone(), workspace=torch.zeros(64, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        hoc.ep_route(x, torch.zeros(7, dtype=torch.int32, device=DEV), torch.zeros(7, device=DEV))
    with pytest.raises(TypeError):
        hoc.ep_route(x, torch.zeros(8, dtype=torch.int64, device=DEV), torch.zeros(8, device=DEV))
    with pytest.raises(ValueError):
        hoc.dropout(x, x, 0.1, torch.zeros(3, dtype=torch.int64, device=DEV))
    with pytest.raises(hoc.HocError):
        hoc.dropout(x, x, 1.0, torch.zeros(2, dtype=torch.int64, device=DEV))
