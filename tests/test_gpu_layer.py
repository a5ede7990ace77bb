"""Expert products grouped by ragged row ranges, the linear layer, and their gradients, against 64-bit plain forms
(tests/layer_ref.py derives the bounds)."""
import pytest
import torch

from collective_communication_schedules_gb300 import hoc
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF = torch.bfloat16


def normal(*shape, seed=0, sigma=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * sigma).to(BF)


def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


# counts [rank][source][expert], in, out: ranges that end inside every tile size, empty experts and sources, one row,
# a rank without rows, all rows at one expert, widths that are and are not whole 16-byte rows
LAYOUTS = {
    "one row": ([[[1]]], 64, 32),
    "aligned": ([[[64, 128]]], 128, 64),
    "ragged": (ref.random_counts(2, 3, 4, 40, 1), 200, 136),
    "many sources": (ref.random_counts(3, 16, 2, 9, 2), 72, 48),
    "tile edges": ([[[255, 256, 257]], [[7, 8, 9]]], 264, 272),
    "empty rank": ([[[0, 0], [0, 0]], [[5, 0], [0, 11]]], 64, 64),
    "one expert": ([[[0, 700, 0, 0], [0, 333, 0, 0]]], 512, 304),
    "odd widths": (ref.random_counts(2, 2, 3, 50, 3), 61, 45),
    "odd in": (ref.random_counts(1, 2, 3, 70, 4), 131, 64),
    "odd out": (ref.random_counts(1, 2, 3, 70, 5), 64, 131),
    "wide": ([[[33, 90]], [[200, 1]]], 1032, 520),
    "many experts": (ref.random_counts(1, 1, 1500, 3, 6), 40, 24),
}


def expert_inputs(name, mul=1, sigma_x=1.0):
    counts, inp, out = LAYOUTS[name]
    L = ref.Routed(counts)
    x = [normal(n, inp, seed=10 + d, sigma=sigma_x) for d, n in enumerate(L.cap)]
    for d in range(L.k):
        x[d][L.of[d] < 0] = float("nan")  # nobody's rows must reach no result
    w = [normal(L.experts, mul * out, inp, seed=20 + d, sigma=inp ** -0.5) for d in range(L.k)]
    b = [normal(L.experts, mul * out, seed=30 + d, sigma=0.5) for d in range(L.k)]
    return L, x, w, b, inp, out


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu", "swiglu"])
@pytest.mark.parametrize("name", list(LAYOUTS))
def test_expert_forward(name, act):
    mul = 2 if act == "swiglu" else 1
    L, x, w, b, inp, out = expert_inputs(name, mul)
    with_bias = act != "relu"
    y = [torch.full((n, out), 7.0, dtype=BF, device=DEV) for n in L.cap]
    pre = [torch.full((n, mul * out), 7.0, dtype=BF, device=DEV) for n in L.cap]
    st = status()
    hoc.expert_mm(x, w, L.seg, y, status=st, bias=b if with_bias else None, act=act, pre=pre)
    y2 = [torch.empty_like(v) for v in y]
    hoc.expert_mm(x, w, L.seg, y2, status=st, bias=b if with_bias else None, act=act)
    torch.cuda.synchronize()
    assert st.item() == 0
    for d in range(L.k):
        nobody = L.of[d] < 0
        assert bool((y[d][nobody] == 7).all()) and bool((pre[d][nobody] == 7).all()), "a row of no range was written"
        assert torch.equal(y[d][~nobody], y2[d][~nobody])
        for e in range(L.experts):
            r = L.rows(d, e)
            if len(r) == 0:
                continue
            z, ez, want, ey = ref.forward(x[d][r], w[d][e], b[d][e] if with_bias else None, act)
            ref.close(pre[d][r], z, ez, f"pre {d} {e}")
            ref.close(y[d][r], want, ey, f"y {d} {e}")


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu", "swiglu"])
@pytest.mark.parametrize("name", list(LAYOUTS))
def test_expert_dgrad(name, act):
    mul = 2 if act == "swiglu" else 1
    counts, inp, out = LAYOUTS[name]
    L = ref.Routed(counts)
    dy = [normal(n, out, seed=40 + d) for d, n in enumerate(L.cap)]
    pre = [normal(n, mul * inp, seed=50 + d, sigma=2.0) for d, n in enumerate(L.cap)]
    for d in range(L.k):
        dy[d][L.of[d] < 0] = float("nan")
    w = [normal(L.experts, out, inp, seed=20 + d, sigma=inp ** -0.5) for d in range(L.k)]
    dx = [torch.full((n, mul * inp), 7.0, dtype=BF, device=DEV) for n in L.cap]
    st = status()
    hoc.expert_mm_dgrad(dy, w, L.seg, dx, status=st, act=act, pre=pre if act != "none" else None)
    torch.cuda.synchronize()
    assert st.item() == 0
    for d in range(L.k):
        assert bool((dx[d][L.of[d] < 0] == 7).all()), "a row of no range was written"
        for e in range(L.experts):
            r = L.rows(d, e)
            if len(r):
                want, err = ref.dgrad(dy[d][r], w[d][e], act, pre[d][r])
                ref.close(dx[d][r], want, err, f"dx {d} {e}")


@pytest.mark.parametrize("dtype,accumulate", [(BF, False), (torch.float32, True), (torch.float32, False), (BF, True)])
@pytest.mark.parametrize("name", list(LAYOUTS))
def test_expert_wgrad(name, dtype, accumulate):
    L, x, _, _, inp, out = expert_inputs(name)
    dy = [normal(n, out, seed=40 + d) for d, n in enumerate(L.cap)]
    for d in range(L.k):
        dy[d][L.of[d] < 0] = float("nan")
    dw = [normal(L.experts, out, inp, seed=60 + d).to(dtype) for d in range(L.k)]
    db = [normal(L.experts, out, seed=70 + d).to(dtype) for d in range(L.k)]
    was = [v.double() for v in dw], [v.double() for v in db]
    st = status()
    hoc.expert_mm_wgrad(dy, x, L.seg, dw, status=st, db=db, accumulate=accumulate)
    torch.cuda.synchronize()
    assert st.item() == 0
    half = ref.BF16 if dtype == BF else ref.F32
    for d in range(L.k):
        for e in range(L.experts):
            r = L.rows(d, e)
            a, v = dy[d][r].double(), x[d][r].double()
            n = max(1, len(r))
            ew, eb = (a.abs().t() @ v.abs()) * n * ref.F32, a.abs().sum(0) * n * ref.F32
            want_w, want_b = a.t() @ v, a.sum(0)
            if accumulate:
                want_w, want_b = want_w + was[0][d][e], want_b + was[1][d][e]
            ref.close(dw[d][e], want_w, ew + want_w.abs() * ref.F32, f"dw {d} {e}", half)
            ref.close(db[d][e], want_b, eb + want_b.abs() * ref.F32, f"db {d} {e}", half)


def test_rows_of_one_expert_stay_out_of_the_others():
    """NaN and inf rows of one expert reach no other expert's results, in any direction."""
    L = ref.Routed([[[37, 21, 5], [3, 0, 44]]])
    inp, out = 128, 96
    x, dy = normal(L.cap[0], inp, seed=1), normal(L.cap[0], out, seed=2)
    bad = L.rows(0, 1)
    x[bad], dy[bad] = float("nan"), float("inf")
    w = [normal(3, out, inp, seed=3, sigma=inp ** -0.5)]
    y, dx = torch.zeros(L.cap[0], out, dtype=BF, device=DEV), torch.zeros(L.cap[0], inp, dtype=BF, device=DEV)
    dw = [torch.zeros(3, out, inp, dtype=BF, device=DEV)]
    db = [torch.zeros(3, out, dtype=BF, device=DEV)]
    st = status()
    hoc.expert_mm([x], w, L.seg, [y], status=st)
    hoc.expert_mm_dgrad([dy], w, L.seg, [dx], status=st)
    hoc.expert_mm_wgrad([dy], [x], L.seg, dw, status=st, db=db)
    torch.cuda.synchronize()
    for e in (0, 2):
        r = L.rows(0, e)
        assert bool(torch.isfinite(y[r]).all()) and bool(torch.isfinite(dx[r]).all())
        assert bool(torch.isfinite(dw[0][e]).all()) and bool(torch.isfinite(db[0][e]).all())
    assert bool(y[bad].isnan().all()) and bool(dw[0][1].isnan().all())


def test_ranges_are_cut_to_the_buffer():
    """Ranges past the buffer's capacity, as after a dispatch that ran out of room, are cut; nothing past it is touched."""
    inp, out, cap = 64, 64, 50
    big = torch.full((cap + 30, inp), float("nan"), dtype=BF, device=DEV)
    x = big[:cap]
    x.copy_(normal(cap, inp, seed=1))
    seg = torch.tensor([[0, 30, 80, 75]], device=DEV)  # the second ends past the buffer, the third before it starts
    w = [normal(3, out, inp, seed=2, sigma=inp ** -0.5)]
    ybig = torch.full((cap + 30, out), 7.0, dtype=BF, device=DEV)
    dw = [torch.zeros(3, out, inp, dtype=BF, device=DEV)]
    st = status()
    dy = normal(cap, out, seed=3)
    hoc.expert_mm([x], w, seg, [ybig[:cap]], status=st)
    hoc.expert_mm_wgrad([dy], [x], seg, dw, status=st)
    torch.cuda.synchronize()
    assert bool((ybig[cap:] == 7).all())
    for e, (lo, hi) in enumerate([(0, 30), (30, 50)]):
        _, _, want, err = ref.forward(x[lo:hi], w[0][e], None, "none")
        ref.close(ybig[lo:hi], want, err, f"y {e}")
        a, v = dy[lo:hi].double(), x[lo:hi].double()
        ref.close(dw[0][e], a.t() @ v, (a.abs().t() @ v.abs()) * (hi - lo) * ref.F32, f"dw {e}")
    assert bool((dw[0][2] == 0).all())


LINEARS = [  # rows, in, out
    (1, 64, 64), (1, 4096, 520), (3, 1032, 264), (8, 512, 4096), (9, 128, 72), (16, 2048, 96), (17, 256, 640),
    (31, 520, 136), (64, 1024, 1024), (100, 136, 2056), (256, 512, 512), (257, 264, 776), (1000, 96, 40),
    (2, 33, 17), (5, 1, 1), (130, 77, 99), (40, 64, 33), (40, 35, 64),
]


@pytest.mark.parametrize("act,residual,pad", [("none", False, 0), ("gelu", True, 8), ("silu", True, 0), ("relu", False, 1),
                                              ("swiglu", False, 0), ("swiglu", True, 16)])
@pytest.mark.parametrize("rows,inp,out", LINEARS)
def test_linear(rows, inp, out, act, residual, pad):
    mul = 2 if act == "swiglu" else 1
    x = normal(rows, inp + pad, seed=1)[:, :inp]
    w, b = normal(mul * out, inp, seed=2, sigma=inp ** -0.5), normal(mul * out, seed=3)
    r = normal(rows, out + pad, seed=4)[:, :out] if residual else None
    ybig = torch.full((rows, out + pad), 7.0, dtype=BF, device=DEV)
    y, pre = ybig[:, :out], torch.empty(rows, mul * out, dtype=BF, device=DEV)
    st = status()
    hoc.linear(x, w, y, status=st, bias=b, act=act, pre=pre, residual=r)
    y2 = r.clone() if residual else torch.empty(rows, out, dtype=BF, device=DEV)
    hoc.linear(x, w, y2, status=st, bias=b, act=act, residual=y2 if residual else None)  # in place on the residual
    torch.cuda.synchronize()
    assert st.item() == 0
    assert bool((ybig[:, out:] == 7).all()), "written past a row's end"
    z, ez, want, ey = ref.forward(x, w, b, act)
    ref.close(pre, z, ez, "pre")
    if residual:
        want = want + r.double()
        ey = ey + want.abs() * ref.F32
    ref.close(y, want, ey, "y")
    assert torch.equal(y2, y)


@pytest.mark.parametrize("act", ["none", "gelu", "swiglu"])
@pytest.mark.parametrize("rows,inp,out", LINEARS)
def test_linear_gradients(rows, inp, out, act):
    mul = 2 if act == "swiglu" else 1
    x, dy = normal(rows, inp + 8, seed=1)[:, :inp], normal(rows, out + 8, seed=2)[:, :out]
    w, pre = normal(out, inp, seed=3, sigma=inp ** -0.5), normal(rows, mul * inp, seed=4)
    dx = torch.empty(rows, mul * inp, dtype=BF, device=DEV)
    dw, db = torch.empty(out, inp, device=DEV), torch.empty(out, device=DEV)
    st = status()
    hoc.linear_dgrad(dy, w, dx, status=st, act=act, pre=pre if act != "none" else None)
    hoc.linear_wgrad(dy, x, dw, status=st, db=db)
    torch.cuda.synchronize()
    assert st.item() == 0
    want, err = ref.dgrad(dy, w, act, pre)
    ref.close(dx, want, err, "dx")
    a, v = dy.double(), x.double()
    ref.close(dw, a.t() @ v, (a.abs().t() @ v.abs()) * rows * ref.F32, "dw", ref.F32)
    ref.close(db, a.sum(0), a.abs().sum(0) * rows * ref.F32, "db", ref.F32)


def test_linear_without_rows():
    w, st = normal(32, 64, seed=1), status()
    x, y = torch.empty(0, 64, dtype=BF, device=DEV), torch.empty(0, 32, dtype=BF, device=DEV)
    hoc.linear(x, w, y, status=st)
    hoc.linear_dgrad(y, w, x, status=st)
    dw, db = torch.full((32, 64), 5.0, device=DEV), torch.full((32,), 5.0, device=DEV)
    hoc.linear_wgrad(y, x, dw, status=st, db=db, accumulate=True)
    assert bool((dw == 5).all()) and bool((db == 5).all())
    hoc.linear_wgrad(y, x, dw, status=st, db=db)
    assert bool((dw == 0).all()) and bool((db == 0).all())


def test_a_few_bytes_off():
    """Operands that start 2 bytes past a 16-byte boundary."""
    n, inp, out = 70, 64, 48
    off = lambda t: torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].view(t.shape)  # noqa: E731
    x, w, b = off(normal(n, inp, seed=1)), off(normal(out, inp, seed=2, sigma=0.1)), off(normal(out, seed=3))
    y, st = off(torch.zeros(n, out, dtype=BF, device=DEV)), status()
    hoc.linear(x, w, y, status=st, bias=b, act="gelu")
    _, _, want, err = ref.forward(x, w, b, "gelu")
    ref.close(y, want, err, "y")


def test_on_another_stream_and_in_a_graph():
    n, inp, out = 300, 256, 128
    x, w, st = normal(n, inp, seed=1), normal(out, inp, seed=2, sigma=inp ** -0.5), status()
    y = torch.zeros(n, out, dtype=BF, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    hoc.linear(x, w, y, status=st, stream=s)
    s.synchronize()
    first = y.clone()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        hoc.linear(x, w, y, status=st, stream=s)
    x.copy_(normal(n, inp, seed=9))
    g.replay()
    torch.cuda.synchronize()
    _, _, want, err = ref.forward(x, w, None, "none")
    ref.close(y, want, err, "replayed")
    assert not torch.equal(first, y)


@pytest.mark.parametrize("act", ["relu", "gelu", "silu", "swiglu"])
@pytest.mark.parametrize("rows,width", [(1, 1), (5, 64), (33, 40), (7, 13)])
def test_act_grad(rows, width, act):
    mul = 2 if act == "swiglu" else 1
    dy, pre = normal(rows, width, seed=1), normal(rows, mul * width, seed=2, sigma=3.0)
    dz = torch.empty_like(pre)
    hoc.act_grad(dy, pre, dz, act)
    want, err = ref.dgrad(dy, torch.eye(width, device=DEV), act, pre)
    ref.close(dz, want, err, "dz")
    again = pre.clone()
    hoc.act_grad(dy, again, again, act)
    assert torch.equal(again, dz)


@pytest.mark.parametrize("act", ["gelu", "silu", "swiglu", "relu"])
def test_activations_at_the_ends_of_the_range(act):
    """Values whose exponentials over- or underflow, and infinite ones; against the limits."""
    v = torch.tensor([0.0, -0.0, 30.0, -30.0, 100.0, -100.0, 3e38, -3e38, 1e-38], device=DEV).to(BF)
    n = len(v)
    eye = torch.ones(1, 1, dtype=BF, device=DEV)
    x = v.view(n, 1).contiguous()
    w = torch.cat([eye, eye]) if act == "swiglu" else eye
    b = torch.tensor([0.0, 1.0], device=DEV).to(BF) if act == "swiglu" else None
    y, st = torch.empty(n, 1, dtype=BF, device=DEV), status()
    hoc.linear(x, w, y, status=st, act=act, bias=b)
    z = v.double()
    want = z.clamp(min=0) if act == "relu" else z * torch.sigmoid(z) if act != "gelu" else ref.act("gelu", z)
    if act == "swiglu":
        want = want * (z + 1)
    over = want.abs() > 3.4e38
    assert bool(torch.isfinite(y[~over]).all())
    ref.close(y[~over, 0], want[~over], want[~over].abs() * ref.MATH + 1e-30, "y")
    dz = torch.empty(n, 2 if act == "swiglu" else 1, dtype=BF, device=DEV)
    pre = torch.cat([x, torch.ones_like(x)], 1) if act == "swiglu" else x
    hoc.act_grad(torch.ones(n, 1, dtype=BF, device=DEV), pre.contiguous(), dz, act)
    assert bool(torch.isfinite(dz).all())
    assert dz[2, 0] == 1 and dz[4, 0] == 1 and dz[6, 0] == 1 and abs(float(dz[5, 0])) < 1e-30 and dz[7, 0] == 0


@pytest.mark.parametrize("act", ["gelu", "silu", "swiglu"])
def test_gradients_against_differences(act):
    """The gradients of sum(act(x W^T) * c) for x and W against central differences of the 64-bit definition."""
    rows, inp, out, mul = 4, 8, 8, 2 if act == "swiglu" else 1
    x, w = normal(rows, inp, seed=1), normal(mul * out, inp, seed=2, sigma=0.5)
    c = normal(rows, out, seed=3)
    y, pre, st = torch.empty(rows, out, dtype=BF, device=DEV), torch.empty(rows, mul * out, dtype=BF, device=DEV), status()
    hoc.linear(x, w, y, status=st, act=act, pre=pre)
    dz, dx, dw = torch.empty_like(pre), torch.empty_like(x), torch.empty(mul * out, inp, device=DEV)
    hoc.act_grad(c, pre, dz, act)
    hoc.linear_dgrad(dz, w, dx, status=st)
    hoc.linear_wgrad(dz, x, dw, status=st)

    def loss(xx, ww):
        return float((ref.forward(xx, ww, None, act)[2] * c.double()).sum())

    h = 1e-5
    for t, got, which in ((x.double(), dx, 0), (w.double(), dw, 1)):
        for i in range(t.shape[0]):
            for j in range(t.shape[1]):
                up, dn = t.clone(), t.clone()
                up[i, j] += h
                dn[i, j] -= h
                args = [(up, w.double()), (dn, w.double())] if which == 0 else [(x.double(), up), (x.double(), dn)]
                want = (loss(*args[0]) - loss(*args[1])) / (2 * h)
                # pre, dz and dx are each rounded to bf16: three roundings of terms of the size of the products
                scale = float((dz.double().abs()[i] @ w.double().abs()[:, j]) if which == 0
                              else (dz.double().abs()[:, i] @ x.double().abs()[:, j]))
                assert abs(float(got[i, j]) - want) <= 6 * ref.BF16 * (scale + abs(want)) + 1e-6, (which, i, j)


def test_segments_follow_the_dispatch():
    """ep_segments gives the ranges in which a fused dispatch leaves each expert's rows; dropped pairs count nowhere."""
    k, tokens, topk, experts, hidden = 4, 77, 3, 8, 16
    g = torch.Generator(device=DEV).manual_seed(3)
    ids = [torch.rand(tokens, experts, generator=g, device=DEV).topk(topk, 1).indices.to(torch.int32).flatten() for _ in range(k)]
    ids[1][5] = -1
    ids[2][9] = experts
    x = [torch.arange(tokens, device=DEV).view(-1, 1).expand(tokens, hidden).to(BF).contiguous() for _ in range(k)]
    cap = [k * tokens * topk] * k
    recv = [torch.full((c, hidden), -1.0, dtype=BF, device=DEV) for c in cap]
    pos = [torch.empty(tokens * topk, dtype=torch.int32, device=DEV) for _ in range(k)]
    counts = torch.empty(k, k, dtype=torch.int64, device=DEV)
    ws = torch.empty(k * hoc.ep_pack_workspace(tokens, topk, experts), dtype=torch.int32, device=DEV)
    hoc.ep_dispatch_fused(ids, x, experts, [t.view(-1) for t in recv], [c * hidden for c in cap], pos, counts, ws, status())
    seg = torch.full((k, experts + 1), -5, dtype=torch.int64, device=DEV)
    hoc.ep_segments(ids, experts, topk, seg)
    per = experts // k
    for d in range(k):
        at = 0
        for s in range(k):
            for e in range(per):
                want = torch.nonzero(ids[s] == d * per + e).flatten() // topk
                lo, hi = seg[d, s * per + e].item(), seg[d, s * per + e + 1].item()
                assert lo == at and hi == at + len(want)
                assert torch.equal(recv[d][lo:hi, 0].long(), want)
                at = hi
    many = [torch.randint(0, 9000, (500,), generator=g, device=DEV, dtype=torch.int32)]
    seg = torch.empty(1, 9001, dtype=torch.int64, device=DEV)
    hoc.ep_segments(many, 9000, 1, seg)
    assert torch.equal(seg[0, 1:], torch.bincount(many[0].long(), minlength=9000).cumsum(0)) and seg[0, 0] == 0


@pytest.mark.parametrize("seed", range(8))
def test_random_expert_layers(seed):
    """Random layouts and widths through all three products."""
    g = torch.Generator().manual_seed(100 + seed)
    pick = lambda *v: v[int(torch.randint(len(v), (1,), generator=g))]  # noqa: E731
    k, sources, experts = pick(1, 2, 5), pick(1, 2, 8), pick(1, 3, 8)
    inp, out, act = pick(8, 96, 192, 328, 50), pick(16, 64, 144, 400, 21), pick("none", "gelu", "swiglu")
    mul = 2 if act == "swiglu" else 1
    L = ref.Routed(ref.random_counts(k, sources, experts, pick(3, 60, 300), seed))
    x = [normal(n, inp, seed=seed + d) for d, n in enumerate(L.cap)]
    w = [normal(experts, mul * out, inp, seed=20 + d, sigma=inp ** -0.5) for d in range(k)]
    y = [torch.empty(n, out, dtype=BF, device=DEV) for n in L.cap]
    pre = [torch.empty(n, mul * out, dtype=BF, device=DEV) for n in L.cap]
    dx = [torch.empty(n, inp, dtype=BF, device=DEV) for n in L.cap]
    dw = [torch.empty(experts, mul * out, inp, dtype=BF, device=DEV) for _ in range(k)]
    st = status()
    hoc.expert_mm(x, w, L.seg, y, status=st, act=act, pre=pre)
    hoc.expert_mm_dgrad(pre, w, L.seg, dx, status=st)
    hoc.expert_mm_wgrad(pre, x, L.seg, dw, status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    for d in range(k):
        for e in range(experts):
            r = L.rows(d, e)
            a, v = pre[d][r].double(), x[d][r].double()
            ref.close(dw[d][e], a.t() @ v, (a.abs().t() @ v.abs()) * max(1, len(r)) * ref.F32, f"dw {d} {e}")
            if len(r):
                z, ez, want, ey = ref.forward(x[d][r], w[d][e], None, act)
                ref.close(y[d][r], want, ey, f"y {d} {e}")
                want, err = ref.dgrad(pre[d][r], w[d][e], "none", None)
                ref.close(dx[d][r], want, err, f"dx {d} {e}")


@pytest.mark.parametrize("product", ["forward", "dgrad", "wgrad"])
def test_a_wait_that_runs_out_sets_the_status(product, monkeypatch):
    """HOC_FAULT=mm_stall makes every copy barrier expect 16 bytes that no copy brings: the kernel's waits run out
    (0.1 s), it sets bit 2 and returns, and the next call is right again."""
    n, inp, out = 300, 256, 512
    x, dy, w = normal(n, inp, seed=1), normal(n, out, seed=2), normal(out, inp, seed=3, sigma=inp ** -0.5)
    y, dx, dw, st = torch.empty_like(dy), torch.empty_like(x), torch.empty_like(w), status()
    call = {"forward": lambda: hoc.linear(x, w, y, status=st), "dgrad": lambda: hoc.linear_dgrad(dy, w, dx, status=st),
            "wgrad": lambda: hoc.linear_wgrad(dy, x, dw, status=st)}[product]
    monkeypatch.setenv("HOC_FAULT", "mm_stall")
    call()
    torch.cuda.synchronize()
    assert st.item() == 4
    monkeypatch.delenv("HOC_FAULT")
    st.zero_()
    call()
    torch.cuda.synchronize()
    assert st.item() == 0
    got, want = {"forward": (y, x.double() @ w.double().t()), "dgrad": (dx, dy.double() @ w.double()),
                 "wgrad": (dw, dy.double().t() @ x.double())}[product]
    assert float((got.double() - want).norm() / want.norm()) < 2 * ref.BF16


@pytest.mark.parametrize("act", ["none", "gelu", "swiglu"])
@pytest.mark.parametrize("rows,inp,out", [(600, 333, 129), (300, 328, 131), (257, 515, 264), (9, 2049, 1031), (20, 1030, 2051),
                                          (130, 514, 250)])
def test_rows_that_are_not_whole_vectors(rows, inp, out, act):
    """Products large enough to run on realigned copies of their operands, with epilogue rows of any alignment."""
    mul = 2 if act == "swiglu" else 1
    x, dy = normal(rows, inp + 3, seed=1)[:, 1: 1 + inp], normal(rows, out + 1, seed=2)[:, :out]
    w, b, r = normal(mul * out, inp, seed=3, sigma=inp ** -0.5), normal(mul * out, seed=4), normal(rows, out + 5, seed=5)[:, 2: 2 + out]
    ybig = torch.full((rows, out + 3), 7.0, dtype=BF, device=DEV)
    y, pre, st = ybig[:, 1: 1 + out], torch.empty(rows, mul * out, dtype=BF, device=DEV), status()
    hoc.linear(x, w, y, status=st, bias=b, act=act, pre=pre, residual=r)
    wd, prd = normal(out, inp, seed=6, sigma=inp ** -0.5), normal(rows, mul * inp, seed=7)
    dx = torch.empty(rows, mul * inp, dtype=BF, device=DEV)
    hoc.linear_dgrad(dy, wd, dx, status=st, act=act, pre=prd if act != "none" else None)
    old = normal(out, inp, seed=8)
    dw, dwf, db = old.clone(), torch.empty(out, inp, device=DEV), torch.zeros(out, dtype=BF, device=DEV)
    hoc.linear_wgrad(dy, x, dw, status=st, db=db, accumulate=True)
    hoc.linear_wgrad(dy, x, dwf, status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    assert bool((ybig[:, 0] == 7).all()) and bool((ybig[:, 1 + out:] == 7).all()), "written outside the rows"
    z, ez, want, ey = ref.forward(x, w, b, act)
    ref.close(pre, z, ez, "pre")
    want = want + r.double()
    ref.close(y, want, ey + want.abs() * ref.F32, "y")
    want, err = ref.dgrad(dy, wd, act, prd)
    ref.close(dx, want, err, "dx")
    a, v = dy.double(), x.double()
    ew = (a.abs().t() @ v.abs()) * rows * ref.F32
    ref.close(dwf, a.t() @ v, ew, "dw", ref.F32)
    want = a.t() @ v + old.double()
    ref.close(dw, want, ew + want.abs() * ref.F32, "dw added")
    ref.close(db, a.sum(0), a.abs().sum(0) * rows * ref.F32, "db")


@pytest.mark.parametrize("act", ["silu", "swiglu"])
def test_expert_rows_that_are_not_whole_vectors(act):
    """The same for expert products: two ranks, two sources, an expert without rows, NaN rows that belong to nobody."""
    mul = 2 if act == "swiglu" else 1
    inp, out = 307, 205
    L = ref.Routed([[[70, 0, 33], [5, 0, 100]], [[1, 64, 9], [200, 8, 0]]])
    x = [normal(n, inp, seed=1 + d) for d, n in enumerate(L.cap)]
    dy = [normal(n, out, seed=3 + d) for d, n in enumerate(L.cap)]
    for d in range(2):
        x[d][L.of[d] < 0] = dy[d][L.of[d] < 0] = float("nan")
    w = [normal(3, mul * out, inp, seed=5 + d, sigma=inp ** -0.5) for d in range(2)]
    wd = [normal(3, out, inp, seed=7 + d, sigma=inp ** -0.5) for d in range(2)]
    prd = [normal(n, mul * inp, seed=9 + d) for d, n in enumerate(L.cap)]
    y = [torch.full((n, out), 7.0, dtype=BF, device=DEV) for n in L.cap]
    dx = [torch.full((n, mul * inp), 7.0, dtype=BF, device=DEV) for n in L.cap]
    dw = [torch.full((3, out, inp), 7.0, dtype=BF, device=DEV) for _ in range(2)]
    st = status()
    hoc.expert_mm(x, w, L.seg, y, status=st, act=act)
    hoc.expert_mm_dgrad(dy, wd, L.seg, dx, status=st, act=act, pre=prd)
    hoc.expert_mm_wgrad(dy, x, L.seg, dw, status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    for d in range(2):
        assert bool((y[d][L.of[d] < 0] == 7).all()) and bool((dx[d][L.of[d] < 0] == 7).all())
        for e in range(3):
            r = L.rows(d, e)
            a, v = dy[d][r].double(), x[d][r].double()
            ref.close(dw[d][e], a.t() @ v, (a.abs().t() @ v.abs()) * max(1, len(r)) * ref.F32, f"dw {d} {e}")
            if len(r):
                _, _, want, ey = ref.forward(x[d][r], w[d][e], None, act)
                ref.close(y[d][r], want, ey, f"y {d} {e}")
                want, err = ref.dgrad(dy[d][r], wd[d][e], act, prd[d][r])
                ref.close(dx[d][r], want, err, f"dx {d} {e}")


def test_realigned_copies_in_a_graph():
    n, inp, out = 300, 333, 129
    x, w, st = normal(n, inp, seed=1), normal(out, inp, seed=2, sigma=inp ** -0.5), status()
    y = torch.zeros(n, out, dtype=BF, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    hoc.linear(x, w, y, status=st, stream=s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        hoc.linear(x, w, y, status=st, stream=s)
    for seed in (9, 10):
        x.copy_(normal(n, inp, seed=seed))
        g.replay()
        torch.cuda.synchronize()
        _, _, want, err = ref.forward(x, w, None, "none")
        ref.close(y, want, err, "replayed")


@pytest.mark.parametrize("most", [5, 90])
def test_more_sources_than_a_warp_has_lanes(most):
    """40 and 70 row ranges to an expert: the ranges are walked 32 at a time."""
    inp, out = 136, 72
    for sources in (40, 70):
        L = ref.Routed(ref.random_counts(1, sources, 2, most, sources + most))
        n = L.cap[0]
        x, dy = normal(n, inp, seed=1), normal(n, out, seed=2)
        x[L.of[0] < 0] = dy[L.of[0] < 0] = float("nan")
        w = [normal(2, out, inp, seed=3, sigma=inp ** -0.5)]
        y, dx = torch.full((n, out), 7.0, dtype=BF, device=DEV), torch.full((n, inp), 7.0, dtype=BF, device=DEV)
        dw, db = [torch.empty(2, out, inp, device=DEV)], [torch.empty(2, out, device=DEV)]
        st = status()
        hoc.expert_mm([x], w, L.seg, [y], status=st)
        hoc.expert_mm_dgrad([dy], w, L.seg, [dx], status=st)
        hoc.expert_mm_wgrad([dy], [x], L.seg, dw, status=st, db=db)
        torch.cuda.synchronize()
        assert st.item() == 0
        assert bool((y[L.of[0] < 0] == 7).all())
        for e in range(2):
            r = L.rows(0, e)
            _, _, want, err = ref.forward(x[r], w[0][e], None, "none")
            ref.close(y[r], want, err, f"y {e}")
            want, err = ref.dgrad(dy[r], w[0][e], "none", None)
            ref.close(dx[r], want, err, f"dx {e}")
            a, v = dy[r].double(), x[r].double()
            ref.close(dw[0][e], a.t() @ v, (a.abs().t() @ v.abs()) * len(r) * ref.F32, f"dw {e}", ref.F32)
            ref.close(db[0][e], a.sum(0), a.abs().sum(0) * len(r) * ref.F32, f"db {e}", ref.F32)


def test_every_expert_tile_order():
    """More experts than are sorted (256), with whole and lower tiles among them, and the two-launch split (more than
    1024): every row is computed once, by its own expert."""
    for experts, most in ((300, 520), (1100, 5)):
        counts = ref.random_counts(1, 1, experts, most, experts, empty=0.5)
        L = ref.Routed(counts)
        n, inp, out = L.cap[0], 16, 8
        x = normal(n, inp, seed=1)
        w = [normal(experts, out, inp, seed=2)]
        y, st = torch.full((n, out), 7.0, dtype=BF, device=DEV), status()
        hoc.expert_mm([x], w, L.seg, [y], status=st)
        own = L.of[0].clamp(min=0)
        want = torch.einsum("rk,rok->ro", x.double(), w[0].double()[own])
        err = torch.einsum("rk,rok->ro", x.double().abs(), w[0].double().abs()[own]) * inp * ref.F32
        has = L.of[0] >= 0
        ref.close(y[has], want[has], err[has], "y")
        assert bool((y[~has] == 7).all()) and st.item() == 0


@pytest.mark.parametrize("act", ["none", "gelu", "swiglu"])
@pytest.mark.parametrize("rows,inp,out", [(33, 8192, 512), (70, 4104, 296), (257, 1000, 256), (40, 328, 8), (130, 520, 2056),
                                          (2100, 40, 24), (1025, 264, 520), (5000, 72, 128)])
def test_a_contraction_shared_by_several_ctas(rows, inp, out, act):
    """Few tiles and a long contraction, of x's or dy's width or of the rows."""
    mul = 2 if act == "swiglu" else 1
    x, w, b = normal(rows, inp, seed=1), normal(mul * out, inp, seed=2, sigma=inp ** -0.5), normal(mul * out, seed=3)
    r, dy = normal(rows, out, seed=4), normal(rows, out, seed=5)
    wd, below = w[:out], normal(rows, mul * inp, seed=6)
    st = status()
    got = []
    for _ in range(3):
        y, pre = torch.empty(rows, out, dtype=BF, device=DEV), torch.empty(rows, mul * out, dtype=BF, device=DEV)
        dx = torch.empty(rows, mul * inp, dtype=BF, device=DEV)
        dw, db = torch.empty(out, inp, device=DEV), torch.empty(out, device=DEV)
        dwb = torch.ones(out, inp, dtype=BF, device=DEV)
        hoc.linear(x, w, y, status=st, bias=b, act=act, pre=pre, residual=r)
        hoc.linear_dgrad(dy, wd, dx, status=st, act=act, pre=below if act != "none" else None)
        hoc.linear_wgrad(dy, x, dw, status=st, db=db)
        hoc.linear_wgrad(dy, x, dwb, status=st, accumulate=True)
        got.append((y, pre, dx, dw, db, dwb))
    torch.cuda.synchronize()
    assert st.item() == 0
    assert all(torch.equal(a, c) for other in got[1:] for a, c in zip(got[0], other)), "the order of the sums changed"
    z, ez, want, ey = ref.forward(x, w, b, act)
    ref.close(pre, z, ez, "pre")
    want = want + r.double()
    ref.close(y, want, ey + want.abs() * ref.F32, "y")
    want, err = ref.dgrad(dy, wd, act, below)
    ref.close(dx, want, err, "dx")
    a, v = dy.double(), x.double()
    err = (a.abs().t() @ v.abs()) * rows * ref.F32
    ref.close(dw, a.t() @ v, err, "dw", ref.F32)
    ref.close(db, a.sum(0), a.abs().sum(0) * rows * ref.F32, "db", ref.F32)
    ref.close(dwb, a.t() @ v + 1, err + ref.F32, "dw added to")


@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("rows", [16, 17, 32])
def test_few_rows_of_large_weights(rows, act):
    inp, out = 4160, 4104
    x, w = normal(rows, inp, seed=1), normal((2 if act == "swiglu" else 1) * out, inp, seed=2, sigma=inp ** -0.5)
    y, st = torch.empty(rows, out, dtype=BF, device=DEV), status()
    hoc.linear(x, w, y, status=st, act=act)
    assert st.item() == 0
    _, _, want, err = ref.forward(x, w, None, act)
    ref.close(y, want, err, "y")


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("rows,inp,out", [(1, 512, 512), (70, 1024, 1048), (515, 2048, 1400), (2047, 512, 520)])
def test_bias_gradient_beside_the_weight_gradient(rows, inp, out, accumulate):
    """Column sums by the product's own warps, their order fixed; rows that lie apart."""
    x, dy = normal(rows, inp, seed=1), normal(rows, out + 8, seed=2)[:, :out]
    w0, b0, st = normal(out, inp, seed=3), normal(out, seed=4), status()
    got = []
    for _ in range(2):
        dw, db = w0.clone(), b0.clone()
        hoc.linear_wgrad(dy, x, dw, status=st, db=db, accumulate=accumulate)
        got.append((dw, db))
    assert st.item() == 0
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    a, v, keep = dy.double(), x.double(), float(accumulate)
    ref.close(got[0][0], a.t() @ v + keep * w0.double(), (a.abs().t() @ v.abs()) * rows * ref.F32 + w0.double().abs() * ref.F32, "dw")
    ref.close(got[0][1], a.sum(0) + keep * b0.double(), a.abs().sum(0) * rows * ref.F32 + b0.double().abs() * ref.F32, "db")


@pytest.mark.parametrize("out", [8, 24, 72, 136, 264])
def test_gates_of_any_multiple_of_eight(out):
    """Gates and values lie `out` rows apart; the last tile holds fewer than its 128."""
    rows, inp = 150, 200
    x, w, b = normal(rows, inp, seed=1), normal(2 * out, inp, seed=2, sigma=inp ** -0.5), normal(2 * out, seed=3)
    y, pre, st = torch.empty(rows, out, dtype=BF, device=DEV), torch.empty(rows, 2 * out, dtype=BF, device=DEV), status()
    hoc.linear(x, w, y, status=st, bias=b, act="swiglu", pre=pre)
    assert st.item() == 0
    z, ez, want, err = ref.forward(x, w, b, "swiglu")
    ref.close(pre, z, ez, "pre")
    ref.close(y, want, err, "y")


@pytest.mark.parametrize("sources", [0, 1, 3])
def test_a_long_contraction_is_not_a_stall(sources, monkeypatch):
    """HOC_FAULT=mm_hurry lets waits run out after a millisecond.  The weight gradient over some 4 million rows of one
    expert, in which the epilogue (and the warps that zero padding rows) wait for longer, is still complete: the limit
    is on standing still.  Values are small whole numbers, so that binary32 sums are exact.  sources 0: a linear layer,
    whose contraction four pairs of CTAs share."""
    rows, inp, out = (1 << 22) + 37, 200, 136
    g = torch.Generator(device=DEV).manual_seed(sources)
    x, dy = (torch.randint(-1, 2, (rows, w), generator=g, device=DEV, dtype=torch.int8).to(BF) for w in (inp, out))
    dw, db, st = torch.zeros(1, out, inp, device=DEV), torch.zeros(1, out, device=DEV), status()
    monkeypatch.setenv("HOC_FAULT", "mm_hurry")
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(2):
        start.record()
        if sources:
            cuts = [0, rows] if sources == 1 else [0, 1_000_003, 3_000_000, rows]
            hoc.expert_mm_wgrad([dy], [x], torch.tensor([cuts], device=DEV), [dw], status=st, db=[db])
        else:
            hoc.linear_wgrad(dy, x, dw[0], status=st, db=db[0])
        end.record()
    torch.cuda.synchronize()
    assert start.elapsed_time(end) > 3, "too short to tell a long wait from a stall"
    assert st.item() == 0
    want = sum(dy[i: i + (1 << 19)].double().t() @ x[i: i + (1 << 19)].double() for i in range(0, rows, 1 << 19))
    assert torch.equal(dw[0].double(), want)
    assert torch.equal(db[0].double(), dy.sum(0, dtype=torch.float64))


def test_scratch_is_given_back():
    """What realigned copies took stays with the library until it is asked for, and later calls are right again."""
    rows, inp, out = 200_000, 1023, 255
    x, w, st = normal(rows, inp, seed=1), normal(out, inp, seed=2, sigma=inp ** -0.5), status()
    y, again = torch.empty(rows, out, dtype=BF, device=DEV), torch.empty(rows, out, dtype=BF, device=DEV)
    mib = 1 << 20

    def taken(since):
        torch.cuda.synchronize()
        return since - torch.cuda.mem_get_info()[0]

    hoc.layer_trim()  # other tests' scratch
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    hoc.linear(x, w, y, status=st)
    assert taken(before) > rows * 1024 * 2 - 64 * mib  # the copy of x is 391 MiB, taken in units of some MiB
    hoc.layer_trim(128 * mib)
    assert taken(before) < 192 * mib
    hoc.linear(x, w, again, status=st)
    hoc.layer_trim()
    torch.cuda.synchronize()
    hoc.layer_trim()
    assert taken(before) < 64 * mib
    assert torch.equal(y, again) and st.item() == 0


def test_a_closed_relu_lets_nothing_through():
    """Where ReLU's input is not above 0 the gradient is 0 whatever comes from above, infinities and NaN among them;
    where it is, what comes is passed on."""
    inf, nan = float("inf"), float("nan")
    above = torch.tensor([1.0, inf, -inf, nan], device=DEV).to(BF)
    below = torch.tensor([-1.0, 0.0, -0.0, -inf, 2.0, inf], device=DEV).to(BF)
    n = len(above)
    dy = above.view(n, 1).expand(n, len(below)).contiguous()  # row i: above[i]
    pre = below.view(1, -1).expand(n, len(below)).contiguous()
    want = torch.where(pre > 0, dy, torch.zeros_like(dy))
    for width in (len(below), 8 * len(below)):  # value by value, and as vectors
        d, z = (t.repeat(1, width // len(below)) for t in (dy, pre))
        dz = torch.full_like(d, 7.0)
        hoc.act_grad(d, z, dz, "relu")
        assert torch.equal(dz.nan_to_num(5.0), want.repeat(1, width // len(below)).nan_to_num(5.0))
    # through a product: every input of the layer below gets above[i]
    for rows, inp in ((n, 6), (n, 48), (64, 48)):
        out = 16 if inp > 6 else 5
        d = torch.zeros(rows, out, device=DEV).to(BF)
        d[:n, 0] = above
        w = torch.zeros(out, inp, device=DEV).to(BF)
        w[0] = 1.0
        z = below.repeat(inp // len(below)).expand(rows, inp).contiguous()
        dx, st = torch.full((rows, inp), 7.0, device=DEV).to(BF), status()
        hoc.linear_dgrad(d, w, dx, status=st, act="relu", pre=z)
        want = torch.where(z > 0, d[:, :1].expand(rows, inp), torch.zeros_like(z))
        assert torch.equal(dx.nan_to_num(5.0), want.nan_to_num(5.0)), (rows, inp)
