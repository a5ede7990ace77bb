"""Gradient norm and clipping over tensor lists, and the gradient of the combine, against 64-bit plain forms."""
import pytest
import torch

from collective_communication_schedules_gb300 import hoc

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF = torch.bfloat16


def make(counts, dtype, seed=0, sigma=1.0, offset=0):
    """Tensors of a flat buffer, each starting `offset` elements after the one before ends."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    flat = (torch.randn(sum(counts) + offset * (len(counts) + 1), generator=g, device=DEV) * sigma).to(dtype)
    out, at = [], offset
    for n in counts:
        out.append(flat[at: at + n])
        at += n + offset
    return flat, out


# Squares and sums in binary32 over at most 32768 / 1024 terms per thread and unroll slot, then binary64: the norm is
# good to 64 * 2^-24 relatively; the coefficient adds two roundings.
NORM = 64 * 2.0 ** -24


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("counts,offset", [
    ([1], 0), ([0], 0), ([], 0), ([5, 0, 7], 1), ([4096], 0), ([1000003], 3), ([1, 2, 3, 4, 5, 6, 7, 8, 9] * 20, 1),
    ([100_000] * 30, 0), ([40_000_001], 1), ([17] * 3000, 1),
])
def test_clip(counts, offset, dtype):
    flat, src = make(counts, dtype, seed=len(counts), offset=offset)
    guard, dst = make(counts, dtype, seed=99, offset=offset)
    before = guard.clone()
    norm = torch.full((1,), -1.0, device=DEV)
    with hoc.TensorList(src) as a, hoc.TensorList(dst) as b:
        ws = torch.full((hoc.grad_workspace(a),), -1, dtype=torch.int32, device=DEV)
        want = sum(float(t.double().square().sum()) for t in src) ** 0.5
        for max_norm in (0.5, 1e9):
            hoc.grad_clip(a, b, max_norm, norm, ws)
            assert abs(norm.item() - want) <= NORM * want
            c = min(1.0, max_norm / (want + 1e-6))
            half = 2.0 ** -8 if dtype == BF else 2.0 ** -24
            for s, d in zip(src, dst):
                if c == 1.0:
                    assert torch.equal(s, d)
                else:
                    assert bool(((d.double() - c * s.double()).abs() <= (half + 2 * NORM) * c * s.double().abs() + 1e-40).all())
        norm2 = torch.empty(1, device=DEV)
        hoc.grad_norm(a, norm2, ws)
        assert torch.equal(norm, norm2)
        hoc.grad_clip(a, b, 0.5, norm, ws)
        kept = [d.clone() for d in dst]
        hoc.grad_clip(a, a, 0.5, norm, ws)  # in place
        for s, d in zip(src, kept):
            assert torch.equal(s, d)
    if offset:
        gaps = torch.ones_like(guard, dtype=torch.bool)
        at = offset
        for n in counts:
            gaps[at: at + n] = False
            at += n + offset
        assert torch.equal(guard[gaps], before[gaps]), "written outside the tensors"


def test_source_and_destination_aligned_differently():
    flat, src = make([1001, 77], torch.float32, seed=1, offset=1)
    out, dst = make([1001, 77], torch.float32, seed=2, offset=2)
    norm = torch.empty(1, device=DEV)
    a, b = hoc.TensorList(src), hoc.TensorList(dst)
    ws = torch.empty(hoc.grad_workspace(a), dtype=torch.int32, device=DEV)
    hoc.grad_clip(a, b, 1.0, norm, ws)
    c = 1.0 / (float(torch.cat(src).double().norm()) + 1e-6)
    for s, d in zip(src, dst):
        assert bool(((d.double() - c * s.double()).abs() <= (2.0 ** -24 + 2 * NORM) * c * s.double().abs()).all())


@pytest.mark.parametrize("value,norm_is", [(float("nan"), "nan"), (float("inf"), "inf"), (3e38, "inf")])
def test_values_that_are_not_finite(value, norm_is):
    _, src = make([5000, 300], torch.float32, seed=1)
    src[1][7] = value
    norm = torch.empty(1, device=DEV)
    with hoc.TensorList(src) as a:
        ws = torch.empty(hoc.grad_workspace(a), dtype=torch.int32, device=DEV)
        hoc.grad_norm(a, norm, ws)
        assert str(norm.item()) == norm_is
        hoc.grad_clip(a, a, 1.0, norm, ws)
        assert bool(src[0].isnan().all()) if norm_is == "nan" else bool((src[0] == 0).all())


def test_same_bits_every_time():
    _, src = make([3_000_001, 5], BF, seed=4)
    norm = torch.empty(20, device=DEV)
    with hoc.TensorList(src) as a:
        ws = torch.empty(hoc.grad_workspace(a), dtype=torch.int32, device=DEV)
        for i in range(20):
            hoc.grad_norm(a, norm[i:i + 1], ws)
        assert len(set(norm.tolist())) == 1


def test_in_a_graph():
    _, src = make([70_000, 11], torch.float32, seed=5)
    norm = torch.empty(1, device=DEV)
    with hoc.TensorList(src) as a:
        ws = torch.empty(hoc.grad_workspace(a), dtype=torch.int32, device=DEV)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        hoc.grad_clip(a, a, 1.0, norm, ws, stream=s)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            hoc.grad_clip(a, a, 1.0, norm, ws, stream=s)
        src[0].fill_(2.0)
        src[1].fill_(0.0)
        g.replay()
        torch.cuda.synchronize()
        want = 2 * 70_000 ** 0.5
        assert abs(norm.item() - want) <= NORM * want
        assert abs(float(src[0][3]) - 2 / want) <= 1e-6


def routed(k, tokens, topk, experts, hidden, seed, drop=True):
    g = torch.Generator(device=DEV).manual_seed(seed)
    ids = [torch.rand(tokens, experts, generator=g, device=DEV).topk(topk, 1).indices.to(torch.int32).flatten().contiguous()
           for _ in range(k)]
    if drop and tokens:
        ids[0][0] = -3
        ids[k - 1][tokens * topk - 1] = experts
    return ids, g


def dispatch(ids, x, experts, caps, tokens, topk, hidden):
    k = len(ids)
    recv = [torch.zeros(c * hidden, dtype=BF, device=DEV) for c in caps]
    pos = [torch.empty(tokens * topk, dtype=torch.int32, device=DEV) for _ in range(k)]
    counts = torch.empty(k, k, dtype=torch.int64, device=DEV)
    ws = torch.empty(k * hoc.ep_pack_workspace(tokens, topk, experts), dtype=torch.int32, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    hoc.ep_dispatch_fused(ids, x, experts, recv, [c * hidden for c in caps], pos, counts, ws, st)
    return recv, pos, counts, st


@pytest.mark.parametrize("k,tokens,topk,experts,hidden", [
    (1, 1, 1, 1, 8), (2, 33, 2, 8, 512), (4, 200, 6, 16, 264), (8, 700, 3, 16, 2056), (16, 9, 4, 32, 64),
    (2, 50, 12, 24, 128), (3, 41, 2, 6, 37), (2, 3000, 2, 4, 96),
])
@pytest.mark.parametrize("packed", [False, True])
def test_combine_gradient(k, tokens, topk, experts, hidden, packed):
    """drows and dweights of the combine; rows found through a dispatch of the same ids (its rows name their tokens)."""
    ids, g = routed(k, tokens, topk, experts, hidden, seed=k)
    n = tokens * topk
    caps = [k * n] * k
    x = [torch.randn(tokens, hidden, generator=g, device=DEV).to(BF) for _ in range(k)]
    dy = [torch.randn(tokens, hidden, generator=g, device=DEV).to(BF) for _ in range(k)]
    w = [torch.rand(n, generator=g, device=DEV) for _ in range(k)]
    if packed:
        rows = [torch.zeros(n * hidden, dtype=BF, device=DEV) for _ in range(k)]
        pos = [torch.empty(n, dtype=torch.int32, device=DEV) for _ in range(k)]
        counts = torch.empty(k, k, dtype=torch.int64, device=DEV)
        ws = torch.empty(k * hoc.ep_pack_workspace(tokens, topk, experts), dtype=torch.int32, device=DEV)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        caps = [n] * k
        hoc.ep_pack_all(ids, x, experts, rows, [n * hidden] * k, pos, counts, ws, st)
    else:
        rows, pos, counts, st = dispatch(ids, x, experts, caps, tokens, topk, hidden)
    drows = [torch.full_like(t, 7.0) for t in rows]
    dw = [torch.full((n,), 7.0, device=DEV) for _ in range(k)]
    elems = [c * hidden for c in caps]
    if packed:
        hoc.ep_combine_grad_all(dy, rows, elems, pos, w, tokens, topk, hidden, drows, dw, st)
    else:
        hoc.ep_combine_grad(dy, rows, elems, ids, pos, counts, w, tokens, topk, hidden, experts, drows, dw, st)
    torch.cuda.synchronize()
    assert st.item() == 0
    per = experts // k
    touched = [torch.zeros(c, dtype=torch.bool, device=DEV) for c in caps]
    cn = counts // hidden
    for s in range(k):
        e = ids[s].long()
        ok = (e >= 0) & (e < experts)
        d = torch.where(ok, e // per, torch.zeros_like(e))
        sd = cn[s].cumsum(0) - cn[s]
        rd = cn[:, :].cumsum(0)[s] - cn[s]
        row = pos[s].long() if packed else rd[d] - sd[d] + pos[s].long()
        where = torch.full_like(d, s) if packed else d
        token = torch.arange(n, device=DEV) // topk
        v = dy[s].double()[token]
        dot = (v * x[s].double()[token]).sum(1)  # the rows are the tokens' own
        err = (v * x[s].double()[token]).abs().sum(1) * hidden * 2.0 ** -24
        assert bool(((dw[s].double() - dot).abs() <= err)[ok].all()) and bool((dw[s][~ok] == 0).all())
        want = (w[s][:, None] * dy[s].float()[token]).to(BF)
        for b in range(k):
            m = ok & (where == b)
            assert torch.equal(drows[b].view(-1, hidden)[row[m]], want[m])
            touched[b][row[m]] = True
    for b in range(k):
        assert bool((drows[b].view(-1, hidden)[~touched[b]] == 7).all()), "a row that no pair names was written"


def test_combine_gradient_past_the_buffers():
    """Rows outside their buffer set status bit 1, add nothing and are not written."""
    k, tokens, topk, experts, hidden = 2, 20, 2, 4, 64
    ids, g = routed(k, tokens, topk, experts, hidden, seed=1, drop=False)
    full = [k * tokens * topk] * k
    x = [torch.randn(tokens, hidden, generator=g, device=DEV).to(BF) for _ in range(k)]
    rows, pos, counts, st = dispatch(ids, x, experts, full, tokens, topk, hidden)
    small = 5
    drows = [torch.full_like(t, 7.0) for t in rows]
    dw = [torch.full((tokens * topk,), 7.0, device=DEV) for _ in range(k)]
    w = [torch.ones(tokens * topk, device=DEV) for _ in range(k)]
    hoc.ep_combine_grad(x, rows, [small * hidden] * k, ids, pos, counts, w, tokens, topk, hidden, experts, drows, dw, st)
    torch.cuda.synchronize()
    assert st.item() == 2
    for b in range(k):
        assert bool((drows[b].view(-1, hidden)[small:] == 7).all())
    assert sum(int((v != 0).sum()) for v in dw) == k * small


def test_combine_gradient_inverts_the_combine():
    """<combine(rows), dy> changes by <drows, step> along any step of the rows: the gradient is the combine's."""
    k, tokens, topk, experts, hidden = 2, 30, 3, 6, 64
    ids, g = routed(k, tokens, topk, experts, hidden, seed=5, drop=False)
    caps = [k * tokens * topk] * k
    x = [torch.randn(tokens, hidden, generator=g, device=DEV).to(BF) for _ in range(k)]
    dy = [torch.randn(tokens, hidden, generator=g, device=DEV).to(BF) for _ in range(k)]
    w = [torch.rand(tokens * topk, generator=g, device=DEV) for _ in range(k)]
    rows, pos, counts, st = dispatch(ids, x, experts, caps, tokens, topk, hidden)
    elems = [c * hidden for c in caps]
    drows, dw = [torch.zeros_like(t) for t in rows], [torch.empty_like(v) for v in w]
    hoc.ep_combine_grad(dy, rows, elems, ids, pos, counts, w, tokens, topk, hidden, experts, drows, dw, st)
    y = [torch.empty(tokens, hidden, dtype=BF, device=DEV) for _ in range(k)]
    hoc.ep_combine_fused(rows, elems, ids, pos, counts, w, tokens, topk, hidden, experts, y, st)
    # the combine is linear in rows and in weights: <y, dy> = <rows, drows> = <w, dw>; y and drows are rounded to bf16
    a = sum(float((p.double() * q.double()).sum()) for p, q in zip(y, dy))
    b = sum(float((p.double() * q.double()).sum()) for p, q in zip(rows, drows))
    c = sum(float((p.double() * q.double()).sum()) for p, q in zip(w, dw))
    size = sum(float((p.double() * q.double()).abs().sum()) for p, q in zip(rows, drows))
    assert abs(a - b) <= 2 * 2.0 ** -8 * size and abs(b - c) <= 2 * 2.0 ** -8 * size
