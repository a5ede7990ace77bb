"""Rank buffers of a call that is split into several launches (more than 1024 experts in all): how the rows of each
launch are moved follows from that launch's own buffers."""
import os
import subprocess

import pytest
import torch

from collective_communication_schedules_gb300 import build, hoc
from tests import layer_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIBDIR = os.path.dirname(hoc.LIB_PATH)
DEV, BF = "cuda", torch.bfloat16


def test_the_rule_looks_at_the_launch_s_own_buffers(tmp_path):
    if not os.path.exists(hoc.LIB_PATH):
        pytest.skip("libhoc.so is not built")
    out = str(tmp_path / "loose")
    cmd = [build.nvcc()] + build.ARCH + ["-std=c++17", "-cudart", "static", "-I", build.INCLUDE, "-I", build.CSRC,
                                         os.path.join(ROOT, "tests", "c", "loose.cu"), "-L", LIBDIR, "-lhoc",
                                         "-Xlinker", f"-rpath={LIBDIR}", "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([out], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "LOOSE OK" in r.stdout, r.stdout + r.stderr


def normal(*shape, seed=0, sigma=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * sigma).to(BF)


def placed(shape, off):
    """A tensor of sevens `off` elements behind a 16-byte boundary, and the buffer around it."""
    n = 1
    for v in shape:
        n *= v
    around = torch.full((n + off + 9,), 7.0, dtype=BF, device=DEV)
    return around[off: off + n].view(shape), around


@pytest.mark.gpu
@pytest.mark.parametrize("first,second", [(0, 1), (1, 0), (3, 0), (0, 4)])
@pytest.mark.parametrize("k,experts", [(2, 600), (3, 400), (2, 1030)])
def test_outputs_of_every_rank_whatever_their_alignment(k, experts, first, second):
    """All three products over more experts than a launch takes: outputs of the first rank `first` elements off a
    16-byte boundary, those of the others `second`; every rank's results, and nothing beside them."""
    inp, out = 24, 16
    L = ref.Routed(ref.random_counts(k, 1, experts, 4, experts + k))
    off = [first] + [second] * (k - 1)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    x, dy = [normal(n, inp, seed=1 + d) for d, n in enumerate(L.cap)], [normal(n, out, seed=9 + d) for d, n in enumerate(L.cap)]
    w = [normal(experts, out, inp, seed=20 + d, sigma=0.2) for d in range(k)]
    below = [placed((n, inp), off[d]) for d, n in enumerate(L.cap)]
    for d, (t, _) in enumerate(below):
        t.copy_(normal(*t.shape, seed=40 + d))
    y, pre = [placed((n, out), off[d]) for d, n in enumerate(L.cap)], [placed((n, out), off[d]) for d, n in enumerate(L.cap)]
    dx, dw = [placed((n, inp), off[d]) for d, n in enumerate(L.cap)], [placed((experts, out, inp), off[d]) for d in range(k)]
    hoc.expert_mm(x, w, L.seg, [t for t, _ in y], status=st, act="silu", pre=[t for t, _ in pre])
    hoc.expert_mm_dgrad(dy, w, L.seg, [t for t, _ in dx], status=st, act="gelu", pre=[t for t, _ in below])
    hoc.expert_mm_wgrad(dy, x, L.seg, [t for t, _ in dw], status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    for d in range(k):
        has = L.of[d] >= 0
        own = L.of[d][has]
        wd = w[d].double()[own]
        xs, ds = x[d][has].double(), dy[d][has].double()
        z, ez = torch.einsum("rk,rok->ro", xs, wd), torch.einsum("rk,rok->ro", xs.abs(), wd.abs()) * inp * ref.F32
        ref.close(pre[d][0][has], z, ez, f"pre {d}")
        want = ref.act("silu", z)
        ref.close(y[d][0][has], want, ez * ref.SLOPE + (want.abs() + z.abs()) * ref.MATH, f"y {d}")
        v, ev = torch.einsum("ro,rok->rk", ds, wd), torch.einsum("ro,rok->rk", ds.abs(), wd.abs()) * out * ref.F32
        p = below[d][0][has].double()
        ref.close(dx[d][0][has], v * ref.slope("gelu", p),
                  ref.SLOPE * ev + v.abs() * 4 * ref.MATH * (1 + p.abs().clamp(max=32)), f"dx {d}")
        pair = torch.einsum("ro,rk->rok", ds, xs)
        want = torch.zeros(experts, out, inp, dtype=torch.float64, device=DEV).index_add_(0, own, pair)
        err = torch.zeros_like(want).index_add_(0, own, pair.abs()) * 4 * ref.F32
        ref.close(dw[d][0], want, err, f"dw {d}")
        for t, around in (y[d], pre[d], dx[d], dw[d]):
            assert bool((around[:off[d]] == 7).all()) and bool((around[off[d] + t.numel():] == 7).all())
        for t, _ in (y[d], pre[d], dx[d]):
            assert bool((t[~has] == 7).all()), "a row of no range was written"
