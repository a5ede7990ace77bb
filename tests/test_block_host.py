"""Refusals of the operators around the dispatch (arguments are checked before anything is queued, so none of this needs a
GPU), the layout of 8-bit rows, and the 64-bit forms that the GPU tests compare with."""
import ctypes as C

import numpy as np
import pytest
import torch

from collective_communication_schedules_gb300 import hoc
from tests import block_ref

P = 4096  # a non-NULL, aligned address that no refused call may follow
BAD = hoc.ERR_INVALID_ARG


def f32(v):
    return None if v is None else C.byref(C.c_float(v))


def f64(v):
    return None if v is None else C.byref(C.c_double(v))


F32, BF = hoc.FLOAT32, hoc.BFLOAT16


def norm(rows=4, width=64, dt=BF, x=P, ldx=64, r=None, ldr=64, w=P, wdt=BF, eps=1e-6, h=None, ldh=64, y=P, ldy=64, wire=None):
    return hoc.lib().hoc_rms_norm(rows, width, dt, x, ldx, r, ldr, w, wdt, f32(eps), h, ldh, y, ldy, wire, None)


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(width=0), dict(width=32769, ldx=40000, ldy=40000), dict(dt=hoc.INT32), dict(wdt=hoc.UINT8),
    dict(x=None), dict(x=P + 1), dict(dt=F32, x=P + 2), dict(ldx=63), dict(r=P, ldr=8), dict(r=P + 1), dict(w=None),
    dict(w=P + 1), dict(wdt=F32, w=P + 2), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=None), dict(h=P), dict(r=P, h=P, ldh=3),
    dict(y=None), dict(ldy=1), dict(wire=P + 8), dict(ldx=2 ** 60),
])
def test_norm_refuses(bad):
    assert norm(**bad) == BAD
    assert hoc.last_error_detail().startswith("hoc_rms_norm: ")


def grad(rows=4, width=64, dt=BF, dy=P, lddy=64, dy2=None, lddy2=64, h=P, ldh=64, w=P, wdt=BF, eps=1e-6, dres=None, lddres=64,
         dx=P, lddx=64, dw=P, dwdt=F32, ws=P, ints=4 * 64):
    return hoc.lib().hoc_rms_norm_grad(rows, width, dt, dy, lddy, dy2, lddy2, h, ldh, w, wdt, f32(eps), dres, lddres, dx, lddx, dw,
                                       dwdt, 0, ws, ints, None)


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(width=0), dict(width=32769), dict(dt=hoc.UINT8), dict(dwdt=hoc.INT32), dict(dy=None), dict(h=None),
    dict(dx=None), dict(w=None), dict(dy2=P + 1), dict(dres=P, lddres=63), dict(ldh=2), dict(dw=P + 2), dict(ws=None),
    dict(ints=4 * 64 - 1), dict(ws=P + 4), dict(eps=float("inf") * 0),
])
def test_norm_gradient_refuses(bad):
    assert grad(**bad) == BAD
    assert hoc.last_error_detail().startswith("hoc_rms_norm_grad: ")


def test_calls_on_no_rows_do_nothing():
    assert norm(rows=0, x=None, y=P) == hoc.SUCCESS
    assert grad(rows=0, dy=None, h=None, dx=None, dw=None, ws=None, ints=0) == hoc.SUCCESS
    assert hoc.lib().hoc_dropout(0, 8, BF, None, 8, None, 0, f64(0.5), P, None, 8, None) == hoc.SUCCESS
    assert hoc.lib().hoc_dropout(8, 0, BF, None, 0, None, 0, f64(0.5), P, None, 0, None) == hoc.SUCCESS
    assert route(tokens=0, logits=None, ids=None, gate=None) == hoc.SUCCESS
    assert widen(cap=(0,), wire=(None,), y=(None,)) == hoc.SUCCESS


def widen(k=1, experts=2, sources=1, seg=P, cap=(8,), wire=(P,), y=(P,), width=64, counts=None):
    g = hoc._RowGroups(k, experts, sources, seg, (C.c_size_t * len(cap))(*cap))
    return hoc.lib().hoc_expert_widen(C.byref(g), (C.c_void_p * len(wire))(*wire), width, (C.c_void_p * len(y))(*y), counts, None)


@pytest.mark.parametrize("bad", [
    dict(k=0), dict(k=17, cap=(1,) * 17), dict(experts=0), dict(sources=0), dict(seg=None), dict(seg=P + 4), dict(cap=(2 ** 31,)),
    dict(wire=(None,)), dict(wire=(P + 8,)), dict(y=(None,)), dict(y=(P + 1,)), dict(width=0), dict(width=32769), dict(counts=P + 4),
])
def test_widen_refuses(bad):
    assert widen(**bad) == BAD


def route(tokens=4, experts=64, topk=6, logits=P, dt=BF, ld=64, score=0, bias=None, groups=1, top=1, renorm=0, scale=1.0, ids=P,
          gate=P):
    return hoc.lib().hoc_ep_route(tokens, experts, topk, logits, dt, ld, score, bias, groups, top, renorm, f32(scale), ids, gate, None)


@pytest.mark.parametrize("bad", [
    dict(tokens=-1), dict(experts=0), dict(experts=1025, ld=1025), dict(topk=0), dict(topk=65), dict(topk=32), dict(logits=None),
    dict(logits=P + 1), dict(dt=hoc.INT32), dict(ld=63), dict(score=2), dict(score=-1), dict(bias=P + 2), dict(groups=0),
    dict(groups=7), dict(groups=64, top=64), dict(groups=8, top=0), dict(groups=8, top=9), dict(groups=16, top=1),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=None), dict(ids=None), dict(gate=None), dict(ids=P + 2),
])
def test_route_refuses(bad):
    assert route(**bad) == BAD
    assert hoc.last_error_detail().startswith("hoc_ep_route: ")


@pytest.mark.parametrize("bad", [
    dict(tokens=-1), dict(experts=0), dict(topk=65), dict(dt=hoc.UINT8), dict(ld=1), dict(score=5), dict(ids=None), dict(dgate=None),
    dict(out=None), dict(out=P + 1), dict(ldd=63), dict(scale=float("nan")),
])
def test_route_gradient_refuses(bad):
    a = dict(tokens=4, experts=64, topk=6, logits=P, dt=BF, ld=64, score=0, renorm=0, scale=1.0, ids=P, dgate=P, out=P, ldd=64)
    a.update(bad)
    assert hoc.lib().hoc_ep_route_grad(a["tokens"], a["experts"], a["topk"], a["logits"], a["dt"], a["ld"], a["score"], a["renorm"],
                                       f32(a["scale"]), a["ids"], a["dgate"], a["out"], a["ldd"], None) == BAD


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(width=-1), dict(dt=hoc.INT32), dict(x=None), dict(x=P + 1), dict(ldx=7), dict(r=P + 1), dict(r=P, ldr=1),
    dict(p=-0.1), dict(p=1.0), dict(p=float("nan")), dict(p=None), dict(seed=None), dict(seed=P + 4), dict(y=None), dict(ldy=7),
])
def test_dropout_refuses(bad):
    a = dict(rows=4, width=8, dt=BF, x=P, ldx=8, r=None, ldr=0, p=0.5, seed=P, y=P, ldy=8)
    a.update(bad)
    assert hoc.lib().hoc_dropout(a["rows"], a["width"], a["dt"], a["x"], a["ldx"], a["r"], a["ldr"], f64(a["p"]), a["seed"], a["y"],
                                 a["ldy"], None) == BAD


def test_the_binding_refuses_what_is_not_on_the_gpu_or_of_another_type():
    x, w = torch.zeros(4, 8), torch.zeros(8)
    with pytest.raises(ValueError):
        hoc.rms_norm(x, w, x, eps=1e-6)
    with pytest.raises(TypeError):
        hoc.rms_norm(x.half(), w, x, eps=1e-6)
    with pytest.raises(TypeError):
        hoc.rms_norm_grad(x.int(), x, w, x, eps=1e-6)
    with pytest.raises(ValueError):
        hoc.ep_route(x, torch.zeros(8, dtype=torch.int32), torch.zeros(8))
    with pytest.raises(ValueError):
        hoc.dropout(x, x, 0.1, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):
        hoc.ep_route_grad(x, torch.zeros(8, dtype=torch.int32), torch.zeros(8), x, score="tanh")
    with pytest.raises(ValueError):
        hoc.wire8_views(torch.zeros(2, 7, dtype=torch.uint8), 64)


@pytest.mark.parametrize("width", [1, 15, 16, 64, 127, 128, 129, 1001, 2048, 4096, 32768])
def test_the_layout_of_rows_of_8_bits(width):
    n, groups = hoc.wire8_bytes(width), -(-width // 128)
    at = -(-width // 16) * 16
    assert n % 16 == 0 and at + 4 * groups <= n < at + 4 * groups + 16
    wire = torch.arange(3 * n, dtype=torch.int64).to(torch.uint8).view(3, n)
    q, scale = hoc.wire8_views(wire, width)
    assert q.shape == (3, width) and scale.shape == (3, groups)
    assert torch.equal(q.view(torch.uint8), wire[:, :width])
    assert scale.data_ptr() == wire.data_ptr() + at


def test_workspaces_grow_with_rows_up_to_a_limit():
    assert hoc.rms_norm_workspace(1, 100) == 100
    assert hoc.rms_norm_workspace(0, 100) == 100
    assert hoc.rms_norm_workspace(7, 100) == 700
    assert hoc.rms_norm_workspace(10 ** 9, 100) == hoc.rms_norm_workspace(10 ** 6, 100)
    with pytest.raises(hoc.HocError):
        hoc.rms_norm_workspace(1, 0)


def test_the_generator_is_the_published_one():
    """Philox4x32-10's known answers for a counter and key of zeros, of ones and of digits of pi (the paper's own test
    vectors)."""
    def words(ctr, key):
        # element 8 g draws from the counter (g, call): g and call hold two words each
        g, call = ctr[0] | ctr[1] << 32, ctr[2] | ctr[3] << 32
        c = [np.array([v], dtype=np.uint64) for v in ctr]
        mask = np.uint64(0xFFFFFFFF)
        k = [np.uint64(key[0]), np.uint64(key[1])]
        for _ in range(10):
            a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
            c = [(b >> np.uint64(32)) ^ c[1] ^ k[0], b & mask, (a >> np.uint64(32)) ^ c[3] ^ k[1], a & mask]
            k = [(k[0] + np.uint64(0x9E3779B9)) & mask, (k[1] + np.uint64(0xBB67AE85)) & mask]
        if g == 0:
            bits = block_ref.philox_bits(8, (key[0] | key[1] << 32, call)).tolist()
            assert [bits[2 * i] | bits[2 * i + 1] << 16 for i in range(4)] == [int(v[0]) for v in c]
        return [int(v[0]) for v in c]

    assert words([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert words([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert words([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0]) == \
        [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_the_routing_form_picks_what_a_sort_picks():
    g = torch.Generator().manual_seed(1)
    z = torch.randn(50, 24, generator=g)
    ids, gate = block_ref.route(z, 5, "softmax")
    want = z.double().sort(dim=1, descending=True, stable=True)
    assert torch.equal(ids.long(), want.indices[:, :5])
    assert torch.allclose(gate, torch.softmax(z.double(), 1).gather(1, want.indices[:, :5]), rtol=1e-12)
    ids, gate = block_ref.route(z, 5, "sigmoid", renormalise=True, scale=2.5)
    assert torch.allclose(gate.sum(1), torch.full((50,), 2.5, dtype=torch.float64))
