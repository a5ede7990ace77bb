"""Counts that an int does not hold, and host numbers, on their way through the binding: a stand-in takes the library's place,
with the same argument types, so that none of this needs a GPU.  The tensors have a shape and no memory."""
import ctypes as C

import pytest
import torch

from collective_communication_schedules_gb300 import hoc

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
TOP = 1 << 31


class Recorder:
    """The library's functions, which keep what ctypes makes of their arguments."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        kinds = hoc._SIGS[name][1]

        def call(*args):
            assert len(args) == len(kinds)
            self.calls.append((name, [k(a).value if k in (C.c_int, C.c_int64, C.c_size_t) else a for k, a in zip(kinds, args)]))
            return hoc.SUCCESS
        return call


@pytest.fixture
def calls(monkeypatch):
    lib = Recorder()
    monkeypatch.setattr(hoc, "_lib", lib)
    monkeypatch.setattr(hoc, "_here", lambda x, what: x.get_device())
    monkeypatch.setattr(hoc, "_queue", lambda stream, device: 0)
    return lib.calls


def empty(*shape, dtype=BF):
    return torch.empty(shape, dtype=dtype, device="meta")


SEED = empty(2, dtype=torch.int64)


@pytest.mark.parametrize("shape", [
    (TOP - 1,), (TOP,), (2 * TOP,), (2 * TOP + 5,), (2 * TOP + 15,), (3, TOP + 1), (2, 2 * TOP), (5, 7, TOP), (TOP, 3, 1), (TOP, 8),
    (2 * TOP + 5, 1), (0, TOP), (TOP, 0), (3, 0, TOP), (4, 5, 6), (),
])
def test_dropout_hands_on_every_element_of_any_shape(calls, shape):
    x = empty(*shape)
    hoc.dropout(x, x, 0.5, SEED, residual=x)
    (name, args), = calls
    rows, width, ldx, ldr, ldy = args[0], args[1], args[4], args[6], args[10]
    assert name == "hoc_dropout" and rows * width == x.numel() and 0 <= width < TOP
    assert ldx == ldr == ldy == max(width, 1) or rows <= 1 or width <= 1


def test_dropout_of_rows_too_wide_for_an_int_wants_them_together(calls):
    x = empty(2, 2 * TOP + 8)[:, :2 * TOP]
    with pytest.raises(ValueError):
        hoc.dropout(x, x, 0.5, SEED)
    assert not calls


def test_dropout_refuses_more_than_a_grid_reaches():
    p = C.c_double(0.5)
    for rows, width in ((1 << 43, 1), (1 << 62, 1), (1 << 40, 8), (1 << 33, 1 << 30), ((1 << 12) + 1, TOP - 1)):
        assert hoc.lib().hoc_dropout(rows, width, hoc.BFLOAT16, 4096, width, None, 0, C.byref(p), 4096, 4096, width, None) == \
            hoc.ERR_INVALID_ARG


@pytest.mark.parametrize("shape", [(TOP, 64), (2 * TOP, 64), (2 * TOP + 5, 8), (1, 2 * TOP + 64), (0, 2 * TOP + 64)])
def test_norms_refuse_counts_that_an_int_does_not_hold(calls, shape):
    x, w = empty(*shape), empty(shape[1], dtype=F32)
    with pytest.raises(ValueError):
        hoc.rms_norm(x, w, x, eps=1e-6)
    with pytest.raises(ValueError):
        hoc.rms_norm_grad(x, x, w, x, eps=1e-6)
    with pytest.raises(ValueError):
        hoc.rms_norm_workspace(*shape)
    assert not calls


@pytest.mark.parametrize("shape,topk", [((TOP, 8), 2), ((2 * TOP + 3, 8), 2), ((1, 2 * TOP + 8), 2), ((1, 8), 2 * TOP + 1)])
def test_routing_refuses_counts_that_an_int_does_not_hold(calls, shape, topk):
    z, ids, gate = empty(*shape), empty(shape[0] * topk, dtype=I32), empty(shape[0] * topk, dtype=F32)
    with pytest.raises(ValueError):
        hoc.ep_route(z, ids, gate)
    with pytest.raises(ValueError):
        hoc.ep_route_grad(z, ids, gate, z)
    assert not calls


@pytest.mark.parametrize("groups", [dict(groups=2 * TOP + 1), dict(groups=2, top_groups=2 * TOP + 1), dict(top_groups=2 * TOP + 1),
                                    dict(groups=1 - 2 * TOP)])
def test_routing_refuses_groups_that_an_int_does_not_hold(calls, groups):
    z, ids, gate = empty(4, 8), empty(8, dtype=I32), empty(8, dtype=F32)
    with pytest.raises(ValueError):
        hoc.ep_route(z, ids, gate, **groups)
    assert not calls


def test_rows_of_8_bits_refuse_counts_that_an_int_does_not_hold(calls):
    with pytest.raises(ValueError):
        hoc.wire8_bytes(2 * TOP + 64)
    y, wire = empty(0, 2 * TOP + 64), empty(0, 80, dtype=torch.uint8)
    with pytest.raises(ValueError):
        hoc.expert_widen([wire], empty(1, 2, dtype=torch.int64), [y])
    with pytest.raises(ValueError):
        hoc.expert_widen([empty(4, 80, dtype=torch.uint8)], empty(1, TOP + 1, dtype=torch.int64), [empty(4, 64)])
    assert all(name == "hoc_wire8_row" for name, _ in calls)


def test_a_number_that_lies_in_a_tensor_is_read_at_every_call():
    for kind in (C.c_float, C.c_double):
        t = torch.tensor(2.0)
        first = hoc._number(t, kind)._obj
        t.fill_(5.0)
        assert hoc._number(t, kind)._obj.value == 5.0 and first.value == 2.0
        p = torch.nn.Parameter(torch.tensor([0.5]), requires_grad=False)
        assert hoc._number(p, kind)._obj.value == 0.5
        p.mul_(0.5)
        assert hoc._number(p, kind)._obj.value == 0.25
    assert all(type(v) is float for _, v in hoc._NUMBERS), "what it holds would live as long as the table"


def test_numbers_reach_the_calls_as_they_are(calls):
    x, w, eps = empty(4, 8), empty(8, dtype=F32), torch.tensor(0.5)
    for want in (0.5, 0.25, 1, 0.125):
        eps.fill_(want)
        hoc.rms_norm(x, w, x, eps=eps)
        hoc.ep_route(x, empty(8, dtype=I32), empty(8, dtype=F32), scale=eps)
        hoc.dropout(x, x, eps, SEED)
        (_, norm), (_, route), (_, drop) = calls[-3:]
        assert norm[9]._obj.value == route[11]._obj.value == drop[7]._obj.value == want


def test_what_is_no_number_is_refused():
    for v in ("0.5", None, torch.zeros(2)):
        with pytest.raises((TypeError, ValueError, RuntimeError)):
            hoc._number(v)


def test_a_width_that_lies_in_a_tensor_is_read_at_every_call():
    w = torch.tensor(64)
    assert hoc.wire8_bytes(w) == hoc.wire8_bytes(64)
    w.fill_(2048)
    assert hoc.wire8_bytes(w) == hoc.wire8_bytes(2048) and all(type(v) is int for v in hoc._WIRE8)
