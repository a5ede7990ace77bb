"""Counts that an int does not hold, on their way through the binding of the expert-parallel and layer calls: a stand-in takes
the library's place, with the same argument types, so that none of this needs a GPU.  The tensors have a shape and no memory."""
import pytest
import torch

from collective_communication_schedules_gb300 import hoc
from tests.test_block_counts import Recorder, empty

TOP = 1 << 31
MUCH = [TOP, 2 * TOP, 2 * TOP + 5]
I32, I64 = torch.int32, torch.int64


@pytest.fixture
def calls(monkeypatch):
    lib = Recorder()
    monkeypatch.setattr(hoc, "_lib", lib)
    monkeypatch.setattr(hoc, "lib", lambda: lib)
    monkeypatch.setattr(hoc, "_ptr", lambda x, *a: 0)
    monkeypatch.setattr(hoc, "_ptr_array", lambda xs, *a: None)
    monkeypatch.setattr(hoc, "_shaped", lambda x, shape, *a: 0)
    monkeypatch.setattr(hoc, "_strided", lambda x, shape, what: (0, shape[1]))
    monkeypatch.setattr(hoc, "_stream", lambda stream: 0)
    return lib.calls


def refused(calls, call, *args, **kw):
    with pytest.raises(ValueError, match="2\\^31"):
        call(*args, **kw)
    assert not calls


@pytest.mark.parametrize("n", MUCH)
def test_expert_parallel_calls(calls, n):
    ws, one = empty(8, dtype=I32), empty(1, dtype=I32)
    ids, x = empty(2 * n, dtype=I32), empty(n, 8)
    refused(calls, hoc.ep_pack_workspace, n, 2, 8)
    refused(calls, hoc.ep_pack_workspace, 8, 2, n)
    refused(calls, hoc.ep_pack, ids, x, 8, 2, x, ids, ids, one, ws)
    refused(calls, hoc.ep_pack, empty(16, dtype=I32), empty(8, 8), n, 2, x, ids, ids, one, ws)
    refused(calls, hoc.ep_pack, empty(16, dtype=I32), empty(8, 8), 8, n, x, ids, ids, one, ws)
    refused(calls, hoc.ep_combine, x, ids, ids, n, 2, 8, x)
    refused(calls, hoc.ep_combine, x, ids, ids, 8, 2, n, x)
    refused(calls, hoc.ep_pack_all, [ids], [x], 8, [x], [8], [ids], one, ws, one)
    refused(calls, hoc.ep_dispatch_fused, [ids], [x], 8, [x], [8], [ids], one, ws, one)
    refused(calls, hoc.ep_combine_all, [x], [8], [ids], [ids], n, 2, 8, [x], one)
    refused(calls, hoc.ep_combine_fused, [x], [8], [ids], [ids], one, [ids], n, 2, 8, 4, [x], one)
    refused(calls, hoc.ep_combine_fused, [x], [8], [ids], [ids], one, [ids], 8, 2, 8, n, [x], one)
    refused(calls, hoc.ep_combine_grad, [x], [x], [8], [ids], [ids], one, [ids], n, 2, 8, 4, [x], [ids], one)
    refused(calls, hoc.ep_combine_grad_all, [x], [x], [8], [ids], [ids], n, 2, 8, [x], [ids], one)
    refused(calls, hoc.ep_segments, [ids], 8, 2, empty(1, 9, dtype=I64))
    refused(calls, hoc.ep_segments, [empty(16, dtype=I32)], n, 2, empty(1, n + 1, dtype=I64))


@pytest.mark.parametrize("n", MUCH)
def test_layer_calls(calls, n):
    one, rows, wide, w = empty(1, dtype=I32), empty(n, 8), empty(4, n), empty(8, 8)
    refused(calls, hoc.linear, rows, w, rows, status=one)
    refused(calls, hoc.linear, wide, empty(8, n), empty(4, 8), status=one)
    refused(calls, hoc.linear, empty(4, 8), empty(n, 8), wide, status=one)
    refused(calls, hoc.linear_dgrad, rows, w, rows, status=one)
    refused(calls, hoc.linear_wgrad, rows, rows, w, status=one)
    refused(calls, hoc.act_grad, rows, rows, rows, "relu")
    refused(calls, hoc.act_grad, wide, wide, wide, "relu")
    seg = empty(1, 5, dtype=I64)
    refused(calls, hoc.expert_mm, [wide], [empty(4, 8, n)], seg, [empty(4, 8)], status=one)
    refused(calls, hoc.expert_mm_dgrad, [wide], [empty(4, n, 8)], seg, [empty(4, 8)], status=one)
    refused(calls, hoc.expert_mm_wgrad, [wide], [empty(4, 8)], seg, [empty(4, n, 8)], status=one)
    refused(calls, hoc.expert_mm, [empty(4, 8)], [empty(1, 8, 8)], empty(1, n + 1, dtype=I64), [empty(4, 8)], status=one)
