"""Tensor lists on other streams than the one that was current when they were made."""
import pytest
import torch

from collective_communication_schedules_gb300 import hoc

pytestmark = pytest.mark.gpu

DEV = "cuda"
BUSY = 200_000_000  # cycles: about a tenth of a second


@pytest.mark.parametrize("tensors", [1, 40, 6000])  # tables of one tile, of a few and of more than 64 KB
def test_a_list_is_on_the_device_when_it_has_been_made(tensors):
    """Creation returns when its upload, which the default stream runs in its turn, is complete."""
    src = [torch.ones(100, device=DEV) for _ in range(tensors)]
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    with hoc.TensorList(src):
        assert torch.cuda.default_stream().query(), "returned with work of the default stream under way"


@pytest.mark.parametrize("tensors", [1, 40, 6000])
def test_a_list_is_used_at_once_on_a_stream_of_its_own(tensors):
    src = [torch.full((100,), 2.0, device=DEV) for _ in range(tensors)]
    norm = torch.empty(1, device=DEV)
    ws = torch.empty(1 << 20, dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    with hoc.TensorList(src) as a:
        hoc.grad_clip(a, a, 1.0, norm, ws, stream=side)
        side.synchronize()
        want = 2 * (100 * tensors) ** 0.5
        assert abs(norm.item() - want) <= 1e-5 * want
        assert all(abs(float(t[99]) - 2 / want) <= 1e-5 for t in (src[0], src[-1]))
