"""The norm's gradient without eps on rows so small that 1 / mean(h^2) is no binary32 number, while every result is one."""
import pytest
import torch

from collective_communication_schedules_gb300 import hoc
from tests import block_ref as ref
from tests.test_gpu_block import BF, DEV, F32, gen, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("width", [64, 1001, 2048, 9000, 16384, 32768])
def test_gradient_of_tiny_rows(width, dtype):
    """Squares near 1e-39 are off by half of 2^-149 each, 2^-20 of their mean, and so is the mean; half of that in 1 / sqrt,
    which an element of dx has three times at most: 2^-18.4 beside the 2^-18 of ordinary rows, of what its terms add up to."""
    g = gen(width)
    h = (torch.randn(5, width, generator=g, device=DEV) * 3e-20).to(dtype)
    dy = torch.randn(5, width, generator=g, device=DEV).to(dtype)
    w, dx, dw = torch.ones(width, device=DEV), torch.empty_like(dy), torch.empty(width, device=DEV)
    ws = torch.empty(hoc.rms_norm_workspace(5, width), dtype=torch.int32, device=DEV)
    hoc.rms_norm_grad(dy, h, w, dx, eps=0.0, dw=dw, workspace=ws)
    want, terms, ww, wterms = ref.norm_grad(dy.cpu(), None, h.cpu(), w.cpu(), 0.0, None)
    within(dx, want, ref.half_step(dtype) * want.abs() + 2.0 ** -17 * terms, "dx")
    within(dw, ww, 2.0 ** -18 * wterms, "dw")
