"""The 8-bit values of a norm bit for bit: binary32 rows also get y as it was before the rounding to 8 bits."""
import pytest
import torch

from collective_communication_schedules_gb300 import hoc

pytestmark = pytest.mark.gpu
DEV, F32 = "cuda", torch.float32


@pytest.mark.parametrize("width", [64, 256, 1001, 2048, 4096, 9000, 20000])
@pytest.mark.parametrize("most", [7, 28, 56, 112, 440])
def test_codes_are_those_of_the_quotient(width, most):
    """Whole numbers times a factor: many quotients lie on a tie of e4m3 or a rounding beside it."""
    g = torch.Generator(device=DEV).manual_seed(width + most)
    x = torch.randint(-most, most + 1, (200, width), generator=g, device=DEV).to(F32)
    x[:, ::64] = most
    y = torch.empty_like(x)
    wire = torch.zeros(200, hoc.wire8_bytes(width), dtype=torch.uint8, device=DEV)
    hoc.rms_norm(x, torch.ones(width, device=DEV), y, eps=1e-6, wire=wire)
    q, scale = (t.cpu() for t in hoc.wire8_views(wire, width))
    y, groups = y.cpu(), scale.shape[1]
    wide = torch.zeros(200, groups * 128)
    wide[:, :width] = y
    want = wide.view(200, groups, 128).abs().amax(2) / 448
    assert torch.equal(scale, want)
    codes = (y / want.repeat_interleave(128, 1)[:, :width]).to(torch.float8_e4m3fn)
    assert torch.equal(q.view(torch.uint8), codes.view(torch.uint8))
