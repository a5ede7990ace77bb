"""Dropout of runs whose length is no product of two ints: 2^32 elements and more, checked at their start, around 2^32 and at
their end."""
import pytest
import torch

from collective_communication_schedules_gb300 import hoc
from tests import block_ref as ref

pytestmark = pytest.mark.gpu
DEV, BF, F64 = "cuda", torch.bfloat16, torch.float64


@pytest.mark.parametrize("n", [2 ** 31, 2 ** 32 + 15])  # (the second is a prime)
@pytest.mark.parametrize("offset", [0, 1])  # vectors, elements
def test_dropout_of_a_run_past_2_to_the_31(n, offset):
    seed, t = (5, 6), 16384
    flat = torch.empty(n + offset, dtype=BF, device=DEV)
    x = flat[offset:]
    x.fill_(3.0)
    hoc.dropout(x, x, 0.25, torch.tensor(seed, device=DEV))
    scaled = torch.tensor(3.0 * 65536 / (65536 - t), dtype=F64).to(BF)  # 4, exactly
    for first in (0, 2 ** 31 - 4096, 2 ** 32 - 4096, n - n % 8 - 4096):
        if first < 0 or first >= n:
            continue
        got = x[first: first + 8192].cpu()
        keep = ref.philox_bits(len(got), seed, first) >= t
        assert torch.equal(got, torch.where(keep, scaled, torch.zeros((), dtype=BF))), first
    assert not bool((x[-1000:] == 3).any())
    gone = sum(int((part == 0).sum()) for part in x.split(1 << 28))
    assert abs(gone - n / 4) <= 6 * (n * 3 / 16) ** 0.5
    assert sum(int((part == 3).sum()) for part in x.split(1 << 28)) == 0
