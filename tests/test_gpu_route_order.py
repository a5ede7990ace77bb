"""Which experts a routing chooses where its binary32 keys alone would choose others."""
import math

import pytest
import torch

from tests.test_gpu_block import BF, DEV, F32, check_route, gen, route

pytestmark = pytest.mark.gpu
F64 = torch.float64


def border_keys(tokens, experts, step, sure, g):
    """Sigmoid keys above 1, in units of 2^-23: expert b a little below or above a multiple of `step` and c too, a at the end of
    the range behind it, d at the start of the one before it, in the order b, a, d, c.  Keys are put in order without their last
    bits, in ranges of `step`, and a range's by their experts: with b rounded up and c down, a is the last that is chosen and d
    the first that is not, which lie far apart, and c behind them may still be larger than b.  `sure` more are chosen anyway."""
    spots = torch.arange(4) * (experts // 8) + (experts > 32)
    base = 1.6 + torch.rand(4, generator=g, dtype=F64)
    bias = torch.zeros(experts)
    bias[spots] = (1 - torch.sigmoid(base)).float()
    bias[experts - sure:] = 1.5 + 0.25 * torch.arange(sure)
    low = torch.tensor([3 * step - 1.0, 4 * step - 4.5, 2 * step + 0.5, 3 * step - 1.0], dtype=F64)
    wide = torch.tensor([1.0, 3.8, 3.0, 1.0], dtype=F64)
    key = 1 + (low + wide * torch.rand(tokens, 4, generator=g, dtype=F64)) * 2.0 ** -23
    z = torch.full((tokens, experts), -3.0)
    z[:, spots] = torch.special.logit(key - bias[spots].double()).float()
    return z.to(DEV), bias.to(DEV)


@pytest.mark.parametrize("tokens,experts,step,sure,calls", [
    (60, 32, 32, 0, 40), (60, 64, 32, 0, 40), (60, 128, 32, 0, 40), (60, 256, 32, 0, 40), (2500, 64, 16, 8, 10),
])
def test_what_follows_the_first_that_is_left_out_may_still_be_chosen(tokens, experts, step, sure, calls):
    g = torch.Generator().manual_seed(experts + step)
    for _ in range(calls):
        z, bias = border_keys(tokens, experts, step, sure, g)
        check_route(z, 2 + sure, bias, "sigmoid")


@pytest.mark.parametrize("experts,groups,top_groups,topk", [(32, 4, 2, 12), (32, 4, 3, 20), (64, 8, 4, 16), (256, 8, 4, 31), (40, 8, 5, 12)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("tokens", [9, 10_000])
def test_groups_closed_by_the_lowest_finite_bias_come_last_and_are_there(experts, groups, top_groups, topk, score, dtype, tokens):
    """The sum of two such keys is no binary32 number.  One group is open, of the others one has an open expert, or none has."""
    g = gen(experts)
    z = torch.randn(tokens, experts, generator=g, device=DEV).to(dtype)
    per = experts // groups
    bias = torch.full((experts,), torch.finfo(F32).min, device=DEV)
    bias[2 * per: 3 * per] = 0.25
    check = z[:500] if tokens > 500 else z  # (the 64-bit form goes token by token)
    for _ in range(2):
        ids, gate = check_route(check, topk, bias, score, groups, top_groups)
        assert bool((ids >= 0).all())
        if tokens > 500:
            all_ids, all_gate = route(z, topk, bias=bias, score=score, groups=groups, top_groups=top_groups)
            assert torch.equal(all_ids[:500], ids) and bool((all_ids >= 0).all())
        bias[0] = 0.5


@pytest.mark.parametrize("masked", [False, True])
def test_groups_of_one_key_are_in_doubt_as_their_keys_are(masked):
    """The same keys, each the only one of its group: alone in it, or beside a masked one."""
    g = torch.Generator().manual_seed(7)
    for _ in range(60):
        z, bias = border_keys(60, 32, 32, 0, g)
        groups = 32
        if masked:
            groups = 16
            z = torch.stack([z[:, :16], torch.full_like(z[:, :16], -math.inf)], 2).reshape(60, 32)
            bias = torch.stack([bias[:16], torch.zeros_like(bias[:16])], 1).reshape(32)
        check_route(z, 2, bias, "sigmoid", groups, 2)
