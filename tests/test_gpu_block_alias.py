"""An expert block without a residual holds x itself for its backward pass, which a forward pass onto x takes away."""
import pytest
import torch

from collective_communication_schedules_gb300.expert_block import ExpertBlock
from tests.test_gpu_expert_block import outputs, problem

pytestmark = pytest.mark.gpu


def run(block, p, y, residual=None):
    block.forward(p["x"], p["norm"], p["router"], p["w_up"], p["w_down"], y, residual=residual, seed=p["seed"])


def back(block, p, o):
    block.backward(p["dy"], p["norm"], p["router"], p["w_up"], p["w_down"], o["dx"], o["dnorm"], o["drouter"], o["dup"], o["ddown"],
                   seed=p["seed"])


@pytest.mark.parametrize("drop", [0.0, 0.25])
def test_forward_onto_x(drop):
    p = problem(2, 40, 128, 64, 8, 3)
    block, o = ExpertBlock(2, 40, 2, 128, 64, 8, drop=drop), outputs(p)
    x = p["x"].clone()
    run(block, p, o["y"])
    back(block, p, o)
    want = {k: o[k].clone() for k in ("y", "dx", "dnorm", "drouter")}
    # with a residual both may be written over: the block keeps their sum
    r = torch.zeros_like(x)
    run(block, p, p["x"], residual=r)
    assert torch.equal(p["x"], want["y"])
    back(block, p, o)
    assert all(torch.equal(o[k], want[k]) for k in ("dx", "dnorm", "drouter"))
    # without one the results are there, and the gradients are refused
    p["x"].copy_(x)
    run(block, p, p["x"])
    assert torch.equal(p["x"], want["y"])
    with pytest.raises(ValueError):
        back(block, p, o)
    p["x"].copy_(x)  # until a forward pass leaves x again
    run(block, p, o["y"])
    back(block, p, o)
    assert all(torch.equal(o[k], want[k]) for k in ("dx", "dnorm", "drouter"))


def test_backward_needs_a_forward():
    p = problem(1, 8, 64, 32, 2, 1)
    block = ExpertBlock(1, 8, 1, 64, 32, 2)
    with pytest.raises(ValueError):
        back(block, p, outputs(p))


def test_backward_needs_the_whole_of_the_last_forward():
    p = problem(1, 8, 64, 32, 2, 1)
    block, o = ExpertBlock(1, 8, 1, 64, 32, 2), outputs(p)
    run(block, p, o["y"])
    with pytest.raises(ValueError):  # the router's shape: what the first pass kept is partly overwritten
        block.forward(p["x"], p["norm"], p["router"][:, :32].contiguous(), p["w_up"], p["w_down"], o["y"], seed=p["seed"])
    with pytest.raises(ValueError):
        back(block, p, o)
    run(block, p, o["y"])
    back(block, p, o)
