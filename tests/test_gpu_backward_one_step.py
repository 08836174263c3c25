"""The backward pass of a single step with no state before it: y is v whatever k
and u are, so gk, gu and gw are exactly zero."""

import pytest
import torch

from rwkv_wkv_linear_b200 import wkv4
from tests.test_gpu_backward import _check, _inputs, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_device_errors(cuda_device):
    yield
    assert wkv4.device_error(reset=True) == 0


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("B,C", [(1, 8), (3, 72), (5, 1027)])
def test_one_step_without_a_state(cuda_device, B, C, gated, dt):
    x = _inputs(B, 1, C, dt, seed=B + C, gated=gated, state=False)
    g, _ = _run(x, cuda_device)
    for name in ("gk", "gu", "gw"):
        assert not getattr(g, name).any(), name
    _check(x, g, None, dt, "one step")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 33, 129])
def test_a_last_chunk_of_one_step(cuda_device, T, dt):
    """With a state, or with steps before it, a chunk of one step is like any other."""
    for state in (False, True):
        x = _inputs(2, T, 70, dt, seed=T, gated=True, state=state)
        g, s = _run(x, cuda_device)
        _check(x, g, s, dt, f"{T} steps")


def test_zero_state_given(cuda_device):
    """The empty state given in so many words is no other than none."""
    x = _inputs(2, 1, 40, "f32", seed=3, gated=False, state=False)
    d = {a: None if t is None else t.to(cuda_device) for a, t in x.items()}
    s = torch.zeros(3, 2, 40, device=cuda_device)
    s[2] = -1e38
    g = wkv4.backward(d["k"], d["v"], d["w"], d["u"], d["gy"], s)
    torch.cuda.synchronize()
    assert not g.gk.any() and not g.gu.any() and not g.gstate_in.any()


def test_a_state_with_a_numerator_alone(cuda_device):
    """A state whose denominator is zero is not an empty one: y is not v."""
    x = _inputs(2, 1, 40, "f32", seed=4, gated=False, state=True)
    x["state_in"][1] = 0
    g, s = _run(x, cuda_device)
    _check(x, g, s, "f32", "numerator alone")
    assert g.gk.any()
