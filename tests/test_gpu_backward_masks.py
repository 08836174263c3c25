"""GPU gradients under finite masks: keys of -1e9, -1e10 or -1e30 in part of a
chunk, in whole chunks, CTAs and rounds, with nothing before them, against the
oracle that holds its sums to a running max; states whose max lies as low; and
what a padded row leaves of the other rows' gradients."""

import numpy as np
import pytest
import torch

from oracle import backward as ob
from rwkv_wkv_linear_b200 import wkv4
from tests import gradcheck
from tests.test_gpu_backward import _inputs, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_device_errors(cuda_device):
    yield
    assert wkv4.device_error(reset=True) == 0


def _check(x, g, s_out, dt, mask, what, extra=0.0):
    """As for usual keys (tests/gradcheck.py), and for the exponents of masked
    steps: 3 passes of up to 64 steps in a chunk and its neighbour, each with 3
    fp64 roundings of an exponent |mask| log2(e) (2^-53 of it, times ln 2 in the
    value), the exponent held to 1.02e9 nats.  From 2^53 on an exponent swallows
    what is added to it in the kernel and in the oracle alike."""
    ref, mag = ob.wkv_backward_any_range(x["k"], x["v"], x["w"], x["u"], x["gy"], x["state_in"], x["r"],
                                         None if s_out is None else s_out.cpu(), x["gstate_out"])
    B, T, C = x["k"].shape
    rounds = -(-T // (512 if dt == "f32" else 1024))
    K = gradcheck.k_backward(rounds) + 16 + rounds + 8 + B + 8 + extra
    if abs(mask) < 2.0 ** 53:
        K += 3 * 64 * 3 * min(abs(mask), 1.02e9) * 2.0 ** -53 / 2.0 ** -24
    for name, got in g._asdict().items():
        if got is not None:
            gradcheck.check(got.cpu(), ref[name], mag[name], dt if name in ("gk", "gv", "gr") else "f32", K,
                            f"{what} {name}")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("mask", [-1e9, -1e10, -1e30])
@pytest.mark.parametrize("T,masked", [(5, (0, 2)), (40, (0, 10)), (100, (0, 64)), (50, (0, 50)), (300, (0, 200)),
                                      (300, (64, 96)), (300, (290, 300)), (2300, (0, 1100)), (2300, (0, 2300)),
                                      (5000, (0, 4200))], ids=str)
def test_gradients_of_finite_masks(cuda_device, T, masked, mask, dt):
    x = _inputs(2, T, 66, dt, seed=T + masked[1], gated=T != 300, state=False)
    x["k"][:, masked[0]:masked[1]] = mask
    g, _ = _run(x, cuda_device)
    _check(x, g, None, dt, mask, f"{mask} in {masked} of {T} {dt}")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("least", [-1e5, -1e7])
def test_gradients_of_mixed_masks(cuda_device, least, dt):
    """Masks of different size behind one another, in every order, with nothing else before them."""
    x = _inputs(2, 200, 66, dt, seed=9, gated=True, state=False)
    sizes = torch.tensor([least, -1e7, -3e8, -1e9, -1e12, -1e30])
    g = torch.Generator().manual_seed(1)
    at = torch.randint(0, len(sizes), (2, 10, 66), generator=g).repeat_interleave(17, 1)
    x["k"][:, :170] = sizes[at].to(x["k"].dtype)
    out, _ = _run(x, cuda_device)
    # Keys up to 2^22 log2 units take the fixed-reference walk where a chunk holds nothing else, and the exact
    # one beside others.  In the first, k log2(e) is a product by the float nearest log2(e), off by 2^-24
    # relative with its rounding: 2 |k| 2^-24 in e^k (tests/gradcheck.py), in each of the three passes.
    walk = 3 * 2 * abs(least) if abs(least) * 1.4427 < 2.0 ** 22 else 0.0
    _check(x, out, None, dt, -1e9, f"mixed masks {dt}", extra=walk)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("low", [-1e9, -1e30])
@pytest.mark.parametrize("T", [1, 45, 2200])
def test_gradients_of_states_with_a_low_max(cuda_device, T, low, dt):
    """A state whose max is as low as its masked steps' keys, carried in and out
    with its gradient."""
    x = _inputs(2, T, 66, dt, seed=T, gated=True, state=True)
    low = float(torch.tensor(low).to(x["k"].dtype))
    x["k"][:] = low
    x["state_in"][2] = low
    # the state after the last step, whose max alone is read: no decay leaves it at another float
    s = x["state_in"].clone()
    d = {a: None if t is None else t.to(cuda_device) for a, t in x.items()}
    g = wkv4.backward(d["k"], d["v"], d["w"], d["u"], d["gy"], d["state_in"], r=d["r"],
                      state_out=s.to(cuda_device), gstate_out=d["gstate_out"])
    torch.cuda.synchronize()
    _check(x, g, s, dt, low, f"state at {low} over {T} steps {dt}")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T", [3, 70, 1500])
def test_gradients_of_a_state_that_stays_empty(cuda_device, T, dt):
    """Keys of -inf behind an empty state: the state passes through, its gradient
    with it, and zero gradients of the outputs stay zero."""
    x = _inputs(2, T, 40, dt, seed=T, gated=False, state=True)
    x["k"][:] = -float("inf")
    x["state_in"][:2] = 0
    x["state_in"][2] = -1e38
    x["gstate_out"].zero_()
    d = {a: None if t is None else t.to(cuda_device) for a, t in x.items()}
    s = torch.stack([torch.zeros(2, 40), torch.zeros(2, 40), torch.full((2, 40), -1e38)]).to(cuda_device)
    g = wkv4.backward(d["k"], d["v"], d["w"], d["u"], torch.zeros_like(d["gy"]), torch.stack([d["state_in"][0],
                      torch.ones_like(d["state_in"][1]), d["state_in"][2]]), state_out=s,
                      gstate_out=d["gstate_out"])
    torch.cuda.synchronize()
    for name in ("gk", "gv", "gw", "gu", "gstate_in"):
        assert not getattr(g, name).any(), name


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("mask", [-60000.0, -1e9, -1e30, -float("inf")])
def test_a_padded_row_leaves_the_others_as_they_are(cuda_device, mask, dt):
    """A row that is all padding (no gradient arrives for it): the other rows' gradients and gw, gu have the
    bits they have when that row holds usual keys, and a row padded on the left has the gradients of the row
    without its padding."""
    if dt == "f16" and mask in (-1e9, -1e30):
        pytest.skip("past the type's range")
    B, T, C, pad = 3, 400, 66, 170
    x = _inputs(B, T, C, dt, seed=5, gated=True, state=False)
    x["gy"][1] = 0
    want, _ = _run(x, cuda_device)
    y = dict(x)
    y["k"] = x["k"].clone()
    y["k"][1] = mask
    y["v"] = x["v"].clone()
    y["v"][1] = 1.0
    if mask > -float("inf"):
        got, _ = _run(y, cuda_device)
        for a, b in zip(got[:3], want[:3]):
            assert torch.equal(a[[0, 2]], b[[0, 2]]) and not a[1].any()
        assert torch.equal(got.gw, want.gw) and torch.equal(got.gu, want.gu)
    z = {a: None if t is None else t.clone() for a, t in x.items()}
    if mask > -float("inf"):
        z["k"][:, :pad] = mask
    else:  # (with nothing before it, a key of -inf has no output at all: behind one usual step)
        z["k"][:, 1:pad] = mask
    z["gy"][:, :pad] = 0
    got, _ = _run(z, cuda_device)
    first = pad if mask > -float("inf") else 0
    cut = {a: t[:, first:].contiguous() if t is not None and t.dim() == 3 else t for a, t in z.items()}
    ref, mag = (ob.wkv_backward_any_range(cut["k"], cut["v"], cut["w"], cut["u"], cut["gy"], None, cut["r"])
                if mask > -float("inf") else
                ob.wkv_backward(cut["k"], cut["v"], cut["w"], cut["u"], cut["gy"], None, cut["r"]))
    assert not got.gk[:, 1:pad].any() and not got.gv[:, 1:pad].any()
    K = gradcheck.k_backward() + 16 + 1 + 8 + B + 8
    for name in ("gk", "gv", "gr"):
        gradcheck.check(getattr(got, name)[:, first:].cpu(), ref[name], mag[name], dt, K, f"padded {name}")
    for name in ("gw", "gu"):
        gradcheck.check(getattr(got, name).cpu(), ref[name], mag[name], "f32", K, f"padded {name}")
