"""A NaN among the inputs of the backward pass shows in the gradients of its
channel, as the formula has it, and nowhere else."""

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


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("path", ["usual", "exact"])
@pytest.mark.parametrize("name", ["r", "k", "v", "gy"])
@pytest.mark.parametrize("T,t", [(40, 17), (700, 300), (2300, 5)])
def test_a_nan_stays_in_its_channel(cuda_device, T, t, name, path, dt):
    """Channel c: gr of the step itself (r, v, gy, k reach it all), gk and gv of that step and of those before
    it (their sums run over it), gw and gu; every other channel has the bits it has without the NaN."""
    B, C, b, c = 2, 66, 1, 11
    x = _inputs(B, T, C, dt, seed=T, gated=True, state=False)
    if path == "exact":  # chunks too wide for one reference
        x["k"][:, ::7] = 60.0
    want, _ = _run(x, cuda_device)
    y = dict(x)
    y[name] = x[name].clone()
    y[name][b, t, c] = float("nan")
    got, _ = _run(y, cuda_device)
    assert torch.isnan(got.gr[b, t, c])
    assert torch.isnan(got.gk[b, :t + 1, c]).all()
    if name == "v":  # (y is linear in v: gv holds none)
        ref, mag = ob.wkv_backward(x["k"], x["v"], x["w"], x["u"], x["gy"], None, x["r"])
        # (as tests/test_gpu_backward.py for keys of 60: the pair (P, Q) is scaled by its larger part, so P
        # may round differently beside a NaN)
        gradcheck.check(got.gv.cpu(), ref["gv"], mag["gv"], dt, gradcheck.k_backward(5) + 34 + 60 * 3 * 1.4427, "gv",
                        terms=B * T)
    else:
        assert torch.isnan(got.gv[b, :t + 1, c]).all()
    assert torch.isnan(got.gw[c]) and torch.isnan(got.gu[c])
    if name in ("r", "gy"):  # the steps' outputs do not depend on them
        assert torch.isfinite(got.gr[b, :t, c]).all() and torch.isfinite(got.gr[b, t + 1:, c]).all()
        assert torch.equal(got.gk[b, t + 1:, c], want.gk[b, t + 1:, c])
    else:
        assert torch.isnan(got.gr[b, t:, c]).all()
    rest = [i for i in range(C) if i != c]
    for g, w in zip(got[:3], want[:3]):
        assert torch.equal(g[..., rest], w[..., rest]) and torch.equal(g[0], w[0])
    assert torch.equal(got.gw[rest], want.gw[rest]) and torch.equal(got.gu[rest], want.gu[rest])
