"""Selection among logits of large magnitude: finite masks of any size over most
of a row, so that whole threads see nothing else, and rows far from zero."""

import numpy as np
import pytest
import torch

from oracle import beam as obeam
from rwkv_wkv_linear_b200 import wkv4
from tests.test_gpu_beam import DT, _check, _scores

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clear_device_errors(cuda_device):
    wkv4.device_error(reset=True)
    yield
    assert wkv4.device_error(reset=True) == 0


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("mask", [-3000.0, -65504.0, -1e6, -1e8, -1e9, -5e9, -1e10, -1e18, -1e30])
@pytest.mark.parametrize("V", [3001, 50277])
def test_selection_under_finite_masks(cuda_device, V, mask, dt):
    """Most tokens at one finite mask; a usual one is left in every row."""
    G, K, n = 2, 4, 9
    g = torch.Generator().manual_seed(V)
    x = (torch.randn(G, K, V, generator=g) * 2.5).to(DT[dt])
    off = torch.rand(G, K, V, generator=g) < 0.999
    off[..., 17] = False
    off[0, 0, 20:40] = False
    x[off] = mask
    _check(cuda_device, x, _scores(G, K, g), n)


def test_selection_under_the_lowest_half(cuda_device):
    g = torch.Generator().manual_seed(2)
    x = (torch.randn(2, 4, 20001, generator=g) * 2.5).half()
    x[torch.rand(2, 4, 20001, generator=g) < 0.999] = -65504.0
    _check(cuda_device, x, _scores(2, 4, g), 9)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("offset", [3e3, -3e3, 1e5, -1e5, 1e6, -1e6, 2e7, -1e8, 1e8, -1e9, 1e12, -1e12, -1e30])
def test_selection_in_rows_far_from_zero(cuda_device, offset, dt):
    """A row moved as a whole has the same log-probabilities, those of the logits as the type holds them."""
    G, K, V, n = 2, 3, 9001, 12
    g = torch.Generator().manual_seed(7)
    x = (torch.randn(G, K, V, generator=g).double() * 2.5 + offset).to(DT[dt])
    _check(cuda_device, x, _scores(G, K, g), n)


@pytest.mark.parametrize("big", [2e3, 4e4, 6e6, 3e9])
def test_log_sums_of_rows_that_climb(cuda_device, big):
    """Logits that rise by steps along the vocabulary, so that a thread's reference moves from far below to far
    above zero while it sums: the best token's score is that of the last step alone."""
    V = 30000
    step = torch.linspace(-big, big, 6).repeat_interleave(V // 6)
    g = torch.Generator().manual_seed(3)
    x = (step + torch.randn(V, generator=g)).view(1, 1, V).float()
    c = torch.tensor([[-1.0]])
    s, p, t = wkv4.beam_select(x.to(cuda_device), c.to(cuda_device), 5)
    torch.cuda.synchronize()
    rs, rp, rt = obeam.select(x.double().numpy(), c.numpy(), 5)
    assert np.array_equal(t.cpu().numpy(), rt)
    assert np.all(np.abs(s.cpu().double().numpy() - rs) <= 2.0 ** -24 * (np.abs(rs) + 4 + 48 + V / 256 + 8))
