"""The exchange of sums between the CTAs of a backward cluster."""

import pytest
import torch

from rwkv_wkv_linear_b200 import wkv4

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_device_errors(cuda_device):
    yield
    assert wkv4.device_error(reset=True) == 0


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T", [1024, 2300])
def test_equal_rows_of_many_clusters_get_the_same_bits(cuda_device, T, dt):
    """Hundreds of clusters, each joining the same sums: one that met a barrier
    or a sum too early or too late would differ."""
    B, C = 96, 192
    g = torch.Generator().manual_seed(T)
    row = [torch.randn(1, T, C, generator=g).to(dt).to(cuda_device) for _ in range(4)]
    k, v, gy, r = (t.expand(B, T, C).contiguous() for t in row)
    w, u = -torch.exp(torch.rand(C, generator=g) * 4 - 5).to(cuda_device), torch.rand(C, generator=g).to(cuda_device)
    for _ in range(3):
        out = wkv4.backward(k, v, w, u, gy, r=r)
        for got in (out.gk, out.gv, out.gr):
            assert torch.equal(got, got[:1].expand_as(got))
