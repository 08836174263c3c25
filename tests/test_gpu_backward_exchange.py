"""The exchange of sums between the CTAs of a backward cluster."""

import os
import subprocess
import sys

import pytest
import torch

from rwkv_wkv_linear_b200 import _build, wkv4

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


@pytest.mark.parametrize("T,rank", [(300, 0), (300, 1), (300, 2), (1000, 3), (5000, 0), (5000, 5), (5000, 13)])
def test_a_silent_rank_leaves_nobody_behind(cuda_device, T, rank):
    """One CTA of each cluster pushes no sums (checked build): those that need
    them give up and are reported, the rest of the exchange goes on into CTAs
    that are still there, and the context stays usable."""
    if not os.path.exists(_build.CHECKED_LIB):
        pytest.fail(f"{_build.CHECKED_LIB} is missing: run __graft_entry__.build()")
    e = dict(os.environ, WKV4_LIB=_build.CHECKED_LIB, WKV4_FAULT="exchange", WKV4_FAULT_RANK=str(rank),
             WKV4_WAIT_ROUNDS="20")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-m", "tests.exchange_failure_child", str(T)], cwd=root, env=e,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout[-3000:] + r.stderr[-3000:]
