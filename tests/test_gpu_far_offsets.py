"""Tensors of more than 2^32 elements: rows at the far end are the ones that are
read and written (backward pass, token shift's, beam selection, state moves)."""

import numpy as np
import pytest
import torch

from oracle import beam as obeam
from rwkv_wkv_linear_b200 import wkv4

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean(cuda_device):
    wkv4.device_error(reset=True)
    if torch.cuda.get_device_properties(cuda_device).total_memory < 100 << 30:
        pytest.skip("needs 100 GB")
    yield
    assert wkv4.device_error(reset=True) == 0
    torch.cuda.empty_cache()


def test_gradients_of_far_batch_rows(cuda_device):
    B, T, C = 2100, 1024, 2048   # 4.4e9 elements a tensor
    g = torch.Generator().manual_seed(3)
    rows = [torch.randn(1, T, C, generator=g).bfloat16().to(cuda_device) for _ in range(3)]
    big = [torch.zeros(B, T, C, dtype=torch.bfloat16, device=cuda_device) for _ in range(3)]
    for t, row in zip(big, rows):
        t[B - 1:] = row
    w = -torch.exp(torch.rand(C, generator=g) * 4 - 3).to(cuda_device)
    u = torch.rand(C, generator=g).to(cuda_device)
    out = wkv4.backward(big[0], big[1], w, u, big[2])
    want = wkv4.backward(rows[0], rows[1], w, u, rows[2])
    torch.cuda.synchronize()
    assert torch.equal(out.gk[B - 1], want.gk[0]) and torch.equal(out.gv[B - 1], want.gv[0])
    # the other rows have no gradient: gout is zero there
    assert torch.equal(out.gw, want.gw) or torch.allclose(out.gw, want.gw, rtol=2.0 ** -18, atol=0)
    assert not torch.any(out.gk[::300]) and not torch.any(out.gv[B // 2])
    del out
    m = torch.rand(C, generator=g).to(cuda_device)
    sb = wkv4.token_shift_backward(big[0], m, m, big[1], big[2])
    sw = wkv4.token_shift_backward(rows[0], m, m, rows[1], rows[2])
    torch.cuda.synchronize()
    assert torch.equal(sb.gx[B - 1], sw.gx[0])


def test_selection_over_far_rows(cuda_device):
    G, K, V, ld = 3, 2, 1000, (1 << 30) + 8
    buf = torch.empty(G * K * ld, dtype=torch.bfloat16, device=cuda_device)
    g = torch.Generator().manual_seed(4)
    x = (torch.randn(G, K, V, generator=g) * 2).bfloat16()
    view = buf.view(G, K, ld)[..., :V]
    view.copy_(x)
    c = -torch.rand(G, K, generator=g)
    s, p, t = wkv4.beam_select(view, c.to(cuda_device), 7)
    torch.cuda.synchronize()
    _, rp, rt = obeam.select(x.double().numpy(), c.numpy(), 7)
    assert np.array_equal(p.cpu().numpy(), rp) and np.array_equal(t.cpu().numpy(), rt)


def test_state_moves_in_a_far_pool(cuda_device):
    P, S, C, K = 2, 70000, 32768, 4   # 4.6e9 elements
    pool = torch.empty(P, S, C, dtype=torch.bfloat16, device=cuda_device)
    ids = torch.tensor([[0, S - 1, S - 2, 40000]], dtype=torch.int32, device=cuda_device)
    rows = torch.randn(P, K, C, generator=torch.Generator().manual_seed(5)).bfloat16().to(cuda_device)
    pool[:, ids[0].long()] = rows
    par = torch.tensor([[1, 1, 3, 1]], dtype=torch.int32, device=cuda_device)
    new = wkv4.state_reorder(pool, ids, par)
    torch.cuda.synchronize()
    assert new.tolist() == [[S - 1, 0, 40000, S - 2]]
    assert torch.equal(pool[:, new[0].long()], rows[:, par[0].long()])
