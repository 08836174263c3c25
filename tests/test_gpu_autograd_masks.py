"""The time mix's operators under torch's autograd on left-padded batches: keys
masked with a finite value before the sequence, over two carried segments."""

import pytest
import torch

from rwkv_wkv_linear_b200 import autograd as wag
from rwkv_wkv_linear_b200 import wkv4

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_device_errors(cuda_device):
    yield
    assert wkv4.device_error(reset=True) == 0


@pytest.mark.parametrize("mask", [-65504.0, -1e9, -1e10, -1e30])
def test_a_masked_segment_trains_like_none(cuda_device, mask):
    """The first segment is all mask and no loss reads it: the second's gradients have the bits they have alone,
    the first's k, v, r get none."""
    B, T, C = 2, 180, 96
    g = torch.Generator().manual_seed(2)
    leaf = lambda *s: torch.randn(*s, generator=g).to(cuda_device).requires_grad_()
    k2, v2, r2, v1, r1, u = leaf(B, T, C), leaf(B, T, C), leaf(B, T, C), leaf(B, T, C), leaf(B, T, C), leaf(C)
    w = (-torch.exp(torch.rand(C, generator=g) * 4 - 3)).to(cuda_device).requires_grad_()
    k1 = torch.full((B, T, C), mask, device=cuda_device, requires_grad=True)
    gy = torch.randn(B, T, C, generator=g).to(cuda_device)
    y, s = wag.wkv(k2, v2, w, u, r2)
    want = torch.autograd.grad((y * gy).sum() + s[:2].sum(), (k2, v2, r2, w, u))
    y1, s1 = wag.wkv(k1, v1, w, u, r1)
    y2, s2 = wag.wkv(k2, v2, w, u, r2, s1)
    got = torch.autograd.grad((y2 * gy).sum() + s2[:2].sum(), (k2, v2, r2, w, u, k1, v1, r1), allow_unused=True)
    torch.cuda.synchronize()
    assert torch.isfinite(y1).all() and torch.equal(y2, y) and torch.equal(s2, s)
    for a, b in zip(got[:5], want):
        assert torch.equal(a, b)
    for a in got[5:]:
        assert a is None or not a.any()


@pytest.mark.parametrize("mask", [-65504.0, -1e9, -1e10, -1e30])
@pytest.mark.parametrize("pad", [7, 64, 150])
def test_left_padding_trains_like_the_cut_row(cuda_device, pad, mask):
    """Padding inside one call, no loss on it: the gradients of the row without it, to a few roundings (the chunks
    lie otherwise), gk and gv of the padding zero."""
    T, C = 300, 64
    g = torch.Generator().manual_seed(pad)
    n = lambda *s: torch.randn(*s, generator=g).to(cuda_device)
    k, v, r, gy = (n(1, T, C) for _ in range(4))
    k[:, :pad] = mask
    gy[:, :pad] = 0
    w, u = -torch.exp(torch.rand(C, generator=g) * 4 - 3).to(cuda_device), n(C)
    def grads(lo):
        x = [t[:, lo:].contiguous().requires_grad_() for t in (k, v, r)]
        p = [t.clone().requires_grad_() for t in (w, u)]
        y, _ = wag.wkv(x[0], x[1], p[0], p[1], x[2])
        return torch.autograd.grad((y * gy[:, lo:]).sum(), x + p)
    got, want = grads(0), grads(pad)
    torch.cuda.synchronize()
    assert not got[0][:, :pad].any() and not got[1][:, :pad].any()
    for i, (a, b) in enumerate(zip(got, want)):
        a = a[:, pad:] if i < 3 else a
        # fp32 sums of 150 to 293 steps in two orders, 3 passes of up to 64 + 20 joins of 3 roundings (tests/
        # gradcheck.py's K of some 450), of terms up to a tenth of the largest gradient's size times their number
        assert (a - b).abs().max() <= 2 * 450 * 2.0 ** -24 * 30 * b.abs().max()
