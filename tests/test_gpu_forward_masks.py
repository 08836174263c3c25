"""The forward under finite masks of any size: whole chunks of keys like -1e10 or
-1e30 with nothing before them, in every kernel, and the state they leave."""

import pytest
import torch

from rwkv_wkv_linear_b200 import wkv4

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
KERNELS = {"auto": wkv4.KERNEL_AUTO, "seq": wkv4.KERNEL_SEQ, "scan": wkv4.KERNEL_SCAN,
           "scan_ldg": wkv4.KERNEL_SCAN_LDG, "step": wkv4.KERNEL_STEP}


@pytest.fixture(autouse=True)
def no_device_errors(cuda_device):
    yield
    assert wkv4.device_error(reset=True) == 0


def _inputs(B, T, C, dt, seed):
    g = torch.Generator().manual_seed(seed)
    k, v = (torch.randn(B, T, C, generator=g).to(DT[dt]) for _ in range(2))
    return k, v, -torch.exp(torch.rand(C, generator=g) * 4 - 3), torch.rand(C, generator=g) - 0.5


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("kernel", sorted(KERNELS))
@pytest.mark.parametrize("mask", [-1e9, -5e9, -1e10, -1e30])
@pytest.mark.parametrize("T,masked", [(100, 64), (300, 170), (70, 70), (2100, 1100)])
def test_masked_steps_weigh_nothing(cuda_device, T, masked, mask, kernel, dt):
    """y is finite under the mask, a weighted mean of v, and behind it what the
    sequence without its masked steps gives, with the same state."""
    B, C = 2, 72
    k, v, w, u = _inputs(B, T, C, dt, T)
    k[:, :masked] = mask
    d = lambda t: t.to(cuda_device)
    y, s = wkv4.forward(d(k), d(v), d(w), d(u), variant=KERNELS[kernel])
    torch.cuda.synchronize()
    head = y[:, :masked].float().cpu()
    # (half a step of the type past the largest |v| before it, and the quotient's few roundings)
    most = v.float().abs().cummax(1).values[:, :masked] * (1 + 2.0 ** -8)
    assert torch.isfinite(head).all() and (head.abs() <= most).all()
    assert torch.isfinite(s).all()
    if masked == T:
        return
    cut = [d(t[:, masked:].contiguous()) for t in (k, v)]
    want, sw = wkv4.forward(*cut, d(w), d(u), variant=wkv4.KERNEL_STEP)
    torch.cuda.synchronize()
    # both are right to a few roundings of fp32 in sums of positive weights (the state's planes num and den
    # held against maxima that may differ by rounding), then one to the type
    eps = 2.0 ** -24 * 256 + (2.0 ** -8 if dt == "bf16" else 0)
    vmax = v.float().abs().amax().item()
    assert (y[:, masked:].float() - want.float()).abs().max().item() <= eps * vmax
    a, b = ((t[:2].double() * torch.exp(t[2].double())).cpu() for t in (s, sw))
    assert ((a - b).abs() <= 2.0 ** -24 * 512 * b[1].abs().clamp(min=0) * max(vmax, 1.0)).all()


@pytest.mark.parametrize("mask", [-1e9, -1e10, -1e30])
def test_a_masked_segment_carries_a_usable_state(cuda_device, mask):
    """A segment of nothing but masks, with slow and fast decays, then a usual one on its state: the first leaves
    no trace."""
    B, T, C = 2, 1200, 64
    k, v, w, u = _inputs(B, T, C, "f32", 3)
    w[::2] *= 4.0
    d = lambda t: t.to(cuda_device)
    for kernel in KERNELS.values():
        _, s = wkv4.forward(d(torch.full_like(k, mask)), d(v), d(w), d(u), variant=kernel)
        assert torch.isfinite(s).all()
        y, s2 = wkv4.forward(d(k), d(v), d(w), d(u), s, variant=kernel)
        want, sw = wkv4.forward(d(k), d(v), d(w), d(u), variant=kernel)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(s2, sw)
