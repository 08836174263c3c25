"""The differentiable functions (rwkv_wkv_linear_b200/autograd.py): a time mix
layer -- token shift, three projections, the gated recurrence, the output
projection -- over two carried segments, its gradients against the same layer
written in fp64 torch and differentiated by torch; unused outputs; expanded
gradients; the backward pass captured into a graph."""

import numpy as np
import pytest
import torch

from rwkv_wkv_linear_b200 import autograd as wag
from rwkv_wkv_linear_b200 import wkv4
from tests import gradcheck

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_device_errors(cuda_device):
    yield
    assert wkv4.device_error(reset=True) == 0


NAMES = ("x", "mk", "mv", "mr", "Wk", "Wv", "Wr", "Wo", "w", "u", "x_prev", "state")


def _layer_inputs(B, T, C, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    p = dict(x=n(B, T, C), mk=torch.rand(C, generator=g), mv=torch.rand(C, generator=g),
             mr=torch.rand(C, generator=g), w=-torch.exp(torch.rand(C, generator=g) * 3 - 2),
             u=n(C) * 0.5, x_prev=n(B, C),
             state=torch.stack([n(B, C), torch.rand(B, C, generator=g) + 0.5, n(B, C)]))
    for m in ("Wk", "Wv", "Wr", "Wo"):
        p[m] = n(C, C) / C ** 0.5
    return p, n(B, T, C)


def _ours(p, gout, cut):
    outs, x_prev, state = [], p["x_prev"], p["state"]
    for x in (p["x"][:, :cut].contiguous(), p["x"][:, cut:].contiguous()):
        xk, xv, xr, x_prev = wag.token_shift(x, p["mk"], p["mv"], p["mr"], x_prev)
        y, state = wag.wkv(xk @ p["Wk"], xv @ p["Wv"], p["w"], p["u"], xr @ p["Wr"], state)
        outs.append(y @ p["Wo"])
    e = torch.exp(state[2].detach())
    return (torch.cat(outs, 1) * gout).sum() + (state[0] * e).sum() + (state[1] * e).square().sum()


def _plain(p, gout):
    x = p["x"]
    prev = torch.cat([p["x_prev"][:, None], x[:, :-1]], 1)
    xk, xv, xr = (prev + p[m] * (x - prev) for m in ("mk", "mv", "mr"))
    k, v, r = xk @ p["Wk"], xv @ p["Wv"], xr @ p["Wr"]
    e0 = torch.exp(p["state"][2])
    A, D = p["state"][0] * e0, p["state"][1] * e0
    ys = []
    for t in range(x.shape[1]):
        own, ek = torch.exp(p["u"] + k[:, t]), torch.exp(k[:, t])
        ys.append((A + own * v[:, t]) / (D + own))
        A, D = torch.exp(p["w"]) * A + ek * v[:, t], torch.exp(p["w"]) * D + ek
    y = torch.stack(ys, 1) * torch.sigmoid(r)
    return ((y @ p["Wo"]) * gout).sum() + A.sum() + D.square().sum()


@pytest.mark.parametrize("shape", [(2, 40, 48, 17), (1, 9, 33, 1)], ids=lambda s: "B%dT%dC%dcut%d" % s)
def test_time_mix_layer_gradients(cuda_device, shape):
    B, T, C, cut = shape
    inp, gout = _layer_inputs(B, T, C, seed=C)
    ours = {n: inp[n].to(cuda_device).requires_grad_() for n in NAMES}
    loss = _ours(ours, gout.to(cuda_device), cut)
    got = torch.autograd.grad(loss, [ours[n] for n in NAMES])
    ref = {n: inp[n].double().requires_grad_() for n in NAMES}
    want = torch.autograd.grad(_plain(ref, gout.double()), [ref[n] for n in NAMES])
    torch.cuda.synchronize()
    for n, a, b in zip(NAMES, got, want):
        a, b = a.cpu().double().numpy(), b.numpy()
        # every path through the layer is a chain of products over C terms of order one and the recurrence's own
        # rounding (tests/gradcheck.py), 2^-24 each: 4 projections of C terms, forward and back, relative to the
        # largest gradient of the tensor
        K = gradcheck.k_backward() + 8 * C + 64
        assert np.max(np.abs(a - b)) <= K * 2.0 ** -24 * np.max(np.abs(b)) * 4, n


def test_unused_outputs_and_expanded_gradients(cuda_device):
    B, T, C = 2, 30, 40
    inp, _ = _layer_inputs(B, T, C, seed=1)
    p = {n: inp[n].to(cuda_device) for n in NAMES}
    k, v, r = (torch.randn(B, T, C, device=cuda_device, requires_grad=True) for _ in range(3))
    y, s = wag.wkv(k, v, p["w"], p["u"], r)
    gk, = torch.autograd.grad(y.sum(), k)                      # an expanded ones
    want = wkv4.backward(k.detach(), v.detach(), p["w"], p["u"], torch.ones_like(k), r=r.detach())
    assert torch.equal(gk, want.gk)
    y, s = wag.wkv(k, v, p["w"], p["u"])                       # the state alone
    gk, gv = torch.autograd.grad(s[0].sum(), (k, v))
    go = torch.zeros_like(s)
    go[0] = 1
    want = wkv4.backward(k.detach(), v.detach(), p["w"], p["u"], torch.zeros_like(k), state_out=s.detach(),
                         gstate_out=go)
    assert torch.equal(gk, want.gk) and torch.equal(gv, want.gv)
    x = p["x"].clone().requires_grad_()
    xk, xv, xr, xl = wag.token_shift(x, p["mk"], p["mv"])
    assert xr is None
    gx, = torch.autograd.grad(xv.square().sum(), x)            # xk and x_last unused
    z = torch.zeros_like(p["x"])
    want = wkv4.token_shift_backward(p["x"], p["mk"], p["mv"], z, 2 * xv.detach())
    assert torch.equal(gx, want.gx)
    xk, xv, xr, xl = wag.token_shift(x, p["mk"], p["mv"])
    gx, = torch.autograd.grad(xl.sum(), x)
    assert torch.all(gx[:, -1] == 1) and torch.all(gx[:, :-1] == 0)
    with pytest.raises(RuntimeError):                          # first order only
        y, _ = wag.wkv(k, v, p["w"], p["u"])
        gk, = torch.autograd.grad(y.sum(), k, create_graph=True)
        gk.sum().backward()


def test_training_step_captured_into_a_graph(cuda_device):
    """Forward and gradients captured on a side stream, after eager steps whose
    graphs are gone, replayed on new inputs."""
    B, T, C = 2, 50, 64
    inp, gout = _layer_inputs(B, T, C, seed=4)
    leaves = {n: inp[n].to(cuda_device).requires_grad_() for n in NAMES}
    gout = gout.to(cuda_device)
    names = NAMES
    torch.autograd.grad(_ours(leaves, gout, 20), [leaves[n] for n in names])
    side = torch.cuda.Stream(cuda_device)
    side.wait_stream(torch.cuda.current_stream(cuda_device))
    with torch.cuda.stream(side):
        for _ in range(2):
            torch.autograd.grad(_ours(leaves, gout, 20), [leaves[n] for n in names])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = torch.autograd.grad(_ours(leaves, gout, 20), [leaves[n] for n in names])
    with torch.no_grad():
        leaves["x"].copy_(_layer_inputs(B, T, C, seed=5)[0]["x"])
    graph.replay()
    torch.cuda.synchronize()
    want = torch.autograd.grad(_ours(leaves, gout, 20), [leaves[n] for n in names])
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
