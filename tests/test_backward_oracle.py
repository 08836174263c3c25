"""The gradients' fp64 oracle against central differences of the forward
oracle's own outputs, and the argument checks of the backward entry points
(which return before any CUDA call)."""

import numpy as np
import pytest
import torch

import oracle
from oracle import backward as ob
from rwkv_wkv_linear_b200 import wkv4


def _case(B, T, C, seed, state, gated):
    g = np.random.default_rng(seed)
    x = dict(k=g.normal(size=(B, T, C)) * 1.5, v=g.normal(size=(B, T, C)), w=-np.exp(g.uniform(-4, 1, C)),
             u=g.uniform(-1, 1, C), gy=g.normal(size=(B, T, C)),
             r=g.normal(size=(B, T, C)) if gated else None, state_in=None)
    if state:
        x["state_in"] = np.stack([g.normal(size=(B, C)), g.uniform(0.5, 2, (B, C)), g.uniform(-2, 2, (B, C))])
    gs = g.normal(size=(2, B, C))
    return x, gs


def _loss(x, gs):
    """sum gy out + sum of gs against the final state's sums in units of e^0."""
    f = oracle.forward_gated if x["r"] is not None else oracle.forward
    args = (x["k"], x["v"]) + ((x["r"],) if x["r"] is not None else ())
    y, s = f(*args, x["w"], x["u"], x["state_in"])
    e = np.exp(s[2])
    return (x["gy"] * y).sum() + (gs[0] * s[0] * e).sum() + (gs[1] * s[1] * e).sum(), s


@pytest.mark.parametrize("T,state,gated", [(1, True, True), (5, False, False), (9, True, True), (6, True, False)])
def test_oracle_gradients_match_differences(T, state, gated):
    x, gs = _case(2, T, 3, 10 + T, state, gated)
    _, s_out = _loss(x, gs)
    # the final state's gradient in the state's own units: dL/dnum = e^max dL/dA
    e = np.exp(s_out[2])
    gso = np.stack([gs[0] * e, gs[1] * e, np.zeros_like(e)])
    out, mag = ob.wkv_backward(x["k"], x["v"], x["w"], x["u"], x["gy"], x["state_in"], x["r"], s_out, gso)
    names = {"k": "gk", "v": "gv", "w": "gw", "u": "gu"}
    if gated:
        names["r"] = "gr"
    if state:
        names["state_in"] = "gstate_in"
    h = 1e-6
    for name, gname in names.items():
        flat = x[name].reshape(-1)
        num = np.empty_like(flat)
        for i in range(flat.size):
            keep = flat[i]
            flat[i] = keep + h
            up = _loss(x, gs)[0]
            flat[i] = keep - h
            num[i] = (up - _loss(x, gs)[0]) / (2 * h)
            flat[i] = keep
        # central difference: truncation h^2, rounding of the loss 2^-53 |L| / h
        err = np.abs(num.reshape(x[name].shape) - out[gname])
        assert np.all(err <= 1e-7 * (1 + np.abs(out[gname]))), (name, err.max())
        assert np.all(np.abs(out[gname]) <= mag[gname] * (1 + 1e-12)), name


def test_oracle_token_shift_gradients_match_differences():
    g = np.random.default_rng(3)
    B, T, C = 2, 4, 3
    x, xp = g.normal(size=(B, T, C)), g.normal(size=(B, C))
    mixes = [g.uniform(size=C) for _ in range(3)]
    grads = [g.normal(size=(B, T, C)) for _ in range(3)]
    gl = g.normal(size=(B, C))

    def loss():
        outs, last = oracle.token_shift(x, xp, mixes)
        return sum((a * b).sum() for a, b in zip(grads, outs)) + (gl * last).sum()

    out, _ = ob.token_shift_backward(x, mixes, grads, xp, gl)
    h = 1e-5
    for arr, ref in [(x, out["gx"]), (xp, out["gx_prev"])] + list(zip(mixes, out["gmix"])):
        flat, want = arr.reshape(-1), np.asarray(ref).reshape(-1)
        for i in range(flat.size):
            keep = flat[i]
            flat[i] = keep + h
            up = loss()
            flat[i] = keep - h
            num = (up - loss()) / (2 * h)
            flat[i] = keep
            assert abs(num - want[i]) <= 1e-8 * (1 + abs(want[i]))


P = 0x7F0000000000  # fake device addresses


def _bwd(B=2, T=8, C=16, w=P, u=P + 0x1000, k=P + 0x10000, v=P + 0x20000, r=None, si=None,
         gy=P + 0x30000, so=None, gso=None, gk=P + 0x40000, gv=P + 0x50000, gr=None, gw=P + 0x2000,
         gu=P + 0x3000, gsi=None, ws=P + 0x100000, nbytes=1 << 20, dtype=wkv4.F32):
    return wkv4.load().wkv4_backward(B, T, C, w, u, k, v, r, si, gy, so, gso, gk, gv, gr, gw, gu, gsi,
                                     ws, nbytes, None, dtype)


def test_backward_argument_checks():
    assert _bwd(B=-1) == -1 and _bwd(T=-1) == -1 and _bwd(C=-1) == -1
    assert _bwd(dtype=4) == -2
    assert _bwd(C=0) == 0
    assert _bwd(T=(1 << 24) + 1) == -1
    assert _bwd(B=65536, T=1, nbytes=1 << 45) == -1  # the grid's two short sides: rows and tiles of 64 channels
    assert _bwd(C=65535 * 64 + 1, T=1, nbytes=1 << 45) == -1
    for name in ("w", "u", "k", "v", "gy", "gk", "gv", "gw", "gu", "ws"):
        assert _bwd(**{name: None}) == -1, name
    assert _bwd(r=P + 0x60000) == -1                                  # r without gr
    assert _bwd(gso=P + 0x70000) == -1                                # gstate_out without state_out
    assert _bwd(gsi=P + 0x70000) == -1                                # gstate_in without state_in
    need = wkv4.load().wkv4_backward_workspace(2, 8, 16, wkv4.F32)
    assert need > 0
    assert _bwd(nbytes=need - 1) == -1
    assert _bwd(ws=P + 0x100004) == -1                                # misaligned workspace
    # gk over k (1024 bytes), gv over gk, gw over w, gstate_in over state_in, the workspace over gy
    assert _bwd(gk=P + 0x10000 + 512) == -3
    assert _bwd(gv=P + 0x40000 + 512) == -3
    assert _bwd(gw=P + 32) == -3
    assert _bwd(si=P + 0x70000, gsi=P + 0x70000) == -3
    assert _bwd(ws=P + 0x30000 + 16) == -3
    assert _bwd(r=P + 0x60000, gr=P + 0x60000) == -3


def test_backward_workspace_sizes():
    f = wkv4.load().wkv4_backward_workspace
    assert f(0, 8, 16, 0) == 0 and f(2, 8, 0, 0) == 0 and f(2, -1, 16, 0) == 0 and f(2, 8, 16, 9) == 0
    assert f(1, 32, 768, 0) == 0              # one CTA a channel tile sums by itself
    assert f(4, 1024, 768, 2) >= 2 * 4 * 8 * 768 * 4
    assert f(1, 16384, 64, 0) > f(1, 1024, 64, 0)


def _sb(B=2, T=8, C=16, x=P + 0x10000, xp=None, mk=P, mv=P + 0x1000, mr=None, gxk=P + 0x20000,
        gxv=P + 0x30000, gxr=None, gl=None, gx=P + 0x40000, gp=None, gmk=P + 0x2000, gmv=P + 0x3000,
        gmr=None, ws=P + 0x100000, nbytes=1 << 20, dtype=wkv4.F32):
    return wkv4.load().wkv4_token_shift_backward(B, T, C, x, xp, mk, mv, mr, gxk, gxv, gxr, gl, gx, gp,
                                                 gmk, gmv, gmr, ws, nbytes, None, dtype)


def test_token_shift_backward_argument_checks():
    assert _sb(B=-1) == -1 and _sb(T=-1) == -1 and _sb(C=-1) == -1 and _sb(dtype=3) == -2
    assert _sb(C=0) == 0
    for name in ("x", "mk", "mv", "gxk", "gxv", "gx", "gmk", "gmv"):
        assert _sb(**{name: None}) == -1, name
    assert _sb(mr=P + 0x4000) == -1 and _sb(mr=P + 0x4000, gmr=P + 0x5000) == -1   # no gxr
    assert _sb(B=70000) == -1
    sizes = wkv4.load().wkv4_token_shift_backward_workspace
    assert sizes(2, 8, 16, 0) == 0             # few enough rows to be summed by one cluster
    need = sizes(20, 8, 16, 0)
    far = dict(B=20, x=P + 0x1000000, gxk=P + 0x2000000, gxv=P + 0x3000000, gx=P + 0x4000000, ws=P + 0x5000000)
    assert need > 0 and _sb(**far, nbytes=need - 1) == -1
    far["ws"] += 8
    assert _sb(**far) == -1
    assert _sb(gx=P + 0x20000) == -3 and _sb(gmv=P + 0x2000) == -3 and _sb(gmk=P + 16) == -3
    far["ws"] = P + 0x4000000 + 64             # the workspace over gx
    assert _sb(**far) == -3


def test_binding_refuses_host_and_mismatched_tensors():
    k = torch.zeros(1, 4, 8)
    with pytest.raises(ValueError):
        wkv4.backward(k, k, torch.zeros(8), torch.zeros(8), k)
    with pytest.raises(ValueError):
        wkv4.backward(k, k, torch.zeros(8), torch.zeros(8), torch.zeros(1, 3, 8))
    with pytest.raises(ValueError):
        wkv4.token_shift_backward(k, torch.zeros(8), torch.zeros(8), k, k, mix_r=torch.zeros(8))


def test_kernel_hash_leaves_out_the_units_the_bench_does_not_launch(tmp_path):
    """The recorded traffic of the bench's workloads is keyed by the sources of
    their kernels: the backward and beam search units are not among them, and
    the forward's kernels include none of their files."""
    import os
    import shutil

    import bench
    csrc = os.path.join(bench.ROOT, "rwkv_wkv_linear_b200", "csrc")
    copy = tmp_path / "csrc"
    shutil.copytree(csrc, copy)
    base = bench.kernel_source_hash(str(copy))
    for name in bench._NOT_KERNEL_SOURCES:
        f = copy / name
        f.write_text(f.read_text() + "\nstatic const int one_more_constant = 3;\n")
    assert bench.kernel_source_hash(str(copy)) == base
    for name in os.listdir(csrc):
        if name not in bench._NOT_KERNEL_SOURCES:
            text = (copy / name).read_text()
            assert not any(f'#include "{other}"' in text for other in bench._NOT_KERNEL_SOURCES), name


@pytest.mark.parametrize("state,gated", [(False, True), (True, False)])
def test_oracle_of_any_range_is_the_oracle_for_usual_keys(state, gated):
    x, gs = _case(2, 30, 3, 5, state, gated)
    _, s_out = _loss(x, gs)
    gso = np.stack([gs[0], gs[1], np.zeros_like(gs[0])])
    args = (x["k"], x["v"], x["w"], x["u"], x["gy"], x["state_in"], x["r"], s_out, gso)
    for a, b in zip(ob.wkv_backward(*args), ob.wkv_backward_any_range(*args)):
        for name in a:
            assert np.max(np.abs(a[name] - b[name])) <= 1e-12 * np.max(np.abs(a[name])), name
    # a shift of all keys and of the state's max changes no gradient of a call that ends in no state
    y = dict(x, k=x["k"] - 1e4)
    if state:
        y["state_in"] = x["state_in"] - np.array([0, 0, 1e4])[:, None, None]
    a, _ = ob.wkv_backward(x["k"], x["v"], x["w"], x["u"], x["gy"], x["state_in"], x["r"])
    b, _ = ob.wkv_backward_any_range(y["k"], y["v"], y["w"], y["u"], y["gy"], y["state_in"], y["r"])
    for name in a:
        assert np.max(np.abs(a[name] - b[name])) <= 1e-10 * np.max(np.abs(a[name])), name
