"""GPU gradients of the WKV recurrence and of the token shift against their
fp64 oracle, element by element: the three types, gated and not, one step to
several rounds, widths that fill no tile, carried states with their gradients,
keys, decays and states that leave the fixed-reference path; chained calls,
streams, captured graphs, repeated runs."""

import numpy as np
import pytest
import torch

from oracle import backward as ob
from rwkv_wkv_linear_b200 import wkv4
from tests import gradcheck

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def no_device_errors(cuda_device):
    yield
    assert wkv4.device_error(reset=True) == 0


def _inputs(B, T, C, dt, seed, gated, state, kstd=1.4, td=(-6.0, 1.0)):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    un = lambda lo, hi, *s: torch.rand(*s, generator=g) * (hi - lo) + lo
    x = dict(k=(n(B, T, C) * kstd).to(DT[dt]), v=n(B, T, C).to(DT[dt]), w=-torch.exp(un(*td, C)),
             u=un(-1.0, 1.0, C), gy=n(B, T, C).to(DT[dt]), r=n(B, T, C).to(DT[dt]) if gated else None,
             state_in=None, gstate_out=None)
    if state:
        x["state_in"] = torch.stack([n(B, C), un(0.5, 2.0, B, C), un(-2.0, 2.0, B, C)])
        x["gstate_out"] = n(3, B, C)
    return x


def _run(x, dev, stream=None, **kw):
    """The forward's state on the device, then the gradients."""
    d = {a: None if t is None else t.to(dev) for a, t in x.items()}
    torch.cuda.synchronize()
    s_out = None
    if d["gstate_out"] is not None:
        if d["r"] is not None:
            _, s_out = wkv4.forward_gated(d["k"], d["v"], d["r"], d["w"], d["u"], d["state_in"])
        else:
            _, s_out = wkv4.forward(d["k"], d["v"], d["w"], d["u"], d["state_in"])
        torch.cuda.synchronize()
    g = wkv4.backward(d["k"], d["v"], d["w"], d["u"], d["gy"], d["state_in"], r=d["r"], state_out=s_out,
                      gstate_out=d["gstate_out"], stream=stream, **kw)
    torch.cuda.synchronize()
    return g, s_out


def _check(x, g, s_out, dt, what):
    ref, mag = ob.wkv_backward(x["k"], x["v"], x["w"], x["u"], x["gy"], x["state_in"], x["r"],
                               None if s_out is None else s_out.cpu(), x["gstate_out"])
    B, T, C = x["k"].shape
    rounds = -(-T // (512 if dt == "f32" else 1024))
    K = gradcheck.k_backward(rounds)
    got = g._asdict()
    assert (got["gr"] is None) == (x["r"] is None) and (got["gstate_in"] is None) == (x["state_in"] is None)
    for name in ref:
        t = dt if name in ("gk", "gv", "gr") else "f32"
        extra = 0 if t == dt and name != "gw" else 16 + rounds + 8 + B + 8
        gradcheck.check(got[name].cpu(), ref[name], mag[name], t, K + extra, f"{what} {name}")


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("shape", [(1, 1, 8), (2, 3, 7), (1, 16, 64), (2, 17, 66), (3, 65, 130), (1, 130, 72),
                                   (2, 300, 72), (2, 500, 33), (1, 700, 130), (1, 1024, 64), (2, 1025, 40), (1, 2500, 24),
                                   (1, 5200, 9)],
                         ids=lambda s: "B%dT%dC%d" % s)
def test_gradients_match_oracle(cuda_device, shape, gated, dt):
    B, T, C = shape
    x = _inputs(B, T, C, dt, seed=B + T + C, gated=gated, state=(T + C) % 2 == 1)
    g, s = _run(x, cuda_device)
    _check(x, g, s, dt, f"{shape} {dt}")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["spikes", "wide", "growing", "large_u", "fast_decay", "no_decay", "high_state",
                                  "low_state", "late_drop", "zero_gradient", "empty_state"])
def test_gradients_outside_the_usual_range(cuda_device, kind, dt):
    """Inputs that leave the fixed-reference path in the whole chunk, in some
    channels of a warp, or only on the way back."""
    B, T, C = 2, 200, 70
    x = _inputs(B, T, C, dt, seed=7, gated=True, state=True)
    g = torch.Generator().manual_seed(8)
    if kind == "spikes":      # chunks wider than the fixed reference takes
        x["k"][torch.rand(B, T, C, generator=g) < 0.02] = 60.0
    elif kind == "wide":
        x["k"] = (torch.randn(B, T, C, generator=g) * 40).to(DT[dt])
    elif kind == "growing":   # w above zero: the past gains weight
        x["w"][::3] = 0.5
        x["w"][1::3] = 0.02
    elif kind == "large_u":
        x["u"][::2] = 50.0
        x["u"][1::2] = -50.0
    elif kind == "fast_decay":
        x["w"] = -torch.exp(torch.rand(C, generator=g) * 2 + 1.5)
    elif kind == "no_decay":
        x["w"].zero_()
    elif kind == "high_state":
        x["state_in"][2] += 60.0
    elif kind == "low_state":
        x["state_in"][2] -= 200.0
    elif kind == "late_drop":  # what follows a chunk weighs far more than its own keys
        x["k"][:, 100:] -= 90.0
        x["w"][::2] = -8.0
    elif kind == "zero_gradient":
        x["gy"][:, 20:150] = 0
        x["gy"][1] = 0
    elif kind == "empty_state":
        x["state_in"][:2] = 0
        x["state_in"][2] = -1e38
    out, s = _run(x, cuda_device)
    ref, mag = ob.wkv_backward(x["k"], x["v"], x["w"], x["u"], x["gy"], x["state_in"], x["r"], s.cpu(),
                               x["gstate_out"])
    # larger keys: the fp32 argument of e^k is off by 2^-24 |k log2(e)| more (a
    # state's max likewise), in each of the three passes
    far = max(float(x["k"].float().abs().max()), 60.0) * 3 * 1.4427
    for name, got in out._asdict().items():
        t = dt if name in ("gk", "gv", "gr") else "f32"
        gradcheck.check(got.cpu(), ref[name], mag[name], t, gradcheck.k_backward() + 34 + far, f"{kind} {name}",
                        terms=B * T)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,masked", [(5, (4, 5)), (40, (0, 3)), (40, (30, 40)), (200, (150, 200)), (300, (32, 64)),
                                      (2200, (2000, 2200))], ids=str)
def test_gradients_of_masked_steps(cuda_device, T, masked, dt):
    """Keys of -inf (padded steps): they weigh nothing and get no gradient, in
    part of a chunk, in whole chunks and in whole CTAs, at either end."""
    x = _inputs(2, T, 70, dt, seed=T + masked[0], gated=True, state=True)
    x["k"][:, masked[0]:masked[1]] = -float("inf")
    g, s = _run(x, cuda_device)
    with np.errstate(all="ignore"):
        _check(x, g, s, dt, f"masked {masked} of {T} {dt}")
    assert not g.gk[:, masked[0]:masked[1]].any()


@pytest.mark.parametrize("dt,off", [("f32", 1), ("bf16", 1), ("f16", 4)])
def test_gradients_of_misaligned_rows(cuda_device, dt, off):
    """Bases off the 16-byte grid: loads and stores element by element, the
    same bits as the vector path."""
    B, T, C = 2, 90, 72
    x = _inputs(B, T, C, dt, seed=3, gated=True, state=True)
    want, s = _run(x, cuda_device)

    def shifted(t):
        buf = torch.empty(t.numel() + off, dtype=t.dtype, device=cuda_device)
        return buf[off:].view(t.shape).copy_(t)

    y = dict(x)
    for name in ("k", "v", "gy", "r"):
        y[name] = shifted(x[name].to(cuda_device))
    got, _ = _run(y, cuda_device)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_gradients_of_chained_calls(cuda_device, dt):
    """A sequence cut in three, the state carried and its gradient carried
    back, against the oracle over the whole."""
    B, T, C = 2, 300, 48
    x = _inputs(B, T, C, dt, seed=21, gated=True, state=True)
    d = {a: None if t is None else t.to(cuda_device) for a, t in x.items()}
    cuts = [0, 70, 71, T]
    states, outs = [d["state_in"]], []
    part = lambda t, i: t[:, cuts[i]:cuts[i + 1]].contiguous()
    for i in range(3):
        _, s = wkv4.forward_gated(part(d["k"], i), part(d["v"], i), part(d["r"], i), d["w"], d["u"], states[-1])
        states.append(s)
    gs = d["gstate_out"]
    for i in reversed(range(3)):
        g = wkv4.backward(part(d["k"], i), part(d["v"], i), d["w"], d["u"], part(d["gy"], i), states[i],
                          r=part(d["r"], i), state_out=states[i + 1], gstate_out=gs)
        gs = g.gstate_in
        outs.insert(0, g)
    torch.cuda.synchronize()
    whole = wkv4.Grads(*(torch.cat([getattr(o, n) for o in outs], 1) for n in ("gk", "gv", "gr")),
                       sum(o.gw for o in outs), sum(o.gu for o in outs), gs)
    ref, mag = ob.wkv_backward(x["k"], x["v"], x["w"], x["u"], x["gy"], x["state_in"], x["r"],
                               states[-1].cpu(), x["gstate_out"])
    for name, got in whole._asdict().items():
        t = dt if name in ("gk", "gv", "gr") else "f32"
        # two more joins through fp32 states each way (7 roundings each) and three sums
        gradcheck.check(got.cpu(), ref[name], mag[name], t, gradcheck.k_backward() + 34 + 3 * 14 + 3,
                        f"chained {name}")


def test_zero_steps_and_empty_batches(cuda_device):
    B, C = 2, 40
    w = -torch.ones(C, device=cuda_device)
    s = torch.stack([torch.randn(B, C), torch.rand(B, C) + 0.5, torch.randn(B, C)]).to(cuda_device)
    gs = torch.randn(3, B, C, device=cuda_device)
    k = torch.empty(B, 0, C, device=cuda_device)
    g = wkv4.backward(k, k, w, w, k, s, state_out=s.clone(), gstate_out=gs)
    torch.cuda.synchronize()
    assert torch.all(g.gw == 0) and torch.all(g.gu == 0)
    # through the scaled form and back: two exponentials and two products
    tol = 2.0 ** -24 * 12
    assert torch.all((g.gstate_in[:2] - gs[:2]).abs() <= tol * gs[:2].abs())
    want = s[0] * gs[0] + s[1] * gs[1]
    assert torch.all((g.gstate_in[2] - want).abs() <= 16 * 2.0 ** -24 * ((s[0] * gs[0]).abs() + (s[1] * gs[1]).abs()))
    e = torch.empty(0, 5, C, device=cuda_device)
    g = wkv4.backward(e, e, w, w, e)
    torch.cuda.synchronize()
    assert torch.all(g.gw == 0) and torch.all(g.gu == 0)


def test_masked_positions_give_no_gradient_and_leave_the_rest(cuda_device):
    """gy = 0 past a row's length (a padded batch): positions past it get
    exactly zero, and the ones before it what the cut row gets."""
    B, T, C, n = 1, 150, 64, 83
    x = _inputs(B, T, C, "f32", seed=31, gated=False, state=False)
    x["gy"][:, n:] = 0
    g, _ = _run(x, cuda_device)
    assert torch.all(g.gk[:, n:] == 0) and torch.all(g.gv[:, n:] == 0)
    cut = {a: t[:, :n].contiguous() if t is not None and t.dim() == 3 else t for a, t in x.items()}
    _check(cut, wkv4.Grads(g.gk[:, :n], g.gv[:, :n], None, g.gw, g.gu, None), None, "f32", "cut row")


def test_repeated_runs_give_the_same_bits_on_any_stream(cuda_device):
    x = _inputs(4, 700, 192, "bf16", seed=41, gated=True, state=True)
    want, _ = _run(x, cuda_device)
    other = torch.cuda.Stream(cuda_device)
    for stream in (None, other, other.cuda_stream):
        got, _ = _run(x, cuda_device, stream=stream)
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_two_calls_at_once_and_a_replayed_graph(cuda_device):
    """Two streams at once (workspaces of their own), then both calls captured
    in one graph and replayed on new inputs."""
    xs = [_inputs(2, 1100, 128, "f16", seed=s, gated=s % 2 == 0, state=False) for s in (50, 51)]
    want = [_run(x, cuda_device)[0] for x in xs]
    ds = [{a: None if t is None else t.to(cuda_device) for a, t in x.items()} for x in xs]
    streams = [torch.cuda.Stream(cuda_device) for _ in xs]
    call = lambda d, s=None: wkv4.backward(d["k"], d["v"], d["w"], d["u"], d["gy"], r=d["r"], stream=s)
    torch.cuda.synchronize()
    for _ in range(3):
        got = [call(d, s) for d, s in zip(ds, streams)]
    torch.cuda.synchronize()
    for g, ref in zip(got, want):
        for a, b in zip(g, ref):
            assert (a is None and b is None) or torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [call(d) for d in ds]
    keep = [{a: None if t is None else t.clone() for a, t in d.items()} for d in ds]
    for d in ds:
        d["gy"].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.all(g.gk == 0) and torch.all(g.gw == 0) for g in got)
    for d, kd in zip(ds, keep):
        d["gy"].copy_(kd["gy"])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for g, ref in zip(got, want):
        for a, b in zip(g, ref):
            assert (a is None and b is None) or torch.equal(a, b)


def test_a_given_workspace_is_all_that_is_used(cuda_device):
    x = _inputs(2, 1500, 64, "f32", seed=61, gated=False, state=False)
    want, _ = _run(x, cuda_device)
    need = wkv4.backward_workspace_bytes(2, 1500, 64, torch.float32)
    ws = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device=cuda_device)
    got, _ = _run(x, cuda_device, workspace=ws[:need])
    assert torch.equal(got.gk, want.gk) and torch.equal(got.gw, want.gw)
    assert torch.all(ws[need:] == 0x5A)
    with pytest.raises(wkv4.Wkv4Error):
        _run(x, cuda_device, workspace=ws[:need - 1])


# ------------------------------------------------------------- token shift


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 8), (2, 7, 33), (3, 65, 130), (2, 300, 256), (1, 1000, 12),
                                   (37, 700, 16), (12, 500, 520)],
                         ids=lambda s: "B%dT%dC%d" % s)
@pytest.mark.parametrize("outs,carry", [(3, True), (2, False)])
def test_token_shift_gradients_match_oracle(cuda_device, shape, outs, carry, dt):
    B, T, C = shape
    g = torch.Generator().manual_seed(B + T + C)
    x = torch.randn(B, T, C, generator=g).to(DT[dt])
    grads = [torch.randn(B, T, C, generator=g).to(DT[dt]) for _ in range(outs)]
    mixes = [torch.rand(C, generator=g) for _ in range(outs)]
    mixes[0][:3] = torch.tensor([0.0, 1.0, 0.5])[:C]
    xp = torch.randn(B, C, generator=g).to(DT[dt]) if carry else None
    gl = torch.randn(B, C, generator=g).to(DT[dt]) if carry else None
    dv = lambda t: None if t is None else t.to(cuda_device)
    pad = [None] * (3 - outs)
    m, gr = [dv(t) for t in mixes] + pad, [dv(t) for t in grads] + pad
    out = wkv4.token_shift_backward(dv(x), m[0], m[1], gr[0], gr[1], m[2], gr[2], dv(xp), gx_last=dv(gl))
    torch.cuda.synchronize()
    ref, mag = ob.token_shift_backward(x, mixes, grads, xp, gl)
    # 1 - m, then a rounding for each of the outputs and rows, gx_last
    gradcheck.check(out.gx.cpu(), ref["gx"], mag["gx"], dt, 8, "gx")
    if carry:
        gradcheck.check(out.gx_prev.cpu(), ref["gx_prev"], mag["gx_prev"], dt, 8, "gx_prev")
    else:
        assert out.gx_prev is None
    # difference, product, then the additions: a run's steps, 4 runs a CTA, rows / 8 + 8
    blocks = max(1, 148 * 8 // max(1, -(-C // 32) * B))
    K = 4 + max(8, -(-T // blocks)) + 4 + B * blocks / 8 + 8
    for i, got in enumerate([out.gmix_k, out.gmix_v, out.gmix_r][:outs]):
        gradcheck.check(got.cpu(), ref["gmix"][i], mag["gmix"][i], "f32", K, f"gmix {i}")


@pytest.mark.parametrize("dt,off", [("bf16", 4), ("f16", 1), ("f32", 2)])
def test_token_shift_gradients_of_unaligned_rows(cuda_device, dt, off):
    """One tensor `off` elements past 16 bytes: fewer channels a thread, the same gradients."""
    B, T, C = 37, 700, 16
    g = torch.Generator().manual_seed(off)
    x, gk, gv = (torch.randn(B, T, C, generator=g).to(DT[dt]) for _ in range(3))
    mk, mv = torch.rand(C, generator=g), torch.rand(C, generator=g)
    buf = torch.empty(B * T * C + off, dtype=DT[dt], device=cuda_device)
    xd = buf[off:].view(B, T, C)
    xd.copy_(x)
    dv = lambda t: t.to(cuda_device)
    out = wkv4.token_shift_backward(xd, dv(mk), dv(mv), dv(gk), dv(gv))
    torch.cuda.synchronize()
    ref, mag = ob.token_shift_backward(x, [mk, mv], [gk, gv])
    gradcheck.check(out.gx.cpu(), ref["gx"], mag["gx"], dt, 8, "gx")
    blocks = max(1, 148 * 8 // B)
    K = 4 + max(8, -(-T // blocks)) + 4 + B * blocks / 8 + 8
    for i, got in enumerate([out.gmix_k, out.gmix_v]):
        gradcheck.check(got.cpu(), ref["gmix"][i], mag["gmix"][i], "f32", K, f"gmix {i}")


def test_token_shift_gradients_of_zero_steps(cuda_device):
    B, C = 2, 24
    x = torch.empty(B, 0, C, device=cuda_device)
    m = torch.rand(C, device=cuda_device)
    xp, gl = torch.randn(B, C, device=cuda_device), torch.randn(B, C, device=cuda_device)
    out = wkv4.token_shift_backward(x, m, m, x, x, x_prev=xp, gx_last=gl)
    torch.cuda.synchronize()
    assert torch.equal(out.gx_prev, gl) and torch.all(out.gmix_k == 0) and torch.all(out.gmix_v == 0)
    out = wkv4.token_shift_backward(x, m, m, x, x, x_prev=xp)
    torch.cuda.synchronize()
    assert torch.all(out.gx_prev == 0)
