"""Child process of tests/test_gpu_train_failure.py, run with the bounds-checked
library (WKV4_LIB pointing at libwkv4_checked.so):

  python -m tests.train_failure_child clean     the backward passes, the beam
                                                selection and the state moves on
                                                valid shapes: right results and an
                                                empty device error word
  python -m tests.train_failure_child launch N  with WKV4_FAULT=launch:N: the call
                                                whose launch is the N-th fails with
                                                WKV4_ERR_CUDA, and everything after
                                                it is right
  python -m tests.train_failure_child exchange  with WKV4_FAULT=exchange and a short
                                                WKV4_WAIT_ROUNDS: the CTAs of a
                                                backward cluster wait for sums that
                                                nobody pushes, give up
                                                (WKV4_ERR_TIMEOUT in the error word)
                                                and return; a call without an
                                                exchange is right afterwards

Prints "ok" on success; any failure raises (non-zero exit).
"""

import sys

import numpy as np
import torch

from oracle import backward as ob
from oracle import beam as obeam
from rwkv_wkv_linear_b200 import wkv4
from tests import gradcheck

DEV = torch.device("cuda:0")
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def backward(B, T, C, dt, gated=True):
    g = torch.Generator().manual_seed(B + T + C)
    n = lambda *s: torch.randn(*s, generator=g)
    k, v, gy = ((n(B, T, C)).to(DT[dt]) for _ in range(3))
    r = n(B, T, C).to(DT[dt]) if gated else None
    w, u = -torch.exp(torch.rand(C, generator=g) * 4 - 3), n(C) * 0.5
    s = torch.stack([n(B, C), torch.rand(B, C, generator=g) + 0.5, n(B, C)])
    d = lambda t: None if t is None else t.to(DEV)
    out = wkv4.backward(d(k), d(v), d(w), d(u), d(gy), d(s), r=d(r))
    torch.cuda.synchronize()
    ref, mag = ob.wkv_backward(k, v, w, u, gy, s, r)
    for name, got in out._asdict().items():
        if got is not None:
            t = dt if name in ("gk", "gv", "gr") else "f32"
            gradcheck.check(got.cpu(), ref[name], mag[name], t, gradcheck.k_backward(4) + 40, f"{dt} {name}")


def shift(B, T, C, dt):
    g = torch.Generator().manual_seed(T)
    x, gk, gv = (torch.randn(B, T, C, generator=g).to(DT[dt]) for _ in range(3))
    mk, mv = torch.rand(C, generator=g), torch.rand(C, generator=g)
    out = wkv4.token_shift_backward(*(t.to(DEV) for t in (x, mk, mv, gk, gv)))
    torch.cuda.synchronize()
    ref, mag = ob.token_shift_backward(x, [mk, mv], [gk, gv])
    gradcheck.check(out.gx.cpu(), ref["gx"], mag["gx"], dt, 8, "gx")


def select(G, K, V, n, dt):
    g = torch.Generator().manual_seed(V)
    x = (torch.randn(G, K, V, generator=g) * 2).to(DT[dt])
    c = -torch.rand(G, K, generator=g)
    s, p, t = wkv4.beam_select(x.to(DEV), c.to(DEV), n)
    torch.cuda.synchronize()
    _, rp, rt = obeam.select(x.double().numpy(), c.numpy(), n)
    assert np.array_equal(p.cpu().numpy(), rp) and np.array_equal(t.cpu().numpy(), rt)


def reorder(P, S, C, G, K, dt):
    g = torch.Generator().manual_seed(S)
    pool = torch.randn(P, S, C, generator=g).to(DT[dt])
    ids = torch.randperm(S, generator=g)[:G * K].int().view(G, K)
    par = torch.randint(0, K, (G, K), generator=g).int()
    pd = pool.to(DEV)
    new = wkv4.state_reorder(pd, ids.to(DEV), par.to(DEV))
    torch.cuda.synchronize()
    rp, ri = obeam.reorder(pool.float().numpy(), ids.numpy(), par.numpy())
    assert np.array_equal(pd.float().cpu().numpy(), rp) and np.array_equal(new.cpu().numpy(), ri)


def clean():
    for dt in ("f32", "f16", "bf16"):
        for shape in ((1, 1, 8), (2, 77, 66), (3, 300, 27), (1, 2100, 72)):
            backward(*shape, dt, gated=shape[1] % 2 == 1)
        for shape in ((1, 1, 8), (2, 77, 66), (3, 301, 64), (9, 33, 24)):
            shift(*shape, dt)
        for shape in ((1, 1, 5, 3), (2, 3, 5003, 9), (1, 4, 50277, 8)):
            select(*shape, dt)
        for shape in ((3, 9, 64, 1, 4), (2, 40, 37, 4, 8)):
            reorder(*shape, dt)
    assert wkv4.device_error(reset=True) == 0


# launches a call makes: several rounds (summary, prefix, main, sums), the shift's two
# (CTAs of more rows than a cluster takes) or one, one each
CALLS = [(4, lambda: backward(1, 2100, 72, "bf16")), (2, lambda: shift(9, 77, 66, "f16")),
         (1, lambda: select(2, 3, 1000, 5, "f32")), (1, lambda: reorder(3, 9, 64, 1, 4, "f32")),
         (1, lambda: shift(2, 77, 66, "f16"))]


def launch(nth):
    count, failed = 0, 0
    for launches, call in CALLS:
        if count < nth <= count + launches:
            try:
                call()
            except wkv4.Wkv4Error as e:
                assert e.status == -4
                failed += 1
            else:
                raise AssertionError("the injected failure was not reported")
        else:
            call()
        count += launches
        if failed == 1 and nth <= count:
            count = 10 ** 9  # the failing call made fewer: none fails any more
    assert failed == 1
    for _, call in CALLS:
        call()
    assert wkv4.device_error(reset=True) == 0


def exchange():
    g = torch.Generator().manual_seed(1)
    k = torch.randn(1, 300, 64, generator=g).bfloat16().to(DEV)
    w = -torch.ones(64, device=DEV)
    wkv4.backward(k, k, w, w, k)
    assert wkv4.device_error(reset=True) == -5
    backward(2, 60, 64, "bf16")      # one CTA a cluster: nothing to wait for
    assert wkv4.device_error(reset=True) == 0


if __name__ == "__main__":
    mode = sys.argv[1]
    {"clean": clean, "launch": lambda: launch(int(sys.argv[2])), "exchange": exchange}[mode]()
    print("ok")
