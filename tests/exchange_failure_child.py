"""Child process of tests/test_gpu_backward_exchange.py, run with the bounds-checked
library, WKV4_FAULT=exchange, WKV4_FAULT_RANK=R and a short WKV4_WAIT_ROUNDS: in
every backward cluster the CTAs of rank R push no sums.  The CTAs that need them
give up (WKV4_ERR_TIMEOUT in the error word) while the others' sums are still on
their way, and every call returns; a call without an exchange is right afterwards.

  python -m tests.exchange_failure_child T

Prints "ok" on success; any failure raises (non-zero exit)."""

import sys

import torch

from rwkv_wkv_linear_b200 import wkv4
from tests.train_failure_child import DEV, backward


def main(T):
    g = torch.Generator().manual_seed(1)
    x = [torch.randn(2, T, 130, generator=g).bfloat16().to(DEV) for _ in range(4)]
    w = -torch.ones(130, device=DEV)
    for r in (None, x[3]):
        wkv4.backward(x[0], x[1], w, w, x[2], r=r)
        assert wkv4.device_error(reset=True) == -5
    backward(2, 60, 64, "bf16")      # one CTA a cluster: nothing to wait for
    assert wkv4.device_error(reset=True) == 0


if __name__ == "__main__":
    main(int(sys.argv[1]))
    print("ok")
