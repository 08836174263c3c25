"""Failure detection of the backward and beam search kernels without a GPU
fault, through the bounds-checked build (libwkv4_checked.so), each case in a
child process of its own (tests/train_failure_child.py): nothing recorded on
valid shapes; a launch that the runtime rejects is returned as WKV4_ERR_CUDA
by its call alone; a bounded wait for a cluster peer that runs out is recorded
as WKV4_ERR_TIMEOUT and the kernel returns."""

import os
import subprocess
import sys

import pytest

from rwkv_wkv_linear_b200 import _build

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _child(*args, **env):
    if not os.path.exists(_build.CHECKED_LIB):
        pytest.fail(f"{_build.CHECKED_LIB} is missing: run __graft_entry__.build()")
    e = dict(os.environ)
    e.pop("WKV4_FAULT", None)
    e.pop("WKV4_WAIT_ROUNDS", None)
    e["WKV4_LIB"] = _build.CHECKED_LIB
    e.update(env)
    r = subprocess.run([sys.executable, "-m", "tests.train_failure_child", *args], cwd=ROOT, env=e,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout[-3000:] + r.stderr[-3000:]


def test_checked_build_records_nothing_on_valid_shapes(cuda_device):
    _child("clean")


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 6, 7, 8, 9])
def test_injected_launch_failure(cuda_device, n):
    _child("launch", str(n), WKV4_FAULT=f"launch:{n}")


def test_exchange_wait_runs_out(cuda_device):
    _child("exchange", WKV4_FAULT="exchange", WKV4_WAIT_ROUNDS="20")
