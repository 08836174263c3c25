"""Every mbarrier that a kernel sets up is fenced by the threads that set it up.

`fence.mbarrier_init.release.cluster` orders the issuing thread's own
initialisations before what it does next, so a fence under another condition
than the initialisation (one thread for four threads' barriers) orders nothing
for the rest: a peer's copy or remote store could meet a barrier that is not
there yet.  No run shows that reliably; the sources do."""

import os
import re

import pytest

from rwkv_wkv_linear_b200 import _build


def _code(path):
    text = open(path).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


def _unfenced(text):
    """Positions of mbar_init calls without a fence_mbar_init() behind them in a
    block that the kernel enters by condition."""
    bad = []
    for call in re.finditer(r"\bmbar_init\(", text):
        if re.search(r"void\s+$", text[:call.start()]):
            continue  # the definition
        opens, depth = [], 0
        for i in range(call.start() - 1, -1, -1):  # the blocks around the call, innermost first
            if text[i] == "}":
                depth += 1
            elif text[i] == "{":
                if depth == 0:
                    opens.append(i)
                else:
                    depth -= 1
        ok = False
        for at in opens:
            head = text[:at].rstrip()
            if not re.search(r"\bif (constexpr )?\([^{};]*\)$", head):
                continue
            depth, end = 0, at
            for end in range(at, len(text)):
                depth += (text[end] == "{") - (text[end] == "}")
                if depth == 0:
                    break
            ok |= "fence_mbar_init()" in text[call.end():end]
        if not ok:
            bad.append(call.start())
    return bad


@pytest.mark.parametrize("path", [p for p in _build.deps() if p.endswith(".cuh")], ids=os.path.basename)
def test_barriers_are_fenced_by_the_threads_that_set_them_up(path):
    text = _code(path)
    for at in _unfenced(text):
        line = text[text.rfind("\n", 0, at) + 1:text.find("\n", at)].strip()
        raise AssertionError(f"{os.path.basename(path)}: no fence by the same threads behind `{line}`")


def test_the_check_itself():
    assert not _unfenced("f() { if (t == 0) { for (;;) mbar_init(b, 1); fence_mbar_init(); } }")
    assert _unfenced("f() { if (t < 4) mbar_init(b + t, 1); if (t == 0) fence_mbar_init(); }")
    assert _unfenced("f() { if (t < 4) { mbar_init(b + t, 1); } if (t == 0) { fence_mbar_init(); } }")
