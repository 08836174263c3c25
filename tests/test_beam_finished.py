"""A finished beam's logits are not read (include/wkv4.h): the selection tests
the flag before it touches the row.  A run cannot show that without memory that
may not be read; the source does."""

import os
import re

from rwkv_wkv_linear_b200 import _build


def _unit():
    text = open(os.path.join(_build.CSRC, "wkv4_beam.cuh")).read()
    text = re.sub(r"//[^\n]*", "", text)
    at = re.search(r"void beam_unit\(", text).start()
    start = text.index("{", at)
    depth = 0
    for end in range(start, len(text)):
        depth += (text[end] == "{") - (text[end] == "}")
        if depth == 0:
            return text[start:end]


def test_the_flag_of_a_finished_beam_comes_before_its_logits():
    body = _unit()
    flag = re.search(r"if \(finished && \*finished\) return;", body)
    assert flag, "the unit does not leave for a finished beam by its flag alone"
    # what touches the row: the loads of whole pieces, and elements of p
    first = min(m.start() for m in re.finditer(r"beam_load\(|\bp\[", body))
    assert flag.start() < first


def test_no_row_is_touched_outside_a_unit():
    """The kernel hands rows to beam_unit and reads none itself."""
    text = open(os.path.join(_build.CSRC, "wkv4_beam.cuh")).read()
    text = re.sub(r"//[^\n]*", "", text)
    kernel = text[text.index("wkv4_beam_select_kernel("):text.index("struct ReorderParams")]
    assert kernel.count("p.logits") == 1 and "beam_unit<IO>(s, static_cast<const IO*>(p.logits)" in kernel
