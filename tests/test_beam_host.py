"""Argument checks of the beam search entry points: they return before any CUDA
call."""

import pytest
import torch

from rwkv_wkv_linear_b200 import wkv4

P = 0x7F0000000000  # fake device addresses


def _select(G=2, K=4, V=100, ld=100, n=4, logits=P + 0x10000, scores=P, finished=None, end_id=0,
            out=P + 0x1000, parents=P + 0x2000, tokens=P + 0x3000, dtype=wkv4.F32):
    return wkv4.load().wkv4_beam_select(G, K, V, ld, n, logits, scores, finished, end_id, out, parents,
                                        tokens, None, dtype)


def test_beam_select_argument_checks():
    assert _select(G=-1) == -1 and _select(K=-1) == -1 and _select(V=-1) == -1
    assert _select(dtype=3) == -2
    assert _select(G=0) == 0
    assert _select(K=0) == -1 and _select(V=0) == -1 and _select(K=33) == -1
    assert _select(n=0) == -1 and _select(n=65) == -1 and _select(n=-3) == -1
    assert _select(K=1, V=3, ld=3, n=4) == -1           # more than there are candidates
    assert _select(ld=99) == -1
    assert _select(K=4, V=1 << 30, ld=1 << 30) == -1    # K V past 31 bits
    assert _select(finished=P + 0x4000, end_id=100) == -1 and _select(finished=P + 0x4000, end_id=-1) == -1
    for name in ("logits", "scores", "out", "parents", "tokens"):
        assert _select(**{name: None}) == -1, name
    assert _select(logits=P + 0x10002) == -1            # off the type's own alignment
    assert _select(out=P + 0x10000 + 128) == -3 and _select(parents=P + 0x1004) == -3
    assert _select(tokens=P + 4) == -3 and _select(finished=P + 0x1000) == -3


def _reorder(P_=3, S=8, C=16, G=1, K=4, pool=P + 0x10000, ids=P, parents=P + 0x100, new=P + 0x200,
             dtype=wkv4.F32):
    return wkv4.load().wkv4_state_reorder(P_, S, C, G, K, pool, ids, parents, new, None, dtype)


def test_state_reorder_argument_checks():
    for bad in (dict(P_=-1), dict(S=-1), dict(C=-1), dict(G=-1), dict(K=-1), dict(K=33), dict(G=65536),
                dict(P_=65536)):
        assert _reorder(**bad) == -1, bad
    assert _reorder(dtype=9) == -2
    assert _reorder(G=0) == 0 and _reorder(K=0) == 0
    for name in ("pool", "ids", "parents", "new"):
        assert _reorder(**{name: None}) == -1, name
    assert _reorder(pool=P + 0x10002) == -1
    assert _reorder(new=P + 8) == -3 and _reorder(new=P + 0x100) == -3 and _reorder(ids=P + 0x10000) == -3


def test_binding_refuses_wrong_shapes():
    x = torch.zeros(2, 3, 5)
    with pytest.raises(ValueError):
        wkv4.beam_select(x[0], torch.zeros(2, 3))
    with pytest.raises(ValueError):
        wkv4.beam_select(x, torch.zeros(2, 3))              # host tensors
    with pytest.raises(ValueError):
        wkv4.state_reorder(x, torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        wkv4.state_reorder(x.int(), torch.zeros(1, 3, dtype=torch.int32), torch.zeros(1, 3, dtype=torch.int32))
