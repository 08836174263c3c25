"""Outputs that a call on another stream has allocated and the caller drops at
once: their memory is not handed on before that stream has passed the call."""

import pytest
import torch

from rwkv_wkv_linear_b200 import wkv4

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_device_errors(cuda_device):
    wkv4.device_error(reset=True)
    yield
    assert wkv4.device_error(reset=True) == 0


B, T, C = 2, 64, 256


def _calls(dev):
    g = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=g).to(dev)
    k, v, r, gy = (n(B, T, C) for _ in range(4))
    w, u, m = -torch.rand(C, generator=g).to(dev), n(C), torch.rand(C, generator=g).to(dev)
    state, pool = n(3, B, C), n(3, 9, C)
    state[1].abs_()
    pool[1].abs_()
    ids = torch.tensor([[0, 3, 5, 7]], dtype=torch.int32, device=dev)
    par = torch.tensor([[1, 1, 2, 0]], dtype=torch.int32, device=dev)
    k1, v1, r1 = (t[:, 0].contiguous() for t in (k, v, r))
    logits, scores = n(2, 4, 1000), n(2, 4)
    return {
        "forward": lambda s: wkv4.forward(k, v, w, u, stream=s),
        "forward_gated": lambda s: wkv4.forward_gated(k, v, r, w, u, stream=s),
        "decode_step": lambda s: wkv4.decode_step(k1, v1, w, u, state, stream=s),
        "decode_step_gated": lambda s: wkv4.decode_step_gated(k1, v1, r1, w, u, state, stream=s),
        "decode_step_slots": lambda s: wkv4.decode_step_slots(k1, v1, w, u, pool, ids[0, :2], stream=s),
        "token_shift": lambda s: wkv4.token_shift(k, m, m, m, stream=s),
        "state_combine": lambda s: wkv4.state_combine(state, state, 3, w, stream=s),
        "backward": lambda s: wkv4.backward(k, v, w, u, gy, state, r=r, stream=s),
        "token_shift_backward": lambda s: wkv4.token_shift_backward(k, m, m, gy, gy, m, gy, k1, stream=s),
        "beam_select": lambda s: wkv4.beam_select(logits, scores, stream=s),
        "state_reorder": lambda s: wkv4.state_reorder(pool, ids, par, stream=s),
    }


@pytest.mark.parametrize("name", sorted(_calls(torch.device("cpu"))))
@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_dropped_outputs_keep_their_memory(cuda_device, name, raw):
    call = _calls(cuda_device)[name]
    side = torch.cuda.Stream(cuda_device)
    out = call(None)  # (what the call returns, for its sizes)
    sizes = [t.shape for t in (out if isinstance(out, tuple) else (out,)) if t is not None]
    dtypes = [t.dtype for t in (out if isinstance(out, tuple) else (out,)) if t is not None]
    del out
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream(cuda_device))
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)  # some 20 ms: the call's kernel runs long after what follows
    call(side.cuda_stream if raw else side)  # nothing of it is kept
    fresh = [torch.empty(s, dtype=t, device=cuda_device).fill_(7) for _ in range(3) for s, t in zip(sizes, dtypes)]
    torch.cuda.synchronize()
    for t in fresh:
        assert (t == 7).all()
