"""GPU beam search: the selection against every candidate sorted in fp64, and
the state moves against rows moved one by one, with the cases where they can go
wrong (ruled-out tokens, rows with nothing left, NaN and infinities, equal
logits, dead and finished beams, fewer candidates than asked for, padded and
odd rows, bad parents), and a search that uses them with the slot decode."""

import numpy as np
import pytest
import torch

import oracle
from oracle import beam as obeam
from rwkv_wkv_linear_b200 import wkv4

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
INF = float("inf")


@pytest.fixture(autouse=True)
def clear_device_errors(cuda_device):
    wkv4.device_error(reset=True)
    yield
    assert wkv4.device_error(reset=True) == 0


def _scores(G, K, g):
    return -torch.sort(torch.rand(G, K, generator=g) * 8 + 4, dim=1).values


def _check(dev, logits, scores, n, finished=None, end_id=0, exact=True):
    ld = lambda t: None if t is None else t.to(dev)
    if logits.is_contiguous():
        x = ld(logits)
    else:  # rows of a padded buffer: the same strides on the device
        G, K, V = logits.shape
        x = torch.full((G, K, logits.stride(1)), 99.0, dtype=logits.dtype, device=dev)[..., :V]
        x.copy_(logits)
    s, p, t = wkv4.beam_select(x, ld(scores), n, finished=ld(finished), end_id=end_id)
    torch.cuda.synchronize()
    fin = None if finished is None else finished.numpy()
    rs, rp, rt = obeam.select(logits.double().numpy(), scores.numpy(), n, fin, end_id)
    assert np.array_equal(p.cpu().numpy(), rp) and np.array_equal(t.cpu().numpy(), rt)
    got = s.cpu().double().numpy()
    live = np.isfinite(rs)
    assert np.array_equal(np.isneginf(got), ~live)
    # rounding to fp32 (half a step), and the log-sum: its terms are off by an
    # ex2.approx (2 ulp), its rounded argument (|x| log2(e) 2^-24 at |x| <= 32)
    # and a running sum of V / 256 + 8 fp32 additions in the worst case
    V = logits.shape[2]
    bound = 2.0 ** -24 * np.abs(rs[live]) + 2.0 ** -24 * (4 + 48 + V / 256 + 8)
    assert np.all(np.abs(got[live] - rs[live]) <= bound)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1), (1, 1, 7, 7), (3, 2, 9, 4), (2, 32, 2, 64), (1, 4, 50277, 4),
                                   (2, 3, 12345, 6), (5, 8, 1000, 16), (1, 32, 4097, 64), (2, 1, 65536, 64),
                                   (300, 2, 300, 3)],
                         ids=lambda s: "G%dK%dV%dn%d" % s)
def test_selection_matches_sorted_candidates(cuda_device, shape, dt):
    G, K, V, n = shape
    g = torch.Generator().manual_seed(G + K + V)
    # distinct beams: equal scores of different beams have no chance but through equal logits and sums
    logits = (torch.randn(G, K, V, generator=g) * 2.5).to(DT[dt])
    _check(cuda_device, logits, _scores(G, K, g), n)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("pad", [1, 3, 8, 64])
def test_selection_over_padded_rows(cuda_device, pad, dt):
    G, K, V, n = 3, 4, 5003, 9
    g = torch.Generator().manual_seed(pad)
    buf = (torch.randn(G, K, V + pad, generator=g) * 2).to(DT[dt])
    buf[..., V:] = 50.0  # what lies behind a row is never a candidate
    _check(cuda_device, buf[..., :V], _scores(G, K, g), n)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind", ["masked", "few_left", "nothing_left", "lowest_value", "nan", "posinf", "dead",
                                  "dead_nan", "finished", "all_finished", "all_dead", "huge", "negative_zero"])
def test_selection_of_masked_and_broken_rows(cuda_device, kind, dt):
    G, K, V, n = 2, 4, 3001, 12
    g = torch.Generator().manual_seed(17)
    x = (torch.randn(G, K, V, generator=g) * 2.5).to(DT[dt])
    scores, finished = _scores(G, K, g), None
    if kind == "masked":
        x[torch.rand(G, K, V, generator=g) < 0.9] = -INF
    elif kind == "few_left":       # fewer candidates than asked for in one group
        keep = x[0, :, :2].clone()
        x[0] = -INF
        x[0, :, 1000:1002] = keep
    elif kind == "nothing_left":
        x[0] = -INF
        x[1, 1] = -INF
    elif kind == "lowest_value":   # a mask of the type's lowest value: those tokens are candidates, last ones
        low = torch.finfo(DT[dt]).min
        keep = x[0, 0, 5:8].clone()
        x[0] = low
        x[0, 0, 5:8] = keep
        scores[0, 1:] = -INF       # one live row, so equal scores go by the token alone
    elif kind == "nan":
        x[0, 2, 77] = float("nan")
        x[1, 0, :] = float("nan")
        x[1, 3] = -INF
        x[1, 3, 3000] = float("nan")
    elif kind == "posinf":
        x[0, 0, 100] = INF
        x[1, 2, 0] = INF
    elif kind == "dead":
        scores[:, 1:] = -INF
        scores[1, 0] = INF
    elif kind == "dead_nan":
        scores[0, 0] = float("nan")
        scores[1, 1] = -3e9
    elif kind == "finished":
        finished = torch.rand(G, K, generator=g) < 0.5
        finished[0, 0] = True
        x[0, 0] = float("nan")     # a finished beam's logits are not read
    elif kind == "all_finished":
        finished = torch.ones(G, K, dtype=torch.bool)
    elif kind == "all_dead":
        scores[:] = -INF
        finished = torch.ones(G, K, dtype=torch.bool)
    elif kind == "huge":           # one logit far above the rest
        x[0, 1, 9] = 60000.0
        x[1, :, 4] = -60000.0
    elif kind == "negative_zero":  # -0 and 0 are one value: the lower token first
        x[0] = -INF
        x[0, 1, 10:30] = 0.0
        x[0, 1, 10:30:2] = -0.0
    _check(cuda_device, x, scores, n, finished, end_id=5)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("V", [2048, 24000])
def test_selection_among_equal_logits(cuda_device, V, dt):
    """More equal logits than a list holds: the lowest tokens of the best row."""
    g = torch.Generator().manual_seed(5)
    x = torch.zeros(2, 3, V).to(DT[dt])
    x[1, 1, V // 2:] = 1.0
    x[1, 1, 7] = 2.0
    x[1, 1, V - 1] = 3.0
    scores = torch.tensor([[-1.0, -2.0, -3.0], [-50.0, -0.5, -60.0]])
    _check(cuda_device, x, scores, 40)


def test_selection_keeps_the_order_of_identical_beams(cuda_device):
    """Rows with the same bits and scores: equal sums, so the lower beam first
    (rows of 16-byte multiples, which are summed in one order)."""
    g = torch.Generator().manual_seed(6)
    x = (torch.randn(1, 1, 4096, generator=g) * 2).repeat(2, 4, 1)
    _check(cuda_device, x, torch.full((2, 4), -1.5), 10)


def test_selection_replayed_from_a_graph(cuda_device):
    g = torch.Generator().manual_seed(9)
    x = (torch.randn(4, 4, 3000, generator=g)).to(cuda_device)
    c = _scores(4, 4, g).to(cuda_device)
    graph = torch.cuda.CUDAGraph()
    wkv4.beam_select(x, c)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = wkv4.beam_select(x, c)
    for seed in (1, 2):
        x.copy_(torch.randn(4, 4, 3000, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        want = wkv4.beam_select(x, c)
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)


# ------------------------------------------------------------ state moves


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(3, 9, 64, 1, 4), (1, 5, 1, 1, 1), (7, 40, 37, 4, 8), (36, 70, 768, 2, 32),
                                   (2, 33, 1030, 3, 11), (3, 300, 130, 37, 6)],
                         ids=lambda s: "P%dS%dC%dG%dK%d" % s)
def test_states_move_like_rows_one_by_one(cuda_device, shape, dt):
    P, S, C, G, K = shape
    g = torch.Generator().manual_seed(S + C)
    pool = torch.randn(P, S, C, generator=g).to(DT[dt])
    pool[0, 0, 0] = float("nan")  # moved as they are
    ids = torch.randperm(S, generator=g)[:G * K].int().view(G, K)
    dev_pool = pool.to(cuda_device)
    cur = ids.to(cuda_device)
    ref, ref_ids = pool.float().numpy(), ids.numpy()
    for step in range(4):
        par = torch.randint(0, K, (G, K), generator=g).int()
        if step == 1:
            par[:] = torch.randint(0, K, (G, 1), generator=g).int()   # one parent for all
        elif step == 2:
            par = torch.argsort(torch.rand(G, K, generator=g), dim=1).int()   # everyone goes on
        ref, ref_ids = obeam.reorder(ref, ref_ids, par.numpy())
        cur = wkv4.state_reorder(dev_pool, cur, par.to(cuda_device))
        torch.cuda.synchronize()
        assert np.array_equal(cur.cpu().numpy(), ref_ids)
        assert np.array_equal(dev_pool.float().cpu().numpy(), ref, equal_nan=True)


def test_pools_that_share_slots_and_misaligned_pools(cuda_device):
    G, K, S = 2, 5, 16
    g = torch.Generator().manual_seed(2)
    ids = torch.randperm(S, generator=g)[:G * K].int().view(G, K).to(cuda_device)
    par = torch.randint(0, K, (G, K), generator=g).int().to(cuda_device)
    buf = torch.randn(1 + 3 * S * 64, generator=g).to(cuda_device)
    pools = [torch.randn(6, S, 64, generator=g).to(cuda_device), buf[1:].view(3, S, 64),
             torch.randn(2, S, 7, generator=g).to(torch.bfloat16).to(cuda_device)]
    refs = [obeam.reorder(p.float().cpu().numpy(), ids.cpu().numpy(), par.cpu().numpy()) for p in pools]
    first = buf[0].clone()
    news = [wkv4.state_reorder(p, ids, par) for p in pools]
    torch.cuda.synchronize()
    for p, new, (rp, ri) in zip(pools, news, refs):
        assert np.array_equal(p.float().cpu().numpy(), rp) and np.array_equal(new.cpu().numpy(), ri)
    assert torch.equal(buf[0], first)


def test_bad_groups_are_reported_and_left_as_they_are(cuda_device):
    S, C, K = 12, 40, 3
    pool = torch.randn(3, S, C, device=cuda_device)
    ids = torch.tensor([[0, 1, 2], [3, 4, S], [5, -1, 6], [7, 7, 8], [9, 10, 11]], dtype=torch.int32)
    par = torch.tensor([[0, 0, 3], [0, 0, 1], [0, 0, 1], [0, 0, 1], [2, 2, 0]], dtype=torch.int32)
    before = pool.clone()
    new = wkv4.state_reorder(pool, ids.to(cuda_device), par.to(cuda_device))
    torch.cuda.synchronize()
    assert wkv4.device_error(reset=True) == -8
    assert torch.equal(new.cpu()[:4], ids[:4])
    rp, ri = obeam.reorder(before.cpu().numpy(), ids[4:].numpy(), par[4:].numpy())
    assert np.array_equal(pool.cpu().numpy(), rp) and np.array_equal(new.cpu().numpy()[4:], ri)


# --------------------------------------------------------- a whole search


@pytest.mark.parametrize("graphed", [False, True], ids=["eager", "graph"])
def test_beam_search_over_a_recurrent_layer(cuda_device, graphed):
    """Several requests' beams through embedding -> token mix -> slot decode ->
    logits -> selection -> state moves: at the end each beam's score is the sum
    of its own tokens' log-probabilities, recomputed from its history alone by
    the fp64 oracle, and the scores descend."""
    dev = cuda_device
    G, K, C, V, steps = 3, 4, 32, 211, 9
    g = torch.Generator().manual_seed(77)
    emb = torch.randn(V, C, generator=g)
    Wk, Wv, Wh = (torch.randn(C, m, generator=g) * s for m, s in ((C, 0.3), (C, 0.3), (V, 0.6)))
    w, u = -torch.exp(torch.rand(C, generator=g) * 3 - 2), torch.rand(C, generator=g)
    D = {n: t.to(dev) for n, t in dict(emb=emb, Wk=Wk, Wv=Wv, Wh=Wh, w=w, u=u).items()}
    S = G * K + 5
    pool = torch.zeros(3, S, C, device=dev)
    pool[2] = -1e38
    last = torch.zeros(1, S, C, device=dev)   # the token before, per slot
    ids = torch.randperm(S, generator=g)[:G * K].int().view(G, K).to(dev)
    tokens = torch.zeros(G, K, dtype=torch.int32, device=dev)
    scores = torch.full((G, K), -INF, device=dev)
    scores[:, 0] = 0.0

    def step():
        x = D["emb"][tokens.view(-1).long()]
        rows = ids.view(-1).long()
        mixed = 0.5 * (x + last[0, rows])
        last[0, rows] = x
        k, v = mixed @ D["Wk"], mixed @ D["Wv"]
        y = wkv4.decode_step_slots(k, v, D["w"], D["u"], pool, ids.view(-1))
        logits = (y @ D["Wh"]).view(G, K, V)
        s, p, t = wkv4.beam_select(logits, scores)
        new = wkv4.state_reorder(pool, ids, p)
        wkv4.state_reorder(last, ids, p)
        ids.copy_(new)
        scores.copy_(s)
        tokens.copy_(t)
        return p

    keep = [t.clone() for t in (pool, last, ids, tokens, scores)]
    hist = [[[0] for _ in range(K)] for _ in range(G)]
    if graphed:
        step()  # warm up, then start over
        for t, old in zip((pool, last, ids, tokens, scores), keep):
            t.copy_(old)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            parents = step()
        for t, old in zip((pool, last, ids, tokens, scores), keep):
            t.copy_(old)
    for _ in range(steps):
        if graphed:
            graph.replay()
            p = parents
        else:
            p = step()
        torch.cuda.synchronize()
        hist = [[hist[a][int(p[a, b])] + [int(tokens[a, b])] for b in range(K)] for a in range(G)]
    got = scores.cpu().double().numpy()
    assert np.all(np.diff(got, axis=1) <= 0)
    for a in range(G):
        assert len({tuple(h) for h in hist[a]}) == K
        for b in range(K):
            seq = hist[a][b]
            x = emb[torch.tensor(seq[:-1])].double().numpy()
            mixed = 0.5 * (x + np.concatenate([np.zeros((1, C)), x[:-1]]))
            k, v = mixed @ Wk.double().numpy(), mixed @ Wv.double().numpy()
            y, _ = oracle.forward(k[None], v[None], w, u, None)
            logits = y[0] @ Wh.double().numpy()
            logp = logits - logits.max(1, keepdims=True)
            logp -= np.log(np.exp(logp).sum(1, keepdims=True))
            want = sum(logp[i, seq[i + 1]] for i in range(steps))
            # per step: two fp32 (at worst tf32-free) products over C = 32 terms of order one and the decode's own
            # rounding, 2^-24 of the terms' magnitudes each: below 2^-24 (32 + 32 + 64) 32 of a logit
            assert abs(got[a, b] - want) <= steps * 2.0 ** -24 * 128 * 32
