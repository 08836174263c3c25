"""The training and beam-search operators of the time mix, as cases to be measured.

Four operators that stand beside the WKV forward, the token shift and the slot decode:

  wkv_backward          gradients of the (gated) WKV recurrence: k, v, r, w, u and the carried state
  token_shift_backward  gradients of the token shift: x, the mixes and the carried token
  beam_select           the n best continuations over beams and vocabulary
  state_reorder         the states of a slot pool moved to the beams that go on

Where `own` is false, `run` computes them in their plain form (elementary torch operations); where it is true it
calls the framework.
"""

import math

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_ES = {"f32": 4, "f16": 2, "bf16": 2}
_DEV = "cuda"


# ------------------------------------------------------------------- cases


def listed():
    return [
        # the latency end of training: one short sequence at the small model's width, fp32
        {"name": "wkv_bwd_short", "op": "wkv_backward", "B": 1, "T": 48, "C": 768, "dtype": "f32",
         "gated": False, "state": False},
        # a training step's layer at the small model's width (B=8, T=1024, C=768, fp16), state carried in and out
        {"name": "wkv_bwd_169m", "op": "wkv_backward", "B": 8, "T": 1024, "C": 768, "dtype": "f16",
         "gated": True, "state": True},
        # the same at the 14B width (B=4, T=1024, C=5120, bf16)
        {"name": "wkv_bwd_14b", "op": "wkv_backward", "B": 4, "T": 1024, "C": 5120, "dtype": "bf16",
         "gated": True, "state": False},
        # one long document in fp32: T far past what one group of blocks holds
        {"name": "wkv_bwd_long", "op": "wkv_backward", "B": 1, "T": 16384, "C": 2048, "dtype": "f32",
         "gated": False, "state": False},
        # odd sizes: no 16-byte rows, a ragged end
        {"name": "wkv_bwd_ragged", "op": "wkv_backward", "B": 3, "T": 777, "C": 1027, "dtype": "bf16",
         "gated": True, "state": True},
        # token shift: a short fine-tuning batch, and the 14B width
        {"name": "shift_bwd_short", "op": "token_shift_backward", "B": 2, "T": 65, "C": 768, "dtype": "f16",
         "outs": 3, "carry": True},
        {"name": "shift_bwd_14b", "op": "token_shift_backward", "B": 4, "T": 1024, "C": 5120, "dtype": "bf16",
         "outs": 3, "carry": False},
        # one request with 4 beams over the model's vocabulary: latency of a decode loop
        {"name": "beam_select_one", "op": "beam_select", "G": 1, "K": 4, "V": 50277, "pad": 0, "n": 4,
         "dtype": "f32", "masked": 0.0, "finished": False},
        # a serving batch, 2K candidates so that finished beams can be set aside, padded vocabulary rows
        {"name": "beam_select_batch", "op": "beam_select", "G": 48, "K": 8, "V": 50277, "pad": 27, "n": 16,
         "dtype": "bf16", "masked": 0.2, "finished": True},
        # the state pool of one request at the small width (12 layers of three planes)
        {"name": "reorder_one", "op": "state_reorder", "P": 36, "S": 16, "C": 768, "G": 1, "K": 4,
         "survivors": 2, "dtype": "f32"},
        # 40 layers at the 14B width for 8 requests of 8 beams
        {"name": "reorder_14b", "op": "state_reorder", "P": 120, "S": 80, "C": 5120, "G": 8, "K": 8,
         "survivors": 5, "dtype": "f32"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["wkv_backward", "wkv_backward", "token_shift_backward", "beam_select", "state_reorder"])
    dt = rng.choice(["f32", "f16", "bf16"])
    if op == "wkv_backward":
        while True:
            B, T, C = _log_int(rng, 1, 12), _log_int(rng, 1, 12000), _log_int(rng, 17, 5200)
            if rng.random() < 0.7:
                C = max(16, C // 8 * 8)
            if 2000 <= B * T * C <= 20_000_000:
                break
        return {"op": op, "B": B, "T": T, "C": C, "dtype": dt, "gated": rng.random() < 0.6,
                "state": rng.random() < 0.4}
    if op == "token_shift_backward":
        while True:
            B, T, C = _log_int(rng, 1, 24), _log_int(rng, 1, 5000), _log_int(rng, 17, 5200)
            if rng.random() < 0.7:
                C = max(16, C // 8 * 8)
            if 2000 <= B * T * C <= 20_000_000:
                break
        return {"op": op, "B": B, "T": T, "C": C, "dtype": dt, "outs": rng.choice([2, 3]),
                "carry": rng.random() < 0.5}
    if op == "beam_select":
        while True:
            G, K, V = _log_int(rng, 1, 64), _log_int(rng, 1, 16), _log_int(rng, 50, 66000)
            if G * K * V <= 18_000_000:
                break
        n = rng.choice([K, 2 * K, 2 * K + 1])
        return {"op": op, "G": G, "K": K, "V": V, "pad": rng.choice([0, 0, 3, 64]), "n": n, "dtype": dt,
                "masked": rng.choice([0.0, 0.3, 0.9]), "finished": rng.random() < 0.5}
    while True:
        P, C, G, K = _log_int(rng, 1, 120), _log_int(rng, 17, 5200), _log_int(rng, 1, 24), _log_int(rng, 1, 16)
        if rng.random() < 0.7:
            C = max(16, C // 8 * 8)
        S = G * K + rng.randint(0, 20)
        if P * S * C <= 45_000_000:
            break
    return {"op": op, "P": P, "S": S, "C": C, "G": G, "K": K, "survivors": rng.randint(1, K), "dtype": dt}


def work(case):
    es = _ES[case["dtype"]]
    op = case["op"]
    if op == "wkv_backward":
        n = case["B"] * case["T"] * case["C"]
        bc = case["B"] * case["C"]
        tensors = 7 if case["gated"] else 5
        state = 12 * bc * 4 if case["state"] else 0  # state in and out, both gradients
        return {"bytes": tensors * n * es + state + 16 * case["C"], "flops": (48 if case["gated"] else 40) * n}
    if op == "token_shift_backward":
        n = case["B"] * case["T"] * case["C"]
        rows = case["B"] * case["C"] * es * (3 if case["carry"] else 0)
        return {"bytes": (case["outs"] + 2) * n * es + rows + 8 * case["outs"] * case["C"],
                "flops": 7 * case["outs"] * n}
    if op == "beam_select":
        rows = case["G"] * case["K"]
        return {"bytes": rows * case["V"] * es + 5 * rows + 12 * case["G"] * case["n"],
                "flops": 4 * rows * case["V"]}
    moved = case["G"] * (case["K"] - case["survivors"])
    return {"bytes": 2 * moved * case["P"] * case["C"] * es + 12 * case["G"] * case["K"], "flops": 0}


# ------------------------------------------------------------------ inputs


def _gen(seed):
    return torch.Generator(device=_DEV).manual_seed(int(seed))


def prepare(case, seed):
    g = _gen(seed)
    dt = _DT[case["dtype"]]
    st = {"case": case}

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=_DEV) * std

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, generator=g, device=_DEV) * (hi - lo) + lo

    if case["op"] == "wkv_backward":
        B, T, C = case["B"], case["T"], case["C"]
        # decays and bonuses over the range of the forward's workloads, activations of order one, a key far
        # above the rest now and then
        st["w"] = -torch.exp(uniform(-6.0, 1.0, C))
        st["u"] = uniform(-1.0, 1.0, C)
        k = normal(B, T, C, std=1.4)
        k[uniform(0.0, 1.0, B, T, C) < 5e-4] += 12.0
        st["k"] = k.to(dt)
        st["v"] = normal(B, T, C).to(dt)
        st["gy"] = normal(B, T, C).to(dt)
        st["r"] = normal(B, T, C).to(dt) if case["gated"] else None
        st["state_in"] = st["state_out"] = st["gstate_out"] = None
        if case["state"]:
            st["state_in"] = torch.stack([normal(B, C), uniform(0.5, 2.0, B, C), uniform(-2.0, 2.0, B, C)])
            a, b, p = _states(st)
            st["state_out"] = torch.stack([a[:, -1], b[:, -1], p[:, -1]])
            st["gstate_out"] = normal(3, B, C)
    elif case["op"] == "token_shift_backward":
        B, T, C = case["B"], case["T"], case["C"]
        st["x"] = normal(B, T, C).to(dt)
        st["mix"] = [uniform(0.0, 1.0, C) for _ in range(case["outs"])]
        st["g"] = [normal(B, T, C).to(dt) for _ in range(case["outs"])]
        st["x_prev"] = normal(B, C).to(dt) if case["carry"] else None
        st["gx_last"] = normal(B, C).to(dt) if case["carry"] else None
    elif case["op"] == "beam_select":
        G, K, V = case["G"], case["K"], case["V"]
        logits = normal(G, K, V + case["pad"], std=2.5)
        logits[..., 0] += 3.0
        if case["masked"] > 0:  # tokens that a grammar or a stop list rules out
            off = uniform(0.0, 1.0, G, 1, V + case["pad"]) < case["masked"]
            logits = logits.masked_fill(off, float("-inf"))
        st["logits"] = logits.to(dt)[..., :V]
        st["scores"] = -torch.sort(uniform(0.0, 1.0, G, K) * 8.0 + 4.0, dim=1).values
        st["finished"] = (uniform(0.0, 1.0, G, K) < 0.15) if case["finished"] else None
        st["end_id"] = 0
    else:
        P, S, C, G, K = (case[x] for x in "PSCGK")
        st["pool"] = normal(P, S, C).to(dt)
        order = torch.argsort(uniform(0.0, 1.0, S))
        st["slot_ids"] = order[:G * K].to(torch.int32).view(G, K).contiguous()
        # exactly `survivors` different parents a group, in any order
        alive = torch.argsort(uniform(0.0, 1.0, G, K), dim=1)[:, :case["survivors"]]
        pick = (uniform(0.0, 1.0, G, K) * case["survivors"]).long().clamp_(max=case["survivors"] - 1)
        pick[:, :case["survivors"]] = torch.arange(case["survivors"], device=_DEV)
        parents = torch.gather(alive, 1, pick)
        mix = torch.argsort(uniform(0.0, 1.0, G, K), dim=1)
        st["parents"] = torch.gather(parents, 1, mix).to(torch.int32).contiguous()
    return st


# -------------------------------------------------------------- plain forms


def _scan(a, b, p, w):
    """Inclusive scan over dim 1 of (a, b, max p) triples, each step decaying what came before by e^w:
    log2(T) rounds of doubling, each joining a window of d steps with the one before it."""
    T, d = a.shape[1], 1
    while d < T:
        px = p[:, :-d] + d * w
        q = torch.maximum(px, p[:, d:])
        fx, fy = torch.exp(px - q), torch.exp(p[:, d:] - q)
        a = torch.cat([a[:, :d], a[:, :-d] * fx + a[:, d:] * fy], 1)
        b = torch.cat([b[:, :d], b[:, :-d] * fx + b[:, d:] * fy], 1)
        p = torch.cat([p[:, :d], q], 1)
        d *= 2
    return a, b, p


def _states(st):
    """The state before every step and after the last one: T + 1 triples a channel."""
    k, v = st["k"].float(), st["v"].float()
    if st["state_in"] is None:
        s = torch.zeros(3, k.shape[0], k.shape[2], device=k.device)
        s[2] = -1e38
    else:
        s = st["state_in"]
    return _scan(torch.cat([s[0][:, None], v], 1), torch.cat([s[1][:, None], torch.ones_like(k)], 1),
                 torch.cat([s[2][:, None], k], 1), st["w"])


def _plain_wkv_backward(st):
    dt = st["k"].dtype
    k, v, gy, w, u = st["k"].float(), st["v"].float(), st["gy"].float(), st["w"], st["u"]
    a, b, p = (x[:, :-1] for x in _states(st))
    m = torch.maximum(p, u + k)
    fa, fe = torch.exp(p - m), torch.exp(u + k - m)
    z = fa * b + fe
    y = (fa * a + fe * v) / z
    gr = None
    if st["r"] is not None:
        s = 1.0 / (1.0 + torch.exp(-st["r"].float()))
        gr = gy * y * s * (1.0 - s)
        gy = gy * s
    al = gy / z
    # dL/dA, dL/dD after every step, in units of e^{-max}
    if st["gstate_out"] is None:
        last = [torch.zeros_like(k[:, :1]), torch.zeros_like(k[:, :1]), torch.full_like(k[:, :1], -1e38)]
    else:
        last = [st["gstate_out"][0][:, None], st["gstate_out"][1][:, None], -st["state_out"][2][:, None]]
    P, Q, h = (x.flip(1) for x in _scan(torch.cat([last[0], al.flip(1)], 1),
                                        torch.cat([last[1], (-al * y).flip(1)], 1),
                                        torch.cat([last[2], (-m).flip(1)], 1), w))
    Pn, Qn, hn = P[:, 1:], Q[:, 1:], h[:, 1:]
    own_step, later = fe * al, torch.exp(k + hn)
    gv = own_step + later * Pn
    gu = own_step * (v - y)
    gk = gu + later * (Pn * v + Qn)
    gw = torch.exp(w + p + hn) * (Pn * a + Qn * b)
    out = {"gk": gk.to(dt), "gv": gv.to(dt), "gw": gw.sum((0, 1)), "gu": gu.sum((0, 1))}
    if gr is not None:
        out["gr"] = gr.to(dt)
    if st["state_in"] is not None:
        f = torch.exp(h[:, 0] + st["state_in"][2])
        ga, gb = P[:, 0] * f, Q[:, 0] * f
        out["gstate_in"] = torch.stack([ga, gb, st["state_in"][0] * ga + st["state_in"][1] * gb])
    return out


def _plain_shift_backward(st):
    x, dt = st["x"].float(), st["x"].dtype
    B, T, C = x.shape
    first = torch.zeros(B, 1, C, device=x.device) if st["x_prev"] is None else st["x_prev"].float()[:, None]
    diff = x - torch.cat([first, x[:, :-1]], 1)
    gx = torch.zeros_like(x)
    gp = torch.zeros(B, C, device=x.device)
    gmix = []
    for mix, g in zip(st["mix"], st["g"]):
        g = g.float()
        gx += mix * g
        gx[:, :-1] += (1.0 - mix) * g[:, 1:]
        gp += (1.0 - mix) * g[:, 0]
        gmix.append((g * diff).sum((0, 1)))
    if st["gx_last"] is not None:
        gx[:, -1] += st["gx_last"].float()
    out = {"gx": gx.to(dt), "gmix": gmix}
    if st["x_prev"] is not None:
        out["gx_prev"] = gp.to(dt)
    return out


def _plain_beam_select(st):
    G, K, V = st["logits"].shape
    x = st["logits"].double()  # 64 bits: candidates of different beams lie as close as their sums' rounding
    top = x.max(-1, keepdim=True).values
    lse = top + torch.log(torch.exp(x - top).sum(-1, keepdim=True))
    s = st["scores"].double()[..., None]
    alive = torch.isfinite(lse) & (s.abs() <= 2e9)
    cand = torch.where(alive, s + (x - lse), float("-inf"))
    if st["finished"] is not None:
        only = torch.full_like(cand, float("-inf"))
        only[..., st["end_id"]] = torch.where(s.abs() <= 2e9, s, float("-inf"))[..., 0]
        cand = torch.where(st["finished"][..., None], only, cand)
    best, at = torch.sort(cand.view(G, K * V), dim=1, descending=True, stable=True)
    at = at[:, :st["case"]["n"]]
    return {"scores": best[:, :st["case"]["n"]].float(), "parents": (at // V).to(torch.int32),
            "tokens": (at % V).to(torch.int32)}


def _plain_state_reorder(st):
    ids, par = st["slot_ids"].long(), st["parents"].long()
    G, K = ids.shape
    src = torch.gather(ids, 1, par)
    j = torch.arange(K, device=ids.device)
    earlier = (par[:, :, None] == par[:, None, :]) & (j[None, :, None] > j[None, None, :])
    first = ~earlier.any(2)  # the first child of its parent keeps the parent's slot
    childless = ~(par[:, None, :] == j[None, :, None]).any(2)
    free = torch.argsort((~childless).to(torch.int32), dim=1, stable=True)  # childless beams first, in order
    rank = (torch.cumsum((~first).to(torch.int64), 1) - 1).clamp(min=0)
    dst = torch.where(first, src, torch.gather(ids, 1, torch.gather(free, 1, rank)))
    st["pool"][:, dst.view(-1)] = st["pool"][:, src.view(-1)]
    return {"pool": st["pool"], "slot_ids": dst.to(torch.int32)}


# --------------------------------------------------------------------- run


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"wkv_backward": _plain_wkv_backward, "token_shift_backward": _plain_shift_backward,
                "beam_select": _plain_beam_select, "state_reorder": _plain_state_reorder}[op](state)
    from rwkv_wkv_linear_b200 import wkv4
    if op == "wkv_backward":
        g = wkv4.backward(state["k"], state["v"], state["w"], state["u"], state["gy"], state["state_in"],
                          r=state["r"], state_out=state["state_out"], gstate_out=state["gstate_out"])
        out = {"gk": g.gk, "gv": g.gv, "gw": g.gw, "gu": g.gu}
        if g.gr is not None:
            out["gr"] = g.gr
        if g.gstate_in is not None:
            out["gstate_in"] = g.gstate_in
        return out
    if op == "token_shift_backward":
        mixes = list(state["mix"]) + [None] * (3 - len(state["mix"]))
        gs = list(state["g"]) + [None] * (3 - len(state["g"]))
        r = wkv4.token_shift_backward(state["x"], mixes[0], mixes[1], gs[0], gs[1], mixes[2], gs[2],
                                      state["x_prev"], gx_last=state["gx_last"])
        out = {"gx": r.gx, "gmix": [m for m in (r.gmix_k, r.gmix_v, r.gmix_r) if m is not None]}
        if r.gx_prev is not None:
            out["gx_prev"] = r.gx_prev
        return out
    if op == "beam_select":
        scores, parents, tokens = wkv4.beam_select(state["logits"], state["scores"], state["case"]["n"],
                                                   finished=state["finished"], end_id=state["end_id"])
        return {"scores": scores, "parents": parents, "tokens": tokens}
    ids = wkv4.state_reorder(state["pool"], state["slot_ids"], state["parents"])
    return {"pool": state["pool"], "slot_ids": ids}


# ------------------------------------------------------------------- exact


def _exact_wkv_backward(st):
    """Step after step in 64 bits on the true sums (no running max: e^k stays far inside the range)."""
    k, v, gy = (st[x].double() for x in ("k", "v", "gy"))
    w, u = st["w"].double(), st["u"].double()
    B, T, C = k.shape
    ew, eu, ek = torch.exp(w), torch.exp(u), torch.exp(k)
    if st["state_in"] is None:
        A = D = torch.zeros(B, C, dtype=torch.float64, device=k.device)
    else:
        s0 = st["state_in"].double()
        e0 = torch.exp(s0[2])
        A, D = s0[0] * e0, s0[1] * e0
    As, Ds = torch.empty_like(k), torch.empty_like(k)
    ekv = ek * v
    for t in range(T):
        As[:, t], Ds[:, t] = A, D
        A = torch.addcmul(ekv[:, t], ew, A)
        D = torch.addcmul(ek[:, t], ew, D)
    Z = Ds + eu * ek
    y = (As + eu * ekv) / Z
    out = {}
    gate = torch.ones_like(k) if st["r"] is None else torch.sigmoid(st["r"].double())
    al = gy * gate / Z
    be = -al * y
    if st["gstate_out"] is None:
        P = Q = torch.zeros(B, C, dtype=torch.float64, device=k.device)
    else:
        f = torch.exp(-st["state_out"][2].double())
        P, Q = st["gstate_out"][0].double() * f, st["gstate_out"][1].double() * f
    Pn, Qn = torch.empty_like(k), torch.empty_like(k)
    for t in range(T - 1, -1, -1):
        Pn[:, t], Qn[:, t] = P, Q
        P = torch.addcmul(al[:, t], ew, P)
        Q = torch.addcmul(be[:, t], ew, Q)
    out["gv"] = ek * (eu * al + Pn)
    out["gk"] = ek * (eu * (al * v + be) + Pn * v + Qn)
    out["gw"] = (ew * (Pn * As + Qn * Ds)).sum((0, 1))
    out["gu"] = (eu * ek * (al * v + be)).sum((0, 1))
    if st["r"] is not None:
        out["gr"] = gy * y * gate * (1.0 - gate)
    if st["state_in"] is not None:
        out["gstate_in"] = torch.stack([P * e0, Q * e0, P * s0[0] * e0 + Q * s0[1] * e0])
    return out


def _exact_shift_backward(st):
    x = st["x"].double()
    B, T, C = x.shape
    n = len(st["mix"])
    # position t of the extended row holds x[t - 1]; its gradient is read off at both places that use it
    gext = torch.zeros(B, T + 1, C, dtype=torch.float64, device=x.device)
    xext = torch.zeros(B, T + 1, C, dtype=torch.float64, device=x.device)
    xext[:, 1:] = x
    if st["x_prev"] is not None:
        xext[:, 0] = st["x_prev"].double()
    gmix = []
    for i in range(n):
        m, g = st["mix"][i].double(), st["g"][i].double()
        gext[:, 1:] += g * m
        gext[:, :T] += g * (1.0 - m)
        gmix.append(torch.einsum("btc,btc->c", g, xext[:, 1:]) - torch.einsum("btc,btc->c", g, xext[:, :T]))
    if st["gx_last"] is not None:
        gext[:, T] += st["gx_last"].double()
    out = {"gx": gext[:, 1:], "gmix": gmix}
    if st["x_prev"] is not None:
        out["gx_prev"] = gext[:, 0]
    return out


def _exact_beam_select(st):
    G, K, V = st["logits"].shape
    n = st["case"]["n"]
    scores = torch.empty(G, n, dtype=torch.float64)
    parents, tokens = torch.empty(G, n, dtype=torch.int32), torch.empty(G, n, dtype=torch.int32)
    for g in range(G):
        row = torch.log_softmax(st["logits"][g].double(), dim=-1) + st["scores"][g].double()[:, None]
        row = torch.nan_to_num(row, nan=float("-inf"), neginf=float("-inf"))
        if st["finished"] is not None:
            for b in range(K):
                if bool(st["finished"][g, b]):
                    row[b] = float("-inf")
                    row[b, st["end_id"]] = st["scores"][g, b].double()
        flat = row.reshape(-1).cpu()
        # everything at or above the n-th value, in order of (value down, index up)
        least = torch.topk(flat, n).values[-1]
        cand = torch.nonzero(flat > least).view(-1).tolist()
        cand.sort(key=lambda i: (-float(flat[i]), i))
        ties = torch.nonzero(flat == least).view(-1)[:n - len(cand)].tolist()
        for j, i in enumerate(cand + ties):
            scores[g, j], parents[g, j], tokens[g, j] = flat[i], i // V, i % V
    return {"scores": scores, "parents": parents, "tokens": tokens}


def _exact_state_reorder(st):
    ids, par = st["slot_ids"].tolist(), st["parents"].tolist()
    src, new = [], []
    for group, parents in zip(ids, par):
        free = [group[b] for b in range(len(group)) if b not in parents]
        seen = set()
        for p in parents:
            src.append(group[p])
            new.append(group[p] if p not in seen else free.pop(0))
            seen.add(p)
    pool = st["pool"].clone()
    for a, b in zip(src, new):
        if a != b:
            pool[:, b] = st["pool"][:, a]
    return {"pool": pool, "slot_ids": torch.tensor(new, dtype=torch.int32).view(len(ids), -1)}


def exact(case, seed):
    st = prepare(case, seed)
    return {"wkv_backward": _exact_wkv_backward, "token_shift_backward": _exact_shift_backward,
            "beam_select": _exact_beam_select, "state_reorder": _exact_state_reorder}[case["op"]](st)
