"""Gradients of the WKV recurrence and of the token shift in fp64, step after
step on the true sums (no running max: keys of a few hundred nats stay inside
fp64), written from the formulas.

Each function returns the gradients and, under the same names, the sums of the
magnitudes of the terms they are made of: the scale that rounding is measured
against where terms cancel.
"""

import numpy as np


def _f64(x):
    if x is None:
        return None
    if hasattr(x, "detach"):
        x = x.detach().to("cpu").double().numpy()
    return np.asarray(x, dtype=np.float64)


def wkv_backward(k, v, w, u, gy, state_in=None, r=None, state_out=None, gstate_out=None):
    """Gradients of out = sigmoid(r) wkv (r None: no gate) and of the state
    after the last step: dict of gk, gv, gr, gw, gu, gstate_in, and the same of
    magnitudes."""
    k, v, w, u, gy, state_in, r, state_out, gstate_out = map(
        _f64, (k, v, w, u, gy, state_in, r, state_out, gstate_out))
    B, T, C = k.shape
    ew, eu, ek = np.exp(w), np.exp(u), np.exp(k)
    zero = np.zeros((B, C))
    if state_in is None:
        e0, A, D = zero, zero, zero
    else:
        e0 = np.exp(state_in[2])
        A, D = state_in[0] * e0, state_in[1] * e0
    As, Ds, Am = np.empty_like(k), np.empty_like(k), np.empty_like(k)
    M = np.abs(A)
    for t in range(T):
        As[:, t], Ds[:, t], Am[:, t] = A, D, M
        A = ew * A + ek[:, t] * v[:, t]
        D = ew * D + ek[:, t]
        M = ew * M + ek[:, t] * np.abs(v[:, t])
    Z = Ds + eu * ek
    y = (As + eu * ek * v) / Z
    ym = (Am + eu * ek * np.abs(v)) / Z
    out, mag = {}, {}
    g = gy
    if r is not None:
        s = 1.0 / (1.0 + np.exp(-r))
        out["gr"] = gy * y * s * (1.0 - s)
        mag["gr"] = np.abs(gy) * ym * s * (1.0 - s)
        g = gy * s
    al = g / Z
    if gstate_out is None:
        P, Q = zero, zero
    else:
        f = np.exp(-state_out[2])
        P, Q = gstate_out[0] * f, gstate_out[1] * f
    Pm, Qm = np.abs(P), np.abs(Q)
    gk, gv, gkm, gvm = (np.empty_like(k) for _ in range(4))
    gw, gu, gwm, gum = (np.zeros(C) for _ in range(4))
    for t in range(T - 1, -1, -1):
        a, am, vt, vm = al[:, t], np.abs(al[:, t]), v[:, t], np.abs(v[:, t])
        own, ownm = eu * a * (vt - y[:, t]), eu * am * (vm + ym[:, t])
        gv[:, t] = ek[:, t] * (eu * a + P)
        gk[:, t] = ek[:, t] * (own + P * vt + Q)
        gvm[:, t] = ek[:, t] * (eu * am + Pm)
        gkm[:, t] = ek[:, t] * (ownm + Pm * vm + Qm)
        gu += (ek[:, t] * own).sum(0)
        gum += (ek[:, t] * ownm).sum(0)
        gw += (ew * (P * As[:, t] + Q * Ds[:, t])).sum(0)
        gwm += (ew * (Pm * Am[:, t] + Qm * Ds[:, t])).sum(0)
        P, Q = a + ew * P, -a * y[:, t] + ew * Q
        Pm, Qm = am + ew * Pm, am * ym[:, t] + ew * Qm
    out.update(gk=gk, gv=gv, gw=gw, gu=gu)
    mag.update(gk=gkm, gv=gvm, gw=gwm, gu=gum)
    if state_in is not None:
        ga, gb, gam, gbm = e0 * P, e0 * Q, e0 * Pm, e0 * Qm
        out["gstate_in"] = np.stack([ga, gb, state_in[0] * ga + state_in[1] * gb])
        mag["gstate_in"] = np.stack([gam, gbm, np.abs(state_in[0]) * gam + np.abs(state_in[1]) * gbm])
    return out, mag


def token_shift_backward(x, mixes, grads, x_prev=None, gx_last=None):
    """Gradients of the token shift: dict of gx, gx_prev, gmix (a list), and the
    same of magnitudes."""
    x, x_prev, gx_last = _f64(x), _f64(x_prev), _f64(gx_last)
    B, T, C = x.shape
    ext = np.concatenate([np.zeros((B, 1, C)) if x_prev is None else x_prev[:, None], x], axis=1)
    g_ext, m_ext = np.zeros((B, T + 1, C)), np.zeros((B, T + 1, C))
    gmix, mmix = [], []
    for m, g in zip(mixes, grads):
        m, g = _f64(m), _f64(g)
        g_ext[:, 1:] += m * g
        g_ext[:, :-1] += (1.0 - m) * g
        m_ext[:, 1:] += np.abs(m * g)
        m_ext[:, :-1] += np.abs((1.0 - m) * g)
        gmix.append((g * (ext[:, 1:] - ext[:, :-1])).sum((0, 1)))
        mmix.append((np.abs(g) * (np.abs(ext[:, 1:]) + np.abs(ext[:, :-1]))).sum((0, 1)))
    if gx_last is not None:
        g_ext[:, -1] += gx_last
        m_ext[:, -1] += np.abs(gx_last)
    return (dict(gx=g_ext[:, 1:], gx_prev=g_ext[:, 0], gmix=gmix),
            dict(gx=m_ext[:, 1:], gx_prev=m_ext[:, 0], gmix=mmix))
