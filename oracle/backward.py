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


def wkv_backward_any_range(k, v, w, u, gy, state_in=None, r=None, state_out=None, gstate_out=None):
    """wkv_backward for keys of any size (masks of -1e9 or -1e30 with nothing
    before them, where the true sums underflow): every sum is held against a
    running max, whose exponents are extended floats.  As in any floating point,
    a decay or a bonus next to a max that swallows it is lost."""
    k, v, w, u, gy, state_in, r, state_out, gstate_out = map(
        _f64, (k, v, w, u, gy, state_in, r, state_out, gstate_out))
    X = np.longdouble
    B, T, C = k.shape
    ex = lambda d: np.exp(np.clip(d, X(-1e4), X(700))).astype(np.float64)  # differences of exponents

    def add(a, p, b, q):
        """Sums a e^p and b e^q (dicts of parts): the parts and the exponent of the sum."""
        m = np.maximum(p, q)
        fa, fb = ex(p - m), ex(q - m)
        return [x * fa + y * fb for x, y in zip(a, b)], m

    kx, wx, ux = k.astype(X), w.astype(X), u.astype(X)
    if state_in is None:
        S, p = [np.zeros((B, C))] * 3, np.full((B, C), X(-1e38))
    else:
        S, p = [state_in[0], state_in[1], np.abs(state_in[0])], state_in[2].astype(X)
    p0, s0 = p, S
    As, Ds, Am, ps = [], [], [], []
    for t in range(T):
        As.append(S[0])
        Ds.append(S[1])
        Am.append(S[2])
        ps.append(p)
        S, p = add(S, p + wx, [v[:, t], np.ones((B, C)), np.abs(v[:, t])], kx[:, t])
    As, Ds, Am, ps = (np.stack(x, 1) for x in (As, Ds, Am, ps))
    m = np.maximum(ps, ux + kx)
    fs, fe = ex(ps - m), ex(ux + kx - m)
    Z = fs * Ds + fe
    y, ym = (fs * As + fe * v) / Z, (fs * Am + fe * np.abs(v)) / Z
    out, mag = {}, {}
    g = gy
    if r is not None:
        s = 1.0 / (1.0 + np.exp(-r))
        out["gr"], mag["gr"] = gy * y * s * (1.0 - s), np.abs(gy) * ym * s * (1.0 - s)
        g = gy * s
    al = g / Z   # in units of e^{-m}
    if gstate_out is None:
        R, h = [np.zeros((B, C))] * 4, np.full((B, C), X(-1e38))
    else:
        R, h = [gstate_out[0], gstate_out[1], np.abs(gstate_out[0]), np.abs(gstate_out[1])], -state_out[2].astype(X)
    zero = lambda parts, at: np.where(sum(np.abs(x) for x in parts) == 0, X(-1e38), at)
    h = zero(R, h)
    gk, gv, gkm, gvm = (np.empty_like(k) for _ in range(4))
    gw, gu, gwm, gum = (np.zeros(C) for _ in range(4))
    for t in range(T - 1, -1, -1):
        a, am, vt, vm = al[:, t], np.abs(al[:, t]), v[:, t], np.abs(v[:, t])
        own, ownm = fe[:, t] * a * (vt - y[:, t]), fe[:, t] * am * (vm + ym[:, t])
        f = ex(h + kx[:, t])
        gv[:, t] = fe[:, t] * a + f * R[0]
        gvm[:, t] = fe[:, t] * am + f * R[2]
        gk[:, t] = own + f * (R[0] * vt + R[1])
        gkm[:, t] = ownm + f * (R[2] * vm + R[3])
        gu += own.sum(0)
        gum += ownm.sum(0)
        fw = ex((h + ps[:, t]) + wx)
        gw += (fw * (R[0] * As[:, t] + R[1] * Ds[:, t])).sum(0)
        gwm += (fw * (R[2] * Am[:, t] + R[3] * Ds[:, t])).sum(0)
        step = [a, -a * y[:, t], am, am * ym[:, t]]
        R, h = add(R, h + wx, step, zero(step, -m[:, t]))
        h = zero(R, h)
    out.update(gk=gk, gv=gv, gw=gw, gu=gu)
    mag.update(gk=gkm, gv=gvm, gw=gwm, gu=gum)
    if state_in is not None:
        ga, gb, gam, gbm = (x * ex(h + p0) for x in R)
        out["gstate_in"] = np.stack([ga, gb, s0[0] * ga + s0[1] * gb])
        mag["gstate_in"] = np.stack([gam, gbm, np.abs(s0[0]) * gam + np.abs(s0[1]) * gbm])
    return out, mag
