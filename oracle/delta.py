"""Plain float64 evaluation of the gated delta rule and of the block norm.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Both are evaluated from
their definitions, the delta rule token by token:

    C_t = f_t C_{t-1} + beta_t (v_t - f_t C_{t-1} k_t) k_t^T,   h_t = C_t q_t / sqrt(dk)

with f = sigma(f~) or exp(f~) and C rows by value; q, k [B, NHK, T, dk], v
[B, NH, T, dv], beta, fgate [B, NH, T], C [B, NH, dv, dk]; value head n reads key
head n // (NH // NHK).  Gradients are the reversed recurrence.
"""

import numpy as np


def _f(fgate, forget):
    x = np.asarray(fgate, np.float64)
    if forget == "exp":
        return np.exp(x)
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0, e) / (1.0 + e)


def _heads(x, group):
    return np.repeat(np.asarray(x, np.float64), group, axis=1)


def delta_forward(q, k, v, beta, fgate, C0=None, forget="sigmoid", all_states=False):
    """-> (h, C_T), or (h, [C_0 ... C_T]) with ``all_states``."""
    v = np.asarray(v, np.float64)
    B, NH, T, dv = v.shape
    dk, group = q.shape[-1], NH // q.shape[1]
    q, k, beta = _heads(q, group) / np.sqrt(dk), _heads(k, group), np.asarray(beta, np.float64)
    f = _f(fgate, forget)
    C = np.zeros((B, NH, dv, dk)) if C0 is None else np.asarray(C0, np.float64)
    h, states = np.empty((B, NH, T, dv)), [C]
    for t in range(T):
        C = f[:, :, t, None, None] * C
        miss = v[:, :, t] - (C @ k[:, :, t, :, None])[..., 0]
        C = C + (beta[:, :, t, None] * miss)[..., None] * k[:, :, t, None, :]
        h[:, :, t] = (C @ q[:, :, t, :, None])[..., 0]
        if all_states:
            states.append(C)
    return h, states if all_states else C


def delta_backward(q, k, v, beta, fgate, dh, C0=None, dC=None, forget="sigmoid", sizes=False):
    """-> (dq, dk, dv, dbeta, dfgate, dC0), and with ``sizes`` the roots of the
    sums of squares of the terms that each dbeta and dfgate adds up."""
    _, states = delta_forward(q, k, v, beta, fgate, C0, forget, all_states=True)
    v, dh = np.asarray(v, np.float64), np.asarray(dh, np.float64)
    B, NH, T, dv_ = v.shape
    dk_, NHK = q.shape[-1], q.shape[1]
    group, scale = NH // NHK, 1.0 / np.sqrt(q.shape[-1])
    q, k, beta = _heads(q, group), _heads(k, group), np.asarray(beta, np.float64)
    f = _f(fgate, forget)
    g = np.zeros_like(states[0]) if dC is None else np.asarray(dC, np.float64).copy()
    dq, dk, dv = np.empty_like(q), np.empty_like(k), np.empty_like(v)
    db, df, db_size, df_size = (np.empty_like(f) for _ in range(4))
    for t in reversed(range(T)):
        kt, bt = k[:, :, t], beta[:, :, t, None]
        faded = f[:, :, t, None, None] * states[t]
        miss = v[:, :, t] - (faded @ kt[..., None])[..., 0]
        dq[:, :, t] = scale * (dh[:, :, t, None, :] @ states[t + 1])[..., 0, :]
        g = g + dh[:, :, t, :, None] * (scale * q[:, :, t, None, :])
        du = (g @ kt[..., None])[..., 0]
        dv[:, :, t] = bt * du
        db[:, :, t] = (du * miss).sum(-1)
        db_size[:, :, t] = np.sqrt((((g * kt[..., None, :]) * miss[..., None]) ** 2).sum((-1, -2)))
        dk[:, :, t] = ((bt * miss)[..., None, :] @ g - dv[:, :, t, None, :] @ faded)[..., 0, :]
        g = g - dv[:, :, t, :, None] * kt[..., None, :]  # through what the memory predicted
        df[:, :, t] = (g * states[t]).sum((-1, -2))
        df_size[:, :, t] = np.sqrt(((g * states[t]) ** 2).sum((-1, -2)))
        g = f[:, :, t, None, None] * g
    slope = f if forget == "exp" else f * _f(-np.asarray(fgate, np.float64), "sigmoid")
    shared = (B, NHK, group, T, dk_)
    out = (dq.reshape(shared).sum(2), dk.reshape(shared).sum(2), dv, db, df * slope, g)
    return (*out, db_size, df_size * slope) if sizes else out


def _norm(x, layer, eps):
    x = x - x.mean(-1, keepdims=True) if layer else x
    inv = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x * inv, inv


def _norm_grad(g, n, inv, layer):
    g = g - n * (g * n).mean(-1, keepdims=True) - (g.mean(-1, keepdims=True) if layer else 0.0)
    return inv * g


def _gate(g, activation):
    s = _f(g, "sigmoid")
    if activation == "sigmoid":
        return s, s * _f(-g, "sigmoid")
    return g * s, s * (1.0 + g * _f(-g, "sigmoid"))


def block_norm(p, weight, gate=None, residual=None, scale=None, next_weight=None, norm="layer",
               activation="sigmoid", eps=1e-5, dr=None, dy=None, grads=False):
    """-> (r, y), or the dict of gradients given dr, dy with ``grads``."""
    as64 = [None if x is None else np.asarray(x, np.float64)
            for x in (p, weight, gate, residual, scale, next_weight, dr, dy)]
    p, w, gate, x, s, w2, dr, dy = as64
    B, NH, T, d = p.shape
    D, layer = NH * d, norm == "layer"

    def rows(a):
        return a.transpose(0, 2, 1, 3).reshape(B, T, D)

    def heads(a):
        return a.reshape(B, T, NH, d).transpose(0, 2, 1, 3)

    n1, inv1 = _norm(p, layer, eps)
    act, slope = _gate(gate, activation) if gate is not None else (np.ones_like(p), None)
    z = rows(act * n1) * w
    r = z if s is None else s * z
    r = r if x is None else x + r
    n2, inv2 = _norm(r, layer, eps)
    if not grads:
        return r, None if w2 is None else w2 * n2
    out = {}
    g = np.zeros_like(r) if dr is None else dr
    if w2 is not None:
        out["dnext_weight"] = (dy * n2).sum((0, 1))
        g = g + _norm_grad(dy * w2, n2, inv2, layer)
    if x is not None:
        out["dresidual"] = g
    if s is not None:
        out["dscale"] = (g * z).sum((0, 1))
    dz = g if s is None else g * s
    out["dweight"] = (dz * rows(act * n1)).sum((0, 1))
    dz = heads(dz * w)
    if gate is not None:
        out["dgate"] = dz * n1 * slope
    out["dp"] = _norm_grad(dz * act, n1, inv1, layer)
    return out
