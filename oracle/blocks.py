"""The short causal convolution, the selective scan and the gated feed-forward in
float64, from their definitions, token by token.  Gradients also return, on
request, the size of each sum's terms (the root of the sum of their squares), to
which a float32 sum's error is relative.
"""
import numpy as np
from scipy.special import erf


def _lengths(lengths, B, T):
    return [T] * B if lengths is None else [min(max(int(n), 0), T) for n in lengths]


def _sigmoid(x):
    return 0.5 * (1.0 + np.tanh(0.5 * x))


def _silu(x):
    s = _sigmoid(x)
    return x * s, s * (1.0 + x * (1.0 - s))


def _heads(rows, heads):
    """[B, T, C] -> [B, heads, T, C / heads]"""
    B, T, C = rows.shape
    return rows.reshape(B, T, heads, C // heads).transpose(0, 2, 1, 3)


def short_conv(x, weight, bias=None, state=None, lengths=None, activation="silu"):
    """x [B, T, C], weight [C, W] -> (y [B, T, C], state [B, W - 1, C])."""
    B, T, C = x.shape
    W = weight.shape[1]
    y, out = np.zeros_like(x), np.zeros((B, W - 1, C))
    for b, n in enumerate(_lengths(lengths, B, T)):
        before = np.zeros((W - 1, C)) if state is None else state[b]
        z = np.concatenate([before, x[b, :n]])
        for t in range(n):
            a = (weight * z[t:t + W].T).sum(1) + (0.0 if bias is None else bias)
            y[b, t] = _silu(a)[0] if activation == "silu" else a
        out[b] = z[n:]
    return y, out


def short_conv_grads(x, weight, dy, bias=None, state=None, dstate=None, lengths=None,
                     activation="silu"):
    """dy [B, T, C] -> (dx, dweight, dbias, dstate, sizes of dweight's and dbias's terms)."""
    B, T, C = x.shape
    W = weight.shape[1]
    dx, dw, db = np.zeros_like(x), np.zeros_like(weight), np.zeros(C)
    ds = np.zeros((B, W - 1, C))
    w_size, b_size = np.zeros_like(weight), np.zeros(C)
    for b, n in enumerate(_lengths(lengths, B, T)):
        before = np.zeros((W - 1, C)) if state is None else state[b]
        z = np.concatenate([before, x[b, :n]])
        dz = np.zeros_like(z)
        if dstate is not None:
            dz[n:] += dstate[b]
        for t in range(n):
            a = (weight * z[t:t + W].T).sum(1) + (0.0 if bias is None else bias)
            g = dy[b, t] * (_silu(a)[1] if activation == "silu" else 1.0)
            db += g
            b_size += g ** 2
            dw += g[:, None] * z[t:t + W].T
            w_size += (g[:, None] * z[t:t + W].T) ** 2
            dz[t:t + W] += (weight * g[:, None]).T
        ds[b], dx[b, :n] = dz[:W - 1], dz[W - 1:]
    return dx, dw, db, ds, np.sqrt(w_size), np.sqrt(b_size)


def selective_scan(u, dt, A, B, C, D=None, gate=None, dt_bias=None, state=None, lengths=None,
                   keep=False):
    """u, dt, gate [n, T, c], A [c, N], B, C [n, T, G, N] -> (y, state [n, c, N]);
    with ``keep`` also what the gradients need."""
    n, T, c = u.shape
    N, rep = A.shape[1], c // B.shape[2]
    x = dt + (0.0 if dt_bias is None else dt_bias)
    delta = np.logaddexp(x, 0.0)
    y = np.zeros_like(u)
    s = np.zeros((n, c, N)) if state is None else state.copy()
    kept, raw = np.zeros((T + 1, n, c, N)) if keep else None, np.zeros_like(u)
    live = np.zeros((n, T, 1))
    for b, m in enumerate(_lengths(lengths, n, T)):
        live[b, :m] = 1.0
    if keep:
        kept[0] = s
    for t in range(T):
        on = live[:, t, :, None] > 0
        Bt, Ct = (m[:, t].repeat(rep, 1) for m in (B, C))
        new = np.exp(delta[:, t, :, None] * A) * s + (delta[:, t] * u[:, t])[..., None] * Bt
        s = np.where(on, new, s)
        raw[:, t] = np.where(on[..., 0], (Ct * s).sum(-1)
                             + (0.0 if D is None else D * u[:, t]), 0.0)
        if keep:
            kept[t + 1] = s
    y = raw if gate is None else np.where(live > 0, raw * _silu(gate)[0], 0.0)
    return (y, s, kept, raw, delta, x, live) if keep else (y, s)


def selective_scan_grads(u, dt, A, B, C, dy, D=None, gate=None, dt_bias=None, state=None,
                         dstate=None, lengths=None):
    """A dict of gradients by name, and a dict of the sizes of the sums' terms (for
    dA, dB, dC, dD and ddt_bias)."""
    n, T, c = u.shape
    N, G = A.shape[1], B.shape[2]
    rep = c // G
    _, _, kept, raw, delta, x, live = selective_scan(u, dt, A, B, C, D, gate, dt_bias, state,
                                                     lengths, keep=True)
    dy = np.where(live > 0, dy, 0.0)
    act, slope = (np.ones_like(u), None) if gate is None else _silu(gate)
    g = np.where(live > 0, dy * act, 0.0)
    Dv = 0.0 if D is None else D
    out = {"du": g * Dv, "ddt": np.zeros_like(u), "dA": np.zeros_like(A),
           "dB": np.zeros_like(B), "dC": np.zeros_like(C)}
    size = {k: np.zeros_like(out[k]) for k in ("dA", "dB", "dC")}
    S = np.zeros((n, c, N)) if dstate is None else dstate.copy()

    def groups(v):
        return v.reshape(n, G, rep, N).sum(2)

    for t in range(T - 1, -1, -1):
        on = live[:, t, :, None] > 0
        Bt, Ct = (np.where(on, m[:, t].repeat(rep, 1), 0.0) for m in (B, C))
        dl = np.where(on, delta[:, t, :, None], 0.0)
        ut, gt = np.where(on, u[:, t, :, None], 0.0), g[:, t, :, None]
        out["dC"][:, t] = groups(gt * np.where(on, kept[t + 1], 0.0))
        size["dC"][:, t] = np.sqrt(groups((gt * kept[t + 1]) ** 2))
        S = S + gt * Ct
        a = np.where(on, np.exp(dl * A), 1.0)
        flow = np.where(on, S * a * kept[t], 0.0)
        out["dA"] += (flow * dl).sum(0)
        size["dA"] += ((flow * dl) ** 2).sum(0)
        out["ddt"][:, t] = (flow * A + np.where(on, S * ut * Bt, 0.0)).sum(-1)
        out["du"][:, t] += (S * Bt * dl).sum(-1)
        out["dB"][:, t] = groups(S * dl * ut)
        size["dB"][:, t] = np.sqrt(groups((S * dl * ut) ** 2))
        S = S * a
    with np.errstate(invalid="ignore"):
        out["ddt"] = np.where(live > 0, out["ddt"] * _sigmoid(x), 0.0)
    size["dA"] = np.sqrt(size["dA"])
    if D is not None:
        gu = np.where(live > 0, g * u, 0.0)
        out["dD"], size["dD"] = gu.sum((0, 1)), np.sqrt((gu ** 2).sum((0, 1)))
    if gate is not None:
        out["dgate"] = np.where(live > 0, dy * raw * slope, 0.0)
    if dt_bias is not None:
        out["ddt_bias"] = out["ddt"].sum((0, 1))
        size["ddt_bias"] = np.sqrt((out["ddt"] ** 2).sum((0, 1)))
    out["dstate"] = S
    return out, size


def _ffn_activation(g, activation):
    if activation == "silu":
        return _silu(g)
    cdf = 0.5 * (1.0 + erf(g / np.sqrt(2.0)))
    return g * cdf, cdf + g * np.exp(-0.5 * g * g) / np.sqrt(2.0 * np.pi)


def gated_ffn(x, w_gate, w_up, activation="silu"):
    return _ffn_activation(x @ w_gate.T, activation)[0] * (x @ w_up.T)


def gated_ffn_grads(x, w_gate, w_up, dh, activation="silu"):
    """(dx, dw_gate, dw_up), and the sizes of their sums' terms."""
    g, u = x @ w_gate.T, x @ w_up.T
    act, slope = _ffn_activation(g, activation)
    dg, du = dh * u * slope, dh * act
    sizes = (np.sqrt(dg ** 2 @ w_gate ** 2 + du ** 2 @ w_up ** 2),
             np.sqrt((dg ** 2).T @ x ** 2), np.sqrt((du ** 2).T @ x ** 2))
    return (dg @ w_gate + du @ w_up, dg.T @ x, du.T @ x), sizes
