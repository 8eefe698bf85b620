"""Timed cases of the short causal convolution, the selective scan and the gated
feed-forward.

Calls of ``linear_recurrent_sequence_amd.mlstm``: ``short_conv_fwd``, ``_bwd``
and ``_step``, ``scan_fwd``, ``_bwd`` and ``_step``, ``gated_ffn_fwd`` and
``_bwd``.

Short convolution, per channel, over W inputs (the W - 1 before the first one are
the state, zeros if there is none):

    y_t = act(b + sum_j w_j x_{t - W + 1 + j})

Selective scan, per channel c with N states, Delta = softplus(dt + bias):

    s_t = exp(Delta_t A_c) s_{t-1} + Delta_t u_t B_t
    y_t = (C_t . s_t + D_c u_t) silu(z_t)

Gated feed-forward, per row: h = act(x Wg^T) * (x Wu^T).

With ``own`` false every case runs in elementary torch operations in 32 bits.
"""
import math

import torch

own = False

BF16, FP32 = "bf16", "fp32"
TYPES = {BF16: torch.bfloat16, FP32: torch.float32}
CHUNK = 64


def _conv(name, op, B, T, NH, d, W, dtype, ragged=False):
    return dict(name=name, op=op, B=B, T=T, NH=NH, d=d, W=W, dtype=dtype, ragged=ragged)


def _scan(name, op, B, T, C, N, G, dtype, ragged=False, gate=True):
    return dict(name=name, op=op, B=B, T=T, C=C, N=N, G=G, dtype=dtype, ragged=ragged, gate=gate)


def _ffn(name, op, M, D, F, dtype, act="silu"):
    return dict(name=name, op=op, M=M, D=D, F=F, dtype=dtype, act=act)


def listed():
    return [
        # one sequence generating through a 125M-shaped layer's convolution: latency
        _conv("conv step 1x4x384", "conv_step", 1, 1, 4, 384, 4, BF16),
        # a training step of the convolution before that layer's 4 heads of 384
        _conv("conv train 8x2048 4x384", "conv_train", 8, 2048, 4, 384, 4, BF16),
        # float32, width 3, sequences of unlike lengths
        _conv("conv train fp32 3x777 5x96", "conv_train", 3, 777, 5, 96, 3, FP32, True),
        # 64 sequences generating through 2048 channels: the state's traffic
        _scan("scan step 64x2048 N16", "scan_step", 64, 1, 2048, 16, 1, BF16),
        # prompts of a batch, as wide as the 125M-shaped layer
        _scan("scan 8x2048 1536 N16", "scan", 8, 2048, 1536, 16, 1, BF16),
        # one long prompt: few channels to fill the card
        _scan("scan 1x16384 2048 N16", "scan", 1, 16384, 2048, 16, 1, BF16),
        # the training step of the batch
        _scan("scan train 8x2048 1536 N16", "scan_train", 8, 2048, 1536, 16, 1, BF16),
        # float32, odd sizes, two groups, sequences of unlike lengths
        _scan("scan train fp32 2x555 208 N20", "scan_train", 2, 555, 208, 20, 2, FP32, True),
        # eight sequences generating: the weights' traffic
        _ffn("ffn 8 rows 1536 4096", "ffn", 8, 1536, 4096, BF16),
        # prompts of a batch through the 125M-shaped layer's block
        _ffn("ffn 16384 rows 1536 4096", "ffn", 16384, 1536, 4096, BF16),
        # a training step of a 1.3B-shaped block
        _ffn("ffn train 8192 rows 2048 5504", "ffn_train", 8192, 2048, 5504, BF16),
        # float32, odd sizes
        _ffn("ffn train fp32 999 rows 392 1048", "ffn_train", 999, 392, 1048, FP32, "gelu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv_step", "conv_train", "conv_train", "scan_step", "scan", "scan",
                     "scan_train", "scan_train", "ffn", "ffn", "ffn_train", "ffn_train"])
    dtype = rng.choice([BF16, BF16, FP32])
    if op.startswith("ffn"):
        D, F = 8 * _log(rng, 16, 320), 8 * _log(rng, 32, 700)
        # at most 16384 rows, and no more work than the listed training step
        M = _log(rng, 1, min(16384, (2 if dtype == FP32 else 8) * 10 ** 10 // (D * F)))
        return dict(op=op, M=M, D=D, F=F, dtype=dtype, act=rng.choice(["silu", "gelu"]))
    ragged = rng.random() < 0.4
    if op.startswith("conv"):
        NH, d, W = rng.choice([1, 2, 3, 4, 8]), 8 * rng.randint(4, 64), rng.randint(2, 8)
        rows = _log(rng, 1, min(16384, 24 * 1024 * 1024 // (NH * d)))
        B = min(rows, rng.choice([1, 2, 3, 8]))
        if op == "conv_step":
            return dict(op=op, B=min(rows, 512), T=1, NH=NH, d=d, W=W, dtype=dtype, ragged=False)
        return dict(op=op, B=B, T=rows // B, NH=NH, d=d, W=W, dtype=dtype, ragged=ragged)
    G, N = rng.choice([1, 1, 2, 3]), rng.choice([1, 4, 8, 11, 16, 16, 16, 24, 32, 64])
    C = 8 * G * _log(rng, 4, 256 // G)
    gate = rng.random() < 0.7
    if op == "scan_step":
        return dict(op=op, B=_log(rng, 1, min(256, 4 * 1024 * 1024 // (C * N))), T=1, C=C, N=N,
                    G=G, dtype=dtype, ragged=False, gate=gate)
    # no more states than the listed cases
    rows = _log(rng, 1, min(16384, 384 * 1024 * 1024 // (C * N)))
    B = min(rows, rng.choice([1, 2, 3, 8]))
    return dict(op=op, B=B, T=rows // B, C=C, N=N, G=G, dtype=dtype, ragged=ragged, gate=gate)


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device=dev).to(dtype)

    s = dict(case=dict(case))
    op = case["op"]
    if op.startswith("ffn"):
        M, D, F = case["M"], case["D"], case["F"]
        # a block norm's output, weights that keep its size
        s["x"] = normal(M, D, dtype=dt)
        s["w_gate"] = (normal(F, D) * D ** -0.5).to(dt)
        s["w_up"] = (normal(F, D) * D ** -0.5).to(dt)
        if op == "ffn_train":
            s["dh"] = normal(M, F, dtype=dt)
        return s
    B, T = case["B"], case["T"]
    s["lengths"] = None
    if case["ragged"]:
        n = torch.randint(0, T + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
        n[0] = T
        s["lengths"] = n
    if op.startswith("conv"):
        NH, d, W = case["NH"], case["d"], case["W"]
        C = NH * d
        s["x"] = normal(B, T, C, dtype=dt)
        s["weight"], s["bias"] = normal(C, W) * W ** -0.5, 0.1 * normal(C)
        s["state"] = normal(B, W - 1, C, dtype=dt)
        if op == "conv_step":
            s["x"] = s["x"][:, 0].contiguous()
            s["out_state"] = torch.empty_like(s["state"])
        else:
            s["dy"] = normal(B, NH, T, d, dtype=dt)
            s["dstate"] = normal(B, W - 1, C, dtype=dt)
        return s
    C, N, G = case["C"], case["N"], case["G"]
    s["u"] = normal(B, T, C, dtype=dt)
    s["dt"] = (0.5 * normal(B, T, C)).to(dt)
    # steps from 0.001 to 0.1 as layers are initialised, rates -1 .. -N
    step = torch.exp(torch.rand(C, generator=gen, device=dev) * math.log(100.0) - math.log(1000.0))
    s["dt_bias"] = torch.log(torch.expm1(step))
    s["A"] = -(torch.arange(1, N + 1, device=dev).float() * (1.0 + 0.1 * torch.rand(
        (C, N), generator=gen, device=dev)))
    s["B"], s["C"] = normal(B, T, G, N, dtype=dt), normal(B, T, G, N, dtype=dt)
    s["D"] = 1.0 + 0.1 * normal(C)
    s["gate"] = normal(B, T, C, dtype=dt) if case["gate"] else None
    s["state"] = 0.1 * normal(B, C, N)
    if op == "scan_step":
        for n in ("u", "dt", "B", "C", "gate"):
            s[n] = s[n][:, 0].contiguous() if s[n] is not None else None
        s["out_state"] = torch.empty_like(s["state"])
    if op == "scan_train":
        s["dy"], s["dstate"] = normal(B, T, C, dtype=dt), normal(B, C, N)
    return s


def run(state):
    op = state["case"]["op"]
    kind = op.split("_")[0]
    if own:
        return {"conv": _conv_own, "scan": _scan_own, "ffn": _ffn_own}[kind](state, op)
    return {"conv": _conv_plain, "scan": _scan_plain, "ffn": _ffn_plain}[kind](state, op)


# ---- the framework's calls


def _conv_own(s, op):
    from linear_recurrent_sequence_amd import mlstm

    NH = s["case"]["NH"]
    if op == "conv_step":
        y, st = mlstm.short_conv_step(s["x"], s["weight"], s["state"], bias=s["bias"], heads=NH,
                                      out_state=s["out_state"])
        return {"y": y, "state": st}
    kw = dict(bias=s["bias"], state=s["state"], lengths=s["lengths"], heads=NH)
    y, st = mlstm.short_conv_fwd(s["x"], s["weight"], **kw)
    return {"y": y, "state": st,
            **mlstm.short_conv_bwd(s["x"], s["weight"], s["dy"], dstate=s["dstate"], **kw)}


def _scan_own(s, op):
    from linear_recurrent_sequence_amd import mlstm

    args = [s[n] for n in ("u", "dt", "A", "B", "C")]
    kw = dict(D=s["D"], gate=s["gate"], dt_bias=s["dt_bias"])
    if op == "scan_step":
        y, st = mlstm.scan_step(*args, s["state"], out_state=s["out_state"], **kw)
        return {"y": y, "state": st}
    kw.update(state=s["state"], lengths=s["lengths"])
    y, st = mlstm.scan_fwd(*args, **kw)
    out = {"y": y, "state": st}
    if op == "scan_train":
        out.update(mlstm.scan_bwd(*args, s["dy"], dstate=s["dstate"], **kw))
    return out


def _ffn_own(s, op):
    from linear_recurrent_sequence_amd import mlstm

    x, wg, wu, act = s["x"], s["w_gate"], s["w_up"], s["case"]["act"]
    h = mlstm.gated_ffn_fwd(x, wg, wu, activation=act)
    if op == "ffn":
        return {"h": h}
    dx, dwg, dwu = mlstm.gated_ffn_bwd(x, wg, wu, s["dh"], activation=act)
    return {"h": h, "dx": dx, "dw_gate": dwg, "dw_up": dwu}


# ---- the plain forms


def _grads(outs, grads, named, kinds):
    """Gradients by name, rounded once to the type of their input."""
    g = torch.autograd.grad(outs, list(named.values()), grads)
    return {"d" + n: x.to(kinds[n].dtype) for n, x in zip(named, g)}


def _leaves(s, names, train):
    t = {n: s[n].detach().float() for n in names if s[n] is not None}
    return {n: x.requires_grad_() for n, x in t.items()} if train else t


def _inside(s):
    """[B, T] truth values: positions before each sequence's length."""
    at = torch.arange(s["case"]["T"], device=s["lengths"].device)
    return at < s["lengths"][:, None]


def _conv_plain(s, op):
    c, dt = s["case"], TYPES[s["case"]["dtype"]]
    NH, W, T = c["NH"], c["W"], c["T"]
    t = _leaves(s, ("x", "weight", "bias", "state"), op == "conv_train")
    x = t["x"].unsqueeze(1) if op == "conv_step" else t["x"]
    if s["lengths"] is not None:
        x = x * _inside(s)[..., None]
    x = torch.cat([t["state"], x], 1)
    y = t["bias"] + sum(x[:, j:j + T] * t["weight"][:, j] for j in range(W))
    y = y * torch.sigmoid(y)
    if s["lengths"] is None:
        st = x[:, T:]
    else:
        y = y * _inside(s)[..., None]
        at = s["lengths"].long()[:, None] + torch.arange(W - 1, device=x.device)
        st = x[torch.arange(x.shape[0], device=x.device)[:, None], at]
    y = y.unflatten(2, (NH, -1)).transpose(1, 2)
    out = {"y": (y.squeeze(2) if op == "conv_step" else y).detach().to(dt).contiguous(),
           "state": st.detach().to(dt).contiguous()}
    if op == "conv_train":
        out.update(_grads((y, st), (s["dy"].float(), s["dstate"].float()), t, s))
    return out


def _softplus(x):
    return x.clamp(min=0.0) + torch.log1p(torch.exp(-x.abs()))


def _scan_chunks(t, lengths):
    """All chunks side by side from zeros, their ends joined, and what the memory
    before a chunk adds: (y before the gate, the last state)."""
    u, Bm, Cm, A = t["u"], t["B"], t["C"], t["A"]
    B, T, C = u.shape
    N, G = A.shape[1], Bm.shape[2]
    size = min(CHUNK, T)
    delta = _softplus(t["dt"] + t["dt_bias"])
    if lengths is not None:
        delta = delta * (torch.arange(T, device=u.device) < lengths[:, None])[..., None]

    def chunks(x):
        pad = -T % size
        if pad:
            x = torch.cat([x, torch.zeros_like(x[:, :1]).expand(B, pad, *x.shape[2:])], 1)
        return x.unflatten(1, (-1, size))

    v = chunks(delta * u)
    delta, Bm, Cm = chunks(delta), chunks(Bm), chunks(Cm)
    a = torch.exp(delta[..., None] * A)
    grouped = (*v.shape[:3], G, C // G, N)
    b = (v.unflatten(-1, (G, -1))[..., None] * Bm[..., None, :]).reshape(a.shape)
    local = [torch.zeros_like(a[:, :, 0])]
    for ai, bi in zip(a.unbind(2), b.unbind(2)):
        local.append(ai * local[-1] + bi)
    local = torch.stack(local[1:], 2)
    kept = torch.exp(delta.cumsum(2)[..., None] * A)
    starts = [t["state"]]
    for p, e in zip(kept[:, :, -1].unbind(1), local[:, :, -1].unbind(1)):
        starts.append(p * starts[-1] + e)
    s = local + kept * torch.stack(starts[:-1], 1).unsqueeze(2)
    y = (s.view(grouped) * Cm[..., None, :]).sum(-1).flatten(-2)
    return y.flatten(1, 2)[:, :T], starts[-1]


def _scan_plain(s, op):
    c, dt = s["case"], TYPES[s["case"]["dtype"]]
    t = _leaves(s, ("u", "dt", "A", "B", "C", "D", "gate", "dt_bias", "state"),
                op == "scan_train")
    if op == "scan_step":
        t = {n: x.unsqueeze(1) if n in ("u", "dt", "B", "C", "gate") else x for n, x in t.items()}
    y, st = _scan_chunks(t, s["lengths"])
    y = y + t["D"] * t["u"]
    if c["gate"]:
        y = y * (t["gate"] * torch.sigmoid(t["gate"]))
    if s["lengths"] is not None:
        y = y * _inside(s)[..., None]
    out = {"y": (y.squeeze(1) if op == "scan_step" else y).detach().to(dt),
           "state": st.detach().contiguous()}
    if op == "scan_train":
        out.update(_grads((y, st), (s["dy"].float(), s["dstate"]), t, s))
    return out


def _ffn_plain(s, op):
    dt = TYPES[s["case"]["dtype"]]
    t = _leaves(s, ("x", "w_gate", "w_up"), op == "ffn_train")
    g, u = t["x"] @ t["w_gate"].T, t["x"] @ t["w_up"].T
    if s["case"]["act"] == "silu":
        h = g * torch.sigmoid(g) * u
    else:
        h = 0.5 * g * (1.0 + torch.erf(g * math.sqrt(0.5))) * u
    out = {"h": h.detach().to(dt)}
    if op == "ffn_train":
        out.update(_grads((h,), (s["dh"].float(),), t, s))
    return out


# ---- the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["op"].split("_")[0]
    return {"conv": _conv_exact, "scan": _scan_exact, "ffn": _ffn_exact}[kind](s, case)


def _lengths(s, case):
    return [case["T"]] * case["B"] if s["lengths"] is None else s["lengths"].tolist()


def _conv_exact(s, case):
    """Sequence by sequence; the gradients tap by tap."""
    NH, d, W, T, B = (case[n] for n in ("NH", "d", "W", "T", "B"))
    w, bias = s["weight"].double(), s["bias"].double()
    x = s["x"].double().view(B, T, NH * d)
    y = torch.zeros_like(x)
    st = torch.empty_like(s["state"].double())
    train = case["op"] == "conv_train"
    if train:
        dy = s["dy"].double().transpose(1, 2).reshape(B, T, NH * d)
        dx, dst = torch.zeros_like(x), torch.zeros_like(st)
        dw, db = torch.zeros_like(w), torch.zeros_like(bias)
    for b, n in enumerate(_lengths(s, case)):
        z = torch.cat([s["state"][b].double(), x[b, :n]])
        pre = bias.expand(n, -1).clone()
        for j in range(W):
            pre += w[:, j] * z[j:j + n]
        sig = 1.0 / (1.0 + torch.exp(-pre))
        y[b, :n] = pre * sig
        st[b] = z[n:]
        if train:
            g = dy[b, :n] * sig * (1.0 + pre * (1.0 - sig))
            dz = torch.zeros_like(z)
            dz[n:] += s["dstate"][b].double()
            for j in range(W):
                dz[j:j + n] += w[:, j] * g
                dw[:, j] += (g * z[j:j + n]).sum(0)
            db += g.sum(0)
            dst[b], dx[b, :n] = dz[:W - 1], dz[W - 1:]
    y = y.view(B, T, NH, d).transpose(1, 2)
    out = {"y": y[:, :, 0] if case["op"] == "conv_step" else y, "state": st}
    if train:
        out.update(dx=dx, dweight=dw, dbias=db, dstate=dst)
    return out


def _scan_exact(s, case):
    """Token by token, and the reversed recurrence of the gradients."""
    T, C, N, G, Bn = (case[n] for n in ("T", "C", "N", "G", "B"))
    rows = {n: s[n].double().reshape(Bn, T, *s[n].shape[-k:])
            for n, k in (("u", 1), ("dt", 1), ("B", 2), ("C", 2))}
    u, x = rows["u"], rows["dt"] + s["dt_bias"].double()
    A, D = s["A"].double(), s["D"].double()
    live = torch.ones(Bn, T, 1, dtype=torch.float64, device=u.device)
    for b, n in enumerate(_lengths(s, case)):
        live[b, n:] = 0.0
    delta = torch.logaddexp(x, torch.zeros_like(x)) * live

    def wide(m, t):  # [B, C, N] of a group's [B, G, N]
        return m[:, t].repeat_interleave(C // G, 1)

    S = s["state"].double()
    kept, raw = [S], torch.empty_like(u)
    train = case["op"] == "scan_train"
    for t in range(T):
        S = torch.exp(delta[:, t, :, None] * A) * S \
            + (delta[:, t] * u[:, t])[..., None] * wide(rows["B"], t)
        raw[:, t] = (S * wide(rows["C"], t)).sum(-1)
        if train:
            kept.append(S)
    raw += D * u
    act = torch.ones_like(u)
    if s["gate"] is not None:
        z = s["gate"].double().view(Bn, T, C)
        sz = 1.0 / (1.0 + torch.exp(-z))
        act = z * sz
    y = raw * act * live
    out = {"y": y[:, 0] if case["op"] == "scan_step" else y, "state": S}
    if not train:
        return out
    dy = s["dy"].double() * live
    g = dy * act
    du, dd = g * D, torch.zeros_like(u)
    dA = torch.zeros_like(A)
    dB, dC = torch.zeros_like(rows["B"]), torch.zeros_like(rows["C"])
    dS = s["dstate"].double()
    for t in range(T - 1, -1, -1):
        dl, ut, Bt = delta[:, t, :, None], u[:, t, :, None], wide(rows["B"], t)
        gt = g[:, t, :, None]
        dC[:, t] = (gt * kept[t + 1]).unflatten(1, (G, -1)).sum(2)
        dS = dS + gt * wide(rows["C"], t)
        a = torch.exp(dl * A)
        flow = dS * a * kept[t]
        dA += (flow * dl).sum(0)
        dd[:, t] = (flow * A + dS * ut * Bt).sum(-1)
        du[:, t] += (dS * Bt * dl).sum(-1)
        dB[:, t] = (dS * dl * ut).unflatten(1, (G, -1)).sum(2)
        dS = dS * a
    ddt = dd * live / (1.0 + torch.exp(-x))
    out.update(du=du, ddt=ddt, dA=dA, dB=dB, dC=dC, dD=(g * u).sum((0, 1)))
    if s["gate"] is not None:
        out["dgate"] = dy * raw * sz * (1.0 + z * (1.0 - sz))
    out.update(ddt_bias=ddt.sum((0, 1)), dstate=dS)
    return out


def _ffn_exact(s, case):
    x, wg, wu = (s[n].double() for n in ("x", "w_gate", "w_up"))
    g, u = torch.matmul(x, wg.t()), torch.matmul(x, wu.t())
    if case["act"] == "silu":
        p = 1.0 / (1.0 + torch.exp(-g))
        act, slope = g * p, p * (1.0 + g * (1.0 - p))
    else:
        p = 0.5 * torch.erfc(-g / math.sqrt(2.0))
        act, slope = g * p, p + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    out = {"h": act * u}
    if case["op"] == "ffn_train":
        dh = s["dh"].double()
        dg, du = dh * u * slope, dh * act
        out.update(dx=torch.matmul(dg, wg) + torch.matmul(du, wu),
                   dw_gate=torch.matmul(dg.t(), x), dw_up=torch.matmul(du.t(), x))
    return out


def work(case):
    size, op = 2 if case["dtype"] == BF16 else 4, case["op"]
    if op.startswith("ffn"):
        M, D, F = case["M"], case["D"], case["F"]
        if op == "ffn":
            return {"bytes": (M * (D + F) + 2 * F * D) * size, "flops": 4 * M * D * F}
        # x, dh and the weights in, h, dx and the weights' gradients out; two products
        # forward, four backward
        return {"bytes": (2 * M * (D + F) + 4 * F * D) * size, "flops": 12 * M * D * F}
    B, T = case["B"], case["T"]
    if op.startswith("conv"):
        C, W = case["NH"] * case["d"], case["W"]
        rows, state, weights = B * T * C, 2 * B * (W - 1) * C, C * (W + 1) * 4
        if op == "conv_step":
            return {"bytes": (2 * rows + state) * size + weights, "flops": (2 * W + 6) * rows}
        return {"bytes": (4 * rows + 2 * state) * size + 2 * weights,
                "flops": (8 * W + 20) * rows}
    C, N, G = case["C"], case["N"], case["G"]
    rows, bc, state = B * T * C, 2 * B * T * G * N, 2 * B * C * N * 4
    n = 3 + (1 if case["gate"] else 0)
    weights = (C * N + 2 * C) * 4
    if op == "scan_train":
        # u, dt, z, dy in, y, du, ddt, dz out
        return {"bytes": (2 * n * rows + 2 * bc) * size + 2 * state + 2 * weights,
                "flops": 20 * rows * N + 60 * rows}
    return {"bytes": (n * rows + bc) * size + state + weights, "flops": 6 * rows * N + 20 * rows}
