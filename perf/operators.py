"""Timed cases of the gated delta rule and of the block norm.

Five calls of ``linear_recurrent_sequence_amd.mlstm``: ``delta_fwd`` (a whole
sequence in chunks), ``delta_step`` (one token), ``delta_fwd`` with
``delta_bwd`` (a training step of the cell), ``block_norm_fwd`` and
``block_norm_fwd`` with ``block_norm_bwd``.

Gated delta rule, per head, with the memory C (dv x dk, rows by value),
fbar_t = log f_t, and q^_t = q_t / sqrt(dk):

    C_t = f_t C_{t-1} + beta_t (v_t - f_t C_{t-1} k_t) k_t^T
    h_t = C_t q^_t

Block norm, per token, with p in heads of d channels and D = NH d:

    z = act(g) * w1 * norm_head(p),   r = x + s * z,   y = w2 * norm_D(r)

With ``own`` false every case runs in elementary torch operations in 32 bits.
"""
import math

import torch

own = False

CHUNK = 64
BF16, FP32 = "bf16", "fp32"
TYPES = {BF16: torch.bfloat16, FP32: torch.float32}
EPS = 1e-5


def _step(name, B, NHK, NH, dk, dv, dtype):
    return dict(name=name, op="step", B=B, NHK=NHK, NH=NH, T=1, dk=dk, dv=dv, dtype=dtype,
                forget="sigmoid")


def _delta(name, op, B, NHK, NH, T, dk, dv, dtype, forget="sigmoid"):
    return dict(name=name, op=op, B=B, NHK=NHK, NH=NH, T=T, dk=dk, dv=dv, dtype=dtype,
                forget=forget)


def _norm(name, op, B, NH, T, d, dtype, norm="layer", gate="sigmoid", residual=True):
    return dict(name=name, op=op, B=B, NH=NH, T=T, d=d, dtype=dtype, norm=norm, gate=gate,
                residual=residual)


def listed():
    return [
        # one sequence generating: latency
        _step("step 1x4 d64", 1, 4, 4, 64, 64, BF16),
        # a batch of sequences generating, heads of 128: the state's traffic
        _step("step 64x16 d128", 64, 16, 16, 128, 128, BF16),
        # the small, launch-bound layer (4 x 4 heads of 64, 512 positions)
        _delta("fwd 4x4 T512 d64", "fwd", 4, 4, 4, 512, 64, 64, BF16),
        # a training-sized layer with heads of 128
        _delta("fwd 8x16 T2048 d128", "fwd", 8, 16, 16, 2048, 128, 128, BF16),
        # a long prompt: one sequence, few heads, 256 chunks in a row
        _delta("fwd 1x8 T16384 d256", "fwd", 1, 8, 8, 16384, 256, 256, BF16),
        # float32, odd sizes, two value heads to a key head, log decay given directly
        _delta("fwd fp32 2x4 T777 96/160", "fwd", 2, 2, 4, 777, 96, 160, FP32, "exp"),
        # training step of the 125M-shaped layer (8 x 4 heads of 384, 2048 positions)
        _delta("train 8x4 T2048 d384", "train", 8, 4, 4, 2048, 384, 384, BF16),
        # training step in float32, ragged, shared key heads
        _delta("train fp32 2x4 T555 64/128", "train", 2, 2, 4, 555, 64, 128, FP32),
        # the norms around the 125M-shaped layer: one token of 8 sequences, then whole sequences
        _norm("norm 8x1 4x384", "norm", 8, 4, 1, 384, BF16),
        _norm("norm 8x2048 4x384", "norm", 8, 4, 2048, 384, BF16),
        # the training step of the norms around the 1.3B-shaped layer
        _norm("norm train 4x2048 8x512", "norm_train", 4, 8, 2048, 512, BF16),
        # float32, 999 rows, root-mean-square norm with a SiLU gate and no residual
        _norm("norm train fp32 3x333 16x128", "norm_train", 3, 16, 333, 128, FP32, "rms", "silu",
              False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "fwd", "fwd", "train", "train", "norm", "norm_train"])
    dtype = rng.choice([BF16, BF16, FP32])
    if op in ("norm", "norm_train"):
        NH, d = rng.choice([1, 2, 4, 8, 16]), 16 * rng.randint(2, 32)
        rows = _log(rng, 1, min(16384, 4 * 8192 * 1024 // (NH * d)))
        B = rng.choice([1, 2, 3])
        return dict(op=op, B=B, NH=NH, T=max(1, rows // B), d=d, dtype=dtype,
                    norm=rng.choice(["layer", "rms"]), gate=rng.choice(["sigmoid", "silu"]),
                    residual=rng.random() < 0.7)
    dk, dv = 16 * rng.randint(2, 20), 16 * rng.randint(2, 20)
    NHK = rng.choice([1, 2, 4])
    NH = NHK * rng.choice([1, 1, 2, 3])
    forget = rng.choice(["sigmoid", "exp"])
    if op == "step":
        B = _log(rng, 1, max(2, 8 * 1024 * 1024 // (NH * dk * dv)))
        return dict(op=op, B=B, NHK=NHK, NH=NH, T=1, dk=dk, dv=dv, dtype=dtype, forget=forget)
    B = rng.choice([1, 2, 3, 4])
    # at most 2048 positions to a batch row, and fewer where the heads are many
    T = _log(rng, 1, min(2048, 16384 // B))
    return dict(op=op, B=B, NHK=NHK, NH=NH, T=T, dk=dk, dv=dv, dtype=dtype, forget=forget)


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device=dev).to(dtype)

    s = dict(case=dict(case))
    if case["op"] in ("norm", "norm_train"):
        B, NH, T, d = case["B"], case["NH"], case["T"], case["d"]
        D = NH * d
        # the cell's output: heads of unlike sizes, a few channels that stand out
        s["p"] = (normal(B, NH, T, d) * (0.5 + normal(1, NH, 1, 1).abs())
                  + 0.3 * normal(1, NH, 1, d)).to(dt)
        s["gate"] = normal(B, NH, T, d, dtype=dt)
        s["weight"] = 1.0 + 0.1 * normal(D)
        s["residual"] = (3.0 * normal(B, T, D)).to(dt) if case["residual"] else None
        s["scale"] = 0.5 + 0.1 * normal(D) if case["residual"] else None
        s["next_weight"] = 1.0 + 0.1 * normal(D)
        if case["op"] == "norm_train":
            s["dr"], s["dy"] = normal(B, T, D, dtype=dt), normal(B, T, D, dtype=dt)
        return s
    B, NHK, NH, T, dk, dv = (case[x] for x in ("B", "NHK", "NH", "T", "dk", "dv"))
    # unit keys with a common part, as trained layers have them; gates as their
    # projections give them: strengths in (0, 1), most of the memory kept
    k = normal(B, NHK, T, dk) + 0.5 * normal(1, NHK, 1, dk)
    s["k"] = (k / k.square().sum(-1, keepdim=True).sqrt()).to(dt)
    s["q"], s["v"] = normal(B, NHK, T, dk, dtype=dt), normal(B, NH, T, dv, dtype=dt)
    s["beta"] = torch.sigmoid(normal(B, NH, T))
    f = 4.0 + 1.5 * normal(B, NH, T)
    s["fgate"] = f if case["forget"] == "sigmoid" else -torch.log1p(torch.exp(-f))
    s["state"] = normal(B, NH, dv, dk)
    if case["op"] == "step":
        s = {n: x.squeeze(2) if n in ("q", "k", "v", "beta", "fgate") else x
             for n, x in s.items()}
        s["out_state"] = torch.empty_like(s["state"])
    if case["op"] == "train":
        s["dh"], s["dstate"] = normal(B, NH, T, dv, dtype=dt), normal(B, NH, dv, dk)
    return s


def run(state):
    op = state["case"]["op"]
    if op in ("norm", "norm_train"):
        return _norm_own(state, op) if own else _norm_plain(state, op)
    return _delta_own(state, op) if own else _delta_plain(state, op)


# ---- the framework's calls


def _delta_own(s, op):
    from linear_recurrent_sequence_amd import mlstm

    args, forget = [s[n] for n in ("q", "k", "v", "beta", "fgate")], s["case"]["forget"]
    if op == "step":
        h, C = mlstm.delta_step(*args, s["state"], out_state=s["out_state"], forget=forget)
        return {"h": h, "state": C}
    h, C = mlstm.delta_fwd(*args, state=s["state"], forget=forget)
    if op == "fwd":
        return {"h": h, "state": C}
    dq, dk, dv, dbeta, dfgate, dC = mlstm.delta_bwd(*args, s["dh"], state=s["state"],
                                                    dstate=s["dstate"], forget=forget)
    return {"h": h, "state": C, "dq": dq, "dk": dk, "dv": dv, "dbeta": dbeta, "dfgate": dfgate,
            "dstate": dC}


def _norm_own(s, op):
    from linear_recurrent_sequence_amd import mlstm

    c = s["case"]
    kw = dict(gate=s["gate"], residual=s["residual"], scale=s["scale"],
              next_weight=s["next_weight"], norm=c["norm"], activation=c["gate"], eps=EPS)
    r, y = mlstm.block_norm_fwd(s["p"], s["weight"], **kw)
    out = {"r": r, "y": y}
    if op == "norm_train":
        out.update(mlstm.block_norm_bwd(s["p"], s["weight"], s["dr"], s["dy"], **kw))
    return out


# ---- the plain forms


def _log_forget(fgate, forget):
    f = fgate.double()
    if forget == "sigmoid":
        return f.clamp(max=0.0) - torch.log1p(torch.exp(-f.abs()))
    return f


def _unit_lower_inverse(A):
    """(I + A)^-1 for strictly lower triangular A, from blocks of 1 by doubling:
    [[P, 0], [C, Q]]^-1 = [[P^-1, 0], [-Q^-1 C P^-1, Q^-1]]."""
    n = A.shape[-1]
    M = torch.ones(*A.shape[:-2], n, 1, 1, dtype=A.dtype, device=A.device)
    size = 1
    while size < n:
        at = torch.arange(n // (2 * size), device=A.device)
        blocks = A.unflatten(-1, (-1, 2 * size)).unflatten(-3, (-1, 2 * size))
        C = blocks.movedim(-2, -3)[..., at, at, size:, :size]
        P, Q = M[..., 0::2, :, :], M[..., 1::2, :, :]
        low = -(Q @ C @ P)
        M = torch.cat([torch.cat([P, torch.zeros_like(P)], -1), torch.cat([low, Q], -1)], -2)
        size *= 2
    return M.squeeze(-3)


def _delta_chunks(q, k, v, beta, fgate, C, forget):
    """The chunked form in 32 bits (the gates' sums in 64): h and the final memory."""
    B, NH, T, dv = v.shape
    dk, group = k.shape[-1], NH // k.shape[1]
    q, k = (x.repeat_interleave(group, 1) for x in (q * dk ** -0.5, k))
    size = min(CHUNK, 1 << (T - 1).bit_length())
    pad = -T % size

    def chunks(x):
        if pad:
            x = torch.cat([x, torch.zeros_like(x[:, :, :1]).expand(
                *x.shape[:2], pad, *x.shape[3:])], 2)
        return x.unflatten(2, (-1, size))

    q, k, v, beta = (chunks(x) for x in (q, k, v, beta))
    G = chunks(_log_forget(fgate, forget)).cumsum(-1)
    low = torch.ones(size, size, dtype=torch.bool, device=q.device).tril()
    D = torch.exp((G.unsqueeze(-1) - G.unsqueeze(-2)).masked_fill(~low, -math.inf)).float()
    e, to_end = torch.exp(G).float(), torch.exp(G[..., -1:] - G).float()
    kT = k.transpose(-1, -2)
    A = (k @ kT) * D * beta.unsqueeze(-1)
    M = _unit_lower_inverse(A.masked_fill(low.T, 0.0)) * beta.unsqueeze(-2)
    U0, W = M @ v, M @ (k * e.unsqueeze(-1))
    P, qe = (q @ kT) * D, q * e.unsqueeze(-1)
    kT = (k * to_end.unsqueeze(-1)).transpose(-1, -2)
    S, h = C.transpose(-1, -2), []
    for c in range(G.shape[2]):
        U = U0[:, :, c] - W[:, :, c] @ S
        h.append(qe[:, :, c] @ S + P[:, :, c] @ U)
        S = S * e[:, :, c, -1, None, None] + kT[:, :, c] @ U
    return torch.cat(h, 2)[:, :, :T], S.transpose(-1, -2).contiguous()


def _delta_plain(s, op):
    names = ("q", "k", "v", "beta", "fgate", "state")
    dt, forget = TYPES[s["case"]["dtype"]], s["case"]["forget"]
    if op == "step":
        q, k, v, beta, fgate = (s[n].float() for n in names[:5])
        group = v.shape[1] // k.shape[1]
        q, k = (x.repeat_interleave(group, 1) for x in (q * k.shape[-1] ** -0.5, k))
        f = torch.exp(_log_forget(fgate, forget)).float()
        C = s["state"] * f[..., None, None]
        u = beta.unsqueeze(-1) * (v - (C @ k.unsqueeze(-1)).squeeze(-1))
        C = C + u.unsqueeze(-1) * k.unsqueeze(-2)
        return {"h": (C @ q.unsqueeze(-1)).squeeze(-1).to(dt), "state": C}
    x = [s[n].detach().float() for n in names]
    if op == "fwd":
        h, C = _delta_chunks(*x, forget)
        return {"h": h.to(dt), "state": C}
    x = [t.requires_grad_() for t in x]
    h, C = _delta_chunks(*x, forget)
    g = torch.autograd.grad((h, C), x, (s["dh"].float(), s["dstate"]))
    return {"h": h.detach().to(dt), "state": C.detach(), "dq": g[0].to(dt), "dk": g[1].to(dt),
            "dv": g[2].to(dt), "dbeta": g[3], "dfgate": g[4], "dstate": g[5]}


def _norm_rows(x, norm):
    if norm == "layer":
        x = x - x.mean(-1, keepdim=True)
    return x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)


def _norm_plain(s, op):
    c, dt = s["case"], TYPES[s["case"]["dtype"]]
    names = [n for n in ("p", "weight", "gate", "residual", "scale", "next_weight")
             if s[n] is not None]
    t = {n: s[n].detach().float() for n in names}
    if op == "norm_train":
        t = {n: x.requires_grad_() for n, x in t.items()}
    u = _norm_rows(t["p"], c["norm"])
    act = torch.sigmoid(t["gate"])
    if c["gate"] == "silu":
        act = act * t["gate"]
    z = (u * act).transpose(1, 2).flatten(2) * t["weight"]
    r = t["residual"] + t["scale"] * z if c["residual"] else z
    y = _norm_rows(r, c["norm"]) * t["next_weight"]
    out = {"r": r.detach().to(dt), "y": y.detach().to(dt)}
    if op == "norm_train":
        g = torch.autograd.grad((r, y), [t[n] for n in names], (s["dr"].float(), s["dy"].float()))
        out.update({"d" + n: x.to(s[n].dtype) for n, x in zip(names, g)})
    return out


# ---- the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "norm_train"):
        return _norm_exact(s, case)
    return _delta_exact(s, case)


def _delta_exact(s, case):
    """Token by token; the gradients by the reversed recurrence, the memories of
    64 tokens at a time recomputed from the one before them."""
    if case["op"] == "step":
        s = {n: x.unsqueeze(2) if n in ("q", "k", "v", "beta", "fgate") else x
             for n, x in s.items()}
    T, dk, NHK = case["T"], case["dk"], case["NHK"]
    group = case["NH"] // NHK
    q, k = (s[n].double().repeat_interleave(group, 1) for n in ("q", "k"))
    q = q / math.sqrt(dk)
    v, beta, C0 = s["v"].double(), s["beta"].double(), s["state"].double()
    x = s["fgate"].double()
    f = torch.exp(x) if case["forget"] == "exp" else 1.0 / (1.0 + torch.exp(-x))

    def forward(C, t):
        """C_t, and what is taken in with it: the memory's error and the decayed memory."""
        C = C * f[:, :, t, None, None]
        miss = v[:, :, t] - torch.matmul(C, k[:, :, t, :, None])[..., 0]
        u = beta[:, :, t, None] * miss
        return C + u[..., :, None] * k[:, :, t, None, :], miss, C

    h, starts, C = torch.empty_like(v), [], C0
    for t in range(T):
        if t % 64 == 0:
            starts.append(C)
        C = forward(C, t)[0]
        h[:, :, t] = torch.matmul(C, q[:, :, t, :, None])[..., 0]
    if case["op"] == "step":
        return {"h": h[:, :, 0], "state": C}
    out = {"h": h, "state": C}
    if case["op"] == "fwd":
        return out
    dh, dC = s["dh"].double(), s["dstate"].double()
    dq, dk_, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    db, df = torch.empty_like(beta), torch.empty_like(f)
    for a in range((T - 1) // 64 * 64, -1, -64):
        kept, C = [], starts[a // 64]
        for t in range(a, min(a + 64, T)):
            old, (C, miss, faded) = C, forward(C, t)
            kept.append((old, miss, faded, C))
        for t in range(min(a + 64, T) - 1, a - 1, -1):
            old, miss, faded, C = kept[t - a]
            kt, gt = k[:, :, t], dh[:, :, t]
            dq[:, :, t] = torch.matmul(gt[..., None, :], C)[..., 0, :]
            dC = dC + gt[..., :, None] * q[:, :, t, None, :]
            du = torch.matmul(dC, kt[..., :, None])[..., 0]
            u, miss_grad = beta[:, :, t, None] * miss, beta[:, :, t, None] * du
            db[:, :, t] = (du * miss).sum(-1)
            dv[:, :, t] = miss_grad
            dk_[:, :, t] = (torch.matmul(u[..., None, :], dC)
                            - torch.matmul(miss_grad[..., None, :], faded))[..., 0, :]
            dC = dC - miss_grad[..., :, None] * kt[..., None, :]
            df[:, :, t] = (dC * old).sum((-1, -2))
            dC = dC * f[:, :, t, None, None]
    slope = f if case["forget"] == "exp" else f / (1.0 + torch.exp(x))
    out.update(dq=dq.unflatten(1, (NHK, group)).sum(2) / math.sqrt(dk),
               dk=dk_.unflatten(1, (NHK, group)).sum(2), dv=dv, dbeta=db, dfgate=df * slope,
               dstate=dC)
    return out


def _norm_exact(s, case):
    B, NH, T, d = case["B"], case["NH"], case["T"], case["d"]
    centred = case["norm"] == "layer"

    def rows(x):
        x = x - x.mean(-1, keepdim=True) if centred else x
        inv = (x.square().mean(-1, keepdim=True) + EPS) ** -0.5
        return x * inv, inv

    def rows_grad(g, n, inv):
        g = g - n * (g * n).mean(-1, keepdim=True) - (g.mean(-1, keepdim=True) if centred else 0.0)
        return g * inv

    p, g = (s[n].double().permute(0, 2, 1, 3) for n in ("p", "gate"))
    w = s["weight"].double().view(NH, d)
    n1, inv1 = rows(p)
    sig = 1.0 / (1.0 + torch.exp(-g))
    act = sig if case["gate"] == "sigmoid" else g * sig
    z = (act * w * n1).reshape(B, T, NH * d)
    r = z if s["residual"] is None else s["residual"].double() + s["scale"].double() * z
    n2, inv2 = rows(r)
    w2 = s["next_weight"].double()
    out = {"r": r, "y": w2 * n2}
    if case["op"] == "norm":
        return out
    dy, dr = s["dy"].double(), s["dr"].double()
    out["dnext_weight"] = (dy * n2).sum((0, 1))
    dr = dr + rows_grad(dy * w2, n2, inv2)
    dz = dr
    if s["residual"] is not None:
        out["dresidual"], out["dscale"] = dr, (dr * z).sum((0, 1))
        dz = dr * s["scale"].double()
    dz = dz.view(B, T, NH, d)
    out["dweight"] = (dz * act * n1).sum((0, 1)).flatten()
    slope = sig * (1.0 - sig) if case["gate"] == "sigmoid" else sig * (1.0 + g * (1.0 - sig))
    out["dgate"] = (dz * w * n1 * slope).permute(0, 2, 1, 3)
    out["dp"] = rows_grad(dz * w * act, n1, inv1).permute(0, 2, 1, 3)
    return out


def work(case):
    size = 2 if case["dtype"] == BF16 else 4
    B, T, NH = case["B"], case["T"], case["NH"]
    if case["op"] in ("norm", "norm_train"):
        D = NH * case["d"]
        rows, res = B * T * D * size, 1 if case["residual"] else 0
        # read p, g and x, write r and y; backward: dr, dy in, dp, dg and dx out
        n, weights, ops = 4 + res, 2 + res, 25
        if case["op"] == "norm_train":
            n, weights, ops = n + 4 + res, 2 * weights, 80
        return {"bytes": n * rows + weights * D * 4, "flops": ops * B * T * D}
    NHK, dk, dv = case["NHK"], case["dk"], case["dv"]
    tokens = B * T
    qk, vh, gates, C = tokens * NHK * dk * size, tokens * NH * dv * size, tokens * NH * 4, \
        B * NH * dk * dv * 4
    n = 2 * qk + 2 * vh + 2 * gates + 2 * C
    # C k, the rank-one update and C q at each token; about twice that again backward
    flops = 6 * tokens * NH * dk * dv
    if case["op"] == "train":
        n, flops = n + 2 * qk + 2 * vh + 2 * gates + 2 * C, 3 * flops
    return {"bytes": n, "flops": flops}
