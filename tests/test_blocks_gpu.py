"""The short convolution, the selective scan and the gated feed-forward on the GPU
against the float64 oracle.

Tolerances, of float32 results first.  "Size" is the root of the sum of the squares
of a sum's terms: after j of n terms of size a and either sign a partial sum is about
sqrt(j) a, each addition is off by up to 2^-24 of that, and n such errors of either
sign make sqrt(n) 2^-24 of the sum's size sqrt(n) a.
  convolution   at most 9 terms, an activation of about 4 roundings, 8 terms back:
                below 2^-20; a weight's sum has up to 2000 terms: sqrt(2000) 2^-24 =
                2^-18.5 of its size.
  scan          a state takes three roundings a token (factor, product, sum), over at
                most 1000 tokens: sqrt(3000) 2^-24 = 2^-18.2 of its size; then sums of
                up to 64 states or 5000 channels, 2^-20 and 2^-18 of their sizes.
  feed-forward  sums of at most 2000 terms: 2^-18.5 of the sum's size, and three such
                factors follow one another backward.
So 2^-17.5 of the sizes in the 2-norm for all, and at one element 2^-14 of the root mean
square of the sizes (2^-17.5 is the root mean square error; a largest of 10^5 errors
of either sign is below 8 times it, 2^-14.5).
A bf16 result is rounded once more, by at most 2^-8 of its value: 2^-8 + 2^-17 in the
2-norm, 2^-8 |value| + 2^-14 of the sizes' root mean square at one element.  The
operands dg and du of the feed-forward's dx, dw_gate and dw_up are rounded to bf16 for
512 rows and more (below to 16 bits, 2^-17 of each term), each term by up to 2^-8 of itself, 2^-8 / sqrt(3) in the root mean square, of either sign:
2^-8 + 2^-8.7 of the sizes in the 2-norm, and at one element 2^-8 |value| + 6 * 2^-8.7 of
its own size (six times the root mean square of a sum of such errors).
"""
import numpy as np
import pytest
import torch

import oracle
from linear_recurrent_sequence_amd import mlstm

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP = torch.bfloat16, torch.float32


def host(t):
    return None if t is None else t.detach().double().cpu().numpy()


def close(name, t, ref, size=None, rounded_terms=False):
    a, ref = host(t), np.asarray(ref)
    assert a.shape == ref.shape, (name, a.shape, ref.shape)
    assert np.isfinite(a).all(), name
    size = np.abs(ref) if size is None else np.maximum(np.abs(ref), size)
    rms, err = np.sqrt((size ** 2).mean()), np.abs(a - ref)
    bf16 = t.dtype == BF
    most = rms * 2.0 ** -14 + (np.abs(ref) * 2.0 ** -8 if bf16 else 0.0)
    total = 2.0 ** -17.5 + (2.0 ** -8 if bf16 else 0.0)
    if rounded_terms and bf16:
        most = most + 6 * 2.0 ** -8.7 * size
        total += 2.0 ** -8.7
    norm = np.linalg.norm(err) / max(np.linalg.norm(size), 1e-30)
    assert norm <= total, (name, norm, total)
    assert (err <= most + 1e-30).all(), (name, (err / (most + 1e-30)).max())


def gpu(x, dtype=FP):
    return None if x is None else torch.tensor(np.asarray(x), device=DEV).to(dtype)


def i32(x):
    return None if x is None else torch.tensor(x, device=DEV, dtype=torch.int32)


def rows_of(y, heads):
    """[B, heads, T, d] -> [B, T, C] (rows as they are without heads)."""
    return y if heads is None else y.transpose(1, 2).flatten(2)


# ---------------------------------------------------------------- short convolution

def conv_inputs(B, T, C, W, dtype, seed=0, extras=True):
    n = np.random.default_rng(seed).standard_normal
    x, dy = gpu(n((B, T, C)), dtype), gpu(n((B, T, C)), dtype)
    w, b = gpu(n((C, W)) * W ** -0.5), gpu(n(C)) if extras else None
    st, dst = (gpu(n((B, W - 1, C)), dtype) if extras else None for _ in range(2))
    return x, w, b, st, dy, dst


CONVS = [
    # B, T, C, heads, W, dtype, lengths, activation
    (1, 1, 8, 1, 2, BF, None, "silu"),
    (2, 1, 24, 3, 8, FP, None, "none"),
    (3, 2, 16, None, 4, FP, [2, 1, 0], "silu"),
    (2, 5, 40, 5, 7, BF, [0, 5], "silu"),
    (2, 33, 264, 3, 3, FP, None, "silu"),
    (4, 70, 104, 1, 4, BF, [70, 3, 64, 0], "silu"),
    (1, 300, 136, 1, 5, BF, None, "none"),
    (2, 257, 256, 4, 4, FP, [256, 9], "silu"),
    (3, 600, 72, None, 6, FP, [600, 599, 1], "silu"),
    (1, 999, 48, 2, 8, BF, None, "silu"),
]


@pytest.mark.parametrize("B,T,C,heads,W,dtype,lengths,activation", CONVS)
@pytest.mark.parametrize("extras", [True, False])
def test_short_conv(B, T, C, heads, W, dtype, lengths, activation, extras):
    x, w, b, st, dy, dst = conv_inputs(B, T, C, W, dtype, 1, extras)
    kw = dict(bias=b, state=st, heads=heads, lengths=i32(lengths), activation=activation)
    y, new = mlstm.short_conv_fwd(x, w, **kw)
    assert y.dtype == new.dtype == dtype
    assert y.shape == ((B, T, C) if heads is None else (B, heads, T, C // heads))
    yr, sr = oracle.short_conv(host(x), host(w), host(b), host(st), lengths, activation)
    close("y", rows_of(y, heads), yr)
    assert np.array_equal(host(new), sr)  # inputs, unchanged
    by_heads = dy if heads is None else dy.unflatten(2, (heads, -1)).transpose(1, 2).contiguous()
    g = mlstm.short_conv_bwd(x, w, by_heads, dstate=dst, **kw)
    dx, dw, db, ds, w_size, b_size = oracle.short_conv_grads(
        host(x), host(w), host(dy), host(b), host(st), host(dst), lengths, activation)
    close("dx", g["dx"], dx, size=np.full_like(dx, np.sqrt((dx ** 2).mean())))
    close("dweight", g["dweight"], dw, w_size)
    close("dstate", g["dstate"], ds, size=np.full_like(ds, np.sqrt((dx ** 2).mean())))
    if extras:
        close("dbias", g["dbias"], db, b_size)
        kept = st.clone()  # in place
        y2, new2 = mlstm.short_conv_fwd(x, w, out_state=kept, **{**kw, "state": kept})
        assert new2 is kept and torch.equal(kept, new) and torch.equal(y2, y)
    else:
        assert "dbias" not in g


@pytest.mark.parametrize("dtype", [BF, FP])
def test_short_conv_in_pieces_and_steps_is_bitwise_the_whole(dtype):
    x, w, b, st, _, _ = conv_inputs(2, 90, 64, 4, dtype, 2)
    y, new = mlstm.short_conv_fwd(x, w, bias=b, state=st, heads=2)
    s, ys = st, []
    for a, e in ((0, 1), (1, 3), (3, 50), (50, 90)):
        part, s = mlstm.short_conv_fwd(x[:, a:e].contiguous(), w, bias=b, state=s, heads=2)
        ys.append(part)
    assert torch.equal(torch.cat(ys, 2), y) and torch.equal(s, new)
    s = mlstm.conv_state(2, 64, 4, dtype, DEV).copy_(st)
    for t in range(90):
        part, out = mlstm.short_conv_step(x[:, t].contiguous(), w, s, bias=b, heads=2)
        assert out is s and torch.equal(part, y[:, :, t])
    assert torch.equal(s, new)


# ---------------------------------------------------------------- selective scan

def scan_inputs(n, T, c, N, G, dtype, seed=0, extras=True, slow=1.0):
    r = np.random.default_rng(seed)
    z = r.standard_normal
    x = dict(u=gpu(z((n, T, c)), dtype), dt=gpu(0.5 * z((n, T, c)) + (0.0 if extras else -3.0), dtype),
             A=gpu(-slow * np.exp(0.5 * z((c, N))) * np.arange(1, N + 1)),
             B=gpu(z((n, T, G, N)), dtype), C=gpu(z((n, T, G, N)), dtype))
    if extras:
        x.update(D=gpu(z(c)), gate=gpu(z((n, T, c)), dtype),
                 dt_bias=gpu(np.log(np.expm1(np.exp(r.uniform(np.log(1e-3), np.log(0.1), c))))),
                 state=gpu(z((n, c, N))))
    return x, gpu(z((n, T, c)), dtype), gpu(z((n, c, N))) if extras else None


def scan_ref(x, lengths=None):
    return oracle.selective_scan(**{k: host(v) for k, v in x.items()}, lengths=lengths)


def check_scan_grads(g, x, dy, dst, lengths=None):
    ref, size = oracle.selective_scan_grads(**{k: host(v) for k, v in x.items()}, dy=host(dy),
                                            dstate=host(dst), lengths=lengths)
    if x.get("state") is None:
        ref.setdefault("dstate", None)
    assert set(g) == set(ref)
    for k in ref:
        assert g[k].dtype == (x["u"].dtype if k in ("du", "ddt", "dB", "dC", "dgate") else FP), k
        # a token's gradient is a sum over the states of terms as large as its row's
        spread = np.full_like(ref[k], np.sqrt((ref[k] ** 2).mean()))
        close(k, g[k], ref[k], np.maximum(spread, size[k]) if k in size else spread)


SCANS = [
    # n, T, c, N, G, dtype, lengths
    (1, 1, 8, 1, 1, FP, None),
    (2, 1, 16, 16, 2, BF, [1, 0]),
    (2, 2, 24, 3, 3, FP, None),
    (1, 16, 64, 4, 1, FP, None),
    (3, 17, 72, 5, 1, BF, [17, 0, 16]),
    (2, 31, 136, 8, 1, FP, [31, 1]),
    (1, 33, 128, 11, 2, BF, None),
    (2, 64, 40, 16, 1, FP, [33, 64]),
    (2, 65, 208, 16, 2, BF, None),
    (1, 100, 72, 20, 1, FP, None),
    (2, 63, 80, 32, 2, BF, [63, 5]),
    (1, 70, 64, 33, 1, FP, None),
    (1, 129, 24, 64, 3, BF, None),
    (1, 50, 16, 64, 1, FP, [49]),
]


@pytest.mark.parametrize("n,T,c,N,G,dtype,lengths", SCANS)
@pytest.mark.parametrize("extras", [True, False])
def test_scan(n, T, c, N, G, dtype, lengths, extras):
    x, dy, dst = scan_inputs(n, T, c, N, G, dtype, 3, extras)
    kw = {k: v for k, v in x.items() if k not in ("u", "dt", "A", "B", "C")}
    args = [x[k] for k in ("u", "dt", "A", "B", "C")]
    y, st = mlstm.scan_fwd(*args, lengths=i32(lengths), **kw)
    assert y.dtype == dtype and st.dtype == FP
    yr, sr = scan_ref(x, lengths)
    close("y", y, yr, np.full_like(yr, np.sqrt((yr ** 2).mean())))
    close("state", st, sr)
    g = mlstm.scan_bwd(*args, dy, dstate=dst, lengths=i32(lengths), **kw)
    check_scan_grads(g, x, dy, dst, lengths)
    if extras:
        kept = x["state"].clone()  # in place
        y2, st2 = mlstm.scan_fwd(*args, lengths=i32(lengths), **{**kw, "state": kept},
                                 out_state=kept)
        assert st2 is kept and torch.equal(kept, st) and torch.equal(y2, y)


# sequences that are cut into segments (a workspace says so), with each number of
# states to a wave, ragged last segments, and lengths that end in the middle of one
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n,T,c,N,G,lengths", [
    (1, 1000, 8, 3, 1, None), (2, 801, 72, 7, 1, [801, 300]), (1, 900, 64, 16, 2, None),
    (2, 513, 40, 24, 1, [0, 512]), (1, 700, 16, 64, 1, [690])])
def test_scan_in_segments(n, T, c, N, G, lengths, dtype):
    size = mlstm.load_library().mlstm_scan_workspace_bytes
    assert size(n, T, c, G, N, int(dtype == BF), 0) > 0
    x, dy, dst = scan_inputs(n, T, c, N, G, dtype, 4, slow=0.1)
    kw = {k: v for k, v in x.items() if k not in ("u", "dt", "A", "B", "C")}
    args = [x[k] for k in ("u", "dt", "A", "B", "C")]
    y, st = mlstm.scan_fwd(*args, lengths=i32(lengths), **kw)
    yr, sr = scan_ref(x, lengths)
    close("y", y, yr, np.full_like(yr, np.sqrt((yr ** 2).mean())))
    close("state", st, sr)
    check_scan_grads(mlstm.scan_bwd(*args, dy, dstate=dst, lengths=i32(lengths), **kw), x, dy, dst,
                     lengths)


# more workgroups than CUs: four states to a wave, and one piece
@pytest.mark.parametrize("N", [2, 7, 16, 21, 40])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_scan_of_many_channels(N, dtype):
    x, dy, dst = scan_inputs(5, 37, 4168, N, 1, dtype, 19)
    kw = {k: v for k, v in x.items() if k not in ("u", "dt", "A", "B", "C")}
    args = [x[k] for k in ("u", "dt", "A", "B", "C")]
    y, st = mlstm.scan_fwd(*args, **kw)
    yr, sr = scan_ref(x)
    close("y", y, yr, np.full_like(yr, np.sqrt((yr ** 2).mean())))
    close("state", st, sr)
    check_scan_grads(mlstm.scan_bwd(*args, dy, dstate=dst, **kw), x, dy, dst)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_scan_prompt_and_steps(dtype):
    x, _, _ = scan_inputs(3, 40, 72, 12, 3, dtype, 5)
    yr, sr = scan_ref(x)
    cut = {k: v[:, :30].contiguous() if k in ("u", "dt", "B", "C", "gate") else v
           for k, v in x.items()}
    y, st = mlstm.scan_fwd(**cut)
    ys = [y]
    for t in range(30, 40):
        one = {k: v[:, t].contiguous() if k in ("u", "dt", "B", "C", "gate") else v
               for k, v in x.items()}
        y, out = mlstm.scan_step(**{**one, "state": st})
        assert out is st
        ys.append(y.unsqueeze(1))
    close("y", torch.cat(ys, 1), yr, np.full_like(yr, np.sqrt((yr ** 2).mean())))
    close("state", st, sr)


def test_scan_steps_of_many_channels():
    for N in (1, 16, 63):
        x, _, _ = scan_inputs(70, 1, 520, N, 1, BF, 6)
        one = {k: v[:, 0].contiguous() if k in ("u", "dt", "B", "C", "gate") else v
               for k, v in x.items()}
        out = torch.empty_like(one["state"])
        y, st = mlstm.scan_step(**one, out_state=out)
        yr, sr = scan_ref(x)
        assert st is out
        close("y", y, yr[:, 0], np.full_like(yr[:, 0], np.sqrt((yr ** 2).mean())))
        close("state", st, sr)


# ---------------------------------------------------------------- gated feed-forward

def ffn_inputs(M, D, F, dtype, seed=0):
    n = np.random.default_rng(seed).standard_normal
    return (gpu(n((M, D)), dtype), gpu(n((F, D)) * D ** -0.5, dtype),
            gpu(n((F, D)) * D ** -0.5, dtype), gpu(n((M, F)), dtype))


FFNS = [(1, 8, 8), (1, 72, 136), (16, 64, 24), (17, 264, 40), (33, 1000, 72), (64, 136, 520),
        (65, 8, 264), (129, 200, 136), (257, 520, 264), (300, 72, 1048), (1000, 256, 8)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("M,D,F", FFNS)
@pytest.mark.parametrize("activation", ["silu", "gelu"])
def test_gated_ffn(M, D, F, dtype, activation):
    x, wg, wu, dh = ffn_inputs(M, D, F, dtype, 7)
    h = mlstm.gated_ffn_fwd(x, wg, wu, activation)
    ref = oracle.gated_ffn(host(x), host(wg), host(wu), activation)
    close("h", h, ref, np.full_like(ref, np.sqrt((ref ** 2).mean())))
    got = mlstm.gated_ffn_bwd(x, wg, wu, dh, activation)
    refs, sizes = oracle.gated_ffn_grads(host(x), host(wg), host(wu), host(dh), activation)
    for name, a, r, size in zip(("dx", "dw_gate", "dw_up"), got, refs, sizes):
        assert a.dtype == dtype
        close(name, a, r, size, rounded_terms=M >= 512)


# tiles of each kind, whole and split, on more tiles than there are CUs
@pytest.mark.parametrize("M,D,F,dtype", [(2100, 328, 4104, BF), (4200, 72, 2312, BF),
                                         (520, 2056, 1032, BF), (1500, 136, 1544, FP)])
def test_gated_ffn_of_many_tiles(M, D, F, dtype):
    x, wg, wu, dh = ffn_inputs(M, D, F, dtype, 8)
    h = mlstm.gated_ffn_fwd(x, wg, wu)
    ref = oracle.gated_ffn(host(x), host(wg), host(wu))
    close("h", h, ref, np.full_like(ref, np.sqrt((ref ** 2).mean())))
    got = mlstm.gated_ffn_bwd(x, wg, wu, dh)
    refs, sizes = oracle.gated_ffn_grads(host(x), host(wg), host(wu), host(dh))
    for name, a, r, size in zip(("dx", "dw_gate", "dw_up"), got, refs, sizes):
        close(name, a, r, size, rounded_terms=True)


def test_gated_ffn_takes_any_leading_sizes():
    x, wg, wu, dh = ffn_inputs(90, 64, 72, BF, 9)
    h = mlstm.gated_ffn_fwd(x.view(2, 5, 9, 64), wg, wu)
    assert h.shape == (2, 5, 9, 72) and torch.equal(h.view(90, 72), mlstm.gated_ffn_fwd(x, wg, wu))
    dx = mlstm.gated_ffn_bwd(x.view(2, 5, 9, 64), wg, wu, dh.view(2, 5, 9, 72))[0]
    assert dx.shape == (2, 5, 9, 64)
    assert torch.equal(dx.view(90, 64), mlstm.gated_ffn_bwd(x, wg, wu, dh)[0])


def test_gated_ffn_activations_far_from_zero():
    """Where the activation is all or nothing, and at zero."""
    x = torch.tensor([[-60.0, -9.0, 0.0, 9.0, 60.0, -30.0, 30.0, 1e-20]], device=DEV).T.contiguous()
    x = torch.cat([x, torch.zeros(8, 7, device=DEV)], 1)
    w = torch.zeros(8, 8, device=DEV)
    w[:, 0] = 1.0
    for activation in ("silu", "gelu"):
        for rows in (8, 72):
            big = x.repeat(rows // 8, 1)
            h = host(mlstm.gated_ffn_fwd(big, w, w, activation))
            ref = oracle.gated_ffn(host(big), host(w), host(w), activation)
            # absolute below 1e-6: a float32 Phi(-9) or sigma(-60) is exact to its own size only
            assert np.allclose(h, ref, rtol=2.0 ** -20, atol=1e-6)
            assert np.isfinite(host(mlstm.gated_ffn_bwd(big, w, w, torch.ones_like(big))[0])).all()


# ------------------------------------------------- padding, rows, offsets, workspaces

def _poison(t, lengths):
    t = t.clone()
    for b, n in enumerate(lengths):
        t[b, n:] = float("nan")
    return t


@pytest.mark.parametrize("T", [40, 1200])
def test_positions_behind_a_sequence_are_not_read(T):
    """NaN in every input there; 1200 positions are cut into segments."""
    lengths = [T, 0, 17, T - 5]
    x, w, b, st, dy, dst = conv_inputs(4, T, 24, 4, BF, 10)
    kw = dict(bias=b, state=st, lengths=i32(lengths))
    ref = [*mlstm.short_conv_fwd(x, w, **kw),
           *mlstm.short_conv_bwd(x, w, dy, dstate=dst, **kw).values()]
    px, pdy = _poison(x, lengths), _poison(dy, lengths)
    got = [*mlstm.short_conv_fwd(px, w, **kw),
           *mlstm.short_conv_bwd(px, w, pdy, dstate=dst, **kw).values()]
    assert all(torch.equal(a, r) for a, r in zip(got, ref))
    x, dy, dst = scan_inputs(4, T, 24, 6, 1, FP, 11)
    rows = ("u", "dt", "B", "C", "gate")
    p = {k: _poison(v, lengths) if k in rows else v for k, v in x.items()}
    ref = [*mlstm.scan_fwd(**x, lengths=i32(lengths)),
           *mlstm.scan_bwd(**x, dy=dy, dstate=dst, lengths=i32(lengths)).values()]
    got = [*mlstm.scan_fwd(**p, lengths=i32(lengths)),
           *mlstm.scan_bwd(**p, dy=_poison(dy, lengths), dstate=dst,
                           lengths=i32(lengths)).values()]
    assert all(torch.equal(a, r) for a, r in zip(got, ref))
    for out in (got[0], got[2]):  # y, du
        assert not out[1].any() and not out[2, 17:].any()


def test_lengths_out_of_range_are_kept_in_it():
    x, w, b, st, _, _ = conv_inputs(3, 9, 8, 3, FP, 12)
    wild = mlstm.short_conv_fwd(x, w, bias=b, state=st, lengths=i32([-5, 1000, 9]))
    tame = mlstm.short_conv_fwd(x, w, bias=b, state=st, lengths=i32([0, 9, 9]))
    assert all(torch.equal(a, r) for a, r in zip(wild, tame))
    x, dy, dst = scan_inputs(3, 9, 8, 3, 1, FP, 13)
    wild = mlstm.scan_bwd(**x, dy=dy, dstate=dst, lengths=i32([-(2 ** 31), 2 ** 31 - 1, 9]))
    tame = mlstm.scan_bwd(**x, dy=dy, dstate=dst, lengths=i32([0, 9, 9]))
    assert all(torch.equal(wild[k], tame[k]) for k in tame)


def test_a_step_of_minus_infinity_leaves_the_state():
    x, dy, dst = scan_inputs(2, 50, 16, 5, 1, FP, 14)
    x["dt"][:, 20:] = float("-inf")
    y, st = mlstm.scan_fwd(**x)
    cut = {k: v[:, :20].contiguous() if k in ("u", "dt", "B", "C", "gate") else v
           for k, v in x.items()}
    close("state", st, scan_ref(cut)[1])
    g = mlstm.scan_bwd(**x, dy=dy, dstate=dst)
    check_scan_grads(g, x, dy, dst)
    assert not g["ddt"][:, 20:].any()


@pytest.mark.parametrize("dtype", [BF, FP])
def test_rows_of_a_wider_matrix_are_bitwise_the_same(dtype):
    """The parts of one projection: rows that are further apart than they are long."""
    n, T, c, N, G = 2, 300, 40, 5, 1
    x, dy, dst = scan_inputs(n, T, c, N, G, dtype, 15)
    wide = torch.full((n, T, 8 + 3 * c + 2 * N + 6), float("nan"), device=DEV, dtype=dtype)
    wide[..., 8:8 + c], wide[..., 8 + c:8 + 2 * c], wide[..., 8 + 2 * c:8 + 3 * c] = \
        x["u"], x["dt"], x["gate"]
    at = 8 + 3 * c
    wide[..., at + 1:at + 1 + N], wide[..., at + 1 + N:at + 1 + 2 * N] = \
        x["B"].flatten(2), x["C"].flatten(2)
    v = dict(x, u=wide[..., 8:8 + c], dt=wide[..., 8 + c:8 + 2 * c],
             gate=wide[..., 8 + 2 * c:8 + 3 * c],
             B=wide[..., at + 1:at + 1 + N].unflatten(-1, (G, N)),
             C=wide[..., at + 1 + N:at + 1 + 2 * N].unflatten(-1, (G, N)))
    assert wide.shape[-1] % 8 == 0 and not v["u"].is_contiguous()
    for a, b in zip(mlstm.scan_fwd(**v), mlstm.scan_fwd(**x)):
        assert torch.equal(a, b) and a.is_contiguous()
    a, b = mlstm.scan_bwd(**v, dy=dy, dstate=dst), mlstm.scan_bwd(**x, dy=dy, dstate=dst)
    assert all(torch.equal(a[k], b[k]) and a[k].is_contiguous() for k in b)
    rows = ("u", "dt", "B", "C", "gate")
    one = mlstm.scan_step(**{k: t[:, 3] if k in rows else t.clone() for k, t in v.items()})
    ref = mlstm.scan_step(**{k: t[:, 3].contiguous() if k in rows else t.clone()
                             for k, t in x.items()})
    assert all(torch.equal(p, q) for p, q in zip(one, ref))
    _, w, b, st, dy, dst = conv_inputs(n, T, c, 4, dtype, 16)
    kw = dict(bias=b, state=st)
    for p, q in zip(mlstm.short_conv_fwd(v["u"], w, **kw), mlstm.short_conv_fwd(x["u"], w, **kw)):
        assert torch.equal(p, q)
    a = mlstm.short_conv_bwd(v["u"], w, dy, dstate=dst, **kw)
    b = mlstm.short_conv_bwd(x["u"], w, dy, dstate=dst, **kw)
    assert all(torch.equal(a[k], b[k]) and a[k].is_contiguous() for k in b)


def test_refused_on_the_gpu():
    """Sizes and rows that the header rules out; the calls before and after are as ever."""
    w = torch.zeros(40, 4, device=DEV)
    wide = torch.zeros(1, 5, 44, device=DEV)
    with pytest.raises(mlstm.MlstmError, match="pitch"):
        mlstm.short_conv_fwd(wide[..., :40], w)
    with pytest.raises(mlstm.MlstmError, match="multiple of 8"):  # heads of 20
        mlstm.short_conv_fwd(torch.zeros(1, 5, 40, device=DEV), w, heads=2)
    with pytest.raises(ValueError, match="evenly"):  # a part of each sequence of a batch
        mlstm.short_conv_fwd(torch.zeros(2, 9, 40, device=DEV)[:, 2:5], w)
    x, wg, wu, _ = ffn_inputs(3, 64, 40, BF, 50)
    with pytest.raises(mlstm.MlstmError, match="multiple of 8"):
        mlstm.gated_ffn_fwd(x, wg[:36].contiguous(), wu[:36].contiguous())
    with pytest.raises(ValueError, match="GPU tensor"):
        mlstm.gated_ffn_fwd(x, wg, wu.cpu())
    with pytest.raises(mlstm.MlstmError):  # no rows
        mlstm.gated_ffn_fwd(x[:0], wg, wu)


def test_offsets_past_32_bits():
    """Rows 2^20 elements apart: the last of 2200 begin 4.6 GB behind the first."""
    T, c = 2200, 16
    wide = torch.empty(1, T, 1 << 20, device=DEV, dtype=BF)
    x, dy, dst = scan_inputs(1, T, c, 4, 1, BF, 17)
    v = dict(x)
    for i, k in enumerate(("u", "dt", "gate")):
        v[k] = wide[..., i * c:(i + 1) * c].copy_(x[k])
    for i, k in enumerate(("B", "C")):
        v[k] = wide[..., 1000 + 4 * i:1004 + 4 * i].unflatten(-1, (1, 4)).copy_(x[k])
    for a, b in zip(mlstm.scan_fwd(**v), mlstm.scan_fwd(**x)):
        assert torch.equal(a, b)
    a, b = mlstm.scan_bwd(**v, dy=dy, dstate=dst), mlstm.scan_bwd(**x, dy=dy, dstate=dst)
    assert all(torch.equal(a[k], b[k]) for k in b)
    _, w, b, st, dy, dst = conv_inputs(1, T, c, 4, BF, 18)
    a, r = (mlstm.short_conv_bwd(u, w, dy, bias=b, state=st) for u in (v["u"], x["u"]))
    assert all(torch.equal(a[k], r[k]) for k in r)
    del wide, v
    # results of more than 2^32 bytes: the last rows against a call of their own
    M, D, F = 131072 + 72, 64, 16392
    n = np.random.default_rng(19).standard_normal
    x = torch.randn(M, D, device=DEV, dtype=BF)
    wg, wu = (gpu(n((F, D)) * D ** -0.5, BF) for _ in range(2))
    h = mlstm.gated_ffn_fwd(x, wg, wu)
    tail = x[-300:].contiguous()
    ref = oracle.gated_ffn(host(tail), host(wg), host(wu))
    close("h", h[-300:], ref, np.full_like(ref, np.sqrt((ref ** 2).mean())))


def test_workspaces_need_no_clearing(monkeypatch):
    x, w, b, st, dy, dst = conv_inputs(2, 100, 40, 4, BF, 20)
    s, sdy, sdst = scan_inputs(2, 600, 40, 9, 1, FP, 21)
    f = {dt: ffn_inputs(150, 72, 136, dt, 22) for dt in (BF, FP)}

    def everything():
        out = [*mlstm.short_conv_bwd(x, w, dy, bias=b, state=st, dstate=dst).values(),
               *mlstm.scan_fwd(**s), *mlstm.scan_bwd(**s, dy=sdy, dstate=sdst).values()]
        for fx, wg, wu, dh in f.values():
            out += [mlstm.gated_ffn_fwd(fx, wg, wu), *mlstm.gated_ffn_bwd(fx, wg, wu, dh)]
        return out

    ref = everything()
    monkeypatch.setattr(mlstm, "_workspace", lambda n, device: torch.full(
        (n,), 255, dtype=torch.uint8, device=device) if n else None)
    for again in (everything(), everything()):  # bitwise reproducible, too
        assert all(torch.equal(a, r) for a, r in zip(again, ref))


def _padded(shape, dtype):
    """A tensor with 256 bytes of a pattern before and after it, and a check of them."""
    n = int(np.prod(shape)) * (2 if dtype == BF else 4)
    raw = torch.full((n + 512,), 0x5A, dtype=torch.uint8, device=DEV)
    t = raw[256:256 + n].view(dtype).view(shape)
    return t, lambda: bool((raw[:256] == 0x5A).all() and (raw[256 + n:] == 0x5A).all())


@pytest.mark.parametrize("dtype", [BF, FP])
def test_nothing_is_written_beside_the_outputs(monkeypatch, dtype):
    checks = []

    def empty(shape, dtype=None, device=None, **_):
        shape = (shape,) if isinstance(shape, int) else tuple(shape)
        if dtype == torch.uint8:
            raw = torch.full((shape[0] + 256,), 0x5A, dtype=torch.uint8, device=device)
            checks.append(lambda: bool((raw[shape[0]:] == 0x5A).all()))
            return raw[:shape[0]]
        t, ok = _padded(shape, dtype)
        checks.append(ok)
        return t

    x, w, b, st, dy, dst = conv_inputs(2, 37, 24, 4, dtype, 23)
    s, sdy, sdst = scan_inputs(2, 333, 24, 5, 1, dtype, 24)
    f = [(*ffn_inputs(M, 72, 40, dtype, 25),) for M in (3, 70, 150)]
    monkeypatch.setattr(mlstm.torch, "empty", empty)
    monkeypatch.setattr(mlstm.torch, "empty_like", lambda t, **_: empty(t.shape, t.dtype, t.device))
    mlstm.short_conv_fwd(x, w, bias=b, state=st, heads=3)
    mlstm.short_conv_bwd(x, w, dy, bias=b, state=st, dstate=dst)
    mlstm.scan_fwd(**s)
    mlstm.scan_bwd(**s, dy=sdy, dstate=sdst)
    for fx, wg, wu, dh in f:
        mlstm.gated_ffn_fwd(fx, wg, wu)
        mlstm.gated_ffn_bwd(fx, wg, wu, dh)
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert len(checks) > 30 and all(ok() for ok in checks)


# ------------------------------------------------------------------- runs of them together

def _block_weights(C, N, F, W, seed=30):
    r = np.random.default_rng(seed)
    z = r.standard_normal
    return dict(conv=z((C, W)) * W ** -0.5, conv_b=0.1 * z(C), A=-np.exp(0.3 * z((C, N))),
                dt_w=z((C, C)) * C ** -0.5, bc_w=z((2 * N, C)) * C ** -0.5, D=z(C),
                dt_b=np.log(np.expm1(np.exp(r.uniform(np.log(0.01), np.log(0.3), C)))),
                n1=1.0 + 0.1 * z(C), n2=1.0 + 0.1 * z(C), wg=z((F, C)) * C ** -0.5,
                wu=z((F, C)) * C ** -0.5)


def _block(x, z, p, states, lengths=None):
    """conv -> scan -> block norm (gate, residual, next norm) -> feed-forward, float32."""
    C, N = p["A"].shape
    kw = {} if lengths is None else dict(lengths=lengths)
    u, s0 = mlstm.short_conv_fwd(x, p["conv"], bias=p["conv_b"], state=states[0], **kw)
    bc = (u @ p["bc_w"].T).unsqueeze(2)
    y, s1 = mlstm.scan_fwd(u, u @ p["dt_w"].T, p["A"], bc[..., :N], bc[..., N:], D=p["D"],
                           dt_bias=p["dt_b"], state=states[1], **kw)
    norm = dict(gate=z.unsqueeze(1), residual=x, next_weight=p["n2"], norm="rms",
                activation="silu")
    r, q = mlstm.block_norm_fwd(y.unsqueeze(1), p["n1"], **norm)
    h = mlstm.gated_ffn_fwd(q, p["wg"], p["wu"])
    return h, r, (s0, s1), (u, bc, y, norm, q)


def test_a_block_of_them_prompt_and_tokens():
    """A padded batch's prompts, then tokens one at a time, against the whole sequences
    in one call."""
    C, N, F, W, T = 64, 8, 88, 4, 30
    p = {k: gpu(v) for k, v in _block_weights(C, N, F, W).items()}
    n = np.random.default_rng(31).standard_normal
    x, z = gpu(n((3, T, C))), gpu(n((3, T, C)))
    h, r, states, _ = _block(x, z, p, (None, None))
    lengths = [20, 7, 13]
    _, _, s, _ = _block(x[:, :20].contiguous(), z[:, :20].contiguous(), p, (None, None),
                        i32(lengths))
    for t in range(10):
        at = torch.tensor([m + t for m in lengths], device=DEV)
        each = torch.arange(3, device=DEV)
        u, s0 = mlstm.short_conv_step(x[each, at], p["conv"], s[0], bias=p["conv_b"])
        bc = (u @ p["bc_w"].T).unsqueeze(1)
        y, s1 = mlstm.scan_step(u, u @ p["dt_w"].T, p["A"], bc[..., :N], bc[..., N:], s[1],
                                D=p["D"], dt_bias=p["dt_b"])
        assert s0 is s[0] and s1 is s[1]
        rt, qt = mlstm.block_norm_fwd(y.view(3, 1, 1, C), p["n1"], gate=z[each, at].view(3, 1, 1, C),
                                      residual=x[each, at].unsqueeze(1), next_weight=p["n2"],
                                      norm="rms", activation="silu")
        ht = mlstm.gated_ffn_fwd(qt, p["wg"], p["wu"])
        # both are float32 evaluations of one formula: 2^-17.5 each, and the library's
        # products between them
        for a, ref in ((ht[:, 0], h[each, at]), (rt[:, 0], r[each, at])):
            assert ((a - ref).norm() / ref.norm()).item() < 2.0 ** -16


def test_a_block_of_them_trains():
    """The gradients of the whole run against differences of the run in float64."""
    C, N, F, W, T = 16, 3, 24, 4, 11
    w = _block_weights(C, N, F, W, 32)
    n = np.random.default_rng(33).standard_normal
    x, z, dh = n((2, T, C)), n((2, T, C)), n((2, T, F))
    p = {k: gpu(v) for k, v in w.items()}
    h, r, _, (u, bc, y, norm, q) = _block(gpu(x), gpu(z), p, (None, None))
    dq, dwg, dwu = mlstm.gated_ffn_bwd(q, p["wg"], p["wu"], gpu(dh))
    gn = mlstm.block_norm_bwd(y.unsqueeze(1), p["n1"], None, dq, **norm)
    gs = mlstm.scan_bwd(u, u @ p["dt_w"].T, p["A"], bc[..., :N], bc[..., N:], gn["dp"][:, 0],
                        D=p["D"], dt_bias=p["dt_b"])
    dbc = torch.cat([gs["dB"], gs["dC"]], -1)[:, :, 0]
    du = gs["du"] + gs["ddt"] @ p["dt_w"] + dbc @ p["bc_w"]
    gc = mlstm.short_conv_bwd(gpu(x), p["conv"], du, bias=p["conv_b"])
    grads = dict(x=gc["dx"] + gn["dresidual"], conv=gc["dweight"], conv_b=gc["dbias"], A=gs["dA"],
                 D=gs["dD"], dt_b=gs["ddt_bias"], dt_w=torch.einsum("btc,btd->cd", gs["ddt"], u),
                 bc_w=torch.einsum("btc,btd->cd", dbc, u), n1=gn["dweight"],
                 n2=gn["dnext_weight"], wg=dwg, wu=dwu, z=gn["dgate"][:, 0])

    def rms(a):
        return a / np.sqrt((a ** 2).mean(-1, keepdims=True) + 1e-5)

    def loss(**kw):
        v = {**w, "x": x, "z": z, **kw}
        u, _ = oracle.short_conv(v["x"], v["conv"], v["conv_b"])
        bc = (u @ v["bc_w"].T)[:, :, None]
        y, _ = oracle.selective_scan(u, u @ v["dt_w"].T, v["A"], bc[..., :N], bc[..., N:],
                                     D=v["D"], dt_bias=v["dt_b"])
        act = v["z"] / (1.0 + np.exp(-v["z"]))
        r = v["x"] + act * v["n1"] * rms(y)
        return (oracle.gated_ffn(v["n2"] * rms(r), v["wg"], v["wu"]) * dh).sum()

    r = np.random.default_rng(34)
    for name, g in grads.items():
        g, base = host(g), w.get(name, x if name == "x" else z)
        d = r.standard_normal(base.shape)
        diff = (loss(**{name: base + 1e-5 * d}) - loss(**{name: base - 1e-5 * d})) / 2e-5
        # four operators and the library's products follow one another, 2^-17.5 each and
        # factors of up to 2 between them: 2^-14 of the gradient in the 2-norm, and an
        # error of that size has a component below four times it along a random d
        assert abs((g * d).sum() - diff) < 4 * 2.0 ** -14 * np.linalg.norm(g), name


def test_on_other_streams():
    """Two calls at once on two streams, on tensors of a third."""
    s, sdy, sdst = scan_inputs(1, 700, 64, 16, 1, BF, 40)
    f = ffn_inputs(300, 136, 264, BF, 41)
    x, w, b, st, dy, dst = conv_inputs(2, 200, 64, 4, BF, 42)

    def run():
        return [*mlstm.scan_fwd(**s), *mlstm.scan_bwd(**s, dy=sdy, dstate=sdst).values(),
                *mlstm.gated_ffn_bwd(*f), *mlstm.short_conv_bwd(x, w, dy, bias=b).values()]

    ref = run()
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(3):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                outs[i].append(run())
    torch.cuda.synchronize()
    for out in outs[0] + outs[1]:
        assert all(torch.equal(a, r) for a, r in zip(out, ref))


def test_in_graphs():
    """Two captured runs, replayed in turn with new inputs and eager calls between."""
    s, sdy, sdst = scan_inputs(1, 500, 40, 16, 1, FP, 43)
    f = ffn_inputs(200, 72, 136, FP, 44)
    few = ffn_inputs(5, 72, 136, BF, 45)
    x, w, b, st, dy, dst = conv_inputs(2, 100, 40, 4, BF, 46)

    def run():
        return [*mlstm.short_conv_fwd(x, w, bias=b, state=st),
                *mlstm.short_conv_bwd(x, w, dy, bias=b, state=st, dstate=dst).values(),
                *mlstm.scan_fwd(**s), *mlstm.scan_bwd(**s, dy=sdy, dstate=sdst).values(),
                mlstm.gated_ffn_fwd(*f[:3]), *mlstm.gated_ffn_bwd(*f),
                mlstm.gated_ffn_fwd(*few[:3])]

    run()
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for graph in graphs:
        with torch.cuda.graph(graph):
            outs.append(run())
    for i in range(4):
        for t in (x, s["u"], f[0], few[0]):
            t.normal_()
        graphs[i % 2].replay()
        graphs[1 - i % 2].replay()
        ref = run()
        torch.cuda.synchronize()
        for out in outs:
            assert all(torch.equal(a, r) for a, r in zip(out, ref))


@pytest.mark.parametrize("n,T,c", [(1, 4096, 64), (2, 1500, 136)])
def test_a_long_sequence_updates_its_states_in_place(n, T, c):
    """The scan in segments and the convolution in many runs, with a state that other
    workgroups read while the last ones are not done."""
    x, _, _ = scan_inputs(n, T, c, 16, 1, BF, 40)
    args = [x[k] for k in ("u", "dt", "A", "B", "C")]
    kw = {k: x[k] for k in ("D", "gate", "dt_bias")}
    y, st = mlstm.scan_fwd(*args, state=x["state"], **kw)
    kept = x["state"].clone()
    y2, st2 = mlstm.scan_fwd(*args, state=kept, out_state=kept, **kw)
    assert st2 is kept and torch.equal(y, y2) and torch.equal(st, kept)
    w, state = gpu(np.random.default_rng(41).normal(size=(c, 4))), x["u"][:, :3].clone()
    if n == 1:  # the first rows of x themselves
        with pytest.raises(mlstm.MlstmError, match="overlap"):
            mlstm.short_conv_fwd(x["u"], w, state=state, out_state=x["u"][:, :3])
    y, st = mlstm.short_conv_fwd(x["u"], w, state=state)
    y2, st2 = mlstm.short_conv_fwd(x["u"], w, state=state, out_state=state)
    assert st2 is state and torch.equal(y, y2) and torch.equal(st, state)


def _scan_call():
    x, dy, dst = scan_inputs(2, 9, 32, 4, 1, FP, 42)
    return mlstm.scan_bwd, dict(x, dy=dy, dstate=dst, lengths=i32([9, 4]))


def _conv_call():
    r = np.random.default_rng(43)
    z = lambda *s: gpu(r.normal(size=s))
    return mlstm.short_conv_bwd, dict(x=z(2, 9, 16), weight=z(16, 4), dy=z(2, 1, 9, 16),
                                      bias=z(16), state=z(2, 3, 16), dstate=z(2, 3, 16),
                                      lengths=i32([9, 4]), heads=1)


@pytest.mark.parametrize("call", [_scan_call, _conv_call])
def test_each_tensor_is_checked_among_gpu_tensors(call):
    f, good = call()
    f(**good)
    tensors = [k for k, v in good.items() if isinstance(v, torch.Tensor)]
    first = tensors[0]  # its device and type are the call's
    for k in tensors:
        if k != first:
            with pytest.raises(ValueError, match=f"{k} "):
                f(**{**good, k: good[k].cpu()})
        with pytest.raises((TypeError, ValueError)):
            f(**{**good, k: good[k].double()})
        wide = torch.stack([good[k], good[k]], -1)[..., 0]  # every second element
        with pytest.raises(ValueError, match="contiguous"):
            f(**{**good, k: wide})
