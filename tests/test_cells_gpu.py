"""The gated delta rule and the block norm on the GPU against the float64 oracle.

Tolerances.  A float32 result: each of the products that lead to it sums at
most 1024 terms in float32 with errors of either sign, sqrt(1024) 2^-24 = 2^-19
of the sum's size, and four such products follow one another in a chunk
(memory, inverse, scores, memory): 2 * 2^-19 = 2^-18 in the 2-norm, and at most
2^-14 of the root mean square at one element.  A bf16 result: that is below the
one rounding, 2^-8 of the value at most, and the operands of h, dq and dk that
are not inputs carry 16 bits, 2^-16 each: 2^-8 + 2^-12 in the 2-norm, 2^-8 of
the value plus 2^-10 of the root mean square at one element.

"The sum's size" above is the root of the sum of squares of its terms: after j
of n terms of size a and either sign a partial sum is about sqrt(j) a, each
addition is off by up to 2^-24 of that, and n such errors of either sign make
2^-24 n a = sqrt(n) 2^-24 of the size sqrt(n) a.  For most results that is their
own size.  A gate's gradient is a single number, the sum of up to 1024 x 512
products of a memory and its gradient, and may come out far below its size
(a sum of 256 terms of 0.05 that came out at 0.0014 was off by 1e-8, 2^-26 of the
size): dbeta and dfgate are held to their terms' size.
"""
import numpy as np
import pytest
import torch

import oracle
from linear_recurrent_sequence_amd import mlstm

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAMES = ("dq", "dk", "dv", "dbeta", "dfgate", "dstate")


def host(t):
    return t.detach().double().cpu().numpy()


def close(name, t, ref, size=None):
    a, ref = host(t), np.asarray(ref)
    assert a.shape == ref.shape, name
    assert np.isfinite(a).all(), name
    size = np.abs(ref) if size is None else np.maximum(np.abs(ref), size)
    rms, err = np.sqrt((size ** 2).mean()), np.abs(a - ref)
    bf16 = t.dtype == torch.bfloat16
    norm = np.linalg.norm(err) / max(np.linalg.norm(size), 1e-30)
    assert norm <= (2 ** -8 + 2 ** -12 if bf16 else 2 ** -18), (name, norm)
    most = np.abs(ref) * 2 ** -8 + rms * 2 ** -10 if bf16 else rms * 2 ** -14
    assert (err <= most + 1e-30).all(), (name, (err / (most + 1e-30)).max())


def inputs(B, NHK, NH, T, dk, dv, dtype, seed=0, forget="sigmoid", common=0.5, fmean=3.0):
    """Unit keys with a common part; float64 copies of the rounded values for the oracle."""
    rng = np.random.default_rng(seed)
    n = rng.standard_normal
    k = n((B, NHK, T, dk)) + common * n((1, NHK, 1, dk))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    f = fmean + 1.5 * n((B, NH, T))
    if forget == "exp":
        f = -np.log1p(np.exp(-f))
    half = (n((B, NHK, T, dk)), k, n((B, NH, T, dv)), n((B, NH, T, dv)))
    full = (rng.uniform(0, 1, (B, NH, T)), f, n((B, NH, dv, dk)), n((B, NH, dv, dk)))
    q, k, v, dh = (torch.tensor(x, device=DEV).to(dtype) for x in half)
    beta, fgate, C0, dC = (torch.tensor(x, device=DEV).float() for x in full)
    return (q, k, v, beta, fgate), C0, dh, dC


def oracle_of(args, C0, forget="sigmoid"):
    return oracle.delta_forward(*map(host, args), None if C0 is None else host(C0), forget)


def delta_ref(args, dh, C0, dC, forget="sigmoid"):
    """For each gradient (reference, size of its sum's terms or None)."""
    *ref, db_size, df_size = oracle.delta_backward(
        *map(host, args), host(dh), None if C0 is None else host(C0),
        None if dC is None else host(dC), forget, sizes=True)
    return list(zip(ref, (None, None, None, db_size, df_size, None)))


BF, FP = torch.bfloat16, torch.float32
SHAPES = [
    # B, NHK, NH, T, dk, dv, dtype, forget
    (1, 1, 1, 1, 16, 16, BF, "sigmoid"),
    (1, 1, 1, 2, 16, 16, FP, "sigmoid"),
    (2, 1, 2, 63, 32, 48, BF, "exp"),
    (1, 2, 2, 64, 48, 32, FP, "exp"),
    (1, 2, 6, 65, 64, 80, BF, "sigmoid"),
    (3, 1, 1, 127, 80, 64, FP, "sigmoid"),
    (1, 4, 8, 129, 128, 128, BF, "sigmoid"),
    (1, 1, 3, 130, 112, 96, FP, "sigmoid"),
    (1, 1, 1, 191, 192, 208, BF, "exp"),
    (1, 1, 2, 100, 256, 144, FP, "sigmoid"),
    (2, 2, 2, 70, 272, 16, BF, "sigmoid"),
    (1, 1, 1, 66, 384, 400, BF, "sigmoid"),
    (1, 1, 1, 65, 512, 32, FP, "exp"),
    (1, 1, 1, 65, 512, 1024, BF, "sigmoid"),
    (2, 2, 4, 300, 96, 160, FP, "exp"),
]


@pytest.mark.parametrize("B,NHK,NH,T,dk,dv,dtype,forget", SHAPES)
@pytest.mark.parametrize("with_state", [True, False])
def test_delta_forward(B, NHK, NH, T, dk, dv, dtype, forget, with_state):
    args, C0, _, _ = inputs(B, NHK, NH, T, dk, dv, dtype, 1, forget)
    C0 = C0 if with_state else None
    h, C = mlstm.delta_fwd(*args, state=C0, forget=forget)
    hr, Cr = oracle_of(args, C0, forget)
    assert h.dtype == dtype and C.dtype == FP
    close("h", h, hr)
    close("C", C, Cr)
    if with_state:  # in place
        kept = C0.clone()
        h2, C2 = mlstm.delta_fwd(*args, state=kept, out_state=kept, forget=forget)
        assert C2 is kept and torch.equal(h2, h) and torch.equal(kept, C)


@pytest.mark.parametrize("B,NHK,NH,T,dk,dv,dtype,forget", SHAPES)
@pytest.mark.parametrize("with_state", [True, False])
def test_delta_backward(B, NHK, NH, T, dk, dv, dtype, forget, with_state):
    args, C0, dh, dC = inputs(B, NHK, NH, T, dk, dv, dtype, 2, forget)
    C0, dC = (C0, dC) if with_state else (None, None)
    got = mlstm.delta_bwd(*args, dh, state=C0, dstate=dC, forget=forget)
    ref = delta_ref(args, dh, C0, dC, forget)
    for name, a, b in zip(NAMES, got, ref):
        if not with_state and T == 1 and name == "dfgate":
            assert not a.any()  # nothing to forget
            continue
        close(name, a, *b)
    again = mlstm.delta_bwd(*args, dh, state=C0, dstate=dC, forget=forget)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


# the chains of the backward run one after the other where side by side takes no
# fewer rounds of workgroups: 129 to 256 of them
@pytest.mark.parametrize("B,NHK,NH,T,dk,dv,dtype,forget", [
    (2, 5, 35, 131, 32, 80, BF, "sigmoid"), (9, 2, 16, 66, 16, 16, FP, "exp"),
    (1, 3, 33, 65, 112, 272, BF, "exp"), (1, 33, 33, 67, 48, 272, FP, "sigmoid")])
def test_delta_backward_of_many_heads(B, NHK, NH, T, dk, dv, dtype, forget):
    test_delta_backward(B, NHK, NH, T, dk, dv, dtype, forget, True)


@pytest.mark.parametrize("NHK,NH,dk,dv,dtype,forget", [
    (4, 4, 64, 64, BF, "sigmoid"), (1, 3, 16, 48, FP, "exp"), (2, 2, 272, 80, FP, "sigmoid"),
    (1, 2, 512, 1024, BF, "exp"), (1, 1, 80, 16, BF, "sigmoid"), (2, 4, 128, 128, BF, "sigmoid")])
def test_delta_steps(NHK, NH, dk, dv, dtype, forget):
    """Token after token, in place, against the oracle and (the chunked kernel) a whole call."""
    args, C0, _, _ = inputs(2, NHK, NH, 9, dk, dv, dtype, 3, forget)
    hr, Cr = oracle_of(args, C0, forget)
    C, hs = C0.clone(), []
    for t in range(9):
        tok = [x[:, :, t].contiguous() for x in args]
        other = torch.empty_like(C)
        h2, _ = mlstm.delta_step(*tok, C, out_state=other, forget=forget)
        h, C_same = mlstm.delta_step(*tok, C, forget=forget)
        assert C_same is C and torch.equal(C, other) and torch.equal(h, h2)
        hs.append(h)
    close("h", torch.stack(hs, 2), hr)
    close("C", C, Cr)
    h, C = mlstm.delta_fwd(*args, state=C0, forget=forget)
    close("h", h, hr)
    close("C", C, Cr)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_delta_padding_leaves_the_memory(dtype):
    """beta = 0 and f = 1 behind each sequence's end: the memory is that of the sequence alone."""
    args, C0, dh, dC = inputs(3, 2, 4, 200, 48, 32, dtype, 4)
    q, k, v, beta, fgate = (x.clone() for x in args)
    lengths = [200, 77, 1]
    for b, n in enumerate(lengths):
        beta[b, :, n:] = 0.0
        fgate[b, :, n:] = float("inf")
    h, C = mlstm.delta_fwd(q, k, v, beta, fgate, state=C0)
    assert torch.isfinite(h).all()
    for b, n in enumerate(lengths):
        part = [x[b:b + 1, :, :n].contiguous() for x in args]
        hb, Cb = mlstm.delta_fwd(*part, state=C0[b:b + 1].contiguous())
        close("C", C[b:b + 1], host(Cb))
        close("h", h[b:b + 1, :, :n], host(hb))
        if n > 1:  # one token takes the step kernel
            assert torch.equal(C[b:b + 1], Cb) and torch.equal(h[b:b + 1, :, :n], hb)
    # the gradients of a padded batch, with nothing asked of the padding
    for b, n in enumerate(lengths):
        dh[b, :, n:] = 0.0
    got = mlstm.delta_bwd(q, k, v, beta, fgate, dh, state=C0, dstate=dC)
    for b, n in enumerate(lengths):
        part = [x[b:b + 1, :, :n].contiguous() for x in args]
        ref = delta_ref(part, dh[b:b + 1, :, :n], C0[b:b + 1], dC[b:b + 1])
        for name, a, r in zip(NAMES, got, ref):
            a = a[b:b + 1]
            close(name, a if name == "dstate" else a[:, :, :n], *r)
            if name in ("dq", "dk", "dv"):
                assert not a[:, :, n:].any()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("forget,value", [("sigmoid", -np.inf), ("sigmoid", -3e4), ("exp", -np.inf),
                                          ("exp", -200.0)])
def test_delta_forgets_everything(dtype, forget, value):
    """f = 0 at tokens 0, 70 and 71: what came before is gone, and no NaN comes of it."""
    args, C0, dh, dC = inputs(1, 1, 2, 150, 32, 32, dtype, 5, forget)
    fgate = args[4]
    for t in (0, 70, 71):
        fgate[:, :, t] = value
    h, C = mlstm.delta_fwd(*args, state=C0, forget=forget)
    hr, Cr = oracle_of(args, C0, forget)
    close("h", h, hr)
    close("C", C, Cr)
    got = mlstm.delta_bwd(*args, dh, state=C0, dstate=dC, forget=forget)
    for name, a, r in zip(NAMES[:5], got, delta_ref(args, dh, C0, dC, forget)):
        close(name, a, *r)
    assert not got[5].any()  # nothing of the first memory is kept


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("what", ["same keys", "no writes", "full writes", "no decay", "long range"])
def test_delta_extremes(dtype, what):
    T = 140 if what != "long range" else 700
    args, C0, dh, dC = inputs(1, 1, 2, T, 64, 32, dtype, 6)
    q, k, v, beta, fgate = args
    if what == "same keys":
        k[:] = k[:, :, :1]
    elif what == "no writes":
        beta.zero_()
    elif what == "full writes":
        beta.fill_(1.0)
    elif what == "no decay":
        fgate.fill_(float("inf"))
    else:
        fgate.fill_(12.0)
    h, C = mlstm.delta_fwd(*args, state=C0)
    hr, Cr = oracle_of(args, C0)
    close("h", h, hr)
    close("C", C, Cr)
    got = mlstm.delta_bwd(*args, dh, state=C0, dstate=dC)
    for name, a, r in zip(NAMES, got, delta_ref(args, dh, C0, dC)):
        if what == "no decay" and name == "dfgate":
            assert not a.any()  # sigma(-inf) = 0
            continue
        if what == "no writes" and name in ("dk", "dv"):
            assert not a.any()
            continue
        close(name, a, *r)


def test_delta_gradients_by_differences():
    """Directional differences of the float32 forward: its error, 2^-18 of the
    loss's size over a step of 2^-6, and the step's own cubic term, leave 1%."""
    args, C0, dh, dC = inputs(1, 1, 2, 90, 32, 32, FP, 7)
    grads = mlstm.delta_bwd(*args, dh, state=C0, dstate=dC)
    rng = torch.Generator(device=DEV).manual_seed(0)
    for i, g in enumerate(grads):
        x = [t.clone() for t in (*args, C0)]
        to = torch.randn(x[i].shape, generator=rng, device=DEV)
        to = to / to.norm() + g / g.norm()  # with a part along the gradient
        value = []
        for step in (2.0 ** -6, -2.0 ** -6):
            y = list(x)
            y[i] = x[i] + step * to
            h, C = mlstm.delta_fwd(*y[:5], state=y[5])
            value.append((h.double() * dh).sum() + (C.double() * dC).sum())
        slope, want = (value[0] - value[1]) / 2.0 ** -5, (g.double() * to).sum()
        assert abs(slope - want) <= 0.01 * abs(want), NAMES[i]


@pytest.mark.parametrize("dtype", [BF, FP])
def test_delta_in_two_calls(dtype):
    """A sequence in two calls: at a chunk's border bitwise the one call, elsewhere near it."""
    args, C0, _, _ = inputs(2, 1, 2, 192, 64, 48, dtype, 8)
    h, C = mlstm.delta_fwd(*args, state=C0)
    for cut in (128, 100):
        a = [x[:, :, :cut].contiguous() for x in args]
        b = [x[:, :, cut:].contiguous() for x in args]
        h1, C1 = mlstm.delta_fwd(*a, state=C0)
        h2, C2 = mlstm.delta_fwd(*b, state=C1)
        if cut % 64 == 0:
            assert torch.equal(torch.cat([h1, h2], 2), h) and torch.equal(C2, C)
        hr, Cr = oracle_of(args, C0)
        close("h", torch.cat([h1, h2], 2), hr)
        close("C", C2, Cr)


@pytest.mark.parametrize("NHK,NH,T,dk,dv,dtype,forget", [
    (1, 1, 1500, 64, 64, BF, "sigmoid"), (1, 2, 2113, 48, 80, FP, "exp"),
    (1, 1, 1600, 272, 16, BF, "exp"), (2, 4, 3001, 112, 96, BF, "sigmoid"),
    (1, 1, 2048, 512, 32, FP, "sigmoid"), (1, 1, 4160, 16, 144, FP, "sigmoid")])
def test_delta_long_sequences_in_segments(NHK, NH, T, dk, dv, dtype, forget):
    """Few heads and many chunks: the sequence is cut into segments.  In place
    too, where the last segment writes what the first one starts from."""
    args, C0, _, _ = inputs(1, NHK, NH, T, dk, dv, dtype, 15, forget, fmean=6.0)
    hr, Cr = oracle_of(args, C0, forget)
    h, C = mlstm.delta_fwd(*args, state=C0, forget=forget)
    close("h", h, hr)
    close("C", C, Cr)
    kept = C0.clone()
    h2, _ = mlstm.delta_fwd(*args, state=kept, out_state=kept, forget=forget)
    assert torch.equal(h2, h) and torch.equal(kept, C)
    h0, C1 = mlstm.delta_fwd(*args, forget=forget)
    zero, _ = mlstm.delta_fwd(*args, state=torch.zeros_like(C0), forget=forget)
    assert torch.equal(h0, zero)


def test_delta_keeps_heads_and_earlier_chunks_apart():
    """A NaN at one token reaches neither other heads nor earlier chunks."""
    args, C0, _, _ = inputs(2, 2, 4, 200, 32, 32, BF, 9)
    h, C = mlstm.delta_fwd(*args, state=C0)
    v = args[2].clone()
    v[0, 1, 130, 3] = float("nan")
    h2, C2 = mlstm.delta_fwd(args[0], args[1], v, *args[3:], state=C0)
    assert torch.isnan(h2[0, 1, 130, 3]) and torch.isnan(C2[0, 1]).any()
    assert torch.equal(h2[0, 1, :128], h[0, 1, :128])
    h2[0, 1], C2[0, 1] = h[0, 1], C[0, 1]
    assert torch.equal(h2, h) and torch.equal(C2, C)


def test_delta_writes_only_its_outputs():
    """Outputs that lie inside larger buffers: nothing around them changes."""
    args, C0, dh, _ = inputs(1, 1, 2, 75, 48, 32, BF, 10)
    n = C0.numel()
    buf = torch.full((n + 128,), 7.0, device=DEV)
    out = buf[64:64 + n].view_as(C0)
    mlstm.delta_fwd(*args, state=C0, out_state=out)
    assert (buf[:64] == 7).all() and (buf[64 + n:] == 7).all()
    tok = [x[:, :, 0].contiguous() for x in args]
    mlstm.delta_step(*tok, C0, out_state=out)
    assert (buf[:64] == 7).all() and (buf[64 + n:] == 7).all()


def test_delta_past_32_bit_offsets():
    """Memories and values of more than 2^31 elements: the last heads are right."""
    H = 140000
    C = torch.empty((H, 1, 128, 128), device=DEV)
    C[-1].normal_()
    last = C[-1:].clone()
    args, _, _, _ = inputs(1, 1, 1, 1, 128, 128, BF, 11)
    tok = [x[:, :, 0].expand(H, *x.shape[1:2], *x.shape[3:]).contiguous() for x in args]
    C[:-1] = 0.0
    h, C = mlstm.delta_step(*tok, C)
    hr, Cr = oracle_of(args, last)
    close("h", h[-1:], hr[:, :, 0])
    close("C", C[-1:], Cr)
    del C, h, tok
    args, C0, _, _ = inputs(1, 1, 1, 2100, 16, 1024, BF, 12)
    big = [x.expand(1024, *x.shape[1:]).contiguous() for x in args]
    h, C = mlstm.delta_fwd(*big)
    one, C1 = mlstm.delta_fwd(*args)
    assert torch.equal(h[-1:], one) and torch.equal(C[-1:], C1)
    assert torch.equal(h[500:501], one)
    close("C", C1, oracle_of(args, None)[1])
    del big, h
    torch.cuda.empty_cache()


def test_delta_step_of_more_heads_than_a_sequence_may_have():
    """2^18 heads: one token is given no chunks, and takes them."""
    B, NH, dk, dv = 1 << 17, 2, 16, 16
    gen = torch.Generator(device=DEV).manual_seed(9)
    rand = lambda *shape: torch.randn(shape, device=DEV, generator=gen)  # noqa: E731
    k = torch.nn.functional.normalize(rand(B, 1, dk), dim=-1).to(BF)
    args = rand(B, 1, dk).to(BF), k, rand(B, NH, dv).to(BF), rand(B, NH).sigmoid(), rand(B, NH) + 3
    C0 = rand(B, NH, dv, dk)
    h, C = mlstm.delta_step(*args, C0, out_state=torch.empty_like(C0))
    pick = torch.tensor([0, 1, 65535, 65536, B - 1], device=DEV)
    hr, Cr = oracle_of([x[pick].unsqueeze(2) for x in args], C0[pick])
    close("h", h[pick], hr[:, :, 0])
    close("C", C[pick], Cr)
    h2, C2 = mlstm.delta_fwd(*(x.unsqueeze(2) for x in args), state=C0)
    assert torch.equal(h2[:, :, 0], h) and torch.equal(C2, C)
    with pytest.raises(mlstm.MlstmError):
        mlstm.delta_fwd(*(x.unsqueeze(2).repeat_interleave(2, 2) for x in args))


def test_delta_on_other_streams_and_in_graphs():
    """Two calls at once on two streams, and captured forward and backward passes
    replayed with new inputs and eager work in between, against eager calls."""
    a = inputs(2, 2, 4, 150, 64, 48, BF, 13)
    b = inputs(1, 1, 2, 200, 32, 64, FP, 14)

    def both(x):
        args, C0, dh, dC = x
        return (*mlstm.delta_fwd(*args, state=C0),
                *mlstm.delta_bwd(*args, dh, state=C0, dstate=dC))

    want = both(a), both(b)
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        got = []
        for s, x in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                got.append(both(x))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(g, w))
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for gr, x in zip(graphs, (a, b)):
        with torch.cuda.graph(gr):
            outs.append(both(x))
    for seed in (13, 20, 21, 13):
        for x in (inputs(2, 2, 4, 150, 64, 48, BF, seed),):
            for old, new in zip((*a[0], *a[1:]), (*x[0], *x[1:])):
                old.copy_(new)
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for x, got in zip((a, b), outs):
            assert all(torch.equal(p, q) for p, q in zip(got, both(x)))
        torch.cuda.synchronize()


# ----------------------------------------------------------------- block norm

NORM_SHAPES = [
    # B, NH, T, d, dtype, norm, activation, gate, residual, scale, next
    (1, 1, 1, 8, BF, "layer", "sigmoid", 1, 1, 1, 1),
    (2, 3, 5, 16, FP, "rms", "silu", 1, 0, 0, 1),
    (3, 4, 7, 384, BF, "layer", "sigmoid", 1, 1, 1, 1),
    (1, 16, 33, 128, FP, "rms", "silu", 1, 0, 0, 1),
    (2, 8, 9, 512, BF, "layer", "silu", 1, 1, 1, 1),
    (2, 5, 11, 40, FP, "layer", "sigmoid", 0, 1, 0, 1),
    (1, 7, 13, 72, BF, "rms", "sigmoid", 1, 1, 1, 0),
    (1, 2, 6, 96, FP, "layer", "silu", 1, 0, 1, 0),
    (1, 15, 3, 520, FP, "layer", "sigmoid", 1, 1, 1, 1),
    (1, 3, 4, 1032, BF, "rms", "silu", 1, 1, 1, 1),
    (2, 3, 5, 2056, FP, "layer", "sigmoid", 1, 1, 1, 1),
    (3, 1, 2, 8192, BF, "layer", "sigmoid", 1, 1, 1, 1),
    (1, 1, 3, 4104, FP, "rms", "silu", 0, 1, 1, 1),
    (1, 1024, 2, 8, FP, "layer", "sigmoid", 1, 1, 1, 1),
    (1, 31, 2, 264, FP, "rms", "sigmoid", 1, 1, 1, 1),
    (1, 1, 2500, 64, BF, "layer", "sigmoid", 0, 0, 0, 0),
    (2, 2, 3000, 48, FP, "layer", "silu", 1, 1, 1, 1),
    (2, 12, 3, 264, BF, "layer", "sigmoid", 1, 1, 1, 1),
    (1, 7, 3, 1032, FP, "layer", "silu", 1, 1, 1, 1),
]


def norm_inputs(B, NH, T, d, dtype, norm, activation, gate, residual, scale, nxt, seed=0):
    rng = np.random.default_rng(seed)
    n, D = rng.standard_normal, NH * d

    def half(*s):
        return torch.tensor(n(s), device=DEV).to(dtype)

    def weight():
        return torch.tensor(1 + 0.3 * n(D), device=DEV).float()

    p = half(B, NH, T, d) + half(1, NH, 1, d)
    kw = dict(gate=half(B, NH, T, d) * 2 if gate else None,
              residual=half(B, T, D) if residual else None, scale=weight() if scale else None,
              next_weight=weight() if nxt else None, norm=norm, activation=activation)
    return p, weight(), kw, half(B, T, D), half(B, T, D) if nxt else None


def host_kw(kw):
    return {k: host(x) if torch.is_tensor(x) else x for k, x in kw.items()}


@pytest.mark.parametrize("case", NORM_SHAPES, ids=lambda c: "-".join(map(str, c)))
def test_block_norm(case):
    p, w, kw, dr, dy = norm_inputs(*case)
    r, y = mlstm.block_norm_fwd(p, w, **kw)
    rr, yr = oracle.block_norm(host(p), host(w), **host_kw(kw))
    close("r", r, rr)
    assert (y is None) == (yr is None)
    if y is not None:
        close("y", y, yr)
    for d_r in (dr, None) if dy is not None else (dr,):
        got = mlstm.block_norm_bwd(p, w, d_r, dy, **kw)
        ref = oracle.block_norm(host(p), host(w), **host_kw(kw),
                                dr=None if d_r is None else host(d_r),
                                dy=None if dy is None else host(dy), grads=True)
        assert set(got) == set(ref)
        for name in ref:
            close(name, got[name], ref[name])
        again = mlstm.block_norm_bwd(p, w, d_r, dy, **kw)
        assert all(torch.equal(got[n], again[n]) for n in got)


@pytest.mark.parametrize("norm", ["layer", "rms"])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_block_norm_extremes(norm, dtype):
    """Constant and zero rows (eps alone), rows far from zero, and gates at both ends."""
    p, w, kw, dr, dy = norm_inputs(1, 2, 8, 64, dtype, norm, "silu", 1, 1, 1, 1, 3)
    p[0, 0, 0] = 0.0
    p[0, :, 1] = 3.0
    p[0, :, 2] += 1000.0
    kw["gate"][0, :, 3] = 60.0
    kw["gate"][0, :, 4] = -60.0
    kw["gate"][0, :, 5] = -3e4
    kw["residual"][0, 6] += 500.0
    r, y = mlstm.block_norm_fwd(p, w, **kw)
    rr, yr = oracle.block_norm(host(p), host(w), **host_kw(kw))
    close("r", r, rr)
    got = mlstm.block_norm_bwd(p, w, dr, dy, **kw)
    ref = oracle.block_norm(host(p), host(w), **host_kw(kw), dr=host(dr), dy=host(dy), grads=True)
    for t in range(8):
        if dtype == FP and t in (2, 6) and norm == "layer":
            # values of a (1000, 500) whose spread is 1: each difference carries
            # 2^-24 of a, a 2^-24 of the spread
            assert np.abs(host(y[0, t]) - yr[0, t]).max() <= 1000 * 2 ** -22
            continue
        close("y", y[:, t], yr[:, t])
        for name in ("dgate", "dp"):
            a, b = got[name][:, :, t], ref[name][:, :, t]
            if np.abs(b).max() < 1e-20 or (name == "dp" and t in (0, 1, 2)):
                assert torch.isfinite(a).all()
                continue
            close(name, a, b)


def test_block_norm_keeps_rows_apart():
    p, w, kw, _, _ = norm_inputs(2, 4, 9, 96, BF, "layer", "sigmoid", 1, 1, 1, 1)
    r, y = mlstm.block_norm_fwd(p, w, **kw)
    bad = p.clone()
    bad[1, 2, 4, 5] = float("nan")
    bad[0, 0, 0, 0] = float("inf")
    r2, y2 = mlstm.block_norm_fwd(bad, w, **kw)
    assert torch.isnan(y2[1, 4]).all() and torch.isnan(r2[1, 4, 192:288]).all()
    assert torch.equal(r2[1, 4, :192], r[1, 4, :192])
    keep = torch.ones((2, 9), dtype=torch.bool, device=DEV)
    keep[1, 4] = keep[0, 0] = False
    assert torch.equal(r2[keep], r[keep]) and torch.equal(y2[keep], y[keep])


def test_block_norm_past_32_bit_offsets():
    T = (1 << 31) // 512 + 5
    p = torch.empty((1, 2, T, 256), dtype=BF, device=DEV)
    p[:, :, :8].normal_()
    p[:, :, 8:] = p[:, :, 7:8]
    p[:, :, -8:].normal_()
    w = torch.rand(512, device=DEV)
    r, _ = mlstm.block_norm_fwd(p, w)
    for cut in (slice(0, 8), slice(T - 8, T)):
        close("r", r[:, cut], oracle.block_norm(host(p[:, :, cut]), host(w))[0])
    g = mlstm.block_norm_bwd(p, w, r, None)
    ref = oracle.block_norm(host(p[:, :, -8:]), host(w), dr=host(r[:, -8:]), grads=True)
    close("dp", g["dp"][:, :, -8:], ref["dp"])
    del p, r, g
    torch.cuda.empty_cache()


def test_block_norm_on_other_streams_and_in_graphs():
    cases = [norm_inputs(*NORM_SHAPES[2]), norm_inputs(*NORM_SHAPES[16])]

    def both(c):
        p, w, kw, dr, dy = c
        g = mlstm.block_norm_bwd(p, w, dr, dy, **kw)
        return [*mlstm.block_norm_fwd(p, w, **kw), *(g[n] for n in sorted(g))]

    want = [both(c) for c in cases]
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for s, c in zip(streams, cases):
        with torch.cuda.stream(s):
            got.append(both(c))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(g, w))
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for gr, c in zip(graphs, cases):
        with torch.cuda.graph(gr):
            outs.append(both(c))
    for k in range(3):
        cases[0][0].mul_(1.5).add_(0.25 * k)
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for c, o in zip(cases, outs):
            assert all(torch.equal(a, b) for a, b in zip(o, both(c)))


# ------------------------------------------------------------------- together

def test_a_prompt_then_tokens_through_cell_and_norms():
    """delta_fwd over a prompt, delta_step on, block_norm_fwd behind each: the
    outputs of one call over everything."""
    args, _, _, _ = inputs(2, 2, 4, 140, 64, 48, FP, 30)
    p, w, kw, _, _ = norm_inputs(2, 4, 140, 48, FP, "rms", "silu", 1, 1, 1, 1, 31)
    h, C = mlstm.delta_fwd(*(x[:, :, :130].contiguous() for x in args))
    rows = []

    def behind(h, a, b):
        cut = dict(kw, gate=kw["gate"][:, :, a:b].contiguous(),
                   residual=kw["residual"][:, a:b].contiguous())
        return mlstm.block_norm_fwd(h, w, **cut)

    rows.append(behind(h, 0, 130))
    for t in range(130, 140):
        h, C = mlstm.delta_step(*(x[:, :, t].contiguous() for x in args), C)
        rows.append(behind(h.unsqueeze(2), t, t + 1))
    hr, Cr = oracle_of(args, None)
    rr, yr = oracle.block_norm(hr, host(w), **host_kw(kw))
    close("r", torch.cat([r for r, _ in rows], 1), rr)
    close("y", torch.cat([y for _, y in rows], 1), yr)
    close("C", C, Cr)


def test_a_training_step_through_cell_and_norms():
    args, C0, _, dC = inputs(2, 1, 2, 100, 32, 64, FP, 32)
    _, w, kw, dr, dy = norm_inputs(2, 2, 100, 64, FP, "layer", "sigmoid", 1, 1, 1, 1, 33)
    h, C = mlstm.delta_fwd(*args, state=C0)
    r, y = mlstm.block_norm_fwd(h, w, **kw)
    g = mlstm.block_norm_bwd(h, w, dr, dy, **kw)
    grads = mlstm.delta_bwd(*args, g["dp"], state=C0, dstate=dC)
    hr, _ = oracle_of(args, C0)
    ref = oracle.block_norm(hr, host(w), **host_kw(kw), dr=host(dr), dy=host(dy), grads=True)
    for name in ref:
        close(name, g[name], ref[name])
    back = delta_ref(args, torch.tensor(ref["dp"]), C0, dC)
    for name, a, b in zip(NAMES, grads, back):
        close(name, a, *b)


def test_a_block_with_the_mlstm_cell():
    """The mLSTM cell's output through the block norm, as the delta rule's."""
    x = inputs(1, 2, 2, 96, 64, 64, FP, 34)[0]
    igate = torch.randn((1, 2, 96), device=DEV)
    h, _, _ = mlstm.parallel_fwd(x[0], x[1], x[2], igate, x[4])
    p, w, kw, _, _ = norm_inputs(1, 2, 96, 64, FP, "layer", "sigmoid", 1, 1, 1, 1, 35)
    r, y = mlstm.block_norm_fwd(h, w, **kw)
    rr, yr = oracle.block_norm(host(h), host(w), **host_kw(kw))
    close("r", r, rr)
    close("y", y, yr)
