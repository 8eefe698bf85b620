"""Paths of the gated delta rule and the block norm that the shapes of
test_cells_gpu.py do not reach; inputs, oracle and tolerances are that file's.
"""
import numpy as np
import pytest
import torch

import oracle
from linear_recurrent_sequence_amd import mlstm
from test_cells_gpu import (BF, DEV, FP, NAMES, close, delta_ref, host, host_kw, inputs,
                            norm_inputs, oracle_of)

pytestmark = pytest.mark.gpu


def in_segments(NHK, NH, T, dk, dv, dtype):
    """Whether the forward cuts such a sequence: its workspace is then more than
    its chunks' (two of them are never cut)."""
    size = mlstm.load_library().mlstm_delta_workspace_bytes
    code = mlstm.MLSTM_BF16 if dtype == BF else mlstm.MLSTM_FP32
    two = size(1, NHK, NH, 128, dk, dv, code, 0)
    return size(1, NHK, NH, T, dk, dv, code, 0) > two // 2 * -(-T // 64)


# each number of 32-column blocks that the kernels are built for, joins of one and of
# two blocks of 256 rows, ragged last segments and chunks, shared key heads
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("NHK,NH,T,dk,dv,forget", [
    (1, 2, 1100, 16, 144, "exp"), (1, 1, 1500, 64, 16, "sigmoid"), (1, 2, 1801, 176, 32, "exp"),
    (2, 2, 2690, 240, 16, "sigmoid"), (1, 1, 3300, 272, 48, "sigmoid"),
    (1, 1, 5801, 384, 16, "exp"), (1, 2, 6177, 400, 16, "sigmoid"), (1, 1, 9750, 512, 16, "exp")])
def test_delta_segments_of_every_width(NHK, NH, T, dk, dv, dtype, forget):
    assert in_segments(NHK, NH, T, dk, dv, dtype)
    args, C0, _, _ = inputs(1, NHK, NH, T, dk, dv, dtype, 50, forget, fmean=6.0)
    hr, Cr = oracle_of(args, C0, forget)
    h, C = mlstm.delta_fwd(*args, state=C0, forget=forget)
    close("h", h, hr)
    close("C", C, Cr)
    kept = C0.clone()
    h2, _ = mlstm.delta_fwd(*args, state=kept, out_state=kept, forget=forget)
    assert torch.equal(h2, h) and torch.equal(kept, C)
    h3, C3 = mlstm.delta_fwd(*args, forget=forget)
    hr, Cr = oracle_of(args, None, forget)
    close("h", h3, hr)
    close("C", C3, Cr)


# each number of 32-column blocks again, ragged ones (memories whose rows end inside a
# wave's), with the backward's chains side by side (3 heads) and one after the other (130)
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("B,NHK,NH", [(1, 1, 3), (2, 65, 65)])
@pytest.mark.parametrize("dk", [16, 48, 80, 144, 208, 272, 336, 400, 464])
def test_delta_of_every_width(B, NHK, NH, dk, dtype):
    args, C0, dh, dC = inputs(B, NHK, NH, 70, dk, 16, dtype, 58)
    h, C = mlstm.delta_fwd(*args, state=C0)
    hr, Cr = oracle_of(args, C0)
    close("h", h, hr)
    close("C", C, Cr)
    got = mlstm.delta_bwd(*args, dh, state=C0, dstate=dC)
    for name, a, b in zip(NAMES, got, delta_ref(args, dh, C0, dC)):
        close(name, a, *b)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("with_state,with_dstate", [(True, False), (False, True)])
def test_delta_backward_with_one_memory(dtype, with_state, with_dstate):
    args, C0, dh, dC = inputs(2, 1, 2, 100, 48, 32, dtype, 51)
    C0, dC = C0 if with_state else None, dC if with_dstate else None
    got = mlstm.delta_bwd(*args, dh, state=C0, dstate=dC)
    for name, a, b in zip(NAMES, got, delta_ref(args, dh, C0, dC)):
        close(name, a, *b)


def test_delta_backward_without_the_memorys_gradient():
    """The C ABI without dC_out: the other gradients are the same, bit by bit."""
    args, C0, dh, dC = inputs(2, 1, 2, 100, 48, 32, FP, 52)
    want = mlstm.delta_bwd(*args, dh, state=C0, dstate=dC)
    lib, sizes = mlstm.load_library(), (2, 1, 2, 100, 48, 32)
    ws = torch.empty(lib.mlstm_delta_workspace_bytes(*sizes, mlstm.MLSTM_FP32, 1),
                     dtype=torch.uint8, device=DEV)
    out = [torch.empty_like(x) for x in (*args[:3], args[3], args[4])]
    st = lib.mlstm_delta_bwd(*(x.data_ptr() for x in args), C0.data_ptr(), dh.data_ptr(),
                             dC.data_ptr(), *(x.data_ptr() for x in out), None, ws.data_ptr(),
                             ws.numel(), *sizes, mlstm.MLSTM_FP32, 0,
                             torch.cuda.current_stream().cuda_stream)
    assert st == 0 and all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("dtype", [BF, FP])
def test_delta_gates_that_grow_the_memory(dtype):
    """f > 1, as far as a chunk's product of them is a number (e^35 here).  The
    tolerance at one element is meant of results of one size: here a token's are, and
    the root mean square over all tokens is that of the largest few's (2 of 150
    tokens at e^0.55 a token: up to 9 times below theirs), so each token is held to its
    own."""
    args, C0, dh, dC = inputs(1, 1, 2, 150, 48, 32, dtype, 53, "exp")
    rng = np.random.default_rng(54)
    args[4].copy_(torch.tensor(rng.uniform(0.3, 0.8, (1, 2, 150))))
    args[4][:, :, 64:].neg_()
    h, C = mlstm.delta_fwd(*args, state=C0, forget="exp")
    hr, Cr = oracle_of(args, C0, "exp")
    got = mlstm.delta_bwd(*args, dh, state=C0, dstate=dC, forget="exp")
    ref = [(hr, None)] + delta_ref(args, dh, C0, dC, "exp")
    for name, a, (b, size) in zip(("h", *NAMES), (h, *got), ref):
        if name == "dstate":
            close(name, a, b)
            continue
        if size is None:
            size = np.sqrt((b ** 2).mean(-1, keepdims=True))
        err, bf16 = np.abs(host(a) - b), a.dtype == BF
        most = np.abs(b) * 2 ** -8 + size * 2 ** -10 if bf16 else size * 2 ** -14
        assert (err <= most).all(), (name, (err / most).max())
    close("C", C, Cr)


# what torch allocates for a call holds NaN here: nothing is read before it is written
@pytest.mark.parametrize("dtype", [BF, FP])
def test_results_do_not_depend_on_what_the_workspaces_hold(dtype):
    cases = [inputs(*s, dtype, 55) for s in ((2, 2, 2, 70, 272, 16), (1, 2, 4, 200, 48, 80),
                                             (1, 65, 130, 65, 16, 16))]
    long = inputs(1, 1, 1, 1500, 64, 16, dtype, 56)
    norms = [norm_inputs(2, 3, 30, d, dtype, "layer", "silu", 1, 1, 1, 1, 57) for d in (72, 1032)]

    def everything():
        out = [*mlstm.delta_fwd(*long[0], state=long[1])]
        for args, C0, dh, dC in cases:
            out += [*mlstm.delta_fwd(*args, state=C0), *mlstm.delta_fwd(*args)]
            out += [*mlstm.delta_bwd(*args, dh, state=C0, dstate=dC)]
            out += [*mlstm.delta_bwd(*args, dh)]
        for p, w, kw, dr, dy in norms:
            g = mlstm.block_norm_bwd(p, w, dr, dy, **kw)
            out += [*mlstm.block_norm_fwd(p, w, **kw), *(g[n] for n in sorted(g))]
        return out

    want = everything()
    before = torch.are_deterministic_algorithms_enabled()
    torch.use_deterministic_algorithms(True)  # fills what is allocated
    try:
        assert torch.empty(4, device=DEV).isnan().all()
        got = everything()
    finally:
        torch.use_deterministic_algorithms(before)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# ----------------------------------------------------------------- block norm

# every workgroup takes three rows and more, with the rows over several waves (or
# several rows to a workgroup, or both), and not all of them in the last turn
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("NH,d,rows,norm,activation", [
    (4, 384, 5003, "layer", "sigmoid"), (2, 264, 8003, "layer", "silu"),
    (15, 520, 801, "layer", "sigmoid"), (1, 8192, 801, "layer", "sigmoid"),
    (31, 264, 801, "rms", "silu"), (7, 1032, 801, "layer", "silu"), (9, 768, 803, "rms", "sigmoid"),
    (3, 2056, 801, "layer", "sigmoid"), (1, 4096, 803, "rms", "sigmoid"),
    (20, 384, 803, "layer", "silu"), (3, 128, 7001, "layer", "sigmoid")])
def test_block_norm_of_many_rows(NH, d, rows, norm, activation, dtype):
    p, w, kw, dr, dy = norm_inputs(1, NH, rows, d, dtype, norm, activation, 1, 1, 1, 1, 60)
    r, y = mlstm.block_norm_fwd(p, w, **kw)
    rr, yr = oracle.block_norm(host(p), host(w), **host_kw(kw))
    close("r", r, rr)
    close("y", y, yr)
    got = mlstm.block_norm_bwd(p, w, dr, dy, **kw)
    ref = oracle.block_norm(host(p), host(w), **host_kw(kw), dr=host(dr), dy=host(dy), grads=True)
    assert set(got) == set(ref)
    for name in ref:
        close(name, got[name], ref[name])


@pytest.mark.parametrize("norm", ["layer", "rms"])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_block_norm_gradients_of_extreme_rows(norm, dtype):
    """Rows without spread: n1 = 0 exactly and 1 / sqrt(eps) before the gradient.
    Rows far from zero (m = 1000 and 500, spread 1): their mean adds up 64 (128)
    values with at most 12 roundings on the way, so with the layer norm n is off by
    c = 12 * 2^-24 m inv, the same in all of a row (a - mean is exact), and the gradient
    inv (g - n mean(g n) - mean(g)) by inv c (|mean(g n)| + |n mean(g)|) <= 5 c times
    its size, |n| <= 4 here.  The weights' gradients sum eight rows of it."""
    p, w, kw, dr, dy = norm_inputs(1, 2, 8, 64, dtype, norm, "silu", 1, 1, 1, 1, 61)
    p[0, :, 0] = 0.0
    p[0, :, 1] = 3.0
    p[0, :, 2] += 1000.0
    kw["residual"][0, 6] += 500.0
    got = mlstm.block_norm_bwd(p, w, dr, dy, **kw)
    ref = oracle.block_norm(host(p), host(w), **host_kw(kw), dr=host(dr), dy=host(dy), grads=True)

    def far(name, a, b, m):
        a, rms = host(a), np.sqrt((b ** 2).mean())
        rounding = 2 ** -8 * np.abs(b) if got[name].dtype == BF else 0.0
        assert (np.abs(a - b) <= rounding + 5 * 12 * 2 ** -24 * m * rms).all(), name

    for t in range(8):
        for name in ("dp", "dgate", "dresidual"):
            a, b = ((x[:, t] if name == "dresidual" else x[:, :, t]) for x in (got[name], ref[name]))
            if t < 2 and name == "dgate" and not np.abs(b).any():
                assert not a.any()  # n1 = 0
            elif norm == "layer" and t in (2, 6):
                far(name, a, b, 1000.0 if t == 2 else 500.0)
            else:
                close(name, a, b)
    for name in ("dweight", "dscale", "dnext_weight"):
        if norm == "layer":
            far(name, got[name], ref[name], 1000.0)
        else:
            close(name, got[name], ref[name])
