"""Paths of the gated delta rule and the block norm that the shapes of
test_cells_gpu.py do not reach; inputs, oracle and tolerances are that file's.
"""
import numpy as np
import pytest
import torch

from linear_recurrent_sequence_amd import mlstm
from test_cells_gpu import (BF, DEV, FP, NAMES, close, delta_ref, host, inputs,
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
