"""How exact the gated delta rule and the block norm are on the GPU, beyond the
tolerances of test_cells_gpu.py, whose inputs and oracle these tests share.  (Those
allow for 16 bits in the operands of bf16 h, dq and dk, which carry 24 now.)

A bf16 result is the float32 one rounded once.  With heads of 64 every sum has
64 terms: float32 errors of either sign make sqrt(64) 2^-24 = 2^-21 of the sum's
size, and four such products follow one another in a chunk, 2 * 2^-21 = 2^-20 in
the 2-norm (e).  Rounded, a value differs from the oracle's rounded value only
where a rounding border lies between the two, which it does with a chance of
e / u, u <= 2^-7 |y| being the step, and then by u: the sum of the squares is
sum e u <= 2^-20 2^-7 |y|^2, 2^-13.5 of y in the 2-norm.
"""
import numpy as np
import pytest
import torch

from linear_recurrent_sequence_amd import mlstm
from test_cells_gpu import BF, DEV, FP, NAMES, delta_ref, host, inputs, oracle_of

pytestmark = pytest.mark.gpu
ONE_ROUNDING = 2 ** -13.5


def rounded_once(name, t, ref):
    want = host(torch.tensor(ref, device=DEV).to(BF))
    off = np.linalg.norm(host(t) - want) / np.linalg.norm(want)
    assert t.dtype == BF and off <= ONE_ROUNDING, (name, off)


@pytest.mark.parametrize("NHK,NH,T,forget", [(2, 4, 500, "sigmoid"), (1, 1, 2100, "exp")])
def test_delta_forward_rounds_once(NHK, NH, T, forget):
    """(1 x 1 x 2100 runs in segments.)"""
    args, C0, _, _ = inputs(2 if T < 1000 else 1, NHK, NH, T, 64, 64, BF, 40, forget)
    h, _ = mlstm.delta_fwd(*args, state=C0, forget=forget)
    rounded_once("h", h, oracle_of(args, C0, forget)[0])


# the first two run the backward's two chains side by side, the third one after the other
@pytest.mark.parametrize("B,NHK,NH,T,forget", [(2, 2, 4, 500, "sigmoid"), (1, 2, 2, 300, "exp"),
                                               (2, 66, 66, 130, "sigmoid")])
def test_delta_backward_rounds_once(B, NHK, NH, T, forget):
    args, C0, dh, dC = inputs(B, NHK, NH, T, 64, 64, BF, 42, forget)
    got = mlstm.delta_bwd(*args, dh, state=C0, dstate=dC, forget=forget)
    ref = delta_ref(args, dh, C0, dC, forget)
    for name, a, (b, _) in list(zip(NAMES, got, ref))[:3]:
        rounded_once(name, a, b)


@pytest.mark.parametrize("B,H,T,d,dtype", [(1, 2, 150, 64, BF), (1, 2, 150, 64, FP),
                                           (2, 66, 70, 32, BF), (2, 66, 70, 32, FP)])
@pytest.mark.parametrize("forget,fmean", [("sigmoid", 0.0), ("sigmoid", -6.0), ("exp", -3.0),
                                          ("exp", -16.0)])
def test_delta_gate_gradients_where_little_is_kept(B, H, T, d, dtype, forget, fmean):
    """dL/df~_t has f_t as a factor in every term, however small: each one is held
    to the size of its own terms.  (A float32 sum of 64 x 64 terms is within 64 2^-24
    = 2^-18 of that, two such products follow one another, and the largest of
    some thousands of errors is within eight times their size: 2^-14.)  Where f =
    0 it is 0.  (2 x 66 heads run the backward's chains one after the other.)"""
    args, C0, dh, dC = inputs(B, 1, H, T, d, 64, dtype, 43, forget, fmean=fmean)
    args[4][:, :, 40] = args[4][:, :, 64] = -np.inf
    got = mlstm.delta_bwd(*args, dh, state=C0, dstate=dC, forget=forget)[4]
    ref, size = delta_ref(args, dh, C0, dC, forget)[4]
    assert (np.abs(host(got) - ref) <= 2 ** -14 * size).all()
    assert not got[:, :, 40].any() and not got[:, :, 64].any()
