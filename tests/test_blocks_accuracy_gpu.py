"""How exact the feed-forward's bf16 gradients are on the GPU, beyond the tolerances of
test_blocks_gpu.py, whose inputs these tests share.  (Those allow for bf16 operands dg and
du behind dx, dw_gate and dw_up for 512 rows and more; they have 16 bits now.)

A bf16 result is the float32 one rounded once.  dg and du enter their products with 16
bits, off by up to 2^-17 of themselves, 2^-17 / sqrt(3) = 2^-17.8 in the root mean square
and of either sign, so a sum is off by that of its size (the root of the sum of the squares
of its terms).  The sums have up to 2100 terms, float32 errors of sqrt(2100) 2^-24 =
2^-18.5 of their size, and three follow one another: 2^-17.7.  Together 2^-17.2, so
e = 2^-17 in the 2-norm, of a result whose size is its own, as its terms have either sign.
Rounded, a value differs from the oracle's rounded value only where a rounding border
lies between the two, which it does with a chance of e / u, u <= 2^-7 |y| being the step,
and then by u: the sum of the squares is sum e u <= 2^-17 2^-7 |y|^2, 2^-12 of y in the
2-norm.
"""
import numpy as np
import pytest
import torch

import oracle
from linear_recurrent_sequence_amd import mlstm
from test_blocks_gpu import BF, DEV, ffn_inputs, host

pytestmark = pytest.mark.gpu
ONE_ROUNDING = 2 ** -12


def rounded_once(name, t, ref):
    want = host(torch.tensor(ref, device=DEV).to(BF))
    off = np.linalg.norm(host(t) - want) / np.linalg.norm(want)
    assert t.dtype == BF and off <= ONE_ROUNDING, (name, off)


# few and many rows, sums over the rows that are shorter and longer than those over F
@pytest.mark.parametrize("M,D,F", [(500, 264, 520), (512, 264, 520), (1000, 264, 136),
                                   (2100, 328, 1032)])
@pytest.mark.parametrize("activation", ["silu", "gelu"])
def test_ffn_gradients_round_once(M, D, F, activation):
    x, wg, wu, dh = ffn_inputs(M, D, F, BF, 60)
    got = mlstm.gated_ffn_bwd(x, wg, wu, dh, activation)
    refs, _ = oracle.gated_ffn_grads(host(x), host(wg), host(wu), host(dh), activation)
    for name, a, r in zip(("dx", "dw_gate", "dw_up"), got, refs):
        rounded_once(name, a, r)
