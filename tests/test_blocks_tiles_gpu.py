"""The gated feed-forward in every kind of tiles that its products are taken in: 256 x 256,
128 x 256 and 128 x 128 outputs; all of them whole, all split along their sums, or both;
one to a workgroup, or more. SIZES reach them all for each product and type
(test_blocks_tiles_cpu.py holds them to it; those of test_blocks_gpu.py, many tiles among
them, reach a part); results are compared with the definition in float64.

Tolerances, by the sums' lengths: up to 16400 terms, so a float32 sum is off by up to
sqrt(16400) 2^-24 = 2^-17 of its size (the root of the sum of the squares of its terms),
and three follow one another: 2^-16 in the 2-norm, and eight times that, 2^-13 of the root
mean square of the sizes, at one element. (The gradients' 16 bits behind bf16 results add
2^-17.8.) A bf16 result is rounded once more, by at most 2^-8 of its value.
"""
import ctypes

import pytest
import torch

import oracle
from linear_recurrent_sequence_amd import mlstm
from test_blocks_gpu import BF, DEV, FP, ffn_inputs, host

pytestmark = pytest.mark.gpu

# M, D, F
SIZES = {
    BF: [(65, 8, 8), (65, 5504, 520), (65, 8200, 776), (130, 8200, 5504), (300, 392, 8200),
         (300, 8200, 4104), (520, 8200, 5504), (1000, 8, 4104), (1000, 776, 8200),
         (1000, 8200, 776), (2100, 4104, 2056), (6000, 1288, 8), (8190, 264, 5504),
         (8190, 4104, 264), (12000, 4104, 520), (12000, 8200, 136), (16384, 1288, 520)],
    FP: [(65, 8, 8), (65, 264, 72), (65, 2568, 1544), (65, 8200, 264), (65, 8200, 776),
         (300, 8, 8200), (300, 8200, 776), (300, 8200, 4104), (520, 776, 8200),
         (1500, 4104, 2056), (4200, 136, 5504), (6000, 264, 4104), (6000, 1288, 1288),
         (8190, 1544, 1032), (8190, 4104, 264), (12000, 1288, 8), (12000, 1544, 72)],
}
PRODUCTS = ("forward", "again", "dx", "weights")


def tiles_of(M, D, F, dtype, product):
    """(columns, rows) of a tile, tiles taken whole, tiles split, shares of each."""
    t = (ctypes.c_int64 * 5)()
    st = mlstm.load_library().mlstm_gated_ffn_tiles(
        M, D, F, mlstm.MLSTM_BF16 if dtype == BF else mlstm.MLSTM_FP32, PRODUCTS.index(product), t)
    assert st == 0, mlstm.strerror(st)
    return (t[0], t[1]), *t[2:]


def reference(x, wg, wu, dh):
    """((h, dx, dw_gate, dw_up), the sizes of their sums' terms), float64."""
    x, wg, wu, dh = (t.double() for t in (x, wg, wu, dh))
    g, u = x @ wg.T, x @ wu.T
    s = torch.sigmoid(g)
    dg, du = dh * u * (s * (1.0 + g * (1.0 - s))), dh * (g * s)
    h = g * s * u
    del g, u, s
    outs = h, dg @ wg + du @ wu, dg.T @ x, du.T @ x
    dg, du, x, wg, wu = (t.square_() for t in (dg, du, x, wg, wu))
    sizes = (dg @ wg).add_(du @ wu), dg.T @ x, du.T @ x
    return outs, [torch.full_like(h, h.square().mean().sqrt())] + [t.sqrt_() for t in sizes]


def close(name, t, ref, size):
    err, size = (t.double() - ref).abs(), torch.maximum(ref.abs(), size)
    bf16 = 2.0 ** -8 if t.dtype == BF else 0.0
    norm = (err.norm() / size.norm()).item()
    assert norm <= 2.0 ** -16 + bf16, (name, norm)
    most = size.square().mean().sqrt() * 2.0 ** -13 + ref.abs() * bf16
    assert (err <= most).all(), (name, (err / most).max().item())


def test_the_reference_is_the_oracle():
    f = ffn_inputs(33, 24, 40, FP, 70)
    (h, *grads), (_, *sizes) = reference(*f)
    x, wg, wu, dh = map(host, f)
    ref, ref_sizes = oracle.gated_ffn_grads(x, wg, wu, dh)
    for a, b in zip([h, *grads, *sizes], [oracle.gated_ffn(x, wg, wu), *ref, *ref_sizes]):
        assert abs(host(a) - b).max() < 1e-13 * abs(b).max()


@pytest.mark.parametrize("dtype,M,D,F", [(dt, *s) for dt, sizes in SIZES.items() for s in sizes])
def test_gated_ffn_in_tiles(dtype, M, D, F):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(71)
    x, wg, wu, dh = (torch.randn(s, generator=gen, device=DEV)
                     for s in ((M, D), (F, D), (F, D), (M, F)))
    f = x.to(dtype), (wg * D ** -0.5).to(dtype), (wu * D ** -0.5).to(dtype), dh.to(dtype)
    got = mlstm.gated_ffn_fwd(*f[:3]), *mlstm.gated_ffn_bwd(*f)
    for name, a, ref, size in zip(("h", "dx", "dw_gate", "dw_up"), got, *reference(*f)):
        assert a.dtype == dtype
        close(name, a, ref, size)
