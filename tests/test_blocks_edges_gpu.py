"""Calls of the short convolution, the selective scan and the gated feed-forward at the
ends of what their documentation allows; inputs, oracle and tolerances are those of
test_blocks_gpu.py and test_blocks_tiles_gpu.py.
"""
import numpy as np
import pytest
import torch

from linear_recurrent_sequence_amd import mlstm
from test_blocks_gpu import (BF, DEV, FP, check_scan_grads, close, conv_inputs, ffn_inputs, i32,
                             scan_inputs, scan_ref)
from test_blocks_tiles_gpu import reference

pytestmark = pytest.mark.gpu
ROWS = ("u", "dt", "B", "C", "gate")


def _shifted(t):
    """The same values 16 bytes behind a 256-byte border."""
    if t is None:
        return None
    raw = torch.empty(t.numel() * t.element_size() + 16, dtype=torch.uint8, device=DEV)
    out = raw[16:].view(t.dtype).view(t.shape).copy_(t)
    assert out.data_ptr() % 256 == 16
    return out


def _calls(move, dtype):
    x, w, b, st, dy, dst = map(move, conv_inputs(2, 70, 40, 4, dtype, 80))
    kw = dict(bias=b, state=st)
    yield mlstm.short_conv_fwd(x, w, **kw)
    yield mlstm.short_conv_bwd(x, w, dy, dstate=dst, **kw).values()
    x, dy, dst = scan_inputs(1, 600, 40, 12, 1, dtype, 81)
    x, dy, dst = {k: move(v) for k, v in x.items()}, move(dy), move(dst)
    yield mlstm.scan_fwd(**x)
    yield mlstm.scan_bwd(**x, dy=dy, dstate=dst).values()
    yield mlstm.scan_step(**{k: move(v[:, 0].contiguous()) if k in ROWS else v
                             for k, v in x.items()})
    for M in (5, 70, 300):
        f = list(map(move, ffn_inputs(M, 72, 136, dtype, 82)))
        yield (mlstm.gated_ffn_fwd(*f[:3]), *mlstm.gated_ffn_bwd(*f))


@pytest.mark.parametrize("dtype", [BF, FP])
def test_tensors_that_are_aligned_to_16_bytes_and_no_more(dtype):
    for a, b in zip(_calls(_shifted, dtype), _calls(lambda t: t, dtype)):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


# float32 sums of n terms: sqrt(n) 2^-24 of their size, three of them one after the other;
# 2^20 terms 2^-14 and 2^-12.4, the others below
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("M,D,F", [(1 << 20, 8, 16), (70, 1 << 16, 8), (70, 8, 1 << 16),
                                   (3, 1 << 16, 8), (3, 8, 1 << 16)])
def test_gated_ffn_of_the_largest_sizes(M, D, F, dtype):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(83)
    x, wg, wu, dh = (torch.randn(s, generator=gen, device=DEV)
                     for s in ((M, D), (F, D), (F, D), (M, F)))
    f = x.to(dtype), (wg * D ** -0.5).to(dtype), (wu * D ** -0.5).to(dtype), dh.to(dtype)
    got = mlstm.gated_ffn_fwd(*f[:3]), *mlstm.gated_ffn_bwd(*f)
    bf16 = 2.0 ** -8 if dtype == BF else 0.0
    for name, a, ref, size in zip(("h", "dx", "dw_gate", "dw_up"), got, *reference(*f)):
        err, size = (a.double() - ref).abs(), torch.maximum(ref.abs(), size)
        assert err.norm() <= size.norm() * (2.0 ** -12.4 + bf16), name
        assert (err <= size.square().mean().sqrt() * 2.0 ** -9.4 + ref.abs() * bf16).all(), name


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("T", [30, 700])
def test_scan_of_growing_states(T, dtype):
    """A above zero: e^(A sum Delta) is at most about e^12 here."""
    x, dy, dst = scan_inputs(2, T, 24, 6, 1, dtype, 84)
    x["A"] = x["A"].abs().clamp(max=0.3)
    x["dt_bias"] = x["dt_bias"].clamp(max=-3.0)  # Delta of 0.05 at most, on average
    y, st = mlstm.scan_fwd(**x)
    yr, sr = scan_ref(x)
    close("y", y, yr, np.full_like(yr, np.sqrt((yr ** 2).mean())))
    close("state", st, sr)
    check_scan_grads(mlstm.scan_bwd(**x, dy=dy, dstate=dst), x, dy, dst)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("T", [40, 700])
def test_scan_of_extreme_steps_and_rates(T, dtype):
    """dt of the type's lowest value or minus infinity (no step), rates of float32's lowest
    value (a state of one token), gates that are shut, and padding."""
    x, dy, dst = scan_inputs(2, T, 24, 6, 1, dtype, 85, slow=0.1)
    low, lengths = torch.finfo(dtype).min, [T, T // 2 + 3]
    x["dt"][:, 3:T // 2:4], x["dt"][:, 5:T // 2:4] = low, float("-inf")
    x["gate"][:, ::7] = low
    x["A"][3], x["A"][4], x["A"][5, :3] = torch.finfo(FP).min, 0.0, -(2.0 ** 100)
    y, st = mlstm.scan_fwd(**x, lengths=i32(lengths))
    g = mlstm.scan_bwd(**x, dy=dy, dstate=dst, lengths=i32(lengths))
    with np.errstate(over="ignore"):
        yr, sr = scan_ref(x, lengths)
        close("y", y, yr, np.full_like(yr, np.sqrt((yr ** 2).mean())))
        close("state", st, sr)
        check_scan_grads(g, x, dy, dst, lengths)
    assert not g["ddt"][:, 3:T // 2:4].any() and not g["ddt"][:, 5:T // 2:4].any()
    # a token of a sequence whose length is 0, and one of no step
    one = {k: v[:, 3].contiguous() if k in ROWS else v.clone() for k, v in x.items()}
    kept = one["state"].clone()
    y, st = mlstm.scan_step(**one)
    assert torch.equal(st, kept) and y.isfinite().all()
    y, st = mlstm.scan_fwd(**{k: v[:, :1].contiguous() if k in ROWS else v for k, v in x.items()},
                           lengths=i32([0, 0]))
    assert torch.equal(st, kept) and not y.any()


@pytest.mark.parametrize("dtype", [BF, FP])
def test_one_token_of_a_long_batch(dtype):
    """Rows that are a whole sequence apart, 2^24 elements: a position of every sequence."""
    n, pitch = 3, 1 << 24
    wide = torch.empty(n, pitch, device=DEV, dtype=dtype)
    x, _, _ = scan_inputs(n, 1, 40, 5, 1, dtype, 86)
    one = {k: v[:, 0].contiguous() if k in ROWS else v for k, v in x.items()}
    far, at = dict(one), 0
    for k in ROWS:
        c = one[k].flatten(1).shape[1]
        far[k] = wide[:, at:at + c].copy_(one[k].flatten(1)).view(one[k].shape)
        assert far[k].stride(0) == pitch
        at += c + 8 - c % 8
    ref, got = (mlstm.scan_step(**{**v, "state": x["state"].clone()}) for v in (one, far))
    assert all(torch.equal(a, r) for a, r in zip(got, ref))
    _, w, b, st, _, _ = conv_inputs(n, 1, 40, 4, dtype, 87)
    ref, got = (mlstm.short_conv_step(u, w, st.clone(), bias=b) for u in (one["u"], far["u"]))
    assert all(torch.equal(a, r) for a, r in zip(got, ref))
    with pytest.raises(mlstm.MlstmError, match="pitch"):  # a sequence's rows
        mlstm.scan_fwd(**{k: v.unsqueeze(0) if k in ROWS else v for k, v in far.items()
                          if k != "state"})
