"""Paths of the selective scan that the shapes of test_blocks_gpu.py do not reach; inputs,
oracle and tolerances are that file's.
"""
import numpy as np
import pytest

from linear_recurrent_sequence_amd import mlstm
from test_blocks_gpu import BF, FP, check_scan_grads, close, i32, scan_inputs, scan_ref

pytestmark = pytest.mark.gpu


def _pad(n):
    return (n + 255) // 256 * 256


def forward_segments(n, T, c, N, G, dtype):
    """Into how many segments the forward cuts a sequence: its workspace has a state and
    a sum of steps for each."""
    size = mlstm.load_library().mlstm_scan_workspace_bytes(n, T, c, G, N, int(dtype == BF), 0)
    return next(s for s in range(1, 65) if size == (
        0 if s == 1 else _pad(4 * s * n * N * c) + _pad(4 * s * n * c)))


def backward_is_cut(n, T, c, N, G, dtype):
    """Whether the backward's workspace is more than a sequence in one piece takes."""
    size = mlstm.load_library().mlstm_scan_workspace_bytes(n, T, c, G, N, int(dtype == BF), 1)
    tiles = -(-T // (16 if N <= 32 else 8))
    return size > (_pad(4 * n * tiles * N * c) + _pad(4 * n * (N + 2) * c)
                   + _pad(8 * G * -(-c // G // 64) * n * T * N))


def workgroups(n, c, G):
    return n * G * -(-c // G // 64)


def scan_case(n, T, c, N, G, dtype, seed, left_out):
    """Inputs without some of those that may be left out (with smaller steps where the
    bias, which makes them small, is)."""
    x, dy, dst = scan_inputs(n, T, c, N, G, dtype, seed, slow=0.1)
    if "dt_bias" in left_out:
        x["dt"] = x["dt"] - 3.0
    if "state" in left_out:
        dst = None
    return {k: v for k, v in x.items() if k not in left_out}, dy, dst


def check_scan(x, dy, dst, lengths):
    y, st = mlstm.scan_fwd(**x, lengths=i32(lengths))
    yr, sr = scan_ref(x, lengths)
    close("y", y, yr, np.full_like(yr, np.sqrt((yr ** 2).mean())))
    close("state", st, sr)
    check_scan_grads(mlstm.scan_bwd(**x, dy=dy, dstate=dst, lengths=i32(lengths)), x, dy, dst,
                     lengths)


ALL = ("gate", "D", "dt_bias", "state")


# segments, with each number of states to a wave, ragged last ones, and lengths that end
# in the middle of one
@pytest.mark.parametrize("left_out", [ALL, ("gate",), ("D", "state"), ("dt_bias",)])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n,T,c,N,G,lengths", [
    (1, 1000, 8, 3, 1, None), (2, 801, 72, 7, 1, [801, 300]), (1, 900, 64, 16, 2, None),
    (2, 513, 40, 24, 1, [0, 512]), (1, 700, 16, 64, 1, [690])])
def test_scan_in_segments_with_inputs_left_out(n, T, c, N, G, lengths, dtype, left_out):
    assert forward_segments(n, T, c, N, G, dtype) > 1
    assert backward_is_cut(n, T, c, N, G, dtype)
    check_scan(*scan_case(n, T, c, N, G, dtype, 64, left_out), lengths)


# segments on more workgroups than CUs: four states to a wave for few states as well
@pytest.mark.parametrize("left_out", [(), ALL])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("c,N,G", [(2056, 3, 1), (2056, 7, 1), (2048, 16, 1), (4176, 16, 2)])
def test_scan_in_segments_of_many_channels(c, N, G, dtype, left_out):
    T = 800
    segments = forward_segments(1, T, c, N, G, dtype)
    assert segments > 1 and workgroups(1, c, G) * segments > 256
    assert backward_is_cut(1, T, c, N, G, dtype)
    check_scan(*scan_case(1, T, c, N, G, dtype, 65, left_out), None)


# and one piece there, without what may be left out
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("N", [2, 7, 16, 21, 40])
def test_scan_of_many_channels_without_a_gate(N, dtype):
    n, T, c = 5, 37, 4168
    assert forward_segments(n, T, c, N, 1, dtype) == 1 and workgroups(n, c, 1) > 256
    assert not backward_is_cut(n, T, c, N, 1, dtype)
    check_scan(*scan_case(n, T, c, N, 1, dtype, 66, ALL), None)
