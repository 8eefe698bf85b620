"""That every result of the short convolution, the selective scan and the gated
feed-forward lies in memory whose surroundings a test watches, and that these stay as
they were; inputs are those of test_blocks_gpu.py.
"""
import pytest
import torch

from linear_recurrent_sequence_amd import mlstm
from test_blocks_gpu import BF, FP, _padded, conv_inputs, ffn_inputs, scan_inputs

pytestmark = pytest.mark.gpu


def _conv(dtype):
    x, w, b, st, dy, dst = conv_inputs(2, 37, 24, 4, dtype, 61)
    heads = dy.unflatten(2, (3, 8)).transpose(1, 2).contiguous()
    return lambda: [*mlstm.short_conv_fwd(x, w, bias=b, state=st, heads=3),
                    *mlstm.short_conv_fwd(x, w),
                    mlstm.short_conv_step(x[:, 0].contiguous(), w, st.clone(), heads=3)[0],
                    *mlstm.short_conv_bwd(x, w, heads, bias=b, state=st, dstate=dst,
                                          heads=3).values()]


def _scan(dtype):
    s, dy, dst = scan_inputs(2, 333, 24, 5, 1, dtype, 62)
    one = {k: v[:, 0].contiguous() if k in ("u", "dt", "B", "C", "gate") else v
           for k, v in s.items()}
    return lambda: [*mlstm.scan_fwd(**s),
                    mlstm.scan_step(**{**one, "state": one["state"].clone()})[0],
                    *mlstm.scan_bwd(**s, dy=dy, dstate=dst).values()]


def _ffn(dtype):
    f = [ffn_inputs(M, 72, 40, dtype, 63) for M in (3, 70, 600)]
    return lambda: [t for x, wg, wu, dh in f for t in (
        mlstm.gated_ffn_fwd(x, wg, wu), *mlstm.gated_ffn_bwd(x, wg, wu, dh))]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("calls", [_conv, _scan, _ffn])
def test_every_result_lies_between_guards(monkeypatch, calls, dtype):
    run, checks, at = calls(dtype), [], set()

    def empty(shape, dtype=None, **_):
        if dtype == torch.uint8:  # a workspace
            t, ok = _padded((-(-shape // 4),), FP)
            t = t.view(torch.uint8)[:shape]
        else:
            t, ok = _padded(tuple(shape), dtype)
        checks.append(ok)
        at.add(t.data_ptr())
        return t

    ref = run()
    monkeypatch.setattr(mlstm.torch, "empty", empty)
    monkeypatch.setattr(mlstm.torch, "empty_like", lambda t, **_: empty(t.shape, t.dtype))
    got = run()
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert all(t.data_ptr() in at for t in got), [t.data_ptr() in at for t in got]
    assert all(ok() for ok in checks)
    assert all(torch.equal(a, r) for a, r in zip(got, ref))
