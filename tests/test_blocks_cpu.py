"""The short convolution, the selective scan and the gated feed-forward without a
GPU: the float64 oracle's pins, and the argument checks of the C ABI and the
binding, which run before any device work.
"""
import itertools
import os

import numpy as np
import pytest
import torch

import oracle
from linear_recurrent_sequence_amd import mlstm

needs_lib = pytest.mark.skipif(not os.path.exists(mlstm.LIB_PATH),
                               reason="libmlstm.so not built (run __graft_entry__.build())")


# ---------------------------------------------------------------- the oracle

def _differences(loss, x, grads, every=3):
    """Central differences against ``grads``: truncation ~ 1e-10, rounding ~ 1e-16 / 1e-5."""
    for name, grad in grads.items():
        for at in itertools.islice(np.ndindex(x[name].shape), 0, None, every):
            up, dn = x[name].copy(), x[name].copy()
            up[at] += 1e-5
            dn[at] -= 1e-5
            d = (loss(**{name: up}) - loss(**{name: dn})) / 2e-5
            assert abs(d - grad[at]) < 1e-7, (name, at)


@pytest.mark.parametrize("activation", ["silu", "none"])
def test_short_conv_gradients_by_differences(activation):
    n = np.random.default_rng(0).standard_normal
    x = dict(x=n((3, 5, 2)), weight=n((2, 4)), bias=n(2), state=n((3, 3, 2)))
    dy, dst, lengths = n((3, 5, 2)), n((3, 3, 2)), [5, 0, 2]

    def loss(**kw):
        v = {**x, **kw}
        y, st = oracle.short_conv(v["x"], v["weight"], v["bias"], v["state"], lengths, activation)
        return (y * dy).sum() + (st * dst).sum()

    dx, dw, db, ds, _, _ = oracle.short_conv_grads(x["x"], x["weight"], dy, x["bias"], x["state"],
                                                   dst, lengths, activation)
    _differences(loss, x, dict(x=dx, weight=dw, bias=db, state=ds), 1)
    assert not dx[1].any() and not dx[2, 2:].any() and np.array_equal(ds[1], dst[1])


def test_short_conv_shifts_and_sums():
    x = np.arange(1.0, 7.0).reshape(1, 6, 1)
    y, st = oracle.short_conv(x, np.array([[1.0, 0.0, 0.0]]), activation="none")
    assert y[0, :, 0].tolist() == [0, 0, 1, 2, 3, 4] and st[0, :, 0].tolist() == [5, 6]
    y, _ = oracle.short_conv(x, np.ones((1, 2)), np.array([10.0]), np.full((1, 1, 1), 7.0),
                             activation="none")
    assert y[0, :, 0].tolist() == [18, 13, 15, 17, 19, 21]


@pytest.mark.parametrize("gate", [True, False])
def test_scan_gradients_by_differences(gate):
    n = np.random.default_rng(1).standard_normal
    x = dict(u=n((2, 4, 4)), dt=n((2, 4, 4)), A=-np.abs(n((4, 3))), B=n((2, 4, 2, 3)),
             C=n((2, 4, 2, 3)), D=n(4), gate=n((2, 4, 4)), dt_bias=n(4), state=n((2, 4, 3)))
    if not gate:
        del x["gate"], x["D"]
    dy, dst, lengths = n((2, 4, 4)), n((2, 4, 3)), [4, 2]

    def loss(**kw):
        y, st = oracle.selective_scan(**{**x, **kw}, lengths=lengths)
        return (y * dy).sum() + (st * dst).sum()

    g, _ = oracle.selective_scan_grads(**x, dy=dy, dstate=dst, lengths=lengths)
    _differences(loss, x, {k: g["d" + k] for k in x}, 2)


def test_scan_of_constant_steps_is_geometric():
    """u = B = C = 1, one state, Delta log 2 and A = -1: s halves and gains log 2."""
    one = np.ones((1, 5, 1))
    dt = np.full((1, 5, 1), 0.0)  # softplus(0) = log 2
    y, st = oracle.selective_scan(one, dt, np.array([[-1.0]]), one[..., None], one[..., None])
    ref = np.log(2.0) * np.cumsum(0.5 ** np.arange(5))
    np.testing.assert_allclose(y[0, :, 0], ref, rtol=1e-14)
    np.testing.assert_allclose(st[0, 0, 0], ref[-1], rtol=1e-14)
    _, kept = oracle.selective_scan(one, dt - np.inf, np.array([[-1.0]]), one[..., None],
                                    one[..., None], state=np.full((1, 1, 1), 3.0))
    assert kept[0, 0, 0] == 3.0


@pytest.mark.parametrize("activation", ["silu", "gelu"])
def test_ffn_gradients_by_differences(activation):
    n = np.random.default_rng(2).standard_normal
    x = dict(x=n((3, 4)), w_gate=n((5, 4)), w_up=n((5, 4)))
    dh = n((3, 5))

    def loss(**kw):
        return (oracle.gated_ffn(**{**x, **kw}, activation=activation) * dh).sum()

    grads, _ = oracle.gated_ffn_grads(**x, dh=dh, activation=activation)
    _differences(loss, x, dict(zip(x, grads)), 1)


def test_ffn_activations_far_from_zero():
    one, big = np.ones((1, 1)), np.full((1, 1), 40.0)
    for activation in ("silu", "gelu"):
        assert abs(oracle.gated_ffn(big, one, one, activation)[0, 0] - 1600.0) < 1e-12
        assert abs(oracle.gated_ffn(big, -one, one, activation)[0, 0]) < 1e-12


# ------------------------------------------------------- the C ABI's refusals

F = [(i + 1) << 33 for i in range(24)]  # addresses that are not dereferenced, far apart
BIG = 1 << 62


def _call(name, order, good, case):
    args = {**good, **case}
    return getattr(mlstm.load_library(), name)(*[args[n] for n in order.split()])


CONV = dict(x=F[0], x_row=96, weight=F[1], bias=F[2], state=F[3], lengths=F[4], y=F[5], so=F[6],
            dy=F[7], dstate=F[8], dx=F[9], dweight=F[10], dbias=F[11], dso=F[12], ws=F[13],
            nws=1 << 30, B=2, NH=2, T=10, d=48, width=4, dtype=1, act=1, stream=0)
CFWD = "x x_row weight bias state lengths y so B NH T d width dtype act stream"
CBWD = ("x x_row weight bias state lengths dy dstate dx dweight dbias dso ws nws B NH T d width "
        "dtype act stream")
CSIZES = [(dict(dtype=2), -3), (dict(B=0), -2), (dict(T=0), -2), (dict(NH=0), -2), (dict(d=0), -2),
          (dict(B=BIG), -2), (dict(T=BIG), -2), (dict(B=1 << 20, T=1 << 14), -2), (dict(d=44), -4),
          (dict(NH=1 << 20), -4), (dict(width=1), -14), (dict(width=9), -14), (dict(act=2), -10),
          (dict(x=0), -1), (dict(weight=0), -1), (dict(x_row=95), -15), (dict(x_row=88), -15),
          (dict(x_row=100), -15), (dict(x_row=BIG), -15), (dict(x=F[0] + 8), -5),
          (dict(bias=F[2] + 4), -5), (dict(state=F[3] + 2), -5), (dict(lengths=F[4] + 2), -5)]


@needs_lib
@pytest.mark.parametrize("case,status", CSIZES + [
    (dict(y=0), -1), (dict(so=0), -1), (dict(y=F[5] + 8), -5), (dict(y=F[0]), -9),
    (dict(so=F[3] + 16), -9), (dict(so=F[5]), -9), (dict(y=F[4]), -9)])
def test_short_conv_fwd_rejects_before_device_work(case, status):
    assert _call("mlstm_short_conv_fwd", CFWD, CONV, case) == status


@needs_lib
@pytest.mark.parametrize("case,status", CSIZES + [
    (dict(dy=0), -1), (dict(dx=0), -1), (dict(dweight=0), -1), (dict(ws=0), -1),
    (dict(dbias=0), -1), (dict(bias=0), -1), (dict(ws=F[13] + 16), -5), (dict(nws=100), -7),
    (dict(dx=F[0]), -9), (dict(dx=F[7]), -9), (dict(dso=F[8]), -9), (dict(dweight=F[11]), -9),
    (dict(dso=F[3]), -9)])
def test_short_conv_bwd_rejects_before_device_work(case, status):
    assert _call("mlstm_short_conv_bwd", CBWD, CONV, case) == status


SCAN = dict(u=F[0], ur=32, dt=F[1], dr=32, A=F[2], B=F[3], br=24, C=F[4], cr=24, D=F[5],
            gate=F[6], gr=32, bias=F[7], state=F[8], lengths=F[9], y=F[10], so=F[11], dy=F[12],
            dstate=F[13], du=F[14], ddt=F[15], dA=F[16], dB=F[17], dC=F[18], dD=F[19],
            dgate=F[20], dbias=F[21], dso=F[22], ws=F[23], nws=1 << 30, n=2, T=10, ch=32, G=2,
            N=12, dtype=0, stream=0)
SIN = "u ur dt dr A B br C cr D gate gr bias state lengths "
SFWD = SIN + "y so ws nws n T ch G N dtype stream"
SBWD = SIN + "dy dstate du ddt dA dB dC dD dgate dbias dso ws nws n T ch G N dtype stream"
SSIZES = [(dict(dtype=-1), -3), (dict(n=0), -2), (dict(T=0), -2), (dict(ch=0), -2),
          (dict(G=0), -2), (dict(N=0), -2), (dict(n=BIG), -2), (dict(T=BIG), -2),
          (dict(T=1 << 30), -2), (dict(n=1 << 25), -2), (dict(G=3), -12), (dict(G=8), -4),
          (dict(ch=1 << 21), -4), (dict(N=65), -14), (dict(u=0), -1), (dict(dt=0), -1),
          (dict(A=0), -1), (dict(B=0), -1), (dict(C=0), -1), (dict(ur=31), -15),
          (dict(dr=36), -15), (dict(gr=24), -15), (dict(br=23), -15), (dict(cr=BIG), -15),
          (dict(u=F[0] + 4), -5), (dict(gate=F[6] + 8), -5), (dict(A=F[2] + 4), -5),
          (dict(state=F[8] + 4), -5), (dict(B=F[3] + 2), -5), (dict(lengths=F[9] + 1), -5)]


@needs_lib
@pytest.mark.parametrize("case,status", SSIZES + [
    (dict(y=0), -1), (dict(so=0), -1), (dict(y=F[10] + 4), -5), (dict(ws=F[23] + 8), -5),
    (dict(y=F[0]), -9), (dict(so=F[8] + 16), -9), (dict(y=F[11]), -9),
    (dict(T=4000, nws=64), -7), (dict(T=4000, ws=0), -1), (dict(T=4000, ws=F[6]), -9)])
def test_scan_fwd_rejects_before_device_work(case, status):
    assert _call("mlstm_scan_fwd", SFWD, SCAN, case) == status


@needs_lib
@pytest.mark.parametrize("case,status", SSIZES + [
    (dict(dy=0), -1), (dict(du=0), -1), (dict(ddt=0), -1), (dict(dA=0), -1), (dict(dB=0), -1),
    (dict(dC=0), -1), (dict(ws=0), -1), (dict(dD=0), -1), (dict(D=0), -1), (dict(dgate=0), -1),
    (dict(gate=0), -1), (dict(dbias=0), -1), (dict(bias=0), -1), (dict(nws=64), -7),
    (dict(dC=F[18] + 4), -5), (dict(du=F[0]), -9), (dict(dso=F[13]), -9), (dict(dB=F[18]), -9),
    (dict(ddt=F[12]), -9)])
def test_scan_bwd_rejects_before_device_work(case, status):
    assert _call("mlstm_scan_bwd", SBWD, SCAN, case) == status


FFN = dict(x=F[0], wg=F[1], wu=F[2], h=F[3], dh=F[4], dx=F[5], dwg=F[6], dwu=F[7], ws=F[8],
           nws=1 << 32, M=100, D=64, F=40, dtype=0, act=0, stream=0)
FFWD = "x wg wu h ws nws M D F dtype act stream"
FBWD = "x wg wu dh dx dwg dwu ws nws M D F dtype act stream"
FSIZES = [(dict(dtype=5), -3), (dict(M=0), -2), (dict(D=0), -2), (dict(F=0), -2),
          (dict(M=(1 << 20) + 1), -2), (dict(M=1 << 20, F=1 << 13), -2), (dict(D=60), -4),
          (dict(F=36), -4), (dict(D=1 << 17), -4), (dict(F=BIG), -4), (dict(act=2), -10),
          (dict(x=0), -1), (dict(wg=0), -1), (dict(wu=0), -1), (dict(x=F[0] + 4), -5),
          (dict(ws=F[8] + 16), -5), (dict(nws=1000), -7), (dict(ws=0), -1)]


@needs_lib
@pytest.mark.parametrize("case,status", FSIZES + [
    (dict(h=0), -1), (dict(h=F[3] + 8), -5), (dict(h=F[0]), -9), (dict(h=F[2]), -9),
    (dict(ws=F[1]), -9)])
def test_gated_ffn_fwd_rejects_before_device_work(case, status):
    assert _call("mlstm_gated_ffn_fwd", FFWD, FFN, case) == status


@needs_lib
@pytest.mark.parametrize("case,status", FSIZES + [
    (dict(dh=0), -1), (dict(dx=0), -1), (dict(dwg=0), -1), (dict(dwu=0), -1),
    (dict(dwu=F[7] + 8), -5), (dict(dx=F[0]), -9), (dict(dwg=F[7]), -9), (dict(dx=F[4]), -9)])
def test_gated_ffn_bwd_rejects_before_device_work(case, status):
    assert _call("mlstm_gated_ffn_bwd", FBWD, FFN, case) == status


@needs_lib
def test_block_workspace_sizes():
    lib = mlstm.load_library()
    scan, ffn = lib.mlstm_scan_workspace_bytes, lib.mlstm_gated_ffn_workspace_bytes
    assert scan(1, 1, 64, 1, 16, 1, 0) == 0 < scan(1, 1, 64, 1, 16, 1, 1)
    assert scan(1, 100000, 64, 1, 16, 1, 0) > 0  # segments
    assert scan(1, 100, 60, 1, 16, 1, 1) == scan(1, 100, 64, 1, 65, 1, 1) == 0
    assert ffn(8, 64, 64, 0, 0) == 0 < ffn(8, 64, 64, 0, 1)
    assert ffn(1000, 64, 63, 0, 1) == 0 < ffn(1000, 64, 64, 0, 0)
    assert lib.mlstm_short_conv_workspace_bytes(1, 1, 8, 16, 4, 1) > 0
    assert lib.mlstm_short_conv_workspace_bytes(1, 1, 8, 16, 1, 1) == 0
    assert "width" in mlstm.strerror(-14) and "pitch" in mlstm.strerror(-15)


# ------------------------------------------------------- the binding's refusals

def _t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def _scan_args(T=True):
    n = (9,) if T else ()
    return [_t(2, *n, 32), _t(2, *n, 32), _t(32, 4), _t(2, *n, 2, 4), _t(2, *n, 2, 4)]


CALLS = {
    "short_conv_fwd": (lambda **k: mlstm.short_conv_fwd(**k), dict(
        x=_t(2, 9, 16), weight=_t(16, 4), bias=_t(16), state=_t(2, 3, 16),
        out_state=_t(2, 3, 16), lengths=_t(2, dtype=torch.int32))),
    "short_conv_step": (lambda **k: mlstm.short_conv_step(**k), dict(
        x=_t(2, 16), weight=_t(16, 4), state=_t(2, 3, 16), bias=_t(16), out_state=_t(2, 3, 16))),
    "short_conv_bwd": (lambda **k: mlstm.short_conv_bwd(heads=2, **k), dict(
        x=_t(2, 9, 16), weight=_t(16, 4), dy=_t(2, 2, 9, 8), bias=_t(16), state=_t(2, 3, 16),
        dstate=_t(2, 3, 16), lengths=_t(2, dtype=torch.int32))),
    "scan_fwd": (lambda **k: mlstm.scan_fwd(**k), dict(
        zip("u dt A B C".split(), _scan_args()), D=_t(32), gate=_t(2, 9, 32), dt_bias=_t(32),
        state=_t(2, 32, 4), out_state=_t(2, 32, 4), lengths=_t(2, dtype=torch.int32))),
    "scan_step": (lambda **k: mlstm.scan_step(**k), dict(
        zip("u dt A B C".split(), _scan_args(False)), state=_t(2, 32, 4), D=_t(32),
        gate=_t(2, 32), dt_bias=_t(32), out_state=_t(2, 32, 4))),
    "scan_bwd": (lambda **k: mlstm.scan_bwd(**k), dict(
        zip("u dt A B C".split(), _scan_args()), dy=_t(2, 9, 32), D=_t(32), gate=_t(2, 9, 32),
        dt_bias=_t(32), state=_t(2, 32, 4), dstate=_t(2, 32, 4),
        lengths=_t(2, dtype=torch.int32))),
    "gated_ffn_fwd": (lambda **k: mlstm.gated_ffn_fwd(**k), dict(
        x=_t(2, 3, 16), w_gate=_t(24, 16), w_up=_t(24, 16))),
    "gated_ffn_bwd": (lambda **k: mlstm.gated_ffn_bwd(**k), dict(
        x=_t(2, 3, 16), w_gate=_t(24, 16), w_up=_t(24, 16), dh=_t(2, 3, 24))),
}


@needs_lib
@pytest.mark.parametrize("call", CALLS)
def test_binding_wants_gpu_tensors(call):
    f, good = CALLS[call]
    with pytest.raises(ValueError, match="GPU tensor"):
        f(**good)


@needs_lib
@pytest.mark.parametrize("call,arg", [(c, a) for c, (_, good) in CALLS.items() for a in good])
def test_binding_checks_every_tensor(monkeypatch, call, arg):
    monkeypatch.setattr(mlstm, "_require_device", lambda *a: None)
    f, good = CALLS[call]
    bad = [(good[arg].double(), (TypeError, ValueError)), ([1.0], TypeError),
           (good[arg][..., :1], ValueError)]
    if (call, arg) != ("gated_ffn_fwd", "x"):  # which may have any number of rows
        bad.append((torch.cat([good[arg], good[arg]]), ValueError))
    for bad, errors in bad:
        with pytest.raises(errors):
            f(**{**good, arg: bad})


@needs_lib
def test_binding_refuses_malformed_calls(monkeypatch):
    monkeypatch.setattr(mlstm, "_require_device", lambda *a: None)
    f, conv = CALLS["short_conv_fwd"]
    for kw, match in ((dict(heads=3), "divisor"), (dict(heads=0), "divisor"),
                      (dict(heads="2"), "divisor"), (dict(activation="gelu"), "activation"),
                      (dict(x=_t(2, 16, 9).transpose(1, 2)), "contiguous"),
                      (dict(x=_t(9, 2, 16).transpose(0, 1)), "evenly")):
        with pytest.raises(ValueError, match=match):
            f(**{**conv, **kw})
    f, scan = CALLS["scan_fwd"]
    for kw, match in ((dict(B=_t(2, 9, 4, 2).transpose(2, 3)), "contiguous"),
                      (dict(gate=_t(9, 2, 32).transpose(0, 1)), "evenly"),
                      (dict(u=_t(2, 32)), "channels"), (dict(B=_t(2, 9, 4)), "G, N")):
        with pytest.raises(ValueError, match=match):
            f(**{**scan, **kw})
    f, ffn = CALLS["gated_ffn_fwd"]
    with pytest.raises(ValueError, match="activation"):
        f(**ffn, activation="relu")
    with pytest.raises(ValueError, match="contiguous"):
        f(**{**ffn, "w_up": _t(16, 24).T})


@needs_lib
@pytest.mark.parametrize("call,arg", [
    (c, a) for c, (_, good) in CALLS.items() for a in good
    if a in "x weight u dt A B C dy w_gate w_up dh".split() or (c.endswith("step") and a == "state")])
def test_binding_wants_what_is_not_optional(monkeypatch, call, arg):
    monkeypatch.setattr(mlstm, "_require_device", lambda *a: None)
    f, good = CALLS[call]
    with pytest.raises(TypeError, match=f"{arg} must be a torch.Tensor, got NoneType"):
        f(**{**good, arg: None})


def test_pitches_of_rows(monkeypatch):
    """Rows of a wider matrix: one pitch for all of them."""
    monkeypatch.setattr(mlstm, "_require_device", lambda *a: None)
    wide = _t(3, 5, 64)

    def pitch(t, row):
        return mlstm._require_rows([("x", t, t.shape, t.dtype, row)], t.device)[0]

    assert pitch(wide, 64) == 64 and pitch(wide[..., 8:24], 16) == 64
    assert pitch(wide[:1, :, :16], 16) == 64 and pitch(wide[:, :1, :16], 16) == 5 * 64
    assert pitch(wide[:1, :1, :16], 16) == 16
    assert pitch(wide[..., :24].unflatten(-1, (2, 12)), 24) == 64
    with pytest.raises(ValueError, match="evenly"):
        pitch(wide[:, :4, :16], 16)
    with pytest.raises(ValueError, match="contiguous"):
        pitch(wide[..., :32].unflatten(-1, (2, 16))[..., :12], 24)
