"""The gated delta rule and the block norm without a GPU: the float64 oracle's
pins, and the argument checks of the C ABI and the binding, which run before
any device work.
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

def _delta(rng, B=1, NHK=1, NH=2, T=5, dk=4, dv=3):
    n = rng.standard_normal
    k = n((B, NHK, T, dk))
    return dict(q=n((B, NHK, T, dk)), k=k / np.linalg.norm(k, axis=-1, keepdims=True),
                v=n((B, NH, T, dv)), beta=rng.uniform(0, 1, (B, NH, T)), fgate=n((B, NH, T)),
                C0=n((B, NH, dv, dk)))


def test_delta_holds_the_last_value_of_a_repeated_unit_key():
    """beta = 1, f = 1: writing a unit key replaces what the memory returns for it."""
    rng = np.random.default_rng(0)
    x = _delta(rng, NH=1, T=6)
    x["k"][:] = x["k"][:, :, :1]
    x["q"][:] = x["k"] * np.sqrt(4)  # q / sqrt(dk) is the key
    h, C = oracle.delta_forward(x["q"], x["k"], x["v"], np.ones((1, 1, 6)),
                                np.full((1, 1, 6), np.inf), x["C0"])
    np.testing.assert_allclose(h, x["v"], atol=1e-12)
    np.testing.assert_allclose(C[0, 0] @ x["k"][0, 0, 0], x["v"][0, 0, -1], atol=1e-12)


def test_delta_with_orthogonal_keys_is_gated_linear_attention():
    rng = np.random.default_rng(1)
    x = _delta(rng, NH=1, T=4)
    x["k"][0, 0] = np.eye(4)
    f = 1 / (1 + np.exp(-x["fgate"][0, 0]))
    h, C = oracle.delta_forward(x["q"], x["k"], x["v"], x["beta"], x["fgate"])
    for t in range(4):
        ref = sum(np.prod(f[j + 1:t + 1]) * x["beta"][0, 0, j] * x["v"][0, 0, j]
                  * x["q"][0, 0, t, j] / 2.0 for j in range(t + 1))
        np.testing.assert_allclose(h[0, 0, t], ref, atol=1e-12)
    assert np.array_equal(C[0, 0][:, 3], x["beta"][0, 0, 3] * x["v"][0, 0, 3])


@pytest.mark.parametrize("forget", ["sigmoid", "exp"])
def test_delta_gradients_by_differences(forget):
    rng = np.random.default_rng(2)
    x = _delta(rng, B=2, NHK=1, NH=2)
    dh, dC = rng.standard_normal((2, 2, 5, 3)), rng.standard_normal((2, 2, 3, 4))

    def loss(**kw):
        y = {**x, **kw}
        h, C = oracle.delta_forward(y["q"], y["k"], y["v"], y["beta"], y["fgate"], y["C0"], forget)
        return (h * dh).sum() + (C * dC).sum()

    g = oracle.delta_backward(x["q"], x["k"], x["v"], x["beta"], x["fgate"], dh, x["C0"], dC,
                              forget)
    for name, grad in zip(("q", "k", "v", "beta", "fgate", "C0"), g):
        for at in itertools.islice(np.ndindex(x[name].shape), 0, None, 3):
            up, dn = x[name].copy(), x[name].copy()
            up[at] += 1e-5
            dn[at] -= 1e-5
            # central difference: truncation ~ 1e-10, rounding ~ 1e-16 / 1e-5
            assert abs((loss(**{name: up}) - loss(**{name: dn})) / 2e-5 - grad[at]) < 1e-7, name


@pytest.mark.parametrize("norm,activation", [("layer", "sigmoid"), ("rms", "silu")])
def test_block_norm_gradients_by_differences(norm, activation):
    rng = np.random.default_rng(3)
    n = rng.standard_normal
    x = dict(p=n((1, 2, 3, 4)), weight=n(8), gate=n((1, 2, 3, 4)), residual=n((1, 3, 8)),
             scale=n(8), next_weight=n(8))
    dr, dy = n((1, 3, 8)), n((1, 3, 8))
    kw = dict(norm=norm, activation=activation)

    def loss(**c):
        r, y = oracle.block_norm(**{**x, **c}, **kw)
        return (r * dr).sum() + (y * dy).sum()

    g = oracle.block_norm(**x, **kw, dr=dr, dy=dy, grads=True)
    for name in x:
        for at in np.ndindex(x[name].shape):
            up, dn = x[name].copy(), x[name].copy()
            up[at] += 1e-5
            dn[at] -= 1e-5
            assert abs((loss(**{name: up}) - loss(**{name: dn})) / 2e-5
                       - g["d" + name][at]) < 1e-6, name


# -------------------------------------------------------- the C ABI's refusals

F = [(i + 1) << 32 for i in range(24)]  # aligned addresses far apart; never dereferenced
BIG = 1 << 31


def _call(fn, order, args, case):
    args = {**args, **case}
    return getattr(mlstm.load_library(), fn)(
        *[args[n] or None if n in PTRS else args[n] for n in order])


PTRS = set("q k v beta fgate C_in h C_out dh dC_in dq dk dv dbeta dfgate dC_out ws p gate residual "
           "weight scale next_weight r y dr dy dp dgate dresidual dweight dscale dnext_weight "
           "stream".split())
DELTA = dict(q=F[0], k=F[1], v=F[2], beta=F[3], fgate=F[4], C_in=F[5], h=F[6], C_out=F[7], ws=F[8],
             dh=F[9], dC_in=F[10], dq=F[11], dk=F[12], dv=F[13], dbeta=F[14], dfgate=F[15],
             dC_out=F[16], nws=1 << 30, B=2, NHK=2, NH=4, T=100, ddk=64, ddv=48, dtype=1,
             forget=0, stream=0)
FWD = "q k v beta fgate C_in h C_out ws nws B NHK NH T ddk ddv dtype forget stream".split()
BWD = ("q k v beta fgate C_in dh dC_in dq dk dv dbeta dfgate dC_out ws nws B NHK NH T ddk ddv "
       "dtype forget stream").split()
STEP = "q k v beta fgate C_in C_out h B NHK NH ddk ddv dtype forget stream".split()

SIZES = [(dict(B=0), -2), (dict(NH=0), -2), (dict(NHK=0), -2), (dict(ddk=0), -2),
         (dict(ddv=-16), -2), (dict(dtype=2), -3), (dict(ddk=24), -4), (dict(ddk=528), -4), (dict(ddv=40), -4),
         (dict(ddv=1040), -4), (dict(NH=5), -12), (dict(NHK=8), -12), (dict(forget=2), -10),
         (dict(forget=-1), -10), (dict(B=BIG), -2), (dict(B=1 << 20, NH=1 << 16, NHK=1), -2)]


@needs_lib
@pytest.mark.parametrize("case,status", SIZES + [
    (dict(T=0), -2), (dict(T=1 << 40), -2), (dict(T=1 << 30, B=64), -2), (dict(B=1 << 16), -2),
    (dict(q=0), -1), (dict(C_out=0), -1), (dict(h=0), -1), (dict(ws=0), -1), (dict(beta=0), -1),
    (dict(q=F[0] + 8), -5), (dict(beta=F[3] + 2), -5), (dict(ws=F[8] + 128), -5),
    (dict(C_in=F[5] + 4), -5), (dict(nws=100), -7),
    (dict(h=F[2]), -9), (dict(C_out=F[5] + 16), -9), (dict(C_out=F[6]), -9), (dict(ws=F[0]), -9),
])
def test_delta_fwd_rejects_before_device_work(case, status):
    assert _call("mlstm_delta_fwd", FWD, DELTA, case) == status


@needs_lib
@pytest.mark.parametrize("case,status", SIZES + [
    (dict(T=0), -2), (dict(dh=0), -1), (dict(dq=0), -1), (dict(dfgate=0), -1), (dict(ws=0), -1),
    (dict(dC_out=F[16] + 4), -5), (dict(dbeta=F[14] + 1), -5), (dict(nws=100), -7),
    (dict(dq=F[0]), -9), (dict(dv=F[9]), -9), (dict(dk=F[11]), -9), (dict(dC_out=F[10]), -9),
    (dict(ws=F[9]), -9),
])
def test_delta_bwd_rejects_before_device_work(case, status):
    assert _call("mlstm_delta_bwd", BWD, DELTA, case) == status


@needs_lib
@pytest.mark.parametrize("case,status", SIZES + [
    (dict(B=1 << 18, NH=32), -2), (dict(C_in=0), -1), (dict(h=0), -1), (dict(v=F[2] + 2), -5),
    (dict(C_out=F[5] + 64), -9), (dict(h=F[0]), -9)])
def test_delta_step_rejects_before_device_work(case, status):
    assert _call("mlstm_delta_step", STEP, DELTA, case) == status


NORM = dict(p=F[0], gate=F[1], residual=F[2], weight=F[3], scale=F[4], next_weight=F[5], r=F[6],
            y=F[7], dr=F[8], dy=F[9], dp=F[10], dgate=F[11], dresidual=F[12], dweight=F[13],
            dscale=F[14], dnext_weight=F[15], ws=F[16], nws=1 << 30, B=2, NH=4, T=10, d=40,
            dtype=1, norm=0, act=0, eps=1e-5, stream=0)
NFWD = "p gate residual weight scale next_weight r y B NH T d dtype norm act eps stream".split()
NBWD = ("p gate residual weight scale next_weight dr dy dp dgate dresidual dweight dscale "
        "dnext_weight ws nws B NH T d dtype norm act eps stream").split()
NSIZES = [(dict(B=0), -2), (dict(T=0), -2), (dict(d=0), -2), (dict(dtype=-1), -3), (dict(d=4), -4),
          (dict(d=44), -4), (dict(d=8200), -4), (dict(d=4096, NH=3), -4), (dict(B=BIG), -2),
          (dict(T=1 << 40), -2), (dict(B=1 << 20, T=1 << 29), -2), (dict(norm=2), -13),
          (dict(act=-1), -13), (dict(eps=-1.0), -13), (dict(eps=float("nan")), -13),
          (dict(eps=float("inf")), -13), (dict(p=0), -1), (dict(weight=0), -1),
          (dict(p=F[0] + 2), -5), (dict(scale=F[4] + 4), -5)]


@needs_lib
@pytest.mark.parametrize("case,status", NSIZES + [
    (dict(r=0), -1), (dict(y=0), -1), (dict(next_weight=0), -1), (dict(r=F[2]), -9),
    (dict(y=F[6]), -9), (dict(y=F[5]), -9)])
def test_block_norm_fwd_rejects_before_device_work(case, status):
    assert _call("mlstm_block_norm_fwd", NFWD, NORM, case) == status


@needs_lib
@pytest.mark.parametrize("case,status", NSIZES + [
    (dict(dp=0), -1), (dict(dweight=0), -1), (dict(ws=0), -1), (dict(dgate=0), -1),
    (dict(gate=0), -1), (dict(dresidual=0), -1), (dict(scale=0), -1), (dict(dnext_weight=0), -1),
    (dict(dy=0), -1), (dict(next_weight=0), -1), (dict(nws=64), -7), (dict(ws=F[16] + 16), -5),
    (dict(dp=F[0]), -9), (dict(dresidual=F[8]), -9), (dict(dweight=F[13], dscale=F[13]), -9)])
def test_block_norm_bwd_rejects_before_device_work(case, status):
    assert _call("mlstm_block_norm_bwd", NBWD, NORM, case) == status


@needs_lib
def test_workspace_sizes():
    lib = mlstm.load_library()
    size = lib.mlstm_delta_workspace_bytes
    one = size(1, 1, 1, 64, 64, 16, 1, 0)
    assert one > 0 and size(1, 1, 1, 65, 64, 16, 1, 0) == 2 * one
    assert size(1, 1, 1, 1, 32, 16, 1, 0) == 0 < size(1, 1, 1, 1, 32, 16, 1, 1)
    assert size(1, 3, 4, 64, 32, 16, 1, 0) == size(0, 1, 1, 64, 32, 16, 1, 1) == 0
    assert lib.mlstm_block_norm_workspace_bytes(1, 1, 1, 9) == 0
    assert lib.mlstm_block_norm_workspace_bytes(1, 4, 7, 384) > 0
    assert "multiple" in mlstm.strerror(-12) and "norm" in mlstm.strerror(-13)


# ------------------------------------------------------- the binding's refusals

def _t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def _args(T=True):
    n = (64,) if T else ()
    b = torch.bfloat16
    return [_t(1, 2, *n, 32, dtype=b), _t(1, 2, *n, 32, dtype=b), _t(1, 4, *n, 16, dtype=b),
            _t(1, 4, *n), _t(1, 4, *n)]


def _norm_kw():
    return dict(gate=_t(1, 4, 8, 16), residual=_t(1, 8, 64), scale=_t(64), next_weight=_t(64))


class Stop(Exception):
    pass


CALLS = {
    "delta_fwd": (lambda: mlstm.delta_fwd(*_args(), state=_t(1, 4, 16, 32),
                                          out_state=_t(1, 4, 16, 32)),
                  "q k v beta fgate state out_state"),
    "delta_bwd": (lambda: mlstm.delta_bwd(*_args(), _args()[2], state=_t(1, 4, 16, 32),
                                          dstate=_t(1, 4, 16, 32)),
                  "q k v beta fgate dh state dstate"),
    "delta_step": (lambda: mlstm.delta_step(*_args(False), _t(1, 4, 16, 32), _t(1, 4, 16, 32)),
                   "q k v beta fgate state out_state"),
    "block_norm_fwd": (lambda: mlstm.block_norm_fwd(_t(1, 4, 8, 16), _t(64), **_norm_kw()),
                       "p weight gate residual scale next_weight"),
    "block_norm_bwd": (lambda: mlstm.block_norm_bwd(_t(1, 4, 8, 16), _t(64), _t(1, 8, 64),
                                                    _t(1, 8, 64), **_norm_kw()),
                       "p weight gate residual scale next_weight dr dy"),
}


@needs_lib
@pytest.mark.parametrize("call,arg", [(c, a) for c, (_, s) in CALLS.items() for a in s.split()])
def test_every_tensor_argument_is_validated(monkeypatch, call, arg):
    def fake(name, t, *rest):
        if name == arg:
            raise Stop
    monkeypatch.setattr(mlstm, "_require", fake)
    monkeypatch.setattr(mlstm, "_require_device", lambda *a: None)
    with pytest.raises(Stop):
        CALLS[call][0]()


@needs_lib
def test_binding_refuses_malformed_calls():
    a = _args()
    with pytest.raises(ValueError, match="GPU tensor"):
        mlstm.delta_fwd(*a)
    with pytest.raises(ValueError, match="shape"):
        mlstm.delta_fwd(a[0], a[1][:, :, :5], *a[2:])
    with pytest.raises(ValueError, match="NHK"):
        mlstm.delta_fwd(a[0][0], *a[1:])
    with pytest.raises(ValueError, match="NHK"):
        mlstm.delta_step(*a, _t(1, 4, 16, 32))
    with pytest.raises(TypeError):
        mlstm.delta_fwd(a[0].half(), *a[1:])
    with pytest.raises(TypeError):
        mlstm.delta_fwd(a[0], a[1], None, *a[3:])
    p, w = _t(1, 4, 8, 16), _t(64)
    with pytest.raises(ValueError, match="GPU tensor"):
        mlstm.block_norm_fwd(p, w)
    with pytest.raises(ValueError, match=r"\[B, NH, T, d\]"):
        mlstm.block_norm_fwd(p[0], w)
    with pytest.raises(TypeError):
        mlstm.block_norm_fwd(p.double(), w)


@needs_lib
def test_binding_refuses_unknown_names(monkeypatch):
    monkeypatch.setattr(mlstm, "_require", lambda *a: None)
    monkeypatch.setattr(mlstm, "_require_device", lambda *a: None)
    p, w = _t(1, 4, 8, 16), _t(64)
    with pytest.raises(ValueError, match="norm"):
        mlstm.block_norm_fwd(p, w, norm="batch")
    with pytest.raises(ValueError, match="activation"):
        mlstm.block_norm_fwd(p, w, activation="relu")
    with pytest.raises(ValueError, match="together"):
        mlstm.block_norm_bwd(p, w, None, None, next_weight=w)
    with pytest.raises(ValueError, match="together"):
        mlstm.block_norm_bwd(p, w, None, _t(1, 8, 64))
    with pytest.raises(ValueError, match="forget"):
        mlstm.delta_fwd(*_args(), forget="relu")
