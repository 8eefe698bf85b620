"""Thin ctypes binding over libmlstm.so (the C ABI in include/mlstm.h).

Argument marshalling only: every step of the forward pass runs in the HIP
kernels of the library.  PyTorch supplies device memory and the current
stream.  There is no fallback: if the library is missing or the tensors are
not on a GPU, the call raises.

    h, m, n = parallel_fwd(q, k, v, igate, fgate)

q, k, v: [B, NH, T, d] contiguous, float32 or bfloat16, on the current GPU.
igate, fgate: [B, NH, T] contiguous float32 (input / forget gate pre-activations).
Returns h~ (same dtype as q), m and n (float32), as defined by Eqs. 80, 84 and
86 of the xLSTM appendix ("Parallel mLSTM Backward Pass" restates the
stabilized forward pass).

Beside the cell: the gated delta rule (``delta_fwd``, ``delta_bwd``,
``delta_step``), the block norm (``block_norm_fwd``, ``block_norm_bwd``), the short
causal convolution (``short_conv_fwd``, ``short_conv_bwd``, ``short_conv_step``), the
selective scan (``scan_fwd``, ``scan_bwd``, ``scan_step``) and the gated feed-forward
(``gated_ffn_fwd``, ``gated_ffn_bwd``), with the same conventions.
"""

import contextlib
import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmlstm.so")

MLSTM_FP32, MLSTM_BF16 = 0, 1
KERNELS = {"auto": 0, "mfma": 1, "vector": 2, "mfma_all_tiles": 3, "mfma_single": 4,
           "mfma_wide": 5}
FORGET_ACTIVATIONS = {"sigmoid": 0, "exp": 1}
NORMS = {"layer": 0, "rms": 1}
GATE_ACTIVATIONS = {"sigmoid": 0, "silu": 1}
CONV_ACTIVATIONS = {"none": 0, "silu": 1}
FFN_ACTIVATIONS = {"silu": 0, "gelu": 1}

_lib = None


class MlstmError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {strerror(status)} (status {status})")


def load_library():
    """Load libmlstm.so once; raise if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m linear_recurrent_sequence_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i64, i32, f = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    lib.mlstm_parallel_fwd.argtypes = [vp] * 8 + [i64] * 4 + [i32]
    lib.mlstm_parallel_fwd.restype = i32
    lib.mlstm_parallel_fwd_stream.argtypes = [vp] * 8 + [i64] * 4 + [i32, vp]
    lib.mlstm_parallel_fwd_stream.restype = i32
    lib.mlstm_parallel_fwd_noalloc.argtypes = [vp] * 8 + [i64] * 4 + [i32, vp]
    lib.mlstm_parallel_fwd_noalloc.restype = i32
    lib.mlstm_parallel_fwd_gated.argtypes = [vp] * 10 + [i64] * 4 + [i32, vp]
    lib.mlstm_parallel_fwd_gated.restype = i32
    lib.mlstm_recurrent_step.argtypes = [vp] * 13 + [i64] * 3 + [i32, i32, vp]
    lib.mlstm_recurrent_step.restype = i32
    lib.mlstm_parallel_fwd_train.argtypes = [vp] * 9 + [i64] * 4 + [i32, i32, vp]
    lib.mlstm_parallel_fwd_train.restype = i32
    lib.mlstm_parallel_bwd.argtypes = [vp] * 15 + [i64] * 4 + [i32, i32, vp]
    lib.mlstm_parallel_bwd.restype = i32
    lib.mlstm_workspace_bytes.argtypes = [i64] * 3
    lib.mlstm_workspace_bytes.restype = f
    lib.mlstm_gate_scan.argtypes = [vp] * 4 + [f] + [i64] * 4 + [i32, vp]
    lib.mlstm_gate_scan.restype = i32
    lib.mlstm_causal_tiles.argtypes = [vp] * 5 + [f] + [vp] * 2 + [i64] * 4 + [i32, i32, vp]
    lib.mlstm_causal_tiles.restype = i32
    lib.mlstm_delta_workspace_bytes.argtypes = [i64] * 6 + [i32, i32]
    lib.mlstm_delta_workspace_bytes.restype = f
    lib.mlstm_delta_fwd.argtypes = [vp] * 9 + [f] + [i64] * 6 + [i32, i32, vp]
    lib.mlstm_delta_fwd.restype = i32
    lib.mlstm_delta_bwd.argtypes = [vp] * 15 + [f] + [i64] * 6 + [i32, i32, vp]
    lib.mlstm_delta_bwd.restype = i32
    lib.mlstm_delta_step.argtypes = [vp] * 8 + [i64] * 5 + [i32, i32, vp]
    lib.mlstm_delta_step.restype = i32
    fl = ctypes.c_float
    lib.mlstm_block_norm_fwd.argtypes = [vp] * 8 + [i64] * 4 + [i32] * 3 + [fl, vp]
    lib.mlstm_block_norm_fwd.restype = i32
    lib.mlstm_block_norm_workspace_bytes.argtypes = [i64] * 4
    lib.mlstm_block_norm_workspace_bytes.restype = f
    lib.mlstm_block_norm_bwd.argtypes = [vp] * 15 + [f] + [i64] * 4 + [i32] * 3 + [fl, vp]
    lib.mlstm_block_norm_bwd.restype = i32
    lib.mlstm_short_conv_fwd.argtypes = [vp, i64] + [vp] * 6 + [i64] * 5 + [i32, i32, vp]
    lib.mlstm_short_conv_fwd.restype = i32
    lib.mlstm_short_conv_workspace_bytes.argtypes = [i64] * 5 + [i32]
    lib.mlstm_short_conv_workspace_bytes.restype = f
    lib.mlstm_short_conv_bwd.argtypes = [vp, i64] + [vp] * 11 + [f] + [i64] * 5 + [i32, i32, vp]
    lib.mlstm_short_conv_bwd.restype = i32
    lib.mlstm_scan_workspace_bytes.argtypes = [i64] * 5 + [i32, i32]
    lib.mlstm_scan_workspace_bytes.restype = f
    scan = [vp, i64, vp, i64, vp, vp, i64, vp, i64, vp, vp, i64, vp, vp, vp]
    lib.mlstm_scan_fwd.argtypes = scan + [vp] * 3 + [f] + [i64] * 5 + [i32, vp]
    lib.mlstm_scan_fwd.restype = i32
    lib.mlstm_scan_bwd.argtypes = scan + [vp] * 12 + [f] + [i64] * 5 + [i32, vp]
    lib.mlstm_scan_bwd.restype = i32
    lib.mlstm_gated_ffn_workspace_bytes.argtypes = [i64] * 3 + [i32, i32]
    lib.mlstm_gated_ffn_workspace_bytes.restype = f
    lib.mlstm_gated_ffn_tiles.argtypes = [i64] * 3 + [i32, i32, ctypes.POINTER(i64)]
    lib.mlstm_gated_ffn_tiles.restype = i32
    lib.mlstm_gated_ffn_fwd.argtypes = [vp] * 5 + [f] + [i64] * 3 + [i32, i32, vp]
    lib.mlstm_gated_ffn_fwd.restype = i32
    lib.mlstm_gated_ffn_bwd.argtypes = [vp] * 8 + [f] + [i64] * 3 + [i32, i32, vp]
    lib.mlstm_gated_ffn_bwd.restype = i32
    lib.mlstm_strerror.argtypes = [i32]
    lib.mlstm_strerror.restype = ctypes.c_char_p
    _lib = lib
    return lib


def strerror(status):
    return load_library().mlstm_strerror(int(status)).decode()


def _dtype_code(t):
    if t.dtype == torch.float32:
        return MLSTM_FP32
    if t.dtype == torch.bfloat16:
        return MLSTM_BF16
    raise TypeError(f"q/k/v must be float32 or bfloat16, got {t.dtype}")


def _forget_code(forget):
    """The C-ABI code of a forget-gate activation name ("sigmoid" or "exp")."""
    if forget not in FORGET_ACTIVATIONS:
        raise ValueError(f"forget must be one of {tuple(FORGET_ACTIVATIONS)}, got {forget!r}")
    return FORGET_ACTIVATIONS[forget]


def _require(name, t, shape, dtype, device=None):
    """Raise unless ``t`` is a contiguous tensor of exactly ``shape`` and
    ``dtype`` (and, if ``device`` is given, on that GPU).  Every tensor handed
    to the C ABI goes through here first: a host pointer, a wrong element type
    or a short buffer would otherwise reach the kernels."""
    # the common case in one expression (each tensor attribute read costs the
    # host time of a small kernel launch); the messages below on failure
    if (isinstance(t, torch.Tensor) and t.dtype == dtype and t.shape == shape
            and t.is_contiguous() and (device is None or t.device == device)):
        if device is None or device.type == "cuda":
            return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None:
        _require_device(name, t, device)


def _require_device(name, t, device):
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor (there is no CPU path), got {t.device}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the other tensors on {device}")


def _require_workspace(ws, device):
    """A workspace: a contiguous 1-D uint8 GPU tensor on ``device`` (its size
    is checked by the library against mlstm_workspace_bytes)."""
    if not isinstance(ws, torch.Tensor) or ws.dim() != 1:
        raise ValueError("workspace must be a 1-D tensor (see alloc_workspace)")
    _require("workspace", ws, ws.shape, torch.uint8, device)


def _check_inputs(q, k, v, igate, fgate):
    if not isinstance(q, torch.Tensor):
        raise TypeError(f"q must be a torch.Tensor, got {type(q).__name__}")
    if q.dim() != 4:
        raise ValueError(f"q must be [B, NH, T, d], got shape {tuple(q.shape)}")
    if q.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"q/k/v must be float32 or bfloat16, got {q.dtype}")
    B, NH, T, d = q.shape
    named = (("q", q), ("k", k), ("v", v), ("igate", igate), ("fgate", fgate))
    for name, t in named[:3]:
        _require(name, t, q.shape, q.dtype)
    for name, t in named[3:]:
        _require(name, t, (B, NH, T), torch.float32)
    dev = q.device
    if dev.type == "cuda" and k.device == dev and v.device == dev and igate.device == dev \
            and fgate.device == dev:
        return B, NH, T, d
    for name, t in named:  # devices last: a malformed tensor is named first
        _require_device(name, t, dev)
    return B, NH, T, d


def _stream_ptr(device):
    """The current HIP stream of ``device`` (torch's raw-stream query where
    this build has it: it skips building a Stream object)."""
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None:
        return ctypes.c_void_p(raw(device.index if device.index is not None
                                   else torch.cuda.current_device()))
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _on(device):
    """torch.cuda.device(device), or nothing when it is already current."""
    if device.index is None or device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def parallel_fwd(q, k, v, igate, fgate, out=None):
    """Stabilized parallel mLSTM forward for B x NH heads -> (h, m, n).

    ``out`` may be a tuple (h, m, n) of preallocated outputs.
    """
    lib = load_library()
    B, NH, T, d = _check_inputs(q, k, v, igate, fgate)
    if out is None:
        h = torch.empty_like(q)
        m = torch.empty((B, NH, T), dtype=torch.float32, device=q.device)
        n = torch.empty((B, NH, T), dtype=torch.float32, device=q.device)
    else:
        h, m, n = out
        _require("h", h, q.shape, q.dtype, q.device)
        _require("m", m, (B, NH, T), torch.float32, q.device)
        _require("n", n, (B, NH, T), torch.float32, q.device)
    with _on(q.device):
        st = lib.mlstm_parallel_fwd_stream(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), igate.data_ptr(), fgate.data_ptr(),
            h.data_ptr(), m.data_ptr(), n.data_ptr(), B, NH, T, d, _dtype_code(q),
            _stream_ptr(q.device))
    if st != 0:
        raise MlstmError(st, "mlstm_parallel_fwd")
    return h, m, n


def parallel_fwd_noalloc(q, k, v, igate, fgate, out):
    """parallel_fwd through mlstm_parallel_fwd_noalloc: the library allocates
    nothing (its workspace is a fixed per-GPU array, shared by every call on
    that GPU, so calls must not overlap).  ``out`` = (h, m, n) is required:
    this path allocates no outputs either."""
    lib = load_library()
    B, NH, T, d = _check_inputs(q, k, v, igate, fgate)
    h, m, n = out
    _require("h", h, q.shape, q.dtype, q.device)
    _require("m", m, (B, NH, T), torch.float32, q.device)
    _require("n", n, (B, NH, T), torch.float32, q.device)
    with _on(q.device):
        st = lib.mlstm_parallel_fwd_noalloc(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), igate.data_ptr(), fgate.data_ptr(),
            h.data_ptr(), m.data_ptr(), n.data_ptr(), B, NH, T, d, _dtype_code(q),
            _stream_ptr(q.device))
    if st != 0:
        raise MlstmError(st, "mlstm_parallel_fwd_noalloc")
    return h, m, n


def parallel_fwd_gated(q, k, v, igate, fgate, ogate, htilde=False):
    """Forward pass with the output gate of Eq. 78 fused into the epilogue.

    ogate: O~, same shape, dtype and device as q.  Returns (h, m, n), or
    (h, h_tilde, m, n) with ``htilde=True``, where h = sigmoid(O~) * h_tilde.
    """
    lib = load_library()
    B, NH, T, d = _check_inputs(q, k, v, igate, fgate)
    _require("ogate", ogate, q.shape, q.dtype, q.device)
    h = torch.empty_like(q)
    ht = torch.empty_like(q) if htilde else None
    m = torch.empty((B, NH, T), dtype=torch.float32, device=q.device)
    n = torch.empty((B, NH, T), dtype=torch.float32, device=q.device)
    with _on(q.device):
        st = lib.mlstm_parallel_fwd_gated(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), igate.data_ptr(), fgate.data_ptr(),
            ogate.data_ptr(), h.data_ptr(), ht.data_ptr() if htilde else None, m.data_ptr(),
            n.data_ptr(), B, NH, T, d, _dtype_code(q), _stream_ptr(q.device))
    if st != 0:
        raise MlstmError(st, "mlstm_parallel_fwd_gated")
    return (h, ht, m, n) if htilde else (h, m, n)


def workspace_bytes(B, NH, T):
    return int(load_library().mlstm_workspace_bytes(B, NH, T))


def alloc_workspace(B, NH, T, device):
    """A device workspace for gate_scan / causal_tiles (256-byte aligned)."""
    nbytes = workspace_bytes(B, NH, T)
    if nbytes == 0:
        raise ValueError("invalid sizes")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def gate_scan(igate, fgate, d, workspace, m=None, forget="sigmoid"):
    """Stage 1: m (Eq. 80) and the exponent terms, written into ``workspace``."""
    lib = load_library()
    if not isinstance(igate, torch.Tensor) or igate.dim() != 3:
        raise ValueError("igate must be a [B, NH, T] tensor")
    B, NH, T = igate.shape
    _require("igate", igate, (B, NH, T), torch.float32, igate.device)
    _require("fgate", fgate, (B, NH, T), torch.float32, igate.device)
    _require_workspace(workspace, igate.device)
    if m is None:
        m = torch.empty((B, NH, T), dtype=torch.float32, device=igate.device)
    else:
        _require("m", m, (B, NH, T), torch.float32, igate.device)
    with _on(igate.device):
        st = lib.mlstm_gate_scan(igate.data_ptr(), fgate.data_ptr(), m.data_ptr(),
                                 workspace.data_ptr(), workspace.numel(), B, NH, T, d,
                                 _forget_code(forget), _stream_ptr(igate.device))
    if st != 0:
        raise MlstmError(st, "mlstm_gate_scan")
    return m


def causal_tiles(q, k, v, m, workspace, kernel="auto", out=None):
    """Stage 2: h~ and n from q, k, v and the stage-1 results -> (h, n)."""
    lib = load_library()
    B, NH, T, d = _check_inputs(q, k, v, m, m)
    _require_workspace(workspace, q.device)
    if kernel not in KERNELS:
        raise ValueError(f"kernel must be one of {tuple(KERNELS)}, got {kernel!r}")
    if out is None:
        h = torch.empty_like(q)
        n = torch.empty((B, NH, T), dtype=torch.float32, device=q.device)
    else:
        h, n = out
        _require("h", h, q.shape, q.dtype, q.device)
        _require("n", n, (B, NH, T), torch.float32, q.device)
    with _on(q.device):
        st = lib.mlstm_causal_tiles(q.data_ptr(), k.data_ptr(), v.data_ptr(), m.data_ptr(),
                                    workspace.data_ptr(), workspace.numel(), h.data_ptr(),
                                    n.data_ptr(), B, NH, T, d, _dtype_code(q), KERNELS[kernel],
                                    _stream_ptr(q.device))
    if st != 0:
        raise MlstmError(st, "mlstm_causal_tiles")
    return h, n


def parallel_fwd_staged(q, k, v, igate, fgate, kernel="auto", forget="sigmoid"):
    """Both stages with an explicit workspace and a chosen tile kernel."""
    B, NH, T, d = _check_inputs(q, k, v, igate, fgate)
    ws = alloc_workspace(B, NH, T, q.device)
    m = gate_scan(igate, fgate, d, ws, forget=forget)
    h, n = causal_tiles(q, k, v, m, ws, kernel=kernel)
    return h, m, n


def recurrent_state(B, NH, d, device):
    """A fresh recurrent state (C = 0, n = 0, m = -inf), float32."""
    C = torch.zeros((B, NH, d, d), dtype=torch.float32, device=device)
    n = torch.zeros((B, NH, d), dtype=torch.float32, device=device)
    m = torch.full((B, NH), float("-inf"), dtype=torch.float32, device=device)
    return C, n, m


def recurrent_step(q, k, v, igate, fgate, state, out_state=None, den=False, forget="sigmoid"):
    """One stabilized recurrent step -> (h, new_state[, den]).

    q, k, v: [B, NH, d] (float32 or bfloat16); igate, fgate: [B, NH] float32;
    state = (C [B,NH,d,d], n [B,NH,d], m [B,NH]) float32.  ``out_state``
    receives the new state (its C may be the input C: updated in place); by
    default C is updated in place and new n, m are allocated.
    """
    lib = load_library()
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a [B, NH, d] tensor")
    if q.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"q/k/v must be float32 or bfloat16, got {q.dtype}")
    B, NH, d = q.shape
    C, n, m = state
    for name, t in (("q", q), ("k", k), ("v", v)):
        _require(name, t, q.shape, q.dtype, q.device)
    for name, t, shp in (("igate", igate, (B, NH)), ("fgate", fgate, (B, NH)),
                         ("C", C, (B, NH, d, d)), ("n", n, (B, NH, d)), ("m", m, (B, NH))):
        _require(name, t, shp, torch.float32, q.device)
    if out_state is None:
        out_state = (C, torch.empty_like(n), torch.empty_like(m))
    Co, no, mo = out_state
    for name, t, shp in (("C_out", Co, (B, NH, d, d)), ("n_out", no, (B, NH, d)),
                         ("m_out", mo, (B, NH))):
        _require(name, t, shp, torch.float32, q.device)
    h = torch.empty_like(q)
    dn = torch.empty((B, NH), dtype=torch.float32, device=q.device) if den else None
    with _on(q.device):
        st = lib.mlstm_recurrent_step(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), igate.data_ptr(), fgate.data_ptr(),
            C.data_ptr(), n.data_ptr(), m.data_ptr(), Co.data_ptr(), no.data_ptr(), mo.data_ptr(),
            h.data_ptr(), dn.data_ptr() if den else None, B, NH, d, _dtype_code(q),
            _forget_code(forget), _stream_ptr(q.device))
    if st != 0:
        raise MlstmError(st, "mlstm_recurrent_step")
    return (h, out_state, dn) if den else (h, out_state)


def parallel_fwd_train(q, k, v, igate, fgate, forget="sigmoid"):
    """Forward pass that also returns the row sums b -> (h, m, n, b)."""
    lib = load_library()
    B, NH, T, d = _check_inputs(q, k, v, igate, fgate)
    h = torch.empty_like(q)
    m, n, b = (torch.empty((B, NH, T), dtype=torch.float32, device=q.device) for _ in range(3))
    with _on(q.device):
        st = lib.mlstm_parallel_fwd_train(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), igate.data_ptr(), fgate.data_ptr(),
            h.data_ptr(), m.data_ptr(), n.data_ptr(), b.data_ptr(), B, NH, T, d, _dtype_code(q),
            _forget_code(forget), _stream_ptr(q.device))
    if st != 0:
        raise MlstmError(st, "mlstm_parallel_fwd_train")
    return h, m, n, b


def parallel_bwd(q, k, v, igate, fgate, h, m, n, b, dh, forget="sigmoid"):
    """Gradients (dq, dk, dv, digate, dfgate) of the forward pass given dh = dL/dh~."""
    lib = load_library()
    B, NH, T, d = _check_inputs(q, k, v, igate, fgate)
    for name, t in (("h", h), ("dh", dh)):
        _require(name, t, q.shape, q.dtype, q.device)
    for name, t in (("m", m), ("n", n), ("b", b)):
        _require(name, t, (B, NH, T), torch.float32, q.device)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dig, dfg = torch.empty_like(igate), torch.empty_like(fgate)
    with _on(q.device):
        st = lib.mlstm_parallel_bwd(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), igate.data_ptr(), fgate.data_ptr(),
            h.data_ptr(), m.data_ptr(), n.data_ptr(), b.data_ptr(), dh.data_ptr(),
            dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dig.data_ptr(), dfg.data_ptr(),
            B, NH, T, d, _dtype_code(q), _forget_code(forget), _stream_ptr(q.device))
    if st != 0:
        raise MlstmError(st, "mlstm_parallel_bwd")
    return dq, dk, dv, dig, dfg



def _require_all(named, device):
    """_require for each (name, tensor, shape, dtype), all on ``device``, a GPU.
    The common case in one pass (a call's host time is that of a small kernel);
    on failure the messages of _require, devices last, so that a malformed
    tensor is named first."""
    if device.type == "cuda":
        index = device.index
        for _, t, shape, dtype in named:
            if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
                    and t.get_device() == index and t.is_contiguous()):
                break
        else:
            return
    for name, t, shape, dtype in named:
        _require(name, t, shape, dtype)
    for name, t, _, _ in named:
        _require_device(name, t, device)


def _check_delta(q, k, v, beta, fgate, dims, dh=None, **states):
    """Checks the gated delta rule's tensors (``states``: memories, None where
    they are left out); ``dims`` 4 with a length, 3 for one token."""
    if not isinstance(q, torch.Tensor):
        raise TypeError(f"q must be a torch.Tensor, got {type(q).__name__}")
    if not isinstance(v, torch.Tensor):
        raise TypeError(f"v must be a torch.Tensor, got {type(v).__name__}")
    form = "T, " if dims == 4 else ""
    if q.dim() != dims:
        raise ValueError(f"q must be [B, NHK, {form}dk], got shape {tuple(q.shape)}")
    if v.dim() != dims:
        raise ValueError(f"v must be [B, NH, {form}dv], got shape {tuple(v.shape)}")
    if q.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"q/k/v must be float32 or bfloat16, got {q.dtype}")
    B, NHK, dk = q.shape[0], q.shape[1], q.shape[-1]
    NH, dv = v.shape[1], v.shape[-1]
    T = q.shape[2] if dims == 4 else 1
    rows = (B, NH, T) if dims == 4 else (B, NH)
    named = [("q", q, q.shape, q.dtype), ("k", k, q.shape, q.dtype),
             ("v", v, (*rows, dv), q.dtype), ("beta", beta, rows, torch.float32),
             ("fgate", fgate, rows, torch.float32)]
    if dh is not None:
        named.append(("dh", dh, v.shape, v.dtype))
    for name, t in states.items():
        if t is not None:
            named.append((name, t, (B, NH, dv, dk), torch.float32))
    _require_all(named, q.device)
    return B, NHK, NH, T, dk, dv


def delta_state(B, NH, dk, dv, device):
    """A fresh memory of the gated delta rule: zeros [B, NH, dv, dk], float32."""
    return torch.zeros((B, NH, dv, dk), dtype=torch.float32, device=device)


def _delta_workspace(lib, sizes, dtype, backward, device):
    n = lib.mlstm_delta_workspace_bytes(*sizes, dtype, int(backward))
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def _ptr(t):
    return None if t is None else t.data_ptr()


def delta_fwd(q, k, v, beta, fgate, state=None, out_state=None, forget="sigmoid"):
    """The gated delta rule over a sequence -> (h, new state).

        C_t = f_t C_{t-1} + beta_t (v_t - f_t C_{t-1} k_t) k_t^T,  h_t = C_t q_t / sqrt(dk)

    q, k: [B, NHK, T, dk], v: [B, NH, T, dv] (float32 or bfloat16), NH a
    multiple of NHK (value head n reads key head n // (NH // NHK)); beta, fgate:
    [B, NH, T] float32 (write strengths, forget gate pre-activations).
    ``state``: the memory before the sequence, [B, NH, dv, dk] float32 (zeros by
    default); ``out_state`` receives the memory after it and may be ``state``;
    by default a new one is allocated.
    """
    lib = load_library()
    sizes = _check_delta(q, k, v, beta, fgate, 4, state=state, out_state=out_state)
    B, NHK, NH, T, dk, dv = sizes
    forget_code, code = _forget_code(forget), _dtype_code(q)
    with _on(q.device):
        if out_state is None:
            out_state = torch.empty((B, NH, dv, dk), dtype=torch.float32, device=q.device)
        h = torch.empty_like(v)
        ws = _delta_workspace(lib, sizes, code, False, q.device)
        st = lib.mlstm_delta_fwd(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), beta.data_ptr(), fgate.data_ptr(),
            _ptr(state), h.data_ptr(), out_state.data_ptr(), _ptr(ws),
            0 if ws is None else ws.numel(), *sizes, code, forget_code, _stream_ptr(q.device))
    if st != 0:
        raise MlstmError(st, "mlstm_delta_fwd")
    return h, out_state


def delta_bwd(q, k, v, beta, fgate, dh, state=None, dstate=None, forget="sigmoid"):
    """Gradients of ``delta_fwd`` given dh = dL/dh and ``dstate`` = dL/d(new
    state) (zeros by default) -> (dq, dk, dv, dbeta, dfgate, d(state)).

    q, k, v, beta, fgate, ``state``: as given to ``delta_fwd``.
    """
    lib = load_library()
    if not isinstance(dh, torch.Tensor):
        raise TypeError(f"dh must be a torch.Tensor, got {type(dh).__name__}")
    sizes = _check_delta(q, k, v, beta, fgate, 4, dh=dh, state=state, dstate=dstate)
    B, NHK, NH, T, dk, dv = sizes
    forget_code, code = _forget_code(forget), _dtype_code(q)
    with _on(q.device):
        dq, dk_, dv_ = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        db, df = torch.empty_like(beta), torch.empty_like(fgate)
        dC = torch.empty((B, NH, dv, dk), dtype=torch.float32, device=q.device)
        ws = _delta_workspace(lib, sizes, code, True, q.device)
        st = lib.mlstm_delta_bwd(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), beta.data_ptr(), fgate.data_ptr(),
            _ptr(state), dh.data_ptr(), _ptr(dstate), dq.data_ptr(), dk_.data_ptr(),
            dv_.data_ptr(), db.data_ptr(), df.data_ptr(), dC.data_ptr(), _ptr(ws),
            0 if ws is None else ws.numel(), *sizes, code, forget_code, _stream_ptr(q.device))
    if st != 0:
        raise MlstmError(st, "mlstm_delta_bwd")
    return dq, dk_, dv_, db, df, dC


def delta_step(q, k, v, beta, fgate, state, out_state=None, forget="sigmoid"):
    """One token of the gated delta rule -> (h, new state).

    q, k: [B, NHK, dk], v: [B, NH, dv]; beta, fgate: [B, NH]; ``state`` as for
    ``delta_fwd``, updated in place unless ``out_state`` is given.
    """
    lib = load_library()
    if not isinstance(state, torch.Tensor):
        raise TypeError(f"state must be a torch.Tensor, got {type(state).__name__}")
    B, NHK, NH, _, dk, dv = _check_delta(q, k, v, beta, fgate, 3, state=state,
                                         out_state=out_state)
    if out_state is None:
        out_state = state
    h = torch.empty_like(v)
    with _on(q.device):
        st = lib.mlstm_delta_step(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), beta.data_ptr(), fgate.data_ptr(),
            state.data_ptr(), out_state.data_ptr(), h.data_ptr(), B, NHK, NH, dk, dv,
            _dtype_code(q), _forget_code(forget), _stream_ptr(q.device))
    if st != 0:
        raise MlstmError(st, "mlstm_delta_step")
    return h, out_state


def _check_block_norm(p, weight, gate, residual, scale, next_weight, norm, activation, dr=None,
                      dy=None):
    if not isinstance(p, torch.Tensor):
        raise TypeError(f"p must be a torch.Tensor, got {type(p).__name__}")
    if p.dim() != 4:
        raise ValueError(f"p must be [B, NH, T, d], got shape {tuple(p.shape)}")
    if p.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"p must be float32 or bfloat16, got {p.dtype}")
    B, NH, T, d = p.shape
    D = NH * d
    named = [("p", p, p.shape, p.dtype), ("weight", weight, (D,), torch.float32)]
    if gate is not None:
        named.append(("gate", gate, p.shape, p.dtype))
    if residual is not None:
        named.append(("residual", residual, (B, T, D), p.dtype))
    for name, t in (("scale", scale), ("next_weight", next_weight)):
        if t is not None:
            named.append((name, t, (D,), torch.float32))
    for name, t in (("dr", dr), ("dy", dy)):
        if t is not None:
            named.append((name, t, (B, T, D), p.dtype))
    _require_all(named, p.device)
    if norm not in NORMS:
        raise ValueError(f"norm must be one of {tuple(NORMS)}, got {norm!r}")
    if activation not in GATE_ACTIVATIONS:
        raise ValueError(f"activation must be one of {tuple(GATE_ACTIVATIONS)}, got {activation!r}")
    return B, NH, T, d


def block_norm_fwd(p, weight, gate=None, residual=None, scale=None, next_weight=None,
                   norm="layer", activation="sigmoid", eps=1e-5):
    """The norms, gate and scaled residual between a cell and the next block -> (r, y).

        z = act(gate) * weight * norm(p),  r = residual + scale * z,  y = next_weight * norm(r)

    p, gate: [B, NH, T, d] (a cell's output by heads, each normed over its d
    channels; NH = 1 for plain rows); residual, r, y: [B, T, NH * d] rows, all
    float32 or all bfloat16; weight, scale, next_weight: [NH * d] float32.  What
    is None is left out (y is None without next_weight).  norm: "layer" or
    "rms"; activation of the gate: "sigmoid" or "silu".
    """
    lib = load_library()
    B, NH, T, d = _check_block_norm(p, weight, gate, residual, scale, next_weight, norm,
                                    activation)
    r = torch.empty((B, T, NH * d), dtype=p.dtype, device=p.device)
    y = None if next_weight is None else torch.empty_like(r)
    with _on(p.device):
        st = lib.mlstm_block_norm_fwd(
            p.data_ptr(), _ptr(gate), _ptr(residual), weight.data_ptr(), _ptr(scale),
            _ptr(next_weight), r.data_ptr(), _ptr(y), B, NH, T, d, _dtype_code(p), NORMS[norm],
            GATE_ACTIVATIONS[activation], eps, _stream_ptr(p.device))
    if st != 0:
        raise MlstmError(st, "mlstm_block_norm_fwd")
    return r, y


def block_norm_bwd(p, weight, dr, dy, gate=None, residual=None, scale=None, next_weight=None,
                   norm="layer", activation="sigmoid", eps=1e-5):
    """Gradients of ``block_norm_fwd`` given dr and dy (either may be None; dy
    comes with next_weight) -> a dict with "dp", "dweight" and, for the inputs
    that are given, "dgate", "dresidual", "dscale", "dnext_weight"."""
    lib = load_library()
    B, NH, T, d = _check_block_norm(p, weight, gate, residual, scale, next_weight, norm,
                                    activation, dr, dy)
    if (dy is None) != (next_weight is None):
        raise ValueError("dy and next_weight are given together or not at all")
    g = {"dp": torch.empty_like(p), "dweight": torch.empty_like(weight)}
    for name, t in (("dgate", gate), ("dresidual", residual), ("dscale", scale),
                    ("dnext_weight", next_weight)):
        if t is not None:
            g[name] = torch.empty_like(t)
    ws = torch.empty(lib.mlstm_block_norm_workspace_bytes(B, NH, T, d), dtype=torch.uint8,
                     device=p.device)
    with _on(p.device):
        st = lib.mlstm_block_norm_bwd(
            p.data_ptr(), _ptr(gate), _ptr(residual), weight.data_ptr(), _ptr(scale),
            _ptr(next_weight), _ptr(dr), _ptr(dy), g["dp"].data_ptr(), _ptr(g.get("dgate")),
            _ptr(g.get("dresidual")), g["dweight"].data_ptr(), _ptr(g.get("dscale")),
            _ptr(g.get("dnext_weight")), ws.data_ptr(), ws.numel(), B, NH, T, d, _dtype_code(p),
            NORMS[norm], GATE_ACTIVATIONS[activation], eps, _stream_ptr(p.device))
    if st != 0:
        raise MlstmError(st, "mlstm_block_norm_bwd")
    return g


def _require_rows(named, device):
    """Raise unless each (name, tensor, shape, dtype) is rows of contiguous
    elements with one pitch, on ``device`` -> the pitches, in elements.  ``shape``:
    its first two (B, T) or first (B) sizes count rows, ``row`` elements each."""
    pitches = []
    for name, t, shape, dtype, row in named:
        if t is None:
            pitches.append(row)
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        if t.is_contiguous():
            pitches.append(row)
            continue
        size, stride = list(t.shape), list(t.stride())
        inner, step = 1, 1  # the elements of a row
        while inner < row:
            n, st = size.pop(), stride.pop()
            if n > 1 and st != step:
                raise ValueError(f"{name}'s rows must be contiguous")
            inner, step = inner * n, step * n
        pitch = None  # of the rows: the last dimension with more than one of them
        while size:
            n, st = size.pop(), stride.pop()
            if n > 1 and pitch is None:
                pitch, span = st, st * n
            elif n > 1:
                if st != span:
                    raise ValueError(f"{name}'s rows must be evenly spaced")
                span *= n
        pitches.append(row if pitch is None else pitch)
    for name, t, *_ in named:
        if t is not None:
            _require_device(name, t, device)
    return pitches


def _all_plain(device, checks):
    """Whether every (tensor or None, shape, dtype) is a contiguous tensor of that
    shape and type on ``device``, a GPU: the common case of a call's checks in one
    pass, since a small kernel takes less time than its checks."""
    if device.type != "cuda":
        return False
    index = device.index
    for t, shape, dtype in checks:
        if t is not None and not (isinstance(t, torch.Tensor) and t.dtype is dtype
                                  and t.shape == shape and t.get_device() == index
                                  and t.is_contiguous()):
            return False
    return True


def _named_code(what, table, name):
    if name not in table:
        raise ValueError(f"{what} must be one of {tuple(table)}, got {name!r}")
    return table[name]


def _check_floats(name, t):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")


def _workspace(n, device):
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def _check_conv(x, weight, bias, heads, lengths, dims, states, dy=None):
    _check_floats("x", x)
    if x.dim() != dims:
        raise ValueError(f"x must be [B, {'T, ' if dims == 3 else ''}C], got shape "
                         f"{tuple(x.shape)}")
    if not isinstance(weight, torch.Tensor):
        raise TypeError(f"weight must be a torch.Tensor, got {type(weight).__name__}")
    if weight.dim() != 2:
        raise ValueError(f"weight must be [C, W], got shape {tuple(weight.shape)}")
    B, C, W = x.shape[0], x.shape[-1], weight.shape[1]
    T = x.shape[1] if dims == 3 else 1
    NH = 1 if heads is None else heads
    if not isinstance(NH, int) or NH < 1 or C % NH:
        raise ValueError(f"heads must be a divisor of the {C} channels, got {heads!r}")
    sizes = (B, NH, T, C // NH, W)
    kind, f32, state = x.dtype, torch.float32, (B, W - 1, C)
    y_shape = _conv_shape(B, heads, T, C, dims)
    if _all_plain(x.device, ((x, x.shape, kind), (weight, (C, W), f32), (bias, (C,), f32),
                             (lengths, (B,), torch.int32), (dy, y_shape, kind),
                             *((t, state, kind) for t in states.values()))):
        return C, y_shape, sizes
    x_row, = _require_rows([("x", x, x.shape, x.dtype, C)], x.device)
    named = [("weight", weight, (C, W), torch.float32)]
    if bias is not None:
        named.append(("bias", bias, (C,), torch.float32))
    if lengths is not None:
        named.append(("lengths", lengths, (B,), torch.int32))
    if dy is not None:
        named.append(("dy", dy, y_shape, kind))
    for name, t in states.items():
        if t is not None:
            named.append((name, t, state, kind))
    _require_all(named, x.device)
    return x_row, y_shape, sizes


def _conv_shape(B, heads, T, C, dims):
    """The shape of y: rows without heads, else head-major."""
    if dims == 2:
        return (B, C) if heads is None else (B, heads, C // heads)
    return (B, T, C) if heads is None else (B, heads, T, C // heads)


def conv_state(B, C, width, dtype, device):
    """A fresh state of the short convolution: zeros [B, width - 1, C]."""
    return torch.zeros((B, width - 1, C), dtype=dtype, device=device)


def _short_conv(x, weight, bias, state, out_state, heads, lengths, activation, dims):
    lib = load_library()
    x_row, y_shape, sizes = _check_conv(x, weight, bias, heads, lengths, dims,
                                        {"state": state, "out_state": out_state})
    B, NH, _, d, W = sizes
    code = _named_code("activation", CONV_ACTIVATIONS, activation)
    with _on(x.device):
        if out_state is None:
            out_state = torch.empty((B, W - 1, NH * d), dtype=x.dtype, device=x.device)
        y = torch.empty(y_shape, dtype=x.dtype, device=x.device)
        st = lib.mlstm_short_conv_fwd(
            x.data_ptr(), x_row, weight.data_ptr(), _ptr(bias), _ptr(state), _ptr(lengths),
            y.data_ptr(), out_state.data_ptr(), *sizes, _dtype_code(x), code,
            _stream_ptr(x.device))
    if st != 0:
        raise MlstmError(st, "mlstm_short_conv_fwd")
    return y, out_state


def short_conv_fwd(x, weight, bias=None, state=None, out_state=None, heads=None, lengths=None,
                   activation="silu"):
    """The causal convolution before a recurrent cell -> (y, new state).

        y_t = act(bias + sum_j weight[:, j] x_{t - W + 1 + j})   channel by channel

    x: [B, T, C] float32 or bfloat16, rows of contiguous channels (they may be part
    of wider rows); weight: [C, W] and bias: [C], float32, W from 2 to 8.
    ``state``: the W - 1 inputs before the sequence, [B, W - 1, C] (zeros by
    default); ``out_state`` receives the last W - 1 after it and may be ``state``.
    heads: y is [B, heads, T, C // heads], as the cells read it; None: [B, T, C].
    lengths: [B] int32, each sequence's positions (beyond them y is zeros);
    activation: "silu" or "none".
    """
    return _short_conv(x, weight, bias, state, out_state, heads, lengths, activation, 3)


def short_conv_step(x, weight, state, bias=None, heads=None, out_state=None, activation="silu"):
    """One token of ``short_conv_fwd``: x [B, C] -> (y [B, heads, C // heads] or
    [B, C], new state); ``state`` is updated in place unless ``out_state`` is given."""
    if not isinstance(state, torch.Tensor):
        raise TypeError(f"state must be a torch.Tensor, got {type(state).__name__}")
    return _short_conv(x, weight, bias, state, state if out_state is None else out_state, heads,
                       None, activation, 2)


def short_conv_bwd(x, weight, dy, bias=None, state=None, dstate=None, heads=None, lengths=None,
                   activation="silu"):
    """Gradients of ``short_conv_fwd`` given dy and ``dstate`` = dL/d(new state)
    (zeros by default) -> a dict with "dx", "dweight", with bias "dbias", and
    "dstate", that of the state before the sequence."""
    lib = load_library()
    if not isinstance(dy, torch.Tensor):
        raise TypeError(f"dy must be a torch.Tensor, got {type(dy).__name__}")
    x_row, _, sizes = _check_conv(x, weight, bias, heads, lengths, 3,
                                  {"state": state, "dstate": dstate}, dy)
    B, NH, _, d, W = sizes
    code, dtype = _named_code("activation", CONV_ACTIVATIONS, activation), _dtype_code(x)
    with _on(x.device):
        g = {"dx": torch.empty_like(x, memory_format=torch.contiguous_format),
             "dweight": torch.empty_like(weight)}
        if bias is not None:
            g["dbias"] = torch.empty_like(bias)
        g["dstate"] = torch.empty((B, W - 1, NH * d), dtype=x.dtype, device=x.device)
        ws = _workspace(lib.mlstm_short_conv_workspace_bytes(*sizes, dtype), x.device)
        st = lib.mlstm_short_conv_bwd(
            x.data_ptr(), x_row, weight.data_ptr(), _ptr(bias), _ptr(state), _ptr(lengths),
            dy.data_ptr(), _ptr(dstate), g["dx"].data_ptr(), g["dweight"].data_ptr(),
            _ptr(g.get("dbias")), g["dstate"].data_ptr(), _ptr(ws),
            0 if ws is None else ws.numel(), *sizes, dtype, code, _stream_ptr(x.device))
    if st != 0:
        raise MlstmError(st, "mlstm_short_conv_bwd")
    return g


def _check_scan(u, dt, A, B, C, D, gate, dt_bias, lengths, dims, states, dy=None):
    """Checks the scan's tensors -> (the arguments that a call begins with, sizes);
    ``dims`` 3 with a length, 2 for one token."""
    _check_floats("u", u)
    form = "T, " if dims == 3 else ""
    if u.dim() != dims:
        raise ValueError(f"u must be [B, {form}channels], got shape {tuple(u.shape)}")
    for name, t in (("dt", dt), ("A", A), ("B", B), ("C", C)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if A.dim() != 2:
        raise ValueError(f"A must be [channels, N], got shape {tuple(A.shape)}")
    if B.dim() != dims + 1:
        raise ValueError(f"B must be [B, {form}G, N], got shape {tuple(B.shape)}")
    batch, channels, N, G = u.shape[0], u.shape[-1], A.shape[1], B.shape[-2]
    T = u.shape[1] if dims == 3 else 1
    rows, kind, f32 = u.shape, u.dtype, torch.float32
    shared = (*rows[:-1], G, N)
    sizes, state = (batch, T, channels, G, N), (batch, channels, N)
    if _all_plain(u.device, (
            (u, rows, kind), (dt, rows, kind), (A, (channels, N), f32), (B, shared, kind),
            (C, shared, kind), (D, (channels,), f32), (gate, rows, kind),
            (dt_bias, (channels,), f32), (lengths, (batch,), torch.int32), (dy, rows, kind),
            *((t, state, f32) for t in states.values()))):
        pitches = (channels, channels, G * N, G * N, channels)
        return _scan_args(u, dt, A, B, C, D, gate, dt_bias, states["state"], lengths,
                          pitches), sizes
    pitches = _require_rows([("u", u, rows, kind, channels), ("dt", dt, rows, kind, channels),
                             ("B", B, shared, kind, G * N), ("C", C, shared, kind, G * N),
                             ("gate", gate, rows, kind, channels)], u.device)
    named = [("A", A, (channels, N), torch.float32)]
    for name, t in (("D", D), ("dt_bias", dt_bias)):
        if t is not None:
            named.append((name, t, (channels,), torch.float32))
    if lengths is not None:
        named.append(("lengths", lengths, (batch,), torch.int32))
    if dy is not None:
        named.append(("dy", dy, u.shape, u.dtype))
    for name, t in states.items():
        if t is not None:
            named.append((name, t, state, torch.float32))
    _require_all(named, u.device)
    return _scan_args(u, dt, A, B, C, D, gate, dt_bias, states["state"], lengths, pitches), sizes


def _scan_args(u, dt, A, B, C, D, gate, dt_bias, state, lengths, pitches):
    return (u.data_ptr(), pitches[0], dt.data_ptr(), pitches[1], A.data_ptr(), B.data_ptr(),
            pitches[2], C.data_ptr(), pitches[3], _ptr(D), _ptr(gate), pitches[4], _ptr(dt_bias),
            _ptr(state), _ptr(lengths))


def scan_state(B, channels, N, device):
    """A fresh state of the selective scan: zeros [B, channels, N], float32."""
    return torch.zeros((B, channels, N), dtype=torch.float32, device=device)


def _scan(u, dt, A, B, C, D, gate, dt_bias, state, out_state, lengths, dims):
    lib = load_library()
    args, sizes = _check_scan(u, dt, A, B, C, D, gate, dt_bias, lengths, dims,
                              {"state": state, "out_state": out_state})
    code = _dtype_code(u)
    with _on(u.device):
        if out_state is None:
            out_state = torch.empty((sizes[0], *A.shape), dtype=torch.float32, device=u.device)
        y = torch.empty_like(u, memory_format=torch.contiguous_format)
        ws = None
        if sizes[1] > 1:
            ws = _workspace(lib.mlstm_scan_workspace_bytes(*sizes, code, 0), u.device)
        st = lib.mlstm_scan_fwd(*args, y.data_ptr(), out_state.data_ptr(), _ptr(ws),
                                0 if ws is None else ws.numel(), *sizes, code,
                                _stream_ptr(u.device))
    if st != 0:
        raise MlstmError(st, "mlstm_scan_fwd")
    return y, out_state


def scan_fwd(u, dt, A, B, C, D=None, gate=None, dt_bias=None, state=None, out_state=None,
             lengths=None):
    """The selective state space scan over a sequence -> (y, new state).

        s_t = exp(Delta_t A) s_{t-1} + Delta_t u_t B_t,   Delta_t = softplus(dt_t + dt_bias)
        y_t = (C_t . s_t + D u_t) silu(gate_t)

    u, dt, gate: [B, T, channels], B, C: [B, T, G, N] (channel c reads group
    c // (channels // G)), all float32 or all bfloat16, rows of contiguous elements
    that may be part of wider rows; A: [channels, N], D, dt_bias: [channels],
    float32.  D, gate and dt_bias are left out where None.  ``state``: before the
    sequence, [B, channels, N] float32 (zeros by default); ``out_state`` receives
    the state after it and may be ``state``.  lengths: [B] int32, each sequence's
    positions (beyond them y is zeros and the state stays).
    """
    return _scan(u, dt, A, B, C, D, gate, dt_bias, state, out_state, lengths, 3)


def scan_step(u, dt, A, B, C, state, D=None, gate=None, dt_bias=None, out_state=None):
    """One token of ``scan_fwd``: u, dt, gate [B, channels], B, C [B, G, N] -> (y,
    new state); ``state`` is updated in place unless ``out_state`` is given."""
    if not isinstance(state, torch.Tensor):
        raise TypeError(f"state must be a torch.Tensor, got {type(state).__name__}")
    return _scan(u, dt, A, B, C, D, gate, dt_bias, state,
                 state if out_state is None else out_state, None, 2)


def scan_bwd(u, dt, A, B, C, dy, D=None, gate=None, dt_bias=None, state=None, dstate=None,
             lengths=None):
    """Gradients of ``scan_fwd`` given dy and ``dstate`` = dL/d(new state) (zeros by
    default) -> a dict with "du", "ddt", "dA", "dB", "dC", "dstate" (of the state
    before the sequence) and, for the inputs that are given, "dD", "dgate",
    "ddt_bias"."""
    lib = load_library()
    if not isinstance(dy, torch.Tensor):
        raise TypeError(f"dy must be a torch.Tensor, got {type(dy).__name__}")
    args, sizes = _check_scan(u, dt, A, B, C, D, gate, dt_bias, lengths, 3,
                              {"state": state, "dstate": dstate}, dy)
    code = _dtype_code(u)

    def like(t):
        return None if t is None else torch.empty_like(t, memory_format=torch.contiguous_format)

    with _on(u.device):
        g = {n: like(t) for n, t in (("du", u), ("ddt", dt), ("dA", A), ("dB", B), ("dC", C),
                                     ("dD", D), ("dgate", gate), ("ddt_bias", dt_bias))}
        g["dstate"] = torch.empty((sizes[0], *A.shape), dtype=torch.float32, device=u.device)
        ws = _workspace(lib.mlstm_scan_workspace_bytes(*sizes, code, 1), u.device)
        st = lib.mlstm_scan_bwd(
            *args, dy.data_ptr(), _ptr(dstate), *(_ptr(t) for t in g.values()), _ptr(ws),
            0 if ws is None else ws.numel(), *sizes, code, _stream_ptr(u.device))
    if st != 0:
        raise MlstmError(st, "mlstm_scan_bwd")
    return {n: t for n, t in g.items() if t is not None}


def _check_ffn(x, w_gate, w_up, activation, dh=None):
    _check_floats("x", x)
    if x.dim() < 2:
        raise ValueError(f"x must be [..., D], got shape {tuple(x.shape)}")
    if not isinstance(w_gate, torch.Tensor):
        raise TypeError(f"w_gate must be a torch.Tensor, got {type(w_gate).__name__}")
    if w_gate.dim() != 2:
        raise ValueError(f"w_gate must be [F, D], got shape {tuple(w_gate.shape)}")
    F, D = w_gate.shape[0], x.shape[-1]
    named = [("x", x, x.shape, x.dtype), ("w_gate", w_gate, (F, D), x.dtype),
             ("w_up", w_up, (F, D), x.dtype)]
    if dh is not None:
        named.append(("dh", dh, (*x.shape[:-1], F), x.dtype))
    _require_all(named, x.device)
    return (x.numel() // D if D else 0, D, F), _named_code("activation", FFN_ACTIVATIONS,
                                                           activation)


def gated_ffn_fwd(x, w_gate, w_up, activation="silu"):
    """The gated feed-forward's input half -> h = act(x w_gate^T) * (x w_up^T).

    x: [..., D], w_gate, w_up: [F, D] (as a linear layer's weights), all float32 or
    all bfloat16, contiguous; h: [..., F].  activation: "silu" or "gelu" (g Phi(g)).
    """
    lib = load_library()
    sizes, act = _check_ffn(x, w_gate, w_up, activation)
    code = _dtype_code(x)
    with _on(x.device):
        h = torch.empty((*x.shape[:-1], sizes[2]), dtype=x.dtype, device=x.device)
        ws = _workspace(lib.mlstm_gated_ffn_workspace_bytes(*sizes, code, 0), x.device)
        st = lib.mlstm_gated_ffn_fwd(x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(),
                                     h.data_ptr(), _ptr(ws), 0 if ws is None else ws.numel(),
                                     *sizes, code, act, _stream_ptr(x.device))
    if st != 0:
        raise MlstmError(st, "mlstm_gated_ffn_fwd")
    return h


def gated_ffn_bwd(x, w_gate, w_up, dh, activation="silu"):
    """Gradients of ``gated_ffn_fwd`` given dh -> (dx, dw_gate, dw_up)."""
    lib = load_library()
    if not isinstance(dh, torch.Tensor):
        raise TypeError(f"dh must be a torch.Tensor, got {type(dh).__name__}")
    sizes, act = _check_ffn(x, w_gate, w_up, activation, dh)
    code = _dtype_code(x)
    with _on(x.device):
        dx, dwg, dwu = torch.empty_like(x), torch.empty_like(w_gate), torch.empty_like(w_up)
        ws = _workspace(lib.mlstm_gated_ffn_workspace_bytes(*sizes, code, 1), x.device)
        st = lib.mlstm_gated_ffn_bwd(x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(),
                                     dh.data_ptr(), dx.data_ptr(), dwg.data_ptr(),
                                     dwu.data_ptr(), _ptr(ws), 0 if ws is None else ws.numel(),
                                     *sizes, code, act, _stream_ptr(x.device))
    if st != 0:
        raise MlstmError(st, "mlstm_gated_ffn_bwd")
    return dx, dwg, dwu
