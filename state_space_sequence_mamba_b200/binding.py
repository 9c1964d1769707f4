"""ctypes binding of the C ABI in include/m3.h. Argument marshalling only.

torch supplies device memory and streams; every step of the computation runs in the CUDA
kernels of ``libm3.so``. If the library is missing this module raises: there is no fallback
implementation.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libm3.so")

M3_OK, M3_ERR_INVALID_ARG, M3_ERR_UNSUPPORTED, M3_ERR_CUDA, M3_ERR_TIMEOUT = range(5)
M3_F32, M3_BF16 = 0, 1
# m3_dims.flags: the step scalars arrive raw and the kernels apply softplus / sigmoid; the
# zero-order-hold discretisation; the backward in fp32 on the CUDA cores
M3_DT_SOFTPLUS, M3_LAM_SIGMOID, M3_DISC_ZOH, M3_BWD_FP32 = 1, 2, 4, 8
BWD_FP32 = M3_BWD_FP32
# m3_group_norm_dims.flags
M3_GN_CENTER, M3_GN_SILU = 1, 2
# m3_gated_scan_dims.flags, and the tokens between two of its marks
M3_GS_LERP, M3_GS_BLOCK = 1, 8
# m3_rotary_dims.flags
M3_ROT_INTERLEAVED, M3_ROT_INVERSE, M3_ROT_POS64 = 1, 2, 4
# m3_block_norm_dims.flags
M3_BN_POST_RMS, M3_BN_POST_LAYER, M3_BN_PRE_RMS, M3_BN_PRE_LAYER, M3_BN_SIGMOID, M3_BN_SILU = 1, 2, 4, 8, 16, 32


class M3Error(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"m3 status {status}: {msg}")
        self.status = status


class Dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("nheads", ctypes.c_int64), ("ngroups", ctypes.c_int64),
                ("headdim", ctypes.c_int64), ("dstate", ctypes.c_int64),
                ("rank", ctypes.c_int64), ("chunk", ctypes.c_int64),
                ("in_dtype", ctypes.c_int32), ("bc_norm", ctypes.c_int32),
                ("norm_eps", ctypes.c_float), ("flags", ctypes.c_uint32)]


class Inputs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("x", "B", "C", "theta", "dt", "A", "lam", "B_bias", "C_bias", "dt_bias")]


class StateC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("h", "phi", "prev_B", "prev_x")]


class SegState(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("h", "phi", "lam_sum")]


class Proj(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("x_in", "z_in", "W_X", "W_Z", "W_O")]


class View(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch", ctypes.c_int64), ("token", ctypes.c_int64),
                ("head", ctypes.c_int64)]


class LinattnDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("nseq", "seqlen", "nheads", "qheads", "kheads",
                                              "vheads", "kdim", "vdim")] + [
                   ("in_dtype", ctypes.c_int32), ("scale", ctypes.c_float)]


class LinattnInputs(ctypes.Structure):
    _fields_ = [("q", View), ("k", View), ("v", View), ("log_decay", ctypes.c_void_p),
                ("cu_seqlens", ctypes.c_void_p)]


class LinattnGrads(ctypes.Structure):
    _fields_ = [("dq", View), ("dk", View), ("dv", View)]


class GroupNormDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("rows", ctypes.c_int64), ("channels", ctypes.c_int64),
                ("groups", ctypes.c_int64), ("in_dtype", ctypes.c_int32), ("eps", ctypes.c_float), ("flags", ctypes.c_uint32)]


class GatedScanDims(ctypes.Structure):
    _fields_ = [("nseq", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("channels", ctypes.c_int64),
                ("in_dtype", ctypes.c_int32), ("power", ctypes.c_float), ("flags", ctypes.c_uint32)]


class GatedScanInputs(ctypes.Structure):
    _fields_ = [("x", View), ("r", View), ("i", View), ("decay", ctypes.c_void_p),
                ("cu_seqlens", ctypes.c_void_p)]


class GatedScanGrads(ctypes.Structure):
    _fields_ = [("dx", View), ("dr", View), ("di", View)]


class RotaryDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("nseq", "seqlen", "qheads", "kheads", "headdim", "rotdim",
                                              "offset")] + [
                   ("in_dtype", ctypes.c_int32), ("scale", ctypes.c_float), ("flags", ctypes.c_uint32)]


class BlockNormDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("rows", ctypes.c_int64), ("channels", ctypes.c_int64),
                ("in_dtype", ctypes.c_int32), ("res_dtype", ctypes.c_int32), ("eps", ctypes.c_float),
                ("alpha", ctypes.c_float), ("flags", ctypes.c_uint32)]


class BlockNormInputs(ctypes.Structure):
    _fields_ = [("y", View), ("residual", View), ("z", View)] + [
        (n, ctypes.c_void_p) for n in ("post_weight", "post_bias", "pre_weight", "pre_bias")]


class BlockNormGrads(ctypes.Structure):
    _fields_ = [("dy", View), ("dresidual", View), ("dz", View)] + [
        (n, ctypes.c_void_p) for n in ("dpost_weight", "dpost_bias", "dpre_weight", "dpre_bias")]


class Grads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("dx", "dB", "dC", "dtheta", "ddt", "dA", "dlam",
                                               "dB_bias", "dC_bias", "ddt_bias")]


# Symbols include/m3.h declares (checked by the CPU test suite).
EXPORTS = ("m3_scan_workspace_bytes", "m3_scan_fwd", "m3_decode_step", "m3_scan_check",
           "m3_status_str", "m3_last_error", "m3_scan_fwd_noalloc", "m3_decode_step_proj",
           "m3_scan_state", "m3_state_combine", "m3_scan_bwd_workspace_bytes", "m3_scan_bwd",
           "m3_linattn_workspace_bytes", "m3_linattn_fwd", "m3_linattn_step",
           "m3_linattn_bwd_workspace_bytes", "m3_linattn_bwd", "m3_linattn_check",
           "m3_group_norm_fwd", "m3_group_norm_bwd_workspace_bytes", "m3_group_norm_bwd",
           "m3_gated_scan_fwd", "m3_gated_scan_step", "m3_gated_scan_bwd_workspace_bytes",
           "m3_gated_scan_bwd", "m3_rotary", "m3_block_norm_fwd",
           "m3_block_norm_bwd_workspace_bytes", "m3_block_norm_bwd")

_lib = None


def load_library(path: str = LIB_PATH):
    """Loads libm3.so and declares the signatures. Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with "
                          "`python -m state_space_sequence_mamba_b200.build`")
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER
    lib.m3_scan_workspace_bytes.argtypes = [P(Dims)]
    lib.m3_scan_workspace_bytes.restype = ctypes.c_size_t
    lib.m3_scan_fwd.argtypes = [P(Dims), P(Inputs), P(StateC), P(StateC), ctypes.c_void_p,
                                ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    lib.m3_scan_fwd.restype = ctypes.c_int
    lib.m3_decode_step.argtypes = [P(Dims), P(Inputs), P(StateC), P(StateC), ctypes.c_void_p,
                                   ctypes.c_void_p]
    lib.m3_decode_step.restype = ctypes.c_int
    lib.m3_decode_step_proj.argtypes = [P(Dims), P(Inputs), P(Proj), P(StateC), P(StateC),
                                        ctypes.c_void_p, ctypes.c_void_p]
    lib.m3_decode_step_proj.restype = ctypes.c_int
    lib.m3_scan_state.argtypes = [P(Dims), P(Inputs), P(StateC), P(SegState), ctypes.c_void_p,
                                  ctypes.c_size_t, ctypes.c_void_p]
    lib.m3_scan_state.restype = ctypes.c_int
    lib.m3_state_combine.argtypes = [P(Dims), ctypes.c_int, P(SegState), ctypes.c_void_p,
                                     ctypes.c_void_p, ctypes.c_void_p]
    lib.m3_state_combine.restype = ctypes.c_int
    lib.m3_scan_bwd_workspace_bytes.argtypes = [P(Dims)]
    lib.m3_scan_bwd_workspace_bytes.restype = ctypes.c_size_t
    lib.m3_scan_bwd.argtypes = [P(Dims), P(Inputs), P(StateC), ctypes.c_void_p, P(StateC),
                                P(Grads), P(StateC), ctypes.c_void_p, ctypes.c_size_t,
                                ctypes.c_void_p]
    lib.m3_scan_bwd.restype = ctypes.c_int
    lib.m3_scan_check.argtypes = [ctypes.c_void_p]
    lib.m3_scan_check.restype = ctypes.c_int
    lib.m3_status_str.argtypes = [ctypes.c_int]
    lib.m3_status_str.restype = ctypes.c_char_p
    lib.m3_last_error.argtypes = []
    lib.m3_last_error.restype = ctypes.c_char_p
    lib.m3_scan_fwd_noalloc.argtypes = [P(Dims), P(Inputs), P(StateC), P(StateC),
                                        ctypes.c_void_p, ctypes.c_void_p]
    lib.m3_scan_fwd_noalloc.restype = ctypes.c_int
    _declare_linattn(lib)
    _lib = lib
    return lib


def _declare_linattn(lib):
    P, vp, i64, sz = ctypes.POINTER, ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
    for name in ("m3_linattn_workspace_bytes", "m3_linattn_bwd_workspace_bytes"):
        f = getattr(lib, name)
        f.argtypes, f.restype = [P(LinattnDims), ctypes.c_int], sz
    D, I, V = P(LinattnDims), P(LinattnInputs), P(View)
    lib.m3_linattn_fwd.argtypes = [D, I, vp, vp, V, vp, sz, vp]
    lib.m3_linattn_step.argtypes = [D, I, vp, vp, i64, vp, V, vp]
    lib.m3_linattn_bwd.argtypes = [D, I, vp, V, vp, P(LinattnGrads), vp, vp, sz, vp]
    lib.m3_linattn_check.argtypes = []
    G = P(GroupNormDims)
    lib.m3_group_norm_bwd_workspace_bytes.argtypes = [G]
    lib.m3_group_norm_bwd_workspace_bytes.restype = sz
    lib.m3_group_norm_fwd.argtypes = [G, V, V, vp, vp, V, vp]
    lib.m3_group_norm_bwd.argtypes = [G, V, V, vp, vp, V, V, V, vp, vp, vp, sz, vp]
    S, SI = P(GatedScanDims), P(GatedScanInputs)
    lib.m3_gated_scan_fwd.argtypes = [S, SI, vp, vp, V, vp, vp]
    lib.m3_gated_scan_step.argtypes = [S, SI, vp, vp, i64, vp, V, vp]
    lib.m3_gated_scan_bwd_workspace_bytes.argtypes = [S, ctypes.c_int, ctypes.c_int]
    lib.m3_gated_scan_bwd_workspace_bytes.restype = sz
    lib.m3_gated_scan_bwd.argtypes = [S, SI, vp, vp, V, vp, P(GatedScanGrads), vp, vp, vp, sz, vp]
    lib.m3_rotary.argtypes = [P(RotaryDims), V, V, vp, vp, i64, i64, vp, V, V, vp]
    B, BI = P(BlockNormDims), P(BlockNormInputs)
    lib.m3_block_norm_bwd_workspace_bytes.argtypes = [B]
    lib.m3_block_norm_bwd_workspace_bytes.restype = sz
    lib.m3_block_norm_fwd.argtypes = [B, BI, V, V, vp]
    lib.m3_block_norm_bwd.argtypes = [B, BI, V, V, P(BlockNormGrads), vp, sz, vp]
    for name in ("m3_linattn_fwd", "m3_linattn_step", "m3_linattn_bwd", "m3_linattn_check",
                 "m3_group_norm_fwd", "m3_group_norm_bwd", "m3_gated_scan_fwd", "m3_gated_scan_step",
                 "m3_gated_scan_bwd", "m3_rotary", "m3_block_norm_fwd", "m3_block_norm_bwd"):
        getattr(lib, name).restype = ctypes.c_int


def _check(rc: int):
    if rc != M3_OK:
        lib = load_library()
        raise M3Error(rc, lib.m3_last_error().decode() or lib.m3_status_str(rc).decode())


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return M3_BF16
    if dt == torch.float32:
        return M3_F32
    raise ValueError(f"unsupported input dtype {dt}")


class State:
    """Device state of every (batch, head) unit: h [b,H,N,P] fp32, phi [b,H,N/2] fp32,
    prev_B [b,H,R,N] and prev_x [b,H,R,P] in the input dtype."""

    def __init__(self, h, phi, prev_B, prev_x):
        self.h, self.phi, self.prev_B, self.prev_x = h, phi, prev_B, prev_x

    @staticmethod
    def empty(batch, nheads, dstate, headdim, rank, dtype, device):
        return State(torch.empty(batch, nheads, dstate, headdim, device=device),
                     torch.empty(batch, nheads, dstate // 2, device=device),
                     torch.empty(batch, nheads, rank, dstate, dtype=dtype, device=device),
                     torch.empty(batch, nheads, rank, headdim, dtype=dtype, device=device))

    @staticmethod
    def from_dict(d):
        return State(d["h"], d["phi"], d["prev_B"], d["prev_x"])

    def as_dict(self):
        return dict(h=self.h, phi=self.phi, prev_B=self.prev_B, prev_x=self.prev_x)

    def c(self):
        return StateC(*(_ptr(t) for t in (self.h, self.phi, self.prev_B, self.prev_x)))


def make_dims(x, B, chunk, bc_norm, norm_eps, flags=0):
    b, L, H, R, P = x.shape
    G, N = B.shape[2], B.shape[4]
    return Dims(b, L, H, G, P, N, R, int(chunk), _dtype_code(x.dtype), 1 if bc_norm else 0,
                float(norm_eps), int(flags))


def scan_workspace_bytes(dims: Dims) -> int:
    return int(load_library().m3_scan_workspace_bytes(ctypes.byref(dims)))


def _stream_handle(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def scan_fwd(x, B, C, theta, dt, A, lam, B_bias=None, C_bias=None, init: State | None = None,
             final: State | None | bool = True, y=None, workspace=None, chunk=64,
             bc_norm=False, norm_eps=1e-6, stream=None, dt_bias=None, flags=0):
    """m3_scan_fwd on torch CUDA tensors (shapes as in include/m3.h). ``flags``
    (M3_DT_SOFTPLUS | M3_LAM_SIGMOID) passes dt and lam raw, with ``dt_bias`` [H].

    ``final=True`` allocates a new State for the result, ``False``/None skips it, or pass a
    State (it may be ``init`` itself). Returns (y, final State or None)."""
    lib = load_library()
    dims = make_dims(x, B, chunk, bc_norm, norm_eps, flags)
    dev = x.device
    if y is None:
        y = torch.empty_like(x)
    if final is True:
        final = State.empty(dims.batch, dims.nheads, dims.dstate, dims.headdim, dims.rank,
                            x.dtype, dev)
    elif final is False:
        final = None
    need = scan_workspace_bytes(dims)
    if need == 0:
        # invalid or unsupported dims: let the call report why
        need = 256
    if workspace is None:
        workspace = torch.zeros(need, dtype=torch.uint8, device=dev)
    ins = Inputs(*(_ptr(t) for t in (x, B, C, theta, dt, A, lam, B_bias, C_bias, dt_bias)))
    ic = init.c() if init is not None else None
    fc = final.c() if final is not None else None
    rc = lib.m3_scan_fwd(ctypes.byref(dims), ctypes.byref(ins),
                         ctypes.byref(ic) if ic is not None else None,
                         ctypes.byref(fc) if fc is not None else None,
                         _ptr(y), _ptr(workspace), workspace.numel(), _stream_handle(stream))
    _check(rc)
    return y, final


def scan_check(workspace):
    _check(load_library().m3_scan_check(_ptr(workspace)))


def decode_step(x, B, C, theta, dt, A, lam, B_bias=None, C_bias=None, state_in: State = None,
                state_out: State | None = None, y=None, bc_norm=False, norm_eps=1e-6,
                stream=None, dt_bias=None, flags=0):
    """m3_decode_step: x [b,1,H,R,P], B, C [b,1,G,R,N], theta [b,1,H,N/2], dt/A/lam [b,1,H].

    ``state_out`` defaults to ``state_in`` (in-place). Returns (y [b,H,R,P], state_out)."""
    lib = load_library()
    dims = make_dims(x, B, 1, bc_norm, norm_eps, flags)
    if state_out is None:
        state_out = state_in
    if y is None:
        y = torch.empty(dims.batch, dims.nheads, dims.rank, dims.headdim, dtype=x.dtype,
                        device=x.device)
    ins = Inputs(*(_ptr(t) for t in (x, B, C, theta, dt, A, lam, B_bias, C_bias, dt_bias)))
    si, so = state_in.c(), state_out.c()
    rc = lib.m3_decode_step(ctypes.byref(dims), ctypes.byref(ins), ctypes.byref(si),
                            ctypes.byref(so), _ptr(y), _stream_handle(stream))
    _check(rc)
    return y, state_out


def decode_step_proj(xp, zp, W_X, W_Z, W_O, B, C, theta, dt, A, lam, B_bias=None, C_bias=None,
                     state_in: State = None, state_out: State | None = None, o=None,
                     bc_norm=False, norm_eps=1e-6, stream=None, dt_bias=None, flags=0):
    """m3_decode_step_proj: one token with the MIMO projections. xp, zp [b,1,H,P] (X', Z');
    W_X, W_Z, W_O [H,R,P] fp32; B, C [b,1,G,R,N]; theta [b,1,H,N/2]; dt/A/lam [b,1,H].
    ``state_out`` defaults to ``state_in``. Returns (O' [b,H,P], state_out)."""
    lib = load_library()
    b, _, H, P = xp.shape
    R = W_X.shape[1]
    dims = make_dims(xp.reshape(b, 1, H, 1, P).expand(b, 1, H, R, P), B, 1, bc_norm, norm_eps,
                     flags)
    if state_out is None:
        state_out = state_in
    if o is None:
        o = torch.empty(b, H, P, dtype=xp.dtype, device=xp.device)
    ins = Inputs(*(_ptr(t) for t in (None, B, C, theta, dt, A, lam, B_bias, C_bias, dt_bias)))
    pr = Proj(*(_ptr(t) for t in (xp, zp, W_X, W_Z, W_O)))
    si, so = state_in.c(), state_out.c()
    rc = lib.m3_decode_step_proj(ctypes.byref(dims), ctypes.byref(ins), ctypes.byref(pr),
                                 ctypes.byref(si), ctypes.byref(so), _ptr(o),
                                 _stream_handle(stream))
    _check(rc)
    return o, state_out


def scan_state(x, B, C, theta, dt, A, lam, B_bias=None, C_bias=None, init: State | None = None,
               chunk=64, bc_norm=False, norm_eps=1e-6, stream=None, dt_bias=None, flags=0,
               workspace=None):
    """m3_scan_state: the state after the last token (h [b,H,N,P], phi [b,H,N/2]) and the summed
    log-decay [b,H], without y. Returns (h, phi, lam_sum)."""
    lib = load_library()
    dims = make_dims(x, B, chunk, bc_norm, norm_eps, flags)
    b, L, H, R, P = x.shape
    N = B.shape[4]
    dev = x.device
    h = torch.empty(b, H, N, P, device=dev)
    phi = torch.empty(b, H, N // 2, device=dev)
    lam_sum = torch.empty(b, H, device=dev)
    if workspace is None:
        workspace = torch.zeros(max(256, scan_workspace_bytes(dims)), dtype=torch.uint8,
                                device=dev)
    ins = Inputs(*(_ptr(t) for t in (x, B, C, theta, dt, A, lam, B_bias, C_bias, dt_bias)))
    ic = init.c() if init is not None else None
    out = SegState(_ptr(h), _ptr(phi), _ptr(lam_sum))
    rc = lib.m3_scan_state(ctypes.byref(dims), ctypes.byref(ins),
                           ctypes.byref(ic) if ic is not None else None, ctypes.byref(out),
                           _ptr(workspace), workspace.numel(), _stream_handle(stream))
    _check(rc)
    return h, phi, lam_sum


def state_combine(h, phi, lam_sum, stream=None):
    """m3_state_combine on stacked segment states h [S,b,H,N,P], phi [S,b,H,N/2], lam_sum
    [S,b,H]: the state after segment S-1. Returns (h [b,H,N,P], phi [b,H,N/2])."""
    lib = load_library()
    S, b, H, N, P = h.shape
    dims = Dims(b, 1, H, 1, P, N, 1, 1, M3_F32, 0, 1e-6, 0)
    h_out = torch.empty(b, H, N, P, device=h.device)
    phi_out = torch.empty(b, H, N // 2, device=h.device)
    seg = SegState(_ptr(h), _ptr(phi), _ptr(lam_sum))
    rc = lib.m3_state_combine(ctypes.byref(dims), int(S), ctypes.byref(seg), _ptr(h_out),
                              _ptr(phi_out), _stream_handle(stream))
    _check(rc)
    return h_out, phi_out


def scan_bwd_workspace_bytes(dims: Dims) -> int:
    return int(load_library().m3_scan_bwd_workspace_bytes(ctypes.byref(dims)))


def scan_bwd(x, B, C, theta, dt, A, lam, dy, B_bias=None, C_bias=None, init: State | None = None,
             dfinal: dict | None = None, bc_norm=False, norm_eps=1e-6, stream=None, dt_bias=None,
             flags=0, want_init=True, workspace=None):
    """m3_scan_bwd: gradients of sum(y * dy) + <final state, dfinal> for the forward that
    scan_fwd runs on the same arguments. ``dfinal``: dict of fp32 h, phi, prev_B, prev_x (any
    may be missing = 0). Returns a dict of fp32 tensors dx, dB, dC, dtheta, ddt, dA, dlam,
    dB_bias, dC_bias, ddt_bias and (with want_init) dinit, a dict of the initial state's."""
    lib = load_library()
    dims = make_dims(x, B, 1, bc_norm, norm_eps, flags)
    b, L, H, R, P = x.shape
    G, N = B.shape[2], B.shape[4]
    dev = x.device
    f32 = dict(device=dev, dtype=torch.float32)
    g = dict(dx=torch.empty(b, L, H, R, P, **f32), dB=torch.empty(b, L, G, R, N, **f32),
             dC=torch.empty(b, L, G, R, N, **f32), dtheta=torch.empty(b, L, H, N // 2, **f32),
             ddt=torch.empty(b, L, H, **f32), dA=torch.empty(b, L, H, **f32),
             dlam=torch.empty(b, L, H, **f32), dB_bias=torch.empty(H, R, N, **f32),
             dC_bias=torch.empty(H, R, N, **f32), ddt_bias=torch.empty(H, **f32))
    gc = Grads(*(_ptr(g[k]) for k in ("dx", "dB", "dC", "dtheta", "ddt", "dA", "dlam",
                                       "dB_bias", "dC_bias", "ddt_bias")))
    dinit = None
    if want_init:
        dinit = dict(h=torch.empty(b, H, N, P, **f32), phi=torch.empty(b, H, N // 2, **f32),
                     prev_B=torch.empty(b, H, R, N, **f32), prev_x=torch.empty(b, H, R, P, **f32))
    if workspace is None:
        workspace = torch.empty(max(256, scan_bwd_workspace_bytes(dims)), dtype=torch.uint8,
                                device=dev)
    ins = Inputs(*(_ptr(t) for t in (x, B, C, theta, dt, A, lam, B_bias, C_bias, dt_bias)))
    ic = init.c() if init is not None else None
    df = None
    if dfinal is not None:
        df = StateC(*(_ptr(dfinal.get(k)) for k in ("h", "phi", "prev_B", "prev_x")))
    di = StateC(*(_ptr(dinit[k]) for k in ("h", "phi", "prev_B", "prev_x"))) if dinit else None
    rc = lib.m3_scan_bwd(ctypes.byref(dims), ctypes.byref(ins),
                         ctypes.byref(ic) if ic is not None else None, _ptr(dy),
                         ctypes.byref(df) if df is not None else None, ctypes.byref(gc),
                         ctypes.byref(di) if di is not None else None, _ptr(workspace),
                         workspace.numel(), _stream_handle(stream))
    _check(rc)
    g["dinit"] = dinit
    return g


# ---- linear attention with a decay for each head, the grouped norm behind it, the gated scan, rotary
# positions and the norms around a block ----
# Marshalled in C++ (csrc/m3_torch.cpp), since these calls' kernels may be as short as the
# marshalling. They run on the tensors' device and, unless a stream is given, on its current
# stream; what they allocate is allocated on the stream they run on. They are no autograd functions:
# results are detached from inputs that require a gradient, whose gradients the _bwd calls
# (and rotary with ``inverse``) compute; tensors given to be written count as changed. Wrong shapes, types, strides
# and devices raise ValueError, the library's own refusals M3Error.

_native = None


def _ext():
    """The native marshalling module, bound to the loaded library. Raises if it is missing."""
    global _native
    if _native is None:
        lib = load_library()
        from .build import TORCH_EXT, ext_target
        try:
            from . import _m3torch
            if _m3torch.built_for != ext_target():
                raise ImportError(f"built for {_m3torch.built_for}")
        except ImportError as e:
            raise ImportError(f"{TORCH_EXT} does not load under {ext_target()}: build it with "
                              "`python -m state_space_sequence_mamba_b200.build`") from e
        _m3torch.bind(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in (
            "m3_linattn_workspace_bytes", "m3_linattn_bwd_workspace_bytes", "m3_linattn_fwd",
            "m3_linattn_step", "m3_linattn_bwd", "m3_group_norm_fwd",
            "m3_group_norm_bwd_workspace_bytes", "m3_group_norm_bwd", "m3_gated_scan_fwd",
            "m3_gated_scan_step", "m3_gated_scan_bwd_workspace_bytes", "m3_gated_scan_bwd", "m3_rotary",
            "m3_block_norm_fwd", "m3_block_norm_bwd_workspace_bytes", "m3_block_norm_bwd")))
        _native = _m3torch
    return _native


def _run(name, stream, ref, *args):
    f = getattr(_native or _ext(), name)
    if stream is None:
        r = f(*args)
    else:
        if stream.device != ref.device:
            raise ValueError(f"stream on {stream.device}, tensors on {ref.device}")
        with torch.cuda.stream(stream):
            r = f(*args)
    if type(r) is int:
        _check(r)
    return r


def linattn_workspace_bytes(dims: LinattnDims, packed=False, backward=False) -> int:
    lib = load_library()
    f = lib.m3_linattn_bwd_workspace_bytes if backward else lib.m3_linattn_workspace_bytes
    return f(ctypes.byref(dims), int(packed))


def linattn_fwd(q, k, v, log_decay, scale=1.0, init=None, final=True, o=None, cu_seqlens=None,
                workspace=None, stream=None):
    """m3_linattn_fwd: linear attention with decay exp(log_decay[h]) over prompts.

    q [b, L, Hq, K], k [b, L, Hk, K], v [b, L, Hv, V] (any strides, the last dimension
    contiguous), log_decay [H] fp32 with Hq, Hk and Hv dividing H, init [b, H, K, V] fp32 or None.
    ``cu_seqlens`` [n + 1] int32: n sequences packed in tensors of batch 1, states [n, H, K, V].
    ``final=True`` allocates the final state, ``False``/None skips it, or pass a tensor (it may be
    ``init``). ``o`` [b, L, H, V] is allocated unless given (packed: zeroed, since rows behind the
    last sequence are not written). Returns (o, final state or None)."""
    return _run("linattn_fwd", stream, q, q, k, v, log_decay, scale, init, final, o, cu_seqlens, workspace)


def linattn_step(q, k, v, log_decay, state, state_out=None, slots=None, scale=1.0, o=None,
                 stream=None):
    """m3_linattn_step: one token of every sequence. q [b, Hq, K], k [b, Hk, K], v [b, Hv, V];
    ``state`` [b, H, K, V] fp32, or with ``slots`` [b] int32 a pool [n, H, K, V] of which sequence
    i has state slots[i] (outside [0, n): the sequence is skipped and its o row is zero).
    ``state_out`` defaults to ``state`` (in place). Returns (o [b, H, V], state_out)."""
    return _run("linattn_step", stream, q, q, k, v, log_decay, scale, state, state_out, slots, o)


def linattn_bwd(q, k, v, log_decay, do, scale=1.0, init=None, dfinal=None, cu_seqlens=None,
                grads=None, want_init=True, workspace=None, stream=None):
    """m3_linattn_bwd: gradients of sum(o * do) + <final state, dfinal> for linattn_fwd on the
    same arguments. do [b, L, H, V]; ``grads``: tensors (dq, dk, dv) to write, in the input's type
    and shapes (packed: allocated ones are zeroed, since rows behind the last sequence are not
    written). Returns a dict of dq, dk, dv and dinit ([n, H, K, V] fp32; None without
    ``want_init``; pass a tensor as ``want_init`` to have it written there)."""
    dq, dk, dv = grads if grads is not None else (None, None, None)
    r = _run("linattn_bwd", stream, q, q, k, v, log_decay, scale, do, init, dfinal, cu_seqlens,
             dq, dk, dv, want_init, workspace)
    return dict(dq=r[0], dk=r[1], dv=r[2], dinit=r[3])


def linattn_check(device=None):
    """m3_linattn_check on a device (the current one): raises M3Error after a timed-out wait."""
    with torch.cuda.device(device):
        _check(load_library().m3_linattn_check())


def group_norm_fwd(x, groups, weight=None, bias=None, z=None, center=True, silu=True, eps=1e-5,
                   out=None, stream=None):
    """m3_group_norm_fwd: x [..., C] normalised over each row's groups of C / groups channels,
    times weight plus bias (fp32 [C], optional), then times silu(z) with a gate ``z`` [..., C],
    or through silu without one (``silu=False``: times z, or as it is). ``center=False`` divides
    by the root mean square instead. Rows may be slices of wider ones. Returns out."""
    return _run("group_norm_fwd", stream, x, x, groups, weight, bias, z, center, silu, eps, out)


def group_norm_bwd(dout, x, groups, weight=None, bias=None, z=None, center=True, silu=True,
                   eps=1e-5, dx=None, dz=None, workspace=None, stream=None):
    """m3_group_norm_bwd: gradients of sum(out * dout) for group_norm_fwd on the same arguments.
    Returns a dict of dx, dz (None without z), dweight and dbias (fp32 [C]; None without weight
    or bias)."""
    r = _run("group_norm_bwd", stream, x, dout, x, groups, weight, bias, z, center, silu, eps, dx, dz,
             workspace)
    return dict(dx=r[0], dz=r[1], dweight=r[2], dbias=r[3])


def gated_scan_fwd(x, r, i=None, decay=None, power=8.0, lerp=False, init=None, final=True, y=None,
                   cu_seqlens=None, marks=False, stream=None):
    """m3_gated_scan_fwd: the gated linear recurrence h_t = a_t h_{t-1} + w_t sigmoid(i_t) x_t of every
    channel over prompts, with a_t = exp(-power softplus(decay) sigmoid(r_t)) and w_t = sqrt(1 - a_t^2), or with
    ``lerp`` a_t = sigmoid(r_t + decay) and w_t = 1 - a_t.

    x, r, i [b, L, C] (any strides, channels contiguous; no ``i``: no input gate), decay [C] fp32 (optional with
    ``lerp``), init [b, C] fp32 or None. ``cu_seqlens`` [n + 1] int32, not descending: n sequences packed in
    tensors of batch 1, states [n, C]. ``final=True`` allocates the final state, ``False``/None skips it, or
    pass a tensor (it may be ``init``). ``y`` is allocated unless given (packed: zeroed, since rows of no sequence
    are not written). ``marks=True`` allocates the states that spare gated_scan_bwd a pass, [b or 1,
    ceil(L / 8), C] fp32, or pass a tensor. Returns (y, final state or None, marks or None)."""
    return _run("gated_scan_fwd", stream, x, x, r, i, decay, power, lerp, init, final, y, cu_seqlens, marks)


def gated_scan_step(x, r, state, i=None, decay=None, power=8.0, lerp=False, state_out=None, slots=None,
                    y=None, stream=None):
    """m3_gated_scan_step: one token of every sequence. x, r, i [b, C]; ``state`` [b, C] fp32, or with
    ``slots`` [b] int32 a pool [n, C] of which sequence s has state slots[s] (outside [0, n): the sequence is
    skipped and its y row is zero). ``state_out`` defaults to ``state`` (in place). Returns (y, state_out)."""
    return _run("gated_scan_step", stream, x, x, r, i, decay, power, lerp, state, state_out, slots, y)


def gated_scan_bwd(dy, x, r, i=None, decay=None, power=8.0, lerp=False, init=None, dfinal=None,
                   cu_seqlens=None, marks=None, grads=None, want_init=True, workspace=None, stream=None):
    """m3_gated_scan_bwd: gradients of sum(y * dy) + <final state, dfinal> for gated_scan_fwd on the same
    arguments. ``marks``: that call's, or None (one more pass over the inputs). ``grads``: tensors (dx, dr, di) to
    write (di None without ``i``; packed: allocated ones are zeroed). Returns a dict of dx, dr, di (None without
    ``i``), ddecay ([C] fp32; None without ``decay``) and dinit ([n, C] fp32; None without ``want_init``;
    pass a tensor to have it written there)."""
    dx, dr, di = grads if grads is not None else (None, None, None)
    g = _run("gated_scan_bwd", stream, x, x, r, i, decay, power, lerp, dy, init, dfinal, cu_seqlens, marks,
             dx, dr, di, want_init, workspace)
    return dict(dx=g[0], dr=g[1], di=g[2], ddecay=g[3], dinit=g[4])


def rotary_frequencies(rotdim, base=10000.0, scaling=None, factor=1.0, trained=8192, fast=32.0, slow=1.0,
                       device=None):
    """The frequencies [rotdim / 2] (fp64, radians per position) for ``rotary``, and the scale that goes with them.

    base^(-2 j / rotdim), reaching ``factor`` times beyond ``trained`` tokens by ``scaling``: None;
    "linear" (all divided by the factor); "ntk" (base times factor^(rotdim / (rotdim - 2)), which divides the
    slowest one by it); "yarn" (pairs that turn more than ``fast`` times in ``trained`` tokens stay, those
    below ``slow`` turns are divided, a ramp over the pairs between; scale 0.1 ln(factor) + 1); "bands" (the
    same with a ramp over the turns themselves, scale 1; use fast=4)."""
    if rotdim < 0 or rotdim % 2:
        raise ValueError(f"rotdim must be even and >= 0, not {rotdim}")
    if scaling not in (None, "linear", "ntk", "yarn", "bands"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if not (base > 1 and factor > 0 and trained > 0 and fast > slow > 0):
        raise ValueError("base > 1, factor > 0, trained > 0 and fast > slow > 0 are needed")
    n, scale = rotdim, 1.0
    if scaling == "ntk" and n > 2:
        base = base * factor ** (n / (n - 2))
    j = torch.arange(n // 2, dtype=torch.float64)
    f = base ** (-2 * j / max(n, 1))
    keep = torch.ones_like(f)
    if scaling == "linear":
        keep = torch.zeros_like(f)
    elif scaling == "yarn":
        lo, hi = (n * math.log(trained / (t * 2 * math.pi)) / (2 * math.log(base)) for t in (fast, slow))
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), n - 1)
        keep = 1 - ((j - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        scale = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    elif scaling == "bands":
        keep = ((trained * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
    return (f / factor * (1 - keep) + f * keep).to(device), scale


def rotary(q, k, freq, positions=None, offset=0, cu_seqlens=None, interleaved=False, inverse=False,
           scale=1.0, q_out=None, k_out=None, stream=None):
    """m3_rotary: q [b, L, Hq, D] (a step: [b, Hq, D]) and k (or None) with the first 2 len(freq) dimensions of
    every head turned by position * freq, pairs (j, j + len(freq)) or with ``interleaved`` (2 j, 2 j + 1), times
    ``scale``; the rest is copied. ``inverse`` turns back: the gradient. freq: fp64 (``rotary_frequencies``).
    ``positions``: int32 or int64 [b, L] or [L] (a step: [b]), or None: the token's index in its sequence
    (``cu_seqlens`` [n + 1] int32: n sequences packed in tensors of batch 1); ``offset`` is added. ``q_out``
    and ``k_out`` are allocated unless given (packed: zeroed) and may be q and k. Returns (q_out, k_out)."""
    return _run("rotary", stream, q, q, k, freq, positions, offset, cu_seqlens, interleaved, inverse, scale,
                q_out, k_out)


_POST = {None: 0, "rms": M3_BN_POST_RMS, "layer": M3_BN_POST_LAYER}
_PRE = {None: 0, "rms": M3_BN_PRE_RMS, "layer": M3_BN_PRE_LAYER}
_GATE = {None: 0, "sigmoid": M3_BN_SIGMOID, "silu": M3_BN_SILU}


def _block_flags(post, pre, gate):
    for name, value, known in (("post", post, _POST), ("pre", pre, _PRE), ("gate", gate, _GATE)):
        if value not in known:
            raise ValueError(f"{name} must be one of {tuple(known)}, not {value!r}")
    return _POST[post] | _PRE[pre] | _GATE[gate]


def block_norm_fwd(y, residual, z=None, gate=None, alpha=1.0, post=None, post_weight=None, post_bias=None,
                   pre="rms", pre_weight=None, pre_bias=None, eps=1e-5, h=None, out=None, stream=None):
    """m3_block_norm_fwd: what stands between two blocks, in one pass: h = residual + alpha post(y) act(z),
    out = pre(h). y, z, out [..., C]; residual, h [..., C] of y's type or fp32. post and pre: None, "rms" or
    "layer" (mean taken off), times weight plus bias (fp32 [C], optional; post's also without its norm). ``gate``:
    None (z as it is), "sigmoid" or "silu". Rows may be slices of wider ones, z may be expanded over rows. h may
    be residual, out may be y. Returns (h, out or None)."""
    return _run("block_norm_fwd", stream, y, y, residual, z, post_weight, post_bias, pre_weight, pre_bias,
                alpha, eps, _block_flags(post, pre, gate), h, out)


def block_norm_bwd(dh, dout, y, residual, z=None, gate=None, alpha=1.0, post=None, post_weight=None,
                   post_bias=None, pre="rms", pre_weight=None, pre_bias=None, eps=1e-5, dy=None,
                   dresidual=None, dz=None, workspace=None, stream=None):
    """m3_block_norm_bwd: gradients of sum(h * dh) + sum(out * dout) for block_norm_fwd on the same arguments;
    dh None: zero, dout None: without a pre norm. dresidual may be dh, dy may be dout. Returns a dict of dy,
    dresidual, dz (None without z; of z's full shape where it is expanded), and dpost_weight, dpost_bias,
    dpre_weight, dpre_bias (fp32 [C]; None where the parameter is)."""
    g = _run("block_norm_bwd", stream, y, y, residual, z, post_weight, post_bias, pre_weight, pre_bias, alpha,
             eps, _block_flags(post, pre, gate), dh, dout, dy, dresidual, dz, workspace)
    return dict(zip(("dy", "dresidual", "dz", "dpost_weight", "dpost_bias", "dpre_weight", "dpre_bias"), g))
