"""Thin Python binding of ``libssm.so`` (ctypes; argument marshalling only).

Every function here has the name of the C entry point it calls.  Tensors
are torch CUDA tensors; this module only checks that they are contiguous
CUDA tensors of the expected dtype, allocates outputs when the caller does
not pass them (PyTorch is the memory allocator), and passes raw pointers
and the current CUDA stream.  All arithmetic happens in the library's
kernels.  There is no fallback: if the library is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libssm.so")

SSM_F32, SSM_BF16 = 0, 1
_DT = {torch.float32: SSM_F32, torch.bfloat16: SSM_BF16}
_TORCH_DT = {SSM_F32: torch.float32, SSM_BF16: torch.bfloat16}

STATUS_NAMES = {0: "SSM_OK", 1: "SSM_ERR_NULL", 2: "SSM_ERR_SHAPE", 3: "SSM_ERR_ALIGN",
                4: "SSM_ERR_DTYPE", 5: "SSM_ERR_UNSUPPORTED", 6: "SSM_ERR_WORKSPACE",
                7: "SSM_ERR_TIMEOUT", 8: "SSM_ERR_CUDA", 9: "SSM_ERR_ALIAS"}

# every symbol include/ssm.h declares
EXPORTS = ["ssm_abi_version", "ssm_status_string", "ssm_scan_workspace_bytes", "ssm_scan_fwd",
           "ssd_chunked_fwd", "ssd_mamba3_fwd", "ssd_mamba3_mimo_fwd", "ssm_decode_step",
           "ssm_decode_step_mamba3", "ssm_decode_step_mamba3_mimo", "ssm_last_device_status",
           "ssm_scan_fwd_noalloc", "ssm_scan_bwd_workspace_bytes", "ssm_scan_bwd",
           "ssd_chunked_bwd_workspace_bytes", "ssd_chunked_bwd", "ssm_scan_fwd_host_workspace_bytes",
           "ssm_scan_fwd_host", "ssm_scan_checkpoint_bytes", "ssm_scan_fwd_ckpt",
           "ssd_chunked_checkpoint_bytes", "ssd_chunked_fwd_ckpt", "ssd_mamba3_bwd_workspace_bytes",
           "ssd_mamba3_bwd", "ssd_mamba3_mimo_bwd_workspace_bytes", "ssd_mamba3_mimo_bwd",
           "ssd_mamba3_fwd_ckpt", "ssd_mamba3_mimo_fwd_ckpt", "ssm_debug_set_lookback",
           "ssm_debug_set_scan_path", "ssm_noalloc_last_status", "ssm_mamba3_rope",
           "ssm_add_rmsnorm_fwd", "ssm_add_rmsnorm_e4m3_fwd", "ssm_add_rmsnorm_bwd_workspace_bytes",
           "ssm_add_rmsnorm_bwd", "ssm_linrec_checkpoint_bytes", "ssm_linrec_workspace_bytes",
           "ssm_linrec_fwd", "ssm_linrec_bwd_workspace_bytes", "ssm_linrec_bwd",
           "ssm_vocab_ce_workspace_bytes", "ssm_vocab_ce_fwd", "ssm_vocab_ce_bwd_workspace_bytes",
           "ssm_vocab_ce_bwd", "ssm_qk_norm_rope_fwd", "ssm_qk_norm_rope_bwd_workspace_bytes",
           "ssm_qk_norm_rope_bwd", "ssm_gated_delta_checkpoint_bytes",
           "ssm_gated_delta_workspace_bytes", "ssm_gated_delta_walked_steps", "ssm_gated_delta_fwd",
           "ssm_gated_delta_bwd_workspace_bytes", "ssm_gated_delta_bwd"]


class SSMError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)} "
                         f"({status_string(status)})")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it first "
                               "(python -c 'import __graft_entry__ as g; g.build()')")
        L = ctypes.CDLL(LIB_PATH)
        vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L.ssm_abi_version.restype = i
        L.ssm_status_string.restype = ctypes.c_char_p
        L.ssm_status_string.argtypes = [i]
        L.ssm_scan_workspace_bytes.restype = sz
        L.ssm_scan_workspace_bytes.argtypes = [i] * 5
        L.ssm_scan_fwd.restype = i
        L.ssm_scan_fwd.argtypes = [vp] * 8 + [i] + [vp] * 3 + [i] * 7 + [vp, sz, vp]
        L.ssd_chunked_fwd.restype = i
        L.ssd_chunked_fwd.argtypes = [vp] * 5 + [i] + [vp] * 3 + [i] * 8 + [vp]
        L.ssm_decode_step.restype = i
        L.ssm_decode_step.argtypes = [vp] * 9 + [i] * 6 + [vp]
        L.ssd_mamba3_fwd.restype = i
        L.ssd_mamba3_fwd.argtypes = [vp] * 6 + [i] + [vp] * 5 + [i] * 8 + [vp]
        L.ssm_decode_step_mamba3.restype = i
        L.ssm_decode_step_mamba3.argtypes = [vp] * 12 + [i] * 6 + [vp]
        L.ssd_mamba3_mimo_fwd.restype = i
        L.ssd_mamba3_mimo_fwd.argtypes = [vp] * 6 + [i] * 2 + [vp] * 5 + [i] * 8 + [vp]
        L.ssm_decode_step_mamba3_mimo.restype = i
        L.ssm_decode_step_mamba3_mimo.argtypes = [vp] * 12 + [i] * 7 + [vp]
        L.ssm_scan_fwd_noalloc.restype = i
        L.ssm_scan_fwd_noalloc.argtypes = [vp] * 8 + [i] + [vp] * 3 + [i] * 7 + [vp]
        L.ssm_scan_bwd_workspace_bytes.restype = sz
        L.ssm_scan_bwd_workspace_bytes.argtypes = [i] * 5
        L.ssm_scan_bwd.restype = i
        L.ssm_scan_bwd.argtypes = [vp] * 8 + [i] + [vp] * 13 + [i] * 6 + [vp, sz, vp]
        L.ssm_scan_checkpoint_bytes.restype = sz
        L.ssm_scan_checkpoint_bytes.argtypes = [i] * 4
        L.ssm_scan_fwd_ckpt.restype = i
        L.ssm_scan_fwd_ckpt.argtypes = [vp] * 8 + [i] + [vp] * 4 + [i] * 7 + [vp, sz, vp]
        L.ssd_chunked_bwd_workspace_bytes.restype = sz
        L.ssd_chunked_bwd_workspace_bytes.argtypes = [i] * 6
        L.ssd_chunked_bwd.restype = i
        L.ssd_chunked_bwd.argtypes = [vp] * 5 + [i] + [vp] * 10 + [i] * 7 + [vp, sz, vp]
        L.ssd_mamba3_bwd_workspace_bytes.restype = sz
        L.ssd_mamba3_bwd_workspace_bytes.argtypes = [i] * 6
        L.ssd_mamba3_bwd.restype = i
        L.ssd_mamba3_bwd.argtypes = [vp] * 6 + [i] + [vp] * 15 + [i] * 7 + [vp, sz, vp]
        L.ssd_mamba3_fwd_ckpt.restype = i
        L.ssd_mamba3_fwd_ckpt.argtypes = [vp] * 6 + [i] + [vp] * 6 + [i] * 7 + [vp]
        L.ssd_mamba3_mimo_fwd_ckpt.restype = i
        L.ssd_mamba3_mimo_fwd_ckpt.argtypes = [vp] * 6 + [i, i] + [vp] * 6 + [i] * 7 + [vp]
        L.ssd_mamba3_mimo_bwd_workspace_bytes.restype = sz
        L.ssd_mamba3_mimo_bwd_workspace_bytes.argtypes = [i] * 7
        L.ssd_mamba3_mimo_bwd.restype = i
        L.ssd_mamba3_mimo_bwd.argtypes = [vp] * 6 + [i, i] + [vp] * 15 + [i] * 7 + [vp, sz, vp]
        L.ssd_chunked_checkpoint_bytes.restype = sz
        L.ssd_chunked_checkpoint_bytes.argtypes = [i] * 5
        L.ssd_chunked_fwd_ckpt.restype = i
        L.ssd_chunked_fwd_ckpt.argtypes = [vp] * 5 + [i] + [vp] * 4 + [i] * 8 + [vp]
        L.ssm_scan_fwd_host_workspace_bytes.restype = sz
        L.ssm_scan_fwd_host_workspace_bytes.argtypes = [i] * 7
        L.ssm_scan_fwd_host.restype = i
        L.ssm_scan_fwd_host.argtypes = [vp] * 8 + [i] + [vp] * 3 + [i] * 7 + [vp, sz, vp]
        L.ssm_last_device_status.restype = i
        L.ssm_last_device_status.argtypes = [vp, vp]
        L.ssm_debug_set_lookback.restype = i
        L.ssm_debug_set_lookback.argtypes = [i, ctypes.c_uint]
        L.ssm_debug_set_scan_path.restype = i
        L.ssm_debug_set_scan_path.argtypes = [i, i]
        L.ssm_noalloc_last_status.restype = i
        L.ssm_noalloc_last_status.argtypes = [vp]
        L.ssm_mamba3_rope.restype = i
        L.ssm_mamba3_rope.argtypes = [vp] * 8 + [i] * 7 + [vp]
        ll, fl = ctypes.c_longlong, ctypes.c_float
        L.ssm_add_rmsnorm_fwd.restype = i
        L.ssm_add_rmsnorm_fwd.argtypes = [vp] * 3 + [fl] + [vp] * 2 + [i] * 5 + [vp]
        L.ssm_add_rmsnorm_e4m3_fwd.restype = i
        L.ssm_add_rmsnorm_e4m3_fwd.argtypes = [vp] * 3 + [fl, i] + [vp] * 3 + [i] * 4 + [vp]
        L.ssm_add_rmsnorm_bwd_workspace_bytes.restype = sz
        L.ssm_add_rmsnorm_bwd_workspace_bytes.argtypes = [i] * 2
        L.ssm_add_rmsnorm_bwd.restype = i
        L.ssm_add_rmsnorm_bwd.argtypes = [vp] * 2 + [fl] + [vp] * 5 + [i] * 5 + [vp, sz, vp]
        for f in (L.ssm_linrec_checkpoint_bytes, L.ssm_linrec_workspace_bytes,
                  L.ssm_linrec_bwd_workspace_bytes, L.ssm_vocab_ce_workspace_bytes,
                  L.ssm_vocab_ce_bwd_workspace_bytes):
            f.restype = sz
            f.argtypes = [i] * 3
        L.ssm_linrec_fwd.restype = i
        L.ssm_linrec_fwd.argtypes = [vp] * 3 + [ll] * 3 + [vp] * 4 + [i] * 5 + [vp, sz, vp]
        L.ssm_linrec_bwd.restype = i
        L.ssm_linrec_bwd.argtypes = [vp] * 3 + [ll] * 3 + [vp] * 8 + [i] * 5 + [vp, sz, vp]
        L.ssm_vocab_ce_fwd.restype = i
        L.ssm_vocab_ce_fwd.argtypes = [vp] * 5 + [i] * 4 + [vp, sz, vp]
        L.ssm_vocab_ce_bwd.restype = i
        L.ssm_vocab_ce_bwd.argtypes = [vp] * 7 + [i] * 5 + [vp, sz, vp]
        L.ssm_qk_norm_rope_fwd.restype = i
        L.ssm_qk_norm_rope_fwd.argtypes = ([vp] * 2 + [ll] * 2 + [vp] * 4 + [fl, i, i] + [vp] * 2 +
                                           [ll] + [i] * 5 + [vp])
        L.ssm_qk_norm_rope_bwd_workspace_bytes.restype = sz
        L.ssm_qk_norm_rope_bwd_workspace_bytes.argtypes = [ll] + [i] * 3
        L.ssm_qk_norm_rope_bwd.restype = i
        L.ssm_qk_norm_rope_bwd.argtypes = ([vp] * 4 + [ll] * 2 + [vp] * 4 + [fl, i, i] + [vp] * 4 +
                                           [ll] + [i] * 5 + [vp, sz, vp])
        for f in (L.ssm_gated_delta_checkpoint_bytes, L.ssm_gated_delta_workspace_bytes,
                  L.ssm_gated_delta_bwd_workspace_bytes):
            f.restype = sz
            f.argtypes = [i] * 5
        L.ssm_gated_delta_walked_steps.restype = i
        L.ssm_gated_delta_walked_steps.argtypes = []
        L.ssm_gated_delta_fwd.restype = i
        L.ssm_gated_delta_fwd.argtypes = ([vp] * 3 + [ll] * 3 + [vp] * 6 + [i] * 9 +
                                          [vp, sz, vp])
        L.ssm_gated_delta_bwd.restype = i
        L.ssm_gated_delta_bwd.argtypes = ([vp] * 3 + [ll] * 3 + [vp] * 12 + [i] * 9 +
                                          [vp, sz, vp])
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().ssm_status_string(int(status)).decode()


def ssm_abi_version() -> int:
    return int(lib().ssm_abi_version())


def _check(status: int, where: str):
    if status != 0:
        raise SSMError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _req(t, name, dtype=None, ndim=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")
    return t


def _opt(t, name, dtype=None, ndim=None):
    return None if t is None else _req(t, name, dtype, ndim)


def _shape(t, name, shape):
    """Raises ValueError unless tensor ``t`` (when given) has exactly ``shape``."""
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _scan_shapes(u, delta, A, B, C, D, z, delta_bias, initial_state, y, final_state,
                 dy=None, dfinal_state=None):
    """Checks every scan tensor against u's (batch, dim, seqlen), A's dstate and
    B's ngroups, so that no kernel reads or writes past a buffer the caller passed."""
    batch, dim, seqlen = u.shape
    if A.dim() != 2 or A.shape[0] != dim:
        raise ValueError(f"A must have shape ({dim}, dstate), got {tuple(A.shape)}")
    dstate = A.shape[1]
    if B.dim() != 4 or B.shape[0] != batch or B.shape[2] != dstate or B.shape[3] != seqlen:
        raise ValueError(f"B must have shape ({batch}, ngroups, {dstate}, {seqlen}), "
                         f"got {tuple(B.shape)}")
    ngroups = B.shape[1]
    act = (batch, dim, seqlen)
    _shape(delta, "delta", act)
    _shape(z, "z", act)
    _shape(y, "y", act)
    _shape(dy, "dy", act)
    _shape(C, "C", (batch, ngroups, dstate, seqlen))
    _shape(D, "D", (dim,))
    _shape(delta_bias, "delta_bias", (dim,))
    for t, name in ((initial_state, "initial_state"), (final_state, "final_state"),
                    (dfinal_state, "dfinal_state")):
        _shape(t, name, (batch, dim, dstate))
    return batch, dim, seqlen, dstate, ngroups


def _use_out(g, out):
    """Puts the caller's preallocated fp32 tensors (``out``: name -> tensor) in
    place of the gradient buffers ``g`` would allocate."""
    for k, t in (out or {}).items():
        if k not in g or g[k] is None:
            raise ValueError(f"out[{k!r}] is not an output of this call")
        _req(t, f"out[{k!r}]", torch.float32)
        if t.shape != g[k].shape:
            raise ValueError(f"out[{k!r}] must have shape {tuple(g[k].shape)}")
        g[k] = t


def ssm_scan_workspace_bytes(batch, dim, seqlen, dstate=16, ngroups=1) -> int:
    return int(lib().ssm_scan_workspace_bytes(batch, dim, seqlen, dstate, ngroups))


def ssm_scan_checkpoint_bytes(batch, dim, seqlen, dstate=16) -> int:
    return int(lib().ssm_scan_checkpoint_bytes(batch, dim, seqlen, dstate))


def ssm_scan_fwd(u, delta, A, B, C, D=None, z=None, delta_bias=None, delta_softplus=False,
                 initial_state=None, out_dtype=None, y=None, final_state=None,
                 workspace=None, return_final_state=True, stream=None, checkpoints=None):
    """Selective scan.  u, delta, z: (batch, dim, seqlen); A: (dim, dstate) fp32;
    B, C: (batch, ngroups, dstate, seqlen); D, delta_bias: (dim,) fp32;
    initial_state: (batch, dim, dstate) fp32.  With ``checkpoints`` (a CUDA fp32
    tensor of ssm_scan_checkpoint_bytes bytes) the states ssm_scan_bwd needs are
    kept too (ssm_scan_fwd_ckpt).  Returns (y, final_state)."""
    _req(u, "u", ndim=3)
    in_dt = u.dtype
    if in_dt not in _DT:
        raise TypeError("u must be float32 or bfloat16")
    batch, dim, seqlen = u.shape
    _req(delta, "delta", in_dt)
    _req(A, "A", torch.float32, 2)
    dstate = A.shape[1]
    _req(B, "B", in_dt, 4)
    _req(C, "C", in_dt, 4)
    ngroups = B.shape[1]
    _opt(D, "D", torch.float32)
    _opt(z, "z", in_dt)
    _opt(delta_bias, "delta_bias", torch.float32)
    _opt(initial_state, "initial_state", torch.float32)
    out_dt = in_dt if out_dtype is None else out_dtype
    if y is None:
        y = torch.empty((batch, dim, seqlen), dtype=out_dt, device=u.device)
    _req(y, "y", out_dt)
    if final_state is None and return_final_state:
        final_state = torch.empty((batch, dim, dstate), dtype=torch.float32, device=u.device)
    _opt(final_state, "final_state", torch.float32)
    _scan_shapes(u, delta, A, B, C, D, z, delta_bias, initial_state, y, final_state)
    need = ssm_scan_workspace_bytes(batch, dim, seqlen, dstate, ngroups)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=u.device)
    _req(workspace, "workspace", torch.uint8)
    if checkpoints is not None:
        _req(checkpoints, "checkpoints", torch.float32)
        if checkpoints.numel() * 4 < ssm_scan_checkpoint_bytes(batch, dim, seqlen, dstate):
            raise ValueError("checkpoints is smaller than ssm_scan_checkpoint_bytes(...)")
        st = lib().ssm_scan_fwd_ckpt(_ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                     _ptr(z), _ptr(delta_bias), int(bool(delta_softplus)),
                                     _ptr(initial_state), _ptr(y), _ptr(final_state),
                                     _ptr(checkpoints), batch, dim, seqlen, dstate, ngroups,
                                     _DT[in_dt], _DT[out_dt], _ptr(workspace), workspace.numel(),
                                     _stream(stream))
        _check(st, "ssm_scan_fwd_ckpt")
        return y, final_state
    st = lib().ssm_scan_fwd(_ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                            _ptr(delta_bias), int(bool(delta_softplus)), _ptr(initial_state),
                            _ptr(y), _ptr(final_state), batch, dim, seqlen, dstate, ngroups,
                            _DT[in_dt], _DT[out_dt], _ptr(workspace), workspace.numel(),
                            _stream(stream))
    _check(st, "ssm_scan_fwd")
    return y, final_state


def ssm_scan_bwd_workspace_bytes(batch, dim, seqlen, dstate=16, ngroups=1) -> int:
    return int(lib().ssm_scan_bwd_workspace_bytes(batch, dim, seqlen, dstate, ngroups))


def ssm_scan_bwd(u, delta, A, B, C, dy, D=None, z=None, delta_bias=None, delta_softplus=False,
                 initial_state=None, dfinal_state=None, workspace=None, want_dD=None,
                 want_ddelta_bias=None, want_dinitial_state=True, out=None, stream=None,
                 checkpoints=None):
    """Gradient of ``ssm_scan_fwd`` for the loss sum(dy * y) + sum(dfinal_state *
    final_state).  Inputs as for ``ssm_scan_fwd``; dy (batch, dim, seqlen) in u's
    dtype; dfinal_state (batch, dim, dstate) fp32 or None.  Returns a dict of fp32
    tensors: du, ddelta, dz (batch, dim, seqlen); dA (dim, dstate); dB, dC
    (batch, ngroups, dstate, seqlen); dD, ddelta_bias (dim,); dinitial_state
    (batch, dim, dstate).  dz is None without z; dD / ddelta_bias are computed
    when D / delta_bias is given, or when want_dD / want_ddelta_bias is true.
    ``out`` may map any of these names to a preallocated fp32 tensor to write.
    ``checkpoints``: what ``ssm_scan_fwd(..., checkpoints=...)`` kept for the same
    inputs (the forward recurrence is then not run again)."""
    _req(u, "u", ndim=3)
    in_dt = u.dtype
    if in_dt not in _DT:
        raise TypeError("u must be float32 or bfloat16")
    batch, dim, seqlen = u.shape
    _req(delta, "delta", in_dt)
    _req(A, "A", torch.float32, 2)
    dstate = A.shape[1]
    _req(B, "B", in_dt, 4)
    _req(C, "C", in_dt, 4)
    ngroups = B.shape[1]
    _req(dy, "dy", in_dt, 3)
    _opt(D, "D", torch.float32)
    _opt(z, "z", in_dt)
    _opt(delta_bias, "delta_bias", torch.float32)
    _opt(initial_state, "initial_state", torch.float32)
    _opt(dfinal_state, "dfinal_state", torch.float32)
    _scan_shapes(u, delta, A, B, C, D, z, delta_bias, initial_state, None, None, dy=dy,
                 dfinal_state=dfinal_state)
    dev, f32 = u.device, torch.float32
    g = {"du": torch.empty((batch, dim, seqlen), dtype=f32, device=dev),
         "ddelta": torch.empty((batch, dim, seqlen), dtype=f32, device=dev),
         "dA": torch.empty((dim, dstate), dtype=f32, device=dev),
         "dB": torch.empty(tuple(B.shape), dtype=f32, device=dev),
         "dC": torch.empty(tuple(C.shape), dtype=f32, device=dev),
         "dD": None, "dz": None, "ddelta_bias": None, "dinitial_state": None}
    if D is not None or want_dD:
        g["dD"] = torch.empty(dim, dtype=f32, device=dev)
    if delta_bias is not None or want_ddelta_bias:
        g["ddelta_bias"] = torch.empty(dim, dtype=f32, device=dev)
    if z is not None:
        g["dz"] = torch.empty((batch, dim, seqlen), dtype=f32, device=dev)
    if want_dinitial_state:
        g["dinitial_state"] = torch.empty((batch, dim, dstate), dtype=f32, device=dev)
    _use_out(g, out)
    need = ssm_scan_bwd_workspace_bytes(batch, dim, seqlen, dstate, ngroups)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    _req(workspace, "workspace", torch.uint8)
    st = lib().ssm_scan_bwd(_ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                            _ptr(delta_bias), int(bool(delta_softplus)), _ptr(initial_state),
                            _ptr(dy), _ptr(dfinal_state), _ptr(_opt(checkpoints, "checkpoints",
                                                                   torch.float32)),
                            _ptr(g["du"]), _ptr(g["ddelta"]),
                            _ptr(g["dA"]), _ptr(g["dB"]), _ptr(g["dC"]), _ptr(g["dD"]),
                            _ptr(g["dz"]), _ptr(g["ddelta_bias"]), _ptr(g["dinitial_state"]),
                            batch, dim, seqlen, dstate, ngroups, _DT[in_dt], _ptr(workspace),
                            workspace.numel(), _stream(stream))
    _check(st, "ssm_scan_bwd")
    return g


def ssm_scan_fwd_host_workspace_bytes(batch, dim, seqlen, dstate=16, ngroups=1,
                                      in_dtype=torch.bfloat16, out_dtype=torch.float32) -> int:
    return int(lib().ssm_scan_fwd_host_workspace_bytes(batch, dim, seqlen, dstate, ngroups,
                                                       _DT[in_dtype], _DT[out_dtype]))


def _pinned(t, name, dtype=None, ndim=None):
    # an empty tensor is never read or written, and may not be page-locked
    if (not isinstance(t, torch.Tensor) or t.is_cuda
            or (t.numel() > 0 and not t.is_pinned())):
        raise TypeError(f"{name} must be a pinned (page-locked) CPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")
    return t


def ssm_scan_fwd_host(u, delta, A, B, C, y, final_state=None, D=None, z=None, delta_bias=None,
                      delta_softplus=False, initial_state=None, workspace=None, stream=None):
    """``ssm_scan_fwd`` on pinned host tensors: u, delta, z, B, C, initial_state, y and
    final_state are pinned CPU tensors (same layouts); A, D, delta_bias and the workspace
    are CUDA tensors.  The copies in and out are pipelined with the scan on the library's
    copy streams; the call returns once everything is enqueued on ``stream``."""
    _pinned(u, "u", ndim=3)
    in_dt = u.dtype
    if in_dt not in _DT:
        raise TypeError("u must be float32 or bfloat16")
    batch, dim, seqlen = u.shape
    _pinned(delta, "delta", in_dt)
    _req(A, "A", torch.float32, 2)
    dstate = A.shape[1]
    _pinned(B, "B", in_dt, 4)
    _pinned(C, "C", in_dt, 4)
    ngroups = B.shape[1]
    _opt(D, "D", torch.float32)
    _opt(delta_bias, "delta_bias", torch.float32)
    if z is not None:
        _pinned(z, "z", in_dt)
    if initial_state is not None:
        _pinned(initial_state, "initial_state", torch.float32)
    _pinned(y, "y")
    if y.dtype not in _DT:
        raise TypeError("y must be float32 or bfloat16")
    if final_state is not None:
        _pinned(final_state, "final_state", torch.float32)
    _scan_shapes(u, delta, A, B, C, D, z, delta_bias, initial_state, y, final_state)
    need = ssm_scan_fwd_host_workspace_bytes(batch, dim, seqlen, dstate, ngroups, in_dt, y.dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=A.device)
    _req(workspace, "workspace", torch.uint8)
    st = lib().ssm_scan_fwd_host(_ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                 _ptr(z), _ptr(delta_bias), int(bool(delta_softplus)),
                                 _ptr(initial_state), _ptr(y), _ptr(final_state), batch, dim,
                                 seqlen, dstate, ngroups, _DT[in_dt], _DT[y.dtype],
                                 _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "ssm_scan_fwd_host")
    return y, final_state


def ssm_scan_fwd_noalloc(u, delta, A, B, C, y, final_state=None, D=None, z=None,
                         delta_bias=None, delta_softplus=False, initial_state=None, stream=None):
    """The selective scan without a workspace, for callers that cannot
    allocate: its scratch is a fixed array inside the library.  The caller
    passes every input and output (y, and final_state or None); nothing is
    allocated here or in the library.  Same layouts as ssm_scan_fwd."""
    _req(u, "u", ndim=3)
    in_dt = u.dtype
    if in_dt not in _DT:
        raise TypeError("u must be float32 or bfloat16")
    batch, dim, seqlen = u.shape
    _req(delta, "delta", in_dt)
    _req(A, "A", torch.float32, 2)
    _req(B, "B", in_dt, 4)
    _req(C, "C", in_dt, 4)
    _opt(D, "D", torch.float32)
    _opt(z, "z", in_dt)
    _opt(delta_bias, "delta_bias", torch.float32)
    _opt(initial_state, "initial_state", torch.float32)
    _req(y, "y")
    if y.dtype not in _DT:
        raise TypeError("y must be float32 or bfloat16")
    _opt(final_state, "final_state", torch.float32)
    _scan_shapes(u, delta, A, B, C, D, z, delta_bias, initial_state, y, final_state)
    st = lib().ssm_scan_fwd_noalloc(_ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                    _ptr(z), _ptr(delta_bias), int(bool(delta_softplus)),
                                    _ptr(initial_state), _ptr(y), _ptr(final_state), batch, dim,
                                    seqlen, A.shape[1], B.shape[1], _DT[in_dt], _DT[y.dtype],
                                    _stream(stream))
    _check(st, "ssm_scan_fwd_noalloc")
    return y, final_state


def ssd_chunked_bwd_workspace_bytes(batch, seqlen, nheads, headdim=64, dstate=128,
                                    ngroups=1) -> int:
    return int(lib().ssd_chunked_bwd_workspace_bytes(batch, seqlen, nheads, headdim, dstate,
                                                     ngroups))


def ssd_chunked_checkpoint_bytes(batch, seqlen, nheads, headdim=64, dstate=128) -> int:
    return int(lib().ssd_chunked_checkpoint_bytes(batch, seqlen, nheads, headdim, dstate))


def ssd_chunked_bwd(x, dt, A_head, B, C, dy, chunk=64, initial_state=None, dfinal_state=None,
                    workspace=None, want_dinitial_state=True, out=None, stream=None,
                    block_states=None):
    """Gradient of ``ssd_chunked_fwd`` for the loss sum(dy * y) + sum(dfinal_state *
    final_state).  Inputs as for ``ssd_chunked_fwd``; dy like x (bf16); dfinal_state
    (batch, nheads, headdim, dstate) fp32 or None.  Returns a dict of fp32 tensors:
    dx (like x), ddt (like dt), dA_head (nheads,), dB, dC (like B) and dinitial_state
    (batch, nheads, headdim, dstate, or None).  ``out`` may map any of these names to
    a preallocated fp32 tensor to write.  ``block_states``: what
    ``ssd_chunked_fwd(..., block_states=...)`` kept for the same inputs."""
    _req(x, "x", torch.bfloat16, 4)
    batch, seqlen, nheads, headdim = x.shape
    _req(dt, "dt", torch.float32, 3)
    _req(A_head, "A_head", torch.float32, 1)
    _req(B, "B", torch.bfloat16, 4)
    _req(C, "C", torch.bfloat16, 4)
    _req(dy, "dy", torch.bfloat16, 4)
    ngroups, dstate = B.shape[2], B.shape[3]
    _opt(initial_state, "initial_state", torch.float32)
    _opt(dfinal_state, "dfinal_state", torch.float32)
    dev, f32 = x.device, torch.float32
    g = {"dx": torch.empty(tuple(x.shape), dtype=f32, device=dev),
         "ddt": torch.empty(tuple(dt.shape), dtype=f32, device=dev),
         "dA_head": torch.empty(nheads, dtype=f32, device=dev),
         "dB": torch.empty(tuple(B.shape), dtype=f32, device=dev),
         "dC": torch.empty(tuple(C.shape), dtype=f32, device=dev),
         "dinitial_state": (torch.empty((batch, nheads, headdim, dstate), dtype=f32, device=dev)
                            if want_dinitial_state else None)}
    _use_out(g, out)
    need = ssd_chunked_bwd_workspace_bytes(batch, seqlen, nheads, headdim, dstate, ngroups)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    _req(workspace, "workspace", torch.uint8)
    st = lib().ssd_chunked_bwd(_ptr(x), _ptr(dt), _ptr(A_head), _ptr(B), _ptr(C), int(chunk),
                               _ptr(initial_state), _ptr(dy), _ptr(dfinal_state),
                               _ptr(_opt(block_states, "block_states", torch.float32)),
                               _ptr(g["dx"]),
                               _ptr(g["ddt"]), _ptr(g["dA_head"]), _ptr(g["dB"]), _ptr(g["dC"]),
                               _ptr(g["dinitial_state"]), batch, seqlen, nheads, headdim, dstate,
                               ngroups, _DT[torch.bfloat16], _ptr(workspace), workspace.numel(),
                               _stream(stream))
    _check(st, "ssd_chunked_bwd")
    return g


def ssd_mamba3_bwd_workspace_bytes(batch, seqlen, nheads, headdim=64, dstate=128,
                                   ngroups=1) -> int:
    return int(lib().ssd_mamba3_bwd_workspace_bytes(batch, seqlen, nheads, headdim, dstate,
                                                    ngroups))


def ssd_mamba3_bwd(x, dt, lam, A_head, B, C, dy, chunk=64, initial_state=None, prev_B=None,
                   prev_x=None, dfinal_state=None, workspace=None, want_dinitial_state=True,
                   stream=None, block_states=None, out=None):
    """Gradient of ``ssd_mamba3_fwd`` for the loss sum(dy * y) + sum(dfinal_state *
    final_state).  Inputs as for ``ssd_mamba3_fwd`` (bf16 x, B, C, prev_B, prev_x);
    dy like x (bf16).  Returns a dict of fp32 tensors: dx, ddt, dlam, dA_head, dB, dC,
    dinitial_state (or None) and dprev_B, dprev_x (None without a previous token).
    ``out`` may map any of these names to a preallocated fp32 tensor to write."""
    _req(x, "x", torch.bfloat16, 4)
    batch, seqlen, nheads, headdim = x.shape
    _req(dt, "dt", torch.float32, 3)
    _req(lam, "lam", torch.float32, 3)
    _req(A_head, "A_head", torch.float32, 1)
    _req(B, "B", torch.bfloat16, 4)
    _req(C, "C", torch.bfloat16, 4)
    _req(dy, "dy", torch.bfloat16, 4)
    ngroups, dstate = B.shape[2], B.shape[3]
    _opt(initial_state, "initial_state", torch.float32)
    _opt(dfinal_state, "dfinal_state", torch.float32)
    _opt(prev_B, "prev_B", torch.bfloat16)
    _opt(prev_x, "prev_x", torch.bfloat16)
    has_prev = prev_B is not None
    dev, f32 = x.device, torch.float32
    g = {"dx": torch.empty(tuple(x.shape), dtype=f32, device=dev),
         "ddt": torch.empty(tuple(dt.shape), dtype=f32, device=dev),
         "dlam": torch.empty(tuple(dt.shape), dtype=f32, device=dev),
         "dA_head": torch.empty(nheads, dtype=f32, device=dev),
         "dB": torch.empty(tuple(B.shape), dtype=f32, device=dev),
         "dC": torch.empty(tuple(C.shape), dtype=f32, device=dev),
         "dinitial_state": (torch.empty((batch, nheads, headdim, dstate), dtype=f32, device=dev)
                            if want_dinitial_state else None),
         "dprev_B": (torch.empty((batch, ngroups, dstate), dtype=f32, device=dev)
                     if has_prev else None),
         "dprev_x": (torch.empty((batch, nheads, headdim), dtype=f32, device=dev)
                     if has_prev else None)}
    _use_out(g, out)
    need = ssd_mamba3_bwd_workspace_bytes(batch, seqlen, nheads, headdim, dstate, ngroups)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    _req(workspace, "workspace", torch.uint8)
    st = lib().ssd_mamba3_bwd(_ptr(x), _ptr(dt), _ptr(lam), _ptr(A_head), _ptr(B), _ptr(C),
                              int(chunk), _ptr(initial_state), _ptr(prev_B), _ptr(prev_x),
                              _ptr(dy), _ptr(dfinal_state),
                              _ptr(_opt(block_states, "block_states", torch.float32)),
                              _ptr(g["dx"]), _ptr(g["ddt"]),
                              _ptr(g["dlam"]), _ptr(g["dA_head"]), _ptr(g["dB"]), _ptr(g["dC"]),
                              _ptr(g["dinitial_state"]), _ptr(g["dprev_B"]), _ptr(g["dprev_x"]),
                              batch, seqlen, nheads, headdim, dstate, ngroups,
                              _DT[torch.bfloat16], _ptr(workspace), workspace.numel(),
                              _stream(stream))
    _check(st, "ssd_mamba3_bwd")
    return g


def ssd_mamba3_mimo_bwd_workspace_bytes(batch, seqlen, rank, nheads, headdim=64, dstate=128,
                                        ngroups=1) -> int:
    return int(lib().ssd_mamba3_mimo_bwd_workspace_bytes(batch, seqlen, rank, nheads, headdim,
                                                         dstate, ngroups))


def ssd_mamba3_mimo_bwd(x, dt, lam, A_head, B, C, dy, chunk=None, initial_state=None,
                        prev_B=None, prev_x=None, dfinal_state=None, workspace=None,
                        want_dinitial_state=True, stream=None, block_states=None, out=None):
    """Gradient of ``ssd_mamba3_mimo_fwd``.  x, dy: (batch, seqlen, rank, nheads,
    headdim) bf16; B, C: (batch, seqlen, rank, ngroups, dstate) bf16; prev_B (batch,
    rank, ngroups, dstate), prev_x (batch, rank, nheads, headdim) bf16 or None.
    ``chunk`` defaults to 64 // rank.  Returns a dict of fp32 tensors like
    ``ssd_mamba3_bwd``'s, with dx, dB, dC, dprev_B, dprev_x shaped like their inputs;
    ``out`` as for ``ssd_mamba3_bwd``."""
    _req(x, "x", torch.bfloat16, 5)
    batch, seqlen, rank, nheads, headdim = x.shape
    _req(dt, "dt", torch.float32, 3)
    _req(lam, "lam", torch.float32, 3)
    _req(A_head, "A_head", torch.float32, 1)
    _req(B, "B", torch.bfloat16, 5)
    _req(C, "C", torch.bfloat16, 5)
    _req(dy, "dy", torch.bfloat16, 5)
    ngroups, dstate = B.shape[3], B.shape[4]
    _opt(initial_state, "initial_state", torch.float32)
    _opt(dfinal_state, "dfinal_state", torch.float32)
    _opt(prev_B, "prev_B", torch.bfloat16)
    _opt(prev_x, "prev_x", torch.bfloat16)
    has_prev = prev_B is not None
    chunk = 64 // rank if chunk is None else chunk
    dev, f32 = x.device, torch.float32
    g = {"dx": torch.empty(tuple(x.shape), dtype=f32, device=dev),
         "ddt": torch.empty(tuple(dt.shape), dtype=f32, device=dev),
         "dlam": torch.empty(tuple(dt.shape), dtype=f32, device=dev),
         "dA_head": torch.empty(nheads, dtype=f32, device=dev),
         "dB": torch.empty(tuple(B.shape), dtype=f32, device=dev),
         "dC": torch.empty(tuple(C.shape), dtype=f32, device=dev),
         "dinitial_state": (torch.empty((batch, nheads, headdim, dstate), dtype=f32, device=dev)
                            if want_dinitial_state else None),
         "dprev_B": (torch.empty(tuple(prev_B.shape), dtype=f32, device=dev)
                     if has_prev else None),
         "dprev_x": (torch.empty(tuple(prev_x.shape), dtype=f32, device=dev)
                     if has_prev else None)}
    _use_out(g, out)
    need = ssd_mamba3_mimo_bwd_workspace_bytes(batch, seqlen, rank, nheads, headdim, dstate,
                                               ngroups)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    _req(workspace, "workspace", torch.uint8)
    st = lib().ssd_mamba3_mimo_bwd(_ptr(x), _ptr(dt), _ptr(lam), _ptr(A_head), _ptr(B), _ptr(C),
                                   int(chunk), int(rank), _ptr(initial_state), _ptr(prev_B),
                                   _ptr(prev_x), _ptr(dy), _ptr(dfinal_state),
                                   _ptr(_opt(block_states, "block_states", torch.float32)),
                                   _ptr(g["dx"]),
                                   _ptr(g["ddt"]), _ptr(g["dlam"]), _ptr(g["dA_head"]),
                                   _ptr(g["dB"]), _ptr(g["dC"]), _ptr(g["dinitial_state"]),
                                   _ptr(g["dprev_B"]), _ptr(g["dprev_x"]), batch, seqlen, nheads,
                                   headdim, dstate, ngroups, _DT[torch.bfloat16], _ptr(workspace),
                                   workspace.numel(), _stream(stream))
    _check(st, "ssd_mamba3_mimo_bwd")
    return g


def ssd_chunked_fwd(x, dt, A_head, B, C, chunk=64, out_dtype=None, y=None, final_state=None,
                    return_final_state=True, stream=None, initial_state=None, block_states=None):
    """Chunked SSD.  x: (batch, seqlen, nheads, headdim); dt: (batch, seqlen, nheads) fp32;
    A_head: (nheads,) fp32; B, C: (batch, seqlen, ngroups, dstate); initial_state (optional,
    may be ``final_state`` itself): (batch, nheads, headdim, dstate) fp32.
    Returns (y, final_state)."""
    _req(x, "x", ndim=4)
    in_dt = x.dtype
    if in_dt not in _DT:
        raise TypeError("x must be float32 or bfloat16")
    batch, seqlen, nheads, headdim = x.shape
    _req(dt, "dt", torch.float32, 3)
    _req(A_head, "A_head", torch.float32, 1)
    _req(B, "B", in_dt, 4)
    _req(C, "C", in_dt, 4)
    ngroups, dstate = B.shape[2], B.shape[3]
    out_dt = in_dt if out_dtype is None else out_dtype
    if y is None:
        y = torch.empty_like(x, dtype=out_dt)
    _req(y, "y", out_dt)
    if final_state is None and return_final_state:
        final_state = torch.empty((batch, nheads, headdim, dstate), dtype=torch.float32,
                                  device=x.device)
    _opt(final_state, "final_state", torch.float32)
    _opt(initial_state, "initial_state", torch.float32)
    _shape(dt, "dt", (batch, seqlen, nheads))
    _shape(A_head, "A_head", (nheads,))
    if B.shape[0] != batch or B.shape[1] != seqlen:
        raise ValueError(f"B must have shape ({batch}, {seqlen}, ngroups, dstate), "
                         f"got {tuple(B.shape)}")
    _shape(C, "C", tuple(B.shape))
    _shape(y, "y", tuple(x.shape))
    _shape(initial_state, "initial_state", (batch, nheads, headdim, dstate))
    _shape(final_state, "final_state", (batch, nheads, headdim, dstate))
    if block_states is not None:
        _req(block_states, "block_states", torch.float32)
        if block_states.numel() * 4 < ssd_chunked_checkpoint_bytes(batch, seqlen, nheads, headdim,
                                                                   dstate):
            raise ValueError("block_states is smaller than ssd_chunked_checkpoint_bytes(...)")
        st = lib().ssd_chunked_fwd_ckpt(_ptr(x), _ptr(dt), _ptr(A_head), _ptr(B), _ptr(C),
                                        int(chunk), _ptr(initial_state), _ptr(y),
                                        _ptr(final_state), _ptr(block_states), batch, seqlen,
                                        nheads, headdim, dstate, ngroups, _DT[in_dt], _DT[out_dt],
                                        _stream(stream))
        _check(st, "ssd_chunked_fwd_ckpt")
        return y, final_state
    st = lib().ssd_chunked_fwd(_ptr(x), _ptr(dt), _ptr(A_head), _ptr(B), _ptr(C), int(chunk),
                               _ptr(initial_state), _ptr(y), _ptr(final_state), batch, seqlen,
                               nheads, headdim, dstate,
                               ngroups, _DT[in_dt], _DT[out_dt], _stream(stream))
    _check(st, "ssd_chunked_fwd")
    return y, final_state


def ssm_decode_step(state, x, dt, A, B, C, D=None, z=None, y=None, stream=None):
    """One decode step; ``state`` (batch, nheads, headdim, dstate) fp32 is updated in place.
    x, z: (batch, nheads, headdim); dt: (batch, nheads) fp32; A, D: (nheads,) fp32;
    B, C: (batch, ngroups, dstate).  Returns y (batch, nheads, headdim)."""
    _req(state, "state", torch.float32, 4)
    batch, nheads, headdim, dstate = state.shape
    _req(x, "x", ndim=3)
    dt_ = x.dtype
    if dt_ not in _DT:
        raise TypeError("x must be float32 or bfloat16")
    _req(dt, "dt", torch.float32, 2)
    _req(A, "A", torch.float32, 1)
    _req(B, "B", dt_, 3)
    _req(C, "C", dt_, 3)
    ngroups = B.shape[1]
    _opt(D, "D", torch.float32)
    _opt(z, "z", dt_)
    if y is None:
        y = torch.empty_like(x)
    _req(y, "y", dt_)
    _shape(x, "x", (batch, nheads, headdim))
    _shape(z, "z", (batch, nheads, headdim))
    _shape(y, "y", (batch, nheads, headdim))
    _shape(dt, "dt", (batch, nheads))
    _shape(A, "A", (nheads,))
    _shape(D, "D", (nheads,))
    if B.shape[0] != batch or B.shape[2] != dstate:
        raise ValueError(f"B must have shape ({batch}, ngroups, {dstate}), got {tuple(B.shape)}")
    _shape(C, "C", tuple(B.shape))
    st = lib().ssm_decode_step(_ptr(state), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C),
                               _ptr(D), _ptr(z), _ptr(y), batch, nheads, headdim, dstate,
                               ngroups, _DT[dt_], _stream(stream))
    _check(st, "ssm_decode_step")
    return y


def ssm_last_device_status(workspace, stream=None) -> int:
    """Device-side status recorded in a scan workspace (waits for the stream)."""
    return int(lib().ssm_last_device_status(_ptr(workspace), _stream(stream)))


def ssm_debug_set_lookback(drop_first_publish: bool = False, spin_limit: int = 0) -> None:
    """Test hook of the scan's chained L-chunks: chunk 0 withholds its publish
    (so chunk 1's bounded wait runs out and records SSM_ERR_TIMEOUT) and the
    wait gives up after ``spin_limit`` polls (0: the default).  In the gated delta rule, where
    records and chains run at once, the first record is not told of.  Process-wide;
    call with no arguments to restore the defaults."""
    _check(lib().ssm_debug_set_lookback(1 if drop_first_publish else 0, int(spin_limit)),
           "ssm_debug_set_lookback")


def ssm_debug_set_scan_path(path: int = 0, segments: int = 0) -> None:
    """Test hook choosing the forward scan's kernel: path 0 as planned, 1 the
    chained scan, 2 the sequence-parallel scan (where batch * dim <= 3072);
    segments: the sequence-parallel scan's segments per 128-step chunk (8, 16,
    32; 0 = planned).  Process-wide; call with no arguments to restore."""
    _check(lib().ssm_debug_set_scan_path(int(path), int(segments)), "ssm_debug_set_scan_path")


def ssm_noalloc_last_status(stream=None) -> int:
    """Device-side status the last ``ssm_scan_fwd_noalloc`` on the current device
    recorded in its scratch array (waits for the stream)."""
    return int(lib().ssm_noalloc_last_status(_stream(stream)))


def ssm_mamba3_rope(B, C, dt, theta, angle0=None, B_rot=None, C_rot=None, angle_out=None,
                    return_angle=True, stream=None):
    """Mamba-3's data-dependent RoPE: angles -cumsum(dt * theta) (from angle0),
    B and C rotated by them pair by pair, one row per head.  B, C: (batch, L, G, N)
    or with a rank axis (batch, L, R, G, N); dt (batch, L, H) fp32; theta
    (batch, L, H, N/2) fp32; angle0 (batch, H, N/2) fp32 or None.  Returns
    (B_rot, C_rot, angle_out) with B_rot, C_rot (batch, L, [R,] H, N) in B's dtype;
    angle_out may be angle0 itself (updated in place)."""
    _req(B, "B")
    dt_ = B.dtype
    if dt_ not in _DT:
        raise TypeError("B must be float32 or bfloat16")
    siso = B.dim() == 4
    if B.dim() not in (4, 5):
        raise ValueError("B must have 4 dims (batch, L, G, N) or 5 (batch, L, R, G, N)")
    if siso:
        batch, seqlen, ngroups, dstate = B.shape
        rank = 1
    else:
        batch, seqlen, rank, ngroups, dstate = B.shape
    _req(C, "C", dt_)
    _shape(C, "C", tuple(B.shape))
    _req(dt, "dt", torch.float32, 3)
    nheads = dt.shape[2]
    _shape(dt, "dt", (batch, seqlen, nheads))
    _req(theta, "theta", torch.float32, 4)
    _shape(theta, "theta", (batch, seqlen, nheads, dstate // 2))
    _opt(angle0, "angle0", torch.float32)
    _shape(angle0, "angle0", (batch, nheads, dstate // 2))
    rot = (batch, seqlen, nheads, dstate) if siso else (batch, seqlen, rank, nheads, dstate)
    if B_rot is None:
        B_rot = torch.empty(rot, dtype=dt_, device=B.device)
    if C_rot is None:
        C_rot = torch.empty(rot, dtype=dt_, device=B.device)
    _req(B_rot, "B_rot", dt_)
    _req(C_rot, "C_rot", dt_)
    _shape(B_rot, "B_rot", rot)
    _shape(C_rot, "C_rot", rot)
    if angle_out is None and return_angle:
        angle_out = torch.empty((batch, nheads, dstate // 2), dtype=torch.float32,
                                device=B.device)
    _opt(angle_out, "angle_out", torch.float32)
    _shape(angle_out, "angle_out", (batch, nheads, dstate // 2))
    st = lib().ssm_mamba3_rope(_ptr(B), _ptr(C), _ptr(dt), _ptr(theta), _ptr(angle0),
                               _ptr(B_rot), _ptr(C_rot), _ptr(angle_out), batch, seqlen, rank,
                               nheads, ngroups, dstate, _DT[dt_], _stream(stream))
    _check(st, "ssm_mamba3_rope")
    return B_rot, C_rot, angle_out


def ssd_mamba3_fwd(x, dt, lam, A_head, B, C, chunk=64, out_dtype=None, y=None, final_state=None,
                   return_final_state=True, initial_state=None, prev_B=None, prev_x=None,
                   stream=None, block_states=None):
    """Mamba-3 SISO chunked prefill.  As ``ssd_chunked_fwd`` plus lam: (batch, seqlen,
    nheads) fp32 (lambda after sigmoid) and the token before the first, prev_B:
    (batch, ngroups, dstate) and prev_x: (batch, nheads, headdim) in x's dtype (both or
    neither).  B and C are taken already rotated.  ``block_states`` (fp32, at least
    ``ssd_chunked_checkpoint_bytes(batch, seqlen, nheads)`` bytes) also keeps the
    states ``ssd_mamba3_bwd`` starts from.  Returns (y, final_state)."""
    _req(x, "x", ndim=4)
    in_dt = x.dtype
    if in_dt not in _DT:
        raise TypeError("x must be float32 or bfloat16")
    batch, seqlen, nheads, headdim = x.shape
    _req(dt, "dt", torch.float32, 3)
    _req(lam, "lam", torch.float32, 3)
    _req(A_head, "A_head", torch.float32, 1)
    _req(B, "B", in_dt, 4)
    _req(C, "C", in_dt, 4)
    ngroups, dstate = B.shape[2], B.shape[3]
    out_dt = in_dt if out_dtype is None else out_dtype
    if y is None:
        y = torch.empty_like(x, dtype=out_dt)
    _req(y, "y", out_dt)
    if final_state is None and return_final_state:
        final_state = torch.empty((batch, nheads, headdim, dstate), dtype=torch.float32,
                                  device=x.device)
    _opt(final_state, "final_state", torch.float32)
    _opt(initial_state, "initial_state", torch.float32)
    _opt(prev_B, "prev_B", in_dt)
    _opt(prev_x, "prev_x", in_dt)
    if block_states is not None:
        _req(block_states, "block_states", torch.float32)
        if block_states.numel() * 4 < ssd_chunked_checkpoint_bytes(batch, seqlen, nheads, headdim,
                                                                   dstate):
            raise ValueError("block_states is smaller than ssd_chunked_checkpoint_bytes(...)")
        st = lib().ssd_mamba3_fwd_ckpt(_ptr(x), _ptr(dt), _ptr(lam), _ptr(A_head), _ptr(B),
                                       _ptr(C), int(chunk), _ptr(initial_state), _ptr(prev_B),
                                       _ptr(prev_x), _ptr(y), _ptr(final_state),
                                       _ptr(block_states), batch, seqlen, nheads, headdim,
                                       dstate, ngroups, _DT[in_dt], _DT[out_dt], _stream(stream))
        _check(st, "ssd_mamba3_fwd_ckpt")
        return y, final_state
    st = lib().ssd_mamba3_fwd(_ptr(x), _ptr(dt), _ptr(lam), _ptr(A_head), _ptr(B), _ptr(C),
                              int(chunk), _ptr(initial_state), _ptr(prev_B), _ptr(prev_x),
                              _ptr(y), _ptr(final_state), batch, seqlen, nheads, headdim, dstate,
                              ngroups, _DT[in_dt], _DT[out_dt], _stream(stream))
    _check(st, "ssd_mamba3_fwd")
    return y, final_state


def ssm_decode_step_mamba3(state, prev_B, prev_x, x, dt, lam, A, B, C, D=None, z=None, y=None,
                           stream=None):
    """One Mamba-3 SISO decode step; ``state`` (batch, nheads, headdim, dstate) fp32 is
    updated in place.  As ``ssm_decode_step`` plus lam: (batch, nheads) fp32 and the
    previous token's prev_B (batch, ngroups, dstate) and prev_x (batch, nheads, headdim).
    Returns y (batch, nheads, headdim)."""
    _req(state, "state", torch.float32, 4)
    batch, nheads, headdim, dstate = state.shape
    _req(x, "x", ndim=3)
    dt_ = x.dtype
    if dt_ not in _DT:
        raise TypeError("x must be float32 or bfloat16")
    _req(dt, "dt", torch.float32, 2)
    _req(lam, "lam", torch.float32, 2)
    _req(A, "A", torch.float32, 1)
    _req(B, "B", dt_, 3)
    _req(C, "C", dt_, 3)
    _req(prev_B, "prev_B", dt_, 3)
    _req(prev_x, "prev_x", dt_, 3)
    ngroups = B.shape[1]
    _opt(D, "D", torch.float32)
    _opt(z, "z", dt_)
    if y is None:
        y = torch.empty_like(x)
    _req(y, "y", dt_)
    st = lib().ssm_decode_step_mamba3(_ptr(state), _ptr(prev_B), _ptr(prev_x), _ptr(x),
                                      _ptr(dt), _ptr(lam), _ptr(A), _ptr(B), _ptr(C), _ptr(D),
                                      _ptr(z), _ptr(y), batch, nheads, headdim, dstate, ngroups,
                                      _DT[dt_], _stream(stream))
    _check(st, "ssm_decode_step_mamba3")
    return y


def ssd_mamba3_mimo_fwd(x, dt, lam, A_head, B, C, chunk=16, out_dtype=None, y=None,
                        final_state=None, return_final_state=True, initial_state=None,
                        prev_B=None, prev_x=None, stream=None, block_states=None):
    """Mamba-3 MIMO (rank R) chunked prefill.  x: (batch, seqlen, R, nheads, headdim);
    B, C: (batch, seqlen, R, ngroups, dstate); dt, lam: (batch, seqlen, nheads) fp32;
    prev_B: (batch, R, ngroups, dstate), prev_x: (batch, R, nheads, headdim) (both or
    neither).  ``block_states`` (fp32, at least ``ssd_chunked_checkpoint_bytes(batch,
    seqlen * R, nheads)`` bytes) also keeps the states ``ssd_mamba3_mimo_bwd`` starts
    from.  Returns (y (batch, seqlen, R, nheads, headdim), final_state)."""
    _req(x, "x", ndim=5)
    in_dt = x.dtype
    if in_dt not in _DT:
        raise TypeError("x must be float32 or bfloat16")
    batch, seqlen, rank, nheads, headdim = x.shape
    _req(dt, "dt", torch.float32, 3)
    _req(lam, "lam", torch.float32, 3)
    _req(A_head, "A_head", torch.float32, 1)
    _req(B, "B", in_dt, 5)
    _req(C, "C", in_dt, 5)
    ngroups, dstate = B.shape[3], B.shape[4]
    out_dt = in_dt if out_dtype is None else out_dtype
    if y is None:
        y = torch.empty_like(x, dtype=out_dt)
    _req(y, "y", out_dt)
    if final_state is None and return_final_state:
        final_state = torch.empty((batch, nheads, headdim, dstate), dtype=torch.float32,
                                  device=x.device)
    _opt(final_state, "final_state", torch.float32)
    _opt(initial_state, "initial_state", torch.float32)
    _opt(prev_B, "prev_B", in_dt)
    _opt(prev_x, "prev_x", in_dt)
    if block_states is not None:
        _req(block_states, "block_states", torch.float32)
        if block_states.numel() * 4 < ssd_chunked_checkpoint_bytes(batch, seqlen * rank, nheads,
                                                                   headdim, dstate):
            raise ValueError("block_states is smaller than ssd_chunked_checkpoint_bytes(...)")
        st = lib().ssd_mamba3_mimo_fwd_ckpt(_ptr(x), _ptr(dt), _ptr(lam), _ptr(A_head), _ptr(B),
                                            _ptr(C), int(chunk), int(rank), _ptr(initial_state),
                                            _ptr(prev_B), _ptr(prev_x), _ptr(y), _ptr(final_state),
                                            _ptr(block_states), batch, seqlen, nheads, headdim,
                                            dstate, ngroups, _DT[in_dt], _DT[out_dt],
                                            _stream(stream))
        _check(st, "ssd_mamba3_mimo_fwd_ckpt")
        return y, final_state
    st = lib().ssd_mamba3_mimo_fwd(_ptr(x), _ptr(dt), _ptr(lam), _ptr(A_head), _ptr(B), _ptr(C),
                                   int(chunk), int(rank), _ptr(initial_state), _ptr(prev_B),
                                   _ptr(prev_x), _ptr(y), _ptr(final_state), batch, seqlen,
                                   nheads, headdim, dstate, ngroups, _DT[in_dt], _DT[out_dt],
                                   _stream(stream))
    _check(st, "ssd_mamba3_mimo_fwd")
    return y, final_state


def ssm_decode_step_mamba3_mimo(state, prev_B, prev_x, x, dt, lam, A, B, C, D=None, z=None,
                                y=None, stream=None):
    """One Mamba-3 MIMO (rank R) decode step; ``state`` (batch, nheads, headdim, dstate)
    fp32 is updated in place.  x, z, prev_x: (batch, R, nheads, headdim); B, C, prev_B:
    (batch, R, ngroups, dstate); dt, lam: (batch, nheads) fp32; A, D: (nheads,) fp32.
    Returns y (batch, R, nheads, headdim)."""
    _req(state, "state", torch.float32, 4)
    batch, nheads, headdim, dstate = state.shape
    _req(x, "x", ndim=4)
    dt_ = x.dtype
    if dt_ not in _DT:
        raise TypeError("x must be float32 or bfloat16")
    rank = x.shape[1]
    _req(dt, "dt", torch.float32, 2)
    _req(lam, "lam", torch.float32, 2)
    _req(A, "A", torch.float32, 1)
    _req(B, "B", dt_, 4)
    _req(C, "C", dt_, 4)
    _req(prev_B, "prev_B", dt_, 4)
    _req(prev_x, "prev_x", dt_, 4)
    ngroups = B.shape[2]
    _opt(D, "D", torch.float32)
    _opt(z, "z", dt_)
    if y is None:
        y = torch.empty_like(x)
    _req(y, "y", dt_)
    st = lib().ssm_decode_step_mamba3_mimo(_ptr(state), _ptr(prev_B), _ptr(prev_x), _ptr(x),
                                           _ptr(dt), _ptr(lam), _ptr(A), _ptr(B), _ptr(C),
                                           _ptr(D), _ptr(z), _ptr(y), batch, rank, nheads,
                                           headdim, dstate, ngroups, _DT[dt_], _stream(stream))
    _check(st, "ssm_decode_step_mamba3_mimo")
    return y


# ---------------------------------------------------- norm, recurrence, loss
#
# Tensors a call allocates for itself (outputs, workspaces) belong to the
# stream the call runs on, so that their memory is not handed out again before
# the kernels there are done with it.

def _new(like, shape, dtype, stream):
    if stream is None:
        if shape == like.shape:  # the cheaper call of the two
            return torch.empty_like(like, dtype=dtype, memory_format=torch.contiguous_format)
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _out(t, name, like, shape, dtype, stream):
    """The given output, checked, or a new one."""
    return _new(like, shape, dtype, stream) if t is None else _like(t, name, shape, dtype)


def _work(t, like, need, stream):
    """The given workspace, or a new one."""
    return (_new(like, max(need, 256), torch.uint8, stream) if t is None else
            _req(t, "workspace", torch.uint8))


def _p(t):
    return None if t is None else t.data_ptr()


def _raw(stream, t):
    """The stream's handle: the given one's, or the current one's of t's device (without
    the Stream object, whose making takes half as long as a kernel launch)."""
    return (torch._C._cuda_getCurrentRawStream(t.get_device()) if stream is None else
            stream.cuda_stream)


def _like(t, name, ref, dtype):
    """Checks a given output against the tensor it has to be shaped like."""
    _req(t, name, dtype)
    if t.shape != ref:
        _shape(t, name, ref)
    return t


def _norm_args(x, weight, residual):
    _req(x, "x")
    if x.dim() < 1 or x.dtype not in _DT:
        raise TypeError("x must be a float32 or bfloat16 tensor of at least one dimension")
    dim = x.shape[-1]
    _req(weight, "weight", torch.float32)
    _shape(weight, "weight", (dim,))
    if residual is not None:
        _req(residual, "residual")
        _shape(residual, "residual", x.shape)
        if residual.dtype not in (x.dtype, torch.float32):
            raise TypeError(f"residual must be {x.dtype} or float32, got {residual.dtype}")
    return x.numel() // dim if dim else 0, dim


def ssm_add_rmsnorm_fwd(x, weight, residual=None, eps=1e-5, out_dtype=None, sum_dtype=None, y=None,
                        sum_out=None, return_sum=True, stream=None):
    """RMS norm of x + residual over the last dimension.  x, residual: (..., dim);
    weight: (dim,) fp32.  The sum is kept in ``sum_dtype`` (the residual's type, or
    x's; float32 where the residual stream is kept in 32 bits).  ``sum_out`` may be
    ``residual`` itself.  Returns (y, sum); sum is None with ``return_sum`` false
    and no ``sum_out``."""
    rows, dim = _norm_args(x, weight, residual)
    out_dt = x.dtype if out_dtype is None else out_dtype
    res_dt = _sum_dtype(x, residual, sum_dtype, sum_out)
    y = _out(y, "y", x, x.shape, out_dt, stream)
    if sum_out is not None or return_sum:
        sum_out = _out(sum_out, "sum_out", x, x.shape, res_dt, stream)
    st = lib().ssm_add_rmsnorm_fwd(_p(x), _p(residual), _p(weight), float(eps), _p(y),
                                   _p(sum_out), rows, dim, _DT[x.dtype], _DT[res_dt],
                                   _dt_code(out_dt, "out_dtype"), _raw(stream, x))
    _check(st, "ssm_add_rmsnorm_fwd")
    return y, sum_out


def _dt_code(dt, name):
    if dt not in _DT:
        raise TypeError(f"{name} must be float32 or bfloat16, got {dt}")
    return _DT[dt]


def _sum_dtype(x, residual, sum_dtype, sum_out):
    """The type the residual stream is kept in: the residual's where there is one."""
    dt = (residual.dtype if residual is not None else
          sum_out.dtype if sum_out is not None else
          x.dtype if sum_dtype is None else sum_dtype)
    if sum_dtype is not None and dt != sum_dtype:
        raise TypeError(f"sum_dtype must be the residual's type {dt}, got {sum_dtype}")
    if dt not in (x.dtype, torch.float32):
        raise TypeError(f"the sum must be {x.dtype} or float32, got {dt}")
    return dt


def ssm_add_rmsnorm_e4m3_fwd(x, weight, residual=None, eps=1e-5, group=128, sum_dtype=None, q=None,
                             scales=None, sum_out=None, return_sum=True, stream=None):
    """ssm_add_rmsnorm_fwd with y in 8 bits: q (float8_e4m3fn, like x) and fp32
    scales (..., ceil(dim / group)) with y = q * scale of its ``group`` of 32, 64, 128 or
    256 consecutive values (group 0: one scale a row).  Returns (q, scales, sum)."""
    rows, dim = _norm_args(x, weight, residual)
    res_dt = _sum_dtype(x, residual, sum_dtype, sum_out)
    group = int(group)
    if group not in (0, 32, 64, 128, 256):
        raise SSMError(5, "ssm_add_rmsnorm_e4m3_fwd")
    sshape = tuple(x.shape[:-1]) + (1 if group == 0 else -(-dim // group),)
    q = _out(q, "q", x, x.shape, torch.float8_e4m3fn, stream)
    scales = _out(scales, "scales", x, sshape, torch.float32, stream)
    if sum_out is not None or return_sum:
        sum_out = _out(sum_out, "sum_out", x, x.shape, res_dt, stream)
    st = lib().ssm_add_rmsnorm_e4m3_fwd(_p(x), _p(residual), _p(weight), float(eps), group,
                                        _p(q), _p(scales), _p(sum_out), rows, dim,
                                        _DT[x.dtype], _DT[res_dt], _raw(stream, x))
    _check(st, "ssm_add_rmsnorm_e4m3_fwd")
    return q, scales, sum_out


def ssm_add_rmsnorm_bwd_workspace_bytes(rows, dim) -> int:
    return int(lib().ssm_add_rmsnorm_bwd_workspace_bytes(rows, dim))


def ssm_add_rmsnorm_bwd(dy, sum, weight, dsum=None, eps=1e-5, x_dtype=None, dx=None,
                        dresidual=None, dweight=None, workspace=None, stream=None):
    """Gradient of ``ssm_add_rmsnorm_fwd`` at the sum it returned.  dy: like y; dsum: the
    gradient arriving at the sum itself, in its type, or None.  ``x_dtype``: the type of
    x's gradient (dy's where the sum is fp32, else the sum's).  Returns a dict: dx,
    dresidual (the same values in the sum's type; the same tensor as dx where the types
    agree) and dweight (fp32)."""
    _req(sum, "sum")
    if sum.dim() < 1 or sum.dtype not in _DT:
        raise TypeError("sum must be a float32 or bfloat16 tensor of at least one dimension")
    dim = sum.shape[-1]
    rows = sum.numel() // dim if dim else 0
    _req(weight, "weight", torch.float32)
    _shape(weight, "weight", (dim,))
    _req(dy, "dy")
    _shape(dy, "dy", sum.shape)
    if dsum is not None:
        _like(dsum, "dsum", sum.shape, sum.dtype)
    dx_dt = x_dtype or (dx.dtype if dx is not None else
                        dy.dtype if sum.dtype == torch.float32 else sum.dtype)
    same = dx_dt == sum.dtype
    dx = _out(dx, "dx", sum, sum.shape, dx_dt, stream)
    if dresidual is not None or not same:
        dresidual = _out(dresidual, "dresidual", sum, sum.shape, sum.dtype, stream)
    dweight = _out(dweight, "dweight", sum, (dim,), torch.float32, stream)
    workspace = _work(workspace, sum, ssm_add_rmsnorm_bwd_workspace_bytes(rows, dim), stream)
    st = lib().ssm_add_rmsnorm_bwd(_p(sum), _p(weight), float(eps), _p(dy), _p(dsum),
                                   _p(dx), _p(dresidual), _p(dweight), rows, dim,
                                   _dt_code(dx_dt, "x_dtype"), _DT[sum.dtype],
                                   _dt_code(dy.dtype, "dy"), _p(workspace), workspace.numel(),
                                   _raw(stream, sum))
    _check(st, "ssm_add_rmsnorm_bwd")
    return {"dx": dx, "dresidual": dx if dresidual is None else dresidual, "dweight": dweight}


def ssm_linrec_checkpoint_bytes(batch, seqlen, dim) -> int:
    return int(lib().ssm_linrec_checkpoint_bytes(batch, seqlen, dim))


def ssm_linrec_workspace_bytes(batch, seqlen, dim) -> int:
    return int(lib().ssm_linrec_workspace_bytes(batch, seqlen, dim))


def ssm_linrec_bwd_workspace_bytes(batch, seqlen, dim) -> int:
    return int(lib().ssm_linrec_bwd_workspace_bytes(batch, seqlen, dim))


def _steps(t, name, dtype, shape):
    """Elements between the steps of a (batch, seqlen, dim) tensor whose channels are
    contiguous and whose batches follow one another: a contiguous tensor, or a range
    of the last dimension of one."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    batch, seqlen, dim = shape
    if t.is_contiguous():
        return dim
    sb, st, sd = t.stride()
    # a dimension of one element may carry any stride
    step = st if seqlen > 1 else sb if batch > 1 else dim
    if ((dim > 1 and sd != 1) or step < dim or
            (batch > 1 and seqlen > 1 and sb != seqlen * st)):
        raise ValueError(f"{name} must be contiguous, or a range of the last dimension of a "
                         f"contiguous tensor")
    return step


def _linrec_args(f, x, z, initial_state):
    if not isinstance(x, torch.Tensor) or x.dtype not in _DT:
        raise TypeError("x must be a float32 or bfloat16 tensor")
    if x.dim() != 3:
        raise ValueError(f"x must have 3 dims, got {x.dim()}")
    sx = _steps(x, "x", x.dtype, x.shape)
    sf = _steps(f, "f", x.dtype, x.shape)
    sz = 0 if z is None else _steps(z, "z", x.dtype, x.shape)
    batch, seqlen, dim = x.shape
    if initial_state is not None:
        _like(initial_state, "initial_state", (batch, dim), torch.float32)
    return sf, sx, sz


def ssm_linrec_fwd(f, x, z=None, initial_state=None, out_dtype=None, y=None, final_state=None,
                   checkpoints=None, workspace=None, return_final_state=True, stream=None):
    """Gated linear recurrence h_t = a_t h_{t-1} + (1 - a_t) x_t with a = sigmoid(f), and
    y = h * silu(z) (y = h without z).  f, x, z: (batch, seqlen, dim), each contiguous or a
    range of the last dimension of a contiguous tensor; initial_state, final_state:
    (batch, dim) fp32, which may be the same tensor (a decode step in place).  With
    ``checkpoints`` (a CUDA fp32 tensor of ssm_linrec_checkpoint_bytes bytes) the states
    ssm_linrec_bwd needs are kept.  Returns (y, final_state)."""
    sf, sx, sz = _linrec_args(f, x, z, initial_state)
    batch, seqlen, dim = x.shape
    out_dt = x.dtype if out_dtype is None else out_dtype
    y = _out(y, "y", x, x.shape, out_dt, stream)
    if final_state is not None or return_final_state:
        final_state = _out(final_state, "final_state", x, (batch, dim), torch.float32, stream)
    if workspace is not None or seqlen > 16:  # shorter sequences run without one
        workspace = _work(workspace, x, ssm_linrec_workspace_bytes(batch, seqlen, dim), stream)
    _kept(checkpoints, batch, seqlen, dim)
    st = lib().ssm_linrec_fwd(_p(f), _p(x), _p(z), sf, sx, sz, _p(initial_state), _p(y),
                              _p(final_state), _p(checkpoints), batch, seqlen, dim,
                              _DT[x.dtype], _dt_code(out_dt, "out_dtype"), _p(workspace),
                              0 if workspace is None else workspace.numel(), _raw(stream, x))
    _check(st, "ssm_linrec_fwd")
    return y, final_state


def _kept(checkpoints, batch, seqlen, dim):
    if checkpoints is not None:
        _req(checkpoints, "checkpoints", torch.float32)
        if checkpoints.numel() * 4 < ssm_linrec_checkpoint_bytes(batch, seqlen, dim):
            raise ValueError("checkpoints is smaller than ssm_linrec_checkpoint_bytes(...)")


def ssm_linrec_bwd(f, x, dy, z=None, initial_state=None, dfinal_state=None, checkpoints=None,
                   grad_dtype=None, workspace=None, want_dinitial_state=True, stream=None,
                   out=None):
    """Gradient of ``ssm_linrec_fwd`` for the loss sum(dy * y) + sum(dfinal_state *
    final_state).  Inputs as for the forward; dy like x and contiguous; checkpoints: what
    the forward kept, or None (its recurrence is run again).  Returns a dict: df, dx, dz
    (None without z) in ``grad_dtype`` (x's type by default), dinitial_state fp32 (or
    None).  ``out`` may map any of these names to a preallocated tensor to write."""
    sf, sx, sz = _linrec_args(f, x, z, initial_state)
    batch, seqlen, dim = x.shape
    _like(dy, "dy", x.shape, x.dtype)
    if dfinal_state is not None:
        _like(dfinal_state, "dfinal_state", (batch, dim), torch.float32)
    _kept(checkpoints, batch, seqlen, dim)
    gd = x.dtype if grad_dtype is None else grad_dtype
    names = ["df", "dx"] + ([] if z is None else ["dz"])
    if want_dinitial_state or (out and "dinitial_state" in out):
        names.append("dinitial_state")
    g = dict.fromkeys(("df", "dx", "dz", "dinitial_state"))
    out = out or {}
    for k in out:
        if k not in names:
            raise ValueError(f"out[{k!r}] is not an output of this call")
    for k in names:
        shape, dt = ((batch, dim), torch.float32) if k == "dinitial_state" else (x.shape, gd)
        g[k] = _out(out.get(k), f"out[{k!r}]", x, shape, dt, stream)
    workspace = _work(workspace, x, ssm_linrec_bwd_workspace_bytes(batch, seqlen, dim), stream)
    st = lib().ssm_linrec_bwd(_p(f), _p(x), _p(z), sf, sx, sz, _p(initial_state), _p(dy),
                              _p(dfinal_state), _p(checkpoints), _p(g["df"]), _p(g["dx"]),
                              _p(g["dz"]), _p(g["dinitial_state"]), batch, seqlen, dim,
                              _DT[x.dtype], _dt_code(gd, "grad_dtype"), _p(workspace),
                              workspace.numel(), _raw(stream, x))
    _check(st, "ssm_linrec_bwd")
    return g


def ssm_vocab_ce_workspace_bytes(tokens, dim, vocab) -> int:
    return int(lib().ssm_vocab_ce_workspace_bytes(tokens, dim, vocab))


def ssm_vocab_ce_bwd_workspace_bytes(tokens, dim, vocab) -> int:
    return int(lib().ssm_vocab_ce_bwd_workspace_bytes(tokens, dim, vocab))


def _vector(t, stream):
    """t, or a copy of it where it starts off a 16-byte boundary: the labels shifted by one
    (``labels[1:]``) are contiguous and 8-byte aligned."""
    if t.data_ptr() % 16 == 0:
        return t
    with torch.cuda.stream(stream):  # no other stream for None
        return t.clone()


def _ce_args(h, W, targets):
    _req(h, "h", torch.bfloat16, 2)
    _req(W, "W", torch.bfloat16, 2)
    if W.shape[1] != h.shape[1]:
        raise ValueError(f"W must have shape (vocab, {h.shape[1]}), got {tuple(W.shape)}")
    _like(targets, "targets", (h.shape[0],), torch.int64)
    return h.shape[0], h.shape[1], W.shape[0]


def ssm_vocab_ce_fwd(h, W, targets, loss=None, lse=None, workspace=None, stream=None):
    """Softmax cross entropy of the logits h W^T without the logits in memory.  h:
    (tokens, dim), W: (vocab, dim) bf16, dim a multiple of 8; targets: (tokens,) int64, a
    negative one for a token without loss.  Returns (loss, lse), (tokens,) fp32 each."""
    tokens, dim, vocab = _ce_args(h, W, targets)
    targets = _vector(targets, stream)
    loss = _out(loss, "loss", h, (tokens,), torch.float32, stream)
    lse = _out(lse, "lse", h, (tokens,), torch.float32, stream)
    workspace = _work(workspace, h, ssm_vocab_ce_workspace_bytes(tokens, dim, vocab), stream)
    st = lib().ssm_vocab_ce_fwd(_p(h), _p(W), _p(targets), _p(loss), _p(lse), tokens, dim,
                                vocab, _DT[h.dtype], _p(workspace), workspace.numel(),
                                _raw(stream, h))
    _check(st, "ssm_vocab_ce_fwd")
    return loss, lse


def ssm_vocab_ce_bwd(h, W, targets, lse, dloss, grad_dtype=None, workspace=None, stream=None,
                     out=None):
    """Gradient of ``ssm_vocab_ce_fwd`` for the loss sum(dloss * loss), with the lse it
    returned; dloss: (tokens,) fp32.  Returns a dict: dh, dW in ``grad_dtype`` (h's type by
    default).  ``out`` may map either name to a preallocated tensor to write."""
    tokens, dim, vocab = _ce_args(h, W, targets)
    _like(lse, "lse", (tokens,), torch.float32)
    _like(dloss, "dloss", (tokens,), torch.float32)
    targets, lse, dloss = (_vector(t, stream) for t in (targets, lse, dloss))
    gd = h.dtype if grad_dtype is None else grad_dtype
    code = _dt_code(gd, "grad_dtype")
    out = out or {}
    g = {}
    for k in out:
        if k not in ("dh", "dW"):
            raise ValueError(f"out[{k!r}] is not an output of this call")
    for k, t in (("dh", h), ("dW", W)):
        g[k] = _out(out.get(k), f"out[{k!r}]", h, t.shape, gd, stream)
    workspace = _work(workspace, h, ssm_vocab_ce_bwd_workspace_bytes(tokens, dim, vocab), stream)
    st = lib().ssm_vocab_ce_bwd(_p(h), _p(W), _p(targets), _p(lse), _p(dloss),
                                _p(g["dh"]), _p(g["dW"]), tokens, dim, vocab, _DT[h.dtype], code,
                                _p(workspace), workspace.numel(), _raw(stream, h))
    _check(st, "ssm_vocab_ce_bwd")
    return g


# ------------------------------- query and key heads, gated delta rule

def _token_step(t, name, dtype, shape):
    """Elements between the tokens of a (batch, seqlen, heads, dim) tensor whose heads are
    contiguous and whose batches follow one another: a contiguous tensor, or a range of
    the columns of a projection."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    batch, seqlen, heads, dim = shape
    if t.is_contiguous():
        return heads * dim
    sb, st, sh, sd = t.stride()
    # a dimension of one element may carry any stride
    step = st if seqlen > 1 else sb if batch > 1 else heads * dim
    if ((dim > 1 and sd != 1) or (heads > 1 and sh != dim) or step < heads * dim or
            (batch > 1 and seqlen > 1 and sb != seqlen * st)):
        raise ValueError(f"{name} must be contiguous, or a range of the columns of a "
                         f"contiguous projection")
    return step


def _one_device(first, *others):
    if _devices() == 1:
        return
    device = first.get_device()
    for t in others:
        if t is not None and t.get_device() != device:
            raise ValueError("all tensors must be on one device")
    if device != torch.cuda.current_device():  # where the kernels would run
        raise ValueError(f"the tensors are on device {device}, which is not the current one")


@functools.lru_cache(None)
def _devices():
    return torch.cuda.device_count()


def _outputs(given, wants, stream):
    """The tensors of ``wants`` (name: what it is shaped like, shape, dtype), given or new."""
    if given:
        for name in given:
            if name not in wants:
                raise ValueError(f"out[{name!r}] is not an output of this call")
    g = {}
    for name, (like, shape, dtype) in wants.items():
        t = given.get(name) if given else None
        g[name] = (_new(like, shape, dtype, stream) if t is None else
                   _like(t, f"out[{name!r}]", shape, dtype))
    return g


def _qk_args(q, k, q_weight, k_weight, positions, inv_freq):
    """(q, its step, k's step, tokens, heads of both, headdim, rot_dim)."""
    if not isinstance(q, torch.Tensor) or q.dtype not in _DT:
        raise TypeError("q must be a float32 or bfloat16 tensor")
    if q.dim() != 4:
        raise ValueError(f"q must have 4 dims, got {q.dim()}")
    batch, seqlen, qheads, dim = q.shape
    sq = _token_step(q, "q", q.dtype, q.shape)
    kheads = sk = 0
    if k is not None:
        if not isinstance(k, torch.Tensor) or k.dim() != 4:
            raise TypeError("k must be a CUDA tensor of 4 dims")
        kheads = k.shape[2]
        sk = _token_step(k, "k", q.dtype, (batch, seqlen, kheads, dim))
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            _like(w, name, (dim,), torch.float32)
    rot = 0
    if inv_freq is not None and inv_freq.numel():
        _req(inv_freq, "inv_freq", torch.float64, 1)
        rot = 2 * inv_freq.numel()
        if rot > dim:
            raise ValueError(f"inv_freq must have at most {dim // 2} elements, got {rot // 2}")
        if positions is None:
            raise ValueError("positions are needed with inv_freq")
        _like(positions, "positions", (batch, seqlen), torch.int64)
    _one_device(q, k, q_weight, k_weight, positions if rot else None, inv_freq if rot else None)
    return sq, sk, batch * seqlen, qheads, kheads, dim, rot


def ssm_qk_norm_rope_fwd(q, k=None, q_weight=None, k_weight=None, positions=None, inv_freq=None,
                         eps=1e-5, interleaved=False, out_dtype=None, q_out=None, k_out=None,
                         stream=None):
    """RMS norm of every head of q (batch, seqlen, qheads, headdim) and k (batch, seqlen,
    kheads, headdim) over its own columns, and the rotation by position, in one pass.  q
    and k may be ranges of the columns of one projection; k may be None.  weights:
    (headdim,) fp32 or None (ones; 1 / sqrt(headdim) gives heads of length one).
    positions: (batch, seqlen) int64; inv_freq: (rot_dim / 2,) fp64, or None for no
    rotation; pairs are (i, i + rot_dim / 2), or (2 i, 2 i + 1) with ``interleaved``.
    Returns (q_out, k_out), contiguous, in ``out_dtype`` (q's type by default)."""
    sq, sk, tokens, qheads, kheads, dim, rot = _qk_args(q, k, q_weight, k_weight, positions,
                                                        inv_freq)
    out_dt = q.dtype if out_dtype is None else out_dtype
    code = _dt_code(out_dt, "out_dtype")
    q_out = _out(q_out, "q_out", q, q.shape, out_dt, stream)
    if k is not None:
        k_out = _out(k_out, "k_out", k, k.shape, out_dt, stream)
        _one_device(q, q_out, k_out)
    elif k_out is not None:
        raise ValueError("k_out without k")
    st = lib().ssm_qk_norm_rope_fwd(_p(q), _p(k), sq, sk, _p(q_weight), _p(k_weight),
                                    _p(positions) if rot else None, _p(inv_freq) if rot else None,
                                    float(eps), rot, int(bool(interleaved)), _p(q_out), _p(k_out),
                                    tokens, qheads, kheads, dim, _DT[q.dtype], code,
                                    _raw(stream, q))
    _check(st, "ssm_qk_norm_rope_fwd")
    return q_out, k_out


def ssm_qk_norm_rope_bwd_workspace_bytes(tokens, qheads, kheads, headdim) -> int:
    return int(lib().ssm_qk_norm_rope_bwd_workspace_bytes(tokens, qheads, kheads, headdim))


def ssm_qk_norm_rope_bwd(dq_out, dk_out, q, k=None, q_weight=None, k_weight=None, positions=None,
                         inv_freq=None, eps=1e-5, interleaved=False, workspace=None, stream=None,
                         out=None):
    """Gradient of ``ssm_qk_norm_rope_fwd`` for the loss sum(dq_out * q_out) + sum(dk_out *
    k_out), dq_out and dk_out contiguous and of the outputs' type; the other arguments as
    given to the forward.  Returns a dict: dq, dk in q's type, contiguous, and dq_weight,
    dk_weight fp32 (None where there was no weight).  ``out`` may map any of these names
    to a preallocated tensor to write."""
    sq, sk, tokens, qheads, kheads, dim, rot = _qk_args(q, k, q_weight, k_weight, positions,
                                                        inv_freq)
    _req(dq_out, "dq_out")
    code = _dt_code(dq_out.dtype, "dq_out")
    _like(dq_out, "dq_out", q.shape, dq_out.dtype)
    wants = {"dq": (q, q.shape, q.dtype)}
    if k is not None:
        _like(dk_out, "dk_out", k.shape, dq_out.dtype)
        wants["dk"] = (k, k.shape, q.dtype)
    if q_weight is not None:
        wants["dq_weight"] = (q_weight, q_weight.shape, torch.float32)
    if k is not None and k_weight is not None:
        wants["dk_weight"] = (k_weight, k_weight.shape, torch.float32)
    g = dict.fromkeys(("dq", "dk", "dq_weight", "dk_weight"))
    g.update(_outputs(out, wants, stream))
    if g["dq_weight"] is not None or g["dk_weight"] is not None or workspace is not None:
        workspace = _work(workspace, q, ssm_qk_norm_rope_bwd_workspace_bytes(tokens, qheads, kheads,
                                                                             dim), stream)
    _one_device(q, dq_out, dk_out if k is not None else None, workspace, *g.values())
    st = lib().ssm_qk_norm_rope_bwd(_p(dq_out), _p(dk_out) if k is not None else None, _p(q), _p(k),
                                    sq, sk, _p(q_weight), _p(k_weight),
                                    _p(positions) if rot else None, _p(inv_freq) if rot else None,
                                    float(eps), rot, int(bool(interleaved)), _p(g["dq"]),
                                    _p(g["dk"]), _p(g["dq_weight"]), _p(g["dk_weight"]), tokens,
                                    qheads, kheads, dim, _DT[q.dtype], code, _p(workspace),
                                    0 if workspace is None else workspace.numel(), _raw(stream, q))
    _check(st, "ssm_qk_norm_rope_bwd")
    return g


def ssm_gated_delta_checkpoint_bytes(batch, seqlen, nheads, dstate, headdim) -> int:
    return int(lib().ssm_gated_delta_checkpoint_bytes(batch, seqlen, nheads, dstate, headdim))


def ssm_gated_delta_workspace_bytes(batch, seqlen, nheads, dstate, headdim) -> int:
    return int(lib().ssm_gated_delta_workspace_bytes(batch, seqlen, nheads, dstate, headdim))


@functools.lru_cache(None)
def ssm_gated_delta_walked_steps() -> int:
    """Steps a bf16 sequence is walked up to, without a workspace, where nothing is kept."""
    return int(lib().ssm_gated_delta_walked_steps())


def _delta_args(q, k, v, g, beta, initial_state):
    """(steps of q, k, v; batch, seqlen, nheads, ngroups, dstate, headdim)."""
    for t, name in ((q, "q"), (v, "v")):
        if not isinstance(t, torch.Tensor) or t.dtype not in _DT:
            raise TypeError(f"{name} must be a float32 or bfloat16 tensor")
        if t.dim() != 4:
            raise ValueError(f"{name} must have 4 dims, got {t.dim()}")
    batch, seqlen, ngroups, dstate = q.shape
    nheads, headdim = v.shape[2], v.shape[3]
    if (nheads % ngroups or not nheads if ngroups else nheads):
        raise ValueError(f"nheads {nheads} must be a multiple of ngroups {ngroups}")
    sq = _token_step(q, "q", q.dtype, q.shape)
    sk = _token_step(k, "k", q.dtype, q.shape)
    sv = _token_step(v, "v", q.dtype, (batch, seqlen, nheads, headdim))
    _req(g, "g")
    _dt_code(g.dtype, "g")
    _like(g, "g", (batch, seqlen, nheads), g.dtype)
    _like(beta, "beta", (batch, seqlen, nheads), g.dtype)
    if initial_state is not None:
        _like(initial_state, "initial_state", (batch, nheads, headdim, dstate), torch.float32)
    return sq, sk, sv, batch, seqlen, nheads, ngroups, dstate, headdim


def _delta_kept(checkpoints, *sizes):
    if checkpoints is not None:
        _req(checkpoints, "checkpoints", torch.uint8)
        if checkpoints.numel() < ssm_gated_delta_checkpoint_bytes(*sizes):
            raise ValueError("checkpoints is smaller than ssm_gated_delta_checkpoint_bytes(...)")


def ssm_gated_delta_fwd(q, k, v, g, beta, initial_state=None, out_dtype=None, y=None,
                        final_state=None, checkpoints=None, workspace=None,
                        return_final_state=True, stream=None):
    """Gated delta rule S = exp(g) S; u = beta (v - S k); S += u k^T; y = S q per head.  q,
    k: (batch, seqlen, ngroups, dstate), v: (batch, seqlen, nheads, headdim), each contiguous
    or a range of the columns of a projection; g, beta: (batch, seqlen, nheads) fp32 or
    bf16; initial_state, final_state: (batch, nheads, headdim, dstate) fp32, which may be
    the same tensor (a decode step in place).  A beta of 0 masks a step, a g of -inf starts
    the state anew.  With ``checkpoints`` (a CUDA uint8 tensor of
    ssm_gated_delta_checkpoint_bytes bytes) what ssm_gated_delta_bwd needs is kept.
    Returns (y, final_state)."""
    sq, sk, sv, *sizes = _delta_args(q, k, v, g, beta, initial_state)
    batch, seqlen, nheads, ngroups, dstate, headdim = sizes
    out_dt = q.dtype if out_dtype is None else out_dtype
    code = _dt_code(out_dt, "out_dtype")
    y = _out(y, "y", v, v.shape, out_dt, stream)
    if final_state is not None or return_final_state:
        final_state = _out(final_state, "final_state", v if initial_state is None else initial_state,
                           (batch, nheads, headdim, dstate), torch.float32, stream)
    five = batch, seqlen, nheads, dstate, headdim
    _delta_kept(checkpoints, *five)
    if workspace is not None or (q.dtype == torch.bfloat16 and
                                 (checkpoints is not None or
                                  seqlen > ssm_gated_delta_walked_steps())):
        need = 1024 if checkpoints is not None else ssm_gated_delta_workspace_bytes(*five)
        workspace = _work(workspace, q, need, stream)
    _one_device(q, k, v, g, beta, initial_state, y, final_state, checkpoints, workspace)
    st = lib().ssm_gated_delta_fwd(_p(q), _p(k), _p(v), sq, sk, sv, _p(g), _p(beta),
                                   _p(initial_state), _p(y), _p(final_state), _p(checkpoints),
                                   *sizes, _DT[q.dtype], _DT[g.dtype], code, _p(workspace),
                                   0 if workspace is None else workspace.numel(), _raw(stream, q))
    _check(st, "ssm_gated_delta_fwd")
    return y, final_state


def ssm_gated_delta_bwd_workspace_bytes(batch, seqlen, nheads, dstate, headdim) -> int:
    return int(lib().ssm_gated_delta_bwd_workspace_bytes(batch, seqlen, nheads, dstate, headdim))


def ssm_gated_delta_bwd(q, k, v, g, beta, dy, initial_state=None, dfinal_state=None,
                        checkpoints=None, grad_dtype=None, workspace=None,
                        want_dinitial_state=True, stream=None, out=None):
    """Gradient of ``ssm_gated_delta_fwd`` for the loss sum(dy * y) + sum(dfinal_state *
    final_state), bf16 inputs.  Inputs as for the forward; dy like v and contiguous;
    checkpoints: what the forward kept, or None (it is run again).  Returns a dict: dq, dk, dv
    in ``grad_dtype`` (q's type by default), dg, dbeta in g's type, dinitial_state fp32 (or
    None).  ``out`` may map any of these names to a preallocated tensor to write."""
    sq, sk, sv, *sizes = _delta_args(q, k, v, g, beta, initial_state)
    batch, seqlen, nheads, ngroups, dstate, headdim = sizes
    _like(dy, "dy", v.shape, q.dtype)
    if dfinal_state is not None:
        _like(dfinal_state, "dfinal_state", (batch, nheads, headdim, dstate), torch.float32)
    five = batch, seqlen, nheads, dstate, headdim
    _delta_kept(checkpoints, *five)
    gd = q.dtype if grad_dtype is None else grad_dtype
    code = _dt_code(gd, "grad_dtype")
    wants = {"dq": (q, q.shape, gd), "dk": (q, q.shape, gd), "dv": (v, v.shape, gd),
             "dg": (g, g.shape, g.dtype), "dbeta": (g, g.shape, g.dtype)}
    if want_dinitial_state or (out and "dinitial_state" in out):
        wants["dinitial_state"] = (v, (batch, nheads, headdim, dstate), torch.float32)
    grads = {"dinitial_state": None}
    grads.update(_outputs(out, wants, stream))
    need = ssm_gated_delta_bwd_workspace_bytes(*five)
    if checkpoints is None:
        need += ssm_gated_delta_checkpoint_bytes(*five)
    workspace = _work(workspace, q, need, stream)
    _one_device(q, k, v, g, beta, initial_state, dy, dfinal_state, checkpoints, workspace,
                *grads.values())
    st = lib().ssm_gated_delta_bwd(_p(q), _p(k), _p(v), sq, sk, sv, _p(g), _p(beta),
                                   _p(initial_state), _p(dy), _p(dfinal_state), _p(checkpoints),
                                   _p(grads["dq"]), _p(grads["dk"]), _p(grads["dv"]),
                                   _p(grads["dg"]), _p(grads["dbeta"]),
                                   _p(grads["dinitial_state"]), *sizes, _DT[q.dtype],
                                   _DT[g.dtype], code, _p(workspace), workspace.numel(),
                                   _raw(stream, q))
    _check(st, "ssm_gated_delta_bwd")
    return grads
