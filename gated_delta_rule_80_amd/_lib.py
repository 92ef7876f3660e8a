"""ctypes binding of libkda (include/kda.h): argument marshalling only.

Every function here fills the C argument struct from torch tensors (device
memory and the current stream come from torch) and calls the entry point of the
same name.  Nothing is computed in Python; if the library is missing the call
raises instead of falling back to anything.
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
_ROOT = os.path.dirname(_PKG)
LIB_PATH = os.path.join(_PKG, "libkda.so")
HEADER_PATH = os.path.join(_ROOT, "include", "kda.h")

KDA_OK = 0
KDA_BF16 = 0
KDA_FP32 = 1
KDA_FLAG_L2NORM_QK = 1
KDA_FLAG_BETA_LOGITS = 2
ABI_VERSION = 7
KDA_STAGE_PREP, KDA_STAGE_STATE, KDA_STAGE_CONV_TAIL, KDA_STAGE_OUTPUT = 0, 1, 2, 3
KDA_STAGE_STATE_TAIL = 4  # stages 1 and 2 in one launch, as kda_prefill runs them
NUM_STAGES = 4
STATUS_NAMES = {0: "KDA_OK", 1: "KDA_ERR_NULL", 2: "KDA_ERR_SHAPE", 3: "KDA_ERR_DTYPE",
                4: "KDA_ERR_ALIGN", 5: "KDA_ERR_ALIAS", 6: "KDA_ERR_UNSUPPORTED",
                7: "KDA_ERR_WORKSPACE", 8: "KDA_ERR_HIP", 9: "KDA_ERR_VALUE",
                10: "KDA_ERR_SCRATCH"}
KDA_ERR_SCRATCH = 10

_vp = ctypes.c_void_p


class PrefillArgs(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32),
                ("D", ctypes.c_int32), ("chunk", ctypes.c_int32), ("conv_k", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("l2_eps", ctypes.c_float), ("scale", ctypes.c_float),
                ("io", ctypes.c_int32),
                ("q", _vp), ("k", _vp), ("v", _vp), ("g", _vp), ("beta", _vp), ("conv_w", _vp),
                ("conv_state_in", _vp), ("S0", _vp), ("o", _vp), ("S_T", _vp),
                ("conv_state_out", _vp),
                ("A_log", _vp), ("dt_bias", _vp), ("o_norm_w", _vp), ("o_norm_eps", ctypes.c_float),
                ("o_gate", _vp), ("cu_seqlens", _vp), ("n_seqs", ctypes.c_int32)]


class ConvNormArgs(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32),
                ("D", ctypes.c_int32), ("conv_k", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("l2_eps", ctypes.c_float), ("io", ctypes.c_int32),
                ("q", _vp), ("k", _vp), ("v", _vp), ("conv_w", _vp), ("conv_state_in", _vp),
                ("q_out", _vp), ("k_out", _vp), ("v_out", _vp), ("conv_state_out", _vp)]


class DecodeArgs(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("D", ctypes.c_int32),
                ("conv_k", ctypes.c_int32), ("flags", ctypes.c_uint32), ("l2_eps", ctypes.c_float),
                ("scale", ctypes.c_float), ("io", ctypes.c_int32),
                ("q", _vp), ("k", _vp), ("v", _vp), ("g", _vp), ("beta", _vp), ("conv_w", _vp),
                ("conv_state", _vp), ("S", _vp), ("o", _vp),
                ("A_log", _vp), ("dt_bias", _vp), ("o_norm_w", _vp), ("o_norm_eps", ctypes.c_float),
                ("o_gate", _vp)]


class BackwardArgs(ctypes.Structure):
    _fields_ = [("fwd", PrefillArgs), ("dO", _vp), ("dS_T", _vp), ("dq", _vp), ("dk", _vp),
                ("dv", _vp), ("dg", _vp), ("dbeta", _vp), ("dS0", _vp), ("dconv_w", _vp),
                ("dconv_state", _vp), ("dA_log", _vp), ("ddt_bias", _vp), ("do_norm_w", _vp),
                ("do_gate", _vp)]


class KdaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        name = STATUS_NAMES.get(self.status, str(status))
        super().__init__(f"{where}: {name} ({_status_str(self.status)})")


_lib = None


def declared_functions() -> list[str]:
    """Names of the functions include/kda.h declares (used by the export test)."""
    text = open(HEADER_PATH).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(kda_[a-z0-9_]+)\s*\(", text)))


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libkda.so (built in-tree).  Raises if it is not built."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is missing: build it with `python -m gated_delta_rule_80_amd.build` "
                           "(there is no fallback implementation)")
    lib = ctypes.CDLL(p)
    P = ctypes.POINTER
    lib.kda_abi_version.restype = ctypes.c_int
    lib.kda_status_str.restype = ctypes.c_char_p
    lib.kda_status_str.argtypes = [ctypes.c_int]
    lib.kda_validate_prefill.restype = ctypes.c_int
    lib.kda_validate_prefill.argtypes = [P(PrefillArgs)]
    lib.kda_prefill_workspace_bytes.restype = ctypes.c_size_t
    lib.kda_prefill_workspace_bytes.argtypes = [P(PrefillArgs)]
    lib.kda_prefill.restype = ctypes.c_int
    lib.kda_prefill.argtypes = [P(PrefillArgs), _vp, ctypes.c_size_t, _vp]
    lib.kda_prefill_static.restype = ctypes.c_int
    lib.kda_prefill_static.argtypes = [P(PrefillArgs), _vp]
    lib.kda_prefill_stage.restype = ctypes.c_int
    lib.kda_prefill_stage.argtypes = [P(PrefillArgs), _vp, ctypes.c_size_t, ctypes.c_int, _vp]
    lib.kda_prefill_walk_segments.restype = ctypes.c_int
    lib.kda_prefill_walk_segments.argtypes = [P(PrefillArgs)]
    lib.kda_prefill_state_map_workspace_bytes.restype = ctypes.c_size_t
    lib.kda_prefill_state_map_workspace_bytes.argtypes = [P(PrefillArgs)]
    lib.kda_prefill_state_map.restype = ctypes.c_int
    lib.kda_prefill_state_map.argtypes = [P(PrefillArgs), _vp, ctypes.c_size_t, _vp, _vp, _vp]
    lib.kda_validate_conv_norm.restype = ctypes.c_int
    lib.kda_validate_conv_norm.argtypes = [P(ConvNormArgs)]
    lib.kda_conv_norm.restype = ctypes.c_int
    lib.kda_conv_norm.argtypes = [P(ConvNormArgs), _vp]
    lib.kda_validate_decode.restype = ctypes.c_int
    lib.kda_validate_decode.argtypes = [P(DecodeArgs)]
    lib.kda_decode_step.restype = ctypes.c_int
    lib.kda_decode_step.argtypes = [P(DecodeArgs), _vp]
    lib.kda_validate_backward.restype = ctypes.c_int
    lib.kda_validate_backward.argtypes = [P(BackwardArgs)]
    lib.kda_backward_workspace_bytes.restype = ctypes.c_size_t
    lib.kda_backward_workspace_bytes.argtypes = [P(BackwardArgs)]
    lib.kda_prefill_backward.restype = ctypes.c_int
    lib.kda_prefill_backward.argtypes = [P(BackwardArgs), _vp, ctypes.c_size_t, _vp]
    lib.kda_training_workspace_bytes.restype = ctypes.c_size_t
    lib.kda_training_workspace_bytes.argtypes = [P(PrefillArgs)]
    lib.kda_prefill_forward_saved.restype = ctypes.c_int
    lib.kda_prefill_forward_saved.argtypes = [P(PrefillArgs), _vp, ctypes.c_size_t, _vp]
    lib.kda_prefill_backward_saved.restype = ctypes.c_int
    lib.kda_prefill_backward_saved.argtypes = [P(BackwardArgs), _vp, ctypes.c_size_t, _vp]
    from . import _gdr
    _gdr.declare(lib)
    if lib.kda_abi_version() != ABI_VERSION:
        raise RuntimeError("libkda ABI version mismatch")
    if path is None:
        _lib = lib
    return lib


def _status_str(status: int) -> str:
    try:
        return load().kda_status_str(int(status)).decode()
    except Exception:  # pragma: no cover - library absent
        return "?"


def kda_abi_version() -> int:
    return int(load().kda_abi_version())


def kda_status_str(status: int) -> str:
    return load().kda_status_str(int(status)).decode()


# ------------------------------------------------------------------ marshalling
def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t or None
    if t.numel() == 0:
        return None
    if not t.is_contiguous():
        raise ValueError("libkda needs contiguous tensors")
    return t.data_ptr()


def _io_of(t) -> int:
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    if t.dtype == torch.float32:
        return KDA_FP32
    raise TypeError(f"unsupported dtype {t.dtype} (bfloat16 or float32)")


def _stream(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _check(status: int, where: str):
    if status != KDA_OK:
        raise KdaError(status, where)


def _flags(l2norm_qk: bool, beta_logits: bool) -> int:
    return (KDA_FLAG_L2NORM_QK if l2norm_qk else 0) | (KDA_FLAG_BETA_LOGITS if beta_logits else 0)


def _stages(a, A_log, dt_bias, o_norm_w, o_norm_eps, o_gate):
    a.A_log, a.dt_bias, a.o_norm_w, a.o_gate = _ptr(A_log), _ptr(dt_bias), _ptr(o_norm_w), _ptr(o_gate)
    a.o_norm_eps = o_norm_eps


def prefill_args(q, k, v, g, beta, conv_w=None, conv_state_in=None, S0=None, o=None, S_T=None,
                 conv_state_out=None, *, chunk=64, scale=1.0, l2norm_qk=True, eps=1e-6,
                 conv_k=None, B=None, T=None, H=None, D=None, io=None, A_log=None, dt_bias=None,
                 beta_logits=False, o_norm_w=None, o_norm_eps=1e-6, o_gate=None,
                 cu_seqlens=None) -> PrefillArgs:
    """Fill kda_prefill_args from tensors (shapes from q unless given explicitly)."""
    a = PrefillArgs()
    if q is not None and not isinstance(q, int):
        B0, T0, H0, D0 = q.shape
        io0 = _io_of(q)
    else:
        B0 = T0 = H0 = D0 = 0
        io0 = KDA_BF16
    a.B, a.T, a.H, a.D = (B0 if B is None else B, T0 if T is None else T,
                          H0 if H is None else H, D0 if D is None else D)
    a.chunk = chunk
    a.conv_k = (4 if conv_w is not None else 0) if conv_k is None else conv_k
    a.flags = _flags(l2norm_qk, beta_logits)
    a.l2_eps = eps
    a.scale = scale
    a.io = io0 if io is None else io
    a.q, a.k, a.v, a.g, a.beta = _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta)
    a.conv_w, a.conv_state_in, a.S0 = _ptr(conv_w), _ptr(conv_state_in), _ptr(S0)
    a.o, a.S_T, a.conv_state_out = _ptr(o), _ptr(S_T), _ptr(conv_state_out)
    _stages(a, A_log, dt_bias, o_norm_w, o_norm_eps, o_gate)
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int32:
            raise TypeError("cu_seqlens must be int32")
        a.cu_seqlens = _ptr(cu_seqlens)
        a.n_seqs = cu_seqlens.numel() - 1
    return a


def kda_validate_prefill(args: PrefillArgs) -> int:
    return int(load().kda_validate_prefill(ctypes.byref(args)))


def kda_prefill_workspace_bytes(args: PrefillArgs) -> int:
    return int(load().kda_prefill_workspace_bytes(ctypes.byref(args)))


def _workspace(args: PrefillArgs, device, workspace=None):
    need = kda_prefill_workspace_bytes(args)
    if workspace is not None:
        return workspace, need
    if need == 0:
        return None, 0
    return torch.empty(need, dtype=torch.uint8, device=device), need


def kda_prefill(q, k, v, g, beta, conv_w=None, conv_state=None, S0=None, *, chunk=64, scale=1.0,
                l2norm_qk=True, eps=1e-6, o=None, S_T=None, conv_state_out=None, workspace=None,
                stream=None, A_log=None, dt_bias=None, beta_logits=False, o_norm_w=None,
                o_norm_eps=1e-6, o_gate=None, cu_seqlens=None):
    """Whole-sequence KDA forward.  Returns (o, S_T, conv_state_out).

    q, k, v, g: [B, T, H, D] (bf16 or fp32, same dtype); beta [B, T, H];
    conv_w [3, H*D, 4] fp32 or None (no conv); conv_state [B, 3, 3, H*D] or None;
    S0 [B, H, D, D] fp32 or None.  Outputs are allocated unless given.
    Optional stages: A_log [H] and dt_bias [H*D] fp32 (g then holds the raw gate
    projection), beta_logits (beta holds logits), o_norm_w [D] fp32 and o_gate
    [B, T, H, D] for the output RMSNorm and sigmoid gate.
    Packed sequences: cu_seqlens int32 [N + 1] on the device with B = 1; then S0,
    S_T are [N, H, D, D] and the conv states [N, 3, 3, H*D].
    """
    B, T, H, D = q.shape
    dev = q.device
    NS = B if cu_seqlens is None else cu_seqlens.numel() - 1
    if o is None:
        o = torch.empty_like(q)
    if S_T is None:
        S_T = torch.empty(NS, H, D, D, dtype=torch.float32, device=dev)
    if conv_state_out is None and conv_w is not None:
        conv_state_out = torch.empty(NS, 3, 3, H * D, dtype=q.dtype, device=dev)
    a = prefill_args(q, k, v, g, beta, conv_w, conv_state, S0, o, S_T, conv_state_out, chunk=chunk,
                     scale=scale, l2norm_qk=l2norm_qk, eps=eps, A_log=A_log, dt_bias=dt_bias,
                     beta_logits=beta_logits, o_norm_w=o_norm_w, o_norm_eps=o_norm_eps,
                     o_gate=o_gate, cu_seqlens=cu_seqlens)
    _check(kda_validate_prefill(a), "kda_prefill")
    ws, need = _workspace(a, dev, workspace)
    _check(load().kda_prefill(ctypes.byref(a), _ptr(ws) if ws is not None else None, need if
                              workspace is None else workspace.numel(), _stream(stream)),
           "kda_prefill")
    return o, S_T, conv_state_out


def kda_prefill_walk_segments(args: PrefillArgs) -> int:
    """Segments the state walk of kda_prefill(args) is split into (1: not split;
    0: invalid arguments).  Host only."""
    return int(load().kda_prefill_walk_segments(ctypes.byref(args)))


def kda_prefill_state_map_workspace_bytes(args: PrefillArgs) -> int:
    return int(load().kda_prefill_state_map_workspace_bytes(ctypes.byref(args)))


def kda_prefill_state_map_raw(args: PrefillArgs, workspace, M, N, stream=None):
    """kda_prefill_state_map on a pre-filled argument struct whose preparation
    stage has run on `workspace` (no allocation)."""
    ws = _ptr(workspace) if workspace is not None else None
    nbytes = workspace.numel() if workspace is not None else 0
    _check(load().kda_prefill_state_map(ctypes.byref(args), ws, nbytes, _ptr(M), _ptr(N),
                                        _stream(stream)), "kda_prefill_state_map")


def kda_prefill_state_map(q, k, v, g, beta, conv_w=None, conv_state=None, *, chunk=64, scale=1.0,
                          l2norm_qk=True, eps=1e-6, A_log=None, dt_bias=None, beta_logits=False,
                          stream=None):
    """The affine state map of a prefill over these tokens: (M, N), each
    [B, H, D, D] fp32, with S_T = M S_start + N for any start state.  Runs the
    preparation stage, then the map (o and S_T of the arguments are allocated for
    the call but not written)."""
    B, T, H, D = q.shape
    dev = q.device
    o = torch.empty_like(q)
    S_T = torch.empty(B, H, D, D, dtype=torch.float32, device=dev)
    a = prefill_args(q, k, v, g, beta, conv_w, conv_state, None, o, S_T, None, chunk=chunk,
                     scale=scale, l2norm_qk=l2norm_qk, eps=eps, A_log=A_log, dt_bias=dt_bias,
                     beta_logits=beta_logits)
    _check(kda_validate_prefill(a), "kda_prefill_state_map")
    M = torch.empty(B, H, D, D, dtype=torch.float32, device=dev)
    N = torch.empty_like(M)
    need = kda_prefill_state_map_workspace_bytes(a)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need > 0 else None
    if T > 0:
        kda_prefill_stage(a, ws, 0, stream)
    kda_prefill_state_map_raw(a, ws, M, N, stream)
    return M, N


def kda_prefill_stage(args: PrefillArgs, workspace, stage: int, stream=None):
    """Enqueue one stage of kda_prefill (0 prep, 1 state walk, 2 conv hand-over,
    3 separate output-stage pass)."""
    ws = _ptr(workspace) if workspace is not None else None
    nbytes = workspace.numel() if workspace is not None else 0
    _check(load().kda_prefill_stage(ctypes.byref(args), ws, nbytes, int(stage), _stream(stream)),
           "kda_prefill_stage")


def kda_prefill_raw(args: PrefillArgs, workspace, stream=None):
    """kda_prefill on a pre-filled argument struct (no allocation)."""
    ws = _ptr(workspace) if workspace is not None else None
    nbytes = workspace.numel() if workspace is not None else 0
    _check(load().kda_prefill(ctypes.byref(args), ws, nbytes, _stream(stream)), "kda_prefill")


def kda_prefill_static_raw(args: PrefillArgs, stream=None) -> int:
    """kda_prefill_static on a pre-filled argument struct: the library's static
    per-GPU scratch is the workspace (nothing is allocated).  Returns the status
    (KDA_OK, or KDA_ERR_SCRATCH when the request does not fit)."""
    return int(load().kda_prefill_static(ctypes.byref(args), _stream(stream)))


def conv_norm_args(q, k, v, conv_w, conv_state_in=None, q_out=None, k_out=None, v_out=None,
                   conv_state_out=None, *, l2norm_qk=True, eps=1e-6) -> ConvNormArgs:
    a = ConvNormArgs()
    a.B, a.T, a.H, a.D = q.shape
    a.conv_k = 4
    a.flags = KDA_FLAG_L2NORM_QK if l2norm_qk else 0
    a.l2_eps = eps
    a.io = _io_of(q)
    a.q, a.k, a.v, a.conv_w, a.conv_state_in = (_ptr(q), _ptr(k), _ptr(v), _ptr(conv_w),
                                                _ptr(conv_state_in))
    a.q_out, a.k_out, a.v_out, a.conv_state_out = (_ptr(q_out), _ptr(k_out), _ptr(v_out),
                                                   _ptr(conv_state_out))
    return a


def kda_validate_conv_norm(args: ConvNormArgs) -> int:
    return int(load().kda_validate_conv_norm(ctypes.byref(args)))


def kda_conv_norm(q, k, v, conv_w, conv_state=None, *, l2norm_qk=True, eps=1e-6,
                  conv_state_out=None, stream=None):
    """Conv + SiLU (+ L2 for q, k) alone.  Returns (q_hat, k_hat, v_hat, conv_state_out)."""
    B, T, H, D = q.shape
    qo, ko, vo = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    if conv_state_out is None:
        conv_state_out = torch.empty(B, 3, 3, H * D, dtype=q.dtype, device=q.device)
    a = conv_norm_args(q, k, v, conv_w, conv_state, qo, ko, vo, conv_state_out,
                       l2norm_qk=l2norm_qk, eps=eps)
    _check(load().kda_conv_norm(ctypes.byref(a), _stream(stream)), "kda_conv_norm")
    return qo, ko, vo, conv_state_out


def decode_args(q, k, v, g, beta, S, o, conv_w=None, conv_state=None, *, scale=1.0,
                l2norm_qk=True, eps=1e-6, A_log=None, dt_bias=None, beta_logits=False,
                o_norm_w=None, o_norm_eps=1e-6, o_gate=None) -> DecodeArgs:
    a = DecodeArgs()
    a.B, a.H, a.D = q.shape
    a.conv_k = 4 if conv_w is not None else 0
    a.flags = _flags(l2norm_qk, beta_logits)
    a.l2_eps = eps
    a.scale = scale
    a.io = _io_of(q)
    a.q, a.k, a.v, a.g, a.beta = _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta)
    a.conv_w, a.conv_state, a.S, a.o = _ptr(conv_w), _ptr(conv_state), _ptr(S), _ptr(o)
    _stages(a, A_log, dt_bias, o_norm_w, o_norm_eps, o_gate)
    return a


def kda_validate_decode(args: DecodeArgs) -> int:
    return int(load().kda_validate_decode(ctypes.byref(args)))


def kda_decode_step(q, k, v, g, beta, S, conv_w=None, conv_state=None, *, scale=1.0,
                    l2norm_qk=True, eps=1e-6, o=None, stream=None, A_log=None, dt_bias=None,
                    beta_logits=False, o_norm_w=None, o_norm_eps=1e-6, o_gate=None):
    """One decode step; S [B,H,D,D] fp32 and conv_state [B,3,3,H*D] are updated in place.

    q, k, v, g: [B, H, D]; beta [B, H].  Returns o [B, H, D].  Optional stages as
    in kda_prefill (o_gate [B, H, D]).
    """
    if o is None:
        o = torch.empty_like(q)
    a = decode_args(q, k, v, g, beta, S, o, conv_w, conv_state, scale=scale, l2norm_qk=l2norm_qk,
                    eps=eps, A_log=A_log, dt_bias=dt_bias, beta_logits=beta_logits,
                    o_norm_w=o_norm_w, o_norm_eps=o_norm_eps, o_gate=o_gate)
    _check(load().kda_decode_step(ctypes.byref(a), _stream(stream)), "kda_decode_step")
    return o


def kda_decode_raw(args: DecodeArgs, stream=None):
    _check(load().kda_decode_step(ctypes.byref(args), _stream(stream)), "kda_decode_step")


# ------------------------------------------------------------------- backward
def backward_args(fwd: PrefillArgs, do, dS_T, grads: dict) -> BackwardArgs:
    a = BackwardArgs()
    a.fwd = fwd
    a.dO, a.dS_T = _ptr(do), _ptr(dS_T)
    for n in ("dq", "dk", "dv", "dg", "dbeta", "dS0", "dconv_w", "dconv_state", "dA_log", "ddt_bias",
              "do_norm_w", "do_gate"):
        setattr(a, n, _ptr(grads.get(n)))
    return a


def kda_validate_backward(args: BackwardArgs) -> int:
    return int(load().kda_validate_backward(ctypes.byref(args)))


def kda_backward_workspace_bytes(args: BackwardArgs) -> int:
    return int(load().kda_backward_workspace_bytes(ctypes.byref(args)))


def kda_prefill_backward(q, k, v, g, beta, conv_w=None, conv_state=None, S0=None, *, do,
                         dS_T=None, chunk=64, scale=1.0, l2norm_qk=True, eps=1e-6, workspace=None,
                         stream=None, A_log=None, dt_bias=None, beta_logits=False, o_norm_w=None,
                         o_norm_eps=1e-6, o_gate=None, cu_seqlens=None):
    """Gradients of L = <o, do> + <S_T, dS_T> (the forward is recomputed).

    Returns (grads, o, S_T): grads is a dict of float32 tensors dq, dk, dv, dg
    [B, T, H, D], dbeta [B, T, H], dS0 [B, H, D, D], with the convolution
    dconv_w [3, H*D, 4] and dconv_state [B, 3, 3, H*D], and with the optional
    stages (arguments as kda_prefill) dA_log [H] and ddt_bias [H*D] (dg is then
    the gradient of the raw gate projection), do_norm_w [D], do_gate [B, T, H, D];
    with beta_logits dbeta is the gradient of the logits.  Packed sequences
    (cu_seqlens as kda_prefill): dS_T, dS0 [N, H, D, D], dconv_state [N, 3, 3, H*D].
    """
    B, T, H, D = q.shape
    dev = q.device
    NS = B if cu_seqlens is None else cu_seqlens.numel() - 1
    f32 = dict(dtype=torch.float32, device=dev)
    o = torch.empty_like(q)
    S_T = torch.empty(NS, H, D, D, **f32)
    cso = torch.empty(NS, 3, 3, H * D, dtype=q.dtype, device=dev) if conv_w is not None else None
    fwd = prefill_args(q, k, v, g, beta, conv_w, conv_state, S0, o, S_T, cso, chunk=chunk,
                       scale=scale, l2norm_qk=l2norm_qk, eps=eps, A_log=A_log, dt_bias=dt_bias,
                       beta_logits=beta_logits, o_norm_w=o_norm_w, o_norm_eps=o_norm_eps,
                       o_gate=o_gate, cu_seqlens=cu_seqlens)
    grads = dict(dq=torch.empty(B, T, H, D, **f32), dk=torch.empty(B, T, H, D, **f32),
                 dv=torch.empty(B, T, H, D, **f32), dg=torch.empty(B, T, H, D, **f32),
                 dbeta=torch.empty(B, T, H, **f32), dS0=torch.empty(NS, H, D, D, **f32))
    if conv_w is not None:
        grads["dconv_w"] = torch.empty(3, H * D, 4, **f32)
        grads["dconv_state"] = torch.empty(NS, 3, 3, H * D, **f32)
    if A_log is not None:
        grads["dA_log"] = torch.empty(H, **f32)
        grads["ddt_bias"] = torch.empty(H * D, **f32)
    if o_norm_w is not None:
        grads["do_norm_w"] = torch.empty(D, **f32)
    if o_gate is not None:
        grads["do_gate"] = torch.empty(B, T, H, D, **f32)
    a = backward_args(fwd, do, dS_T, grads)
    _check(kda_validate_backward(a), "kda_prefill_backward")
    need = kda_backward_workspace_bytes(a)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    ws = _ptr(workspace) if workspace is not None else None
    nbytes = workspace.numel() if workspace is not None else 0
    _check(load().kda_prefill_backward(ctypes.byref(a), ws, nbytes, _stream(stream)),
           "kda_prefill_backward")
    return grads, o, S_T


def _grads_for(q, NS, conv, A_log, o_norm_w, o_gate):
    B, T, H, D = q.shape
    f32 = dict(dtype=torch.float32, device=q.device)
    grads = dict(dq=torch.empty(B, T, H, D, **f32), dk=torch.empty(B, T, H, D, **f32),
                 dv=torch.empty(B, T, H, D, **f32), dg=torch.empty(B, T, H, D, **f32),
                 dbeta=torch.empty(B, T, H, **f32), dS0=torch.empty(NS, H, D, D, **f32))
    if conv:
        grads["dconv_w"] = torch.empty(3, H * D, 4, **f32)
        grads["dconv_state"] = torch.empty(NS, 3, 3, H * D, **f32)
    if A_log is not None:
        grads["dA_log"] = torch.empty(H, **f32)
        grads["ddt_bias"] = torch.empty(H * D, **f32)
    if o_norm_w is not None:
        grads["do_norm_w"] = torch.empty(D, **f32)
    if o_gate is not None:
        grads["do_gate"] = torch.empty(B, T, H, D, **f32)
    return grads


def kda_training_workspace_bytes(args: PrefillArgs) -> int:
    return int(load().kda_training_workspace_bytes(ctypes.byref(args)))


def kda_prefill_forward_saved_raw(args: PrefillArgs, workspace, stream=None):
    ws = _ptr(workspace) if workspace is not None else None
    nbytes = workspace.numel() if workspace is not None else 0
    _check(load().kda_prefill_forward_saved(ctypes.byref(args), ws, nbytes, _stream(stream)),
           "kda_prefill_forward_saved")


def kda_prefill_backward_saved_raw(args: BackwardArgs, workspace, stream=None):
    ws = _ptr(workspace) if workspace is not None else None
    nbytes = workspace.numel() if workspace is not None else 0
    _check(load().kda_prefill_backward_saved(ctypes.byref(args), ws, nbytes, _stream(stream)),
           "kda_prefill_backward_saved")


class SavedForward:
    """What kda_prefill_forward_saved hands to kda_prefill_backward_saved: the
    forward's argument struct, its workspace, and the tensors both refer to."""

    def __init__(self, args, workspace, keep, NS, conv, stages):
        self.args, self.workspace, self.keep = args, workspace, keep
        self.NS, self.conv, self.stages = NS, conv, stages


def kda_prefill_forward_saved(q, k, v, g, beta, conv_w=None, conv_state=None, S0=None, *, chunk=64,
                              scale=1.0, l2norm_qk=True, eps=1e-6, stream=None, A_log=None,
                              dt_bias=None, beta_logits=False, o_norm_w=None, o_norm_eps=1e-6,
                              o_gate=None, cu_seqlens=None):
    """The forward of a training step, kept for its backward: returns (o, S_T,
    conv_state_out, saved), the outputs as kda_prefill's and `saved` for
    kda_prefill_backward_saved (the inputs must not change in between)."""
    B, T, H, D = q.shape
    dev = q.device
    NS = B if cu_seqlens is None else cu_seqlens.numel() - 1
    o = torch.empty_like(q)
    S_T = torch.empty(NS, H, D, D, dtype=torch.float32, device=dev)
    cso = torch.empty(NS, 3, 3, H * D, dtype=q.dtype, device=dev) if conv_w is not None else None
    a = prefill_args(q, k, v, g, beta, conv_w, conv_state, S0, o, S_T, cso, chunk=chunk,
                     scale=scale, l2norm_qk=l2norm_qk, eps=eps, A_log=A_log, dt_bias=dt_bias,
                     beta_logits=beta_logits, o_norm_w=o_norm_w, o_norm_eps=o_norm_eps,
                     o_gate=o_gate, cu_seqlens=cu_seqlens)
    _check(kda_validate_prefill(a), "kda_prefill_forward_saved")
    need = kda_training_workspace_bytes(a)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need > 0 else None
    kda_prefill_forward_saved_raw(a, ws, stream)
    keep = (q, k, v, g, beta, conv_w, conv_state, S0, o, S_T, cso, A_log, dt_bias, o_norm_w, o_gate,
            cu_seqlens)
    saved = SavedForward(a, ws, keep, NS, conv_w is not None, (A_log, o_norm_w, o_gate))
    return o, S_T, cso, saved


def kda_prefill_backward_saved(saved: SavedForward, *, do, dS_T=None, stream=None) -> dict:
    """The backward of a kda_prefill_forward_saved call, without recomputing the
    forward.  Returns the gradients as kda_prefill_backward does."""
    q = saved.keep[0]
    A_log, o_norm_w, o_gate = saved.stages
    grads = _grads_for(q, saved.NS, saved.conv, A_log, o_norm_w, o_gate)
    a = backward_args(saved.args, do, dS_T, grads)
    _check(kda_validate_backward(a), "kda_prefill_backward_saved")
    kda_prefill_backward_saved_raw(a, saved.workspace, stream)
    return grads


def kda_prefill_backward_raw(args: BackwardArgs, workspace, stream=None):
    ws = _ptr(workspace) if workspace is not None else None
    nbytes = workspace.numel() if workspace is not None else 0
    _check(load().kda_prefill_backward(ctypes.byref(args), ws, nbytes, _stream(stream)),
           "kda_prefill_backward")
