"""ctypes binding of the gated delta rule with one decay per head and of the page
operations (include/kda.h): argument marshalling only, as in ``_lib``.

Shapes, types and devices are checked here, since the C side sees addresses only;
everything else is the library's own validation.  q, k and v may be views into
wider rows (one fused projection): the last two dimensions dense, a constant
stride between tokens.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib

_vp = ctypes.c_void_p
_i32, _i64, _u32, _f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_float


class GdrArgs(ctypes.Structure):
    _fields_ = [("B", _i32), ("T", _i32), ("Hk", _i32), ("Hv", _i32), ("Dk", _i32), ("Dv", _i32),
                ("flags", _u32), ("l2_eps", _f32), ("scale", _f32), ("io", _i32),
                ("q_stride", _i64), ("k_stride", _i64), ("v_stride", _i64),
                ("q", _vp), ("k", _vp), ("v", _vp), ("g", _vp), ("beta", _vp), ("S0", _vp),
                ("o", _vp), ("S_T", _vp), ("A_log", _vp), ("dt_bias", _vp), ("cu_seqlens", _vp),
                ("n_seqs", _i32)]


class GdrBackwardArgs(ctypes.Structure):
    _fields_ = [("fwd", GdrArgs), ("dO", _vp), ("dS_T", _vp), ("dq", _vp), ("dk", _vp),
                ("dv", _vp), ("dg", _vp), ("dbeta", _vp), ("dS0", _vp), ("dA_log", _vp),
                ("ddt_bias", _vp)]


class GdrDecodeArgs(ctypes.Structure):
    _fields_ = [("N", _i32), ("n_slots", _i32), ("Hk", _i32), ("Hv", _i32), ("Dk", _i32),
                ("Dv", _i32), ("flags", _u32), ("l2_eps", _f32), ("scale", _f32), ("io", _i32),
                ("q_stride", _i64), ("k_stride", _i64), ("v_stride", _i64),
                ("q", _vp), ("k", _vp), ("v", _vp), ("g", _vp), ("beta", _vp), ("A_log", _vp),
                ("dt_bias", _vp), ("S", _vp), ("slots", _vp), ("o", _vp)]


class PagesPool(ctypes.Structure):
    _fields_ = [("data", _vp), ("layer_stride", _i64), ("page_bytes", _i64), ("n_layers", _i32),
                ("n_pages", _i32)]


def declare(lib):
    P = ctypes.POINTER
    size = ctypes.c_size_t
    for name, args, ret in [
            ("kda_validate_gdr_prefill", [P(GdrArgs)], ctypes.c_int),
            ("kda_gdr_prefill_workspace_bytes", [P(GdrArgs)], size),
            ("kda_gdr_prefill", [P(GdrArgs), _vp, size, _vp], ctypes.c_int),
            ("kda_validate_gdr_backward", [P(GdrBackwardArgs)], ctypes.c_int),
            ("kda_gdr_backward_workspace_bytes", [P(GdrBackwardArgs)], size),
            ("kda_gdr_prefill_backward", [P(GdrBackwardArgs), _vp, size, _vp], ctypes.c_int),
            ("kda_validate_gdr_decode", [P(GdrDecodeArgs)], ctypes.c_int),
            ("kda_gdr_decode", [P(GdrDecodeArgs), _vp], ctypes.c_int),
            ("kda_pages_workspace_bytes", [P(PagesPool), _i32], size),
            ("kda_pages_fork", [P(PagesPool), _vp, _vp, _vp, _vp, _i32, _vp, size, _vp], ctypes.c_int),
            ("kda_pages_free", [_vp, _vp, _i32, _vp, _i32, _vp], ctypes.c_int),
            ("kda_pages_compact", [P(PagesPool), _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp, size, _vp],
             ctypes.c_int),
            ("kda_pages_copy", [P(PagesPool), P(PagesPool), _vp, _vp, _vp, _i32, _vp, size, _vp],
             ctypes.c_int)]:
        f = getattr(lib, name)
        f.argtypes, f.restype = args, ret


# ------------------------------------------------------------------ helpers
# A call on a small model is a few microseconds of GPU time, so the checks below are
# plain comparisons and only a failing one formats anything; devices go by their index
# (get_device: -1 is the host).
def _wrong(name, t, shape, dtype, device):
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype}, expected {dtype}")
    raise ValueError(f"{name} is on {t.device}, expected {_name(device)}")


def _name(device):
    return "cpu" if device < 0 else f"cuda:{device}"


def _dense(t, name, shape, dtype, device):
    """Address of a contiguous tensor of this shape, type and device (None stays None)."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device:
        _wrong(name, t, shape, dtype, device)
    if not t.is_contiguous():
        raise ValueError(f"{name}: libkda needs contiguous tensors")
    return t.data_ptr() or None


def _rows(t, name, shape, dtype, device):
    """(address, elements between tokens; 0 = packed) of [B, T, H, D] or [N, H, D]."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != device:
        _wrong(name, t, shape, dtype, device)
    if t.is_contiguous():
        return t.data_ptr() or None, 0
    st = t.stride()
    if (shape[-1] > 1 and st[-1] != 1) or (shape[-2] > 1 and st[-2] != shape[-1]):
        raise ValueError(f"{name}: the last two dimensions must be dense")
    lead = shape[:-2]
    step = st[len(lead) - 1]
    if len(lead) == 2:
        if lead[1] == 1:
            step = st[0]
        elif lead[0] > 1 and st[0] != lead[1] * st[1]:
            raise ValueError(f"{name}: rows of the batch must follow one another")
    if lead.numel() == 1:
        step = 0
    elif step < shape[-2] * shape[-1]:  # an expanded view, say
        raise ValueError(f"{name}: the rows of two tokens overlap")
    return t.data_ptr(), step


def _elsewhere(t):
    """The context that makes t's device current; None if it is."""
    d = t.get_device()
    if d < 0:
        raise ValueError(f"libkda works on GPU tensors, not on {t.device}")
    if d == torch.cuda.current_device():
        return None
    return torch.cuda.device(d)


# the current stream's handle without making a Stream object of it (2 us)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _handle(stream, device):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(device)
        return torch.cuda.current_stream(device).cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _made(stream, device, *tensors):
    """Tensors made here on the current stream for a call on the caller's own: that
    stream waits for what the current one still does (with their memory, or filling
    them), and torch keeps the memory until that stream is done with it."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
    current = torch.cuda.current_stream(device)
    if stream == current:
        return
    stream.wait_stream(current)
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def _scratch(need, device, stream, own):
    """(address, bytes) of the workspace, and what keeps it."""
    if own is not None:
        if own.get_device() != device:
            raise ValueError(f"workspace is on {own.device}, expected {_name(device)}")
        return (_lib._ptr(own), own.numel() * own.element_size()), own
    if need == 0:
        return (None, 0), None
    ws = torch.empty(need, dtype=torch.uint8, device=device)
    if stream is not None:
        _made(stream, device, ws)
    return (ws.data_ptr(), need), ws


def _ws(ws):
    return (None, 0) if ws is None else (_lib._ptr(ws), ws.numel() * ws.element_size())


def _list(t, name, device):
    """Address of an int32 list on the device."""
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, expected {_name(device)}")
    return _lib._ptr(t)


def _sequences(cu_seqlens):
    if cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens needs an offset before and one after every sequence")
    return cu_seqlens.numel() - 1


# ------------------------------------------------------------------ prefill
def gdr_args(q, k, v, g, beta, S0=None, o=None, S_T=None, *, scale=1.0, l2norm_qk=True, eps=1e-6,
             A_log=None, dt_bias=None, beta_logits=False, cu_seqlens=None) -> GdrArgs:
    """Fill kda_gdr_args from tensors (shapes as kda_gdr_prefill)."""
    qs, vs = q.shape, v.shape
    B, T, Hk, Dk = qs
    Hv, Dv = vs[2:]
    io, dev, f32 = q.dtype, q.get_device(), torch.float32
    gates = (B, T, Hv)
    cu, n, NS = None, 0, B
    if cu_seqlens is not None:
        cu, NS = _list(cu_seqlens, "cu_seqlens", dev), _sequences(cu_seqlens)
        n = NS
    state = (NS, Hv, Dk, Dv)
    pq, sq = _rows(q, "q", qs, io, dev)
    pk, sk = _rows(k, "k", qs, io, dev)
    pv, sv = _rows(v, "v", torch.Size((B, T, Hv, Dv)), io, dev)
    return GdrArgs(B, T, Hk, Hv, Dk, Dv, _lib._flags(l2norm_qk, beta_logits), eps, scale, _lib._io_of(q),
                   sq, sk, sv, pq, pk, pv, _dense(g, "g", gates, io, dev), _dense(beta, "beta", gates, io, dev),
                   _dense(S0, "S0", state, f32, dev), _dense(o, "o", vs, io, dev),
                   _dense(S_T, "S_T", state, f32, dev), _dense(A_log, "A_log", (Hv,), f32, dev),
                   _dense(dt_bias, "dt_bias", (Hv,), f32, dev), cu, n)


def kda_validate_gdr_prefill(args: GdrArgs) -> int:
    return int(_lib.load().kda_validate_gdr_prefill(ctypes.byref(args)))


def kda_gdr_prefill_workspace_bytes(args: GdrArgs) -> int:
    return int(_lib.load().kda_gdr_prefill_workspace_bytes(ctypes.byref(args)))


def kda_gdr_prefill_raw(args: GdrArgs, workspace, stream=None):
    """kda_gdr_prefill on a pre-filled argument struct (no allocation)."""
    _lib._check(_lib.load().kda_gdr_prefill(ctypes.byref(args), *_ws(workspace), _lib._stream(stream)),
                "kda_gdr_prefill")


def kda_gdr_prefill(q, k, v, g, beta, S0=None, *, scale=1.0, l2norm_qk=True, eps=1e-6, A_log=None,
                    dt_bias=None, beta_logits=False, cu_seqlens=None, o=None, S_T=None,
                    workspace=None, stream=None):
    """Whole-sequence forward of the gated delta rule with one decay per head.
    Returns (o, S_T).

    q, k: [B, T, Hk, Dk]; v: [B, T, Hv, Dv] (Hv a multiple of Hk: value head h uses
    key head h // (Hv // Hk)); g, beta: [B, T, Hv], all bf16 or all fp32; S0
    [B, Hv, Dk, Dv] fp32 or None.  Outputs are allocated unless given; S_T may be
    S0.  A_log, dt_bias [Hv] fp32: g holds the raw decay projection; beta_logits:
    beta holds logits.  Packed sequences: cu_seqlens int32 [N + 1] on the device
    with B = 1; then S0, S_T are [N, Hv, Dk, Dv].
    """
    away = _elsewhere(q)
    if away is not None:
        with away:
            return kda_gdr_prefill(q, k, v, g, beta, S0, scale=scale, l2norm_qk=l2norm_qk, eps=eps, A_log=A_log,
                                   dt_bias=dt_bias, beta_logits=beta_logits, cu_seqlens=cu_seqlens, o=o, S_T=S_T,
                                   workspace=workspace, stream=stream)
    dev = q.get_device()
    if o is None:
        o = torch.empty(v.shape, dtype=q.dtype, device=dev)
        if stream is not None:
            _made(stream, dev, o)
    if S_T is None:
        NS = q.shape[0] if cu_seqlens is None else _sequences(cu_seqlens)
        S_T = torch.empty(NS, v.shape[2], q.shape[3], v.shape[3], dtype=torch.float32, device=dev)
        if stream is not None:
            _made(stream, dev, S_T)
    a = ctypes.byref(gdr_args(q, k, v, g, beta, S0, o, S_T, scale=scale, l2norm_qk=l2norm_qk, eps=eps,
                              A_log=A_log, dt_bias=dt_bias, beta_logits=beta_logits, cu_seqlens=cu_seqlens))
    lib = _lib.load()
    ws, keep = _scratch(lib.kda_gdr_prefill_workspace_bytes(a), dev, stream, workspace)
    status = lib.kda_gdr_prefill(a, *ws, _handle(stream, dev))
    if status:
        _lib._check(status, "kda_gdr_prefill")
    return o, S_T


# ------------------------------------------------------------------ backward
_GRADS = ("dq", "dk", "dv", "dg", "dbeta", "dS0", "dA_log", "ddt_bias")


def gdr_backward_args(fwd: GdrArgs, do, dS_T, grads: dict) -> GdrBackwardArgs:
    """Fill kda_gdr_backward_args (grads: the outputs by name)."""
    return GdrBackwardArgs(fwd, _lib._ptr(do), _lib._ptr(dS_T), *(_lib._ptr(grads.get(n)) for n in _GRADS))


def kda_validate_gdr_backward(args: GdrBackwardArgs) -> int:
    return int(_lib.load().kda_validate_gdr_backward(ctypes.byref(args)))


def kda_gdr_backward_workspace_bytes(args: GdrBackwardArgs) -> int:
    return int(_lib.load().kda_gdr_backward_workspace_bytes(ctypes.byref(args)))


def kda_gdr_prefill_backward_raw(args: GdrBackwardArgs, workspace, stream=None):
    """kda_gdr_prefill_backward on a pre-filled argument struct (no allocation)."""
    _lib._check(_lib.load().kda_gdr_prefill_backward(ctypes.byref(args), *_ws(workspace),
                                                     _lib._stream(stream)), "kda_gdr_prefill_backward")


def kda_gdr_prefill_backward(q, k, v, g, beta, S0=None, *, do, dS_T=None, scale=1.0, l2norm_qk=True,
                             eps=1e-6, A_log=None, dt_bias=None, beta_logits=False, cu_seqlens=None,
                             workspace=None, stream=None) -> dict:
    """Gradients of L = <o, do> + <S_T, dS_T> (arguments as kda_gdr_prefill; the
    forward is recomputed): dq, dk [B, T, Hk, Dk], dv [B, T, Hv, Dv], dg, dbeta
    [B, T, Hv] in the inputs' type, dS0 fp32, and with A_log the fp32 dA_log and
    ddt_bias [Hv] (dg and dbeta are then those of the raw projection and logits).
    Tokens outside every packed sequence get zero gradients."""
    away = _elsewhere(q)
    if away is not None:
        with away:
            return kda_gdr_prefill_backward(q, k, v, g, beta, S0, do=do, dS_T=dS_T, scale=scale, l2norm_qk=l2norm_qk,
                                            eps=eps, A_log=A_log, dt_bias=dt_bias, beta_logits=beta_logits,
                                            cu_seqlens=cu_seqlens, workspace=workspace, stream=stream)
    dev, io = q.get_device(), q.dtype
    B, T, Hk, Dk = q.shape
    Hv, Dv = v.shape[2:]
    NS = B if cu_seqlens is None else _sequences(cu_seqlens)
    fwd = gdr_args(q, k, v, g, beta, S0, None, None, scale=scale, l2norm_qk=l2norm_qk, eps=eps, A_log=A_log,
                   dt_bias=dt_bias, beta_logits=beta_logits, cu_seqlens=cu_seqlens)
    if cu_seqlens is None:
        new = torch.empty
    else:  # packed offsets may leave tokens out: those gradients are not written
        new = torch.zeros
    grads = dict(dq=new(B, T, Hk, Dk, dtype=io, device=dev), dk=new(B, T, Hk, Dk, dtype=io, device=dev),
                 dv=new(B, T, Hv, Dv, dtype=io, device=dev), dg=new(B, T, Hv, dtype=io, device=dev),
                 dbeta=new(B, T, Hv, dtype=io, device=dev),
                 dS0=torch.empty(NS, Hv, Dk, Dv, dtype=torch.float32, device=dev))
    if A_log is not None:
        grads["dA_log"] = torch.empty(Hv, dtype=torch.float32, device=dev)
        grads["ddt_bias"] = torch.empty(Hv, dtype=torch.float32, device=dev)
    if stream is not None:
        _made(stream, dev, *grads.values())
    a = GdrBackwardArgs(fwd, _dense(do, "do", v.shape, io, dev),
                        _dense(dS_T, "dS_T", (NS, Hv, Dk, Dv), torch.float32, dev),
                        *(_lib._ptr(grads.get(n)) for n in _GRADS))
    lib = _lib.load()
    r = ctypes.byref(a)
    _lib._check(lib.kda_validate_gdr_backward(r), "kda_gdr_prefill_backward")
    ws, keep = _scratch(lib.kda_gdr_backward_workspace_bytes(r), dev, stream, workspace)
    _lib._check(lib.kda_gdr_prefill_backward(r, *ws, _handle(stream, dev)), "kda_gdr_prefill_backward")
    return grads


# ------------------------------------------------------------------ decode
def gdr_decode_args(q, k, v, g, beta, S, slots=None, o=None, *, scale=1.0, l2norm_qk=True, eps=1e-6,
                    A_log=None, dt_bias=None, beta_logits=False) -> GdrDecodeArgs:
    """Fill kda_gdr_decode_args from tensors (shapes as kda_gdr_decode)."""
    qs, vs = q.shape, v.shape
    N, Hk, Dk = qs
    Hv, Dv = vs[1:]
    io, dev, f32 = q.dtype, q.get_device(), torch.float32
    at = None
    if slots is not None:
        if slots.shape != (N,):
            raise ValueError(f"slots has shape {tuple(slots.shape)}, expected {(N,)}")
        at = _list(slots, "slots", dev)
    pq, sq = _rows(q, "q", qs, io, dev)
    pk, sk = _rows(k, "k", qs, io, dev)
    pv, sv = _rows(v, "v", torch.Size((N, Hv, Dv)), io, dev)
    n = S.shape[0]
    return GdrDecodeArgs(N, n, Hk, Hv, Dk, Dv, _lib._flags(l2norm_qk, beta_logits), eps, scale, _lib._io_of(q),
                         sq, sk, sv, pq, pk, pv, _dense(g, "g", (N, Hv), io, dev),
                         _dense(beta, "beta", (N, Hv), io, dev), _dense(A_log, "A_log", (Hv,), f32, dev),
                         _dense(dt_bias, "dt_bias", (Hv,), f32, dev), _dense(S, "S", (n, Hv, Dk, Dv), f32, dev),
                         at, _dense(o, "o", vs, io, dev))


def kda_validate_gdr_decode(args: GdrDecodeArgs) -> int:
    return int(_lib.load().kda_validate_gdr_decode(ctypes.byref(args)))


def kda_gdr_decode_raw(args: GdrDecodeArgs, stream=None):
    """kda_gdr_decode on a pre-filled argument struct."""
    _lib._check(_lib.load().kda_gdr_decode(ctypes.byref(args), _lib._stream(stream)), "kda_gdr_decode")


def kda_gdr_decode(q, k, v, g, beta, S, slots=None, *, scale=1.0, l2norm_qk=True, eps=1e-6, A_log=None,
                   dt_bias=None, beta_logits=False, o=None, stream=None):
    """Single tokens on a pool of states S [n_slots, Hv, Dk, Dv] fp32, updated in
    place; row i belongs to slots[i] (int32; outside the pool: a padding row, whose
    o is left as it was -- zeros if o is allocated here).  Rows with one slot are
    consecutive tokens of its sequence.  q, k [N, Hk, Dk], v [N, Hv, Dv], g, beta
    [N, Hv].  Returns o [N, Hv, Dv]."""
    away = _elsewhere(q)
    if away is not None:
        with away:
            return kda_gdr_decode(q, k, v, g, beta, S, slots, scale=scale, l2norm_qk=l2norm_qk, eps=eps, A_log=A_log,
                                  dt_bias=dt_bias, beta_logits=beta_logits, o=o, stream=stream)
    dev = q.get_device()
    if o is None:
        o = (torch.empty if slots is None else torch.zeros)(v.shape, dtype=q.dtype, device=dev)
        if stream is not None:
            _made(stream, dev, o)
    a = gdr_decode_args(q, k, v, g, beta, S, slots, o, scale=scale, l2norm_qk=l2norm_qk, eps=eps, A_log=A_log,
                        dt_bias=dt_bias, beta_logits=beta_logits)
    status = _lib.load().kda_gdr_decode(ctypes.byref(a), _handle(stream, dev))
    if status:
        _lib._check(status, "kda_gdr_decode")
    return o


# ------------------------------------------------------------------ pages
def pages_pool(pool) -> PagesPool:
    """kda_pages_pool of a tensor [layers, pages, ...] whose pages are dense (the
    layers may be further apart)."""
    if pool.dim() < 3:
        raise ValueError("a pool is [layers, pages, ...]")
    shape, es, layer = pool.shape, pool.element_size(), 0
    page = shape[2:].numel()
    if not pool.is_contiguous():
        if not pool[0, 0].is_contiguous() or (shape[1] > 1 and pool.stride(1) != page):
            raise ValueError("the pages of a layer must be dense")
        if shape[0] > 1 and pool.stride(0) < shape[1] * page:
            raise ValueError("two layers overlap")
        layer = pool.stride(0) * es if shape[0] > 1 else 0
    return PagesPool(pool.data_ptr(), layer, page * es, shape[0], shape[1])


def kda_pages_workspace_bytes(pool: PagesPool, n: int) -> int:
    return int(_lib.load().kda_pages_workspace_bytes(ctypes.byref(pool), n))


def kda_pages_fork(pool, refs, src, *, refs_out=None, dst=None, workspace=None, stream=None):
    """Forks pages of `pool` [layers, pages, ...]: request i gets the next free page
    (refs[p] <= 0), filled from page src[i] (zeros where -1).  Returns (dst, refs_out):
    the pages (-1 where a request could not be met) and the new counts."""
    away = _elsewhere(pool)
    if away is not None:
        with away:
            return kda_pages_fork(pool, refs, src, refs_out=refs_out, dst=dst, workspace=workspace, stream=stream)
    dev, i32 = pool.get_device(), torch.int32
    p = pages_pool(pool)
    n, pages = src.numel(), (p.n_pages,)
    if refs_out is None:
        refs_out = torch.empty(pages, dtype=i32, device=dev)
        if stream is not None:
            _made(stream, dev, refs_out)
    if dst is None:
        dst = torch.empty(n, dtype=i32, device=dev)
        if stream is not None:
            _made(stream, dev, dst)
    r, lib = ctypes.byref(p), _lib.load()
    ws, keep = _scratch(lib.kda_pages_workspace_bytes(r, n), dev, stream, workspace)
    _lib._check(lib.kda_pages_fork(r, _dense(refs, "refs", pages, i32, dev),
                                   _dense(refs_out, "refs_out", pages, i32, dev), _list(src, "src", dev),
                                   _dense(dst, "dst", (n,), i32, dev), n, *ws, _handle(stream, dev)),
                "kda_pages_fork")
    return dst, refs_out


def kda_pages_free(refs, pages, *, refs_out=None, stream=None):
    """Lowers the count of every listed page (once for each time it is listed, not
    below 0).  Returns refs_out."""
    away = _elsewhere(refs)
    if away is not None:
        with away:
            return kda_pages_free(refs, pages, refs_out=refs_out, stream=stream)
    dev, i32, shape = refs.get_device(), torch.int32, (refs.numel(),)
    if refs_out is None:
        refs_out = torch.empty(shape, dtype=i32, device=dev)
        if stream is not None:
            _made(stream, dev, refs_out)
    _lib._check(_lib.load().kda_pages_free(_dense(refs, "refs", shape, i32, dev),
                                           _dense(refs_out, "refs_out", shape, i32, dev), shape[0],
                                           _list(pages, "pages", dev), pages.numel(), _handle(stream, dev)),
                "kda_pages_free")
    return refs_out


def kda_pages_compact(pool, refs, table=None, *, refs_out=None, new_id=None, table_out=None,
                      workspace=None, stream=None):
    """Moves the pages in use to the front of the pool.  Returns (n_used [1],
    new_id, refs_out, table_out): the new index of every page (-1: free), the new
    counts, and the table's entries renamed (None without a table)."""
    away = _elsewhere(pool)
    if away is not None:
        with away:
            return kda_pages_compact(pool, refs, table, refs_out=refs_out, new_id=new_id, table_out=table_out,
                                     workspace=workspace, stream=stream)
    dev, i32 = pool.get_device(), torch.int32
    p = pages_pool(pool)
    pages = (p.n_pages,)
    if refs_out is None:
        refs_out = torch.empty(pages, dtype=i32, device=dev)
    if new_id is None:
        new_id = torch.empty(pages, dtype=i32, device=dev)
    n_used = torch.empty(1, dtype=i32, device=dev)
    n, tab = 0, None
    if table is not None:
        n, tab = table.numel(), _list(table, "table", dev)
        if table_out is None:
            table_out = torch.empty(table.shape, dtype=i32, device=dev)
    else:
        table_out = None
    if stream is not None:
        _made(stream, dev, refs_out, new_id, n_used, table_out)
    r, lib = ctypes.byref(p), _lib.load()
    ws, keep = _scratch(lib.kda_pages_workspace_bytes(r, 0), dev, stream, workspace)
    _lib._check(lib.kda_pages_compact(
        r, _dense(refs, "refs", pages, i32, dev), _dense(refs_out, "refs_out", pages, i32, dev),
        _dense(new_id, "new_id", pages, i32, dev), n_used.data_ptr(), tab,
        _dense(table_out, "table_out", table.shape if table is not None else (), i32, dev), n, *ws,
        _handle(stream, dev)), "kda_pages_compact")
    return n_used, new_id, refs_out, table_out


def kda_pages_copy(src_pool, dst_pool, src, dst, *, done=None, workspace=None, stream=None):
    """Copies page src[i] of src_pool to page dst[i] of dst_pool (zeros where src[i]
    is -1) in every layer.  Returns done [n]: 1 where the pair was copied, 0 where it
    was left out (include/kda.h says which)."""
    away = _elsewhere(dst_pool)
    if away is not None:
        with away:
            return kda_pages_copy(src_pool, dst_pool, src, dst, done=done, workspace=workspace, stream=stream)
    dev = dst_pool.get_device()
    if src_pool.get_device() != dev:
        raise ValueError("both pools must be on one device")
    ps, pd = pages_pool(src_pool), pages_pool(dst_pool)
    n = src.numel()
    if dst.numel() != n:
        raise ValueError("src and dst differ in length")
    if done is None:
        done = torch.empty(n, dtype=torch.int32, device=dev)
        if stream is not None:
            _made(stream, dev, done)
    lib = _lib.load()
    ws, keep = _scratch(lib.kda_pages_workspace_bytes(ctypes.byref(pd), n), dev, stream, workspace)
    _lib._check(lib.kda_pages_copy(ctypes.byref(ps), ctypes.byref(pd), _list(src, "src", dev), _list(dst, "dst", dev),
                                   _dense(done, "done", (n,), torch.int32, dev), n, *ws, _handle(stream, dev)),
                "kda_pages_copy")
    return done
