"""ctypes binding of the gated delta rule with one decay per head and of the page
operations (include/kda.h): argument marshalling only, as in ``_lib``.

Shapes, types and devices are checked here, since the C side sees addresses only;
everything else is the library's own validation.  q, k and v may be views into
wider rows (one fused projection): the last two dimensions dense, a constant
stride between tokens.
"""
from __future__ import annotations

import contextlib
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
def _expect(t, name, shape, dtype, device):
    if t is None:
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _rows(t, name):
    """(address, elements between tokens; 0 = packed) of [B, T, H, D] or [N, H, D]."""
    if t.numel() == 0:
        return None, 0
    if t.is_contiguous():
        return t.data_ptr(), 0
    H, D = t.shape[-2:]
    lead, st = t.shape[:-2], t.stride()
    if (D > 1 and st[-1] != 1) or (H > 1 and st[-2] != D):
        raise ValueError(f"{name}: the last two dimensions must be dense")
    step = st[len(lead) - 1]
    if len(lead) == 2:
        if lead[1] == 1:
            step = st[0]
        elif lead[0] > 1 and st[0] != lead[1] * st[1]:
            raise ValueError(f"{name}: rows of the batch must follow one another")
    if lead.numel() == 1:
        step = 0
    return t.data_ptr(), step


def _device(t):
    """The context that makes t's device current, if it is not."""
    if t.device.type != "cuda" or t.device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(t.device)


def _stream(stream, device):
    return torch.cuda.current_stream(device) if stream is None else stream


def _handle(stream):
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _scratch(need, device, stream, own):
    """A workspace of `need` bytes; where the call runs on another stream than the
    one torch allocates for, torch keeps the memory until that stream is done."""
    if own is not None or need == 0:
        return own
    ws = torch.empty(need, dtype=torch.uint8, device=device)
    _used(stream, ws)
    return ws


def _used(stream, *tensors):
    if isinstance(stream, torch.cuda.Stream) and stream != torch.cuda.current_stream(stream.device):
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _ws(ws):
    return (None, 0) if ws is None else (_lib._ptr(ws), ws.numel() * ws.element_size())


def _int32(t, name, device):
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return _lib._ptr(t)


# ------------------------------------------------------------------ prefill
def gdr_args(q, k, v, g, beta, S0=None, o=None, S_T=None, *, scale=1.0, l2norm_qk=True, eps=1e-6,
             A_log=None, dt_bias=None, beta_logits=False, cu_seqlens=None) -> GdrArgs:
    """Fill kda_gdr_args from tensors (shapes as kda_gdr_prefill)."""
    B, T, Hk, Dk = q.shape
    Hv, Dv = v.shape[2:]
    io, dev = q.dtype, q.device
    a = GdrArgs()
    a.io = _lib._io_of(q)
    _expect(k, "k", (B, T, Hk, Dk), io, dev)
    _expect(v, "v", (B, T, Hv, Dv), io, dev)
    _expect(g, "g", (B, T, Hv), io, dev)
    _expect(beta, "beta", (B, T, Hv), io, dev)
    NS = B if cu_seqlens is None else cu_seqlens.numel() - 1
    _expect(S0, "S0", (NS, Hv, Dk, Dv), torch.float32, dev)
    _expect(S_T, "S_T", (NS, Hv, Dk, Dv), torch.float32, dev)
    _expect(o, "o", (B, T, Hv, Dv), io, dev)
    _expect(A_log, "A_log", (Hv,), torch.float32, dev)
    _expect(dt_bias, "dt_bias", (Hv,), torch.float32, dev)
    a.B, a.T, a.Hk, a.Hv, a.Dk, a.Dv = B, T, Hk, Hv, Dk, Dv
    a.flags = _lib._flags(l2norm_qk, beta_logits)
    a.l2_eps, a.scale = eps, scale
    a.q, a.q_stride = _rows(q, "q")
    a.k, a.k_stride = _rows(k, "k")
    a.v, a.v_stride = _rows(v, "v")
    p = _lib._ptr
    a.g, a.beta, a.S0, a.o, a.S_T = p(g), p(beta), p(S0), p(o), p(S_T)
    a.A_log, a.dt_bias = p(A_log), p(dt_bias)
    if cu_seqlens is not None:
        a.cu_seqlens = _int32(cu_seqlens, "cu_seqlens", dev)
        a.n_seqs = NS
    return a


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
    dev = q.device
    with _device(q):
        st = _stream(stream, dev)
        NS = q.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1
        if o is None:
            o = torch.empty(v.shape, dtype=q.dtype, device=dev)
            _used(st, o)
        if S_T is None:
            S_T = torch.empty(NS, v.shape[2], q.shape[3], v.shape[3], dtype=torch.float32, device=dev)
            _used(st, S_T)
        a = gdr_args(q, k, v, g, beta, S0, o, S_T, scale=scale, l2norm_qk=l2norm_qk, eps=eps,
                     A_log=A_log, dt_bias=dt_bias, beta_logits=beta_logits, cu_seqlens=cu_seqlens)
        lib = _lib.load()
        ws = _scratch(lib.kda_gdr_prefill_workspace_bytes(ctypes.byref(a)), dev, st, workspace)
        _lib._check(lib.kda_gdr_prefill(ctypes.byref(a), *_ws(ws), _handle(st)), "kda_gdr_prefill")
    return o, S_T


# ------------------------------------------------------------------ backward
def gdr_backward_args(fwd: GdrArgs, do, dS_T, grads: dict) -> GdrBackwardArgs:
    a = GdrBackwardArgs()
    a.fwd = fwd
    a.dO, a.dS_T = _lib._ptr(do), _lib._ptr(dS_T)
    for n in ("dq", "dk", "dv", "dg", "dbeta", "dS0", "dA_log", "ddt_bias"):
        setattr(a, n, _lib._ptr(grads.get(n)))
    return a


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
    dev, io = q.device, q.dtype
    B, T, Hk, Dk = q.shape
    Hv, Dv = v.shape[2:]
    NS = B if cu_seqlens is None else cu_seqlens.numel() - 1
    with _device(q):
        st = _stream(stream, dev)
        fwd = gdr_args(q, k, v, g, beta, S0, None, None, scale=scale, l2norm_qk=l2norm_qk, eps=eps,
                       A_log=A_log, dt_bias=dt_bias, beta_logits=beta_logits, cu_seqlens=cu_seqlens)
        _expect(do, "do", (B, T, Hv, Dv), io, dev)
        _expect(dS_T, "dS_T", (NS, Hv, Dk, Dv), torch.float32, dev)
        # packed offsets may leave tokens out: those gradients are not written
        new = torch.empty if cu_seqlens is None else torch.zeros
        grads = dict(dq=new(B, T, Hk, Dk, dtype=io, device=dev), dk=new(B, T, Hk, Dk, dtype=io, device=dev),
                     dv=new(B, T, Hv, Dv, dtype=io, device=dev), dg=new(B, T, Hv, dtype=io, device=dev),
                     dbeta=new(B, T, Hv, dtype=io, device=dev),
                     dS0=torch.empty(NS, Hv, Dk, Dv, dtype=torch.float32, device=dev))
        if A_log is not None:
            grads["dA_log"] = torch.empty(Hv, dtype=torch.float32, device=dev)
            grads["ddt_bias"] = torch.empty(Hv, dtype=torch.float32, device=dev)
        if isinstance(st, torch.cuda.Stream) and cu_seqlens is not None:
            st.wait_stream(torch.cuda.current_stream(dev))  # the zeros
        _used(st, *grads.values())
        a = gdr_backward_args(fwd, do, dS_T, grads)
        lib = _lib.load()
        ws = _scratch(lib.kda_gdr_backward_workspace_bytes(ctypes.byref(a)), dev, st, workspace)
        _lib._check(lib.kda_gdr_prefill_backward(ctypes.byref(a), *_ws(ws), _handle(st)),
                    "kda_gdr_prefill_backward")
    return grads


# ------------------------------------------------------------------ decode
def gdr_decode_args(q, k, v, g, beta, S, slots=None, o=None, *, scale=1.0, l2norm_qk=True, eps=1e-6,
                    A_log=None, dt_bias=None, beta_logits=False) -> GdrDecodeArgs:
    """Fill kda_gdr_decode_args from tensors (shapes as kda_gdr_decode)."""
    N, Hk, Dk = q.shape
    Hv, Dv = v.shape[1:]
    io, dev = q.dtype, q.device
    a = GdrDecodeArgs()
    a.io = _lib._io_of(q)
    _expect(k, "k", (N, Hk, Dk), io, dev)
    _expect(v, "v", (N, Hv, Dv), io, dev)
    _expect(g, "g", (N, Hv), io, dev)
    _expect(beta, "beta", (N, Hv), io, dev)
    _expect(S, "S", (S.shape[0], Hv, Dk, Dv), torch.float32, dev)
    _expect(o, "o", (N, Hv, Dv), io, dev)
    _expect(A_log, "A_log", (Hv,), torch.float32, dev)
    _expect(dt_bias, "dt_bias", (Hv,), torch.float32, dev)
    a.N, a.n_slots, a.Hk, a.Hv, a.Dk, a.Dv = N, S.shape[0], Hk, Hv, Dk, Dv
    a.flags = _lib._flags(l2norm_qk, beta_logits)
    a.l2_eps, a.scale = eps, scale
    a.q, a.q_stride = _rows(q, "q")
    a.k, a.k_stride = _rows(k, "k")
    a.v, a.v_stride = _rows(v, "v")
    p = _lib._ptr
    a.g, a.beta, a.S, a.o = p(g), p(beta), p(S), p(o)
    a.A_log, a.dt_bias = p(A_log), p(dt_bias)
    if slots is not None:
        if tuple(slots.shape) != (N,):
            raise ValueError(f"slots has shape {tuple(slots.shape)}, expected {(N,)}")
        a.slots = _int32(slots, "slots", dev)
    return a


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
    dev = q.device
    with _device(q):
        st = _stream(stream, dev)
        if o is None:
            new = torch.empty if slots is None else torch.zeros
            o = new(v.shape, dtype=q.dtype, device=dev)
            _used(st, o)
            if isinstance(st, torch.cuda.Stream) and slots is not None:
                st.wait_stream(torch.cuda.current_stream(dev))  # the zeros
        a = gdr_decode_args(q, k, v, g, beta, S, slots, o, scale=scale, l2norm_qk=l2norm_qk, eps=eps,
                            A_log=A_log, dt_bias=dt_bias, beta_logits=beta_logits)
        _lib._check(_lib.load().kda_gdr_decode(ctypes.byref(a), _handle(st)), "kda_gdr_decode")
    return o


# ------------------------------------------------------------------ pages
def pages_pool(pool) -> PagesPool:
    """kda_pages_pool of a tensor [layers, pages, ...] whose pages are dense (the
    layers may be further apart)."""
    if pool.dim() < 3:
        raise ValueError("a pool is [layers, pages, ...]")
    page = pool[0, 0]
    if not page.is_contiguous() or (pool.shape[1] > 1 and pool.stride(1) != page.numel()):
        raise ValueError("the pages of a layer must be dense")
    es = pool.element_size()
    p = PagesPool()
    p.data = pool.data_ptr()
    p.page_bytes = page.numel() * es
    p.layer_stride = pool.stride(0) * es if pool.shape[0] > 1 else 0
    p.n_layers, p.n_pages = pool.shape[:2]
    return p


def kda_pages_workspace_bytes(pool: PagesPool, n: int) -> int:
    return int(_lib.load().kda_pages_workspace_bytes(ctypes.byref(pool), n))


def kda_pages_fork(pool, refs, src, *, refs_out=None, dst=None, workspace=None, stream=None):
    """Forks pages of `pool` [layers, pages, ...]: request i gets the next free page
    (refs[p] <= 0), filled from page src[i] (zeros where -1).  Returns (dst, refs_out):
    the pages (-1 where a request could not be met) and the new counts."""
    dev = pool.device
    with _device(pool):
        st = _stream(stream, dev)
        p = pages_pool(pool)
        _expect(refs, "refs", (p.n_pages,), torch.int32, dev)
        _expect(refs_out, "refs_out", (p.n_pages,), torch.int32, dev)
        n = src.numel()
        _expect(dst, "dst", (n,), torch.int32, dev)
        if refs_out is None:
            refs_out = torch.empty_like(refs)
            _used(st, refs_out)
        if dst is None:
            dst = torch.empty(n, dtype=torch.int32, device=dev)
            _used(st, dst)
        ws = _scratch(kda_pages_workspace_bytes(p, n), dev, st, workspace)
        _lib._check(_lib.load().kda_pages_fork(ctypes.byref(p), _lib._ptr(refs), _lib._ptr(refs_out),
                                               _int32(src, "src", dev), _lib._ptr(dst), n, *_ws(ws),
                                               _handle(st)), "kda_pages_fork")
    return dst, refs_out


def kda_pages_free(refs, pages, *, refs_out=None, stream=None):
    """Lowers the count of every listed page (once for each time it is listed, not
    below 0).  Returns refs_out."""
    dev = refs.device
    with _device(refs):
        st = _stream(stream, dev)
        _expect(refs, "refs", (refs.numel(),), torch.int32, dev)
        _expect(refs_out, "refs_out", (refs.numel(),), torch.int32, dev)
        if refs_out is None:
            refs_out = torch.empty_like(refs)
            _used(st, refs_out)
        _lib._check(_lib.load().kda_pages_free(_lib._ptr(refs), _lib._ptr(refs_out), refs.numel(),
                                               _int32(pages, "pages", dev), pages.numel(), _handle(st)),
                    "kda_pages_free")
    return refs_out


def kda_pages_compact(pool, refs, table=None, *, refs_out=None, new_id=None, table_out=None,
                      workspace=None, stream=None):
    """Moves the pages in use to the front of the pool.  Returns (n_used [1],
    new_id, refs_out, table_out): the new index of every page (-1: free), the new
    counts, and the table's entries renamed (None without a table)."""
    dev = pool.device
    with _device(pool):
        st = _stream(stream, dev)
        p = pages_pool(pool)
        _expect(refs, "refs", (p.n_pages,), torch.int32, dev)
        _expect(refs_out, "refs_out", (p.n_pages,), torch.int32, dev)
        _expect(new_id, "new_id", (p.n_pages,), torch.int32, dev)
        if refs_out is None:
            refs_out = torch.empty_like(refs)
        if new_id is None:
            new_id = torch.empty_like(refs)
        n_used = torch.empty(1, dtype=torch.int32, device=dev)
        n = 0
        if table is not None:
            _int32(table, "table", dev)
            n = table.numel()
            if table_out is None:
                table_out = torch.empty_like(table)
            _expect(table_out, "table_out", table.shape, torch.int32, dev)
        _used(st, refs_out, new_id, n_used, table_out)
        ws = _scratch(kda_pages_workspace_bytes(p, 0), dev, st, workspace)
        _lib._check(_lib.load().kda_pages_compact(
            ctypes.byref(p), _lib._ptr(refs), _lib._ptr(refs_out), _lib._ptr(new_id), _lib._ptr(n_used),
            _lib._ptr(table), _lib._ptr(table_out), n, *_ws(ws), _handle(st)), "kda_pages_compact")
    return n_used, new_id, refs_out, table_out


def kda_pages_copy(src_pool, dst_pool, src, dst, *, done=None, workspace=None, stream=None):
    """Copies page src[i] of src_pool to page dst[i] of dst_pool (zeros where src[i]
    is -1) in every layer.  Returns done [n]: 1 where the pair was copied, 0 where it
    was left out (include/kda.h says which)."""
    dev = dst_pool.device
    if src_pool.device != dev:
        raise ValueError("both pools must be on one device")
    with _device(dst_pool):
        st = _stream(stream, dev)
        ps, pd = pages_pool(src_pool), pages_pool(dst_pool)
        n = src.numel()
        if dst.numel() != n:
            raise ValueError("src and dst differ in length")
        if done is None:
            done = torch.empty(n, dtype=torch.int32, device=dev)
            _used(st, done)
        _expect(done, "done", (n,), torch.int32, dev)
        ws = _scratch(kda_pages_workspace_bytes(pd, n), dev, st, workspace)
        _lib._check(_lib.load().kda_pages_copy(ctypes.byref(ps), ctypes.byref(pd), _int32(src, "src", dev),
                                               _int32(dst, "dst", dev), _lib._ptr(done), n, *_ws(ws),
                                               _handle(st)), "kda_pages_copy")
    return done
