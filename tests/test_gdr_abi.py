"""Arguments of the per-head gated delta rule and of the page operations on the CPU:
what is valid, and that every invalid call is refused with its own status before
anything is launched.  Pointers are fake addresses (never followed); the binding's own
checks (shapes, types, strides) run on CPU tensors."""
import ctypes
import re

import pytest
import torch

import gated_delta_rule_80_amd as kda
from gated_delta_rule_80_amd import _gdr, _lib

OK, NULL, SHAPE, DTYPE, ALIGN, ALIAS, UNSUP, WS, HIP, VALUE = range(10)


@pytest.fixture(scope="module")
def lib():
    return kda.load()


class Fake:
    def __init__(self):
        self.next = 0x7F0000000000

    def __call__(self, nbytes=1 << 32):
        p = self.next
        self.next += nbytes + 4096
        return p


INPUTS = ("q", "k", "v", "g", "beta", "S0")
GRADS = ("dq", "dk", "dv", "dg", "dbeta", "dS0", "dA_log", "ddt_bias")


def prefill(**kw):
    f = Fake()
    a = _gdr.GdrArgs(2, 100, 2, 4, 64, 128, 1, 1e-6, 0.125, _lib.KDA_BF16)
    for n in INPUTS + ("o", "S_T"):
        setattr(a, n, f())
    for n, x in kw.items():
        setattr(a, n, x)
    return a


def backward(raw=False, **kw):
    f = Fake()
    f.next = 0x6F0000000000
    a = _gdr.GdrBackwardArgs(prefill(o=None, S_T=None))
    for n in ("dO", "dS_T") + GRADS[:6]:
        setattr(a, n, f())
    if raw:
        a.fwd.A_log, a.fwd.dt_bias, a.dA_log, a.ddt_bias = f(), f(), f(), f()
    for n, x in kw.items():
        setattr(a.fwd if hasattr(a.fwd, n) and not hasattr(a, n) else a, n, x)
    return a


def decode(**kw):
    f = Fake()
    a = _gdr.GdrDecodeArgs(8, 20, 2, 4, 64, 128, 1, 1e-6, 0.125, _lib.KDA_BF16)
    for n in ("q", "k", "v", "g", "beta", "S", "slots", "o"):
        setattr(a, n, f())
    for n, x in kw.items():
        setattr(a, n, x)
    return a


MAKE = {"prefill": (prefill, kda.kda_validate_gdr_prefill), "backward": (backward, kda.kda_validate_gdr_backward),
        "decode": (decode, kda.kda_validate_gdr_decode)}


def test_struct_layouts_match_header():
    text = open(_lib.HEADER_PATH).read()
    for struct, cls in (("kda_gdr_args", _gdr.GdrArgs), ("kda_gdr_backward_args", _gdr.GdrBackwardArgs),
                        ("kda_gdr_decode_args", _gdr.GdrDecodeArgs), ("kda_pages_pool", _gdr.PagesPool)):
        body = text[text.index("typedef struct " + struct):]
        body = re.sub(r"/\*.*?\*/", "", body[:body.index("} " + struct)], flags=re.S)
        fields = re.findall(r"(?:const\s+)?(\w+)\s*(\*?)([^;{]*);", body[body.index("{"):])
        names, types = [], []
        for ty, star, rest in fields:
            for n in re.findall(r"(\*?)\s*(\w+)", rest):
                names.append(n[1])
                types.append("ptr" if star or n[0] else ty)
        assert [n for n, _ in cls._fields_] == names, struct
        size = {"ptr": 8, "void": 8, "int32_t": 4, "uint32_t": 4, "float": 4, "int64_t": 8,
                "kda_gdr_args": ctypes.sizeof(_gdr.GdrArgs)}
        for (n, t), ty in zip(cls._fields_, types):
            assert ctypes.sizeof(t) == size[ty], (struct, n)


def test_symbols_and_version(lib):
    names = set(kda.declared_functions())
    assert {"kda_gdr_prefill", "kda_gdr_prefill_backward", "kda_gdr_decode", "kda_pages_fork", "kda_pages_free",
            "kda_pages_compact", "kda_pages_copy"} <= names
    assert lib.kda_abi_version() == 7


@pytest.mark.parametrize("op", MAKE)
@pytest.mark.parametrize("field,value,code", [
    ("io", 2, DTYPE), ("io", -1, DTYPE), ("Hk", 0, SHAPE), ("Hv", 0, SHAPE), ("Hv", 3, SHAPE), ("Dk", 0, SHAPE),
    ("Dv", -128, SHAPE), ("Dk", 48, UNSUP), ("Dv", 256, UNSUP), ("Dk", 16, UNSUP), ("flags", 1 << 20, VALUE),
    ("l2_eps", -1e-6, VALUE), ("l2_eps", float("nan"), VALUE), ("scale", float("inf"), VALUE),
    ("q_stride", 127, SHAPE), ("q_stride", 132, SHAPE), ("k_stride", -128, SHAPE), ("v_stride", 511, SHAPE),
    ("v_stride", (1 << 23) + 8, SHAPE), ("q", None, NULL), ("k", None, NULL), ("v", None, NULL), ("g", None, NULL),
    ("beta", None, NULL), ("A_log", 0x1000, NULL), ("dt_bias", 0x1000, NULL)])
def test_common_refusals(lib, op, field, value, code):
    make, validate = MAKE[op]
    assert validate(make()) == OK
    assert validate(make(**{field: value})) == code


@pytest.mark.parametrize("op,field,value,code", [
    ("prefill", "B", 0, SHAPE), ("prefill", "T", -1, SHAPE), ("prefill", "n_seqs", 1, SHAPE),
    ("prefill", "o", None, NULL), ("prefill", "S_T", None, NULL), ("backward", "T", -1, SHAPE),
    ("backward", "dO", None, NULL), ("backward", "dq", None, NULL), ("backward", "dbeta", None, NULL),
    ("backward", "dA_log", 0x1000, NULL), ("decode", "N", -1, SHAPE), ("decode", "n_slots", 0, SHAPE),
    ("decode", "S", None, NULL), ("decode", "o", None, NULL)])
def test_own_refusals(lib, op, field, value, code):
    make, validate = MAKE[op]
    assert validate(make(**{field: value})) == code
    assert validate(make()) == OK


def test_null_struct(lib):
    assert lib.kda_validate_gdr_prefill(None) == NULL
    assert lib.kda_validate_gdr_backward(None) == NULL
    assert lib.kda_validate_gdr_decode(None) == NULL
    assert lib.kda_gdr_prefill_workspace_bytes(None) == 0
    assert lib.kda_gdr_backward_workspace_bytes(None) == 0
    assert lib.kda_gdr_prefill(None, None, 0, None) == NULL
    assert lib.kda_gdr_prefill_backward(None, None, 0, None) == NULL
    assert lib.kda_gdr_decode(None, None) == NULL


def test_alignment(lib):
    for op, names in (("prefill", INPUTS + ("o", "S_T")), ("decode", ("q", "k", "v", "g", "beta", "S", "slots", "o"))):
        make, validate = MAKE[op]
        for n in names:
            a = make()
            setattr(a, n, getattr(a, n) + 8)
            assert validate(a) == ALIGN, (op, n)
    for n in ("dO", "dS_T") + GRADS:
        a = backward(raw=True)
        setattr(a, n, getattr(a, n) + 4)
        assert kda.kda_validate_gdr_backward(a) == ALIGN, n


def test_aliasing(lib):
    v = kda.kda_validate_gdr_prefill
    a = prefill()
    a.S_T = a.S0
    assert v(a) == OK  # the state in place
    a.S_T = a.S0 + 256
    assert v(a) == ALIAS
    for n in INPUTS:
        a = prefill()
        a.o = getattr(a, n)
        assert v(a) == ALIAS, n
        a = prefill()
        a.S_T = getattr(a, n)
        assert v(a) == (OK if n == "S0" else ALIAS), n
    a = prefill()
    a.S_T = a.o
    assert v(a) == ALIAS
    # one fused projection for q, k, v; o inside its gap would still be an overlap
    a = prefill(q_stride=768, k_stride=768, v_stride=768)
    a.k, a.v = a.q + 128 * 2, a.q + 256 * 2
    assert v(a) == OK
    a.o = a.q + 64 * 768 * 2
    assert v(a) == ALIAS
    for n in GRADS:
        for m in ("q", "S0", "A_log"):
            a = backward(raw=True)
            setattr(a, n, getattr(a.fwd, m))
            assert kda.kda_validate_gdr_backward(a) == ALIAS, (n, m)
        for m in ("dO", "dS_T") + GRADS:
            if n != m:
                a = backward(raw=True)
                setattr(a, n, getattr(a, m))
                assert kda.kda_validate_gdr_backward(a) == ALIAS, (n, m)
    for n in ("q", "k", "v", "g", "beta", "slots", "o"):
        a = decode()
        a.S = getattr(a, n)
        assert kda.kda_validate_gdr_decode(a) == ALIAS, n


def test_packed_arguments(lib):
    v = kda.kda_validate_gdr_prefill
    cu = 0x6D0000000000
    assert v(prefill(B=1, cu_seqlens=cu, n_seqs=5)) == OK
    assert v(prefill(B=2, cu_seqlens=cu, n_seqs=5)) == SHAPE
    assert v(prefill(B=1, cu_seqlens=cu, n_seqs=0)) == SHAPE
    assert v(prefill(B=1, cu_seqlens=cu + 4, n_seqs=5)) == ALIGN
    a = prefill(B=1, cu_seqlens=cu, n_seqs=5)
    a.cu_seqlens = a.S_T
    assert v(a) == ALIAS
    size = kda.kda_gdr_prefill_workspace_bytes
    one, nine = (size(prefill(B=1, cu_seqlens=cu, n_seqs=n)) for n in (1, 9))
    # every sequence may end with a chunk of its own
    assert nine - one == 8 * 4 * (one - 256) // (3 * 4)


def test_sizes_that_do_not_fit(lib):
    v = kda.kda_validate_gdr_prefill
    assert v(prefill(B=0x7FFFFFFF, T=0x7FFFFFFF)) == SHAPE
    assert v(prefill(B=1, T=64 * ((1 << 23) // 4))) == SHAPE           # 2^23 chunks of 4 heads
    assert v(prefill(B=(1 << 21), T=1)) == SHAPE
    assert v(prefill(B=1, T=1, Hk=1, Hv=1 << 17)) == SHAPE             # a row of 2^24 elements
    assert kda.kda_validate_gdr_decode(decode(N=1 << 21, n_slots=1 << 21)) == SHAPE
    assert kda.kda_validate_gdr_decode(decode(N=21, slots=None)) == SHAPE   # rows past the pool
    assert kda.kda_validate_gdr_decode(decode(N=20, slots=None)) == OK


def test_empty_calls(lib):
    empty = dict.fromkeys(("q", "k", "v", "g", "beta", "o"))
    assert kda.kda_validate_gdr_prefill(prefill(T=0, **empty)) == OK
    assert kda.kda_gdr_prefill_workspace_bytes(prefill(T=0, **empty)) == 0
    a = backward(T=0, dO=None, dq=None, dk=None, dv=None, dg=None, dbeta=None)
    for n in ("q", "k", "v", "g", "beta"):
        setattr(a.fwd, n, None)
    assert kda.kda_validate_gdr_backward(a) == OK
    assert kda.kda_validate_gdr_decode(decode(N=0, **empty)) == OK


def test_workspace_refusals(lib):
    for a, need, run in ((prefill(), lib.kda_gdr_prefill_workspace_bytes, lib.kda_gdr_prefill),
                         (backward(), lib.kda_gdr_backward_workspace_bytes, lib.kda_gdr_prefill_backward)):
        r = ctypes.byref(a)
        n = need(r)
        assert n > 0
        assert run(r, None, n, None) == WS
        assert run(r, 0x5D0000000100, n - 1, None) == WS
        assert run(r, 0x5D0000000010, n, None) == WS
        q = a.q if hasattr(a, "q") else a.fwd.q
        assert run(r, q, n, None) == ALIAS


# ------------------------------------------------------------------ pages
def pool(**kw):
    p = _gdr.PagesPool(0x7E0000000000, 0, 4096, 3, 50)
    for n, x in kw.items():
        setattr(p, n, x)
    return p


def fork(lib, p=None, refs=0x100000, refs_out=0x100000, src=0x200000, dst=0x300000, n=7, ws=0x400000, size=1 << 20):
    return lib.kda_pages_fork(None if p is None else ctypes.byref(p), refs, refs_out, src, dst, n, ws, size, None)


def compact(lib, p, refs=0x100000, refs_out=0x100000, new_id=0x200000, used=0x300000, table=0x500000, out=0x500000,
            n=7, ws=0x400000, size=1 << 20):
    return lib.kda_pages_compact(ctypes.byref(p), refs, refs_out, new_id, used, table, out, n, ws, size, None)


def copy(lib, a, b, src=0x100000, dst=0x200000, done=0x300000, n=7, ws=0x400000, size=1 << 20):
    return lib.kda_pages_copy(ctypes.byref(a), ctypes.byref(b), src, dst, done, n, ws, size, None)


@pytest.mark.parametrize("field,value,code", [
    ("data", None, NULL), ("data", 0x7E0000000004, ALIGN), ("n_layers", 0, SHAPE), ("n_pages", 0, SHAPE),
    ("page_bytes", 0, SHAPE), ("page_bytes", 24, ALIGN), ("page_bytes", -16, SHAPE), ("layer_stride", -16, SHAPE),
    ("layer_stride", 4096 * 49, SHAPE), ("layer_stride", 4096 * 50 + 8, ALIGN), ("page_bytes", 1 << 62, SHAPE),
    ("layer_stride", (1 << 63) - 16, SHAPE)])
def test_pool_refusals(lib, field, value, code):
    p = pool(**{field: value})
    if field == "layer_stride" and value > 1 << 40:
        p.n_layers = 100  # the whole pool passes 64 bits
    assert fork(lib, p) == code
    assert compact(lib, p) == code
    assert copy(lib, p, pool()) == code
    assert copy(lib, pool(), p) == code
    assert lib.kda_pages_workspace_bytes(ctypes.byref(p), 4) == 0


def test_pages_refusals(lib):
    p = pool()
    assert fork(lib) == NULL
    assert fork(lib, p, n=-1) == SHAPE
    for n in ("refs", "refs_out", "src", "dst"):
        assert fork(lib, p, **{n: None}) == NULL, n
        assert fork(lib, p, **{n: 0x100008}) == ALIGN, n
    assert fork(lib, p, refs_out=0x100040) == ALIAS       # counts in place or apart
    assert fork(lib, p, dst=0x200010) == ALIAS            # src and dst
    assert fork(lib, p, dst=0x100000) == ALIAS
    assert fork(lib, p, src=0x7E0000000000) == ALIAS
    assert fork(lib, p, ws=None) == WS and fork(lib, p, size=64) == WS and fork(lib, p, ws=0x400010) == WS
    assert fork(lib, p, ws=0x7E0000000000) == ALIAS

    free = lambda **kw: lib.kda_pages_free(*dict(dict(refs=0x1000, out=0x1000, n_pages=50, pages=0x2000, n=3,  # noqa: E731
                                                      stream=None), **kw).values())
    assert free(n_pages=0) == SHAPE and free(n=-1) == SHAPE
    assert free(refs=None) == NULL and free(out=None) == NULL and free(pages=None) == NULL
    assert free(pages=0x2004) == ALIGN and free(out=0x1040) == ALIAS and free(pages=0x1000) == ALIAS

    assert compact(lib, p, n=-1) == SHAPE
    for n in ("refs", "refs_out", "new_id", "used", "table", "out"):
        assert compact(lib, p, **{n: None}) == NULL, n
        assert compact(lib, p, **{n: 0x600004}) == ALIGN, n
    assert compact(lib, p, new_id=0x100000) == ALIAS and compact(lib, p, used=0x500000) == ALIAS
    assert compact(lib, p, out=0x500010) == ALIAS and compact(lib, p, table=0x200000, out=0x600000) == ALIAS
    assert compact(lib, p, size=0) == WS

    q = pool(data=0x6E0000000000)
    assert copy(lib, p, pool(data=0x6E0000000000, n_layers=4)) == SHAPE
    assert copy(lib, p, pool(data=0x6E0000000000, page_bytes=8192)) == SHAPE
    assert copy(lib, p, q, n=-1) == SHAPE
    assert copy(lib, p, q, src=None) == NULL and copy(lib, p, q, dst=None) == NULL
    assert copy(lib, p, q, done=0x300008) == ALIGN
    assert copy(lib, p, pool(data=0x7E0000000000 + 4096)) == ALIAS  # pools that overlap in part
    assert copy(lib, p, pool(n_pages=40)) == ALIAS
    assert copy(lib, p, q, done=0x200000) == ALIAS
    assert copy(lib, p, q, size=16) == WS
    assert copy(lib, p, q, n=0, src=None, dst=None, done=None) == OK  # nothing to do: nothing is launched


# ------------------------------------------------------------------ the binding
def tensors(B=2, T=5, Hk=2, Hv=4, Dk=32, Dv=64, dt=torch.bfloat16):
    z = lambda *s: torch.zeros(*s, dtype=dt)  # noqa: E731
    return dict(q=z(B, T, Hk, Dk), k=z(B, T, Hk, Dk), v=z(B, T, Hv, Dv), g=z(B, T, Hv), beta=z(B, T, Hv),
                S0=torch.zeros(B, Hv, Dk, Dv))


def test_binding_strides():
    row = torch.zeros(2, 5, 2 * 2 * 32 + 4 * 64, dtype=torch.bfloat16)
    t = tensors()
    t["q"] = row[..., :64].unflatten(-1, (2, 32))
    t["v"] = row[..., 128:].unflatten(-1, (4, 64))
    a = kda.gdr_args(**t)
    assert a.q_stride == a.v_stride == 384 and a.k_stride == 0
    t["q"] = row[:, :1, :64].unflatten(-1, (2, 32))  # one token a row: the rows' distance
    t = dict(tensors(T=1), q=t["q"])
    assert kda.gdr_args(**t).q_stride == 5 * 384


@pytest.mark.parametrize("name,make", [
    ("q", lambda t: torch.zeros(2, 1, 2, 32, dtype=t.dtype).expand(2, 5, 2, 32)),
    ("q", lambda t: torch.zeros(1, 5, 2, 32, dtype=t.dtype).expand(2, 5, 2, 32)),
    ("k", lambda t: t.transpose(1, 2).contiguous().transpose(1, 2)),
    ("k", lambda t: torch.zeros(2, 5, 2, 64, dtype=t.dtype)[..., ::2]),
    ("v", lambda t: torch.zeros(2, 7, 4, 64, dtype=t.dtype)[:, :5]),
    ("v", lambda t: t[..., :32]), ("g", lambda t: t[:, :4]),
    ("beta", lambda t: t.transpose(1, 2).contiguous().transpose(1, 2)),
    ("S0", lambda t: t[:1]), ("q", lambda t: t[:, :, :1])])
def test_binding_shape_refusals(name, make):
    t = tensors()
    t[name] = make(t[name])
    with pytest.raises(ValueError):
        kda.gdr_args(**t)


def test_binding_type_refusals():
    for n in ("k", "v", "g", "beta"):
        t = tensors()
        t[n] = t[n].float()
        with pytest.raises(TypeError):
            kda.gdr_args(**t)
    t = tensors()
    t["S0"] = t["S0"].bfloat16()
    with pytest.raises(TypeError):
        kda.gdr_args(**t)
    t = tensors(B=1)
    with pytest.raises(TypeError):
        kda.gdr_args(**t, cu_seqlens=torch.tensor([0, 5]))
    with pytest.raises(ValueError):
        kda.gdr_args(**t, cu_seqlens=torch.zeros(0, dtype=torch.int32))
    with pytest.raises((TypeError, ValueError)):
        kda.gdr_args(**tensors(dt=torch.float16))
    d = dict(q=torch.zeros(3, 2, 32), k=torch.zeros(3, 2, 32), v=torch.zeros(3, 4, 64), g=torch.zeros(3, 4),
             beta=torch.zeros(3, 4), S=torch.zeros(9, 4, 32, 64))
    kda.gdr_decode_args(**d)
    with pytest.raises(ValueError):
        kda.gdr_decode_args(**d, slots=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError):
        kda.gdr_decode_args(**d, slots=torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        kda.gdr_decode_args(**dict(d, S=torch.zeros(9, 4, 64, 32)))


def test_binding_refuses_host_memory():
    t = tensors()
    with pytest.raises(ValueError):
        kda.kda_gdr_prefill(**t)
    with pytest.raises(ValueError):
        kda.kda_gdr_prefill_backward(**t, do=t["v"])
    with pytest.raises(ValueError):
        kda.kda_gdr_decode(*(t[n][:, 0].contiguous() for n in ("q", "k", "v", "g", "beta")), t["S0"])
    p, i = torch.zeros(1, 4, 8), torch.zeros(4, dtype=torch.int32)
    for call in (lambda: kda.kda_pages_fork(p, i, i), lambda: kda.kda_pages_free(i, i),
                 lambda: kda.kda_pages_compact(p, i), lambda: kda.kda_pages_copy(p, p, i, i)):
        with pytest.raises(ValueError):
            call()


def test_binding_pools():
    p = torch.zeros(3, 10, 4, 8)
    a = kda.pages_pool(p)
    assert (a.n_layers, a.n_pages, a.page_bytes, a.layer_stride) == (3, 10, 128, 0)
    a = kda.pages_pool(p[:, :6])
    assert (a.n_pages, a.layer_stride) == (6, 10 * 128)
    for bad in (p.transpose(0, 1), p[..., :4], p[:, ::2], p[:1].expand(3, 10, 4, 8), torch.zeros(3, 10)):
        with pytest.raises(ValueError):
            kda.pages_pool(bad)
