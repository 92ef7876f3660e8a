"""The gated delta rule with one decay per head on the GPU against its float64
statement (oracle/gdr_oracle.py): whole prompts, their gradients, single tokens on a
pool of states, and a run of them together.

Tolerances, relative L2 per tensor.  A bf16 rounding is off by at most 2^-8 of the
value, a float32 one by 2^-24.  With bf16 inputs:
  S_T, dS0   the products on their path read S (or dS), Tm and P in two bf16 terms
             (2^-16 each) and the rest in three (2^-24); float32 sums of at most 512
             terms:                                      3 2^-16 + 512 2^-24
  o          the output's own rounding and that of P:    2 2^-8
  dv         its own rounding, beside the above:         2 2^-8
  gradients  Y, dX, S, dS and the output, one each:      5 2^-8
With float32 inputs every step is float32; sums of at most 512 terms, two of them in
a row (the gradients of norms and gates add a third):     1024 (1536) 2^-24
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_80_amd as kda
from oracle import gdr_oracle as ref

pytestmark = pytest.mark.gpu

STATE = {"bf16": 3 * 2.0 ** -16 + 512 * 2.0 ** -24, "fp32": 1024 * 2.0 ** -24}
OUT = {"bf16": 2 * 2.0 ** -8, "fp32": 1024 * 2.0 ** -24}
GRAD = {"bf16": 5 * 2.0 ** -8, "fp32": 1536 * 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def rel(x, y):
    x = np.asarray(x.double().cpu() if torch.is_tensor(x) else x, np.float64)
    n = np.linalg.norm(y)
    assert np.isfinite(x).all()
    return np.linalg.norm(x - y) / n if n else np.linalg.norm(x)


def make(B, T, Hk, Hv, Dk, Dv, io, *, n_seqs=None, s0=True, raw=False, seed=0, rate=(-3.0, 2.0)):
    g = torch.Generator().manual_seed(seed)
    dt = DT[io]
    x = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    NS = B if n_seqs is None else n_seqs
    d = dict(q=torch.nn.functional.silu(x(B, T, Hk, Dk)).to(dt), k=torch.nn.functional.silu(x(B, T, Hk, Dk)).to(dt),
             v=x(B, T, Hv, Dv).to(dt))
    A = torch.rand(Hv, generator=g) * (rate[1] - rate[0]) + rate[0]
    f, b, bias = x(B, T, Hv), x(B, T, Hv) * 1.4, x(Hv) * 0.5
    if raw:
        d.update(g=f.to(dt), beta=b.to(dt))
        opt = dict(A_log=A, dt_bias=bias, beta_logits=True)
    else:
        d.update(g=(-A.exp() * torch.nn.functional.softplus(f + bias)).to(dt), beta=torch.sigmoid(b).to(dt))
        opt = {}
    d["S0"] = x(NS, Hv, Dk, Dv) * 0.1 if s0 else None
    d["do"] = x(B, T, Hv, Dv).to(dt)
    d["dS_T"] = x(NS, Hv, Dk, Dv) * 0.1
    return d, opt


def num(x):
    return None if x is None else x.double().numpy()


def dev(x):
    return x.cuda() if torch.is_tensor(x) else x


def forward(d, opt, cu=None, **kw):
    o, S = kda.kda_gdr_prefill(*[dev(d[n]) for n in ("q", "k", "v", "g", "beta", "S0")],
                               cu_seqlens=dev(cu), **{n: dev(x) for n, x in opt.items()}, **kw)
    torch.cuda.synchronize()
    return o, S


def check_forward(d, opt, io, cu=None, l2=True, scale=1.0):
    o, S = forward(d, opt, cu, l2norm_qk=l2, scale=scale)
    ro, rS = ref.gdr_reference(*[num(d[n]) for n in ("q", "k", "v", "g", "beta", "S0")], l2=l2, scale=scale,
                               cu_seqlens=None if cu is None else cu.tolist(),
                               **{n: num(x) if torch.is_tensor(x) else x for n, x in opt.items()})
    eo, eS = rel(o, ro), rel(S, rS)
    print(f"o {eo:.2e} S {eS:.2e}", flush=True)
    assert eo <= OUT[io] and eS <= STATE[io]
    return o, S


CASES = [  # B, T, Hk, Hv, Dk, Dv
    (1, 1, 1, 1, 32, 32), (1, 2, 1, 2, 64, 64), (2, 31, 2, 2, 32, 64), (1, 32, 1, 3, 64, 32),
    (1, 33, 2, 4, 128, 32), (1, 63, 1, 1, 128, 128), (2, 64, 1, 2, 128, 128), (1, 65, 3, 3, 64, 128),
    (1, 127, 1, 2, 32, 128), (3, 129, 2, 6, 128, 64), (1, 300, 1, 2, 128, 128), (1, 17, 1, 5, 64, 64),
]


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", CASES, ids=str)
def test_prefill(shape, io):
    d, opt = make(*shape, io, seed=sum(shape))
    check_forward(d, opt, io)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_prefill_options(io):
    shape = (2, 100, 2, 4, 64, 64)
    check_forward(*make(*shape, io, s0=False), io)
    check_forward(*make(*shape, io, raw=True), io)
    check_forward(*make(*shape, io), io, scale=-0.125)
    # rows as given: keys of norm below one, as a caller who normalised them has
    d, opt = make(*shape, io)
    for n in ("q", "k"):
        d[n] = torch.nn.functional.normalize(d[n].float(), dim=-1).to(DT[io])
    check_forward(d, opt, io, l2=False)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("shape,rate", [((1, 1100, 1, 2, 128, 128), (-8.0, -5.0)), ((2, 1601, 2, 2, 64, 32), (-9.0, 0.0)),
                                        ((1, 2573, 1, 1, 32, 64), (-7.0, -4.0)), ((1, 1537, 1, 3, 128, 64), (-3.0, 2.0))],
                         ids=str)
def test_prefill_split(shape, rate, io):
    """Few long rows, whose walks are cut into segments; the state carries far, so
    the segments' maps count."""
    d, opt = make(*shape, io, seed=shape[1], rate=rate)
    o, S = check_forward(d, opt, io)
    check_forward(dict(d, S0=None), opt, io)
    x = d["S0"].cuda()  # the state in place
    o2, _ = kda.kda_gdr_prefill(*[d[n].cuda() for n in ("q", "k", "v", "g", "beta")], x, S_T=x)
    assert torch.equal(o, o2) and torch.equal(S, x)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("B", [5, 8, 9])
def test_many_walks(B, io):
    """More walks than the card holds workgroups, also a few more than that many."""
    d, opt = make(B, 70, 8, 32, 32, 128, io, seed=B)
    check_forward(d, opt, io)
    check_backward(d, opt, io)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("Hk,Hv", [(1, 40), (3, 9), (1, 7)])
def test_many_heads_on_one_key_head(Hk, Hv, io):
    d, opt = make(2, 75, Hk, Hv, 64, 32, io, seed=Hv)
    check_forward(d, opt, io)
    check_backward(d, opt, io)


LENS = [[0, 1, 0, 70, 64, 3, 0, 129, 32, 0], [5], [0, 0, 0], [1] * 40]


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("lens", LENS, ids=lambda x: "-".join(map(str, x[:4])))
def test_prefill_packed(lens, io):
    T = sum(lens)
    d, opt = make(1, T, 2, 4, 64, 128, io, n_seqs=len(lens), seed=T)
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)
    if T:
        check_forward(d, opt, io, cu)
    else:
        _, S = forward(d, opt, cu)
        assert torch.equal(S.cpu(), d["S0"])


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_packed_many_sequences(io):
    lens = [i * 7 % 4 for i in range(2500)]
    T = sum(lens)
    d, opt = make(1, T, 1, 2, 32, 32, io, n_seqs=len(lens), seed=1)
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)
    check_forward(d, opt, io, cu)
    check_backward(d, opt, io, cu)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("lens", [[0, 2000, 1, 0, 4100, 700, 257, 0], [3000], [0, 5000, 0], [900, 2600, 63, 1700]], ids=str)
def test_packed_split(lens, io):
    """Long prompts of few heads: each sequence's walk is cut into its own segments."""
    T = sum(lens)
    d, opt = make(1, T, 1, 2, 64, 64, io, n_seqs=len(lens), seed=T, rate=(-9.0, -5.0))
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)
    o, S = check_forward(d, opt, io, cu)
    x = d["S0"].cuda()  # the states in place
    o2, _ = kda.kda_gdr_prefill(*[d[n].cuda() for n in ("q", "k", "v", "g", "beta")], x, S_T=x, cu_seqlens=cu.cuda())
    assert torch.equal(o, o2) and torch.equal(S, x)
    check_forward(dict(d, S0=None), opt, io, cu)
    # offsets that leave a gap, or go down (read as their running maximum)
    cu[0], cu[-1] = min(lens[0], 40), T - 3
    o = torch.full((1, T, 2, 64), 7.0, dtype=DT[io], device="cuda")
    _, S = forward(d, opt, cu, o=o)
    at = np.maximum.accumulate(cu.numpy()).tolist()
    ro, rS = ref.gdr_reference(*[num(d[n]) for n in ("q", "k", "v", "g", "beta", "S0")], cu_seqlens=at)
    a, b = at[0], at[-1]
    assert rel(o[:, a:b], ro[:, a:b]) <= OUT[io] and rel(S, rS) <= STATE[io]
    assert (o[:, :a] == 7).all() and (o[:, b:] == 7).all()


def test_prefill_no_tokens():
    d, opt = make(2, 0, 1, 2, 32, 64, "bf16")
    o, S = forward(d, opt)
    assert o.shape == (2, 0, 2, 64) and torch.equal(S.cpu(), d["S0"])
    assert not forward(dict(d, S0=None), opt)[1].any()


def test_prefill_tokens_outside_sequences_are_left():
    d, opt = make(1, 200, 1, 2, 64, 64, "bf16", n_seqs=3)
    cu = torch.tensor([20, 90, 90, 150], dtype=torch.int32)
    o = torch.full((1, 200, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    _, S = forward(d, opt, cu, o=o)
    assert (o[:, :20] == 7).all() and (o[:, 150:] == 7).all()
    ro, rS = ref.gdr_reference(*[num(d[n]) for n in ("q", "k", "v", "g", "beta", "S0")], cu_seqlens=cu.tolist())
    assert rel(o[:, 20:150], ro[:, 20:150]) <= OUT["bf16"] and rel(S, rS) <= STATE["bf16"]
    # offsets that go down or leave the row are read as their running maximum in [0, T]
    bad = torch.tensor([-5, 90, 30, 999], dtype=torch.int32)
    _, S = forward(d, opt, bad)
    _, rS = ref.gdr_reference(*[num(d[n]) for n in ("q", "k", "v", "g", "beta", "S0")], cu_seqlens=[0, 90, 90, 200])
    assert rel(S, rS) <= STATE["bf16"]


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_prefill_decays(io):
    """No decay, strong ones, and a state that is forgotten (g = -inf)."""
    d, opt = make(1, 150, 1, 4, 64, 64, io)
    d["g"][..., 0] = 0
    d["g"][..., 1] = -30
    d["g"][:, ::7, 2] = float("-inf")
    d["g"][..., 3] = float("-inf")
    check_forward(d, opt, io)
    d["beta"][..., 0] = 0          # nothing is written
    d["beta"][..., 2] = 2          # a full reflection
    check_forward(d, opt, io)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_prefill_equal_keys(io):
    """All keys alike: the chunk's triangular matrix is as far from I as it gets."""
    d, opt = make(1, 130, 1, 2, 64, 64, io, rate=(-9.0, -8.0))
    d["k"][:] = d["k"][:, :1]
    d["beta"][:] = 1
    check_forward(d, opt, io)


def test_prefill_strided_projection():
    """q, k, v as parts of one fused projection, and the state updated in place."""
    d, opt = make(2, 77, 2, 4, 64, 64, "bf16")
    row = torch.cat([d[n].flatten(2) for n in ("q", "k", "v")], -1).cuda()
    row = torch.nn.functional.pad(row, (0, 16))
    q, k, v = row[..., :128].unflatten(-1, (2, 64)), row[..., 128:256].unflatten(-1, (2, 64)), row[
        ..., 256:512].unflatten(-1, (4, 64))
    o, S = forward(d, opt)
    S2 = d["S0"].cuda()
    o2, S3 = kda.kda_gdr_prefill(q, k, v, d["g"].cuda(), d["beta"].cuda(), S2, S_T=S2)
    assert S3 is S2 and torch.equal(o2, o) and torch.equal(S2, S)


def test_prefill_in_parts_equals_whole():
    d, opt = make(1, 200, 1, 2, 128, 128, "fp32")
    _, S = forward(d, opt)
    part = lambda a, b: {n: (x[:, a:b].contiguous() if n not in ("S0", "dS_T") else x) for n, x in d.items()}  # noqa: E731
    d1, d2 = part(0, 83), part(83, 200)
    _, S1 = forward(d1, opt)
    d2["S0"] = S1.cpu()
    _, S2 = forward(d2, opt)
    assert rel(S2, S.double().cpu().numpy()) <= STATE["fp32"]


# ------------------------------------------------------------------ gradients
def check_backward(d, opt, io, cu=None, l2=True, scale=1.0, with_dS=True):
    args = [dev(d[n]) for n in ("q", "k", "v", "g", "beta", "S0")]
    got = kda.kda_gdr_prefill_backward(*args, do=dev(d["do"]), dS_T=dev(d["dS_T"]) if with_dS else None,
                                       cu_seqlens=dev(cu), l2norm_qk=l2, scale=scale,
                                       **{n: dev(x) for n, x in opt.items()})
    torch.cuda.synchronize()
    want = ref.gdr_reference_backward(*[num(d[n]) for n in ("q", "k", "v", "g", "beta", "S0", "do")],
                                      num(d["dS_T"]) if with_dS else None, l2=l2, scale=scale,
                                      cu_seqlens=None if cu is None else cu.tolist(),
                                      **{n: num(x) if torch.is_tensor(x) else x for n, x in opt.items()})
    assert set(got) == set(want)
    err = {n: rel(got[n], want[n]) for n in want}
    print({n: f"{e:.1e}" for n, e in err.items()}, flush=True)
    for n, e in err.items():
        assert e <= {"dS0": STATE, "dv": OUT}.get(n, GRAD)[io], (n, e)
    return got


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", CASES, ids=str)
def test_backward(shape, io):
    d, opt = make(*shape, io, seed=sum(shape) + 1)
    check_backward(d, opt, io)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_backward_options(io):
    shape = (2, 100, 2, 4, 64, 64)
    check_backward(*make(*shape, io, s0=False), io, with_dS=False)
    check_backward(*make(*shape, io, raw=True), io)
    check_backward(*make(*shape, io), io, scale=-0.125)
    d, opt = make(*shape, io)
    for n in ("q", "k"):
        d[n] = torch.nn.functional.normalize(d[n].float(), dim=-1).to(DT[io])
    check_backward(d, opt, io, l2=False)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("lens", LENS[:2] + LENS[3:], ids=lambda x: "-".join(map(str, x[:4])))
def test_backward_packed(lens, io):
    T = sum(lens)
    d, opt = make(1, T, 2, 4, 64, 128, io, n_seqs=len(lens), seed=T, raw=True)
    check_backward(d, opt, io, torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32))


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("shape,rate", [((1, 1100, 1, 2, 128, 128), (-8.0, -5.0)), ((2, 1601, 2, 2, 64, 32), (-9.0, 0.0)),
                                        ((1, 2573, 1, 1, 32, 64), (-7.0, -4.0)), ((1, 1537, 1, 3, 128, 64), (-3.0, 2.0)),
                                        ((1, 6 * 256, 2, 2, 64, 128), (-9.0, -5.0))], ids=str)
def test_backward_split(shape, rate, io):
    """Few long rows, whose walks are cut into segments; states and gradients carry far."""
    d, opt = make(*shape, io, seed=shape[1] + 1, rate=rate)
    check_backward(d, opt, io)
    check_backward(dict(d, S0=None), opt, io, with_dS=False)


def test_backward_empty():
    d, opt = make(2, 0, 1, 2, 32, 32, "bf16", raw=True)
    got = check_backward(d, opt, "bf16")
    assert torch.equal(got["dS0"].cpu(), d["dS_T"]) and not got["dA_log"].any()


def test_backward_deterministic():
    d, opt = make(1, 150, 1, 4, 64, 64, "bf16")
    a, b = check_backward(d, opt, "bf16"), check_backward(d, opt, "bf16")
    assert all(torch.equal(a[n], b[n]) for n in a)


# ------------------------------------------------------------------ decode
def check_decode(io, N, slots, n_slots, Hk, Hv, Dk, Dv, raw=False, seed=0, scale=1.0, l2=True):
    d, opt = make(1, N, Hk, Hv, Dk, Dv, io, raw=raw, seed=seed)
    g = torch.Generator().manual_seed(seed + 1)
    S = torch.randn(n_slots, Hv, Dk, Dv, generator=g) * 0.1
    o = torch.full((N, Hv, Dv), 7.0).to(DT[io])
    x = [d[n][0] for n in ("q", "k", "v", "g", "beta")]
    gS, go = S.cuda(), o.cuda()
    kda.kda_gdr_decode(*[y.cuda() for y in x], gS, None if slots is None else torch.tensor(slots, dtype=torch.int32).cuda(),
                       o=go, scale=scale, l2norm_qk=l2, **{n: dev(y) for n, y in opt.items()})
    torch.cuda.synchronize()
    at = list(range(N)) if slots is None else slots
    ro, rS = ref.gdr_reference_decode(*[num(y) for y in x], num(S), at, num(o), scale=scale, l2=l2,
                                      **{n: num(y) if torch.is_tensor(y) else y for n, y in opt.items()})
    # one float32 step: no bf16 term on any path but the output's rounding
    assert rel(go, ro) <= (2.0 ** -8 if io == "bf16" else OUT[io]) and rel(gS, rS) <= STATE["fp32"]
    idle = [i for i, s in enumerate(at) if not 0 <= s < n_slots]
    assert (go[idle] == 7).all()
    rest = [s for s in range(n_slots) if s not in at]
    assert torch.equal(gS[rest].cpu(), S[rest])


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("Dk,Dv", [(32, 32), (32, 128), (64, 64), (128, 32), (128, 128), (64, 128)])
def test_decode(io, Dk, Dv):
    check_decode(io, 1, None, 1, 1, 1, Dk, Dv)
    check_decode(io, 5, [3, -1, 0, 9, 2], 4, 2, 4, Dk, Dv, raw=True, scale=0.3)
    check_decode(io, 3, None, 6, 1, 3, Dk, Dv, l2=False)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_decode_tokens_of_one_slot(io):
    """Rows with one slot are its tokens in order, wherever they stand."""
    check_decode(io, 12, [4, 1, 4, -1, 4, 0, 1, 100, 4, 2, 2, 4], 5, 2, 4, 64, 64, raw=True)
    check_decode(io, 300, [7] * 300, 9, 1, 1, 32, 32)
    check_decode(io, 700, [(i * 7) % 13 - 1 for i in range(700)], 12, 1, 2, 32, 64)


def test_decode_strided():
    d, _ = make(1, 6, 2, 2, 64, 64, "bf16")
    x = {n: d[n][0].cuda() for n in ("q", "k", "v", "g", "beta")}
    row = torch.nn.functional.pad(torch.cat([x[n].flatten(1) for n in ("q", "k", "v")], -1), (0, 8))
    q, k, v = (row[:, 128 * i:128 * i + 128].unflatten(-1, (2, 64)) for i in range(3))
    S = torch.randn(6, 2, 64, 64, device="cuda")
    S2 = S.clone()
    o = kda.kda_gdr_decode(x["q"], x["k"], x["v"], x["g"], x["beta"], S)
    assert torch.equal(kda.kda_gdr_decode(q, k, v, x["g"], x["beta"], S2), o) and torch.equal(S, S2)


def test_prefill_equals_decode():
    """A prompt in one call and token by token from the same state."""
    d, opt = make(1, 70, 1, 2, 64, 64, "fp32")
    o, S = forward(d, opt)
    S2 = d["S0"].cuda()
    x = [d[n][0].cuda() for n in ("q", "k", "v", "g", "beta")]
    o2 = kda.kda_gdr_decode(*x, S2, torch.zeros(70, dtype=torch.int32, device="cuda"))
    assert rel(o2, o[0].double().cpu().numpy()) <= 2 * OUT["fp32"]
    assert rel(S2, S.double().cpu().numpy()) <= 2 * STATE["fp32"]
