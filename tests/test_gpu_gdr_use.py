"""The per-head gated delta rule and the page operations as programs use them: on the
caller's stream, captured into graphs and replayed, beside each other, with garbage in
what a call must not read, and at offsets that pass 32 bits.  Results of the same call
are compared bit by bit: every sum has one order."""
import numpy as np
import pytest
import torch

import gated_delta_rule_80_amd as kda
from oracle import gdr_oracle as ref
from test_gpu_gdr import GRAD, OUT, check_backward, dev, make, num, rel

pytestmark = pytest.mark.gpu

NAMES = ("q", "k", "v", "g", "beta", "S0")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def call(d, opt, **kw):
    return kda.kda_gdr_prefill(*[d[n] for n in NAMES], **opt, **kw)


def grads(d, opt, **kw):
    return kda.kda_gdr_prefill_backward(*[d[n] for n in NAMES], do=d["do"], dS_T=d["dS_T"], **opt, **kw)


def on_gpu(*shape, **kw):
    d, opt = make(*shape, **kw)
    return {n: dev(x) for n, x in d.items()}, {n: dev(x) for n, x in opt.items()}


def decode_case(d, n, slots, pages):
    S = torch.zeros(pages, *d["S0"].shape[1:], device="cuda")
    x = [d[m][0, :n].contiguous() for m in ("q", "k", "v", "g", "beta")]
    return x, S, i32(slots)


# ------------------------------------------------------------------ gradients
@pytest.mark.parametrize("Hk,Hv,Dk,Dv", [(1, 2, 64, 32), (2, 2, 32, 128)])
def test_gradients_against_differences(Hk, Hv, Dk, Dv):
    """Along the gradient itself, every input at once: D(h) = (L(x + h e) - L(x - h e)) / 2h
    is off by c h^2, so D(1/2) is by a third of D(1) - D(1/2), beside the loss's own
    rounding."""
    d, opt = on_gpu(2, 97, Hk, Hv, Dk, Dv, io="fp32", raw=True, seed=7)
    got = grads(d, opt)
    names = [n for n in NAMES] + ["A_log", "dt_bias"]
    x = {**{n: d[n] for n in NAMES}, **{n: opt[n] for n in ("A_log", "dt_bias")}}
    step = {n: got["d" + n] * (0.02 * x[n].norm() / got["d" + n].norm()) for n in names}
    want = sum((got["d" + n].double() * step[n].double()).sum().item() for n in names)

    def loss(h):
        y = {n: x[n] + h * step[n] for n in names}
        o, S = kda.kda_gdr_prefill(*[y[n] for n in NAMES], A_log=y["A_log"], dt_bias=y["dt_bias"], beta_logits=True)
        return (o.double() * d["do"].double()).sum().item() + (S.double() * d["dS_T"].double()).sum().item(), o, S

    D = {}
    for h in (1.0, 0.5):
        (up, o, S), (down, _, _) = loss(h), loss(-h)
        D[h] = (up - down) / (2 * h)
    noise = 2 * 2.0 ** -24 * (o.norm() * d["do"].norm() + S.norm() * d["dS_T"].norm()).item() / 0.5
    tol = abs(D[1.0] - D[0.5]) + noise
    assert tol < 0.05 * want  # the test says something
    assert abs(D[0.5] - want) <= tol


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_backward_decays(io):
    """No decay, strong ones, and states that are forgotten (g = -inf)."""
    d, opt = make(1, 150, 1, 4, 64, 64, io)
    d["g"][..., 0] = 0
    d["g"][..., 1] = -30
    d["g"][:, ::7, 2] = float("-inf")
    d["g"][..., 3] = float("-inf")
    d["beta"][..., 2] = 2
    # the states before a forgotten one take no gradient; in float64, e^-1000 stands for it
    e = dict(d, g=d["g"].clamp(min=-1000))
    got = kda.kda_gdr_prefill_backward(*[dev(d[n]) for n in NAMES], do=dev(d["do"]), dS_T=dev(d["dS_T"]))
    want = ref.gdr_reference_backward(*[num(e[n]) for n in NAMES], num(e["do"]), num(e["dS_T"]))
    for n in want:
        assert rel(got[n], want[n]) <= GRAD[io], n
    assert not got["dS0"][:, 3].any()


# ------------------------------------------------------------------ what must not be read
@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_garbage_outside_sequences(io):
    d, opt = make(1, 260, 1, 2, 64, 64, io, n_seqs=4, raw=True)
    cu = [13, 80, 80, 81, 209]
    clean = [t for s, e in zip(cu[:-1], cu[1:]) for t in range(s, e)]
    dirty = sorted(set(range(260)) - set(clean))
    e = {n: x.clone() for n, x in d.items()}
    for n in ("q", "k", "v", "g", "beta", "do"):
        e[n][:, dirty] = float("nan")
    d, e, opt = ({n: dev(x) for n, x in y.items()} for y in (d, e, opt))
    o = torch.zeros_like(d["v"])
    o2 = torch.zeros_like(o)
    S, S2 = call(d, opt, cu_seqlens=i32(cu), o=o)[1], call(e, opt, cu_seqlens=i32(cu), o=o2)[1]
    assert torch.equal(o, o2) and torch.equal(S, S2) and not o2[:, dirty].any()
    a, b = grads(d, opt, cu_seqlens=i32(cu)), grads(e, opt, cu_seqlens=i32(cu))
    for n in a:
        assert torch.equal(a[n], b[n]), n
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        assert not b[n][:, dirty].any(), n


def test_garbage_outside_long_sequences():
    d, opt = make(1, 3000, 1, 2, 64, 64, "bf16", n_seqs=3, raw=True)
    cu = [37, 1500, 1500, 2900]
    e = {n: x.clone() for n, x in d.items()}
    for n in ("q", "k", "v", "g", "beta"):
        e[n][:, :37] = e[n][:, 2900:] = float("nan")
    d, e, opt = ({n: dev(x) for n, x in y.items()} for y in (d, e, opt))
    o, o2 = torch.zeros_like(d["v"]), torch.zeros_like(d["v"])
    S, S2 = call(d, opt, cu_seqlens=i32(cu), o=o)[1], call(e, opt, cu_seqlens=i32(cu), o=o2)[1]
    assert torch.equal(o, o2) and torch.equal(S, S2) and torch.equal(S[1], d["S0"][1])
    assert not o[:, :37].any() and not o[:, 2900:].any()


def test_garbage_in_padding_rows_and_free_pages():
    d, _ = on_gpu(1, 8, 2, 4, 64, 64, io="bf16")
    x, S, slots = decode_case(d, 8, [2, -1, 0, 7, 2, 1 << 30, -(1 << 31), 1], 4)
    S[3] = float("nan")  # nobody's
    y = [t.clone() for t in x]
    for t in y:
        t[[1, 3, 5, 6]] = float("nan")
    S2 = S.clone()
    o, o2 = kda.kda_gdr_decode(*x, S, slots), kda.kda_gdr_decode(*y, S2, slots)
    assert torch.equal(o, o2) and torch.equal(S[:3], S2[:3]) and not o2[[1, 3, 5, 6]].any()


# ------------------------------------------------------------------ streams and graphs
def test_on_another_stream():
    d, opt = on_gpu(2, 333, 2, 4, 64, 128, io="bf16", raw=True)
    o, S = call(d, opt)
    g = grads(d, opt)
    x, P, slots = decode_case(d, 6, [1, 0, 1, -1, 3, 2], 4)
    od = kda.kda_gdr_decode(*x, P, slots)
    refs = i32([1, 1, 0, 0])
    dst, left = kda.kda_pages_fork(P[None], refs, i32([0, 1]))
    P2 = torch.zeros_like(P)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        P2.zero_()
        s.wait_stream(torch.cuda.current_stream())
        # memory that kernels on the current stream are still writing, freed at once: the
        # calls' own tensors may come from it
        for _ in range(20):
            torch.full((64 << 20,), 3.0, device="cuda")
        o2, S2 = call(d, opt, stream=stream)
        g2 = grads(d, opt, stream=stream)
        od2 = kda.kda_gdr_decode(*x, P2, slots, stream=stream)
        dst2, left2 = kda.kda_pages_fork(P2[None], refs, i32([0, 1]), stream=stream)
        s.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(S, S2) and torch.equal(od, od2) and torch.equal(P, P2)
        assert all(torch.equal(g[n], g2[n]) for n in g)
        assert torch.equal(dst, dst2) and torch.equal(left, left2)


def test_two_calls_at_once():
    a, oa = on_gpu(1, 700, 2, 4, 128, 128, io="bf16", seed=1)
    b, ob = on_gpu(1, 2300, 1, 2, 128, 64, io="bf16", seed=2)
    want = call(a, oa), call(b, ob), grads(a, oa)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(4):
        got = call(a, oa, stream=s), call(b, ob, stream=t), grads(a, oa, stream=s)
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for x, y in zip(w.values() if isinstance(w, dict) else w, g.values() if isinstance(g, dict) else g):
            assert torch.equal(x, y)


def test_captured_and_replayed():
    """A prompt, its gradients, the state into a pool, a fork and tokens on both pages,
    as one graph: every replay on new inputs against the eager calls."""
    d, opt = on_gpu(1, 200, 2, 4, 64, 64, io="bf16", raw=True)
    pool = torch.zeros(1, 5, 4, 64, 64, device="cuda")
    refs = i32([0, 1, 0, 0, 0])
    out_refs, n = torch.empty_like(refs), 3

    def run():
        o, S = call(d, opt)
        g = grads(d, opt)
        pool.zero_()
        pool[0, 1].copy_(S[0])
        dst, _ = kda.kda_pages_fork(pool, refs, i_src, refs_out=out_refs)
        x = [d[m][0, :n].contiguous() for m in ("q", "k", "v", "g", "beta")]
        od = kda.kda_gdr_decode(*x, pool[0], slots, **opt)
        used = kda.kda_pages_compact(pool, out_refs)
        return [o, S, dst, od, pool, out_refs, *used[:3], *g.values()]

    i_src, slots = i32([1, -1]), i32([0, 1, 2])
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = run()
    for seed in range(4):
        e, _ = on_gpu(1, 200, 2, 4, 64, 64, io="bf16", raw=True, seed=10 + seed)
        for m in d:
            d[m].copy_(e[m])
        refs.copy_(i32([0, 1 + seed, 0, seed % 2, 0]))
        graph.replay()
        got = [x.clone() for x in kept]
        want = run()
        torch.cuda.synchronize()
        for i, (x, y) in enumerate(zip(got, want)):
            assert torch.equal(x, y), (seed, i)


def test_split_walks_captured_and_replayed():
    """Long rows of few heads, equal and packed: the segments' tables, maps and starts are
    made anew by every replay."""
    d, opt = on_gpu(1, 3000, 1, 2, 64, 64, io="bf16", raw=True)
    e, _ = on_gpu(1, 3000, 1, 2, 64, 64, io="bf16", raw=True, n_seqs=2)
    cu = i32([0, 1400, 3000])

    def run():
        o, S = call(d, opt)
        o2, S2 = call({**d, "S0": e["S0"]}, opt, cu_seqlens=cu)
        return [o, S, o2, S2, *grads(d, opt).values()]

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = run()
    for seed, at in enumerate([10, 1700, 2999]):
        x, _ = on_gpu(1, 3000, 1, 2, 64, 64, io="bf16", raw=True, seed=20 + seed)
        for m in d:
            d[m].copy_(x[m])
        cu.copy_(i32([0, at, 3000]))
        graph.replay()
        got = [y.clone() for y in kept]
        want = run()
        torch.cuda.synchronize()
        for i, (y, w) in enumerate(zip(got, want)):
            assert torch.equal(y, w), (seed, i)


def test_two_graphs_with_their_own_workspaces():
    cases = [on_gpu(1, 150 + 900 * i, 1, 2, 64, 64, io="bf16", seed=i) for i in range(2)]
    graphs = []
    for d, opt in cases:
        want = call(d, opt)
        torch.cuda.synchronize()
        need = kda.kda_gdr_prefill_workspace_bytes(kda.gdr_args(*[d[n] for n in NAMES], *want))
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        o, S = torch.empty_like(want[0]), torch.empty_like(want[1])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(d, opt, o=o, S_T=S, workspace=ws)
        graphs.append((g, o, S, want, torch.cuda.Stream()))
    for _ in range(3):
        for g, o, S, _, s in graphs:
            o.zero_()
            S.zero_()
            s.wait_stream(torch.cuda.current_stream())
        for g, _, _, _, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for _, o, S, want, _ in graphs:
            assert torch.equal(o, want[0]) and torch.equal(S, want[1])


# ------------------------------------------------------------------ large offsets
def test_rows_far_apart():
    """q, k, v in rows of 2^23 elements: the last tokens lie 2^31 elements in."""
    T = 300
    d, opt = on_gpu(1, T, 1, 2, 64, 64, io="bf16")
    want, wg = call(d, opt), grads(d, opt)
    row = torch.empty(1, T, 1 << 23, dtype=torch.bfloat16, device="cuda")
    e, at = dict(d), (1 << 23) - 512
    for n in ("q", "k", "v"):
        w = d[n][0, 0].numel()
        e[n] = row[..., at:at + w].unflatten(-1, d[n].shape[2:])
        e[n].copy_(d[n])
        at += w
    got, gg = call(e, opt), grads(e, opt)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert all(torch.equal(gg[n], wg[n]) for n in wg)


def test_large_pool():
    """Slots and pages past 2^31 elements of a pool."""
    pool = torch.empty(2, 2200, 32, 128, 128, device="cuda")  # 9.2 GB, 1.15e9 elements a layer
    d, _ = on_gpu(1, 3, 16, 32, 128, 128, io="bf16")
    x, S, _ = decode_case(d, 3, [0], 3)
    S.normal_()
    far = pool.flatten(0, 1)[2 * 2200 - 5:]
    far[[4, 0, 2]] = S
    o = kda.kda_gdr_decode(*x, S, i32([0, 1, 2]))
    o2 = kda.kda_gdr_decode(*x, pool.flatten(0, 1), i32([4399, 4395, 4397]))
    assert torch.equal(o, o2) and torch.equal(far[[4, 0, 2]], S)
    refs = torch.ones(2200, dtype=torch.int32, device="cuda")
    refs[2190] = 0
    pool[0, 2199], pool[1, 2190] = 1.5, 0
    dst, _ = kda.kda_pages_fork(pool, refs, i32([2199]))
    assert dst.item() == 2190 and torch.equal(pool[:, 2190], pool[:, 2199]) and (pool[0, 2190] == 1.5).all()


def test_long_row():
    """Outputs and gradients past 2^31 elements: the end of one long row against that end
    by itself, from the state before it (chunks begin at the same tokens)."""
    T, cut, Hv = 66048, 65536, 256
    g = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    d = dict(q=rnd(1, T, 1, 32), k=rnd(1, T, 1, 32), v=rnd(1, T, Hv, 128), g=-rnd(1, T, Hv).abs() * 0.1,
             beta=rnd(1, T, Hv).sigmoid(), S0=None, do=rnd(1, T, Hv, 128),
             dS_T=torch.randn(1, Hv, 32, 128, generator=g, device="cuda"))
    assert d["v"].numel() > 1 << 31
    o, S = call(d, {})
    head = {n: (x[:, :cut].contiguous() if n in ("q", "k", "v", "g", "beta") else x) for n, x in d.items()}
    Sc = call(head, {})[1]
    del head
    tail = {n: (x if n in ("S0", "dS_T") else x[:, cut:].contiguous()) for n, x in d.items()}
    tail["S0"] = Sc
    o2, S2 = call(tail, {})
    assert torch.equal(o[:, cut:], o2) and torch.equal(S, S2)
    a, b = grads(d, {}), grads(tail, {})
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        assert torch.equal(a[n][:, cut:], b[n]), n


# ------------------------------------------------------------------ a layer's two passes
@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_layer_forward_and_gradients_through_the_convolution(io):
    """kda_conv_norm (short convolution, SiLU, norm) before this rule, as a layer runs
    them, against the same chain in float64 (the rule then takes the rows as given)."""
    B, T, H, D = 2, 90, 2, 64
    d, _ = make(B, T, H, H, D, D, io)
    g = torch.Generator().manual_seed(5)
    w = torch.randn(3, H * D, 4, generator=g) * 0.5
    out = kda.kda_conv_norm(dev(d["q"]), dev(d["k"]), dev(d["v"]), dev(w))
    q, k, v = out[:3]
    o, S = kda.kda_gdr_prefill(q, k, v, dev(d["g"]), dev(d["beta"]), dev(d["S0"]), l2norm_qk=False)
    e = dict(d, q=q.cpu(), k=k.cpu(), v=v.cpu())
    ro, rS = ref.gdr_reference(*[num(e[n]) for n in NAMES], l2=False)
    assert rel(o, ro) <= OUT[io]
    check_backward(e, {}, io, l2=False)
