"""Page operations on pools against their statement (oracle/gdr_oracle.py): moved
bytes, counts and indexes are exact.  And a server's run of them with the gated
delta rule: prompts into pages, forks, tokens, frees, a compaction, more tokens."""
import numpy as np
import pytest
import torch

import gated_delta_rule_80_amd as kda
from oracle import gdr_oracle as ref

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def pool_of(layers, pages, shape, seed=0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-999, 999, (layers, pages, *shape), generator=g).to(dtype)


SHAPES = [((4,), 1), ((5, 4), 3), ((3, 32, 32), 2), ((2, 64, 65, 4), 1)]


@pytest.mark.parametrize("shape,layers", SHAPES, ids=str)
@pytest.mark.parametrize("n_pages", [1, 2, 9, 70])
def test_fork(shape, layers, n_pages):
    rng = np.random.default_rng(n_pages)
    for trial in range(3):
        pool = pool_of(layers, n_pages, shape, trial)
        refs = rng.integers(-1, 3, n_pages).tolist() if trial else [0] * n_pages
        src = rng.integers(-2, n_pages + 2, rng.integers(1, 2 * n_pages + 2)).tolist()
        p = pool.cuda()
        dst, out = kda.kda_pages_fork(p, i32(refs), i32(src))
        wp, wd, wr = ref.pages_fork(pool.numpy(), refs, src)
        assert dst.tolist() == wd and out.tolist() == wr and np.array_equal(p.cpu().numpy(), wp)


def test_fork_in_place_counts_and_layer_stride():
    whole = pool_of(3, 12, (16,), dtype=torch.int32)
    p = whole.cuda()
    pool = p[:, :8]  # layers further apart than the pages need
    refs = i32([1, 0, 0, 2, 0, 1, 0, 0])
    dst, out = kda.kda_pages_fork(pool, refs, i32([3, 3, 0, -1, 4]), refs_out=refs)
    wp, wd, wr = ref.pages_fork(whole[:, :8].numpy(), [1, 0, 0, 2, 0, 1, 0, 0], [3, 3, 0, -1, 4])
    assert out is refs and dst.tolist() == wd and refs.tolist() == wr
    assert np.array_equal(p[:, :8].cpu().numpy(), wp) and torch.equal(p[:, 8:].cpu(), whole[:, 8:])


def test_many_pages():
    """Lists longer than the planning workgroup."""
    n = 5000
    rng = np.random.default_rng(0)
    pool, refs = pool_of(1, n, (8,)), (rng.random(n) < 0.4).astype(int).tolist()
    src = rng.integers(-1, n, 2500).tolist()
    p = pool.cuda()
    dst, out = kda.kda_pages_fork(p, i32(refs), i32(src))
    wp, wd, wr = ref.pages_fork(pool.numpy(), refs, src)
    assert dst.tolist() == wd and out.tolist() == wr and np.array_equal(p.cpu().numpy(), wp)
    gone = rng.integers(-3, n + 3, 6000).tolist()
    freed = kda.kda_pages_free(out, i32(gone))
    wf = ref.pages_free(wr, gone)
    assert freed.tolist() == wf
    table = rng.integers(-2, n + 2, 70000).tolist()
    count, new, refs2, tab = kda.kda_pages_compact(p, freed, i32(table))
    cp, cn, ci, cr, ct = ref.pages_compact(wp, wf, table)
    assert count.item() == cn and new.tolist() == ci and refs2.tolist() == cr and tab.tolist() == ct
    assert np.array_equal(p.cpu().numpy(), cp)


def test_free():
    refs = [0, 1, 5, 2, -3]
    assert kda.kda_pages_free(i32(refs), i32([1, 1, 2, 2, 2, 9, -1, 0, 4])).tolist() == [0, 0, 2, 2, -3]
    r = i32(refs)
    assert kda.kda_pages_free(r, i32([]), refs_out=r).tolist() == refs
    assert kda.kda_pages_free(i32([3] * 3000), i32([7] * 5000)).tolist() == [3] * 7 + [0] + [3] * 2992


@pytest.mark.parametrize("refs", [[0, 0, 0], [1, 1, 1], [0, 0, 2], [1, 0, 3, 0, 0, 7, 1, 0, 2], [5], [0]], ids=str)
def test_compact(refs):
    pool = pool_of(2, len(refs), (3, 4))
    table = list(range(-1, len(refs) + 1))
    p, r, t = pool.cuda(), i32(refs), i32(table)
    count, new, out, tab = kda.kda_pages_compact(p, r, t, refs_out=r, table_out=t)
    wp, wn, wi, wr, wt = ref.pages_compact(pool.numpy(), refs, table)
    assert count.item() == wn and new.tolist() == wi and r.tolist() == wr and t.tolist() == wt
    assert np.array_equal(p.cpu().numpy()[:, :wn], wp[:, :wn])
    count, _, out, none = kda.kda_pages_compact(p, r)
    assert none is None and count.item() == wn and out.tolist() == wr


def test_copy():
    a, b = pool_of(2, 6, (8,), 1), pool_of(2, 9, (8,), 2)
    src, dst = [0, 5, -1, 6, 3, 3, -2, 2], [8, 1, 2, 3, 1, 9, 4, 0]
    pa, pb = a.cuda(), b.cuda()
    done = kda.kda_pages_copy(pa, pb, i32(src), i32(dst))
    want, wd = ref.pages_copy(a.numpy(), b.numpy(), src, dst, False)
    assert done.tolist() == wd and np.array_equal(pb.cpu().numpy(), want) and torch.equal(pa.cpu(), a)
    # within one pool: a chain, a swap and a page onto itself are left out
    src, dst = [0, 1, 3, 4, 5, 2], [1, 2, 4, 3, 5, 0]
    done = kda.kda_pages_copy(pa, pa, i32(src), i32(dst))
    want, wd = ref.pages_copy(a.numpy(), a.numpy(), src, dst, True)
    assert done.tolist() == wd and np.array_equal(pa.cpu().numpy(), want)
    src, dst = [0, 0, -1], [4, 5, 1]
    done = kda.kda_pages_copy(pa, pa, i32(src), i32(dst))
    want, wd = ref.pages_copy(want, want, src, dst, True)
    assert done.tolist() == wd == [1, 1, 1] and np.array_equal(pa.cpu().numpy(), want)


def test_serving_run():
    """Two prompts in one packed prefill, their states into pages, a request forked,
    everybody decodes, one is freed, the pool compacted, and decoding goes on."""
    Hk, Hv, D, T = 1, 2, 64, 150
    g = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    draw = lambda n: [rnd(n, Hk, D), rnd(n, Hk, D), rnd(n, Hv, D), -rnd(n, Hv).abs() * 0.3,  # noqa: E731
                      torch.sigmoid(rnd(n, Hv))]
    cuda = lambda x: [y.cuda() for y in x]  # noqa: E731
    num = lambda x: [y.double().numpy() for y in x]  # noqa: E731
    pool = torch.zeros(1, 8, Hv, D, D, device="cuda")
    refs = i32([1, 0, 2, 0, 0, 0, 0, 0])  # others hold pages 0 and 2

    x = draw(T)
    cu = [0, 67, T]
    o, S = kda.kda_gdr_prefill(*[y[None] for y in cuda(x)], cu_seqlens=i32(cu))
    ro, rS = ref.gdr_reference(*[y[None] for y in num(x)], cu_seqlens=cu)
    pages, refs = kda.kda_pages_fork(pool, refs, i32([-1, -1]))
    assert pages.tolist() == [1, 3]
    assert kda.kda_pages_copy(S[None], pool, i32([0, 1]), pages).tolist() == [1, 1]
    beam, refs = kda.kda_pages_fork(pool, refs, pages[:1].contiguous())
    assert beam.tolist() == [4]
    states = np.stack([rS[0], rS[1], rS[0]])

    x = draw(3)
    o = kda.kda_gdr_decode(*cuda(x), pool[0], torch.cat([pages, beam]))
    ro, states = ref.gdr_reference_decode(*num(x), states, [0, 1, 2], np.zeros((3, Hv, D)))
    tol = 2048 * 2.0 ** -24  # float32 throughout: a prefill's bound and a token's
    err = lambda a, b: np.linalg.norm(a.double().cpu().numpy() - b) / np.linalg.norm(b)  # noqa: E731
    assert err(o, ro) <= tol

    refs = kda.kda_pages_free(refs, pages[:1].contiguous())  # the first request is done
    count, new, refs, table = kda.kda_pages_compact(pool, refs, torch.cat([pages[1:], beam]))
    assert count.item() == 4 and table.tolist() == [3, 1] and refs.tolist() == [1, 1, 2, 1, 0, 0, 0, 0]
    x = draw(2)
    o = kda.kda_gdr_decode(*cuda(x), pool[0], table)
    ro, states = ref.gdr_reference_decode(*num(x), states[1:], [0, 1], np.zeros((2, Hv, D)))
    assert err(o, ro) <= tol and err(pool[0, table.long()], states) <= tol
