"""Pins for the float64 statement of the per-head gated delta rule and of the page
operations: values by hand, the matrix form, the per-channel rule where both agree,
and every gradient against central differences.  CPU only."""
import numpy as np
import pytest

from oracle import gdr_oracle as ref
from oracle import kda_reference


def case(rng, T=7, Hk=2, Hv=4, Dk=5, Dv=3, raw=False):
    x = rng.standard_normal
    d = dict(q=x((T, Hk, Dk)), k=x((T, Hk, Dk)), v=x((T, Hv, Dv)), g=-np.abs(x((T, Hv))),
             beta=1 / (1 + np.exp(-x((T, Hv)))), S0=x((Hv, Dk, Dv)))
    opt = {}
    if raw:
        d["g"], d["beta"] = x((T, Hv)), x((T, Hv))
        opt = dict(A_log=x(Hv) * 0.5, dt_bias=x(Hv), beta_logits=True)
    return d, opt


def test_one_token_by_hand():
    # S0 = [[1, 2], [3, 4]], decay 1/2, k = (1, 0), v = (2, 0), beta = 1/2, q = (1, 1):
    # S_bar = [[.5, 1], [1.5, 2]], y = v - (.5, 1) = (1.5, -1), S = S_bar + (1, 0) (.75, -.5)
    o, S = ref.gdr_sequence(*(np.array(a, float) for a in ([[[1, 1]]], [[[1, 0]]], [[[2, 0]]], [[np.log(0.5)]], [[0.5]],
                                                           [[[1, 2], [3, 4]]])), scale=2.0, l2=False)
    np.testing.assert_allclose(S[0], [[1.25, 0.5], [1.5, 2.0]], atol=1e-15)
    np.testing.assert_allclose(o[0, 0], [5.5, 5.0], atol=1e-15)


def test_matrix_form_and_shared_heads():
    d, _ = case(np.random.default_rng(0))
    o, S = ref.gdr_sequence(**d, scale=0.3)
    for h in range(4):
        X = d["S0"][h]
        for t in range(7):
            k, q = (d[n][t, h // 2] / np.sqrt((d[n][t, h // 2] ** 2).sum() + 1e-6) for n in ("k", "q"))
            b = d["beta"][t, h]
            X = np.exp(d["g"][t, h]) * (np.eye(5) - b * np.outer(k, k)) @ X + b * np.outer(k, d["v"][t, h])
            np.testing.assert_allclose(o[t, h], 0.3 * X.T @ q, atol=1e-12)
        np.testing.assert_allclose(S[h], X, atol=1e-12)


def test_agrees_with_the_rule_with_a_decay_per_channel():
    rng = np.random.default_rng(1)
    d, _ = case(rng, Hk=3, Hv=3, Dk=4, Dv=4)
    o, S = ref.gdr_sequence(**d)
    b = {n: x[None] for n, x in d.items()}
    b["g"] = np.repeat(b["g"][..., None], 4, -1)
    S0 = b.pop("S0")
    ko, kS, _ = kda_reference(b["q"], b["k"], b["v"], b["g"], b["beta"], conv_w=None, S0=S0, l2norm_qk=True)
    np.testing.assert_allclose(o, ko[0], atol=1e-12)
    np.testing.assert_allclose(S, kS[0], atol=1e-12)


def test_gates():
    g, b = ref.gdr_gates([[0.0, 800.0]], [[0.0, -700.0]], np.log([2.0, 3.0]), np.zeros(2), True)
    np.testing.assert_allclose(g, [[-2 * np.log(2), -2400.0]], rtol=1e-14)
    np.testing.assert_allclose(b, [[0.5, 0.0]], atol=1e-300)


def test_state_is_handed_on():
    d, opt = case(np.random.default_rng(2), raw=True)
    o, S = ref.gdr_sequence(**d, **opt)
    head = {n: x[:3] for n, x in d.items() if n != "S0"}
    tail = {n: x[3:] for n, x in d.items() if n != "S0"}
    o1, S1 = ref.gdr_sequence(**head, S0=d["S0"], **opt)
    o2, S2 = ref.gdr_sequence(**tail, S0=S1, **opt)
    np.testing.assert_allclose(np.concatenate([o1, o2]), o, atol=1e-14)
    np.testing.assert_allclose(S2, S, atol=1e-14)


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("l2", [True, False])
def test_gradients_against_differences(raw, l2):
    """Central differences with step h: error h^2 |f'''| / 6 + 2^-52 |f| / h, about
    1e-9 for h = 1e-5 and values and derivatives below a few tens."""
    rng = np.random.default_rng(3)
    d, opt = case(rng, T=5, raw=raw)
    if not l2:
        d["q"], d["k"] = d["q"] * 0.4, d["k"] * 0.4
    do, dS = rng.standard_normal((5, 4, 3)), rng.standard_normal((4, 5, 3))
    kw = dict(scale=0.7, l2=l2)

    def loss(x, y):
        o, S = ref.gdr_sequence(**x, **y, **kw)
        return (o * do).sum() + (S * dS).sum()

    got = ref.gdr_sequence_backward(d["q"], d["k"], d["v"], d["g"], d["beta"], d["S0"], do, dS, **opt, **kw)
    h = 1e-5
    for where, names in ((d, list(d)), (opt, [n for n in opt if n != "beta_logits"])):
        for n in names:
            for i in np.ndindex(where[n].shape):
                old = where[n][i]
                where[n][i] = old + h
                up = loss(d, opt)
                where[n][i] = old - h
                down = loss(d, opt)
                where[n][i] = old
                assert abs(got["d" + n][i] - (up - down) / (2 * h)) < 1e-7, (n, i)


def test_packed_and_decode_agree_with_sequences():
    rng = np.random.default_rng(4)
    d, _ = case(rng, T=9)
    S0 = rng.standard_normal((4, 4, 5, 3))
    b = {n: x[None] for n, x in d.items() if n != "S0"}
    o, S = ref.gdr_reference(**b, S0=S0, cu_seqlens=[0, 4, 4, 5, 8])
    o1, S1 = ref.gdr_sequence(**{n: x[0, 5:8] for n, x in b.items()}, S0=S0[3])
    np.testing.assert_array_equal(o[0, 5:8], o1)
    np.testing.assert_array_equal(S[3], S1)
    np.testing.assert_array_equal(S[1], S0[1])
    assert not o[0, 8].any()
    # token by token on a pool, the rows of two sequences interleaved, one row padding
    rows = [5, 0, 6, 8, 1, 7, 2, 3]
    slots = [2, 0, 2, -1, 0, 2, 0, 0]
    od, Sd = ref.gdr_reference_decode(*(d[n][rows] for n in ("q", "k", "v", "g", "beta")), S0[[0, 1, 3]], slots,
                                      np.full((8, 4, 3), 7.0))
    np.testing.assert_allclose(od[[0, 2, 5]], o1, atol=1e-14)
    np.testing.assert_allclose(Sd, S[[0, 1, 3]], atol=1e-14)
    assert (od[3] == 7).all()


def test_pages_by_hand():
    pool = np.arange(5.0)[None, :, None] + np.zeros((2, 5, 1))
    out, dst, refs = ref.pages_fork(pool, [1, 0, 2, -1, 0], [2, 3, 7, 0, -1, -1, 2])
    assert dst == [1, -1, -1, 3, 4, -1, -1] and refs == [1, 1, 2, 1, 1]
    assert out[0, :, 0].tolist() == [0, 2, 2, 0, 0]
    assert ref.pages_free([1, 2, 0, 1], [1, 1, 1, 2, 0, 9, -1]) == [0, 0, 0, 1]
    out, used, new, refs, tab = ref.pages_compact(pool, [0, 3, 0, 1, 1], [1, 3, 4, 0, -1, 9])
    assert used == 3 and new == [-1, 1, -1, 0, 2] and refs == [1, 3, 1, 0, 0] and tab == [1, 0, 2, -1, -1, -1]
    assert out[1, :3, 0].tolist() == [3, 1, 4]
    out, done = ref.pages_copy(pool, pool, [0, 1, 4, -1, 9, 2], [3, 3, 0, 2, 1, 8], True)
    # page 0 is written by the third pair, so the first is left out, and with it its page
    assert done == [0, 0, 1, 1, 0, 0] and out[0, :, 0].tolist() == [4, 1, 0, 3, 4]
