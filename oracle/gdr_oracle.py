"""Plain float64 statement of the gated delta rule with one decay per head, token by
token, with reverse-mode gradients and the page operations on pools.  Test
infrastructure only: it shares no code with the library.

    S_t = e^{g_t} (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,  o_t = scale S_t^T q_t
"""
from __future__ import annotations

import numpy as np


def _l2(x, eps):
    return x / np.sqrt((x * x).sum(-1, keepdims=True) + eps)


def gdr_gates(g, beta, A_log=None, dt_bias=None, beta_logits=False):
    g, beta = np.asarray(g, np.float64), np.asarray(beta, np.float64)
    if A_log is not None:
        g = -np.exp(np.asarray(A_log, np.float64)) * np.logaddexp(g + np.asarray(dt_bias, np.float64), 0.0)
    if beta_logits:
        beta = 1.0 / (1.0 + np.exp(-beta))
    return g, beta


def gdr_token(S, q, k, v, g, beta, scale):
    """One token of every head: S [H, Dk, Dv], q, k [H, Dk], v [H, Dv], g, beta [H]."""
    X = S * np.exp(g)[:, None, None]
    y = v - np.einsum("hkv,hk->hv", X, k)
    X = X + k[:, :, None] * (beta[:, None] * y)[:, None, :]
    return X, scale * np.einsum("hkv,hk->hv", X, q)


def gdr_sequence(q, k, v, g, beta, S0=None, *, scale=1.0, l2=True, eps=1e-6, A_log=None, dt_bias=None,
                 beta_logits=False):
    """One sequence: q, k [T, Hk, Dk], v [T, Hv, Dv], g, beta [T, Hv]; returns o, S_T."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    g, beta = gdr_gates(g, beta, A_log, dt_bias, beta_logits)
    T, Hk, Dk = q.shape
    Hv, Dv = v.shape[1:]
    if l2:
        q, k = _l2(q, eps), _l2(k, eps)
    q, k = (np.repeat(x, Hv // Hk, axis=1) for x in (q, k))
    S = np.zeros((Hv, Dk, Dv)) if S0 is None else np.array(S0, np.float64)
    o = np.zeros((T, Hv, Dv))
    for t in range(T):
        S, o[t] = gdr_token(S, q[t], k[t], v[t], g[t], beta[t], scale)
    return o, S


def gdr_sequence_backward(q, k, v, g, beta, S0, do, dS_T, *, scale=1.0, l2=True, eps=1e-6, A_log=None,
                          dt_bias=None, beta_logits=False):
    """Gradients of <o, do> + <S_T, dS_T> of one sequence, the recurrence reversed
    step by step: dict of dq, dk, dv, dg, dbeta, dS0 (and dA_log, ddt_bias)."""
    raw_q, raw_k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    raw_g, raw_b = np.asarray(g, np.float64), np.asarray(beta, np.float64)
    g, beta = gdr_gates(g, beta, A_log, dt_bias, beta_logits)
    do = np.asarray(do, np.float64)
    T, Hk, Dk = raw_q.shape
    Hv, Dv = v.shape[1:]
    rep = Hv // Hk
    qh, kh = (_l2(raw_q, eps), _l2(raw_k, eps)) if l2 else (raw_q, raw_k)
    qr, kr = (np.repeat(x, rep, axis=1) for x in (qh, kh))
    S = np.zeros((Hv, Dk, Dv)) if S0 is None else np.array(S0, np.float64)
    states = [S]
    for t in range(T):
        S, _ = gdr_token(S, qr[t], kr[t], v[t], g[t], beta[t], scale)
        states.append(S)
    dS = np.zeros((Hv, Dk, Dv)) if dS_T is None else np.array(dS_T, np.float64)
    dq, dk, dv = np.zeros((T, Hv, Dk)), np.zeros((T, Hv, Dk)), np.zeros((T, Hv, Dv))
    dg, db = np.zeros((T, Hv)), np.zeros((T, Hv))
    for t in reversed(range(T)):
        a = np.exp(g[t])[:, None, None]
        X = states[t] * a
        y = v[t] - np.einsum("hkv,hk->hv", X, kr[t])
        u = beta[t][:, None] * y
        dq[t] = scale * np.einsum("hkv,hv->hk", states[t + 1], do[t])
        dS = dS + scale * qr[t][:, :, None] * do[t][:, None, :]
        du = np.einsum("hkv,hk->hv", dS, kr[t])
        db[t] = (du * y).sum(-1)
        dy = beta[t][:, None] * du
        dv[t] = dy
        dk[t] = np.einsum("hkv,hv->hk", dS, u) - np.einsum("hkv,hv->hk", X, dy)
        dX = dS - kr[t][:, :, None] * dy[:, None, :]
        dg[t] = (dX * X).sum((-1, -2))
        dS = a * dX
    dq, dk = (x.reshape(T, Hk, rep, Dk).sum(2) for x in (dq, dk))

    def through(x, d):
        if not l2:
            return d
        n = np.sqrt((x * x).sum(-1, keepdims=True) + eps)
        return d / n - x * (x * d).sum(-1, keepdims=True) / n ** 3

    out = dict(dq=through(raw_q, dq), dk=through(raw_k, dk), dv=dv, dS0=dS)
    if A_log is not None:
        rate = np.exp(np.asarray(A_log, np.float64))
        z = raw_g + np.asarray(dt_bias, np.float64)
        df = -rate * dg / (1.0 + np.exp(-z))
        out["dA_log"], out["ddt_bias"] = (dg * g).sum(0), df.sum(0)
        dg = df
    if beta_logits:
        db = db * beta * (1.0 - beta)
    out["dg"], out["dbeta"] = dg, db
    return out


def _sequences(q, cu):
    B, T = q.shape[:2]
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    return [(0, int(s), int(e)) for s, e in zip(cu[:-1], cu[1:])]


def gdr_reference(q, k, v, g, beta, S0=None, *, cu_seqlens=None, **kw):
    """A batch [B, T, ...], or packed sequences: returns o, S_T."""
    o = np.zeros(v.shape)
    S = []
    for i, (b, s, e) in enumerate(_sequences(q, cu_seqlens)):
        o[b, s:e], St = gdr_sequence(q[b, s:e], k[b, s:e], v[b, s:e], g[b, s:e], beta[b, s:e],
                                     None if S0 is None else S0[i], **kw)
        S.append(St)
    return o, np.stack(S)


def gdr_reference_backward(q, k, v, g, beta, S0, do, dS_T, *, cu_seqlens=None, **kw):
    out = dict(dq=np.zeros(q.shape), dk=np.zeros(k.shape), dv=np.zeros(v.shape), dg=np.zeros(g.shape),
               dbeta=np.zeros(beta.shape))
    states, sums = [], {}
    for i, (b, s, e) in enumerate(_sequences(q, cu_seqlens)):
        d = gdr_sequence_backward(q[b, s:e], k[b, s:e], v[b, s:e], g[b, s:e], beta[b, s:e],
                                  None if S0 is None else S0[i], do[b, s:e],
                                  None if dS_T is None else dS_T[i], **kw)
        for n in out:
            out[n][b, s:e] = d[n]
        states.append(d["dS0"])
        for n in ("dA_log", "ddt_bias"):
            if n in d:
                sums[n] = sums.get(n, 0) + d[n]
    return dict(out, dS0=np.stack(states), **sums)


def gdr_reference_decode(q, k, v, g, beta, S, slots, o, *, scale=1.0, l2=True, eps=1e-6, A_log=None,
                         dt_bias=None, beta_logits=False):
    """Rows in order, each a token of its slot's sequence; rows outside the pool keep
    their o.  Returns o, S."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    g, beta = gdr_gates(g, beta, A_log, dt_bias, beta_logits)
    S, o = np.array(S, np.float64), np.array(o, np.float64)
    if l2:
        q, k = _l2(q, eps), _l2(k, eps)
    rep = v.shape[1] // q.shape[1]
    for i, s in enumerate(slots):
        if 0 <= s < len(S):
            S[s], o[i] = gdr_token(S[s], np.repeat(q[i], rep, 0), np.repeat(k[i], rep, 0), v[i], g[i],
                                   beta[i], scale)
    return o, S


# ------------------------------------------------------------------ pages
def pages_fork(pool, refs, src):
    """pool [layers, pages, ...]; returns pool, dst, refs."""
    pool, refs, before, old, dst = pool.copy(), list(refs), list(refs), pool, []
    for s in src:
        free = [p for p, r in enumerate(refs) if r <= 0]
        if not (s == -1 or (0 <= s < len(refs) and before[s] > 0)) or not free:
            dst.append(-1)
            continue
        refs[free[0]] = 1
        pool[:, free[0]] = old[:, s] if s >= 0 else 0
        dst.append(free[0])
    return pool, dst, refs


def pages_free(refs, pages):
    refs = list(refs)
    for p in pages:
        if 0 <= p < len(refs) and refs[p] > 0:
            refs[p] -= 1
    return refs


def pages_compact(pool, refs, table):
    """Returns pool, n_used, new_id, refs, table."""
    pool, refs = pool.copy(), list(refs)
    n_used = sum(r > 0 for r in refs)
    new_id = [p if r > 0 else -1 for p, r in enumerate(refs)]
    holes = [p for p in range(n_used) if refs[p] <= 0]
    for p in range(n_used, len(refs)):
        if refs[p] > 0:
            to = holes.pop(0)
            pool[:, to] = pool[:, p]
            refs[to], new_id[p] = refs[p], to
        refs[p] = 0
    table = [new_id[t] if 0 <= t < len(refs) else -1 for t in table]
    return pool, n_used, new_id, refs, table


def pages_copy(src_pool, dst_pool, src, dst, same):
    """Returns the destination pool and which pairs were copied."""
    n_src, n_dst = src_pool.shape[1], dst_pool.shape[1]
    inside = [-1 <= s < n_src and 0 <= d < n_dst for s, d in zip(src, dst)]
    taken = {d for d, ok in zip(dst, inside) if ok}
    out, done, seen = dst_pool.copy(), [], set()
    for s, d, ok in zip(src, dst, inside):
        first = ok and d not in seen
        if ok:
            seen.add(d)
        good = first and not (same and s >= 0 and s in taken)
        if good:
            out[:, d] = src_pool[:, s] if s >= 0 else 0
        done.append(int(good))
    return out, done
