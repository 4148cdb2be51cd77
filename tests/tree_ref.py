"""Trees of drafted tokens in 64 bits (numpy), from the definitions, with the error bounds the GPU tests assert.

A tree is a list of parents: -1 a child of the last committed token, an earlier row, -2 no node.

Bounds of the rule.  Every product of two inputs is exact in fp32 or summed with at most 2^-23 of each term lost a
step (a tensor core may cut what it adds): GAMMA = 2 (128 + 64 + 16) 2^-24 covers an inner size of 128, a path's
sum of 64, and the exponentials, norms and sigmoids, each a few 2^-24.  With N and P of the paths, T = (I + N)^-1 and
bars for absolute values throughout (N-bar from |beta| and |k| . |k|, and so on),
    R-bar = |beta| (|v| + e^G |S|^T |k|),   Y = |T| R-bar
a relative error GAMMA of every N, P, T and R moves u by at most GAMMA (Y + |T| N-bar Y) and o by at most
GAMMA (e^G |S|^T |q| + P-bar Y + P-bar |T| N-bar Y), to first order; a bf16 output adds its rounding, 2^-8 |o|.
The committed state e^G S + sum w k u^T is off by at most GAMMA of its terms' absolute values.
"""

from __future__ import annotations

import numpy as np

from tests import attn_ref as ar

GAMMA = 2 * (128 + 64 + 16) * 2.0 ** -24


def make(rng, n, kind):
    """Parents of one tree of n rows."""
    if kind == "chain":
        return [j - 1 for j in range(n)]
    if kind == "star":
        return [-1 if j == 0 else 0 for j in range(n)]
    if kind == "roots":
        return [-1] * n
    if kind == "none":
        return [-2] * n
    if kind == "forest":
        return [int(rng.integers(-1, j)) if j else -1 for j in range(n)]
    if kind == "binary":
        return [(j - 1) // 2 if j else -1 for j in range(n)]
    if kind == "deep":  # mostly a chain
        return [max(-1, j - 1 - int(rng.integers(0, 3) == 0) * int(rng.integers(0, 3))) for j in range(n)]
    if kind == "holes":  # rows that are no nodes among the others
        out, nodes = [], []
        for j in range(n):
            if rng.random() < 0.3:
                out.append(-2)
            else:
                out.append(int(rng.choice([-1] + nodes)))
                nodes.append(j)
        return out
    real = n if kind == "draft" else max(1, n - int(rng.integers(0, n)))  # "padded"
    return [int(rng.integers(0, j)) if j else -1 for j in range(real)] + [-2] * (n - real)


def paths(parents):
    """A_j as sorted lists, empty where the row is no node (a bad parent makes it none)."""
    out = []
    for j, p in enumerate(parents):
        ok = p == -1 or (0 <= p < j and out[p])
        out.append((out[p] if p >= 0 else []) + [j] if ok else [])
    return out


def rule(parents, q, k, v, g, beta, state):
    """One sequence and V head: q, k, v [n, d]; g, beta [n]; state [d, d].  o, u and their bounds, and every
    node's state."""
    n, d = v.shape
    p = paths(parents)
    o, u = np.zeros((n, d)), np.zeros((n, d))
    states = [None] * n
    for j in range(n):
        if not p[j]:
            continue
        old = np.exp(g[j]) * (state if parents[j] < 0 else states[parents[j]])
        u[j] = beta[j] * (v[j] - old.T @ k[j])
        states[j] = old + np.outer(k[j], u[j])
        o[j] = states[j].T @ q[j]
    real = [j for j in range(n) if p[j]]
    bu, bo = np.zeros((n, d)), np.zeros((n, d))
    if real:
        total = np.array([g[a].sum() for a in p])
        nn, nb, pb = np.zeros((n, n)), np.zeros((n, n)), np.zeros((n, n))
        for j in real:
            f = np.exp(total[j] - total[p[j]])
            pb[j, p[j]] = f * (np.abs(k[p[j]]) @ np.abs(q[j]))
            nn[j, p[j]] = beta[j] * f * (k[p[j]] @ k[j])
            nb[j, p[j]] = abs(beta[j]) * f * (np.abs(k[p[j]]) @ np.abs(k[j]))
            nn[j, j] = nb[j, j] = 0.0
        t = np.abs(np.linalg.inv(np.eye(n) + nn))
        grown = np.exp(total)[:, None]
        qz, kz = (np.where([[bool(x)] for x in p], y, 0.0) for y in (q, k))
        r = np.where([[bool(x)] for x in p], np.abs(beta)[:, None] * (np.abs(v) + grown * (np.abs(kz) @ np.abs(state))), 0.0)
        y = t @ r
        bu = GAMMA * (y + t @ nb @ y)
        bo = GAMMA * (grown * (np.abs(qz) @ np.abs(state)) + pb @ y + pb @ t @ nb @ y)
    return o, u, bo, bu, states


def settle(parents, last, k, g, u, state):
    """The state after node `last` from the corrections, and its bound."""
    path = paths(parents)[last] if last >= 0 else []
    out, size = state.copy(), np.abs(state)
    for j in path:
        out = np.exp(g[j]) * out + np.outer(k[j], u[j])
        size = np.exp(g[j]) * size + np.outer(np.abs(k[j]), np.abs(u[j]))
    return out, (GAMMA * size if path else np.zeros_like(size))


def attend(parents, q, k_cache, v_cache, table, lens, scale, dtype):
    """q [n * n_tok, h_q, d], parents [n][n_tok]; o, lse and their bounds."""
    n_tok = len(parents[0])
    o, bo = np.zeros(q.shape), np.zeros(q.shape)
    lse, bl = np.full(q.shape[:2], -np.inf), np.zeros(q.shape[:2])
    group = q.shape[1] // k_cache.shape[2]
    for s, m in enumerate(lens):
        if m < n_tok:
            continue
        k, v = ar.gather(k_cache, table[s], m), ar.gather(v_cache, table[s], m)
        for j, path in enumerate(paths(parents[s])):
            if not path:
                continue
            seen = np.r_[0:m - n_tok, [m - n_tok + i for i in path]].astype(np.int64)
            r = s * n_tok + j
            for h in range(q.shape[1]):
                x = ar.attend(q[r, h][None], k[seen, h // group], v[seen, h // group], scale, [len(seen)], dtype)
                o[r, h], lse[r, h], bo[r, h], bl[r, h] = (y[0] for y in x)
    return o, lse, bo, bl
