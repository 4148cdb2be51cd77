"""The reference of the tree operators against other definitions of the same, and a model of how the rule's kernel
joins blocks of levels (no GPU needed)."""

import numpy as np
import pytest

import oracle
from tests import attn_ref as ar
from tests import tree_ref as tr

KINDS = ("chain", "star", "roots", "none", "forest", "binary", "deep", "holes", "draft", "padded")


def inputs(rng, n, d):
    q, k = (x / np.linalg.norm(x, axis=1, keepdims=True) for x in rng.standard_normal((2, n, d)))
    return q, k, rng.standard_normal((n, d)), -rng.uniform(0.01, 2, n), rng.uniform(0, 1, n), 0.3 * rng.standard_normal((d, d))


def test_a_chain_is_the_sequential_rule():
    rng = np.random.default_rng(1)
    n, d = 12, 16
    q, k, v, g, beta, s0 = inputs(rng, n, d)
    f32 = [np.float32(x) for x in (q, k, v, g, beta, s0)]
    o, _, _, _, states = tr.rule(tr.make(rng, n, "chain"), *(x.astype(np.float64) for x in f32))
    want, s = oracle.gdr_sequential(np.array([0, n]), f32[0][:, None], f32[1][:, None], f32[2][:, None], f32[3][:, None],
                                    f32[4][:, None], f32[5][None, None].astype(np.float64))
    assert np.allclose(o, want[:, 0], rtol=0, atol=1e-10) and np.allclose(states[-1], s[0, 0], rtol=0, atol=1e-10)


@pytest.mark.parametrize("kind", KINDS)
def test_every_node_is_its_path_by_itself(kind):
    rng = np.random.default_rng(2)
    n, d = 23, 8
    parents = tr.make(rng, n, kind)
    q, k, v, g, beta, s0 = inputs(rng, n, d)
    o, u, bo, bu, states = tr.rule(parents, q, k, v, g, beta, s0)
    for j, path in enumerate(tr.paths(parents)):
        if not path:
            assert not o[j].any() and not u[j].any()
            continue
        x = [y[path] for y in (q, k, v, g, beta)]
        alone = tr.rule(list(range(-1, len(path) - 1)), *x, s0)
        assert np.allclose(alone[0][-1], o[j], atol=1e-12) and np.allclose(alone[1][-1], u[j], atol=1e-12)
        s, _ = tr.settle(parents, j, k, g, u, s0)
        assert np.allclose(s, states[j], atol=1e-12)
    assert np.all(bo >= 0) and np.all(bu >= 0)


def test_attention_of_a_chain_is_decode():
    rng = np.random.default_rng(3)
    page, n_tok, lens = 5, 4, [4, 17, 0, 9]
    cache = rng.standard_normal((2, 20, page, 2, 8))
    table = rng.permutation(20)[:16].reshape(4, 4)
    q = rng.standard_normal((4 * n_tok, 4, 8))
    chain = [tr.make(rng, n_tok, "chain")] * 4
    for a, b in zip(tr.attend(chain, q, *cache, table, lens, 0.3, "bf16"),
                    ar.decode(q, *cache, table, lens, n_tok, 0.3, "bf16")):
        assert np.allclose(a[np.isfinite(b)], b[np.isfinite(b)])
        assert np.array_equal(np.isfinite(a), np.isfinite(b))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [1, 2, 17, 64])
def test_joins_of_blocks_of_levels_give_the_inverse(kind, n):
    """The kernel's way to T = (I + N)^-1: with b = 1, 2, 4, ..., entry (t, j) whose levels differ first in bit b is
    -sum_s T_ts Y_sj over t's odd block, Y_sj = sum_i N_si T_ij over j's even block; lists and their order as there."""
    rng = np.random.default_rng(n)
    p = tr.paths(tr.make(rng, n, kind))
    nn = np.zeros((n, n))
    for j, path in enumerate(p):
        nn[j, path[:-1]] = rng.uniform(-1, 1, max(0, len(path) - 1))
    t, y = np.zeros((n, n)), np.zeros((n, n))
    done, b = 0, 1
    deepest = max(len(x) for x in p) - 1
    while b <= deepest:
        mine = [(j, r) for j, path in enumerate(p) for r in range(len(path) - 1) if b <= (len(path) - 1 ^ r) < 2 * b]
        assert len(mine) == sum(b for path in p if path and len(path) - 1 & b)
        for j, r in mine:
            path = p[j]
            i = path[r]
            y[j, i] = nn[j, i] + sum(nn[j, path[x]] * t[path[x], i] for x in range(r + 1, (r | b - 1) + 1))
        for j, r in mine:
            path = p[j]
            i, d = path[r], len(path) - 1
            t[j, i] = -(y[j, i] + sum(t[j, path[x]] * y[path[x], i] for x in range(d & -b, d)))
        done += len(mine)
        b *= 2
    assert done == sum(max(0, len(x) - 1) for x in p)
    assert np.allclose(t + np.eye(n), np.linalg.inv(np.eye(n) + nn), atol=1e-9 * max(1.0, np.abs(t).max()))
