"""The 64-bit attention reference against closed forms and brute force (CPU)."""

import numpy as np
import pytest

from tests import attn_ref as ar


def test_equal_scores_give_running_means():
    rng = np.random.default_rng(0)
    v = rng.standard_normal((7, 3, 8))
    q, k = rng.standard_normal((7, 3, 8)), np.zeros((7, 3, 8))
    o, lse, _, _ = ar.prefill(q, k, v, 0.3, [4, 0, 3], "bf16")
    for t0, n in ((0, 4), (4, 3)):
        for i in range(n):
            assert np.allclose(o[t0 + i], v[t0:t0 + i + 1].mean(0))
            assert np.allclose(lse[t0 + i], np.log(i + 1))


def test_grouped_heads_and_brute_force():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((5, 6, 4)), rng.standard_normal((5, 2, 4)), rng.standard_normal((5, 2, 4))
    o, lse, _, _ = ar.prefill(q, k, v, 0.5, [5], "f16")
    for i in range(5):
        for h in range(6):
            w = [np.exp(0.5 * sum(q[i, h, x] * k[j, h // 3, x] for x in range(4))) for j in range(i + 1)]
            want = sum(w[j] * v[j, h // 3] for j in range(i + 1)) / sum(w)
            assert np.allclose(o[i, h], want) and np.allclose(lse[i, h], np.log(sum(w)))


def test_decode_of_the_last_tokens_is_the_prompts_rows():
    rng = np.random.default_rng(2)
    n, n_tok, page = 11, 4, 3
    q, k, v = (rng.standard_normal((n, h, 8)) for h in (4, 2, 2))
    cache_k, cache_v = np.full((6, page, 2, 8), np.nan), np.full((6, page, 2, 8), np.nan)
    table = np.array([[4, 1, 5, 0]])
    for p in range(n):
        cache_k[table[0, p // page], p % page], cache_v[table[0, p // page], p % page] = k[p], v[p]
    want = ar.prefill(q, k, v, 0.35, [n], "bf16")
    got = ar.decode(q[-n_tok:], cache_k, cache_v, table, [n], n_tok, 0.35, "bf16")
    for w, g in zip(want, got):
        assert np.allclose(w[-n_tok:], g)
    # fewer tokens than queries: the first queries see nothing
    o, lse, _, _ = ar.decode(q[-n_tok:], cache_k, cache_v, table, [2], n_tok, 0.35, "bf16")
    assert np.all(o[:2] == 0) and np.all(np.isneginf(lse[:2])) and np.all(np.isfinite(lse[2:]))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_turns_pairs_and_keeps_the_rest(interleaved):
    x = np.random.default_rng(3).standard_normal((3, 2, 10))
    inv = np.array([1.0, 0.25, 0.01], dtype=np.float32)
    out, _ = ar.rotate(x, [0, 5, 1000003], inv, interleaved)
    assert np.array_equal(out[0], x[0]) and np.array_equal(out[..., 6:], x[..., 6:])
    one, two = (slice(0, 6, 2), slice(1, 6, 2)) if interleaved else (slice(0, 3), slice(3, 6))
    z = (x[..., one] + 1j * x[..., two]) * np.exp(1j * np.array([0, 5, 1000003])[:, None, None] * inv.astype(float))
    assert np.allclose(out[..., one], z.real) and np.allclose(out[..., two], z.imag)
