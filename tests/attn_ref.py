"""Attention, the position rotation and the paged append in 64 bits (numpy), from
their definitions, with the error bounds the GPU tests assert.

A 16-bit rounding is off by at most h = eps / 2 of the value (bf16 2^-8, fp16
2^-11).  For one output row, with weights p_j and A_x = sum_j p_j |v_jx|:
  - the scores are fp32 sums of d exact products: off by at most
    g = d 2^-24 max_j scale sum_x |q_x k_jx|, which moves every weight by a factor
    within exp(+-g) and their sum likewise;
  - the weights enter the product with v rounded to 16 bits: h of each;
  - exponentials, sums over the tokens (in any order, split and joined) and the
    division: 2^-16 covers 2^-22 each for exp2 and its argument, and fp32 sums of up
    to a few hundred rounded partial results;
  - the output is rounded once: h |o|.
So |o - o*| <= h |o*| + (1 + h) (h + 2 g + 2^-16) A, and lse is off by g + 2^-16 + 2^-22 |lse|.
"""

from __future__ import annotations

import numpy as np

HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
SMALLEST = {"bf16": 2.0 ** -133, "f16": 2.0 ** -25}  # half the spacing of subnormals


def attend(q, k, v, scale, seen, dtype):
    """One head: q [n, d], k, v [m, d]; query i sees tokens [0, seen[i]).
    Returns o, lse and their bounds."""
    n, d = q.shape
    o, bo = np.zeros((n, v.shape[1])), np.zeros((n, v.shape[1]))
    lse, bl = np.full(n, -np.inf), np.zeros(n)
    h = HALF[dtype]
    for i in range(n):
        m = max(0, int(seen[i]))
        if m == 0:
            continue
        x = scale * (k[:m] @ q[i])
        top = x.max()
        w = np.exp(x - top)
        l = w.sum()
        p = w / l
        o[i] = p @ v[:m]
        lse[i] = top + np.log(l)
        g = d * 2.0 ** -24 * abs(scale) * np.max(np.abs(k[:m]) @ np.abs(q[i]))
        a = p @ np.abs(v[:m])
        bo[i] = h * np.abs(o[i]) + (1 + h) * (h + 2 * g + 2.0 ** -16) * a + SMALLEST[dtype]
        bl[i] = g + 2.0 ** -16 + 2.0 ** -22 * abs(lse[i])
    return o, lse, bo, bl


def prefill(q, k, v, scale, lens, dtype):
    """Packed prompts: q [T, h_q, d]; k, v [T, h_kv, d]."""
    o, bo = np.zeros(q.shape), np.zeros(q.shape)
    lse, bl = np.zeros(q.shape[:2]), np.zeros(q.shape[:2])
    group = q.shape[1] // k.shape[1]
    t = 0
    for n in lens:
        for h in range(q.shape[1]):
            r = slice(t, t + n)
            o[r, h], lse[r, h], bo[r, h], bl[r, h] = attend(q[r, h], k[r, h // group], v[r, h // group], scale,
                                                           np.arange(1, n + 1), dtype)
        t += n
    return o, lse, bo, bl


def gather(cache, table, n):
    """The first n tokens of one sequence: cache [pages, page, h, d], table one row of page ids."""
    page = cache.shape[1]
    pos = np.arange(n)
    return cache[table[pos // page], pos % page]


def decode(q, k_cache, v_cache, table, lens, n_tok, scale, dtype):
    o, bo = np.zeros(q.shape), np.zeros(q.shape)
    lse, bl = np.zeros(q.shape[:2]), np.zeros(q.shape[:2])
    group = q.shape[1] // k_cache.shape[2]
    for s, n in enumerate(lens):
        k, v = gather(k_cache, table[s], n), gather(v_cache, table[s], n)
        r = slice(s * n_tok, (s + 1) * n_tok)
        for h in range(q.shape[1]):
            o[r, h], lse[r, h], bo[r, h], bl[r, h] = attend(q[r, h], k[:, h // group], v[:, h // group], scale,
                                                           n - n_tok + np.arange(1, n_tok + 1), dtype)
    return o, lse, bo, bl


def rotate(x, pos, inv_freq, interleaved):
    """x [n, heads, d] at positions pos [n]; the rotated rows and |x| + |y| of every value's pair."""
    r = len(inv_freq)
    out, size = x.copy(), np.zeros(x.shape)
    one = slice(0, 2 * r, 2) if interleaved else slice(0, r)
    two = slice(1, 2 * r, 2) if interleaved else slice(r, 2 * r)
    angle = (np.asarray(pos, np.float64)[:, None] * inv_freq.astype(np.float64))[:, None, :]
    a, b = x[..., one], x[..., two]
    out[..., one] = a * np.cos(angle) - b * np.sin(angle)
    out[..., two] = a * np.sin(angle) + b * np.cos(angle)
    size[..., one] = size[..., two] = np.abs(a) + np.abs(b)
    return out, size


def rotate_bound(out, size, dtype, rot):
    """One 16-bit rounding, and of the pair's size: cos and sin of an fp32 angle within half a turn (2^-24 of
    pi, and 2^-23 each for their values) and two fp32 products and a sum: 2^-20 covers them.  Copied values are
    exact."""
    b = HALF[dtype] * np.abs(out) + 2.0 ** -20 * size + SMALLEST[dtype]
    b[..., rot:] = 0.0
    return b
