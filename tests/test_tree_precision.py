"""How exactly the rule over trees is computed, as an error of whole outputs.

The bounds of tests/tree_ref.py are of the worst case, value by value: a kernel that lost its third bf16 part would still
keep them.  Here the 2-norm of what o and u are off, over the norm of the 64-bit result, is held to what the tensor-core
kernel's sums lose.  Its accumulators are fp32 and cut towards zero what they add up, after every 16 products: by
half a unit of the last place on average, which is 0.36 * 2^-23 of a value (half of the mean of 2^-23 / m over mantissas
m of 1 .. 2, evenly in their logarithm), always in the same direction, so steps add up.  o and u take d / 16 steps at the
size of S_0^T k or q (the small parts come first), and 6 ceil(n / 16) more on top of those.  What the parts leave out is
under 2^-21 of a product each, a third of that on average, and counts as one step more; fp32 sums on CUDA cores round and
lose less.

On the CPU the kernel's products are done in numpy, part by part and step by step with such accumulators: they keep the
limit, and do not if a part or a product is left out, so the limit finds that."""

import numpy as np
import pytest

from tests import gpu_util as gu
from tests import tree_ref as tr

KINDS = ("draft", "chain", "deep", "forest")
# parts of R and of T and W, 0 the largest, in the order the kernel adds their products
PRODUCTS = ((2, 0), (1, 1), (0, 2), (1, 0), (0, 1), (0, 0))


def limit(d, n):
    return 0.36 * 2.0 ** -23 * (d // 16 + 6 * -(-n // 16) + 1)


def off(got, want):
    return np.linalg.norm(got - want) / np.linalg.norm(want)


# --- the kernel's arithmetic on the CPU ----------------------------------------------------------------------

def cut(x):
    """To the 16 upper bits of a float."""
    return (x.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)


def split(x):
    x = np.ascontiguousarray(x, dtype=np.float32)
    hi = cut(x)
    mid = cut(x - hi)
    return hi, mid, cut(x - hi - mid)


def to_bf16(x):
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32)
    return ((u + np.uint32(0x7FFF) + (u >> np.uint32(16) & np.uint32(1))) & np.uint32(0xFFFF0000)).view(np.float32)


def towards_zero(x):
    y = x.astype(np.float32)
    far = np.abs(y.astype(np.float64)) > np.abs(x)
    y[far] = np.nextafter(y[far], np.float32(0))
    return y.astype(np.float64)


def accumulate(acc, pairs):
    """acc + the products of pairs (a, b), 16 inner values at a time."""
    for a, b in pairs:
        for k in range(0, a.shape[1], 16):
            acc = towards_zero(acc + a[:, k:k + 16].astype(np.float64) @ b[k:k + 16].astype(np.float64))
    return acc


def as_the_kernel(parents, q, k, v, g, beta, state, state_parts=(2, 1, 0), products=PRODUCTS):
    """o and u of one V head, [n, d]; N, P, T and W in 64 bits and rounded once, the two large products as they are made."""
    n, d = v.shape
    paths = tr.paths(parents)
    total = np.array([g[a].sum() for a in paths])
    grown = np.exp(total)[:, None]
    nn, pp = np.zeros((n, n)), np.zeros((n, n))
    for j, a in enumerate(paths):
        f = np.exp(total[j] - total[a])
        nn[j, a], pp[j, a] = beta[j] * f * (k[a] @ k[j]), f * (k[a] @ q[j])
        nn[j, j] = 0.0
    t = np.linalg.inv(np.eye(n) + nn)
    x = accumulate(np.zeros((d, 2 * n)), [(split(state)[p].T, np.r_[k, q].T) for p in state_parts]).T
    r = (beta[:, None] * (v - grown * x[:n])).astype(np.float32)
    rs, ts = split(r), split(np.r_[t - np.eye(n), pp @ t])
    out = np.r_[r, (grown * x[n:]).astype(np.float32)].T.astype(np.float64)
    out = accumulate(out, [(rs[a].T, ts[b].T) for a, b in products]).T
    return out[n:], out[:n]


def inputs(rng, n, d, kind):
    q, k = rng.standard_normal((2, n, d))
    q, k = (to_bf16(x / np.linalg.norm(x, axis=1, keepdims=True)).astype(np.float64) for x in (q, k))
    return (tr.make(rng, n, kind), q, k, to_bf16(rng.standard_normal((n, d))).astype(np.float64),
            -rng.uniform(0.001, 0.3, n), rng.uniform(0.3, 1.0, n), 0.5 * rng.standard_normal((d, d)).astype(np.float32))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,n", [(128, 24), (128, 64), (64, 41), (32, 24), (32, 64)])
def test_the_limit_finds_what_is_left_out(d, n, kind):
    x = inputs(np.random.default_rng(d + n), n, d, kind)
    wo, wu = tr.rule(*x[:6], x[6].astype(np.float64))[:2]
    o, u = as_the_kernel(*x)
    assert off(o, wo) <= limit(d, n) and off(u, wu) <= limit(d, n)
    faults = [dict(state_parts=(1, 0))]  # S_0 in two parts
    faults += [dict(products=[p for p in PRODUCTS if p != gone]) for gone in PRODUCTS]
    faults += [dict(products=[p for p in PRODUCTS if sum(p) < 2])]  # two parts of R, T and W
    faults += [dict(products=[(a, 1 if b == 2 else b) for a, b in PRODUCTS])]  # the wrong part
    for fault in faults:
        o, _ = as_the_kernel(*x, **fault)
        assert off(o, wo) > limit(d, n), fault


# --- on the GPU ----------------------------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,n_tok", [(128, 24), (128, 64), (64, 41), (32, 24), (32, 64), (64, 64)])
def test_outputs_as_a_whole(d, n_tok, dtype):
    torch = gu.require_gpu()
    from tests.test_gpu_attn import f64, no_error
    from tests.test_gpu_tree_rule import Batch

    rng = np.random.default_rng(d + n_tok)
    b = Batch(rng, [tr.make(rng, n_tok, kind) for kind in KINDS], 2, 4, d, dtype, g_max=0.3)
    b.beta.copy_(0.3 + 0.7 * b.beta)
    o, u = b.run()
    torch.cuda.synchronize()
    no_error()
    wo, wu, _, _ = b.want()
    o, u = f64(o), f64(u)
    for s, kind in enumerate(KINDS):
        r = slice(s * n_tok, (s + 1) * n_tok)
        for h in range(4):
            for got, want, what in ((o, wo, "o"), (u, wu, "u")):
                assert off(got[r, h], want[r, h]) <= limit(d, n_tok), (kind, h, what)
