"""Tree operators on the GPU at the edges of what their documentation allows."""

import numpy as np
import pytest

import gated_deltanet_scan_gb300 as gdr
from tests import gpu_util as gu
from tests import tree_ref as tr
from tests.test_gpu_attn import Paged, ints, no_error, randn
from tests.test_gpu_tree_attn import attend, parents_of

pytestmark = pytest.mark.gpu

TREE = [-1, -1, 1, 0, 2, -2, 4, 3]


@pytest.mark.parametrize("layers", [0, 3])
@pytest.mark.parametrize("stale,last", [
    ([-1, 0, 1, 2, 3, 4, 5, 6], 7), ([-2] * 8, 3), ([9, -7, 1 << 30, 3, 4, 5, -(1 << 31), 7], -1), (TREE, 1 << 30), (TREE, -9),
])
def test_compaction_of_a_batch_with_empty_places(stale, last, layers):
    """A sequence of no tokens is not in the batch: whatever its parents and last node hold, nothing is recorded, its
    new length is 0, and the others' rows move as they do without it."""
    torch = gu.require_gpu()
    rng = np.random.default_rng(61)
    c = Paged(rng, [40, 24, 30], 8, 2, 64, "bf16")
    if layers:
        c.k, c.v = (torch.stack([x + i for i in range(layers)]) for x in (c.k, c.v))
    k0, v0 = c.k.clone(), c.v.clone()

    def run(lens, trees, nodes):
        c.k.copy_(k0), c.v.copy_(v0)
        out = ints([-9] * 3)
        gdr.gdr_attn_commit_tree(c.k, c.v, c.table, ints(lens), parents_of(trees), ints(nodes), out)
        torch.cuda.synchronize()
        return c.k.clone(), c.v.clone(), out.tolist()

    want = run([40, 24, 30], [TREE, TREE, TREE], [6, -1, 7])
    no_error()
    got = run([40, 0, 30], [TREE, stale, TREE], [6, last, 7])
    no_error()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and got[2] == [36, 0, 25]
    assert not torch.equal(got[0], k0)


def test_one_workspace_for_trees_of_several_sizes():
    """The bytes do not grow with every token of a tree: a buffer of the largest of the sizes' bytes serves them all."""
    torch = gu.require_gpu()
    rng = np.random.default_rng(62)
    c = Paged(rng, [700, 64, 0, 3000], 16, 2, 128, "bf16")
    sizes = (24, 4, 5, 1, 17, 64, 16)
    calls = []
    for n_tok in sizes:
        parents = parents_of([tr.make(rng, n_tok, kind) for kind in ("draft", "chain", "holes", "forest")])
        calls.append((randn(rng, (4 * n_tok, 8, 128), "bf16"), parents))
    need = [gdr.gdr_attn_decode_tree_workspace_bytes(q, c.k, p) for q, p in calls]
    assert need[1] > need[0]
    ws = torch.full((max(need),), 255, dtype=torch.uint8, device="cuda")
    for (q, p), size in zip(calls, need):
        want, lse = attend(c, q, p)
        got, lse2 = attend(c, q, p, workspace=ws)
        assert torch.equal(got, want) and torch.equal(lse, lse2)
        attend(c, q, p, workspace=ws[:size])
        with pytest.raises(gdr.GdrError):
            attend(c, q, p, workspace=ws[:size - 1])
    no_error()


def test_example_verifies_and_accepts_trees():
    import importlib.util
    import os

    torch = gu.require_gpu()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_decode.py")
    spec = importlib.util.spec_from_file_location("hybrid_decode", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    tokens, one, lens, want = mod.run_tree(lengths=(130, 61))
    no_error()
    assert lens == want and tokens.shape == one.shape == (7, mod.WIDTH)
    assert torch.isfinite(tokens).all() and torch.isfinite(one).all()
