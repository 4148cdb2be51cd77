"""gdr_attn_commit_tree's new lengths: what they would overlap, or could not be told from, is refused on the host (no GPU
needed)."""

import pytest

import gated_deltanet_scan_gb300 as gdr
from gated_deltanet_scan_gb300 import build as gbuild
from tests.test_tree_refusals import BAD, UNSUP, attn_dims, cache

LENS, LAST, PARENTS = 0x200000, 0x300000, 0x400000


@pytest.fixture(scope="module")
def L():
    gbuild.build()
    return gdr.lib()


@pytest.mark.parametrize("n,n_tok", [(1, 1), (5, 24), (300, 64)])
def test_new_lengths_must_not_overlap_what_is_read(L, n, n_tok):
    def compact(lens_out):
        # more layers than a launch takes: what passes the lengths' check is refused for them
        return L.gdr_attn_commit_tree(attn_dims(), n, n_tok, PARENTS, LAST, 1 << 20, 6553600, cache(), LENS, lens_out, None)

    for at, count in ((LENS, n), (LAST, n), (PARENTS, n * n_tok)):
        for off in (-4 * (n - 1), 0, 4 * (count - 1)):
            assert compact(at + off) == BAD, (hex(at), off)
        for off in (-4 * n, 4 * count):
            assert compact(at + off) == UNSUP, (hex(at), off)


def test_no_layers_give_no_lengths(L):
    torch = pytest.importorskip("torch")
    i32 = torch.int32
    none = torch.zeros(0, 5, 16, 2, 64, dtype=torch.bfloat16)
    args = none, none.clone(), torch.zeros(2, 3, dtype=i32), torch.full((2,), 7, dtype=i32), \
        torch.full((2, 3), -1, dtype=i32), torch.zeros(2, dtype=i32)
    gdr.gdr_attn_commit_tree(*args)
    with pytest.raises(ValueError):
        gdr.gdr_attn_commit_tree(*args, torch.zeros(2, dtype=i32))
