"""Bytes of gdr_attn_decode_tree's workspace, as its documentation has them (no GPU needed)."""

import pytest

import gated_deltanet_scan_gb300 as gdr
from gated_deltanet_scan_gb300 import build as gbuild


@pytest.fixture(scope="module")
def L():
    gbuild.build()
    return gdr.lib()


@pytest.mark.parametrize("h_q,h_kv,d", [(16, 4, 256), (32, 8, 128), (12, 3, 64), (64, 1, 128), (2, 2, 64)])
def test_bytes_grow_with_sequences_and_not_always_with_tokens(L, h_q, h_kv, d):
    dims = gdr.gdr_attn_dims(h_q, h_kv, d, gdr.GDR_BF16, 0.1)
    for n_tok in range(1, 65):
        need = [L.gdr_attn_decode_tree_workspace_bytes(dims, n, n_tok) for n in range(1, 200)]
        assert all(a <= b for a, b in zip(need, need[1:])), n_tok
    most = 16 // (h_q // h_kv)  # tokens of up to 16 rows
    if most >= 1:
        few, more = (L.gdr_attn_decode_tree_workspace_bytes(dims, 8, n) for n in (most, most + 1))
        assert few > more
