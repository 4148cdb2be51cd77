"""Attention operators: what the host checks let through and what they refuse, at the borders (no GPU needed)."""

import pytest

import gated_deltanet_scan_gb300 as gdr
from tests.test_attn_refusals import A, BAD, L, OK, append, cache, decode, dims, prefill, rows  # noqa: F401


def test_empty_batches_need_no_addresses(L):
    """Tensors of no rows have a null address."""
    none, no_cache = rows(ptr=None), cache(k=None, v=None, page_table=None, n_pages=0)
    tensors = dict(q=none, k=none, v=none)
    for n in (0, 2):
        assert prefill(L, n=n, t=0, cu=None, o=none, **tensors) == OK
        assert append(L, n=n, t=0, cu=None, qo=none, ko=none, c=no_cache, lens=None, inv=None, **tensors) == OK
    assert decode(L, n=0, q=none, o=none, c=no_cache, lens=None, ws=None, wsb=0) == OK
    # the sizes are still looked at
    assert append(L, d=dims(h_q=15), n=0, t=0) == BAD and append(L, n=0, t=0, rot=3) == BAD
    assert decode(L, n=0, n_tok=17) == BAD
