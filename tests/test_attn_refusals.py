"""Attention operators: bad arguments are refused on the host before any launch, by
the C ABI and by the binding (no GPU needed)."""

import ctypes

import pytest

import gated_deltanet_scan_gb300 as gdr
from gated_deltanet_scan_gb300 import build as gbuild

A = 0x100000  # a 16-byte aligned stand-in address: validation never dereferences it
BAD, UNSUP, OK = gdr.GDR_ERR_INVALID_ARG, gdr.GDR_ERR_UNSUPPORTED, gdr.GDR_OK


@pytest.fixture(scope="module")
def L():
    gbuild.build()
    return gdr.lib()


def dims(**kw):
    d = dict(h_q=16, h_kv=4, d=256, dtype=gdr.GDR_BF16, scale=0.0625)
    d.update(kw)
    return gdr.gdr_attn_dims(**d)


def rows(ptr=A, ts=4096, hs=256):
    return gdr.gdr_rows(ptr, ts, hs)


def cache(**kw):
    c = dict(k=A, v=A, page_stride=65536, token_stride=1024, head_stride=256, page_table=A, table_stride=8,
             n_pages=100, page_size=64, max_pages=8)
    c.update(kw)
    return gdr.gdr_kv_cache(**c)


def append(L, d=None, n=2, cu=A, t=10, q=None, k=None, v=None, qo=None, ko=None, c=None, lens=A, inv=A, rot=64, il=0):
    r = rows()
    return L.gdr_attn_append(d or dims(), n, cu, t, q or r, k or r, v or r, qo or r, ko, c or cache(), lens, inv, rot,
                             il, None)


def prefill(L, d=None, n=2, cu=A, t=10, q=None, k=None, v=None, o=None, lse=None):
    r = rows()
    return L.gdr_attn_prefill(d or dims(), n, cu, t, q or r, k or r, v or r, o or r, lse, None)


def decode(L, d=None, n=2, n_tok=1, q=None, c=None, lens=A, o=None, lse=None, ws=A, wsb=1 << 40):
    r = rows()
    return L.gdr_attn_decode(d or dims(), n, n_tok, q or r, c or cache(), lens, o or r, lse, ws, wsb, None)


@pytest.mark.parametrize("bad,code", [
    (dict(h_q=0), BAD), (dict(h_kv=0), BAD), (dict(h_q=15), BAD), (dict(d=0), BAD), (dict(dtype=3), BAD),
    (dict(dtype=-1), BAD), (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD),
    (dict(dtype=gdr.GDR_F32), UNSUP), (dict(d=96), UNSUP), (dict(d=512), UNSUP), (dict(h_q=4 * 129), UNSUP),
    (dict(h_q=65536, h_kv=65536), UNSUP),
])
def test_dims(L, bad, code):
    for call in (append, prefill, decode):
        assert call(L, d=dims(**bad)) == code
    assert L.gdr_attn_decode_workspace_bytes(dims(**bad), 2, 1) == 0


@pytest.mark.parametrize("bad", [rows(ptr=None), rows(ptr=A + 8), rows(ts=-8), rows(ts=4100), rows(hs=-256),
                                 rows(hs=1), rows(ts=1 << 40)])
def test_rows(L, bad):
    for name in ("q", "k", "v", "qo", "ko"):
        assert append(L, **{name: bad}) == BAD, name
    for name in ("q", "k", "v", "o"):
        assert prefill(L, **{name: bad}) == BAD, name
    for name in ("q", "o"):
        assert decode(L, **{name: bad}) == BAD, name


@pytest.mark.parametrize("bad", [
    dict(k=None), dict(v=A + 2), dict(page_table=None), dict(page_table=A + 2), dict(page_stride=12),
    dict(token_stride=-8), dict(head_stride=4), dict(n_pages=0), dict(page_size=0), dict(max_pages=0),
    dict(table_stride=-1), dict(page_size=1 << 16, max_pages=1 << 15), dict(page_size=1, max_pages=(1 << 31) - 1023),
])
def test_cache(L, bad):
    assert append(L, c=cache(**bad)) == BAD
    assert decode(L, c=cache(**bad)) == BAD


def test_counts_and_pointers(L):
    for call in (append, prefill):
        assert call(L, n=-1) == BAD and call(L, t=-1) == BAD and call(L, n=0, t=3) == BAD
        assert call(L, n=0, t=0) == OK and call(L, t=0) == OK
        assert call(L, t=1 << 31) == UNSUP
        assert call(L, cu=A + 2) == BAD
    assert prefill(L, cu=None) == BAD
    assert append(L, cu=None, n=3, t=10) == BAD  # not the same number of tokens each
    assert prefill(L, lse=A + 1) == BAD and decode(L, lse=A + 2) == BAD
    assert append(L, lens=None) == BAD and append(L, lens=A + 1) == BAD and decode(L, lens=None) == BAD
    assert append(L, rot=3) == BAD and append(L, rot=-2) == BAD and append(L, rot=258) == BAD
    assert append(L, inv=None) == BAD and append(L, inv=A + 2) == BAD
    for n_tok in (0, 17, -1):
        assert decode(L, n_tok=n_tok) == BAD
    assert decode(L, n=-1) == BAD and decode(L, n=0) == OK


def test_queries_come_with_their_output_and_in_place_rows_match(L):
    r = rows()
    call = lambda q, qo: L.gdr_attn_append(dims(), 2, A, 10, q, r, r, qo, None, cache(), A, A, 64, 0, None)
    assert call(r, None) == BAD and call(None, r) == BAD
    assert call(r, rows(ts=8192)) == BAD  # the same pointer, other rows
    assert append(L, ko=rows(hs=512)) == BAD


def test_decode_workspace(L):
    need = L.gdr_attn_decode_workspace_bytes(dims(), 64, 1)
    assert L.gdr_attn_decode_workspace_bytes(dims(), 0, 1) == 0
    for n_tok in (0, 17):
        assert L.gdr_attn_decode_workspace_bytes(dims(), 2, n_tok) == 0
    if need:
        assert decode(L, n=64, ws=None) == BAD and decode(L, n=64, ws=A + 8) == BAD
        assert decode(L, n=64, wsb=need - 1) == BAD


def test_binding_refuses(L):
    torch = pytest.importorskip("torch")
    bf = torch.bfloat16
    q, k = torch.zeros(6, 4, 64, dtype=bf), torch.zeros(6, 2, 64, dtype=bf)
    cu, lens = torch.tensor([0, 4, 6], dtype=torch.int32), torch.tensor([4, 2], dtype=torch.int32)
    kc = torch.zeros(5, 16, 2, 64, dtype=bf)
    table = torch.zeros(2, 3, dtype=torch.int32)

    for wrong, err in (
        (dict(q=q[:5]), ValueError), (dict(k=k.half()), TypeError), (dict(v=k[:, :1]), ValueError),
        (dict(o=q.transpose(0, 1)), ValueError), (dict(cu=cu.long()), TypeError), (dict(q=q[..., ::2]), ValueError),
        (dict(lse=torch.zeros(6, 4, dtype=bf)), TypeError), (dict(lse=torch.zeros(4, 6)), ValueError),
        (dict(o=q.view(6, 256)), ValueError), (dict(q=q.double(), k=k.double()), TypeError),
    ):
        a = dict(q=q, k=k, v=k.clone(), o=q.clone(), cu=cu, lse=None)
        a.update(wrong)
        with pytest.raises(err):
            gdr.gdr_attn_prefill(a["q"], a["k"], a["v"], a["o"], a["cu"], lse=a["lse"])
    for wrong, err in (
        (dict(kc=kc.half()), TypeError), (dict(vc=kc[:4]), ValueError), (dict(table=table[:1]), ValueError),
        (dict(table=table.long()), TypeError), (dict(vc=kc.transpose(1, 2).contiguous().transpose(1, 2)), ValueError),
        (dict(lens=lens.float()), TypeError), (dict(qo=None), ValueError), (dict(inv=torch.zeros(4, 2)), ValueError),
        (dict(kc=kc[..., :32], vc=kc[..., :32]), ValueError), (dict(table=table.t().contiguous().t()), ValueError),
    ):
        a = dict(q=q, k=k, v=k.clone(), qo=q.clone(), ko=None, kc=kc, vc=kc.clone(), table=table, lens=lens,
                 inv=torch.zeros(8), cu=cu)
        a.update(wrong)
        with pytest.raises(err):
            gdr.gdr_attn_append(a["q"], a["k"], a["v"], a["qo"], a["ko"], a["kc"], a["vc"], a["table"], a["lens"],
                                a["inv"], a["cu"])
    with pytest.raises(ValueError):
        gdr.gdr_attn_decode(q[:3], kc, kc.clone(), table, lens, q[:2])
    with pytest.raises(ValueError):  # host memory
        gdr.gdr_attn_prefill(q, k, k.clone(), q.clone(), cu, stream=0)
    assert ctypes.sizeof(gdr.gdr_kv_cache) == 72
