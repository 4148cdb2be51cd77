"""Operators of trees of drafted tokens: bad arguments are refused on the host before any launch, by the C ABI and by
the binding (no GPU needed)."""

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


def rule_dims(**kw):
    d = dict(h_qk=16, h_v=32, d_k=128, d_v=128, chunk=64, in_dtype=gdr.GDR_BF16, out_dtype=gdr.GDR_F32, scale=1.0,
             flags=0)
    d.update(kw)
    return gdr.gdr_dims(**d)


def attn_dims(**kw):
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


def verify(L, d=None, n=2, n_tok=24, parents=A, q=A, k=A, v=A, g=A, beta=A, state=A, o=A, deltas=None):
    return L.gdr_verify_tree(d or rule_dims(), n, n_tok, parents, q, k, v, g, beta, state, o, deltas, None)


def settle(L, d=None, n=2, n_tok=24, parents=A, last=A, k=A, g=A, deltas=A, state=A):
    return L.gdr_verify_tree_commit(d or rule_dims(), n, n_tok, parents, last, k, g, deltas, state, None)


def append(L, d=None, n=2, n_tok=24, parents=A, q=None, k=None, v=None, qo=None, ko=None, c=None, lens=A, inv=A, rot=64):
    r = rows()
    return L.gdr_attn_append_tree(d or attn_dims(), n, n_tok, parents, q or r, k or r, v or r, qo or r, ko,
                                  c or cache(), lens, inv, rot, 0, None)


def attend(L, d=None, n=2, n_tok=24, parents=A, q=None, c=None, lens=A, o=None, lse=None, ws=A, wsb=1 << 40):
    r = rows()
    return L.gdr_attn_decode_tree(d or attn_dims(), n, n_tok, parents, q or r, c or cache(), lens, o or r, lse, ws, wsb,
                                  None)


def compact(L, d=None, n=2, n_tok=24, parents=A, last=A, layers=3, stride=6553600, c=None, lens=A, lens_out=None):
    return L.gdr_attn_commit_tree(d or attn_dims(), n, n_tok, parents, last, layers, stride, c or cache(), lens,
                                  lens_out, None)


CALLS = (verify, settle, append, attend, compact)


@pytest.mark.parametrize("call", CALLS)
def test_counts_and_parents(L, call):
    for n_tok in (0, 65, -1, 1 << 30):
        assert call(L, n_tok=n_tok) == BAD
        assert call(L, n_tok=n_tok, n=0) == BAD
    assert call(L, n=-1) == BAD
    assert call(L, parents=None) == BAD and call(L, parents=A + 2) == BAD
    assert call(L, n=0) == OK and call(L, n=0, parents=None) == OK  # nothing to do, whatever the pointers are


@pytest.mark.parametrize("bad,code", [
    (dict(h_qk=0), BAD), (dict(h_v=0), BAD), (dict(h_qk=3), BAD), (dict(in_dtype=7), BAD), (dict(d_k=0), BAD),
    (dict(flags=1 << 20), BAD), (dict(d_v=64), UNSUP), (dict(d_k=96, d_v=96), UNSUP),
])
def test_rule_dims(L, bad, code):
    for call in (verify, settle):
        assert call(L, d=rule_dims(**bad)) == code
        assert L.gdr_verify_block(rule_dims(**bad), 2, 4, A, A, A, A, A, A, A, A, None, None) == code  # as there


def test_rule_pointers_and_sizes(L):
    for name in ("q", "k", "v", "g", "beta", "state", "o"):
        assert verify(L, **{name: None}) == BAD and verify(L, **{name: A + 8}) == BAD, name
    assert verify(L, deltas=A + 4) == BAD
    for name in ("k", "g", "deltas", "state"):
        assert settle(L, **{name: None}) == BAD and settle(L, **{name: A + 8}) == BAD, name
    assert settle(L, last=None) == BAD and settle(L, last=A + 1) == BAD
    for call in (verify, settle):
        assert call(L, n=1 << 23) == UNSUP  # 2^28 states


@pytest.mark.parametrize("bad,code", [
    (dict(h_q=0), BAD), (dict(h_kv=0), BAD), (dict(h_q=15), BAD), (dict(d=0), BAD), (dict(dtype=3), BAD),
    (dict(scale=float("nan")), BAD), (dict(dtype=gdr.GDR_F32), UNSUP), (dict(d=96), UNSUP),
    (dict(h_q=4 * 129), UNSUP),
])
def test_attention_dims(L, bad, code):
    for call in (append, attend, compact):
        assert call(L, d=attn_dims(**bad)) == code
    assert L.gdr_attn_decode_tree_workspace_bytes(attn_dims(**bad), 2, 24) == 0


@pytest.mark.parametrize("bad", [rows(ptr=None), rows(ptr=A + 8), rows(ts=-8), rows(ts=4100), rows(hs=1)])
def test_rows(L, bad):
    for name in ("q", "k", "v", "qo", "ko"):
        assert append(L, **{name: bad}) == BAD, name
    for name in ("q", "o"):
        assert attend(L, **{name: bad}) == BAD, name


@pytest.mark.parametrize("bad", [
    dict(k=None), dict(v=A + 2), dict(page_table=None), dict(page_stride=12), dict(token_stride=-8), dict(n_pages=0),
    dict(page_size=0), dict(max_pages=0), dict(table_stride=-1), dict(page_size=1 << 16, max_pages=1 << 15),
])
def test_cache(L, bad):
    for call in (append, attend, compact):
        assert call(L, c=cache(**bad)) == BAD


def test_attention_pointers(L):
    for call in (append, attend, compact):
        assert call(L, lens=None) == BAD and call(L, lens=A + 1) == BAD
    assert append(L, rot=3) == BAD and append(L, rot=258) == BAD and append(L, inv=None) == BAD
    assert attend(L, lse=A + 2) == BAD
    assert append(L, n=1 << 27) == UNSUP and attend(L, n=1 << 24) == UNSUP


def test_decode_workspace(L):
    d = attn_dims()
    need = L.gdr_attn_decode_tree_workspace_bytes(d, 64, 24)
    assert need > 0
    for n, n_tok in ((0, 24), (-1, 24), (2, 0), (2, 65)):
        assert L.gdr_attn_decode_tree_workspace_bytes(d, n, n_tok) == 0
    assert attend(L, n=64, ws=None) == BAD and attend(L, n=64, ws=A + 8) == BAD and attend(L, n=64, wsb=need - 1) == BAD
    # for up to 16 rows what gdr_attn_decode needs
    for n_tok in (1, 7, 16):
        assert (L.gdr_attn_decode_tree_workspace_bytes(d, 64, n_tok) == L.gdr_attn_decode_workspace_bytes(d, 64, n_tok))


def test_compaction(L):
    assert compact(L, last=None) == BAD and compact(L, last=A + 2) == BAD
    assert compact(L, layers=0) == BAD and compact(L, layers=-3) == BAD
    for stride in (-8, 12, 1 << 38):
        assert compact(L, stride=stride) == BAD
    # layers that would share values: no stride, one inside a row, a page's, a token's
    for stride in (0, 8, 65536, 1024, 256 * 3):
        assert compact(L, stride=stride) == BAD, stride
    # pages, tokens or heads that share values cannot be written to
    assert compact(L, layers=1, c=cache(token_stride=0)) == BAD
    assert compact(L, layers=1, c=cache(page_stride=64)) == BAD and compact(L, layers=1, c=cache(head_stride=8)) == BAD
    # lengths are read while new ones are written
    for off in (-4, 0, 4):
        assert compact(L, lens_out=A + off) == BAD
    assert compact(L, lens_out=A + 2 + 64) == BAD
    assert compact(L, layers=1 << 20, stride=6553600, d=attn_dims(h_kv=4)) == UNSUP


def test_no_dims(L):
    z = ctypes.POINTER(gdr.gdr_attn_dims)()
    r = rows()
    assert L.gdr_attn_decode_tree(z, 1, 4, A, r, cache(), A, r, None, A, 1 << 30, None) == BAD
    assert L.gdr_attn_append_tree(z, 1, 4, A, r, r, r, r, None, cache(), A, A, 64, 0, None) == BAD
    assert L.gdr_attn_commit_tree(z, 1, 4, A, A, 1, 0, cache(), A, None, None) == BAD
    assert L.gdr_attn_commit_tree(attn_dims(), 1, 4, A, A, 1, 0, None, A, None, None) == BAD
    z = ctypes.POINTER(gdr.gdr_dims)()
    assert L.gdr_verify_tree(z, 1, 4, A, A, A, A, A, A, A, A, None, None) == BAD
    assert L.gdr_verify_tree_commit(z, 1, 4, A, A, A, A, A, A, None) == BAD


def refused(err, call, base, cases):
    for wrong in cases:
        args = dict(base, **wrong)
        with pytest.raises(err) as e:
            call(**args)
        assert "must be on a CUDA device" not in str(e.value), wrong  # which all tensors here fail last


def test_binding_of_the_rule_refuses(L):
    torch = pytest.importorskip("torch")
    n, m, d = 2, 5, 128
    q = torch.zeros(n * m, 2, d, dtype=torch.bfloat16)
    v = torch.zeros(n * m, 4, d, dtype=torch.bfloat16)
    g, state = torch.zeros(n * m, 4), torch.zeros(n, 4, d, d)
    parents, last = torch.full((n, m), -1, dtype=torch.int32), torch.zeros(n, dtype=torch.int32)
    base = dict(q=q, k=q.clone(), v=v, g=g, beta=g.clone(), state=state, o=v.float(), parents=parents)
    refused(ValueError, gdr.gdr_verify_tree, base, (
        dict(parents=parents[:1]), dict(parents=parents.flatten()), dict(parents=parents[:, :4]), dict(v=v[:9]),
        dict(g=g[:, :3]), dict(state=state[:1]), dict(state=state[0]), dict(deltas=torch.zeros(n * m, 4, 64)),
        dict(q=q.transpose(0, 1).contiguous().transpose(0, 1)), dict(o=v.float()[:, :3]),
        dict(parents=parents.t().contiguous().t())))
    refused(TypeError, gdr.gdr_verify_tree, base, (
        dict(parents=parents.long()), dict(g=g.bfloat16()), dict(state=state.bfloat16()), dict(k=q.float()),
        dict(deltas=v), dict(v=v.float())))
    base = dict(k=q, g=g, deltas=v.float(), state=state, parents=parents, last=last)
    refused(ValueError, gdr.gdr_verify_tree_commit, base, (
        dict(last=last[:1]), dict(parents=parents[:, :4]), dict(k=q[:9]), dict(k=q[:, 0]), dict(g=g[:9]),
        dict(deltas=v.float()[:, :2]), dict(state=state.transpose(2, 3))))
    refused(TypeError, gdr.gdr_verify_tree_commit, base, (
        dict(last=last.long()), dict(parents=parents.float()), dict(deltas=v), dict(state=state.half())))


def test_binding_of_attention_refuses(L):
    torch = pytest.importorskip("torch")
    n, m, d = 2, 3, 64
    bf, i32 = torch.bfloat16, torch.int32
    q, k = torch.zeros(n * m, 4, d, dtype=bf), torch.zeros(n * m, 2, d, dtype=bf)
    parents, last, lens = torch.full((n, m), -1, dtype=i32), torch.zeros(n, dtype=i32), torch.full((n,), 7, dtype=i32)
    kc, table = torch.zeros(5, 16, 2, d, dtype=bf), torch.zeros(n, 3, dtype=i32)
    base = dict(q=q, k=k, v=k.clone(), q_out=q.clone(), k_out=None, k_cache=kc, v_cache=kc.clone(), page_table=table,
                kv_lens=lens, inv_freq=torch.zeros(8), parents=parents)
    refused(ValueError, gdr.gdr_attn_append_tree, base, (
        dict(parents=None), dict(parents=parents[:1]), dict(parents=parents[:, :2]), dict(parents=parents[0]),
        dict(page_table=table[:1]), dict(v=k[:, :1]), dict(kv_lens=lens[:1])))
    refused(TypeError, gdr.gdr_attn_append_tree, base, (
        dict(parents=parents.long()), dict(k=k.half()), dict(kv_lens=lens.float())))
    base = dict(q=q, k_cache=kc, v_cache=kc.clone(), page_table=table, kv_lens=lens, o=q.clone(), parents=parents,
                workspace=torch.zeros(1 << 20, dtype=torch.uint8))
    refused(ValueError, gdr.gdr_attn_decode_tree, base, (
        dict(parents=parents[:, :2]), dict(parents=parents[:1]), dict(o=q[:4]), dict(lse=torch.zeros(4, n * m)),
        dict(v_cache=kc[:4])))
    refused(TypeError, gdr.gdr_attn_decode_tree, base, (
        dict(parents=parents.long()), dict(o=q.half()), dict(lse=torch.zeros(n * m, 4, dtype=bf))))
    base = dict(k_cache=kc, v_cache=kc.clone(), page_table=table, kv_lens=lens, parents=parents, last=last)
    many = torch.zeros(3, 5, 16, 2, d, dtype=bf)
    refused(ValueError, gdr.gdr_attn_commit_tree, base, (
        dict(k_cache=kc[0], v_cache=kc[0]), dict(v_cache=many), dict(last=last[:1]), dict(parents=parents[:1]),
        dict(lens_out=last[:1]), dict(v_cache=kc.transpose(1, 2).contiguous().transpose(1, 2)),
        dict(k_cache=many, v_cache=many[:2]), dict(parents=parents[0])))
    refused(TypeError, gdr.gdr_attn_commit_tree, base, (
        dict(last=last.long()), dict(lens_out=last.long()), dict(v_cache=kc.half()), dict(parents=parents.long())))
    gdr.gdr_attn_commit_tree(**dict(base, k_cache=many[:0], v_cache=many[:0]))  # no layers: nothing to move
