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


def test_binding_wants_the_tensors_device_current(L, monkeypatch):
    """On another device a default stream's handle, the kernels and the error word would be the current one's."""
    torch = pytest.importorskip("torch")

    class Elsewhere(torch.Tensor):
        def get_device(self):
            return 1

    def new(*shape, dtype=torch.bfloat16):
        return torch.zeros(*shape, dtype=dtype).as_subclass(Elsewhere)

    called = []
    for name in ("gdr_attn_append", "gdr_attn_prefill", "gdr_attn_decode"):
        monkeypatch.setattr(L, name, lambda *a: called.append(a) or OK)
    monkeypatch.setattr(gdr, "_attn_types", None)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    q, k, kc = new(6, 4, 64), new(6, 2, 64), new(5, 16, 2, 64)
    lens, table = new(2, dtype=torch.int32), new(2, 3, dtype=torch.int32)
    calls = (lambda: gdr.gdr_attn_prefill(q, k, k, q, new(3, dtype=torch.int32), stream=0),
             lambda: gdr.gdr_attn_append(q, k, k, q, k, kc, kc, table, lens, None, stream=0),
             lambda: gdr.gdr_attn_decode(q, kc, kc, table, lens, q, 3, workspace=new(8, dtype=torch.uint8), stream=0))
    for call in calls:
        with pytest.raises(ValueError, match="device 0 is current"):
            call()
    assert not called
    monkeypatch.setattr(gdr, "_attn_types", None)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    for call in calls:
        call()
    assert len(called) == 3
