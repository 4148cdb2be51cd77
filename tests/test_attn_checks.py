"""Attention operators: what the host checks let through and what they refuse, at the borders (no GPU needed)."""

import ctypes
import subprocess

import pytest

import gated_deltanet_scan_gb300 as gdr
from gated_deltanet_scan_gb300 import build as gbuild
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
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
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
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for call in calls:
        call()
    assert len(called) == 3


def pieces_overlap(counts, strides, d):
    at = [0]
    for n, st in zip(counts, strides):
        at = [a + i * st for a in at for i in range(n)]
    at.sort()
    return any(b - a < d for a, b in zip(at, at[1:]))


@pytest.fixture(scope="module")
def overlap(tmp_path_factory):
    """The host's overlap check alone: what the library lets through it launches, so acceptance is tested here."""
    tmp = tmp_path_factory.mktemp("overlap")
    (tmp / "x.cpp").write_text(
        '#include "gdr_overlap.h"\n'
        'extern "C" int x(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int d) '
        '{ return gdr::attn::overlap(n0, s0, n1, s1, d); }\n')
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", gbuild.CSRC, str(tmp / "x.cpp"), "-o",
                    str(tmp / "x.so")], check=True)
    fn = ctypes.CDLL(str(tmp / "x.so")).x
    fn.argtypes = [ctypes.c_int64] * 4 + [ctypes.c_int]
    return fn


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n0,n1", [(1, 1), (1, 4), (4, 1), (3, 4), (10, 2), (2, 8), (5, 5)])
def test_overlap_against_the_places_themselves(overlap, n0, n1, d):
    """Nested strides in either order, runs that interleave, and zeros."""
    strides, seen = (0, 8, 56, 64, 72, 128, 136, 192, 256, 264, 320, 384, 448, 512, 576, 640, 1024), set()
    for s0 in strides:
        for s1 in strides:
            bad = pieces_overlap((n0, n1), (s0, s1), d)
            assert overlap(n0, s0, n1, s1, d) == bad, (s0, s1)
            seen.add(bad)
    assert n0 * n1 == 1 or seen == {False, True}


def test_overlap_of_far_strides(overlap):
    far, most = (1 << 38) - 8, (1 << 31) - 1
    for s0, s1 in ((far, 64), (64, far), (far, far), (far, far - 64), (far - 64, far), (far, 128), (0, far), (far, 0)):
        assert overlap(3, s0, 5, s1, 64) == pieces_overlap((3, 5), (s0, s1), 64), (s0, s1)
    assert overlap(most, far, 65535, far, 64) and overlap(most, 64, 65535, 32 * most, 64)
    assert not overlap(most, 64, 65535, far, 64) and not overlap(65535, far, most, 64, 64)
    assert not overlap(3, far, 65535, 64, 64) and not overlap(most, far, 1, 0, 256) and not overlap(1, 0, most, 256, 256)


def test_written_rows_that_overlap_are_refused(L):
    for bad in (rows(ts=0), rows(hs=0), rows(ts=128), rows(hs=128), rows(ts=2048), rows(ts=512, hs=512)):
        assert prefill(L, o=bad) == BAD and decode(L, n=10, o=bad) == BAD
        assert append(L, qo=bad) == BAD and append(L, q=bad, qo=bad) == BAD
    for bad in (rows(ts=0), rows(hs=0), rows(ts=128), rows(hs=128), rows(ts=512), rows(ts=512, hs=512)):
        assert append(L, ko=bad) == BAD


@pytest.mark.parametrize("bad", [
    dict(page_stride=0), dict(token_stride=0), dict(head_stride=0), dict(head_stride=248), dict(token_stride=512),
    dict(page_stride=1024), dict(page_stride=32768), dict(token_stride=256, head_stride=256),
])
def test_written_caches_that_overlap_are_refused(L, bad):
    assert append(L, c=cache(**bad)) == BAD
