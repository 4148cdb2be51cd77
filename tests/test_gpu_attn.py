"""Attention operators on the GPU against the 64-bit reference (tests/attn_ref.py)
at its derived bounds."""

import ctypes
import math

import numpy as np
import pytest

import gated_deltanet_scan_gb300 as gdr
from tests import attn_ref as ar
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

DT = ("bf16", "f16")


def tdt(name):
    torch = gu.torch_mod()
    return torch.bfloat16 if name == "bf16" else torch.float16


def randn(rng, shape, dtype, scale=1.0):
    torch = gu.torch_mod()
    return torch.from_numpy(scale * rng.standard_normal(shape)).to(tdt(dtype)).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


def ints(x):
    torch = gu.torch_mod()
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def nan_like(shape, dtype):
    torch = gu.torch_mod()
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def close(got, want, bound, what):
    got = f64(got)
    assert np.array_equal(np.isneginf(got), np.isneginf(want)), what
    with np.errstate(invalid="ignore"):
        over = np.where(np.isfinite(want), np.abs(got - want) - bound, 0.0)
    assert np.all(over <= 0), f"{what}: beyond its bound by {np.nanmax(over):.3e} (NaN: {np.isnan(got).sum()})"


def no_error():
    assert gdr.gdr_device_error(device="cuda") == gdr.GDR_OK


# --- prefill ------------------------------------------------------------------------------------------------

def check_prefill(q, k, v, lens, dtype, scale=None, lse=True):
    torch = gu.torch_mod()
    T, hq, d = q.shape
    cu = ints(np.concatenate([[0], np.cumsum(lens)]))
    o = nan_like((T, hq, d), q.dtype)
    ls = nan_like((T, hq), torch.float32) if lse else None
    gdr.gdr_attn_prefill(q, k, v, o, cu, scale=scale, lse=ls)
    torch.cuda.synchronize()
    no_error()
    wo, wl, bo, bl = ar.prefill(f64(q), f64(k), f64(v), d ** -0.5 if scale is None else scale, lens, dtype)
    close(o, wo, bo, "o")
    if lse:
        close(ls, wl, bl, "lse")
    return o, ls


PREFILL = [
    # d, h_q, h_kv, lens
    (64, 1, 1, [1]), (128, 1, 1, [1]), (256, 4, 1, [2]),
    (128, 2, 2, [17]), (256, 8, 2, [63]), (64, 4, 2, [64, 65]), (128, 8, 2, [127, 128, 129]),
    (256, 8, 2, [255, 1, 0, 33]), (128, 2, 2, [257]), (64, 3, 3, [300, 5]), (256, 3, 1, [0, 0, 140, 0]),
    (128, 6, 2, [200, 31]), (128, 5, 1, [1, 2, 3, 4, 5, 90]), (256, 6, 1, [190]), (64, 14, 2, [97, 64]),
    (64, 16, 1, [70, 9]), (128, 33, 1, [40]), (64, 100, 1, [13]), (256, 128, 1, [9]), (128, 128, 1, [130]),
    (256, 2, 2, [513]), (128, 4, 1, [1000]), (256, 4, 1, [700]), (64, 2, 1, [1300]), (128, 1, 1, [900]),
]


# the two-SM kernel's blocks (sequences over 256 tokens): groups that do not divide 128, a
# group as large as a block, several blocks per pair, short sequences between long ones
PREFILL += [
    (128, 33, 1, [300]), (64, 100, 1, [270, 3]), (256, 128, 1, [259]), (128, 5, 1, [601, 258]),
    (64, 3, 3, [257, 384, 385]), (256, 14, 2, [300, 20, 511]), (128, 24, 8, [513, 400, 256, 300]),
    (64, 12, 12, [640, 641]),
]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("d,h_q,h_kv,lens", PREFILL)
def test_prefill(d, h_q, h_kv, lens, dtype):
    gu.require_gpu()
    rng = np.random.default_rng(d + h_q + sum(lens))
    T = sum(lens)
    q, k, v = randn(rng, (T, h_q, d), dtype, 2.0), randn(rng, (T, h_kv, d), dtype), randn(rng, (T, h_kv, d), dtype)
    check_prefill(q, k, v, lens, dtype)


def test_prefill_many_sequences():
    gu.require_gpu()
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 12, 300)]
    T = sum(lens)
    q, k, v = randn(rng, (T, 4, 64), "bf16"), randn(rng, (T, 2, 64), "bf16"), randn(rng, (T, 2, 64), "bf16")
    check_prefill(q, k, v, lens, "bf16")


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prefill_strided_parts_of_a_projection(d):
    torch = gu.require_gpu()
    rng = np.random.default_rng(6)
    lens, hq, hkv = [150, 41], 4, 2
    T = sum(lens)
    x = randn(rng, (T, hq + 2 * hkv, d), "bf16")
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    o1, l1 = check_prefill(q, k, v, lens, "bf16")
    # head-major outputs and inputs give the same values
    qh, kh = q.transpose(0, 1).contiguous().transpose(0, 1), k.transpose(0, 1).contiguous().transpose(0, 1)
    cu = ints([0, 150, 191])
    o2 = nan_like((hq, T, d), q.dtype).transpose(0, 1)
    gdr.gdr_attn_prefill(qh, kh, v, o2, cu)
    torch.cuda.synchronize()
    assert torch.equal(o1, o2)


@pytest.mark.parametrize("scale", [0.0, -0.1, 1.0])
def test_prefill_scales_and_large_scores(scale):
    gu.require_gpu()
    rng = np.random.default_rng(7)
    q, k, v = (randn(rng, (300, 2, 128), "bf16", 2.0) for _ in range(3))
    check_prefill(q, k, v, [300], "bf16", scale=scale, lse=scale != 1.0)


def test_prefill_scores_that_keep_rising():
    """Every later token outweighs all earlier ones by far: each tile moves the running maximum."""
    torch = gu.require_gpu()
    n, d = 700, 128
    rng = np.random.default_rng(8)
    k = torch.zeros(n, 1, d, device="cuda")
    k[:, 0, 0] = torch.arange(n, device="cuda") * 0.25
    q = torch.zeros(n, 2, d, device="cuda")
    q[:, :, 0] = 8.0
    q[::3, :, 0] = -8.0
    check_prefill(q.to(torch.bfloat16), k.to(torch.bfloat16), randn(rng, (n, 1, d), "bf16"), [n], "bf16")


@pytest.mark.parametrize("d,hq", [(64, 2), (128, 2), (128, 1), (256, 4), (256, 1)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_prefill_never_uses_later_tokens_or_other_sequences(d, hq, bad):
    """Keys and values of later tokens and other sequences may hold anything."""
    torch = gu.require_gpu()
    rng = np.random.default_rng(9)
    lens = [97, 300, 75]
    T = sum(lens)
    q, k, v = randn(rng, (T, hq, d), "bf16"), randn(rng, (T, 1, d), "bf16"), randn(rng, (T, 1, d), "bf16")
    cu = ints([0, 97, 397, 472])
    clean = nan_like((T, hq, d), q.dtype)
    gdr.gdr_attn_prefill(q, k, v, clean, cu)
    for at in (97, 250, 396, 397, 471):  # token `at` holds `bad`: only rows of its sequence from it on change
        k2, v2 = k.clone(), v.clone()
        k2[at] = bad
        v2[at, :, 3::5] = bad
        o = nan_like((T, hq, d), q.dtype)
        gdr.gdr_attn_prefill(q, k2, v2, o, cu)
        end = next(int(c) for c in (97, 397, 472) if c > at)
        keep = torch.ones(T, dtype=torch.bool, device="cuda")
        keep[at:end] = False
        assert torch.equal(o[keep], clean[keep]), at
        # with a finite key, the value's columns take the value's infinity or NaN, and the others stay
        o = nan_like((T, hq, d), q.dtype)
        gdr.gdr_attn_prefill(q, k, v2, o, cu)
        assert torch.equal(o[keep], clean[keep]), at
        hit = torch.zeros(d, dtype=torch.bool, device="cuda")
        hit[3::5] = True
        rest = o[at:end]
        assert torch.all(torch.isnan(rest[..., hit]) if math.isnan(bad) else ~torch.isfinite(rest[..., hit])), at
        assert torch.all(torch.isfinite(rest[..., ~hit])), at
    no_error()


def test_prefill_repeats_exactly_and_on_another_stream():
    torch = gu.require_gpu()
    rng = np.random.default_rng(10)
    q, k, v = randn(rng, (500, 8, 128), "bf16"), randn(rng, (500, 2, 128), "bf16"), randn(rng, (500, 2, 128), "bf16")
    cu = ints([0, 333, 500])
    a, b, c = (nan_like((500, 8, 128), q.dtype) for _ in range(3))
    gdr.gdr_attn_prefill(q, k, v, a, cu)
    gdr.gdr_attn_prefill(q, k, v, b, cu)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    gdr.gdr_attn_prefill(q, k, v, c, cu, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c)


# --- the cache ----------------------------------------------------------------------------------------------

class Paged:
    """A cache of random values with shuffled pages; unused table entries are -1."""

    def __init__(self, rng, lens, page, h_kv, d, dtype, by_head=False, spare=2, stale=None):
        torch = gu.torch_mod()
        need = [-(-n // page) for n in lens]
        total = sum(need) + spare
        shape = (total, h_kv, page, d) if by_head else (total, page, h_kv, d)
        self.k, self.v = (randn(rng, shape, dtype) for _ in range(2))
        if by_head:
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        order = rng.permutation(total)
        self.table_np = np.full((len(lens), max(need + [1]) + 1), -1, dtype=np.int32)
        at = 0
        for s, n in enumerate(need):
            self.table_np[s, :n] = order[at:at + n]
            at += n
        self.lens = list(lens)
        self.table, self.kv_lens = torch.from_numpy(self.table_np).cuda(), ints(lens)
        if stale is not None:  # every slot no sequence holds
            used = np.zeros((total, page), dtype=bool)
            for s, n in enumerate(lens):
                p = np.arange(n)
                used[self.table_np[s, p // page], p % page] = True
            free = torch.from_numpy(~used).cuda()
            self.k[free], self.v[free] = stale, stale


def run_decode(c, q, n_tok, scale=None, lse=True, stream=None):
    torch = gu.torch_mod()
    o = nan_like(q.shape, q.dtype)
    ls = nan_like(q.shape[:2], torch.float32) if lse else None
    gdr.gdr_attn_decode(q, c.k, c.v, c.table, c.kv_lens, o, n_tok, scale=scale, lse=ls, stream=stream)
    return o, ls


def check_decode(c, q, n_tok, dtype, scale=None):
    torch = gu.torch_mod()
    o, ls = run_decode(c, q, n_tok, scale)
    torch.cuda.synchronize()
    no_error()
    wo, wl, bo, bl = ar.decode(f64(q), f64(c.k), f64(c.v), c.table_np, c.lens, n_tok,
                               q.shape[-1] ** -0.5 if scale is None else scale, dtype)
    close(o, wo, bo, "o")
    close(ls, wl, bl, "lse")
    return o, ls


DECODE = [
    # d, h_q, h_kv, n_tok, page, by_head, lens
    (256, 4, 1, 1, 64, False, [1]), (128, 1, 1, 1, 16, False, [0]), (64, 8, 2, 1, 1, False, [5, 0, 1, 2]),
    (256, 16, 4, 1, 64, False, [300, 17, 1, 64, 65]), (128, 8, 2, 1, 48, True, [129, 4000, 15, 16]),
    (64, 6, 2, 1, 100, True, [777, 31, 33]), (256, 3, 3, 1, 3, False, [50, 200]), (128, 40, 2, 1, 32, False, [99, 512]),
    (256, 32, 2, 1, 16, True, [140, 9]), (64, 34, 2, 1, 16, True, [140, 9]), (128, 64, 1, 1, 16, False, [333]),
    (64, 128, 1, 1, 16, False, [50, 3]),
    (256, 16, 4, 16, 64, False, [16, 300, 1001]), (128, 8, 2, 16, 48, True, [7, 0, 95, 1500]),
    (64, 6, 2, 5, 16, False, [5, 4, 200]), (256, 4, 1, 2, 128, False, [2, 129, 1]), (128, 3, 3, 9, 7, True, [64, 10]),
    (256, 8, 8, 4, 256, False, [600]), (128, 24, 1, 8, 64, False, [130, 41]), (64, 128, 1, 16, 16, False, [37]),
    (256, 20, 1, 16, 16, False, [85]), (128, 16, 1, 3, 64, False, [260, 2]),
    # 17 rows and more at other tile ends, many triples per worker
    (256, 17, 1, 1, 64, False, [64, 63, 65, 128, 1]), (128, 9, 1, 2, 16, True, [700, 1, 2, 3]),
    (64, 2, 1, 9, 48, False, [513, 8, 9, 10, 1000]), (256, 16, 4, 12, 33, True, [12, 2500, 11, 640]),
]


@pytest.mark.parametrize("n_tok,h_q", [(16, 8), (1, 40)])
def test_decode_wide_rows_many_sequences(n_tok, h_q):
    gu.require_gpu()
    rng = np.random.default_rng(26)
    lens = [int(x) for x in rng.integers(0, 140, 230)]
    c = Paged(rng, lens, 16, 2, 64, "bf16", stale=float("nan"))
    check_decode(c, randn(rng, (230 * n_tok, h_q, 64), "bf16", 2.0), n_tok, "bf16")



@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("d,h_q,h_kv,n_tok,page,by_head,lens", DECODE)
def test_decode(d, h_q, h_kv, n_tok, page, by_head, lens, dtype):
    gu.require_gpu()
    rng = np.random.default_rng(d + h_q + sum(lens))
    c = Paged(rng, lens, page, h_kv, d, dtype, by_head, stale=float("nan"))
    check_decode(c, randn(rng, (len(lens) * n_tok, h_q, d), dtype, 2.0), n_tok, dtype)


@pytest.mark.parametrize("d,n_tok", [(256, 1), (128, 1), (64, 1), (256, 16), (128, 4)])
def test_decode_long_sequence_is_split_and_joined(d, n_tok):
    gu.require_gpu()
    rng = np.random.default_rng(20 + d)
    c = Paged(rng, [30011], 64, 1, d, "bf16")
    check_decode(c, randn(rng, (n_tok, 4, d), "bf16", 3.0), n_tok, "bf16")


@pytest.mark.parametrize("d", [64, 256])
def test_decode_many_sequences_of_every_length(d):
    gu.require_gpu()
    rng = np.random.default_rng(21)
    lens = [int(x) for x in rng.integers(0, 150, 400)]
    c = Paged(rng, lens, 16, 2, d, "f16", stale=float("inf"))
    check_decode(c, randn(rng, (400, 6, d), "f16", 2.0), 1, "f16")


def test_decode_more_heads_and_sequences_than_blocks():
    gu.require_gpu()
    rng = np.random.default_rng(22)
    lens = [int(x) for x in rng.integers(1, 9, 1500)]
    c = Paged(rng, lens, 4, 4, 64, "bf16", stale=float("nan"))
    check_decode(c, randn(rng, (1500, 4, 64), "bf16"), 1, "bf16")


@pytest.mark.parametrize("heads", [4, 1])  # 64 rows and 16: either kernel
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_decode_draft_tokens_never_see_later_ones(d, bad, heads):
    torch = gu.require_gpu()
    rng = np.random.default_rng(23)
    n, n_tok = 203, 16
    c = Paged(rng, [n], 32, 1, d, "bf16")
    q = randn(rng, (n_tok, heads, d), "bf16")
    clean, _ = run_decode(c, q, n_tok)
    for j in (0, 5, 15):
        p = n - n_tok + j
        at = (int(c.table_np[0, p // 32]), p % 32)
        kept = c.k[at].clone(), c.v[at].clone()
        c.v[at[0], at[1], :, 1::3] = bad
        o, _ = run_decode(c, q, n_tok)
        assert torch.equal(o[:j], clean[:j]), j
        hit = torch.zeros(d, dtype=torch.bool, device="cuda")
        hit[1::3] = True
        assert torch.all(~torch.isfinite(o[j:][..., hit])) and torch.all(torch.isfinite(o[j:][..., ~hit])), j
        c.k[at] = bad
        o, _ = run_decode(c, q, n_tok)
        assert torch.equal(o[:j], clean[:j]), j
        c.k[at], c.v[at] = kept
    no_error()


def test_decode_strided_queries_outputs_and_tables():
    torch = gu.require_gpu()
    rng = np.random.default_rng(24)
    c = Paged(rng, [70, 33], 16, 2, 128, "bf16")
    wide = randn(rng, (2, 12, 128), "bf16")
    o, _ = check_decode(c, wide[:, 2:10], 1, "bf16")
    table = torch.full((2, 64), -1, dtype=torch.int32, device="cuda")
    table[:, :c.table.shape[1]] = c.table
    o2 = nan_like((8, 2, 128), torch.bfloat16).transpose(0, 1)
    gdr.gdr_attn_decode(wide[:, 2:10], c.k, c.v, table[:, :c.table.shape[1]], c.kv_lens, o2)
    torch.cuda.synchronize()
    assert torch.equal(o, o2)


def test_decode_repeats_exactly_on_any_stream_and_in_a_graph():
    torch = gu.require_gpu()
    rng = np.random.default_rng(25)
    c = Paged(rng, [5000, 40, 1300], 64, 2, 128, "bf16")
    q = randn(rng, (3, 8, 128), "bf16")
    ws = torch.empty(max(16, gdr.gdr_attn_decode_workspace_bytes(q, c.k, 3)), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)
    a, la = run_decode(c, q, 1)
    b, g = nan_like(q.shape, q.dtype), nan_like(q.shape, q.dtype)
    gdr.gdr_attn_decode(q, c.k, c.v, c.table, c.kv_lens, b, workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o3, l3 = run_decode(c, q, 1, stream=s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdr.gdr_attn_decode(q, c.k, c.v, c.table, c.kv_lens, g, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, o3) and torch.equal(la, l3) and torch.equal(a, g)
    # the lengths and the table are read at replay: a longer sequence needs no new graph
    c.kv_lens[1] = 64
    c.lens[1] = 64
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(g, run_decode(c, q, 1)[0]) and not torch.equal(a, g)


# --- append -------------------------------------------------------------------------------------------------

APPEND = [
    # d, h_q, h_kv, rot, interleaved, page, by_head, new tokens, kv_lens
    (256, 16, 4, 64, False, 64, False, [1], [1500]), (256, 16, 4, 64, False, 64, False, [1, 1, 1], [1, 64, 65]),
    (128, 8, 2, 128, True, 48, True, [100, 0, 49], [100, 7, 50]), (64, 3, 3, 24, False, 16, False, [5, 33], [100, 33]),
    (64, 6, 1, 24, True, 5, True, [11], [11]), (128, 4, 4, 0, False, 16, False, [20], [21]),
    (256, 1, 1, 256, False, 16, True, [3, 3], [4, 9000]), (128, 12, 4, 32, False, 128, False, [257], [300]),
    (64, 4, 2, 64, False, 32, False, [6], [1000000]), (256, 5, 1, 2, False, 32, False, [40], [40]),
    (128, 9, 3, 34, False, 32, True, [70], [71]), (64, 1, 1, 16, True, 32, True, [9], [9]),
]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("d,h_q,h_kv,rot,il,page,by_head,new,lens", APPEND)
def test_append(d, h_q, h_kv, rot, il, page, by_head, new, lens, in_place, dtype):
    torch = gu.require_gpu()
    rng = np.random.default_rng(d + h_q + rot + sum(lens))
    T = sum(new)
    x = randn(rng, (T, h_q + 2 * h_kv, d), dtype)
    q, k, v = x[:, :h_q], x[:, h_q:h_q + h_kv], x[:, h_q + h_kv:]
    inv = torch.from_numpy((10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))).astype(np.float32)).cuda()
    c = Paged(rng, lens, page, h_kv, d, dtype, by_head)
    k0, v0 = c.k.clone(), c.v.clone()
    q64, k64, v64 = f64(q), f64(k), f64(v)
    qo = q if in_place else nan_like((T, h_q, d), q.dtype)
    ko = k if in_place else nan_like((T, h_kv, d), q.dtype)
    cu = None if len(set(new)) == 1 else ints(np.concatenate([[0], np.cumsum(new)]))
    gdr.gdr_attn_append(q, k, v, qo, ko, c.k, c.v, c.table, c.kv_lens, inv if rot else None, cu, interleaved=il)
    torch.cuda.synchronize()
    no_error()
    pos = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, new)])
    seq = np.repeat(np.arange(len(new)), new)
    for got, src, what in ((qo, q64, "q"), (ko, k64, "k")):
        want, size = ar.rotate(src, pos, inv.cpu().numpy(), il)
        close(got, want, ar.rotate_bound(want, size, dtype, rot), what)
    page_of, slot = c.table_np[seq, pos // page], pos % page
    # the cache holds the rotated keys and the values, bit for bit, and nothing else changed
    k0[page_of, slot], v0[page_of, slot] = ko, torch.from_numpy(v64).to(v0.dtype).cuda()
    assert torch.equal(c.k, k0) and torch.equal(c.v, v0)


def test_append_without_queries_or_packed_keys_and_many_tokens():
    torch = gu.require_gpu()
    rng = np.random.default_rng(31)
    new = [4000, 0, 3001, 1]
    lens = [4010, 3, 3001, 12]
    k, v = randn(rng, (7002, 1, 64), "bf16"), randn(rng, (7002, 1, 64), "bf16")
    c = Paged(rng, lens, 64, 1, 64, "bf16")
    inv = torch.from_numpy((1e4 ** (-np.arange(16) / 16)).astype(np.float32)).cuda()
    gdr.gdr_attn_append(None, k, v, None, None, c.k, c.v, c.table, c.kv_lens, inv, ints([0, 4000, 4000, 7001, 7002]))
    torch.cuda.synchronize()
    no_error()
    pos = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, new)])
    seq = np.repeat(np.arange(4), new)
    want, size = ar.rotate(f64(k), pos, inv.cpu().numpy(), False)
    at = (c.table_np[seq, pos // 64], pos % 64)
    close(c.k[at], want, ar.rotate_bound(want, size, "bf16", 32), "k")
    assert torch.equal(c.v[at], v)


def test_append_copies_special_values_past_the_rotation():
    torch = gu.require_gpu()
    rng = np.random.default_rng(32)
    k = randn(rng, (1, 1, 64), "bf16")
    k[0, 0, 32:] = float("nan")
    k[0, 0, 33] = float("inf")
    c = Paged(rng, [9], 16, 1, 64, "bf16")
    gdr.gdr_attn_append(None, k, k.clone(), None, None, c.k, c.v, c.table, c.kv_lens,
                        torch.ones(16, dtype=torch.float32, device="cuda"))
    got = c.k[int(c.table_np[0, 0]), 8]
    assert torch.isfinite(got[..., :32]).all()
    assert torch.equal(got[..., 32:].view(torch.int16), k[0, ..., 32:].view(torch.int16))


# --- what the device checks itself --------------------------------------------------------------------------

def test_bad_lengths_and_pages_are_recorded_and_nothing_is_touched():
    torch = gu.require_gpu()
    rng = np.random.default_rng(40)
    c = Paged(rng, [40, 20], 16, 1, 64, "bf16")
    q = randn(rng, (2, 2, 64), "bf16")
    k = randn(rng, (2, 1, 64), "bf16")
    good, _ = run_decode(c, q, 1)
    k0, v0 = c.k.clone(), c.v.clone()
    most = c.table.shape[1] * 16
    for bad in (-1, most + 1):
        lens = ints([bad, 20])
        o = nan_like(q.shape, q.dtype)
        gdr.gdr_attn_decode(q, c.k, c.v, c.table, lens, o)
        assert gdr.gdr_device_error(device="cuda") == gdr.GDR_ERR_INVALID_ARG
        assert torch.equal(o[1], good[1]) and torch.all(o[0] == 0)
    for page in (-7, c.k.shape[0]):
        table = c.table.clone()
        table[0, 1] = page
        o = nan_like(q.shape, q.dtype)
        gdr.gdr_attn_decode(q, c.k, c.v, table, c.kv_lens, o)
        assert gdr.gdr_device_error(device="cuda") == gdr.GDR_ERR_INVALID_ARG
        assert torch.equal(o[1], good[1])
        table = c.table.clone()
        table[:, :] = page
        gdr.gdr_attn_append(None, k, k, None, None, c.k, c.v, table, c.kv_lens, None)
        assert gdr.gdr_device_error(device="cuda") == gdr.GDR_ERR_INVALID_ARG
        assert torch.equal(c.k, k0) and torch.equal(c.v, v0)
    for bad in (0, -3, most + 1):
        gdr.gdr_attn_append(None, k, k, None, None, c.k, c.v, c.table, ints([bad, bad]), None)
        assert gdr.gdr_device_error(device="cuda") == gdr.GDR_ERR_INVALID_ARG
        assert torch.equal(c.k, k0) and torch.equal(c.v, v0)
    # packed starts out of range: the sequences that use them are skipped
    q3, k3 = randn(rng, (9, 2, 64), "bf16"), randn(rng, (9, 1, 64), "bf16")
    for starts in ([0, -2, 9], [0, 20, 9], [3, 5, 9], [0, 4, 12]):
        o = nan_like(q3.shape, q3.dtype)
        gdr.gdr_attn_prefill(q3, k3, k3, o, ints(starts))
        gdr.gdr_device_error(device="cuda")
        gdr.gdr_attn_append(None, k3, k3, None, None, c.k, c.v, c.table, c.kv_lens, None, ints(starts))
        gdr.gdr_device_error(device="cuda")
    torch.cuda.synchronize()
    assert ctypes.sizeof(gdr.gdr_rows) == 24


# --- together, as they are used -----------------------------------------------------------------------------

def test_example_decodes_step_by_step_what_one_prefill_gives():
    """The hybrid example: prompt, single tokens and a draft block through append, prefill and decode, against
    one prefill of the whole sequences.  Both sides round q and k alike; o differs by the weights' rounding and
    its own (2 x 2^-8 of o's terms), which the output projection (rows of unit norm) sums over 4096 inputs."""
    import importlib.util
    import os

    torch = gu.require_gpu()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_decode.py")
    spec = importlib.util.spec_from_file_location("hybrid_decode", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    got, whole = mod.run(lengths=(130, 1, 77), steps=5, draft=3)
    no_error()
    assert torch.isfinite(got).all()
    # per row: errors of at most 2^-6 of each |o| term reach the row's entries as 2^-6 of their rms; entries
    # are sums of x (|x| a few) and the projection, rounded to 2^-8 of themselves on both sides
    err = (got.float() - whole.float()).abs()
    bound = 2.0 ** -7 * whole.float().abs() + 2.0 ** -4
    assert torch.all(err <= bound), float((err - bound).max())


def test_prefill_inputs_may_be_expanded():
    """Keys and values shared by all heads or all queries alike: zero strides."""
    torch = gu.require_gpu()
    rng = np.random.default_rng(50)
    q = randn(rng, (150, 4, 64), "bf16")
    k = randn(rng, (150, 1, 64), "bf16").expand(150, 2, 64)
    v = randn(rng, (1, 2, 64), "bf16").expand(150, 2, 64)
    check_prefill(q, k, v, [150], "bf16")
    check_prefill(q[:1].expand(150, 4, 64), k, v, [100, 50], "bf16")


# --- offsets past 32 bits -----------------------------------------------------------------------------------

def spread(torch, shape, strides, dtype):
    """An uninitialised tensor of this shape and strides (its own allocation)."""
    size = 1 + sum((n - 1) * s for n, s in zip(shape, strides))
    return torch.empty(size, dtype=dtype, device="cuda").as_strided(shape, strides)


@pytest.mark.parametrize("n_tok,h_q", [(1, 4), (4, 8)])
def test_pages_far_apart(n_tok, h_q):
    """Pages 2^32 elements apart: offsets in the cache pass 32 bits."""
    torch = gu.require_gpu()
    rng = np.random.default_rng(60)
    lens, page, d = [45, 20], 16, 64
    c = Paged(rng, lens, page, 1, d, "bf16", spare=0)
    shape, strides = (c.k.shape[0], page, 1, d), (1 << 32, d, d, 1)
    far_k, far_v = spread(torch, shape, strides, c.k.dtype), spread(torch, shape, strides, c.k.dtype)
    far_k.copy_(c.k)
    far_v.copy_(c.v)
    k, v = randn(rng, (2 * n_tok, 1, d), "bf16"), randn(rng, (2 * n_tok, 1, d), "bf16")
    q = randn(rng, (2 * n_tok, h_q, d), "bf16")
    for cache in ((c.k, c.v), (far_k, far_v)):
        gdr.gdr_attn_append(None, k, v, None, None, *cache, c.table, c.kv_lens, None)
    assert torch.equal(far_k, c.k) and torch.equal(far_v, c.v)
    near, _ = check_decode(c, q, n_tok, "bf16")
    o = nan_like(q.shape, q.dtype)
    gdr.gdr_attn_decode(q, far_k, far_v, c.table, c.kv_lens, o, n_tok)
    torch.cuda.synchronize()
    no_error()
    assert torch.equal(o, near)


@pytest.mark.parametrize("lens", [[40], [20, 20], [300]])
def test_rows_far_apart(lens):
    """Tokens 2^24 and more elements apart: offsets in the rows pass 32 bits."""
    torch = gu.require_gpu()
    rng = np.random.default_rng(61)
    T, d = sum(lens), 64
    q, k, v = randn(rng, (T, 2, d), "bf16"), randn(rng, (T, 1, d), "bf16"), randn(rng, (T, 1, d), "bf16")
    near, _ = check_prefill(q, k, v, lens, "bf16")
    ts = 1 << (27 if T < 100 else 24)
    far = [spread(torch, t.shape, (ts, d, 1), t.dtype) for t in (q, k, v, near)]
    for t, src in zip(far, (q, k, v)):
        t.copy_(src)
    cu = ints(np.concatenate([[0], np.cumsum(lens)]))
    gdr.gdr_attn_prefill(*far, cu)
    torch.cuda.synchronize()
    no_error()
    assert torch.equal(far[3], near)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [40, 400])
@pytest.mark.parametrize("weight", [-14.25, -17.0])
def test_small_weights_keep_their_accuracy(n, d, dtype, weight):
    """The first token outweighs the others by 2^20 or 2^24 but has no value in half of the columns, so these
    are sums of small weights alone."""
    torch = gu.require_gpu()
    rng = np.random.default_rng(n + d)
    q, k, v = torch.zeros(n, 8, d), torch.zeros(n, 2, d), torch.from_numpy(rng.uniform(0.5, 1.5, (n, 2, d)))
    q[:, :, 3], k[1:, :, 3], v[0, :, d // 2:] = 1.0, weight, 0.0
    q, k, v = (x.to(tdt(dtype)).cuda() for x in (q, k, v))

    def check(o, lse, rows):
        wo, wl, bo, bl = ar.prefill(f64(q), f64(k), f64(v), 1.0, [n], dtype)
        # h of every weight holds down to 2^-22 of the largest; below, half a step of 2^-32 each
        loose = 1.5 * n * 2.0 ** -33 if dtype == "f16" and weight < -15.25 else 0.0
        close(o, wo[rows], bo[rows] + loose, "o")
        close(lse, wl[rows], bl[rows], "lse")

    o, lse = nan_like((n, 8, d), q.dtype), nan_like((n, 8), torch.float32)
    gdr.gdr_attn_prefill(q, k, v, o, ints([0, n]), scale=1.0, lse=lse)
    check(o, lse, slice(0, n))
    page = 16
    kc, vc = (torch.zeros(n // page + 1, page, 2, d, dtype=q.dtype, device="cuda") for _ in range(2))
    kc.view(-1, 2, d)[:n], vc.view(-1, 2, d)[:n] = k, v
    for n_tok in (1, 16):  # 4 rows and 64: either kernel
        o, lse = nan_like((n_tok, 8, d), q.dtype), nan_like((n_tok, 8), torch.float32)
        gdr.gdr_attn_decode(q[n - n_tok:], kc, vc, ints(range(n // page + 1)).view(1, -1), ints([n]), o, n_tok,
                            scale=1.0, lse=lse)
        check(o, lse, slice(n - n_tok, n))
    no_error()
