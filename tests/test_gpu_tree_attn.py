"""Attention over trees of drafted tokens on the GPU: gdr_attn_append_tree, gdr_attn_decode_tree and
gdr_attn_commit_tree against the 64-bit reference (tests/tree_ref.py, tests/attn_ref.py) at its derived bounds, and the
five tree operators together."""

import numpy as np
import pytest

import gated_deltanet_scan_gb300 as gdr
from tests import attn_ref as ar
from tests import gpu_util as gu
from tests import tree_ref as tr
from tests.test_gpu_attn import Paged, close, f64, ints, nan_like, no_error, randn
from tests.test_gpu_tree_rule import Batch, below

pytestmark = pytest.mark.gpu

DT = ("bf16", "f16")
INF, NAN = float("inf"), float("nan")
KINDS = ("draft", "chain", "forest", "holes", "padded", "binary", "roots", "star", "deep", "none")


def trees_of(rng, n, n_tok, kinds=KINDS):
    return [tr.make(rng, n_tok, kinds[s % len(kinds)]) for s in range(n)]


def parents_of(trees):
    return gu.torch_mod().tensor(trees, dtype=gu.torch_mod().int32, device="cuda")


def attend(c, q, trees, scale=None, lse=True, stream=None, workspace=None):
    torch = gu.torch_mod()
    o = nan_like(q.shape, q.dtype)
    ls = nan_like(q.shape[:2], torch.float32) if lse else None
    gdr.gdr_attn_decode_tree(q, c.k, c.v, c.table, c.kv_lens, o, trees if torch.is_tensor(trees) else parents_of(trees),
                             scale=scale, lse=ls, stream=stream, workspace=workspace)
    return o, ls


def spoil(c, trees):
    """Slots of rows that are no nodes hold NaN."""
    page = c.k.shape[1]
    for s, tree in enumerate(trees):
        base = c.lens[s] - len(tree)
        for j, path in enumerate(tr.paths(tree)):
            if not path and base >= 0:
                at = int(c.table_np[s, (base + j) // page]), (base + j) % page
                c.k[at], c.v[at] = NAN, NAN


def check_attend(c, q, trees, dtype, scale=None):
    torch = gu.torch_mod()
    spoil(c, trees)
    o, ls = attend(c, q, trees, scale)
    torch.cuda.synchronize()
    no_error()
    wo, wl, bo, bl = tr.attend(trees, f64(q), f64(c.k), f64(c.v), c.table_np, c.lens,
                               q.shape[-1] ** -0.5 if scale is None else scale, dtype)
    close(o, wo, bo, "o")
    close(ls, wl, bl, "lse")
    return o, ls


ATTEND = [
    # d, h_q, h_kv, n_tok, page, by_head, lens.  First: up to 16 rows of a KV head (n_tok times h_q / h_kv)
    (256, 4, 1, 1, 64, False, [1, 70]), (128, 2, 2, 7, 16, False, [7, 0, 300]), (64, 3, 3, 16, 5, True, [16, 33, 2001]),
    (256, 8, 2, 4, 128, False, [4, 129, 1001]), (128, 1, 1, 13, 48, False, [500, 13, 0, 14]), (64, 16, 1, 1, 16, True, [90]),
    # up to 128
    (128, 1, 1, 17, 16, False, [17, 40]), (256, 16, 4, 24, 64, False, [24, 300, 1001]), (64, 2, 2, 64, 48, True, [64, 65, 0, 900]),
    (128, 8, 2, 24, 48, True, [129, 4000, 25]), (256, 2, 1, 41, 7, False, [41, 100]), (64, 6, 2, 33, 16, False, [33, 200, 97]),
    (128, 8, 8, 31, 256, False, [600]), (256, 4, 2, 64, 64, False, [128, 64, 191, 1000]), (64, 34, 2, 2, 16, True, [140, 9]),
    # more
    (128, 8, 2, 48, 16, False, [48, 700, 111]), (256, 16, 4, 41, 64, False, [300, 41]), (64, 12, 2, 64, 100, True, [777, 64]),
    (256, 16, 2, 64, 33, False, [90, 2500]), (128, 5, 1, 64, 64, False, [64, 0, 3000]), (64, 128, 1, 64, 16, False, [70]),
    (128, 24, 1, 11, 64, False, [130, 12]), (256, 32, 1, 9, 16, True, [85, 9]), (128, 9, 3, 55, 128, False, [55, 64, 4001]),
]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("d,h_q,h_kv,n_tok,page,by_head,lens", ATTEND)
def test_attend(d, h_q, h_kv, n_tok, page, by_head, lens, dtype):
    gu.require_gpu()
    rng = np.random.default_rng(d + h_q + n_tok + sum(lens))
    c = Paged(rng, lens, page, h_kv, d, dtype, by_head, stale=NAN)
    check_attend(c, randn(rng, (len(lens) * n_tok, h_q, d), dtype, 2.0), trees_of(rng, len(lens), n_tok), dtype)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("h_q,n_tok", [(1, 15), (4, 24), (4, 63)])
def test_attend_kinds_of_trees_at_every_place_of_a_tile(h_q, n_tok, kind):
    gu.require_gpu()
    rng = np.random.default_rng(h_q + n_tok)
    lens = [n_tok + x for x in (0, 1, 31, 32, 33, 40, 63, 64, 65, 127)]
    c = Paged(rng, lens, 16, 1, 64, "bf16", stale=INF)
    check_attend(c, randn(rng, (len(lens) * n_tok, h_q, 64), "bf16", 2.0), trees_of(rng, len(lens), n_tok, (kind,)), "bf16")


@pytest.mark.parametrize("h_q,n_tok,n", [(2, 3, 400), (4, 24, 260), (8, 40, 60)])
def test_attend_many_sequences(h_q, n_tok, n):
    gu.require_gpu()
    rng = np.random.default_rng(n)
    lens = [int(x) if x >= n_tok else 0 for x in rng.integers(0, n_tok + 100, n)]
    c = Paged(rng, lens, 16, 2, 64, "f16", stale=NAN)
    check_attend(c, randn(rng, (n * n_tok, h_q, 64), "f16", 2.0), trees_of(rng, n, n_tok), "f16")


# more than 128 rows of d <= 128, and more blocks of rows than the kernel has workers: two blocks a worker
TOGETHER = [(128, 4, 1, 48, 33, 80), (64, 12, 3, 64, 16, 27), (128, 10, 2, 27, 64, 40), (128, 16, 1, 64, 48, 21), (64, 5, 1, 40, 5, 90)]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("d,h_q,h_kv,n_tok,page,n", TOGETHER)
def test_attend_blocks_of_rows_together(d, h_q, h_kv, n_tok, page, n, dtype):
    gu.require_gpu()
    rng = np.random.default_rng(d + n)
    lens = [int(x) if x >= n_tok else 0 for x in rng.integers(n_tok // 2, n_tok + 90, n)]
    lens[3], lens[n - 1] = 1500, n_tok
    c = Paged(rng, lens, page, h_kv, d, dtype, by_head=bool(n & 1), stale=NAN)
    check_attend(c, randn(rng, (n * n_tok, h_q, d), dtype, 2.0), trees_of(rng, n, n_tok), dtype)


@pytest.mark.parametrize("d,h_q,n_tok,n", [(128, 4, 40, 90), (64, 4, 64, 80)])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_attend_blocks_of_rows_together_see_their_paths_only(d, h_q, n_tok, n, bad):
    torch = gu.require_gpu()
    rng = np.random.default_rng(29)
    trees = trees_of(rng, n, n_tok, ("forest", "binary", "deep"))
    parents = parents_of(trees)
    c = Paged(rng, [n_tok + int(x) for x in rng.integers(0, 100, n)], 32, 1, d, "bf16")
    q = randn(rng, (n * n_tok, h_q, d), "bf16")
    clean, lse = attend(c, q, parents)
    again, lse2 = attend(c, q, parents)
    assert torch.equal(clean, again) and torch.equal(lse, lse2)
    hit = torch.zeros(d, dtype=torch.bool, device="cuda")
    hit[1::3] = True
    for s, j in ((0, 0), (7, n_tok // 2), (n - 1, 5)):
        under = torch.zeros(n * n_tok, dtype=torch.bool, device="cuda")
        under[s * n_tok:(s + 1) * n_tok] = torch.from_numpy(below(trees[s], j)).cuda()
        p = c.lens[s] - n_tok + j
        at = (int(c.table_np[s, p // 32]), p % 32)
        kept = c.k[at].clone(), c.v[at].clone()
        c.v[at[0], at[1], :, 1::3] = bad
        o, _ = attend(c, q, parents)
        assert torch.equal(o[~under], clean[~under]), (s, j)
        assert torch.all(~torch.isfinite(o[under][..., hit])) and torch.all(torch.isfinite(o[under][..., ~hit])), (s, j)
        c.k[at] = bad
        o, _ = attend(c, q, parents)
        assert torch.equal(o[~under], clean[~under]), (s, j)
        c.k[at], c.v[at] = kept
    no_error()


@pytest.mark.parametrize("d,h_q,n_tok", [(256, 1, 9), (128, 4, 24), (64, 8, 64)])
def test_attend_long_sequence_is_split_and_joined(d, h_q, n_tok):
    gu.require_gpu()
    rng = np.random.default_rng(d)
    c = Paged(rng, [30011], 64, 1, d, "bf16")
    check_attend(c, randn(rng, (n_tok, h_q, d), "bf16", 3.0), trees_of(rng, 1, n_tok), "bf16")


@pytest.mark.parametrize("dtype", DT)
# the same kernels on the same cuts: the same bits (many trees of more than 128 rows are cut otherwise)
@pytest.mark.parametrize("d,h_q,n_tok", [(128, 1, 16), (256, 4, 16), (64, 2, 5), (128, 8, 16), (256, 16, 16)])
def test_attend_a_chain_is_decode(d, h_q, n_tok, dtype):
    torch = gu.require_gpu()
    rng = np.random.default_rng(d + 1)
    c = Paged(rng, [300, 17, 0, 1000], 32, 1, d, dtype)
    q = randn(rng, (4 * n_tok, h_q, d), dtype)
    o, lse = attend(c, q, trees_of(rng, 4, n_tok, ("chain",)))
    o2, lse2 = nan_like(q.shape, q.dtype), nan_like(q.shape[:2], torch.float32)
    gdr.gdr_attn_decode(q, c.k, c.v, c.table, c.kv_lens, o2, n_tok, lse=lse2)
    torch.cuda.synchronize()
    no_error()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("d,h_q,n_tok", [(64, 1, 16), (128, 1, 16), (256, 4, 40), (64, 2, 64), (128, 4, 48), (256, 2, 64)])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_attend_rows_see_their_paths_only(d, h_q, n_tok, bad):
    torch = gu.require_gpu()
    rng = np.random.default_rng(23)
    n = n_tok + 139
    tree = tr.make(rng, n_tok, "forest")
    c = Paged(rng, [n], 32, 1, d, "bf16")
    q = randn(rng, (n_tok, h_q, d), "bf16")
    clean, _ = attend(c, q, [tree])
    for j in (0, 5, n_tok // 2, n_tok - 1):
        under = torch.from_numpy(below(tree, j)).cuda()
        p = n - n_tok + j
        at = (int(c.table_np[0, p // 32]), p % 32)
        kept = c.k[at].clone(), c.v[at].clone()
        c.v[at[0], at[1], :, 1::3] = bad
        o, _ = attend(c, q, [tree])
        assert torch.equal(o[~under], clean[~under]), j
        hit = torch.zeros(d, dtype=torch.bool, device="cuda")
        hit[1::3] = True
        assert torch.all(~torch.isfinite(o[under][..., hit])) and torch.all(torch.isfinite(o[under][..., ~hit])), j
        c.k[at] = bad
        o, _ = attend(c, q, [tree])
        assert torch.equal(o[~under], clean[~under]), j
        c.k[at], c.v[at] = kept
    no_error()


@pytest.mark.parametrize("h_q,n_tok", [(1, 12), (4, 30), (4, 50)])
def test_attend_scores_of_minus_infinity(h_q, n_tok):
    """Roots whose own and only score is minus infinity have nothing; a path with one such node is its others."""
    torch = gu.require_gpu()
    rng = np.random.default_rng(24)
    tree = [-1, -1] + [0] * (n_tok - 2)
    c = Paged(rng, [n_tok, n_tok + 64], 16, 1, 64, "bf16")
    q = randn(rng, (2 * n_tok, h_q, 64), "bf16")
    q[..., 0] = 1.0
    for s in range(2):
        p = c.lens[s] - n_tok  # node 0
        c.k[int(c.table_np[s, p // 16]), p % 16, :, 0] = -INF
    p = 64 // 2  # and a token before the second tree
    c.k[int(c.table_np[1, p // 16]), p % 16, :, 0] = -INF
    o, lse = attend(c, q, [tree] * 2)
    torch.cuda.synchronize()
    no_error()
    assert not o[0].any() and torch.all(lse[0] == -INF)
    for s in range(2):
        base = c.lens[s] - n_tok
        k, v = (ar.gather(f64(x), c.table_np[s], c.lens[s]) for x in (c.k, c.v))
        before = [i for i in range(base) if i != p]
        for j in range(n_tok):
            if s == 0 and j == 0:
                continue
            at = np.array(before + ([] if j == 0 else [base + j]), dtype=np.int64)
            for h in range(h_q):
                wo, wl, bo, bl = ar.attend(f64(q)[s * n_tok + j, h][None], k[at, 0], v[at, 0], 64 ** -0.5, [len(at)], "bf16")
                close(o[s * n_tok + j, h], wo[0], bo[0], "o")
                close(lse[s * n_tok + j, h], wl[0], bl[0], "lse")


def test_attend_strided_queries_outputs_and_tables():
    torch = gu.require_gpu()
    rng = np.random.default_rng(25)
    c = Paged(rng, [70, 33], 16, 2, 128, "bf16")
    trees = trees_of(rng, 2, 20, ("forest", "padded"))
    wide = randn(rng, (40, 12, 128), "bf16")
    o, _ = check_attend(c, wide[:, 2:10], trees, "bf16")
    table = torch.full((2, 64), -1, dtype=torch.int32, device="cuda")
    table[:, :c.table.shape[1]] = c.table
    o2 = nan_like((8, 40, 128), torch.bfloat16).transpose(0, 1)
    gdr.gdr_attn_decode_tree(wide[:, 2:10], c.k, c.v, table[:, :c.table.shape[1]], c.kv_lens, o2, parents_of(trees))
    torch.cuda.synchronize()
    assert torch.equal(o, o2)


@pytest.mark.parametrize("h_q,n_tok", [(4, 3), (8, 24), (8, 60)])
def test_attend_again_on_another_stream_and_in_a_graph(h_q, n_tok):
    torch = gu.require_gpu()
    rng = np.random.default_rng(26)
    c = Paged(rng, [5000, 140, 1300], 64, 2, 128, "bf16")
    trees = trees_of(rng, 3, n_tok)
    parents = parents_of(trees)
    q = randn(rng, (3 * n_tok, h_q, 128), "bf16")
    ws = torch.full((max(16, gdr.gdr_attn_decode_tree_workspace_bytes(q, c.k, parents)),), 255, dtype=torch.uint8, device="cuda")
    a, la = attend(c, q, parents)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b, lb = attend(c, q, parents, stream=s)
    d, _ = attend(c, q, parents, lse=False, workspace=ws)
    torch.cuda.synchronize()
    g = nan_like(q.shape, q.dtype)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdr.gdr_attn_decode_tree(q, c.k, c.v, c.table, c.kv_lens, g, parents, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(la, lb) and torch.equal(a, d) and torch.equal(a, g)
    # lengths and trees are read at replay
    c.kv_lens[1] = c.lens[1] = 192
    parents.copy_(parents_of(trees_of(rng, 3, n_tok, ("binary", "chain", "deep"))))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(g, attend(c, q, parents)[0]) and not torch.equal(a, g)
    no_error()


@pytest.mark.parametrize("h_q,n_tok", [(2, 3), (8, 24), (8, 60)])
def test_attend_on_two_streams_and_by_two_graphs_of_one_workspace(h_q, n_tok):
    torch = gu.require_gpu()
    rng = np.random.default_rng(28)
    cs = [Paged(rng, lens, 32, 2, 64, "bf16") for lens in ([900, 70, 0, 333], [64, 1500])]
    qs = [randn(rng, (len(c.lens) * n_tok, h_q, 64), "bf16") for c in cs]
    trees = [parents_of(trees_of(rng, len(c.lens), n_tok)) for c in cs]
    want = [attend(c, q, p) for c, q, p in zip(cs, qs, trees)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[attend(c, q, p, stream=s) for c, q, p, s in zip(cs, qs, trees, streams)] for _ in range(4)]
    torch.cuda.synchronize()
    for pairs in got:
        assert all(torch.equal(x, y) for a, b in zip(pairs, want) for x, y in zip(a, b))
    size = max(gdr.gdr_attn_decode_tree_workspace_bytes(q, c.k, p) for c, q, p in zip(cs, qs, trees))
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    outs, graphs = [nan_like(q.shape, q.dtype) for q in qs], []
    for c, q, p, o in zip(cs, qs, trees, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            gdr.gdr_attn_decode_tree(q, c.k, c.v, c.table, c.kv_lens, o, p, workspace=ws)
    for _ in range(3):
        for o, g in zip(outs, graphs):
            o.fill_(NAN)
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w[0]) for o, w in zip(outs, want))
    no_error()


@pytest.mark.parametrize("h_q,n_tok", [(1, 9), (4, 24), (4, 60)])
def test_attend_bad_trees_lengths_and_pages_are_recorded(h_q, n_tok):
    torch = gu.require_gpu()
    rng = np.random.default_rng(27)
    trees = trees_of(rng, 3, n_tok, ("chain", "draft", "binary"))
    c = Paged(rng, [200, 150, 90], 16, 1, 64, "bf16")
    q = randn(rng, (3 * n_tok, h_q, 64), "bf16")
    clean, _ = attend(c, q, trees)
    no_error()
    rest = torch.ones(3 * n_tok, dtype=torch.bool, device="cuda")
    rest[n_tok:2 * n_tok] = False
    for at, p in ((3, 3), (2, 1 << 30), (1, -7), (0, -(1 << 31))):
        bad = [list(t) for t in trees]
        bad[1][at] = p
        o, _ = attend(c, q, bad)
        assert gdr.gdr_device_error(device="cuda") == gdr.GDR_ERR_INVALID_ARG
        wo, _, bo, _ = tr.attend(bad, f64(q), f64(c.k), f64(c.v), c.table_np, c.lens, 0.125, "bf16")
        close(o, wo, bo, "o")
    for n in (n_tok - 1, 1, -1, -(1 << 31), 16 * c.table.shape[1] + 1, (1 << 31) - 1):
        c.kv_lens[1] = n
        o, lse = attend(c, q, trees)
        assert gdr.gdr_device_error(device="cuda") == gdr.GDR_ERR_INVALID_ARG, n
        assert torch.equal(o[rest], clean[rest]) and not o[~rest].any() and torch.all(lse[~rest] == -INF)
    c.kv_lens[1] = 0  # not in the batch: its parents may hold anything
    bad[1] = [12345] * n_tok
    o, _ = attend(c, q, bad)
    no_error()
    assert torch.equal(o[rest], clean[rest]) and not o[~rest].any()
    c.kv_lens[1] = 150
    c.table[1, 2] = c.k.shape[0]
    o, _ = attend(c, q, trees)
    assert gdr.gdr_device_error(device="cuda") == gdr.GDR_ERR_INVALID_ARG
    assert torch.equal(o[rest], clean[rest])


# --- append -------------------------------------------------------------------------------------------------

APPEND = [
    # d, h_q, h_kv, rot, interleaved, page, by_head, n_tok, kv_lens
    (256, 16, 4, 64, False, 64, False, 24, [1500]), (128, 8, 2, 128, True, 48, True, 7, [100, 7, 50]),
    (64, 3, 3, 24, False, 16, False, 33, [100, 33]), (64, 6, 1, 24, True, 5, True, 11, [11]),
    (128, 4, 4, 0, False, 16, False, 20, [21]), (256, 1, 1, 256, False, 16, True, 3, [4, 9000]),
    (128, 12, 4, 32, False, 128, False, 64, [300, 64, 128, 129]), (64, 4, 2, 64, False, 32, False, 1, [1000000, 1]),
    (256, 5, 1, 2, False, 32, False, 40, [40]), (64, 1, 1, 16, True, 32, True, 63, [63, 70]),
]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("d,h_q,h_kv,rot,il,page,by_head,n_tok,lens", APPEND)
def test_append(d, h_q, h_kv, rot, il, page, by_head, n_tok, lens, in_place, dtype):
    torch = gu.require_gpu()
    rng = np.random.default_rng(d + h_q + rot + sum(lens))
    n = len(lens)
    trees = trees_of(rng, n, n_tok, ("holes", "draft", "chain", "padded"))
    x = randn(rng, (n * n_tok, h_q + 2 * h_kv, d), dtype)
    real = torch.tensor([bool(p) for t in trees for p in tr.paths(t)], device="cuda")
    x[~real] = NAN
    q, k, v = x[:, :h_q], x[:, h_q:h_q + h_kv], x[:, h_q + h_kv:]
    inv = torch.from_numpy((10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))).astype(np.float32)).cuda()
    c = Paged(rng, lens, page, h_kv, d, dtype, by_head)
    k0, v0 = c.k.clone(), c.v.clone()
    q64, k64, v64 = f64(q), f64(k), f64(v)
    qo = q if in_place else torch.full((n * n_tok, h_q, d), 7.0, dtype=q.dtype, device="cuda")
    ko = k if in_place else torch.full((n * n_tok, h_kv, d), 7.0, dtype=q.dtype, device="cuda")
    gdr.gdr_attn_append_tree(q, k, v, qo, ko, c.k, c.v, c.table, c.kv_lens, inv if rot else None, parents_of(trees),
                             interleaved=il)
    torch.cuda.synchronize()
    no_error()
    at = np.flatnonzero(real.cpu().numpy())
    pos = np.concatenate([[m - n_tok + len(p) - 1 for p in tr.paths(t) if p] for t, m in zip(trees, lens)]).astype(np.int64)
    slot = np.concatenate([[m - n_tok + j for j, p in enumerate(tr.paths(t)) if p] for t, m in zip(trees, lens)]).astype(np.int64)
    for got, src, what in ((qo, q64, "q"), (ko, k64, "k")):
        want, size = ar.rotate(src[at], pos, inv.cpu().numpy(), il)
        close(got[real], want, ar.rotate_bound(want, size, dtype, rot), what)
        assert torch.all(torch.isnan(got[~real]) if in_place else got[~real] == 7.0)  # written nowhere
    page_of = c.table_np[at // n_tok, slot // page]
    k0[page_of, slot % page], v0[page_of, slot % page] = ko[real], torch.from_numpy(v64[at]).to(v0.dtype).cuda()
    assert torch.equal(c.k, k0) and torch.equal(c.v, v0)


def test_append_a_chain_is_append():
    torch = gu.require_gpu()
    rng = np.random.default_rng(30)
    c = Paged(rng, [40, 24, 300], 16, 2, 128, "bf16")
    q, k, v = (randn(rng, (72, h, 128), "bf16") for h in (8, 2, 2))
    inv = torch.from_numpy((10000.0 ** (-np.arange(32) / 32)).astype(np.float32)).cuda()
    out = []
    for tree in (False, True):
        qo, kc, vc = torch.empty_like(q), c.k.clone(), c.v.clone()
        if tree:
            gdr.gdr_attn_append_tree(q, k, v, qo, None, kc, vc, c.table, c.kv_lens, inv, parents_of(trees_of(rng, 3, 24, ("chain",))))
        else:
            gdr.gdr_attn_append(q, k, v, qo, None, kc, vc, c.table, c.kv_lens, inv)
        out.append((qo, kc, vc))
    assert all(torch.equal(a, b) for a, b in zip(*out))
    no_error()


def test_append_keys_alone_and_what_has_no_slot():
    torch = gu.require_gpu()
    rng = np.random.default_rng(31)
    trees = trees_of(rng, 4, 10, ("forest", "draft", "none", "chain"))
    parents = parents_of(trees)
    c = Paged(rng, [40, 30, 20, 50], 16, 2, 64, "bf16")
    k, v = (randn(rng, (40, 2, 64), "bf16") for _ in range(2))
    kc, vc = c.k.clone(), c.v.clone()

    def append(p=parents):
        c.k.copy_(kc), c.v.copy_(vc)
        gdr.gdr_attn_append_tree(None, k, v, None, None, c.k, c.v, c.table, c.kv_lens, None, p)
        return c.k.clone(), c.v.clone()

    whole = append()
    no_error()
    for n in (9, 1, 0, -5, 16 * c.table.shape[1] + 1, -(1 << 31)):
        c.kv_lens[2] = n  # no node in it: nothing to say
        assert all(torch.equal(a, b) for a, b in zip(append(), whole))
        no_error()
    c.kv_lens[2] = 20
    for bad in (11, 10 + 40, -3):
        p = parents.clone()
        p[0, 4] = bad  # the row and those under it are no nodes
        got = append(p)
        assert gdr.gdr_device_error(device="cuda") == gdr.GDR_ERR_INVALID_ARG
        t = [list(x) for x in trees]
        t[0][4] = bad
        for j, path in enumerate(tr.paths(t[0])):
            at = int(c.table_np[0, (30 + j) // 16]), (30 + j) % 16
            assert torch.equal(got[0][at], (whole if path else (kc,))[0][at]), j
    for n in (9, 0, -1, 16 * c.table.shape[1] + 1):  # sequence 3 has no slots
        c.kv_lens[3] = n
        got = append()
        assert gdr.gdr_device_error(device="cuda") == gdr.GDR_ERR_INVALID_ARG, n
        for s in range(3):
            at = torch.from_numpy(c.table_np[s, :-(-c.lens[s] // 16)]).long().cuda()
            assert torch.equal(got[0][at], whole[0][at]), (n, s)


# --- compaction ---------------------------------------------------------------------------------------------

COMPACT = [
    # layers (0: one cache without a layers' dimension), h_kv, d, page, by_head, n_tok, lens
    (0, 2, 64, 16, False, 1, [1, 40]), (1, 4, 256, 64, False, 24, [1500, 24]), (3, 2, 128, 48, True, 7, [100, 7, 0, 50]),
    (8, 1, 64, 5, False, 33, [100, 33]), (2, 3, 64, 1, True, 64, [64, 65, 200]), (5, 4, 256, 33, False, 64, [64, 0, 0, 900]),
    (32, 8, 128, 128, False, 41, [129, 300]), (0, 1, 256, 7, True, 63, [63]),
]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("layers,h_kv,d,page,by_head,n_tok,lens", COMPACT)
def test_compact(layers, h_kv, d, page, by_head, n_tok, lens, dtype):
    torch = gu.require_gpu()
    rng = np.random.default_rng(layers + d + n_tok)
    n = len(lens)
    c = Paged(rng, lens, page, h_kv, d, dtype, by_head)
    shape = (max(1, layers),) + ((c.k.shape[0], h_kv, page, d) if by_head else tuple(c.k.shape))
    kk, vv = randn(rng, shape, dtype), randn(rng, shape, dtype)
    if by_head:
        kk, vv = kk.transpose(2, 3), vv.transpose(2, 3)
    if not layers:
        kk, vv = kk[0], vv[0]
    for kinds in (("holes", "draft"), ("chain", "forest", "deep"), ("padded", "roots", "binary", "star")):
        trees = trees_of(rng, n, n_tok, kinds)
        paths = [tr.paths(t) for t in trees]
        last = [int(rng.choice(np.r_[-1, [j for j in range(n_tok) if p[j]] * 3])) if m else -1 for p, m in zip(paths, lens)]
        k, v = kk.clone(memory_format=torch.preserve_format), vv.clone(memory_format=torch.preserve_format)
        out = ints([-9] * (n + 1))
        gdr.gdr_attn_commit_tree(k, v, c.table, c.kv_lens, parents_of(trees), ints(last), out[:n])
        torch.cuda.synchronize()
        no_error()
        wk, wv = kk.clone(memory_format=torch.preserve_format), vv.clone(memory_format=torch.preserve_format)
        for s in range(n):
            base = lens[s] - n_tok
            path = paths[s][last[s]] if last[s] >= 0 else []
            for i, j in enumerate(path):
                to, frm = base + i, base + j
                for w, src in ((wk, kk), (wv, vv)):
                    w, src = (w, src) if layers else (w[None], src[None])
                    w[:, int(c.table_np[s, to // page]), to % page] = src[:, int(c.table_np[s, frm // page]), frm % page]
            assert int(out[s]) == (base + len(path) if lens[s] else 0)
        assert int(out[n]) == -9
        # the accepted slots and everything before the trees and outside them; not the trees' other slots
        for s in range(n):
            base = lens[s] - n_tok
            if base < 0:
                continue
            for x in range(base + (len(paths[s][last[s]]) if last[s] >= 0 else 0), lens[s]):
                at = int(c.table_np[s, x // page]), x % page
                for got, w in ((k, wk), (v, wv)):
                    got, w = (got, w) if layers else (got[None], w[None])
                    w[:, at[0], at[1]] = got[:, at[0], at[1]]
        assert torch.equal(k, wk) and torch.equal(v, wv)


def test_compact_records_what_it_leaves_out():
    torch = gu.require_gpu()
    rng = np.random.default_rng(41)
    tree = [-1, -1, 1, 0, 2, -2, 4, 3]
    c = Paged(rng, [40, 30], 8, 2, 64, "bf16")
    k0, v0 = c.k.clone(), c.v.clone()

    def run(last, trees=(tree, tree), lens=None):
        c.k.copy_(k0), c.v.copy_(v0)
        out = ints([-9, -9])
        gdr.gdr_attn_commit_tree(c.k, c.v, c.table, ints(lens or c.lens), parents_of(list(trees)), ints(last), out)
        return gdr.gdr_device_error(device="cuda"), out.tolist()

    assert run([-1, -1]) == (gdr.GDR_OK, [32, 22]) and torch.equal(c.k, k0)
    assert run([6, 7]) == (gdr.GDR_OK, [36, 25]) and not torch.equal(c.k, k0)
    for last in (8, -2, 5, 64, 1 << 30, -(1 << 31)):
        assert run([last, -1]) == (gdr.GDR_ERR_INVALID_ARG, [32, 22]) and torch.equal(c.k, k0), last
    bad = [-1, 9, 1, 0, 2, -2, 4, 3]
    assert run([7, -1], (bad, tree)) == (gdr.GDR_ERR_INVALID_ARG, [35, 22])
    assert run([6, -1], (bad, tree)) == (gdr.GDR_ERR_INVALID_ARG, [32, 22]) and torch.equal(c.k, k0)
    top = 8 * c.table.shape[1]
    for n in (7, 1, -1, top + 1, -(1 << 31), (1 << 31) - 1):
        assert run([6, -1], lens=[n, 30]) == (gdr.GDR_ERR_INVALID_ARG, [n, 22]) and torch.equal(c.k, k0), n
    assert run([-1, -1], lens=[0, 30]) == (gdr.GDR_OK, [0, 22])
    run([6, 7])
    moved = c.k.clone()
    c.k.copy_(k0), c.v.copy_(v0)
    gdr.gdr_attn_commit_tree(c.k, c.v, c.table, ints(c.lens), parents_of([tree, tree]), ints([6, 7]))  # no lengths
    assert torch.equal(c.k, moved)
    for page in (-1, c.k.shape[0], 1 << 30):
        kept = c.table.clone()
        c.table[0, 4] = page  # of the slots 32 .. 39
        assert run([6, -1])[0] == gdr.GDR_ERR_INVALID_ARG and torch.equal(c.k, k0) and torch.equal(c.v, v0)
        c.table.copy_(kept)
    with pytest.raises(gdr.GdrError):  # lengths in place
        gdr.gdr_attn_commit_tree(c.k, c.v, c.table, c.kv_lens, parents_of([tree] * 2), ints([0, 0]), c.kv_lens)
    with pytest.raises(gdr.GdrError):  # layers that are one
        gdr.gdr_attn_commit_tree(c.k.expand(3, -1, -1, -1, -1), c.v.expand(3, -1, -1, -1, -1), c.table, c.kv_lens,
                                 parents_of([tree] * 2), ints([0, 0]))
    with pytest.raises(gdr.GdrError):
        gdr.gdr_attn_commit_tree(c.k[:1].expand(4, -1, -1, -1), c.v[:1].expand(4, -1, -1, -1), c.table, c.kv_lens,
                                 parents_of([tree] * 2), ints([0, 0]))
    no_error()


# --- together -----------------------------------------------------------------------------------------------

@pytest.mark.parametrize("n_tok", [6, 24, 64])
def test_draft_verify_accept_and_go_on(n_tok):
    """Three steps of drafting trees and accepting a path in an attention layer pair and a layer of the rule; what is
    left is what the accepted tokens leave when they are fed one after another."""
    torch = gu.require_gpu()
    rng = np.random.default_rng(50 + n_tok)
    n, h_q, h_kv, d, page, layers, rot = 3, 4, 2, 128, 16, 2, 64
    start = [50, 16, 99]
    room = [x + 4 * n_tok for x in start]
    c = Paged(rng, room, page, h_kv, d, "bf16")
    kk, vv = (randn(rng, (layers,) + tuple(c.k.shape), "bf16") for _ in range(2))
    plain_k, plain_v = kk.clone(), vv.clone()
    inv = torch.from_numpy((10000.0 ** (-np.arange(rot // 2) / (rot // 2))).astype(np.float32)).cuda()
    lens = ints(start)
    state = 0.3 * torch.from_numpy(rng.standard_normal((n, 4, d, d))).float().cuda()
    seq_state = state.clone()
    for step in range(3):
        trees = trees_of(rng, n, n_tok, ("draft", "deep", "holes"))
        last = [int(rng.choice([j for j, p in enumerate(tr.paths(t)) if p])) for t in trees]
        if step == 1:
            last[0] = -1  # nothing accepted
        parents = parents_of(trees)
        b = Batch(rng, trees, 2, 4, d, "bf16")
        b.state = state
        o, u = b.run()
        gdr.gdr_verify_tree_commit(b.k, b.g, u, state, parents, ints(last))
        with_tree = lens + n_tok
        qkv = [[randn(rng, (n * n_tok, h, d), "bf16") for h in (h_q, h_kv, h_kv)] for _ in range(layers)]
        out = []
        for l, (q, k, v) in enumerate(qkv):
            qr = torch.empty_like(q)
            gdr.gdr_attn_append_tree(q, k, v, qr, None, kk[l], vv[l], c.table, with_tree, inv, parents)
            a = nan_like(q.shape, q.dtype)
            gdr.gdr_attn_decode_tree(qr, kk[l], vv[l], c.table, with_tree, a, parents)
            out.append(a)
        new = torch.empty_like(lens)
        gdr.gdr_attn_commit_tree(kk, vv, c.table, with_tree, parents, ints(last), new)
        # the accepted tokens one after another
        for s in range(n):
            path = tr.paths(trees[s])[last[s]] if last[s] >= 0 else []
            for i, j in enumerate(path):
                r = slice(s * n_tok + j, s * n_tok + j + 1)
                o1 = torch.empty(1, 4, d, device="cuda")
                gdr.gdr_decode_step(b.q[r], b.k[r], b.v[r], b.g[r], b.beta[r], seq_state[s:s + 1], o1)
                assert float((o1 - o[r]).norm() / o1.norm()) <= 1e-4
                at = lens[s:s + 1] + i + 1
                for l, (q, k, v) in enumerate(qkv):
                    q1 = torch.empty_like(q[r])
                    gdr.gdr_attn_append(q[r], k[r], v[r], q1, None, plain_k[l], plain_v[l], c.table[s:s + 1], at, inv)
                    a1 = torch.empty_like(q1)
                    gdr.gdr_attn_decode(q1, plain_k[l], plain_v[l], c.table[s:s + 1], at, a1)
                    # either is within 2 h = 2^-7 of A (tests/attn_ref.py), which is under max |v| < 6
                    assert float((a1.float() - out[l][r].float()).abs().max()) <= 2.0 ** -6 * 6
            assert int(new[s]) == int(lens[s]) + len(path)
        lens = new
        for s in range(n):
            p = np.arange(int(lens[s]))
            for x, y in ((kk, plain_k), (vv, plain_v)):
                at = torch.from_numpy(c.table_np[s, p // page].astype(np.int64)).cuda(), torch.from_numpy(p % page).cuda()
                assert torch.equal(x[:, at[0], at[1]], y[:, at[0], at[1]])
        assert float((state - seq_state).norm() / seq_state.norm()) <= 1e-5
    no_error()
