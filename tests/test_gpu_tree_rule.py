"""The rule over trees of drafted tokens on the GPU (gdr_verify_tree, gdr_verify_tree_commit) against the 64-bit
reference (tests/tree_ref.py) at its derived bounds."""

import numpy as np
import pytest

import gated_deltanet_scan_gb300 as gdr
from tests import gpu_util as gu
from tests import tree_ref as tr
from tests.test_gpu_attn import close, f64, ints, no_error

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
BF16_STEP = 2.0 ** -8  # at most, of a value's rounding to bf16


class Batch:
    """Inputs of one call; rows that are no nodes hold NaN throughout."""

    def __init__(self, rng, trees, h_qk, h_v, d, dtype, g_max=2.0, raw=False):
        torch = gu.torch_mod()
        io = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.trees, self.n, self.n_tok, self.d, self.raw = trees, len(trees), len(trees[0]), d, raw
        T = self.n * self.n_tok

        def dev(x, dt=torch.float32):
            return torch.from_numpy(x).to(dt).cuda()

        q, k = rng.standard_normal((2, T, h_qk, d))
        if not raw:
            q, k = (x / np.linalg.norm(x, axis=2, keepdims=True) for x in (q, k))
        self.q, self.k, self.v = dev(q, io), dev(k, io), dev(rng.standard_normal((T, h_v, d)), io)
        self.g = dev(-rng.uniform(0.001, g_max, (T, h_v)))
        self.beta = dev(rng.standard_normal((T, h_v)) if raw else rng.uniform(0, 1, (T, h_v)))
        self.state = dev(0.5 * rng.standard_normal((self.n, h_v, d, d)))
        self.parents = torch.tensor(trees, dtype=torch.int32, device="cuda")
        self.real = np.array([[bool(p) for p in tr.paths(t)] for t in trees])
        gone = torch.from_numpy(~self.real.reshape(-1)).cuda()
        for x in (self.q, self.k, self.v, self.g, self.beta):
            x[gone] = NAN

    def run(self, out="f32", deltas=True, scale=1.0, stream=None):
        torch = gu.torch_mod()
        o = torch.full(self.v.shape, NAN, dtype=torch.bfloat16 if out == "bf16" else torch.float32, device="cuda")
        u = torch.full(self.v.shape, NAN, dtype=torch.float32, device="cuda") if deltas else None
        gdr.gdr_verify_tree(self.q, self.k, self.v, self.g, self.beta, self.state, o, self.parents, deltas=u,
                            scale=scale, qk_l2norm=self.raw, beta_logits=self.raw, stream=stream)
        return o, u

    def settle(self, u, last, state=None):
        gdr.gdr_verify_tree_commit(self.k, self.g, u, self.state if state is None else state, self.parents, ints(last),
                                   qk_l2norm=self.raw)

    def host(self):
        """q, k, v, g, beta, state as the rule takes them, rows that are no nodes as zeros."""
        x = [np.nan_to_num(f64(y)) for y in (self.q, self.k, self.v, self.g, self.beta)] + [f64(self.state)]
        if self.raw:
            for i in (0, 1):
                x[i] = x[i] / np.sqrt((x[i] ** 2).sum(2, keepdims=True) + 1e-6)
            x[4] = 1.0 / (1.0 + np.exp(-x[4]))
        return x

    def want(self, scale=1.0):
        q, k, v, g, beta, state = self.host()
        group = v.shape[1] // q.shape[1]
        o, u, bo, bu = (np.zeros(v.shape) for _ in range(4))
        for s in range(self.n):
            r = slice(s * self.n_tok, (s + 1) * self.n_tok)
            for h in range(v.shape[1]):
                o[r, h], u[r, h], bo[r, h], bu[r, h], _ = tr.rule(
                    self.trees[s], scale * q[r, h // group], k[r, h // group], v[r, h], g[r, h], beta[r, h], state[s, h])
        return o, u, bo, bu

    def check(self, out="f32", scale=1.0):
        torch = gu.torch_mod()
        before = self.state.clone()
        o, u = self.run(out, scale=scale)
        torch.cuda.synchronize()
        no_error()
        assert torch.equal(self.state, before)  # only read
        wo, wu, bo, bu = self.want(scale)
        if out == "bf16":
            bo = bo + BF16_STEP * (np.abs(wo) + bo)
        close(u, wu, bu, "u")
        close(o, wo, bo, "o")
        return o, u

    def check_settle(self, u, last):
        torch = gu.torch_mod()
        _, k, _, g, _, state = self.host()
        u64 = np.nan_to_num(f64(u))
        group = u64.shape[1] // k.shape[1]
        new = self.state.clone()
        self.settle(u, last, new)
        torch.cuda.synchronize()
        no_error()
        want, bound = state.copy(), np.zeros_like(state)
        for s in range(self.n):
            r = slice(s * self.n_tok, (s + 1) * self.n_tok)
            for h in range(u64.shape[1]):
                want[s, h], bound[s, h] = tr.settle(self.trees[s], last[s], k[r, h // group], g[r, h], u64[r, h], state[s, h])
        close(new, want, bound, "state")
        return new


RULE = [
    # d, h_qk, h_v, n_tok, trees
    (128, 1, 1, 1, ["roots"]), (128, 2, 2, 2, ["chain", "none"]), (64, 1, 1, 3, ["star"]),
    (128, 16, 32, 24, ["draft"]), (128, 2, 4, 41, ["forest", "holes", "padded"]), (64, 2, 2, 17, ["binary", "roots"]),
    (128, 1, 4, 64, ["chain", "draft"]), (64, 3, 3, 64, ["deep", "holes"]), (128, 4, 4, 33, ["deep", "none", "chain"]),
    (128, 1, 2, 16, ["chain"]), (128, 1, 1, 63, ["binary"]), (128, 2, 6, 31, ["star", "roots", "padded"]),
    (64, 1, 8, 48, ["forest"]), (128, 1, 3, 64, ["binary", "star", "deep"]), (32, 1, 2, 20, ["draft", "padded"]),
    (32, 2, 2, 64, ["chain", "holes"]), (32, 1, 1, 63, ["forest"]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,h_qk,h_v,n_tok,kinds", RULE)
def test_rule_and_settle(d, h_qk, h_v, n_tok, kinds, dtype):
    gu.require_gpu()
    rng = np.random.default_rng(d + h_v + n_tok)
    b = Batch(rng, [tr.make(rng, n_tok, kind) for kind in kinds], h_qk, h_v, d, dtype)
    _, u = b.check()
    nodes = [np.flatnonzero(r) for r in b.real]
    for pick in (lambda x: int(x[-1]), lambda x: int(x[0]), lambda x: int(rng.choice(x))):
        b.check_settle(u, [pick(x) if len(x) else -1 for x in nodes])
    assert gu.torch_mod().equal(b.check_settle(u, [-1] * b.n), b.state)  # none accepted: bit for bit


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("h_qk,h_v,n_seqs,n_tok", [(1, 1, 160, 5), (2, 8, 50, 24), (4, 4, 153, 33), (1, 2, 77, 64)])
def test_more_pairs_than_blocks(h_qk, h_v, n_seqs, n_tok, dtype):
    gu.require_gpu()
    rng = np.random.default_rng(n_seqs)
    kinds = ("padded", "chain", "forest", "holes", "none", "star", "binary", "deep")
    b = Batch(rng, [tr.make(rng, n_tok, kinds[s % len(kinds)]) for s in range(n_seqs)], h_qk, h_v, 64, dtype)
    _, u = b.check()
    last = [int(rng.choice(np.r_[-1, np.flatnonzero(r)])) for r in b.real]
    b.check_settle(u, last)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("h_qk,h_v,n_seqs,n_tok", [(2, 4, 19, 7), (4, 8, 10, 24), (8, 8, 24, 12), (1, 4, 40, 64)])
def test_more_pairs_than_blocks_of_128_columns(h_qk, h_v, n_seqs, n_tok, dtype):
    """76 pairs and more: fp32 kernels on either side of it, and more than a bf16 block each."""
    gu.require_gpu()
    rng = np.random.default_rng(n_seqs + n_tok)
    kinds = ("deep", "holes", "draft", "chain", "padded")
    b = Batch(rng, [tr.make(rng, n_tok, kinds[s % len(kinds)]) for s in range(n_seqs)], h_qk, h_v, 128, dtype)
    _, u = b.check()
    b.check_settle(u, [int(rng.choice(np.r_[-1, np.flatnonzero(r)])) for r in b.real])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_two_streams_at_once(dtype):
    torch = gu.require_gpu()
    rng = np.random.default_rng(13)
    b = Batch(rng, [tr.make(rng, 40, kind) for kind in ("draft", "chain", "forest") * 4], 4, 8, 128, dtype)
    o, u = b.run()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    out = [[b.run(stream=s) for s in streams] for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, o) and torch.equal(y, u) for pair in out for x, y in pair)
    no_error()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1.0, 128 ** -0.5, -0.3, 0.0])
def test_flags_scales_and_bf16_outputs(scale, dtype):
    gu.require_gpu()
    rng = np.random.default_rng(3)
    b = Batch(rng, [tr.make(rng, 40, kind) for kind in ("draft", "holes")], 2, 4, 128, dtype, raw=True)
    _, u = b.check(scale=scale)
    b.check(out="bf16", scale=scale)
    b.check_settle(u, [int(np.flatnonzero(r)[-1]) for r in b.real])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_without_deltas_again_and_on_another_stream(dtype):
    torch = gu.require_gpu()
    rng = np.random.default_rng(4)
    b = Batch(rng, [tr.make(rng, 24, kind) for kind in ("forest", "deep", "none")], 2, 4, 128, dtype)
    o, u = b.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o2, u2 = b.run(stream=s)
    o3, none = b.run(deltas=False)
    torch.cuda.synchronize()
    assert none is None and torch.equal(o, o2) and torch.equal(u, u2) and torch.equal(o, o3)
    gone = torch.from_numpy(~b.real.reshape(-1)).cuda()
    assert not o[gone].any() and not u[gone].any()  # set to zero
    no_error()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_tok", [1, 5, 16])
def test_a_chain_is_a_verify_block(n_tok, dtype):
    torch = gu.require_gpu()
    rng = np.random.default_rng(5)
    b = Batch(rng, [tr.make(rng, n_tok, "chain")] * 3, 2, 4, 128, dtype)
    o, u = b.check()
    state, snap, o2, u2 = b.state.clone(), torch.empty_like(b.state), torch.empty_like(o), torch.empty_like(u)
    gdr.gdr_verify_block(b.q, b.k, b.v, b.g, b.beta, state, snap, o2, n_tok, deltas=u2)
    new = b.check_settle(u, [n_tok - 1] * 3)
    # either is within the reference's bound, the block's by the same count of roundings
    _, _, bo, bu = b.want()
    close(o2, f64(o), 2 * bo, "o")
    close(u2, f64(u), 2 * bu, "u")
    assert float((state - new).norm() / new.norm()) <= 1e-5
    no_error()


def below(parents, at):
    """Rows whose path holds `at`."""
    return np.array([at in p for p in tr.paths(parents)])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_tok", [24, 64])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_what_a_row_holds_reaches_only_the_paths_it_is_on(bad, n_tok, dtype):
    torch = gu.require_gpu()
    rng = np.random.default_rng(6)
    b = Batch(rng, [tr.make(rng, n_tok, kind) for kind in ("forest", "deep", "binary")], 2, 4, 128, dtype)
    clean, cu = b.run()
    hit = torch.zeros(128, dtype=torch.bool, device="cuda")
    hit[3::5] = True
    for at in (0, 7, n_tok // 2, n_tok - 1):
        under = np.concatenate([below(t, at) for t in b.trees])
        keep, under = torch.from_numpy(~under).cuda(), torch.from_numpy(under).cuda()
        row = torch.arange(b.n, device="cuda") * n_tok + at
        for name in ("v", "q", "k", "g", "beta"):
            x = getattr(b, name)
            kept = x.clone()
            if name == "v":
                x[row[:, None], :, 3::5] = bad
            else:
                x[row] = bad
            o, u = b.run()
            assert torch.equal(o[keep], clean[keep]) and torch.equal(u[keep], cu[keep]), (name, at)
            if name == "v":  # its columns, and no others
                assert torch.all(~torch.isfinite(o[under][..., hit])) and torch.all(~torch.isfinite(u[under][..., hit]))
                assert torch.equal(u[under][..., ~hit], cu[under][..., ~hit])
                assert torch.equal(o[under][..., ~hit], clean[under][..., ~hit])
            setattr(b, name, kept)
    no_error()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_bad_state_stays_in_its_column(dtype):
    torch = gu.require_gpu()
    rng = np.random.default_rng(7)
    b = Batch(rng, [tr.make(rng, 30, kind) for kind in ("forest", "draft")], 1, 2, 128, dtype)
    clean, cu = b.run()
    b.state[1, 0, 5, 9], b.state[1, 1, 100, 127], b.state[0, 1, 64, 0] = NAN, INF, -INF
    o, u = b.run()
    hit = torch.zeros_like(o, dtype=torch.bool)
    hit[30:, 0, 9] = hit[30:, 1, 127] = hit[:30, 1, 0] = True
    assert torch.all(~torch.isfinite(o[hit])) and torch.all(~torch.isfinite(u[hit]))
    assert torch.equal(o[~hit], clean[~hit]) and torch.equal(u[~hit], cu[~hit])
    no_error()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("low", [-INF, -1e30, -2e4, -300.0])
def test_a_gate_that_forgets_everything(low, dtype):
    """e^g = 0: the nodes from there on are what they would be on an empty state and path."""
    torch = gu.require_gpu()
    rng = np.random.default_rng(8)
    b = Batch(rng, [tr.make(rng, 33, kind) for kind in ("chain", "binary")], 1, 2, 128, dtype)
    b.g[5] = b.g[33 + 2] = low
    o, u = b.run()
    torch.cuda.synchronize()
    b.g[5] = b.g[33 + 2] = -300.0  # its exponential is below the smallest number of either precision here
    wo, wu, bo, bu = b.want()
    close(u, wu, bu, "u")
    close(o, wo, bo, "o")
    b.g[5] = b.g[33 + 2] = low
    state = b.state.clone()
    b.settle(u, [32, 32], state)
    _, k, _, g, _, s0 = b.host()
    g = np.maximum(f64(b.g), -300.0)
    for s in range(2):
        r = slice(33 * s, 33 * s + 33)
        for h in range(2):
            want, bound = tr.settle(b.trees[s], 32, k[r, 0], g[r, h], f64(u)[r, h], s0[s, h])
            close(state[s, h], want, bound, "state")
    no_error()


def test_long_decays_keep_their_differences():
    """Sums of gates of some -2000 whose differences are small."""
    gu.require_gpu()
    rng = np.random.default_rng(9)
    for dtype in ("bf16", "f32"):
        b = Batch(rng, [tr.make(rng, 64, "chain")], 1, 2, 128, dtype, g_max=0.05)
        b.g[:32] -= 60.0
        b.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_parents_and_last_are_recorded_and_are_no_nodes(dtype):
    torch = gu.require_gpu()
    rng = np.random.default_rng(10)
    good = [-1, 0, 1, -1, 3, 1, -2, 0]
    for at, p, gone in ((2, 2, [2]), (0, 5, [0, 1, 2, 5, 7]), (4, -3, [4]), (7, 6, [7]), (3, 1 << 30, [3, 4]),
                        (1, -(1 << 31), [1, 2, 5])):
        bad = list(good)
        bad[at] = p
        b = Batch(rng, [good, bad], 1, 2, 128, dtype)
        assert set(np.flatnonzero(~b.real[1])) == set(gone + [6])
        o, u = b.run()
        assert gdr.gdr_device_error(device="cuda") == gdr.GDR_ERR_INVALID_ARG
        wo, wu, bo, bu = b.want()
        close(u, wu, bu, "u")
        close(o, wo, bo, "o")
    b = Batch(rng, [good] * 7, 1, 2, 128, dtype)
    _, u = b.run()
    no_error()
    for n in (7, 70):  # a few states, and many
        b = Batch(rng, [good] * n, 1, 2, 128, dtype)
        _, u = b.run()
        for last in (8, -2, 6, 64, 1 << 30, -(1 << 31), 32):
            state = b.state.clone()
            b.settle(u, [4] + [last] + [-1] * (n - 2), state)
            assert gdr.gdr_device_error(device="cuda") == gdr.GDR_ERR_INVALID_ARG, last
            assert torch.equal(state[1:], b.state[1:]) and not torch.equal(state[0], b.state[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_a_graph(dtype):
    """Trees, gates and accepted nodes are read at replay."""
    torch = gu.require_gpu()
    rng = np.random.default_rng(11)
    b = Batch(rng, [tr.make(rng, 24, kind) for kind in ("draft", "forest", "chain")], 2, 4, 128, dtype)
    o, u = b.run()
    last, start = ints([3, -1, 20]), b.state.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdr.gdr_verify_tree(b.q, b.k, b.v, b.g, b.beta, b.state, o, b.parents, deltas=u)
        gdr.gdr_verify_tree_commit(b.k, b.g, u, b.state, b.parents, last)
    for kinds, a in ((("draft", "forest", "chain"), [3, -1, 20]), (("chain", "binary", "star"), [23, 22, 0])):
        b.trees = [tr.make(rng, 24, kind) for kind in kinds]
        b.parents.copy_(torch.tensor(b.trees, dtype=torch.int32))
        last.copy_(torch.tensor(a, dtype=torch.int32))
        b.state.copy_(start)
        o.fill_(NAN), u.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        new = b.state.clone()
        b.state.copy_(start)
        o2, u2 = b.run()
        b.settle(u2, a)
        assert torch.equal(o, o2) and torch.equal(u, u2) and torch.equal(new, b.state)
    no_error()


def test_empty_batches_and_rows_behind_the_last_tree():
    torch = gu.require_gpu()
    rng = np.random.default_rng(12)
    b = Batch(rng, [tr.make(rng, 7, "forest")] * 2, 1, 2, 128, "bf16")
    z = slice(0, 0)
    gdr.gdr_verify_tree(b.q[z], b.k[z], b.v[z], b.g[z], b.beta[z], b.state[z], b.v[z].float(), b.parents[z])
    gdr.gdr_verify_tree_commit(b.k[z], b.g[z], b.v[z].float(), b.state[z], b.parents[z], ints([]))
    o, u = (torch.full((20, 2, 128), 7.0, device="cuda") for _ in range(2))
    gdr.gdr_verify_tree(b.q, b.k, b.v, b.g, b.beta, b.state, o[:14], b.parents, deltas=u[:14])
    state = torch.full((3, 2, 128, 128), 7.0, device="cuda")
    gdr.gdr_verify_tree_commit(b.k, b.g, u[:14], state[:2], b.parents, ints([6, 3]))
    torch.cuda.synchronize()
    for x in (o[14:], u[14:], state[2]):
        assert torch.all(x == 7.0)
    no_error()
