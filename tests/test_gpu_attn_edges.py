"""Attention operators on the GPU at values, scales and arguments where they can go wrong: infinite keys and
values that a token does see, scales near zero, and what the device checks itself."""

import numpy as np
import pytest

import gated_deltanet_scan_gb300 as gdr
from tests import attn_ref as ar
from tests import gpu_util as gu
from tests.test_gpu_attn import Paged, check_decode, check_prefill, close, f64, ints, nan_like, no_error, randn, run_decode

pytestmark = pytest.mark.gpu

INF = float("inf")
NAN = float("nan")


# --- infinite values ------------------------------------------------------------------------------------------

def takes(got, bad):
    """All of got is the infinity `bad`, or NaN where bad is."""
    torch = gu.torch_mod()
    return bool(torch.all(torch.isnan(got) if bad != bad else got == bad))


@pytest.mark.parametrize("dtype", ("bf16", "f16"))
@pytest.mark.parametrize("d,hq", [(64, 1), (64, 3), (128, 2), (256, 1), (256, 4)])
@pytest.mark.parametrize("bad", [INF, -INF, NAN])
def test_prefill_rows_take_the_infinity_of_a_value_they_see(d, hq, bad, dtype):
    """Scores of normal variates divided by their deviation: every weight is over 2^-24 of the largest, so what a
    column of an infinite value gives is that infinity, in both kernels (64 and 90 tokens, and 300)."""
    torch = gu.require_gpu()
    rng = np.random.default_rng(70 + d)
    lens = [64, 300, 90 if hq < 3 else 57]
    T, ends = sum(lens), [int(x) for x in np.cumsum(lens)]
    q, k, v = randn(rng, (T, hq, d), dtype), randn(rng, (T, 1, d), dtype), randn(rng, (T, 1, d), dtype)
    cu = ints([0] + ends)
    hit = torch.zeros(d, dtype=torch.bool, device="cuda")
    hit[3::5] = True
    for at in (0, 31, 32, 63, 64, 64 + 127, 64 + 128, 64 + 250, 363, 364, T - 1):
        v2 = v.clone()
        v2[at, :, 3::5] = bad
        o = nan_like((T, hq, d), q.dtype)
        gdr.gdr_attn_prefill(q, k, v2, o, cu)
        end = next(e for e in ends if e > at)
        assert takes(o[at:end][..., hit], bad), at
        assert torch.all(torch.isfinite(o[at:end][..., ~hit])), at
        rest = torch.ones(T, dtype=torch.bool, device="cuda")
        rest[at:end] = False
        assert torch.all(torch.isfinite(o[rest])), at
    no_error()


@pytest.mark.parametrize("n", [90, 300])
def test_prefill_opposite_infinities_cancel_to_nan(n):
    torch = gu.require_gpu()
    rng = np.random.default_rng(71)
    q, k, v = (randn(rng, (n, 1, 64), "bf16") for _ in range(3))
    v[5, 0, 7], v[n - 20, 0, 7] = INF, -INF
    o = nan_like(q.shape, q.dtype)
    gdr.gdr_attn_prefill(q, k, v, o, ints([0, n]))
    col = o[:, 0, 7]
    assert torch.all(torch.isfinite(col[:5])) and takes(col[5:n - 20], INF) and takes(col[n - 20:], NAN)
    no_error()


@pytest.mark.parametrize("n", [19, 203, 3000])  # in one worker's tile, and split over workers and joined
@pytest.mark.parametrize("heads", [4, 1])  # 64 rows and 16: either kernel
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("bad", [INF, -INF, NAN])
def test_decode_rows_take_the_infinity_of_a_value_they_see(d, bad, heads, n):
    torch = gu.require_gpu()
    rng = np.random.default_rng(72)
    n_tok = 16
    c = Paged(rng, [n], 32, 1, d, "bf16")
    q = randn(rng, (n_tok, heads, d), "bf16")
    hit = torch.zeros(d, dtype=torch.bool, device="cuda")
    hit[1::3] = True
    for p in (0, n - 16, n - 11, n - 1):
        at = (int(c.table_np[0, p // 32]), p % 32)
        kept = c.v[at].clone()
        c.v[at[0], at[1], :, 1::3] = bad
        o, _ = run_decode(c, q, n_tok)
        j = max(0, p - (n - n_tok))
        assert takes(o[j:][..., hit], bad), p
        assert torch.all(torch.isfinite(o[j:][..., ~hit])) and torch.all(torch.isfinite(o[:j])), p
        c.v[at] = kept
    no_error()


# --- scores of minus infinity -------------------------------------------------------------------------------

def hidden_by_keys(rng, n, m, hq, d, dtype, scale):
    """q, k, v of one sequence whose first m tokens have a score of minus infinity for every query."""
    q, k, v = randn(rng, (n, hq, d), dtype), randn(rng, (n, 1, d), dtype), randn(rng, (n, 1, d), dtype)
    q[..., 0] = 1.0
    k[:m, :, 0] = -INF if scale > 0 else INF
    return q, k, v


HIDDEN = [
    # d, h_q, lens, of which so many first tokens
    (64, 2, [90, 60], [40, 33]), (256, 4, [64], [32]),  # the short kernel
    (64, 1, [300], [128]), (128, 2, [400], [130]), (128, 4, [700, 300], [257, 128]), (256, 4, [600], [300]),
    (256, 1, [390], [389]), (64, 5, [520], [500]), (128, 1, [1000], [640]),
]


@pytest.mark.parametrize("dtype", ("bf16", "f16"))
@pytest.mark.parametrize("scale", [0.1, -0.1])
@pytest.mark.parametrize("d,hq,lens,first", HIDDEN)
def test_prefill_scores_of_minus_infinity_weigh_nothing(d, hq, lens, first, scale, dtype):
    """What a row gives is the softmax of its other tokens: the definition's weights of exp(-infinity) = 0."""
    torch = gu.require_gpu()
    rng = np.random.default_rng(73 + d)
    parts = [hidden_by_keys(rng, n, m, hq, d, dtype, scale) for n, m in zip(lens, first)]
    q, k, v = (torch.cat([p[i] for p in parts]) for i in range(3))
    o, lse = nan_like(q.shape, q.dtype), nan_like(q.shape[:2], torch.float32)
    gdr.gdr_attn_prefill(q, k, v, o, ints(np.concatenate([[0], np.cumsum(lens)])), scale=scale, lse=lse)
    torch.cuda.synchronize()
    no_error()
    t = 0
    for n, m in zip(lens, first):
        r = slice(t + m, t + n)
        wo, wl, bo, bl = ar.prefill(f64(q[r]), f64(k[r]), f64(v[r]), scale, [n - m], dtype)
        close(o[r], wo, bo, "o")
        close(lse[r], wl, bl, "lse")
        t += n


@pytest.mark.parametrize("dtype", ("bf16", "f16"))
@pytest.mark.parametrize("d,hq,lens,first", HIDDEN)
def test_prefill_rows_without_a_finite_score_are_zero(d, hq, lens, first, dtype):
    torch = gu.require_gpu()
    rng = np.random.default_rng(74 + d)
    parts = [hidden_by_keys(rng, n, m, hq, d, dtype, 0.1) for n, m in zip(lens, first)]
    q, k, v = (torch.cat([p[i] for p in parts]) for i in range(3))
    o, lse = nan_like(q.shape, q.dtype), nan_like(q.shape[:2], torch.float32)
    gdr.gdr_attn_prefill(q, k, v, o, ints(np.concatenate([[0], np.cumsum(lens)])), scale=0.1, lse=lse)
    t = 0
    for n, m in zip(lens, first):
        assert torch.all(o[t:t + m] == 0) and takes(lse[t:t + m], -INF)
        t += n
    no_error()


HIDDEN_CACHE = [
    # d, h_q, n_tok, lens, of which so many first tokens
    (64, 4, 1, [300], [120]), (256, 4, 1, [4000], [3990]), (128, 8, 2, [40, 200, 16], [20, 190, 7]),
    (256, 4, 16, [300], [120]), (128, 40, 1, [2000, 64], [1990, 10]), (64, 8, 12, [40, 200, 16], [20, 180, 3]),
    (64, 2, 1, [9] * 700, [4] * 700), (64, 20, 1, [70] * 300, [64] * 300),  # sequences that one worker sees whole
]


@pytest.mark.parametrize("dtype", ("bf16", "f16"))
@pytest.mark.parametrize("d,hq,n_tok,lens,first", HIDDEN_CACHE)
def test_decode_scores_of_minus_infinity_weigh_nothing(d, hq, n_tok, lens, first, dtype):
    torch = gu.require_gpu()
    rng = np.random.default_rng(75 + d)
    c = Paged(rng, lens, 16, 1, d, dtype)
    q = randn(rng, (len(lens) * n_tok, hq, d), dtype)
    q[..., 0] = 1.0
    for s, m in enumerate(first):
        p = np.arange(m)
        c.k[c.table_np[s, p // 16], p % 16, :, 0] = -INF
    o, lse = run_decode(c, q, n_tok)
    torch.cuda.synchronize()
    no_error()
    k64, v64, q64 = f64(c.k), f64(c.v), f64(q)
    for s in list(range(len(lens)))[:6]:
        n, m, r = lens[s], first[s], slice(s * n_tok, (s + 1) * n_tok)
        k, v = ar.gather(k64, c.table_np[s], n)[m:], ar.gather(v64, c.table_np[s], n)[m:]
        for h in range(hq):
            wo, wl, bo, bl = ar.attend(q64[r, h], k[:, 0], v[:, 0], d ** -0.5,
                                       n - n_tok - m + np.arange(1, n_tok + 1), dtype)
            close(o[r, h], wo, bo, "o")
            close(lse[r, h], wl, bl, "lse")


@pytest.mark.parametrize("d,hq,n_tok,lens", [
    (64, 4, 1, [300]), (256, 4, 1, [4000, 1]), (128, 8, 2, [40, 200, 16]), (256, 4, 16, [300, 7]),
    (128, 40, 1, [2000, 64]), (64, 2, 1, [9] * 700), (64, 20, 1, [70] * 300)])
def test_decode_rows_without_a_finite_score_are_zero(d, hq, n_tok, lens):
    torch = gu.require_gpu()
    rng = np.random.default_rng(76 + d)
    c = Paged(rng, lens, 16, 1, d, "bf16")
    q = randn(rng, (len(lens) * n_tok, hq, d), "bf16")
    q[..., 0] = 1.0
    c.k[..., 0] = -INF
    o, lse = run_decode(c, q, n_tok)
    assert torch.all(o == 0) and takes(lse, -INF)
    no_error()


# --- scales ---------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("hq", [2, 40])  # 2 rows and 40: either kernel
@pytest.mark.parametrize("scale", [0.0, -0.1, 1.0])
def test_decode_scales(scale, hq):
    gu.require_gpu()
    rng = np.random.default_rng(77)
    c = Paged(rng, [300, 17, 1], 16, 1, 128, "bf16", stale=NAN)
    check_decode(c, randn(rng, (3, hq, 128), "bf16"), 1, "bf16", scale=scale)
    check_decode(c, randn(rng, (12, hq, 128), "bf16"), 4, "bf16", scale=scale)


@pytest.mark.parametrize("power,scale", [(60, 0.0), (55, 2.0 ** -110), (55, -2.0 ** -110), (60, 2.0 ** -135)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_scales_near_zero_and_large_products(d, power, scale):
    """Products near 2^115 with scales that bring them to a few units, or to nothing; fp32 holds both."""
    gu.require_gpu()
    rng = np.random.default_rng(78)
    size = 2.0 ** power
    q, k = randn(rng, (400, 2, d), "bf16", size), randn(rng, (400, 1, d), "bf16", size)
    v = randn(rng, (400, 1, d), "bf16")
    check_prefill(q, k, v, [60, 340], "bf16", scale=scale)
    c = Paged(rng, [300, 17], 16, 1, d, "bf16")
    c.k *= size
    check_decode(c, randn(rng, (4, 4, d), "bf16", size), 2, "bf16", scale=scale)
    check_decode(c, randn(rng, (2, 40, d), "bf16", size), 1, "bf16", scale=scale)


# --- what the device checks itself --------------------------------------------------------------------------

@pytest.mark.parametrize("n_tok,h_q", [(1, 2), (16, 4), (1, 40)])  # 2 rows; 64 and 40, which are the wide kernel's
def test_decode_bad_lengths_and_pages(n_tok, h_q):
    """A bad length counts as none, a bad page is read as zeros; the other sequence is not touched by either."""
    torch = gu.require_gpu()
    rng = np.random.default_rng(80)
    c = Paged(rng, [200, 90], 16, 1, 64, "bf16")
    q = randn(rng, (2 * n_tok, h_q, 64), "bf16")
    good, _ = run_decode(c, q, n_tok)
    no_error()
    most = c.table.shape[1] * 16
    for bad in (-1, most + 1, 2 ** 31 - 1):
        o, lse = nan_like(q.shape, q.dtype), nan_like(q.shape[:2], torch.float32)
        gdr.gdr_attn_decode(q, c.k, c.v, c.table, ints([bad, 90]), o, n_tok, lse=lse)
        assert gdr.gdr_device_error(device="cuda") == gdr.GDR_ERR_INVALID_ARG
        assert torch.all(o[:n_tok] == 0) and takes(lse[:n_tok], -INF)
        # (cut elsewhere on the line, the second sequence's sums are in another order)
        wo, wl, bo, bl = ar.decode(f64(q[n_tok:]), f64(c.k), f64(c.v), c.table_np[1:], [90], n_tok, 0.125, "bf16")
        close(o[n_tok:], wo, bo, "o")
        close(lse[n_tok:], wl, bl, "lse")
    for page in (-7, c.k.shape[0], 2 ** 31 - 1):
        for slot in (0, 12):  # the first page, and the one that holds the last tokens
            table = c.table.clone()
            table[0, slot] = page
            o = nan_like(q.shape, q.dtype)
            gdr.gdr_attn_decode(q, c.k, c.v, table, c.kv_lens, o, n_tok)
            assert gdr.gdr_device_error(device="cuda") == gdr.GDR_ERR_INVALID_ARG
            assert torch.equal(o[n_tok:], good[n_tok:])
            # zeros in the place of the page's keys and values
            k64, v64 = ar.gather(f64(c.k), c.table_np[0], 200), ar.gather(f64(c.v), c.table_np[0], 200)
            k64[16 * slot:16 * slot + 16] = 0.0
            v64[16 * slot:16 * slot + 16] = 0.0
            for h in range(h_q):
                wo, _, bo, _ = ar.attend(f64(q[:n_tok, h]), k64[:, 0], v64[:, 0], 0.125,
                                         200 - n_tok + np.arange(1, n_tok + 1), "bf16")
                close(o[:n_tok, h], wo, bo, "o")


STARTS = [
    # total, starts; a sequence is valid when 0 <= start <= end <= total
    (9, [0, -2, 9]), (9, [0, 20, 9]), (9, [3, 5, 9]), (9, [0, 4, 12]),
    (900, [400, 300, 900]), (900, [0, 400, 1200]), (900, [-1, 400, 900]), (900, [0, 300, -5, 600, 900]),
    (900, [300, 900, 2 ** 31 - 1]), (900, [0, 20, 1000, 20, 900]), (900, [-2 ** 31, 2 ** 31 - 1]),
]


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("total,starts", STARTS)
def test_prefill_bad_starts_skip_their_sequences(total, starts, d):
    """Both prefill kernels: sequences with a start or end out of range or before its start write nothing and are
    recorded, the others give what they give alone."""
    torch = gu.require_gpu()
    rng = np.random.default_rng(81)
    q, k, v = randn(rng, (total, 2, d), "bf16"), randn(rng, (total, 1, d), "bf16"), randn(rng, (total, 1, d), "bf16")
    o = nan_like(q.shape, q.dtype)
    gdr.gdr_attn_prefill(q, k, v, o, ints(starts))
    valid = [0 <= a <= b <= total for a, b in zip(starts, starts[1:])]
    want_code = gdr.GDR_OK if all(valid) else gdr.GDR_ERR_INVALID_ARG
    assert gdr.gdr_device_error(device="cuda") == want_code
    rest = torch.ones(total, dtype=torch.bool, device="cuda")
    for a, b, ok in zip(starts, starts[1:], valid):
        if ok and b > a:
            rest[a:b] = False
            wo, _, bo, _ = ar.prefill(f64(q[a:b]), f64(k[a:b]), f64(v[a:b]), d ** -0.5, [b - a], "bf16")
            close(o[a:b], wo, bo, "o")
    assert takes(o[rest], NAN)


@pytest.mark.parametrize("total,starts,taken", [
    (9, [0, -2, 9], []), (9, [0, 20, 9], []), (9, [3, 5, 9], [0, 1]), (9, [0, 4, 12], [0]), (60, [0, 30, 99], [0]),
])
def test_append_bad_starts_leave_out_their_tokens(total, starts, taken):
    """Tokens of no valid sequence are recorded and written nowhere; valid sequences are appended whole."""
    torch = gu.require_gpu()
    rng = np.random.default_rng(82)
    n = len(starts) - 1
    lens = [40] * n
    c = Paged(rng, lens, 16, 1, 64, "bf16")
    k, v = randn(rng, (total, 1, 64), "bf16"), randn(rng, (total, 1, 64), "bf16")
    want_k, want_v = c.k.clone(), c.v.clone()
    ko = nan_like(k.shape, k.dtype)
    want = ko.clone()
    gdr.gdr_attn_append(None, k, v, None, ko, c.k, c.v, c.table, c.kv_lens, None, ints(starts))
    assert gdr.gdr_device_error(device="cuda") == gdr.GDR_ERR_INVALID_ARG  # each case leaves some token out
    for s in taken:
        a, b = starts[s], starts[s + 1]
        pos = np.arange(40 - (b - a), 40)
        want_k[c.table_np[s, pos // 16], pos % 16], want_v[c.table_np[s, pos // 16], pos % 16] = k[a:b], v[a:b]
        want[a:b] = k[a:b]
    assert torch.equal(c.k, want_k) and torch.equal(c.v, want_v)
    assert torch.equal(ko.view(torch.int16), want.view(torch.int16))


# --- empty batches --------------------------------------------------------------------------------------------

def test_empty_batches_are_no_ops():
    torch = gu.require_gpu()
    bf, cuda = torch.bfloat16, torch.device("cuda")
    q, k = torch.empty(0, 4, 64, dtype=bf, device=cuda), torch.empty(0, 2, 64, dtype=bf, device=cuda)
    kc, vc = (torch.ones(5, 16, 2, 64, dtype=bf, device=cuda) for _ in range(2))
    none, table = ints([]), torch.empty(0, 3, dtype=torch.int32, device=cuda)
    inv = torch.ones(8, device=cuda)
    gdr.gdr_attn_append(q, k, k, q, k, kc, vc, table, none, inv)
    gdr.gdr_attn_append(q, k, k, q, k, kc, vc, table, none, inv, ints([0]))
    gdr.gdr_attn_append(None, k, k, None, None, kc, vc, torch.zeros(2, 3, dtype=torch.int32, device=cuda),
                        ints([3, 4]), inv, ints([0, 0, 0]))  # two sequences, nothing new
    gdr.gdr_attn_prefill(q, k, k, q, ints([0]))
    gdr.gdr_attn_prefill(q, k, k, q, ints([0, 0, 0]))
    gdr.gdr_attn_decode(q, kc, vc, table, none, q)
    gdr.gdr_attn_decode(q, kc, vc, table, none, q, 4, lse=torch.empty(0, 4, device=cuda))
    assert torch.all(kc == 1) and torch.all(vc == 1)
    no_error()


# --- the weights' bits ------------------------------------------------------------------------------------------

@pytest.mark.parametrize("lens", [[40], [3000], [33] * 400])  # cut and joined in a block or by the second launch; whole
@pytest.mark.parametrize("d,n_tok,h_q", [(64, 1, 4), (128, 3, 2), (256, 1, 16), (256, 4, 4)])
def test_decode_weights_hold_16_bits(d, n_tok, h_q, lens):
    """bf16, up to 16 rows.  Half of the tokens weigh 1 and have the value 1, the other half weigh e^-x, between
    two bf16 values, and have -1: what is left shows the weights' rounding, which is the same in all of them.  A
    weight is its first 8 bits and the rest (up to 2^-7 of it) rounded to 8 bits: off by 2^-15.  The other terms are
    those of tests/attn_ref.py, with sum_j p_j |v_j| = 1."""
    torch = gu.require_gpu()
    rng = np.random.default_rng(90)
    c = Paged(rng, lens, 16, 1, d, "bf16")
    q = torch.zeros(len(lens) * n_tok, h_q, d, dtype=torch.bfloat16, device="cuda")
    q[..., 5] = 1.0
    x = torch.tensor([0.0035, 0.0011, 0.0059, 0.0095] * h_q, device="cuda").to(torch.bfloat16)[:h_q]
    c.k.zero_()
    c.v.fill_(1.0)
    for s, n in enumerate(lens):
        p = np.arange(1, n, 2)
        c.k[c.table_np[s, p // 16], p % 16, :, 5] = -1.0
        c.v[c.table_np[s, p // 16], p % 16] = -1.0
    q[..., 5] = x
    o, lse = run_decode(c, q, n_tok, scale=1.0)
    no_error()
    o, w = f64(o), np.exp(-f64(x))
    for s, n in enumerate(lens):
        for j in range(n_tok):
            seen = n - n_tok + j + 1
            one, other = (seen + 1) // 2, seen // 2
            want = (one - other * w) / (one + other * w)  # per head
            bound = 2.0 ** -8 * np.abs(want) + (1 + 2.0 ** -8) * (2.0 ** -15 + 2 * d * 2.0 ** -24 * f64(x) + 2.0 ** -16)
            err = np.abs(o[s * n_tok + j] - want[:, None]) - bound[:, None]
            assert np.all(err <= 0), (s, j, err.max())
