"""The attention operators beside the gated delta rule, as cases to measure and compare.

A hybrid model's softmax-attention layers need three operators next to the rule: the position rotation of
queries and keys with the append of keys and values to a paged cache, causal attention over whole packed
prompts, and attention of one or a few new tokens over the paged cache.  `run` computes a case either in plain
torch operations in 32 bits (`own = False`) or through this package's entry points (`own = True`).

Definitions, for query head h, key/value head h // (h_q / h_kv), head size d:

  append   position p = kv_len - n + j of the j-th of a sequence's n new tokens; the first 2 R values of each
           query and key head are R pairs, pair i turned by the angle p * inv_freq[i]; keys (turned) and values
           go to slot p % page_size of page page_table[s, p // page_size]
  prefill  o_i = sum_{j <= i} softmax_j(scale q_i . k_j) v_j within each packed sequence
  decode   the same for a sequence's last n tokens over the kv_len tokens of its pages; no visible token: zeros

and lse is the natural logarithm of the softmax's denominator (minus infinity where no token is visible).
"""

import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def _case(name, op, heads, d, dtype, lens, **more):
    c = {"name": name, "op": op, "h_q": heads[0], "h_kv": heads[1], "d": d, "dtype": dtype, "lens": lens,
         "n_tok": 0, "page": 64, "by_head": False, "rot": 0, "interleaved": False, "base": 1e7}
    c.update(more)
    return c


def _text(lens):
    return ",".join(str(n) for n in lens)


def _ragged(count, lo, hi, seed):
    """`count` lengths spread over [lo, hi] evenly in their logarithm."""
    rng = random.Random(seed)
    return [min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))) for _ in range(count)]


def listed():
    return [
        # one sequence's next token: a single user's decode step, where latency counts
        _case("append_one", "append", (16, 4), 256, "bf16", _text([1500]), n_tok=1, rot=64),
        # one token of each of 64 sequences: a batch's decode step
        _case("append_decode_64", "append", (16, 4), 256, "bf16", _text(_ragged(64, 512, 8192, 1)), n_tok=1, rot=64),
        # eight whole prompts of 512 to 8192 tokens, head-major pages, the whole head turned, other pairing
        _case("append_prompts", "append", (32, 8), 128, "f16", _text(_ragged(8, 512, 8192, 2)), rot=128, page=48,
              by_head=True, interleaved=True, base=1e6),
        # a user's prompt of 1024 tokens, and the longest prompt of 16384
        _case("prefill_1024", "prefill", (16, 4), 256, "bf16", _text([1024])),
        _case("prefill_16384", "prefill", (16, 4), 256, "bf16", _text([16384])),
        # a packed batch of prompts of 512 to 8192 tokens
        _case("prefill_packed", "prefill", (32, 8), 128, "f16", _text(_ragged(8, 512, 8192, 2))),
        # many short chat turns, odd lengths, every query head with its own key/value head
        _case("prefill_short", "prefill", (16, 16), 128, "bf16", _text(_ragged(24, 1, 300, 3))),
        # one short sequence's next token: the least that a decode step does
        _case("decode_one_short", "decode", (16, 4), 256, "bf16", _text([301]), n_tok=1),
        # a batch of 64 sequences of 512 to 8192 tokens
        _case("decode_64", "decode", (16, 4), 256, "bf16", _text(_ragged(64, 512, 8192, 1)), n_tok=1),
        # one sequence of 131072 tokens: the cache's length has to be split
        _case("decode_one_long", "decode", (16, 4), 256, "bf16", _text([131072]), n_tok=1, page=16),
        # smaller heads, head-major pages of an odd size, a batch of sequences from one token to many
        _case("decode_ragged", "decode", (32, 8), 128, "f16", _text(_ragged(96, 1, 16384, 4)), n_tok=1, page=48,
              by_head=True),
        # the 16 draft tokens of a speculative block for eight sequences
        _case("decode_draft_16", "decode", (16, 4), 256, "bf16", _text(_ragged(8, 512, 8192, 5)), n_tok=16),
    ]


def draw(rng):
    op = rng.choice(["append", "prefill", "decode"])
    d = rng.choice([64, 128, 256])
    h_kv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 6, 8])
    while h_kv * group * d > 4096:
        h_kv, group = (h_kv, group - 1) if group > 1 else (h_kv // 2, group)
    dtype = rng.choice(["bf16", "f16"])
    page = rng.choice([16, 32, 48, 64, 100, 128, 256])
    by_head = rng.random() < 0.5
    count = round(math.exp(rng.uniform(0, math.log(64))))
    more = {"page": page, "by_head": by_head}
    if op == "prefill":
        total = round(math.exp(rng.uniform(0, math.log(16384))))
        cuts = sorted(rng.randint(0, total) for _ in range(min(count, 16) - 1))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    elif op == "decode":
        n_tok = rng.choice([1, 1, 1, 2, 5, 8, 16])
        most = min(131072, (1 << 19) // count // max(1, h_kv * d // 1024))
        lens = [max(0, n - 1) for n in _ragged(count, 1, most, rng.random())]
        more["n_tok"] = n_tok
    else:
        more["n_tok"] = rng.choice([0, 1, 1, 4, 16])
        if more["n_tok"]:
            lens = [n + more["n_tok"] - 1 for n in _ragged(count, 1, 8192, rng.random())]
        else:
            lens = _ragged(min(count, 16), 1, 2048, rng.random())
        more["rot"] = rng.choice([d, d // 2, d // 4, 24])
        more["interleaved"] = rng.random() < 0.5
        more["base"] = rng.choice([1e4, 1e6, 1e7])
    c = _case("", op, (h_kv * group, h_kv), d, dtype, _text(lens), **more)
    del c["name"]
    return c


def _lens(case):
    return [int(n) for n in case["lens"].split(",")]


def _new(case):
    """New tokens of each sequence."""
    lens = _lens(case)
    return [case["n_tok"]] * len(lens) if case["n_tok"] else lens


def work(case):
    h_q, h_kv, d = case["h_q"], case["h_kv"], case["d"]
    lens, new = _lens(case), _new(case)
    t = sum(new)
    if case["op"] == "append":
        # q, k and v in; q, k (packed) and the two cache rows out
        return {"bytes": 2 * t * d * (2 * h_q + 4 * h_kv), "flops": 3 * t * case["rot"] * (h_q + h_kv)}
    if case["op"] == "prefill":
        pairs = sum(n * (n + 1) // 2 for n in lens)
        return {"bytes": 2 * t * d * (2 * h_q + 2 * h_kv) + 4 * t * h_q, "flops": 4 * pairs * h_q * d}
    pairs = sum(max(0, n - case["n_tok"] + j + 1) for n in lens for j in range(case["n_tok"]))
    pages = sum(-(-n // case["page"]) for n in lens)
    return {"bytes": 4 * sum(lens) * h_kv * d + 4 * t * h_q * d + 4 * t * h_q + 4 * pages,
            "flops": 4 * pairs * h_q * d}


def prepare(case, seed):
    dev, dtype = torch.device("cuda"), _DTYPES[case["dtype"]]
    h_q, h_kv, d, page = case["h_q"], case["h_kv"], case["d"], case["page"]
    lens, new = _lens(case), _new(case)
    t, n = sum(new), len(lens)
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)

    # q, k and v as a layer's fused projection leaves them: one row of h_q + 2 h_kv heads a token
    qkv = normal(t, h_q + 2 * h_kv, d)
    s = {"case": dict(case), "lens": lens, "new": new, "q": qkv[:, :h_q], "k": qkv[:, h_q:h_q + h_kv],
         "v": qkv[:, h_q + h_kv:], "scale": 1.0 / math.sqrt(d)}
    cu = [0]
    for m in new:
        cu.append(cu[-1] + m)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    s["lse"] = torch.empty(t, h_q, dtype=torch.float32, device=dev)
    if case["op"] == "prefill":
        # q and k come from the rotation, in buffers of their own; normed heads times a learned gain
        s["q"] = (2.0 * s["q"].float()).to(dtype).contiguous()
        s["k"] = s["k"].contiguous()
        s["o"] = torch.empty(t, h_q, d, dtype=dtype, device=dev)
        return s
    need = [-(-m // page) for m in lens]
    width = max(need + [1])
    spare = 3
    order = torch.randperm(sum(need) + spare, generator=gen, device=dev).to(torch.int32)
    table = torch.full((n, width), -1, dtype=torch.int32, device=dev)
    rows = torch.repeat_interleave(torch.arange(n), torch.tensor(need)).to(dev)
    cols = torch.cat([torch.arange(m) for m in need] + [torch.arange(0)]).to(dev)
    table[rows, cols] = order[:sum(need)]
    s["table"], s["kv_lens"] = table, torch.tensor(lens, dtype=torch.int32, device=dev)
    shape = (sum(need) + spare, h_kv, page, d) if case["by_head"] else (sum(need) + spare, page, h_kv, d)
    for name in ("k_cache", "v_cache"):
        c = normal(*shape)
        s[name] = c.transpose(1, 2) if case["by_head"] else c  # [pages, page, h_kv, d] either way
    if case["op"] == "append":
        r = case["rot"] // 2
        s["inv_freq"] = (case["base"] ** (-torch.arange(r, dtype=torch.float64) / r)).float().to(dev)
        s["q_out"] = torch.empty(t, h_q, d, dtype=dtype, device=dev)
        s["k_out"] = torch.empty(t, h_kv, d, dtype=dtype, device=dev)
        return s
    s["q"] = (2.0 * s["q"].float()).to(dtype).contiguous()
    s["o"] = torch.empty(t, h_q, d, dtype=dtype, device=dev)
    s["workspace"] = None
    if own:
        import gated_deltanet_scan_gb300 as gdr

        need = gdr.gdr_attn_decode_workspace_bytes(s["q"], s["k_cache"], n, case["n_tok"])
        s["workspace"] = torch.empty(max(16, need), dtype=torch.uint8, device=dev)
    return s


def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "prefill": _own_prefill, "decode": _own_decode}[op](state)
    return {"append": _plain_append, "prefill": _plain_prefill, "decode": _plain_decode}[op](state)


# --- through the package ------------------------------------------------------------------------------------

def _own_append(s):
    import gated_deltanet_scan_gb300 as gdr

    gdr.gdr_attn_append(s["q"], s["k"], s["v"], s["q_out"], s["k_out"], s["k_cache"], s["v_cache"], s["table"],
                        s["kv_lens"], s["inv_freq"], s["cu"], interleaved=s["case"]["interleaved"])
    return s["q_out"], s["k_out"], s["k_cache"], s["v_cache"]


def _own_prefill(s):
    import gated_deltanet_scan_gb300 as gdr

    gdr.gdr_attn_prefill(s["q"], s["k"], s["v"], s["o"], s["cu"], scale=s["scale"], lse=s["lse"])
    return s["o"], s["lse"]


def _own_decode(s):
    import gated_deltanet_scan_gb300 as gdr

    gdr.gdr_attn_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_lens"], s["o"], s["case"]["n_tok"],
                        scale=s["scale"], lse=s["lse"], workspace=s["workspace"])
    return s["o"], s["lse"]


# --- plain forms --------------------------------------------------------------------------------------------

def _plain_append(s):
    case, dev, t = s["case"], s["q"].device, s["q"].shape[0]
    new = s["cu"][1:] - s["cu"][:-1]
    seq = torch.repeat_interleave(torch.arange(len(s["new"]), device=dev), new, output_size=t)
    pos = torch.arange(t, device=dev) - s["cu"][seq] + (s["kv_lens"][seq] - new[seq])
    angle = pos.double()[:, None, None] * s["inv_freq"].double()  # 64 bits: far positions turn many times
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    r = case["rot"] // 2

    def turned(x):
        x = x.float()
        head, tail = x[..., :2 * r], x[..., 2 * r:]
        a, b = (head[..., 0::2], head[..., 1::2]) if case["interleaved"] else (head[..., :r], head[..., r:])
        ta, tb = a * cos - b * sin, a * sin + b * cos
        head = torch.stack((ta, tb), -1).flatten(-2) if case["interleaved"] else torch.cat((ta, tb), -1)
        return torch.cat((head, tail), -1).to(s["q"].dtype)

    s["q_out"].copy_(turned(s["q"]))
    s["k_out"].copy_(turned(s["k"]))
    page = s["table"][seq, pos // case["page"]].long()
    slot = pos % case["page"]
    s["k_cache"][page, slot] = s["k_out"]
    s["v_cache"][page, slot] = s["v"]
    return s["q_out"], s["k_out"], s["k_cache"], s["v_cache"]


def _attend(q, k, v, scale, first):
    """q [n, h_q, d] at positions first, first + 1, ... over k, v [m, h_kv, d], in q's type; o and lse."""
    n, h_q, d = q.shape
    m, h_kv, _ = k.shape
    qh = q.reshape(n, h_kv, h_q // h_kv, d).permute(1, 2, 0, 3).reshape(h_kv, -1, d)
    scores = torch.matmul(qh, k.permute(1, 2, 0)) * scale  # [h_kv, group * n, m]
    scores = scores.view(h_kv, h_q // h_kv, n, m)
    hidden = torch.arange(m, device=q.device) > torch.arange(first, first + n, device=q.device)[:, None]
    scores = scores.masked_fill_(hidden, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(h_kv, -1, m), v.permute(1, 0, 2)).view(h_kv, h_q // h_kv, n, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (total.log() + top).squeeze(-1)
    return o.permute(2, 0, 1, 3).reshape(n, h_q, d), lse.permute(2, 0, 1).reshape(n, h_q)


_ROWS = 1024  # queries at a time: bounds the scores held at once


def _plain_prefill(s):
    t0 = 0
    for n in s["new"]:
        k, v = s["k"][t0:t0 + n].float(), s["v"][t0:t0 + n].float()
        for i in range(0, n, _ROWS):
            j = min(n, i + _ROWS)
            o, lse = _attend(s["q"][t0 + i:t0 + j].float(), k[:j], v[:j], s["scale"], i)
            s["o"][t0 + i:t0 + j] = o.to(s["o"].dtype)
            s["lse"][t0 + i:t0 + j] = lse
        t0 += n
    return s["o"], s["lse"]


def _gathered(s, b, name):
    n, page = s["lens"][b], s["case"]["page"]
    pages = s["table"][b, :-(-n // page)].long()
    c = s[name][pages]
    return c.reshape(-1, *c.shape[2:])[:n]


def _plain_decode(s):
    n_tok = s["case"]["n_tok"]
    for b, n in enumerate(s["lens"]):
        r0, r1 = b * n_tok, (b + 1) * n_tok
        if n == 0:
            s["o"][r0:r1] = 0
            s["lse"][r0:r1] = -math.inf
            continue
        k, v = _gathered(s, b, "k_cache").float(), _gathered(s, b, "v_cache").float()
        o, lse = _attend(s["q"][r0:r1].float(), k, v, s["scale"], n - n_tok)
        s["o"][r0:r1] = o.to(s["o"].dtype)
        s["lse"][r0:r1] = lse
    return s["o"], s["lse"]


# --- in 64 bits, from the definitions -----------------------------------------------------------------------

def exact(case, seed):
    if case["op"] != "append" and work(case)["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    return {"append": _exact_append, "prefill": _exact_prefill, "decode": _exact_decode}[case["op"]](s)


def _exact_append(s):
    case = s["case"]
    r, pairs = case["rot"] // 2, case["interleaved"]
    q, k = s["q"].double().clone(), s["k"].double().clone()
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    t = 0
    for b, n in enumerate(s["new"]):
        pos = torch.arange(s["lens"][b] - n, s["lens"][b], device=q.device)
        z = torch.polar(torch.ones(n, 1, r, dtype=torch.float64, device=q.device),
                        pos.double().view(n, 1, 1) * s["inv_freq"].double())
        for x in (q[t:t + n], k[t:t + n]):
            one = slice(0, 2 * r, 2) if pairs else slice(0, r)
            two = slice(1, 2 * r, 2) if pairs else slice(r, 2 * r)
            w = torch.complex(x[..., one], x[..., two]) * z
            x[..., one], x[..., two] = w.real, w.imag
        flat = s["table"][b].long()[pos // case["page"]]
        kc[flat, pos % case["page"]] = k[t:t + n]
        vc[flat, pos % case["page"]] = s["v"][t:t + n].double()
        t += n
    return q, k, kc, vc


def _exact_rows(q, k, v, scale, first, o, lse):
    """Row block by row block and head by head: the softmax from its definition, with torch.logsumexp."""
    group = q.shape[1] // k.shape[1]
    for h in range(q.shape[1]):
        kh, vh = k[:, h // group].double(), v[:, h // group].double()
        for i in range(0, q.shape[0], 2048):
            rows = q[i:i + 2048, h].double()
            last = first + i + torch.arange(rows.shape[0], device=q.device)
            seen = max(0, min(int(first) + i + rows.shape[0], kh.shape[0]))
            x = scale * (rows @ kh[:seen].T)
            x[torch.arange(seen, device=q.device)[None, :] > last[:, None]] = -math.inf
            z = torch.logsumexp(x, -1)
            lse[i:i + 2048, h] = z
            weights = torch.exp(x - z[:, None])
            weights[z == -math.inf] = 0.0
            o[i:i + 2048, h] = weights @ vh[:seen]


def _exact_prefill(s):
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=s["q"].device)
    t = 0
    for n in s["new"]:
        _exact_rows(s["q"][t:t + n], s["k"][t:t + n], s["v"][t:t + n], s["scale"], 0, o[t:t + n], lse[t:t + n])
        t += n
    return o, lse


def _exact_decode(s):
    n_tok, page = s["case"]["n_tok"], s["case"]["page"]
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=s["q"].device)
    for b, n in enumerate(s["lens"]):
        pos = torch.arange(n, device=o.device)
        where = s["table"][b].long()[pos // page], pos % page
        rows = slice(b * n_tok, (b + 1) * n_tok)
        if n:
            _exact_rows(s["q"][rows], s["k_cache"][where], s["v_cache"][where], s["scale"], n - n_tok, o[rows],
                        lse[rows])
    return o, lse
