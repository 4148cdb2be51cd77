"""Operators for trees of drafted tokens in a hybrid model, as cases to measure and compare.

A drafter that keeps several continuations gives each sequence a tree of up to 64 tokens.  Node j's parent is
`parents[s, j]`: -1 for a child of the sequence's last committed token, an earlier node, or -2 where the row holds
no node (trees of a batch are padded to the same number of rows).  A_j is the set of j and its ancestors, and base
the number of tokens before the tree (kv_len - n_tok: the cache's last n_tok slots are the nodes').  Verifying a
tree takes five operators:

  append  queries and keys turned by the angle (base + |A_j| - 1) inv_freq[i], keys and values put into slot
          base + j of the paged cache; rows of no node are left as they are
  attend  o_j = sum_p softmax_p(scale q_j . k_p) v_p over p < base and the slots of A_j, and the logarithm of the
          softmax's denominator; rows of no node: zeros and minus infinity
  rule    the gated delta rule along every path from one state S_0, which stays as it is:
          S_j = e^{g_j} (I - beta_j k_j k_j^T) S_parent + beta_j k_j v_j^T,  o_j = S_j^T q_j, and the corrections
          u_j = beta_j (v_j - e^{g_j} S_parent^T k_j); rows of no node: zeros
  settle  (rule) S_0 becomes S_a of the last accepted node a, from the corrections
  compact (attention) the slots of A_a move to base, base + 1, ... in every layer's cache, and the new lengths

`run` computes a case either in plain torch operations in 32 bits (`own = False`) or through this package's entry
points (`own = True`).
"""

import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_MOST_FLOPS = 64 << 30  # of a drawn attention case


def _text(lens):
    return ",".join(str(n) for n in lens)


def _ragged(count, lo, hi, seed):
    """`count` lengths spread over [lo, hi] evenly in their logarithm."""
    rng = random.Random(seed)
    return [min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))) for _ in range(count)]


def _attn(name, op, heads, d, dtype, lens, n_tok, tree, **more):
    c = {"name": name, "op": op, "h_q": heads[0], "h_kv": heads[1], "d": d, "dtype": dtype, "lens": lens,
         "n_tok": n_tok, "tree": tree, "tree_seed": 6, "page": 64, "by_head": False, "rot": 0, "interleaved": False,
         "base": 1e7, "layers": 1}
    c.update(more)
    return c


def _rule(name, op, heads, d, dtype, n_seqs, n_tok, tree, **more):
    c = {"name": name, "op": op, "h_qk": heads[0], "h_v": heads[1], "d": d, "dtype": dtype, "out": "f32",
         "n_seqs": n_seqs, "n_tok": n_tok, "tree": tree, "tree_seed": 6, "raw": True}
    c.update(more)
    return c


def listed():
    return [
        # one user's drafted tree: the least that verifying one does, where latency counts
        _attn("append_one_24", "append", (16, 4), 256, "bf16", _text([1500]), 24, "draft", rot=64),
        # trees of different sizes in a batch, head-major pages of an odd size, the whole head turned
        _attn("append_32x64", "append", (32, 8), 128, "f16", _text(_ragged(32, 300, 4096, 2)), 64, "padded", rot=128,
              page=48, by_head=True, interleaved=True, base=1e6),
        # one user's next step: few rows, one sequence's cache
        _attn("attend_one_24", "attend", (16, 4), 256, "bf16", _text([1500]), 24, "draft"),
        # a batch whose trees fill 128 rows of every key/value head
        _attn("attend_32x32", "attend", (16, 4), 256, "bf16", _text(_ragged(32, 512, 8192, 1)), 32, "draft"),
        # trees of up to 64 nodes, 256 rows of a key/value head, smaller heads, ragged trees
        _attn("attend_16x64", "attend", (32, 8), 128, "f16", _text(_ragged(16, 512, 16384, 4)), 64, "padded", page=48,
              by_head=True),
        # the rule's layer for one user's tree
        _rule("rule_one_24", "rule", (16, 32), 128, "bf16", 1, 24, "draft"),
        # eight sequences, an odd number of rows, queries and keys normalised before
        _rule("rule_8x41", "rule", (16, 32), 128, "bf16", 8, 41, "padded", raw=False),
        # the largest batch of the largest trees
        _rule("rule_64x64", "rule", (16, 32), 128, "bf16", 64, 64, "draft"),
        # the accepted path into the states: one user, and a batch
        _rule("settle_one_24", "settle", (16, 32), 128, "bf16", 1, 24, "draft"),
        _rule("settle_64x64", "settle", (16, 32), 128, "bf16", 64, 64, "padded"),
        # the accepted path in the caches of the model's eight attention layers: one user, and a batch
        _attn("compact_one_24", "compact", (16, 4), 256, "bf16", _text([1500]), 24, "draft", layers=8),
        _attn("compact_64x64", "compact", (16, 4), 256, "bf16", _text(_ragged(64, 300, 1500, 3)), 64, "padded",
              layers=8),
    ]


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "rule", "rule", "settle", "compact"])
    n_tok = rng.choice([1, 2, 3, 4, 6, 8, 11, 16, 17, 24, 31, 32, 33, 40, 48, 57, 63, 64])
    tree = rng.choice(["draft", "draft", "padded", "forest", "chain"])
    count = round(math.exp(rng.uniform(0, math.log(64))))
    more = {"tree_seed": rng.randrange(1 << 30)}
    if op in ("rule", "settle"):
        d = rng.choice([128, 128, 128, 64, 32])
        h_qk = rng.choice([1, 2, 4, 8, 16])
        h_v = h_qk * rng.choice([1, 2, 2, 4])
        if h_v > 32:
            h_v = 32
        more["raw"] = rng.random() < 0.5
        more["out"] = rng.choice(["f32", "f32", "bf16"])
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        c = _rule("", op, (h_qk, h_v), d, dtype, min(count, 16) if dtype == "f32" else count, n_tok, tree, **more)
    else:
        d = rng.choice([64, 128, 256])
        h_kv = rng.choice([1, 2, 3, 4, 8])
        group = rng.choice([1, 2, 3, 4, 5, 6, 8])
        while h_kv * group * d > 4096:
            h_kv, group = (h_kv, group - 1) if group > 1 else (h_kv // 2, group)
        more["page"] = rng.choice([16, 32, 48, 64, 100, 128, 256])
        more["by_head"] = rng.random() < 0.5
        if op == "attend":
            most = 80000 // count // max(1, -(-h_kv * d // 1024))
            most = max(1, min(most, _MOST_FLOPS // (4 * h_kv * group * d * n_tok * count)) - n_tok)
        else:
            most = 2048
        lens = [n_tok - 1 + n for n in _ragged(count, 1, most, rng.random())]
        if op == "append":
            more["rot"] = rng.choice([d, d // 2, d // 4, 24])
            more["interleaved"] = rng.random() < 0.5
            more["base"] = rng.choice([1e4, 1e6, 1e7])
        if op == "compact":
            more["layers"] = rng.choice([1, 2, 5, 8]) if h_kv * d <= 1024 else 1
        c = _attn("", op, (h_kv * group, h_kv), d, rng.choice(["bf16", "f16"]), _text(lens), n_tok, tree, **more)
    del c["name"]
    return c


def _trees(case):
    """Every sequence's parents, and its last accepted node (-1: none)."""
    rng = random.Random(case["tree_seed"])
    n_tok, kind = case["n_tok"], case["tree"]
    parents, last = [], []
    for _ in range(case["n_seqs"] if "n_seqs" in case else len(_lens(case))):
        nodes = rng.randint((n_tok + 1) // 2, n_tok) if kind == "padded" else n_tok
        one = []
        for j in range(nodes):
            if kind == "chain":
                one.append(j - 1)
            elif kind == "forest":  # several continuations of the last committed token
                one.append(rng.randrange(-1, j))
            else:  # the token just sampled, and continuations of it
                one.append(rng.randrange(j) if j else -1)
        parents.append(one + [-2] * (n_tok - nodes))
        last.append(rng.randrange(-1 if kind == "forest" else 0, nodes))
    return parents, last


def _paths(parents):
    """A_j as sorted lists (empty where there is no node)."""
    paths = []
    for j, p in enumerate(parents):
        paths.append([] if p == -2 else ([] if p < 0 else paths[p]) + [j])
    return paths


def _lens(case):
    return [int(n) for n in case["lens"].split(",")]


def work(case):
    n_tok, d = case["n_tok"], case["d"]
    parents, last = _trees(case)
    n = len(parents)
    paths = [_paths(p) for p in parents]
    nodes = sum(p != -2 for one in parents for p in one)
    pairs = sum(len(a) for one in paths for a in one)
    ids = 4 * n * n_tok
    if case["op"] in ("rule", "settle"):
        h_qk, h_v = case["h_qk"], case["h_v"]
        w = 4 if case["dtype"] == "f32" else 2
        if case["op"] == "rule":
            o = 4 if case["out"] == "f32" else 2
            return {"bytes": 4 * n * h_v * d * d + w * nodes * d * (2 * h_qk + h_v) + 8 * nodes * h_v
                    + (4 + o) * n * n_tok * h_v * d + ids,
                    "flops": 4 * nodes * h_v * d * d + pairs * 4 * d * (h_qk + h_v)}
        on = sum(len(one[a]) for one, a in zip(paths, last) if a >= 0)
        moved = sum(a >= 0 for a in last)
        return {"bytes": 8 * moved * h_v * d * d + on * (w * h_qk * d + 4 * h_v * d + 4 * h_v) + ids + 4 * n,
                "flops": 2 * on * h_v * d * d + moved * h_v * d * d}
    h_q, h_kv = case["h_q"], case["h_kv"]
    lens = _lens(case)
    if case["op"] == "append":
        return {"bytes": 2 * nodes * d * (2 * h_q + 4 * h_kv) + ids, "flops": 3 * nodes * case["rot"] * (h_q + h_kv)}
    if case["op"] == "compact":
        moved = sum(i != j for one, a in zip(paths, last) if a >= 0 for i, j in enumerate(one[a]))
        return {"bytes": 8 * case["layers"] * moved * h_kv * d + ids + 12 * n, "flops": 0}
    seen = sum((m - n_tok) * sum(p != -2 for p in one) for m, one in zip(lens, parents)) + pairs
    pages = sum(-(-m // case["page"]) for m in lens)
    t = n * n_tok
    return {"bytes": 4 * sum(lens) * h_kv * d + 2 * (t + nodes) * h_q * d + 4 * t * h_q + 4 * pages + ids,
            "flops": 4 * seen * h_q * d}


# --- what a program has in hand -----------------------------------------------------------------------------

def prepare(case, seed):
    dev, dtype = torch.device("cuda"), _DTYPES[case["dtype"]]
    gen = torch.Generator(device=dev).manual_seed(seed)
    parents, last = _trees(case)
    s = {"case": dict(case), "parents": torch.tensor(parents, dtype=torch.int32, device=dev),
         "last": torch.tensor(last, dtype=torch.int32, device=dev), "workspace": None}

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32)

    n, n_tok, d = len(parents), case["n_tok"], case["d"]
    t = n * n_tok
    if case["op"] in ("rule", "settle"):
        h_qk, h_v = case["h_qk"], case["h_v"]
        q, k = normal(t, h_qk, d), normal(t, h_qk, d)
        if not case["raw"]:
            q, k = (x * torch.rsqrt(x.square().sum(-1, keepdim=True) + 1e-6) for x in (q, k))
        s["q"], s["k"], s["v"] = q.to(dtype), k.to(dtype), normal(t, h_v, d).to(dtype)
        s["g"] = -torch.nn.functional.softplus(normal(t, h_v) - 1.0)
        logits = normal(t, h_v)
        s["beta"] = logits if case["raw"] else torch.sigmoid(logits)
        s["state"] = 0.2 * normal(n, h_v, d, d)
        if case["op"] == "settle":
            s["deltas"] = 0.5 * normal(t, h_v, d)
        else:
            s["deltas"] = torch.empty(t, h_v, d, dtype=torch.float32, device=dev)
            s["o"] = torch.empty(t, h_v, d, dtype=_DTYPES[case["out"]], device=dev)
        return s
    h_q, h_kv, page, layers = case["h_q"], case["h_kv"], case["page"], case["layers"]
    lens = _lens(case)
    need = [-(-m // page) for m in lens]
    width, spare = max(need), 3
    order = torch.randperm(sum(need) + spare, generator=gen, device=dev).to(torch.int32)
    table = torch.full((n, width), -1, dtype=torch.int32, device=dev)
    rows = torch.repeat_interleave(torch.arange(n), torch.tensor(need)).to(dev)
    cols = torch.cat([torch.arange(m) for m in need]).to(dev)
    table[rows, cols] = order[:sum(need)]
    s["table"], s["kv_lens"] = table, torch.tensor(lens, dtype=torch.int32, device=dev)
    s["longest"], s["scale"] = max(lens), 1.0 / math.sqrt(d)
    pages = sum(need) + spare
    shape = (layers, pages, h_kv, page, d) if case["by_head"] else (layers, pages, page, h_kv, d)
    for name in ("k_cache", "v_cache"):
        c = torch.stack([normal(*shape[1:]).to(dtype) for _ in range(layers)])
        c = c.transpose(2, 3) if case["by_head"] else c  # [layers, pages, page, h_kv, d] either way
        s[name] = c if case["op"] == "compact" else c[0]
    if case["op"] == "compact":
        s["new_lens"] = torch.empty(n, dtype=torch.int32, device=dev)
        return s
    # q, k and v as a layer's fused projection leaves them: one row of h_q + 2 h_kv heads a token
    qkv = normal(t, h_q + 2 * h_kv, d).to(dtype)
    s["q"], s["k"], s["v"] = qkv[:, :h_q], qkv[:, h_q:h_q + h_kv], qkv[:, h_q + h_kv:]
    if case["op"] == "append":
        r = case["rot"] // 2
        s["inv_freq"] = (case["base"] ** (-torch.arange(r, dtype=torch.float64) / r)).float().to(dev)
        s["q_out"] = torch.zeros(t, h_q, d, dtype=dtype, device=dev)
        s["k_out"] = torch.zeros(t, h_kv, d, dtype=dtype, device=dev)
        return s
    s["q"] = (2.0 * s["q"].float()).to(dtype).contiguous()  # normed heads times a learned gain
    s["o"] = torch.empty(t, h_q, d, dtype=dtype, device=dev)
    s["lse"] = torch.empty(t, h_q, dtype=torch.float32, device=dev)
    return s


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "attend": _plain_attend, "rule": _plain_rule, "settle": _plain_settle,
            "compact": _plain_compact}[state["case"]["op"]](state)


# --- through the package ------------------------------------------------------------------------------------

def _own(s):
    import gated_deltanet_scan_gb300 as gdr

    case = s["case"]
    op = case["op"]
    if op == "append":
        gdr.gdr_attn_append_tree(s["q"], s["k"], s["v"], s["q_out"], s["k_out"], s["k_cache"], s["v_cache"],
                                 s["table"], s["kv_lens"], s["inv_freq"], s["parents"],
                                 interleaved=case["interleaved"])
        return s["q_out"], s["k_out"], s["k_cache"], s["v_cache"]
    if op == "attend":
        if s["workspace"] is None:  # a program keeps it from step to step
            need = gdr.gdr_attn_decode_tree_workspace_bytes(s["q"], s["k_cache"], s["parents"])
            s["workspace"] = torch.empty(max(16, need), dtype=torch.uint8, device=s["q"].device)
        gdr.gdr_attn_decode_tree(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_lens"], s["o"], s["parents"],
                                 scale=s["scale"], lse=s["lse"], workspace=s["workspace"])
        return s["o"], s["lse"]
    if op == "rule":
        gdr.gdr_verify_tree(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], s["o"], s["parents"],
                            deltas=s["deltas"], qk_l2norm=case["raw"], beta_logits=case["raw"])
        return s["o"], s["deltas"]
    if op == "settle":
        gdr.gdr_verify_tree_commit(s["k"], s["g"], s["deltas"], s["state"], s["parents"], s["last"],
                                   qk_l2norm=case["raw"])
        return s["state"]
    gdr.gdr_attn_commit_tree(s["k_cache"], s["v_cache"], s["table"], s["kv_lens"], s["parents"], s["last"],
                             s["new_lens"])
    return s["k_cache"], s["v_cache"], s["new_lens"]


# --- plain forms --------------------------------------------------------------------------------------------

def _ancestors(parents):
    """[n, t, t] truth values: column i is j or one of j's ancestors (as many steps up as there can be)."""
    t = parents.shape[1]
    up = torch.arange(t, device=parents.device) == parents[:, :, None]
    ways = torch.linalg.matrix_power(up.float() + torch.eye(t, device=up.device), t)
    return (ways > 0.5) & (parents != -2)[:, :, None]


def _places(s, pos):
    """Page and slot of positions pos [n, ...] of every sequence."""
    page = s["case"]["page"]
    flat = s["table"].gather(1, (pos // page).flatten(1).long()).view(pos.shape)
    return flat.long(), (pos % page).long()


def _plain_append(s):
    case = s["case"]
    n, n_tok = s["parents"].shape
    real = (s["parents"] != -2).view(-1, 1, 1)
    base = (s["kv_lens"] - n_tok)[:, None]
    pos = (base + _ancestors(s["parents"]).sum(-1) - 1).view(-1)
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

    s["q_out"].copy_(torch.where(real, turned(s["q"]), s["q_out"]))
    s["k_out"].copy_(torch.where(real, turned(s["k"]), s["k_out"]))
    page, slot = (x.view(-1) for x in _places(s, base + torch.arange(n_tok, device=base.device)))
    s["k_cache"][page, slot] = torch.where(real, s["k_out"], s["k_cache"][page, slot])
    s["v_cache"][page, slot] = torch.where(real, s["v"], s["v_cache"][page, slot])
    return s["q_out"], s["k_out"], s["k_cache"], s["v_cache"]


def _plain_attend(s):
    case, parents = s["case"], s["parents"]
    n, n_tok = parents.shape
    h_q, h_kv, d, m = case["h_q"], case["h_kv"], case["d"], s["longest"]
    pos = torch.arange(m, device=parents.device).expand(n, m)
    page, slot = _places(s, pos)
    page = page.clamp_min(0)  # past a sequence's end: masked below
    inside = (pos < s["kv_lens"][:, None])[:, :, None, None]
    k = s["k_cache"][page, slot].float().permute(0, 2, 3, 1)  # [n, h_kv, d, m]
    v = s["v_cache"][page, slot].float().masked_fill_(~inside, 0.0).permute(0, 2, 1, 3)
    q = s["q"].float().view(n, n_tok, h_kv, h_q // h_kv, d).permute(0, 2, 3, 1, 4).reshape(n, h_kv, -1, d)
    x = (torch.matmul(q, k) * s["scale"]).view(n, h_kv, h_q // h_kv, n_tok, m)
    node = pos - (s["kv_lens"] - n_tok)[:, None]  # a slot's node, negative before the tree
    on_path = _ancestors(parents).gather(2, node.clamp(0, n_tok - 1)[:, None].expand(n, n_tok, m))
    seen = torch.where((node < 0)[:, None], (parents != -2)[:, :, None], on_path & (node < n_tok)[:, None])
    x = x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(n, h_kv, -1, m), v).view(n, h_kv, h_q // h_kv, n_tok, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    s["o"].copy_(o.permute(0, 3, 1, 2, 4).reshape(n * n_tok, h_q, d))
    s["lse"].copy_((total.log() + top).squeeze(-1).permute(0, 3, 1, 2).reshape(n * n_tok, h_q))
    return s["o"], s["lse"]


def _unit(x):
    return x * torch.rsqrt(x.square().sum(-1, keepdim=True) + 1e-6)


def _heads(s, name, of):
    """[n, h_v, n_tok, d] in 32 bits; q and k repeated for the value heads that share them."""
    case = s["case"]
    x = s[name].float()
    if of != "v" and case["raw"]:
        x = _unit(x)
    x = x.view(-1, case["n_tok"], x.shape[1], case["d"]).transpose(1, 2)
    return x if of == "v" else x.repeat_interleave(case["h_v"] // case["h_qk"], 1)


def _sums(s, on):
    """G_j: the sum of g along the path to j, [n, h_v, n_tok]; 64 bits, as differences of long sums follow."""
    n, t, _ = on.shape
    g = torch.where(s["parents"].view(-1, 1) == -2, torch.zeros_like(s["g"]), s["g"])
    return (on.double() @ g.double().view(n, t, -1)).transpose(1, 2)


def _plain_rule(s):
    case = s["case"]
    on = _ancestors(s["parents"])
    n, t, _ = on.shape
    real = (s["parents"] != -2)[:, None, :, None]
    q, k, v = _heads(s, "q", "qk"), _heads(s, "k", "qk"), _heads(s, "v", "v")
    beta = torch.sigmoid(s["beta"]) if case["raw"] else s["beta"]
    beta = beta.view(n, t, -1).transpose(1, 2)[..., None]
    total = _sums(s, on)
    decay = torch.where(on[:, None], torch.exp(total[..., :, None] - total[..., None, :]), 0.0).float()
    grown = torch.exp(total).float()[..., None]
    lower = beta * decay * torch.matmul(k, k.transpose(2, 3))
    right = beta * (v - grown * torch.matmul(k, s["state"]))
    u = torch.linalg.solve_triangular(lower, right, upper=False, unitriangular=True)
    u = torch.where(real, u, torch.zeros_like(u))
    o = grown * torch.matmul(q, s["state"]) + torch.matmul(decay * torch.matmul(q, k.transpose(2, 3)), u)
    o = torch.where(real, o, torch.zeros_like(o))
    s["o"].copy_(o.transpose(1, 2).reshape(s["o"].shape))
    s["deltas"].copy_(u.transpose(1, 2).reshape(s["deltas"].shape))
    return s["o"], s["deltas"]


def _accepted(s, on):
    """Truth values [n, n_tok]: the nodes of the accepted path."""
    last = s["last"].long()
    path = on.gather(1, last.clamp_min(0)[:, None, None].expand(-1, 1, on.shape[2]))[:, 0]
    return path & (last >= 0)[:, None]


def _plain_settle(s):
    on = _ancestors(s["parents"])
    path = _accepted(s, on)
    n, t = path.shape
    g = torch.where(path[..., None], s["g"].view(n, t, -1), 0.0).double()
    total = g.sum(1, keepdim=True)
    w = torch.where(path[..., None], torch.exp(total - g.cumsum(1)), 0.0).float().transpose(1, 2)[..., None]
    k = _heads(s, "k", "qk")
    u = s["deltas"].view(n, t, -1, s["case"]["d"]).transpose(1, 2)
    grown = torch.exp(total).float().transpose(1, 2)[..., None]
    s["state"].copy_(grown * s["state"] + torch.matmul((w * k).transpose(2, 3), u))
    return s["state"]


def _plain_compact(s):
    path = _accepted(s, _ancestors(s["parents"]))
    n, t = path.shape
    count = path.sum(1)
    to = torch.arange(t, device=path.device).expand(n, t)
    order = torch.argsort((~path).to(torch.int32), dim=1, stable=True)
    base = (s["kv_lens"] - t)[:, None]
    page, slot = _places(s, base + torch.where(to < count[:, None], order, to))  # other rows stay
    page_to, slot_to = _places(s, base + to)
    s["k_cache"][:, page_to, slot_to] = s["k_cache"][:, page, slot]
    s["v_cache"][:, page_to, slot_to] = s["v_cache"][:, page, slot]
    s["new_lens"].copy_(base[:, 0] + count)
    return s["k_cache"], s["v_cache"], s["new_lens"]


# --- in 64 bits, from the definitions -----------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "rule": _exact_rule, "settle": _exact_settle,
            "compact": _exact_compact}[case["op"]](s)


def _exact_append(s):
    case = s["case"]
    r, pairs, n_tok, page = case["rot"] // 2, case["interleaved"], case["n_tok"], case["page"]
    parents, _ = _trees(case)
    q, k = s["q_out"].double(), s["k_out"].double()
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    for b, (m, one) in enumerate(zip(_lens(case), parents)):
        paths = _paths(one)
        nodes = [j for j in range(n_tok) if paths[j]]
        rows = torch.tensor([b * n_tok + j for j in nodes], device=q.device)
        depth = torch.tensor([m - n_tok + len(paths[j]) - 1 for j in nodes], dtype=torch.float64, device=q.device)
        z = torch.polar(torch.ones(len(nodes), 1, r, dtype=torch.float64, device=q.device),
                        depth.view(-1, 1, 1) * s["inv_freq"].double())
        for x, y in ((s["q"], q), (s["k"], k)):
            x = x[rows].double()
            first = slice(0, 2 * r, 2) if pairs else slice(0, r)
            second = slice(1, 2 * r, 2) if pairs else slice(r, 2 * r)
            w = torch.complex(x[..., first], x[..., second]) * z
            x[..., first], x[..., second] = w.real, w.imag
            y[rows] = x
        at = torch.tensor([m - n_tok + j for j in nodes], device=q.device)
        where = s["table"][b].long()[at // page], at % page
        kc[where], vc[where] = k[rows], s["v"][rows].double()
    return q, k, kc, vc


def _exact_attend(s):
    case = s["case"]
    n_tok, page, group = case["n_tok"], case["page"], case["h_q"] // case["h_kv"]
    parents, _ = _trees(case)
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=s["q"].device)
    for b, (m, one) in enumerate(zip(_lens(case), parents)):
        at = torch.arange(m, device=o.device)
        where = s["table"][b].long()[at // page], at % page
        k, v = s["k_cache"][where].double(), s["v_cache"][where].double()
        hidden = torch.ones(n_tok, m, dtype=torch.bool)
        paths = _paths(one)
        for j, path in enumerate(paths):
            if path:
                hidden[j, :m - n_tok] = False
                hidden[j, [m - n_tok + i for i in path]] = False
        hidden = hidden.to(o.device)
        rows = torch.tensor([b * n_tok + j for j in range(n_tok)], device=o.device)
        kept = torch.tensor([bool(p) for p in paths], device=o.device)
        for h in range(case["h_q"]):
            x = case["d"] ** -0.5 * (s["q"][rows, h].double() @ k[:, h // group].T)
            x[hidden] = -math.inf
            z = torch.logsumexp(x, -1)
            weights = torch.exp(x - z[:, None])
            lse[rows[kept], h] = z[kept]
            o[rows[kept], h] = weights[kept] @ v[:, h // group]
    return o, lse


def _exact_rule(s):
    """The recurrence itself: every node's state from its parent's, 2 GB of states at a time."""
    case = s["case"]
    h_qk, h_v, n_tok, d = case["h_qk"], case["h_v"], case["n_tok"], case["d"]
    parents, _ = _trees(case)
    n, dev = len(parents), s["q"].device
    o = torch.zeros(n, n_tok, h_v, d, dtype=torch.float64, device=dev)
    u = torch.zeros(n, n_tok, h_v, d, dtype=torch.float64, device=dev)
    share = torch.arange(h_v, device=dev) // (h_v // h_qk)
    step = max(1, (1 << 28) // ((n_tok + 1) * h_v * d * d))
    for b in range(0, n, step):
        some = range(b, min(n, b + step))
        states = torch.zeros(len(some), n_tok + 1, h_v, d, d, dtype=torch.float64, device=dev)  # S_0 first
        states[:, 0] = s["state"][b:b + len(some)].double()
        at = torch.arange(len(some), device=dev)
        for j in range(n_tok):
            up = torch.tensor([max(-1, parents[i][j]) + 1 for i in some], device=dev)
            real = torch.tensor([parents[i][j] != -2 for i in some], device=dev).view(-1, 1, 1)
            rows = torch.tensor([i * n_tok + j for i in some], device=dev)
            q, k, v = s["q"][rows].double()[:, share], s["k"][rows].double()[:, share], s["v"][rows].double()
            if case["raw"]:
                q, k = (x / (x.square().sum(-1, keepdim=True) + 1e-6).sqrt() for x in (q, k))
            beta, g = s["beta"][rows].double(), s["g"][rows].double()
            if case["raw"]:
                beta = 1.0 / (1.0 + torch.exp(-beta))
            old = torch.exp(g)[..., None, None] * states[at, up]
            delta = beta[..., None] * (v - torch.einsum("bhkv,bhk->bhv", old, k))
            states[:, j + 1] = old + k[..., :, None] * delta[..., None, :]
            o[b:b + len(some), j] = torch.where(real, torch.einsum("bhkv,bhk->bhv", states[:, j + 1], q), 0.0)
            u[b:b + len(some), j] = torch.where(real, delta, 0.0)
    return o.view(s["o"].shape), u.view(s["deltas"].shape)


def _exact_settle(s):
    """S = e^g S + k u^T along the accepted path, node by node."""
    case = s["case"]
    h_qk, h_v, n_tok = case["h_qk"], case["h_v"], case["n_tok"]
    parents, last = _trees(case)
    state = s["state"].double()
    share = torch.arange(h_v, device=state.device) // (h_v // h_qk)
    for b, a in enumerate(last):
        for j in _paths(parents[b])[a] if a >= 0 else []:
            row = b * n_tok + j
            k = s["k"][row].double()[share]
            if case["raw"]:
                k = k / (k.square().sum(-1, keepdim=True) + 1e-6).sqrt()
            state[b] = torch.exp(s["g"][row].double())[:, None, None] * state[b] \
                + k[:, :, None] * s["deltas"][row].double()[:, None, :]
    return state


def _exact_compact(s):
    case = s["case"]
    n_tok, page = case["n_tok"], case["page"]
    parents, last = _trees(case)
    kc, vc, table = s["k_cache"].double(), s["v_cache"].double(), s["table"].tolist()
    lens = []
    for b, (m, a) in enumerate(zip(_lens(case), last)):
        path = _paths(parents[b])[a] if a >= 0 else []
        lens.append(m - n_tok + len(path))
        for i, j in enumerate(path):
            src, dst = m - n_tok + j, m - n_tok + i
            p, r = table[b][src // page], table[b][dst // page]
            kc[:, r, dst % page] = s["k_cache"][:, p, src % page].double()
            vc[:, r, dst % page] = s["v_cache"][:, p, src % page].double()
    return kc, vc, torch.tensor(lens, dtype=torch.int32, device=kc.device)
