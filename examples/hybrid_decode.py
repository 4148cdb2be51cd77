"""A small hybrid model served with the library: three gated-delta-rule layers, then one softmax-attention layer.

Random weights, head shapes of the 9B model the library was written for (rule: 16 QK and 32 V heads of 128;
attention: 16 query and 4 key/value heads of 256, rotation over 64 of them).  Two prompts of different lengths are
prefilled as one packed batch; then both sequences decode token by token from the rule's states and the paged cache,
and last a block of draft tokens goes through attention at once.  A second run verifies trees of drafted tokens in all
layers and accepts a path of each.

    python examples/hybrid_decode.py
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gated_deltanet_scan_gb300 as gdr  # noqa: E402

WIDTH, PAGE, ROT = 512, 64, 64
RULE_QK, RULE_V, RULE_D = 16, 32, 128
ATT_Q, ATT_KV, ATT_D = 16, 4, 256


def linear(n_in, n_out, gen):
    w = torch.randn(n_in, n_out, generator=gen, device="cuda") * n_in ** -0.5
    return w.to(torch.bfloat16)


def norm(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


class RuleLayer:
    """x + out(norm(rule(q, k, v, g, beta)) gated by z), one state per sequence and V head."""

    def __init__(self, gen, n_seqs):
        self.qkv = linear(WIDTH, (2 * RULE_QK + RULE_V) * RULE_D, gen)
        self.gates = linear(WIDTH, 2 * RULE_V, gen)
        self.z = linear(WIDTH, RULE_V * RULE_D, gen)
        self.out = linear(RULE_V * RULE_D, WIDTH, gen)
        self.weight = torch.ones(RULE_D, device="cuda")
        self.state = torch.zeros(n_seqs, RULE_V, RULE_D, RULE_D, device="cuda")

    def inputs(self, x):
        h = norm(x)
        qkv = (h @ self.qkv).view(-1, 2 * RULE_QK + RULE_V, RULE_D)
        q, k, v = (t.contiguous() for t in qkv.split([RULE_QK, RULE_QK, RULE_V], dim=1))
        a, b = (h @ self.gates).float().split(RULE_V, dim=1)
        return q, k, v, -torch.nn.functional.softplus(a), b.contiguous(), (h @ self.z).view(-1, RULE_V, RULE_D)

    def __call__(self, x, cu):
        q, k, v, g, b, z = self.inputs(x)
        o = torch.empty(v.shape, dtype=torch.float32, device="cuda")
        if cu is not None:
            gdr.gdr_prefill_chunked(q, k, v, g, b, self.state, o, cu, qk_l2norm=True, beta_logits=True)
            gdr.gdr_gated_rmsnorm(o, z, self.weight, o)
        else:
            gdr.gdr_decode_step_gated(q, k, v, g, b, self.state, z, self.weight, o, qk_l2norm=True,
                                      beta_logits=True)
        return x + o.view(x.shape[0], -1).to(torch.bfloat16) @ self.out

    def tree(self, x, parents):
        """Every node of a tree per sequence; what accept() takes.  The states stay."""
        q, k, v, g, b, z = self.inputs(x)
        o, deltas = (torch.empty(v.shape, dtype=torch.float32, device="cuda") for _ in range(2))
        gdr.gdr_verify_tree(q, k, v, g, b, self.state, o, parents, deltas=deltas, qk_l2norm=True, beta_logits=True)
        gdr.gdr_gated_rmsnorm(o, z, self.weight, o)
        return x + o.view(x.shape[0], -1).to(torch.bfloat16) @ self.out, (k, g, deltas)

    def accept(self, kept, parents, last):
        gdr.gdr_verify_tree_commit(*kept, self.state, parents, last, qk_l2norm=True)


class AttentionLayer:
    """x + out(attention(rotated q, rotated k, v)), keys and values in a paged cache."""

    def __init__(self, gen, n_seqs, max_tokens):
        self.qkv = linear(WIDTH, (ATT_Q + 2 * ATT_KV) * ATT_D, gen)
        self.out = linear(ATT_Q * ATT_D, WIDTH, gen)
        width = -(-max_tokens // PAGE)
        self.k_cache = torch.empty(n_seqs * width, PAGE, ATT_KV, ATT_D, dtype=torch.bfloat16, device="cuda")
        self.v_cache = torch.empty_like(self.k_cache)
        self.table = torch.randperm(n_seqs * width, generator=gen, device="cuda").to(torch.int32).view(n_seqs, width)
        self.kv_lens = torch.zeros(n_seqs, dtype=torch.int32, device="cuda")
        self.inv_freq = 1e7 ** (-torch.arange(ROT // 2, device="cuda").float() / (ROT // 2))

    def __call__(self, x, cu, n_tok=1):
        qkv = (norm(x) @ self.qkv).view(-1, ATT_Q + 2 * ATT_KV, ATT_D)
        q, k, v = qkv.split([ATT_Q, ATT_KV, ATT_KV], dim=1)  # strided rows, as they are
        self.kv_lens += n_tok if cu is None else cu[1:] - cu[:-1]
        # rotated in place, keys and values appended
        gdr.gdr_attn_append(q, k, v, q, k, self.k_cache, self.v_cache, self.table, self.kv_lens, self.inv_freq, cu)
        o = torch.empty(x.shape[0], ATT_Q, ATT_D, dtype=torch.bfloat16, device="cuda")
        if cu is not None:  # whole prompts
            gdr.gdr_attn_prefill(q, k, v, o, cu)
        else:  # the last n_tok tokens of every sequence
            gdr.gdr_attn_decode(q, self.k_cache, self.v_cache, self.table, self.kv_lens, o, n_tok)
        return x + o.view(x.shape[0], -1) @ self.out

    def tree(self, x, parents):
        """Every node of a tree per sequence, in the slots after the sequence's tokens."""
        qkv = (norm(x) @ self.qkv).view(-1, ATT_Q + 2 * ATT_KV, ATT_D)
        q, k, v = qkv.split([ATT_Q, ATT_KV, ATT_KV], dim=1)
        self.kv_lens += parents.shape[1]
        gdr.gdr_attn_append_tree(q, k, v, q, None, self.k_cache, self.v_cache, self.table, self.kv_lens, self.inv_freq,
                                 parents)
        o = torch.empty(x.shape[0], ATT_Q, ATT_D, dtype=torch.bfloat16, device="cuda")
        gdr.gdr_attn_decode_tree(q, self.k_cache, self.v_cache, self.table, self.kv_lens, o, parents)
        return x + o.view(x.shape[0], -1) @ self.out

    def accept(self, parents, last):
        new = torch.empty_like(self.kv_lens)  # other sequences' blocks still read the lengths
        gdr.gdr_attn_commit_tree(self.k_cache, self.v_cache, self.table, self.kv_lens, parents, last, new)
        self.kv_lens = new


def run(lengths=(300, 77), steps=8, draft=4, seed=0):
    """The attention layer's outputs: of the prompts, of `steps` decoded tokens per sequence, and of a draft block;
    and the same rows from one prefill of the whole sequences."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n, total = len(lengths), max(lengths) + steps + draft
    rules, att = [RuleLayer(gen, n) for _ in range(3)], AttentionLayer(gen, n, total)

    def embed(count):
        return torch.randn(count, WIDTH, generator=gen, device="cuda").to(torch.bfloat16)

    def starts(lens):
        return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")

    def forward(x, cu):
        for layer in rules:
            x = layer(x, cu)
        return x, att(x, cu)

    hidden = [[] for _ in lengths]  # what the attention layer saw, by sequence
    got = [[] for _ in lengths]
    x, y = forward(embed(sum(lengths)), starts(lengths))
    for s, (a, b) in enumerate(zip(x.split(list(lengths)), y.split(list(lengths)))):
        hidden[s].append(a)
        got[s].append(b)
    for _ in range(steps):
        x, y = forward(embed(n), None)
        for s in range(n):
            hidden[s].append(x[s:s + 1])
            got[s].append(y[s:s + 1])
    x = embed(n * draft)
    y = att(x, None, draft)
    for s in range(n):
        hidden[s].append(x[s * draft:(s + 1) * draft])
        got[s].append(y[s * draft:(s + 1) * draft])

    att.kv_lens.zero_()
    whole = att(torch.cat([t for h in hidden for t in h]), starts([m + steps + draft for m in lengths]))
    return torch.cat([t for g in got for t in g]), whole


def run_tree(lengths=(300, 77), seed=0):
    """Outputs of the accepted nodes of a drafted tree per sequence, by sequence, and of the same tokens decoded one
    after another; and the lengths both leave in the cache."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    trees = [[-1, 0, 0, 1, 3, 2, 3], [-1, -1, 1, 2, -2, -2, -2]]  # the second has three rows that are no nodes
    paths = [[0, 1, 3, 6], [1, 2, 3]]  # accepted
    n, n_tok = len(trees), len(trees[0])
    parents = torch.tensor(trees, dtype=torch.int32, device="cuda")
    last = torch.tensor([p[-1] for p in paths], dtype=torch.int32, device="cuda")
    rules, att = [RuleLayer(gen, n) for _ in range(3)], AttentionLayer(gen, n, max(lengths) + n_tok)
    x = torch.randn(sum(lengths), WIDTH, generator=gen, device="cuda").to(torch.bfloat16)
    cu = torch.tensor([0, lengths[0], sum(lengths)], dtype=torch.int32, device="cuda")
    for layer in rules + [att]:
        x = layer(x, cu)
    before = [layer.state.clone() for layer in rules], att.kv_lens.clone()

    drafted = torch.randn(n * n_tok, WIDTH, generator=gen, device="cuda").to(torch.bfloat16)
    x, kept = drafted, []
    for layer in rules:
        x, k = layer.tree(x, parents)
        kept.append(k)
    tree = att.tree(x, parents)
    for layer, k in zip(rules, kept):  # once a path of each is chosen
        layer.accept(k, parents, last)
    att.accept(parents, last)
    lens = att.kv_lens

    one = []
    for s, path in enumerate(paths):
        for layer, state in zip(rules, before[0]):
            layer.state = state.clone()
        att.kv_lens = before[1].clone()
        for j in path:  # the other sequence takes the same token, and is not looked at
            x = drafted[s * n_tok + j].expand(n, -1)
            for layer in rules + [att]:
                x = layer(x, None)
            one.append(x[s])
    return (torch.stack([tree[s * n_tok + j] for s, path in enumerate(paths) for j in path]), torch.stack(one),
            lens.tolist(), [m + len(path) for m, path in zip(lengths, paths)])


if __name__ == "__main__":
    tokens, whole = run()
    print(f"{tokens.shape[0]} rows; step by step against one prefill: "
          f"largest difference {(tokens.float() - whole.float()).abs().max().item():.3g} "
          f"of {whole.float().abs().max().item():.3g}")
    tokens, one, lens, _ = run_tree()
    print(f"{tokens.shape[0]} accepted nodes of two trees: one after another "
          f"{(tokens.float() - one.float()).abs().max().item():.3g} off, lengths {lens}")
