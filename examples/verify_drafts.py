"""Verifying a tree of drafted tokens with a small FP8 decoder.

    python examples/verify_drafts.py

Layers of random weights keep their keys and values in the paged FP8 cache.  A
few requests of different lengths are fed token by token; then each gets a tree
of drafted tokens, which one pass verifies: the drafts' keys and values are
written into the cache, every draft attends to the context and to its own
ancestors, and the mixture of experts takes the few rows of all the drafts.
The longest path that the model agrees with is accepted, and its rows move to
the places that they would have had token by token.

The same decoder also goes one token at a time.  Both ways compute the same
numbers but for the roundings of sums taken in another order; the program prints
how far apart the hidden rows are and fails if that is more than bf16
activations explain.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_fine_grained_e4m3_amd as dg  # noqa: E402


class Decoder:
    """RMS norm, attention over the FP8 cache and a mixture of experts, `layers` times."""

    def __init__(self, layers, hidden, heads, kv_heads, head_dim, experts, topk, inner, vocab, pages, page_size, seed=0):
        self.heads, self.kv_heads, self.head_dim, self.topk, self.page_size = heads, kv_heads, head_dim, topk, page_size
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape):
            return torch.randn(*shape, generator=gen, device="cuda") / math.sqrt(shape[-1])

        self.embed = torch.randn(vocab, hidden, generator=gen, device="cuda").bfloat16()
        self.layers = [dict(
            qkv=dg.per_block_cast_to_fp8(weight((heads + 2 * kv_heads) * head_dim, hidden)),
            out=dg.per_block_cast_to_fp8(weight(hidden, heads * head_dim)),
            router=weight(experts, hidden),
            up=dg.per_block_cast_to_fp8(weight(experts, 2 * inner, hidden)),
            down=dg.per_block_cast_to_fp8(weight(experts, hidden, inner)),
            cache=dg.make_fp8_kv_cache(pages, kv_heads, page_size, head_dim)) for _ in range(layers)]

    @staticmethod
    def norm(x):
        x = x.float()
        return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()

    @staticmethod
    def linear(x, w):
        y = torch.empty(x.shape[0], w[0].shape[0], dtype=torch.bfloat16, device="cuda")
        return dg.fp8_gemm_nt(dg.per_token_cast_to_fp8(x), w, y)

    def slots(self, table, positions):
        """Cache slots [B, N] of the requests' positions [B, N]; -1 where a position is negative."""
        pages = torch.gather(table, 1, (positions.clamp(min=0) // self.page_size).long())
        return torch.where(positions < 0, -1, pages * self.page_size + positions % self.page_size).int()

    def forward(self, tokens, table, context_lens, tree_lens, mask):
        """Hidden rows [B, N, hidden] of tokens [B, N] that follow the cached context."""
        B, N = tokens.shape
        at = torch.arange(N, dtype=torch.int32, device="cuda")
        live = at < tree_lens[:, None]
        slots = self.slots(table, torch.where(live, context_lens[:, None] + at, -1)).reshape(-1)
        Q, KV, D = self.heads, self.kv_heads, self.head_dim
        embedded = self.embed[tokens].reshape(B * N, -1)
        x = embedded
        for layer in self.layers:
            qkv = self.linear(self.norm(x), layer["qkv"]).view(B * N, Q + 2 * KV, D)
            dg.fp8_kv_cache_write(qkv[:, Q:Q + KV], qkv[:, Q + KV:], layer["cache"], slots)
            o, _ = dg.fp8_tree_attention(qkv[:, :Q].unflatten(0, (B, N)), layer["cache"], table, context_lens, tree_lens, mask)
            x = x + self.linear(o.view(B * N, Q * D), layer["out"])
            rows = self.norm(x)
            # routed by the token alone: by the hidden row, a near tie would send a row to other
            # experts on one way than on the other, and they could not be compared
            weights, ids = torch.topk(torch.softmax(embedded.float() @ layer["router"].t(), -1), self.topk)
            weights = weights / weights.sum(-1, keepdim=True)
            ids = torch.where(live.reshape(-1, 1), ids, -1).int()
            x = x + dg.fp8_moe_few_tokens(rows, layer["up"], layer["down"], ids, weights)
        return x.view(B, N, -1)

    def move(self, source, target):
        """Cache rows of the slots `source` into the slots `target`.  Read and quantised again, a
        row keeps its codes, and its scales but for the last bit."""
        for layer in self.layers:
            k, v = dg.fp8_kv_cache_read(layer["cache"], source, dtype=torch.float32)
            dg.fp8_kv_cache_write(k, v, layer["cache"], target)

    def predict(self, x):
        return (self.norm(x).float() @ self.embed.float().t()).argmax(-1)


def mask_of(parents):
    """Mask words [B, N, ceil(N / 64)] of trees given by each draft's parent (-1: the context)."""
    B, N = len(parents), len(parents[0])
    words = torch.zeros(B, N, -(-N // 64), dtype=torch.int64)
    for b, tree in enumerate(parents):
        for i in range(N):
            j = i
            while j >= 0:
                bit = 1 << (j % 64)
                words[b, i, j // 64] |= bit - (1 << 64) if j % 64 == 63 else bit
                j = tree[j]
    return words.cuda()


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--requests", type=int, default=3)
    p.add_argument("--prompt", type=int, default=40, help="tokens of the longest prompt")
    p.add_argument("--drafts", type=int, default=12, help="drafted tokens of a tree")
    p.add_argument("--layers", type=int, default=2)
    args = p.parse_args(argv)
    B, N = args.requests, args.drafts
    page_size, hidden, vocab = 16, 1024, 64
    max_pages = -(-(args.prompt + N + 1) // page_size)
    model = Decoder(args.layers, hidden, heads=16, kv_heads=4, head_dim=64, experts=16, topk=4, inner=512, vocab=vocab,
                    pages=2 * B * max_pages, page_size=page_size)
    gen = torch.Generator().manual_seed(1)
    tables = torch.randperm(2 * B * max_pages, generator=gen).int().cuda().view(2, B, max_pages)
    tree_table, step_table = tables[0].contiguous(), tables[1].contiguous()
    prompt = torch.randint(vocab, (B, args.prompt), generator=gen).cuda()
    lens = torch.randint(1, args.prompt + 1, (B,), generator=gen).int()
    lens[0] = args.prompt
    lens = lens.cuda()

    # The prompts, one token a pass, into the pages of both tables.
    for table in (tree_table, step_table):
        last = None
        for i in range(args.prompt):
            here = torch.full((B,), i, dtype=torch.int32, device="cuda")
            live = (here < lens).int()
            x = model.forward(prompt[:, i:i + 1], table, here, live, None)
            last = x if last is None else torch.where((live > 0)[:, None, None], x, last)
    first = model.predict(last[:, 0])

    # What the model says next, token by token: the longest that a path of a tree can be.
    none = torch.ones(B, dtype=torch.int32, device="cuda")
    tokens, alone = [first], []
    for i in range(N):
        alone.append(model.forward(tokens[-1][:, None], step_table, lens + i, none, None)[:, 0])
        tokens.append(model.predict(alone[-1]))

    # Random trees of random tokens, but for those on the way to the deepest draft: these are what
    # the model will say, as a good drafter's would be.
    parents = [[-1] + [int(torch.randint(max(0, i - 4), i, (1,), generator=gen)) for i in range(1, N)] for _ in range(B)]
    drafts = torch.randint(vocab, (B, N), generator=gen).cuda()
    for b, tree in enumerate(parents):
        chains = [[0]]
        for i in range(1, N):
            chains.append(chains[tree[i]] + [i])
        for depth, i in enumerate(max(chains, key=len)):
            drafts[b, i] = tokens[depth][b]
    hidden_rows = model.forward(drafts, tree_table, lens, torch.full_like(none, N), mask_of(parents))
    follows = model.predict(hidden_rows).tolist()

    # The longest path on which every draft is what the model predicted at its parent.
    paths = []
    for b in range(B):
        agreed = {0: [0]}
        for i in range(1, N):
            path = agreed.get(parents[b][i])
            if path is not None and follows[b][path[-1]] == int(drafts[b, i]):
                agreed[i] = path + [i]
        paths.append(max(agreed.values(), key=len))
    longest = max(map(len, paths))
    counts = torch.tensor([len(path) for path in paths], dtype=torch.int32, device="cuda")
    accepted = torch.tensor([path + [-1] * (longest - len(path)) for path in paths], dtype=torch.int32, device="cuda")
    at = torch.arange(longest, dtype=torch.int32, device="cuda")
    source = torch.where(accepted < 0, -1, lens[:, None] + accepted)
    target = torch.where(accepted < 0, -1, lens[:, None] + at)
    model.move(model.slots(tree_table, source).reshape(-1), model.slots(tree_table, target).reshape(-1))

    # How far the two ways are apart on the accepted paths, and one step after them.
    def apart(a, b):
        return float(((a.float() - b.float()).norm(dim=-1) / b.float().norm(dim=-1)).max())

    worst = max(apart(hidden_rows[b, path], torch.stack([alone[i][b] for i in range(len(path))]))
                for b, path in enumerate(paths))
    token = torch.stack([tokens[len(path)][b] for b, path in enumerate(paths)])[:, None]
    after = apart(*(model.forward(token, table, lens + counts, none, None)[:, 0] for table in (tree_table, step_table)))
    print(f"{B} requests of {lens.tolist()} tokens, trees of {N} drafts, accepted {counts.tolist()}")
    print(f"hidden rows, tree against token by token: {worst:.1e} apart; the step after: {after:.1e}")
    # A row passes some ten bf16 roundings of 2^-9 a layer, and the FP8 casts in front of the
    # projections turn a last-bit difference into one of 2^-4 in a few of its values.
    bound = args.layers * 2.0 ** -6
    if not (worst <= bound and after <= bound):
        raise SystemExit(f"further apart than {bound:.1e}")
    return paths


if __name__ == "__main__":
    main()
