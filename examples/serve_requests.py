"""Serving a batch of requests that come and go, with a small decoder over the FP4 (or FP8) cache.

    python examples/serve_requests.py [--cache fp8]

The batch has a fixed number of places.  Prompts that arrive are fed together, each a chain of
tokens; then every place takes one token a step, in a captured graph.  Each time the plan gives new
tokens their pages, slots and positions, queries and keys are normalised and rotated, keys and values
go into the paged cache, and attention reads it.  A request that is done gives its pages back, and
another prompt takes its place.  The pool has too few pages for all requests at their longest, so
some wait.

Each step's attention is compared with the same in fp32 over the rows that the cache stands for; the
program fails if they are further apart than the roundings explain, or if a page is lost.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_fine_grained_e4m3_amd as dg  # noqa: E402


class Decoder:
    """Layers of RMS norm, attention and a linear layer, with FP8 weights."""

    def __init__(self, bits, layers, hidden, heads, kv_heads, head_dim, vocab, pages, page_size, seed=0):
        self.heads, self.kv_heads, self.head_dim, self.page_size = heads, kv_heads, head_dim, page_size
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape):
            return torch.randn(*shape, generator=gen, device="cuda") / math.sqrt(shape[-1])

        self.make, self.write, self.read, self.attention = (
            getattr(dg, name) for name in (f"make_{bits}_kv_cache", f"{bits}_kv_cache_write", f"{bits}_kv_cache_read",
                                           f"{bits}_tree_attention"))
        self.embed = torch.randn(vocab, hidden, generator=gen, device="cuda").bfloat16()
        self.inv_freq = (10000.0 ** (-2.0 * torch.arange(head_dim // 2, dtype=torch.float64) / head_dim)).float().cuda()
        self.layers = [dict(
            qkv=dg.per_block_cast_to_fp8(weight((heads + 2 * kv_heads) * head_dim, hidden)),
            out=dg.per_block_cast_to_fp8(weight(hidden, heads * head_dim)),
            q_norm=1 + 0.1 * torch.randn(head_dim, generator=gen, device="cuda"),
            k_norm=1 + 0.1 * torch.randn(head_dim, generator=gen, device="cuda"),
            cache=self.make(pages, kv_heads, page_size, head_dim)) for _ in range(layers)]

    @staticmethod
    def norm(x):
        x = x.float()
        return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()

    @staticmethod
    def linear(x, w):
        y = torch.empty(x.shape[0], w[0].shape[0], dtype=torch.bfloat16, device="cuda")
        return dg.fp8_gemm_nt(dg.per_token_cast_to_fp8(x), w, y)

    def forward(self, tokens, slots, positions, attend, trace=None):
        """Hidden rows of tokens [T]; attend(q, cache) -> o, both [T, heads, head_dim]."""
        Q, KV, D = self.heads, self.kv_heads, self.head_dim
        x = self.embed[tokens]
        for layer in self.layers:
            qkv = self.linear(self.norm(x), layer["qkv"]).view(-1, Q + 2 * KV, D)
            q, k = dg.qk_norm_rope(qkv[:, :Q], qkv[:, Q:Q + KV], layer["q_norm"], layer["k_norm"], positions, self.inv_freq)
            self.write(k, qkv[:, Q + KV:], layer["cache"], slots)
            o = attend(q, layer["cache"])
            if trace is not None:
                trace.append((q, o))
            x = x + self.linear(o.reshape(-1, Q * D), layer["out"])
        return x


def dense_attention(model, q, cache, slots):
    """Attention in fp32 of the last query over the rows that the cache has at slots, in order."""
    k, v = model.read(cache, slots, dtype=torch.float32)
    G = model.heads // model.kv_heads
    s = torch.einsum("hd,thd->ht", q.float(), k.repeat_interleave(G, 1)) * model.head_dim ** -0.5
    return torch.einsum("ht,thd->hd", s.softmax(-1), v.repeat_interleave(G, 1))


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--cache", choices=["fp4", "fp8"], default="fp4")
    p.add_argument("--places", type=int, default=4, help="requests served at a time")
    p.add_argument("--requests", type=int, default=9)
    p.add_argument("--prompt", type=int, default=70, help="tokens of the longest prompt")
    p.add_argument("--answer", type=int, default=24, help="tokens of the longest answer")
    p.add_argument("--layers", type=int, default=2)
    args = p.parse_args(argv)
    B, page, vocab = args.places, 16, 64
    longest = -(-(args.prompt + args.answer) // page)
    pages = max(longest, B * longest // 3)
    model = Decoder(args.cache, args.layers, hidden=512, heads=8, kv_heads=2, head_dim=64, vocab=vocab, pages=pages, page_size=page)
    gen = torch.Generator().manual_seed(1)
    waiting = [(torch.randint(vocab, (int(torch.randint(1, args.prompt + 1, (1,), generator=gen)),), generator=gen),
                int(torch.randint(1, args.answer + 1, (1,), generator=gen))) for _ in range(args.requests)]

    table = torch.full((B, longest), -1, dtype=torch.int32, device="cuda")
    ring, state = dg.make_kv_page_pool(pages)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    ones = torch.zeros(B, dtype=torch.int32, device="cuda")            # 1: the place takes a token this step
    token = torch.zeros(B, dtype=torch.int64, device="cuda")
    hidden = torch.zeros(B, 512, dtype=torch.bfloat16, device="cuda")
    trace = []

    def step():
        """One token of every place that has one."""
        trace.clear()
        slots, positions, after, pool = dg.kv_cache_plan(table, lens, ones, (ring, state), page, 1, padded=True)
        served = after - lens
        x = model.forward(token, slots.view(-1), positions.view(-1), lambda q, cache: model.attention(
            q[:, None], cache, table, lens, served)[0][:, 0], trace)
        hidden.copy_(torch.where(served[:, None] > 0, x, hidden))
        lens.copy_(after), state.copy_(pool)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                                                       # nothing in any place
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()

    def int32(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    def resize(add, rows):
        """The plan of a change of lengths by add; what it leaves is the batch's state."""
        slots, positions, after, pool = dg.kv_cache_plan(table, lens, int32(add), (ring, state), page, rows, padded=True)
        before = lens.clone()
        lens.copy_(after), state.copy_(pool)
        return slots.view(-1), positions.view(-1), before, (after - before)

    places, answers, worst, waits = [None] * B, [], 0.0, 0
    while waiting or any(places):
        # the next prompts into the places that are free, as far as the pool has pages
        free = [b for b in range(B) if places[b] is None]
        arrivals = dict(zip(free, waiting))
        if arrivals:
            N = max(len(prompt) for prompt, _ in arrivals.values())
            rows = torch.zeros(B, N, dtype=torch.int64)
            for b, (prompt, _) in arrivals.items():
                rows[b, :len(prompt)] = prompt
            slots, positions, context, served = resize([len(arrivals[b][0]) if b in arrivals else 0 for b in range(B)], N)
            x = model.forward(rows.view(-1).cuda(), slots, positions, lambda q, cache: model.attention(
                q.unflatten(0, (B, N)), cache, table, context, served)[0].flatten(0, 1)).view(B, N, -1)
            got = served.tolist()
            for b, request in arrivals.items():
                if got[b]:                          # the first ones, in order: later prompts wait
                    waiting.pop(0)
                    places[b] = [request[1], 0]
                    hidden[b] = x[b, got[b] - 1]
                else:
                    waits += 1
        # a token for every place that has a request
        ones.copy_(int32([int(place is not None) for place in places]))
        token.copy_((model.norm(hidden).float() @ model.embed.float().t()).argmax(-1))
        before = lens.clone()
        graph.replay()
        torch.cuda.synchronize()
        took = (lens - before).tolist()
        for b in range(B):
            if took[b]:
                at = torch.arange(int(lens[b]), device="cuda")
                own = (table[b].long()[at // page] * page + at % page).int()
                for (q, o), layer in zip(trace, model.layers):
                    want = dense_attention(model, q[b], layer["cache"], own)
                    worst = max(worst, float((o[b].float() - want).abs().max() / want.abs().max()))
                places[b][1] += took[b]
        # requests that are done give their pages back; so do all where none got a page
        leave = [b for b in range(B) if places[b] and (places[b][1] >= places[b][0] or not any(took))]
        if leave:
            counts = lens.tolist()
            resize([-counts[b] if b in leave else 0 for b in range(B)], 0)
            for b in leave:
                answers.append(places[b][1])
                places[b] = None
    lost = pages - len(set(ring.tolist()) & set(range(pages))) if int(state[1]) == pages else pages - int(state[1])
    print(f"{args.requests} requests over {B} places and {pages} pages of {args.cache}, answers of {answers} tokens; {waits} times a prompt waited")
    print(f"attention against fp32 over the cache's rows: {worst:.1e} of the largest value apart; {lost} pages lost")
    # o is rounded to bf16 once, half a step of which is 2^-8 of a value; weights have 11 bits
    if worst > 2.0 ** -8 + 2.0 ** -10 or lost:
        raise SystemExit("further apart than the roundings, or pages are lost")
    return answers, waits


if __name__ == "__main__":
    main()
