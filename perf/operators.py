"""Cases of the few-token operators: the FP8 key/value cache (written, read back), attention for
drafted tokens over that cache, and a mixture-of-experts layer for a few tokens.

Sizes are this repository's own where it has them (32 experts of 4096 x 4096 with six per token and
K = 2048, K = 7168 weights, head dimension 128) and generic otherwise.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
BLOCK = 128
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ---------------------------------------------------------------------------------

def listed():
    return [
        # a decode batch's new tokens: a handful of rows at scattered slots, latency counts
        dict(name="write_decode_5", op="write", T=5, Hkv=8, D=128, page=64, dtype="bf16", spread=True),
        # a prefill chunk written page after page
        dict(name="write_chunk_16384", op="write", T=16384, Hkv=8, D=128, page=64, dtype="bf16", spread=False),
        # a short prefix read back in fp32, some slots already dropped
        dict(name="read_prefix_333", op="read", T=333, Hkv=4, D=64, page=16, dtype="f32", drop=0.1),
        # a long prefix read back for a chunk's attention
        dict(name="read_prefix_40000", op="read", T=40000, Hkv=8, D=128, page=64, dtype="bf16", drop=0.0),
        # one request, one token, a short context: latency counts
        dict(name="attn_decode_1x1000", op="attn", B=1, N=1, ctx=1000, Hkv=8, G=4, D=128, page=64, idle=False),
        # a decode batch
        dict(name="attn_decode_32x8192", op="attn", B=32, N=1, ctx=8192, Hkv=8, G=4, D=128, page=64, idle=False),
        # ragged draft trees over small pages, the last request of the batch idle
        dict(name="attn_tree_7x24", op="attn", B=7, N=24, ctx=3001, Hkv=4, G=8, D=64, page=16, idle=True),
        # long contexts, 128 query rows per key head
        dict(name="attn_tree_2x16_long", op="attn", B=2, N=16, ctx=100001, Hkv=8, G=8, D=128, page=64, idle=False),
        # one token through a small layer: latency counts
        dict(name="moe_1_small", op="moe", T=1, E=8, k=2, H=1024, I=512, drop=0.0, dtype="bf16"),
        # one token through the repository's 32-expert layer
        dict(name="moe_1", op="moe", T=1, E=32, k=6, H=4096, I=2048, drop=0.0, dtype="bf16"),
        # a small draft tree's tokens, a tenth of the slots routed elsewhere
        dict(name="moe_13", op="moe", T=13, E=32, k=6, H=4096, I=2048, drop=0.1, dtype="bf16"),
        # a decode batch that reaches every expert, fp32 output for a later sum
        dict(name="moe_64", op="moe", T=64, E=64, k=8, H=7168, I=2048, drop=0.0, dtype="f32"),
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, even over its logarithm, odd ones among them."""
    n = min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n + 1 if n == 3072 else n


def draw(rng):
    op = rng.choice(["write", "read", "attn", "attn", "moe", "moe"])
    heads, page = rng.choice([1, 2, 4, 8]), rng.choice([16, 32, 64, 128])
    if op == "write":
        return dict(op=op, T=_log(rng, 1, 16384), Hkv=heads, D=rng.choice([64, 128, 256]), page=page,
                    dtype=rng.choice(["bf16", "f32"]), spread=rng.random() < 0.5)
    if op == "read":
        return dict(op=op, T=_log(rng, 1, 40000), Hkv=heads, D=rng.choice([64, 128, 256]), page=page,
                    dtype=rng.choice(["bf16", "f32"]), drop=rng.choice([0.0, 0.1]))
    if op == "attn":
        B, N, G, D = _log(rng, 1, 64), _log(rng, 1, 64), rng.choice([1, 2, 4, 8, 16]), rng.choice([64, 128, 256])
        # the cache is at most the largest listed one's, the scores of the plain form at most 1 GB
        most = min(100001, (1 << 28) // (B * heads * D), (1 << 28) // (B * N * heads * G))
        return dict(op=op, B=B, N=N, ctx=_log(rng, 16, max(17, most)), Hkv=heads, G=G, D=D, page=page,
                    idle=B > 1 and rng.random() < 0.3)
    E = rng.choice([8, 16, 32, 64])
    return dict(op=op, T=_log(rng, 1, 64), E=E, k=rng.choice([1, 2, 4, 6, 8]),
                H=rng.choice([512, 1024, 1536, 2048, 2944, 4096, 7168]),
                I=rng.choice([128, 384, 512, 768, 1024, 1408, 2048]), drop=rng.choice([0.0, 0.1]),
                dtype=rng.choice(["bf16", "f32"]))


# ---- inputs --------------------------------------------------------------------------------

def _quantise_rows(x):
    """[..., D] fp32 -> e4m3 codes as bytes, one fp32 scale a row."""
    s = x.abs().amax(-1) / E4M3_MAX
    s = torch.where(s == 0, torch.ones_like(s), s)
    return (x / s[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8), s


def _quantise_blocks(w):
    """[N, K] fp32 -> e4m3 codes as bytes, one fp32 scale per 128 x 128 block."""
    N, K = w.shape
    b = w.view(N // BLOCK, BLOCK, K // BLOCK, BLOCK)
    s = b.abs().amax((1, 3)) / E4M3_MAX
    q = (b / s[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.view(N, K), s


def _cache(g, pages, heads, page, D):
    shape = (pages, heads, page, D)
    return tuple(_quantise_rows(torch.randn(shape, generator=g, device="cuda")) for _ in range(2))


def _tree_lens(case):
    """Drafted tokens of each request: from N down to half of it, none where the last request is idle."""
    B, N = case["B"], case["N"]
    n = [N - (N // 2) * b // max(1, B - 1) for b in range(B)]
    return n[:-1] + [0] if case["idle"] else n


def _context_lens(case):
    B, ctx = case["B"], case["ctx"]
    n = [ctx - (ctx // 2) * b // max(1, B - 1) for b in range(B)]
    return n[:-1] + [0] if case["idle"] else n


def _tree_masks(rng, lens, N):
    """Bit j of row i: token j is token i or one of its ancestors in a random tree."""
    masks = torch.zeros(len(lens), N, dtype=torch.int64)
    for b, n in enumerate(lens):
        seen = []
        for i in range(n):
            parent = rng.randrange(max(-1, i - 4), i)
            seen.append((1 << i) | (seen[parent] if parent >= 0 else 0))
        for i, bits in enumerate(seen):
            masks[b, i] = bits - (1 << 64) if bits >> 63 else bits
    return masks[:, :, None]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    s = dict(case)
    if case["op"] == "moe":
        T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
        w1 = torch.empty(E, 2 * I, H, dtype=torch.uint8, device="cuda")
        w2 = torch.empty(E, H, I, dtype=torch.uint8, device="cuda")
        s1 = torch.empty(E, 2 * I // BLOCK, H // BLOCK, device="cuda")
        s2 = torch.empty(E, H // BLOCK, I // BLOCK, device="cuda")
        for e in range(E):
            w1[e], s1[e] = _quantise_blocks(torch.randn(2 * I, H, generator=g, device="cuda") / H ** 0.5)
            w2[e], s2[e] = _quantise_blocks(torch.randn(H, I, generator=g, device="cuda") / I ** 0.5)
        logits = torch.randn(T, E, generator=g, device="cuda")
        top, ids = logits.topk(k, dim=1)
        ids = torch.where(torch.rand(T, k, generator=g, device="cuda") < case["drop"], -1, ids)
        s.update(x=torch.randn(T, H, generator=g, device="cuda").bfloat16(), w1=w1, s1=s1, w2=w2, s2=s2,
                 ids=ids.int(), weights=top.softmax(1))
        return s
    heads, D, page = case["Hkv"], case["D"], case["page"]
    if case["op"] == "attn":
        B, N = case["B"], case["N"]
        ctx, lens = _context_lens(case), _tree_lens(case)
        need = [-(-(c + n) // page) for c, n in zip(ctx, lens)]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=g, device="cuda").int().tolist()
        table = torch.zeros(B, -(-(case["ctx"] + N) // page), dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        s.update(cache=_cache(g, pages, heads, page, D), table=table.cuda(),
                 q=2 * torch.randn(B, N, heads * case["G"], D, generator=g, device="cuda").bfloat16(),
                 ctx_lens=torch.tensor(ctx, dtype=torch.int32, device="cuda"),
                 tree_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                 mask=_tree_masks(rng, lens, N).cuda())
        return s
    T = case["T"]
    pages = -(-T // page) + 3
    if case["op"] == "write":
        cache = tuple((torch.zeros(pages, heads, page, D, dtype=torch.uint8, device="cuda"),
                       torch.ones(pages, heads, page, device="cuda")) for _ in range(2))
        # keys and values as a projection leaves them: side by side in one row, no copy
        kv = torch.randn(T, 2 * heads, D, generator=g, device="cuda").to(DTYPES[case["dtype"]])
        s.update(cache=cache, k=kv[:, :heads], v=kv[:, heads:])
    else:
        s.update(cache=_cache(g, pages, heads, page, D))
    if case["op"] == "write" and case["spread"]:
        slots = torch.randperm(pages * page, generator=g, device="cuda")[:T]
    else:
        order = torch.randperm(pages, generator=g, device="cuda")
        slots = (order[:, None] * page + torch.arange(page, device="cuda")).flatten()[5:5 + T]
    if case["op"] == "read":
        slots = torch.where(torch.rand(T, generator=g, device="cuda") < case["drop"], -1, slots)
    s["slots"] = slots.int()
    return s


# ---- the operators -------------------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import fp8_fine_grained_e4m3_amd as dg
    if s["op"] == "write":
        (k, k_sf), (v, v_sf) = dg.fp8_kv_cache_write(s["k"], s["v"], s["cache"], s["slots"])
        return [k.view(torch.float8_e4m3fn), k_sf, v.view(torch.float8_e4m3fn), v_sf]
    if s["op"] == "read":
        return list(dg.fp8_kv_cache_read(s["cache"], s["slots"], dtype=DTYPES[s["dtype"]]))
    if s["op"] == "attn":
        if "workspace" not in s:
            s["workspace"] = dg.make_fp8_tree_attention_workspace(s["q"], s["cache"], s["table"])
        return list(dg.fp8_tree_attention(s["q"], s["cache"], s["table"], s["ctx_lens"], s["tree_lens"], s["mask"],
                                          workspace=s["workspace"]))
    if "workspace" not in s:
        s["workspace"] = dg.make_fp8_moe_few_tokens_workspace(s["x"], (s["w2"], s["s2"]), s["ids"])
    return dg.fp8_moe_few_tokens(s["x"], (s["w1"], s["s1"]), (s["w2"], s["s2"]), s["ids"], s["weights"],
                                 dtype=DTYPES[s["dtype"]], workspace=s["workspace"])


def _run_plain(s):
    return {"write": _plain_write, "read": _plain_read, "attn": _plain_attention, "moe": _plain_moe}[s["op"]](s)


def _values(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _plain_write(s):
    (kc, ks), (vc, vs) = s["cache"]
    slots = s["slots"].long()
    page, at = slots // s["page"], slots % s["page"]
    q, sf = _quantise_rows(torch.stack((s["k"], s["v"])).float())
    kc[page, :, at], vc[page, :, at] = q[0], q[1]
    ks[page, :, at], vs[page, :, at] = sf[0], sf[1]
    return [kc.view(torch.float8_e4m3fn), ks, vc.view(torch.float8_e4m3fn), vs]


def _plain_rows(pool, slots, page, dtype):
    codes, sf = pool
    at = slots.long().clamp(min=0)
    x = _values(codes[at // page, :, at % page]) * sf[at // page, :, at % page][..., None]
    return torch.where((slots >= 0)[:, None, None], x, 0.0).to(dtype)


def _plain_read(s):
    return [_plain_rows(pool, s["slots"], s["page"], DTYPES[s["dtype"]]) for pool in s["cache"]]


def _plain_gather(pool, table):
    """[B, heads, table's tokens, D] fp32 values of the pages of a table."""
    codes, sf = pool
    x = _values(codes[table]) * sf[table][..., None]
    B, P, heads, page, D = x.shape
    return x.transpose(1, 2).reshape(B, heads, P * page, D)


def _plain_attention(s):
    q = s["q"].float()
    B, N, Hq, D = q.shape
    heads = s["Hkv"]
    G, table = Hq // heads, s["table"].long()
    keys, values = (_plain_gather(pool, table) for pool in s["cache"])
    L = keys.shape[2]
    rows = q.view(B, N, heads, G, D).permute(0, 2, 1, 3, 4).reshape(B, heads, N * G, D)
    scores = torch.matmul(rows, keys.transpose(2, 3)).mul_(D ** -0.5).view(B, heads, N, G, L)
    ctx, n = s["ctx_lens"].view(B, 1, 1), s["tree_lens"].view(B, 1, 1)
    at = torch.arange(L, device=q.device).view(1, 1, L) - ctx            # [B, 1, L], tree token number
    bits = (s["mask"] >> at.clamp(0, 63)) & 1                            # [B, N, L]
    seen = (at < 0) | ((bits == 1) & (at >= 0) & (at < n))
    seen = seen & (torch.arange(N, device=q.device).view(1, N, 1) < n)
    scores = scores.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(top.clamp(min=-3e38)).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(B, heads, N * G, L), values).view(B, heads, N, G, D) / total.clamp(min=1e-30)
    out = out.permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D).to(torch.bfloat16)
    lse = (top + total.log())[..., 0].permute(0, 2, 1, 3).reshape(B, N, Hq)
    return [out, lse]


def _plain_weights(codes, sf):
    w = _values(codes)
    n, N, K = w.shape
    w.view(n, N // BLOCK, BLOCK, K // BLOCK, BLOCK).mul_(sf[:, :, None, :, None])
    return w


def _plain_moe(s):
    x, ids, wt = s["x"].float(), s["ids"].long(), s["weights"]
    T, k = ids.shape
    E, I = s["E"], s["I"]
    wt, ids = torch.where(ids >= 0, wt, 0.0), ids.clamp(min=0)
    if T * k < E:      # few slots: each takes its own copy of its expert's weights
        e = ids.flatten()
        h = torch.matmul(_plain_weights(s["w1"][e], s["s1"][e]), x.repeat_interleave(k, 0)[:, :, None])
        h = torch.nn.functional.silu(h[:, :I]) * h[:, I:]
        y = torch.matmul(_plain_weights(s["w2"][e], s["s2"][e]), h).view(T, k, -1)
        y = (y * wt[:, :, None]).sum(1)
    else:              # every token through every expert, weighted by 0 where it was not routed
        h = torch.matmul(_plain_weights(s["w1"], s["s1"]), x.t().contiguous())
        h = torch.nn.functional.silu(h[:, :I]) * h[:, I:]
        each = torch.zeros(T, E, device=x.device).scatter_add_(1, ids, wt)
        y = (torch.matmul(_plain_weights(s["w2"], s["s2"]), h) * each.t()[:, None, :]).sum(0).t().contiguous()
    return y.to(DTYPES[s["dtype"]])


# ---- the definitions in 64 bits --------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"write": _exact_write, "read": _exact_read, "attn": _exact_attention, "moe": _exact_moe}[case["op"]](s)


def _grid():
    """The finite values of e4m3 codes 0..126, in 64 bits."""
    c = torch.arange(127, device="cuda", dtype=torch.float64)
    e, m = (c / 8).floor(), c % 8
    return torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.pow(2.0, e - 7))


def _exact_codes(y):
    """The e4m3 value nearest to each y, the even code of two that are as near."""
    grid = _grid()
    a = y.abs().clamp(max=E4M3_MAX)
    hi = torch.searchsorted(grid, a).clamp(1, 126)
    lo = hi - 1
    up, down = grid[hi] - a, a - grid[lo]
    pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.copysign(grid[pick], y)


def _exact_write(s):
    out, slots = [], s["slots"].long().tolist()
    place = torch.tensor([(t // s["page"], t % s["page"]) for t in slots], device="cuda")
    for x, (codes, sf) in zip((s["k"], s["v"]), s["cache"]):
        x = x.double()
        scale = (x.abs().max(-1).values / E4M3_MAX)
        scale[scale == 0] = 1
        pool, scales = torch.zeros(codes.shape, device="cuda", dtype=torch.float64), sf.double()
        # the quotient is by the stored scale, a number of 32 bits
        pool[place[:, 0], :, place[:, 1]] = _exact_codes(x / scale.float().double()[..., None])
        scales[place[:, 0], :, place[:, 1]] = scale
        out += [pool, scales]
    return out


def _signed(codes):
    grid = _grid()
    return torch.where(codes >= 128, -1.0, 1.0).double() * grid[(codes & 127).long()]


def _exact_read(s):
    out, page = [], s["page"]
    slots = s["slots"].long()
    live = torch.nonzero(slots >= 0).flatten()
    at = slots[live]
    for codes, sf in s["cache"]:
        x = torch.zeros(len(slots), s["Hkv"], s["D"], device="cuda", dtype=torch.float64)
        x[live] = _signed(codes[at // page, :, at % page]) * sf[at // page, :, at % page].double()[..., None]
        out.append(x)
    return out


def _exact_attention(s):
    B, N, Hq, D = s["q"].shape
    heads, page = s["Hkv"], s["page"]
    G = Hq // heads
    o = torch.zeros(B, N, Hq, D, device="cuda", dtype=torch.float64)
    lse = torch.full((B, N, Hq), -math.inf, device="cuda", dtype=torch.float64)
    for b in range(B):
        c, n = int(s["ctx_lens"][b]), int(s["tree_lens"][b])
        if n == 0:
            continue
        t = torch.arange(c + n, device="cuda")
        pg, off = s["table"][b].long()[t // page], t % page
        tree = torch.tensor([[(int(s["mask"][b, i, 0]) >> j) & 1 for j in range(n)] for i in range(n)],
                            device="cuda", dtype=torch.bool).view(n, n)
        for h in range(heads):
            (kc, ks), (vc, vs) = s["cache"]
            key = _signed(kc[pg, h, off]) * ks[pg, h, off].double()[:, None]
            val = _signed(vc[pg, h, off]) * vs[pg, h, off].double()[:, None]
            for i in range(G):
                S = s["q"][b, :n, h * G + i].double() @ key.t() / math.sqrt(D)
                S[:, c:][~tree] = -math.inf
                l = torch.logsumexp(S, 1)
                lse[b, :n, h * G + i] = l
                o[b, :n, h * G + i] = torch.exp(S - l[:, None]) @ val
    return [o, lse]


def _exact_moe(s):
    T, k = s["ids"].shape
    y = torch.zeros(T, s["H"], device="cuda", dtype=torch.float64)
    x, ids = s["x"].double(), s["ids"]
    for e in range(s["E"]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if len(t) == 0:
            continue
        w1, w2 = ((_signed(s[w][e]).unflatten(1, (-1, BLOCK)).unflatten(0, (-1, BLOCK))
                   * s[f][e].double()[:, None, :, None]).flatten(2, 3).flatten(0, 1)
                  for w, f in (("w1", "s1"), ("w2", "s2")))
        gate, up = (x[t] @ w1.t()).chunk(2, 1)
        h = gate / (1 + torch.exp(-gate)) * up
        y.index_add_(0, t, (h @ w2.t()) * s["weights"][t, j].double()[:, None])
    return y


# ---- what a pass cannot do without -------------------------------------------------------------

def work(case):
    size = {"bf16": 2, "f32": 4}
    if case["op"] in ("write", "read"):
        rows = 2 * case["T"] * case["Hkv"]
        return {"bytes": rows * (case["D"] * (size[case["dtype"]] + 1) + 4) + 4 * case["T"], "flops": 2 * rows * case["D"]}
    if case["op"] == "attn":
        heads, D, Hq = case["Hkv"], case["D"], case["Hkv"] * case["G"]
        ctx, lens = _context_lens(case), _tree_lens(case)
        tokens = sum(c + n for c, n in zip(ctx, lens) if n)
        q = case["B"] * case["N"] * Hq
        return {"bytes": tokens * heads * (2 * D + 8) + q * (4 * D + 4) + 8 * case["B"] * case["N"] + 4 * tokens // case["page"],
                "flops": 4 * Hq * D * sum(n * (c + n) for c, n in zip(ctx, lens))}
    T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
    live = k * (1 - case["drop"])
    experts = E * (1 - (1 - live / E) ** T)      # expected, each token's experts drawn alike
    return {"bytes": experts * 3 * H * I * (1 + 4 / BLOCK ** 2) + T * (H * (2 + size[case["dtype"]]) + 8 * k),
            "flops": 6 * T * live * H * I}
