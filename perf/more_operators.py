"""Cases of the operators around a paged cache: pages and slots from request lengths, norms of queries
and keys with the position rotation (forward and backward), the FP4 key/value cache (written and read
back) and attention for drafted tokens over it.

Sizes are this repository's own where it has them (32 query and 8 key heads of 128, pages of 64,
chunks of 16384 tokens) and generic otherwise.
"""
import math
import random

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK = 32
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
BASE = 10000.0


# ---- cases ---------------------------------------------------------------------------------

def listed():
    return [
        # a decode step of a small batch, a row a request: latency counts
        dict(name="plan_decode_7", op="plan", B=7, N=1, rows=0, ctx=3001, page=16, short=False),
        # ragged prompts of a large batch, packed, beside requests that end or lose drafts
        dict(name="plan_prefill_256", op="plan", B=256, N=0, rows=131072, ctx=1000, page=16, short=False),
        # a decode batch's new tokens at far positions: latency counts
        dict(name="rope_decode_5", op="rope", T=5, Hq=32, H=8, D=128, R=128, dtype="bf16", pairs=False, far=1000000),
        # a prefill chunk
        dict(name="rope_chunk_16384", op="rope", T=16384, Hq=32, H=8, D=128, R=128, dtype="bf16", pairs=False, far=40000),
        # the gradients of a short fp32 batch, neighbours rotated, half of each head
        dict(name="rope_grad_333", op="rope_grad", T=333, Hq=16, H=2, D=64, R=32, dtype="f32", pairs=True, far=5000),
        # the gradients of a training batch
        dict(name="rope_grad_16384", op="rope_grad", T=16384, Hq=32, H=8, D=128, R=128, dtype="bf16", pairs=False, far=8192),
        # a decode batch's new tokens stored, and read as attention will see them: latency counts
        dict(name="fp4_store_5", op="store", T=5, H=8, D=128, page=64, dtype="bf16", drop=0.0),
        # a prefill chunk stored and read back, some tokens not stored
        dict(name="fp4_store_16384", op="store", T=16384, H=8, D=128, page=64, dtype="bf16", drop=0.1),
        # one request, one token, a short context: latency counts
        dict(name="fp4_decode_1x1000", op="attn", B=1, N=1, ctx=1000, H=8, G=4, D=128, page=64, idle=False),
        # a decode batch
        dict(name="fp4_decode_32x8192", op="attn", B=32, N=1, ctx=8192, H=8, G=4, D=128, page=64, idle=False),
        # ragged draft trees over small pages, the last request of the batch idle
        dict(name="fp4_tree_7x24", op="attn", B=7, N=24, ctx=3001, H=4, G=8, D=64, page=16, idle=True),
        # long contexts, 128 query rows per key head
        dict(name="fp4_tree_2x16_long", op="attn", B=2, N=16, ctx=100001, H=8, G=8, D=128, page=64, idle=False),
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, even over its logarithm, odd ones among them."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "rope", "rope_grad", "store", "attn", "attn"])
    page, heads, D = rng.choice([16, 32, 64, 128]), rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256])
    if op == "plan":
        B, ctx, short = _log(rng, 1, 256), _log(rng, 16, 4000), rng.random() < 0.25
        if rng.random() < 0.5:
            return dict(op=op, B=B, N=_log(rng, 1, 64), rows=0, ctx=ctx, page=page, short=short)
        return dict(op=op, B=B, N=0, rows=_log(rng, B, 131072), ctx=ctx, page=page, short=short)
    if op in ("rope", "rope_grad"):
        Hq, dtype = heads * rng.choice([1, 2, 4, 8]), rng.choice(["bf16", "f32"])
        # no more bytes than the listed chunk has
        most = 16384 * 40 * 128 * 2 // ((Hq + heads) * D * (4 if dtype == "f32" else 2))
        return dict(op=op, T=_log(rng, 1, min(16384, most)), Hq=Hq, H=heads, D=D, R=rng.choice([D, D, D // 2, D // 4]),
                    dtype=dtype, pairs=rng.random() < 0.4, far=_log(rng, 100, 1000000))
    if op == "store":
        dtype = rng.choice(["bf16", "f32"])
        most = 16384 * 8 * 128 * 2 // (heads * D * (4 if dtype == "f32" else 2))
        return dict(op=op, T=_log(rng, 1, min(16384, most)), H=heads, D=D, page=page, dtype=dtype,
                    drop=rng.choice([0.0, 0.1]))
    B, N, G = _log(rng, 1, 64), _log(rng, 1, 64), rng.choice([1, 2, 4, 8, 16])
    # the cache is at most the largest listed one's, the scores of the plain form at most 1 GB
    most = min(100001, (1 << 28) // (B * heads * D), (1 << 28) // (B * N * heads * G))
    return dict(op=op, B=B, N=N, ctx=_log(rng, 16, max(17, most)), H=heads, G=G, D=D, page=page,
                idle=B > 1 and rng.random() < 0.3)


# ---- inputs --------------------------------------------------------------------------------

def _round_fp4(a):
    """Codes 0..7 of the e2m1 values nearest to a >= 0, the even code of two that are as near."""
    code = torch.zeros_like(a, dtype=torch.uint8)
    for i in range(7):
        middle = (E2M1[i] + E2M1[i + 1]) / 2
        code += (a > middle) if i % 2 == 0 else (a >= middle)
    return code


def _quantise(x):
    """[..., D] fp32 -> two e2m1 codes a byte (the even value in the low half), an exponent byte a block.
    The scale is the least power of two, from 2^-125 to 2^125, that brings the block's largest value to
    6 at most; 1 for zeros."""
    b = x.unflatten(-1, (-1, BLOCK))
    mantissa, exponent = torch.frexp(b.abs().amax(-1))        # m 2^e with m in [0.5, 1)
    e = (exponent - 3 + (mantissa > 0.75)).clamp(-125, 125)
    e = torch.where(mantissa == 0, 0, e)
    # two factors, each a number of 32 bits
    y = torch.ldexp(torch.ldexp(b, -(e // 2)[..., None]), -(e - e // 2)[..., None])
    code = (_round_fp4(y.abs()) | (torch.signbit(y).to(torch.uint8) << 3)).flatten(-2)
    return code[..., ::2] | (code[..., 1::2] << 4), (e + 127).to(torch.uint8)


def _cache(g, pages, heads, page, D):
    return tuple(_quantise(torch.randn(pages, heads, page, D, generator=g, device="cuda")) for _ in range(2))


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


def _prepare_plan(case, rng, s):
    B, N, rows, page = (case[n] for n in ("B", "N", "rows", "page"))
    # shares of the packed rows, ragged; of a padded batch up to N a request
    weights = [rng.uniform(0.2, 2.0) for _ in range(B)]
    ctx, add = [], []
    for b in range(B):
        what = rng.random()
        ctx.append(rng.randint(case["ctx"] // 2, case["ctx"]))
        if what < 0.08:
            add.append(-ctx[b])                                   # done: all of it goes back
        elif what < 0.16:
            add.append(-rng.randint(1, min(24, ctx[b])))          # rejected drafts
        elif N:
            add.append(rng.randint((N + 1) // 2, N))
        else:
            add.append(int(0.9 * rows * weights[b] / sum(weights)))
            ctx[b] = ctx[b] if rng.random() < 0.5 else 0          # a new request
    held = [-(-c // page) for c in ctx]
    need = [-(-(c + max(a, 0)) // page) for c, a in zip(ctx, add)]
    # sizes by the case alone: the most that a request and all of them may have
    most = N or int(0.9 * rows * 2.0 / (0.2 * (B - 1) + 2.0)) + 1
    width = (case["ctx"] + most) // page + 2
    pages = B * (case["ctx"] // page + 2) + (B * N + rows) // page + 40
    order = list(range(pages))
    rng.shuffle(order)
    table, at = torch.full((B, width), -1, dtype=torch.int32), 0
    for b, n in enumerate(held):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    # other requests hold the rest of a short pool, which then has enough for the first ones only
    free, head = order[at:], rng.randrange(pages)
    if case["short"]:
        free = free[:(sum(need) - sum(held)) * 2 // 3]
    ring = torch.full((pages,), -1, dtype=torch.int32)
    ring[(head + torch.arange(len(free))) % pages] = torch.tensor(free, dtype=torch.int32)
    s.update(table=table.cuda(), ring=ring.cuda(), pages=pages,
             context_lens=torch.tensor(ctx, dtype=torch.int32, device="cuda"),
             add_lens=torch.tensor(add, dtype=torch.int32, device="cuda"),
             state=torch.tensor([head, len(free)], dtype=torch.int32, device="cuda"))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    s = dict(case)
    if case["op"] == "plan":
        _prepare_plan(case, rng, s)
        return s
    if case["op"] in ("rope", "rope_grad"):
        T, Hq, H, D = (case[n] for n in ("T", "Hq", "H", "D"))
        dtype = DTYPES[case["dtype"]]
        # queries, keys and values as a projection leaves them: side by side in one row
        qkv = (torch.randn(T, Hq + 2 * H, D, generator=g, device="cuda") * 1.5).to(dtype)
        first = torch.randint(0, case["far"], (1,), generator=g, device="cuda")
        s.update(q=qkv[:, :Hq], k=qkv[:, Hq:Hq + H],
                 wq=(1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dtype),
                 wk=(1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dtype),
                 positions=(first + torch.arange(T, device="cuda")).int(),
                 inv_freq=(BASE ** (-2.0 * torch.arange(case["R"] // 2, dtype=torch.float64) / case["R"])).float().cuda())
        if case["op"] == "rope_grad":
            s.update(dq=torch.randn(T, Hq, D, generator=g, device="cuda").to(dtype),
                     dk=torch.randn(T, H, D, generator=g, device="cuda").to(dtype))
        return s
    H, D, page = case["H"], case["D"], case["page"]
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
        s.update(cache=_cache(g, pages, H, page, D), table=table.cuda(),
                 q=2 * torch.randn(B, N, H * case["G"], D, generator=g, device="cuda").bfloat16(),
                 ctx_lens=torch.tensor(ctx, dtype=torch.int32, device="cuda"),
                 tree_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                 mask=_tree_masks(rng, lens, N).cuda())
        return s
    T = case["T"]
    pages = -(-T // page) + 3
    cache = tuple((torch.zeros(pages, H, page, D // 2, dtype=torch.uint8, device="cuda"),
                   torch.full((pages, H, page, D // BLOCK), 127, dtype=torch.uint8, device="cuda")) for _ in range(2))
    kv = torch.randn(T, 2 * H, D, generator=g, device="cuda")
    kv *= torch.exp(torch.randn(1, 2 * H, D, generator=g, device="cuda"))        # channels of different sizes
    kv = kv.to(DTYPES[case["dtype"]])
    order = torch.randperm(pages, generator=g, device="cuda")
    slots = (order[:, None] * page + torch.arange(page, device="cuda")).flatten()[5:5 + T]
    slots = torch.where(torch.rand(T, generator=g, device="cuda") < case["drop"], -1, slots)
    s.update(cache=cache, k=kv[:, :H], v=kv[:, H:], slots=slots.int())
    return s


# ---- the operators -------------------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import fp8_fine_grained_e4m3_amd as dg
    if s["op"] == "plan":
        slots, positions, lens, state = dg.kv_cache_plan(s["table"], s["context_lens"], s["add_lens"], (s["ring"], s["state"]),
                                                         s["page"], s["N"] or s["rows"], padded=s["N"] > 0)
        return [s["table"], slots, positions, lens, s["ring"], state]
    if s["op"] == "rope":
        return list(dg.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["positions"], s["inv_freq"], eps=EPS,
                                    interleaved=s["pairs"]))
    if s["op"] == "rope_grad":
        if "workspace" not in s:
            s["workspace"] = dg.make_qk_norm_rope_backward_workspace(s["q"], s["k"])
        return list(dg.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"], s["positions"],
                                             s["inv_freq"], eps=EPS, interleaved=s["pairs"], workspace=s["workspace"]))
    if s["op"] == "store":
        dg.fp4_kv_cache_write(s["k"], s["v"], s["cache"], s["slots"])
        return list(dg.fp4_kv_cache_read(s["cache"], s["slots"], dtype=DTYPES[s["dtype"]]))
    if "workspace" not in s:
        s["workspace"] = dg.make_fp4_tree_attention_workspace(s["q"], s["cache"], s["table"])
    return list(dg.fp4_tree_attention(s["q"], s["cache"], s["table"], s["ctx_lens"], s["tree_lens"], s["mask"],
                                      workspace=s["workspace"]))


def _run_plain(s):
    return {"plan": _plain_plan, "rope": _plain_rope, "rope_grad": _plain_rope_grad, "store": _plain_store,
            "attn": _plain_attention}[s["op"]](s)


def _plain_plan(s):
    table, ring, page, P = s["table"], s["ring"], s["page"], s["pages"]
    ctx, add = s["context_lens"].long(), s["add_lens"].long()
    head, count = s["state"][0].long(), s["state"][1].long()
    held, after = (ctx + page - 1) // page, ((ctx + add).clamp(min=0) + page - 1) // page
    take, give = (after - held).clamp(min=0), (held - after).clamp(min=0)
    taken, given = take.cumsum(0), give.cumsum(0)
    served = (take == 0) | (taken <= count)
    lens = torch.where(served, (ctx + add).clamp(min=0), ctx)
    column = torch.arange(table.shape[1], device=table.device)
    new = (column >= held[:, None]) & (column < after[:, None]) & served[:, None]
    pick = (taken - take)[:, None] + column - held[:, None]
    back = (column >= after[:, None]) & (column < held[:, None])
    put = (given - give)[:, None] + column - after[:, None]
    filled = torch.where(new, ring[(head + pick.clamp(min=0)) % P], table)
    # pages that go back, the others to a place behind the ring
    longer = torch.cat([ring, ring[:1]])
    longer.scatter_(0, torch.where(back, (head + count + put) % P, P).flatten(), table.flatten())
    table.copy_(filled)
    ring.copy_(longer[:P])
    last = torch.where(take > 0, torch.where(taken <= count, taken, 0), 0).amax()
    state = torch.stack([(head + last) % P, count - last + given[-1]]).int()
    rows = add.clamp(min=0)
    if s["N"]:
        at = torch.arange(s["N"], device=table.device).expand(s["B"], -1)
        b = torch.arange(s["B"], device=table.device)[:, None].expand(-1, s["N"])
        live = at < rows[:, None]
    else:
        r = torch.arange(s["rows"], device=table.device)
        upto = rows.cumsum(0)
        b = torch.searchsorted(upto, r, right=True).clamp(max=s["B"] - 1)
        at = r - (upto - rows)[b]
        live = r < upto[-1]
    position = torch.where(live, ctx[b] + at, 0)
    slots = table[b, position // page] * page + position % page
    return [table, torch.where(live & served[b], slots, -1).int(), position.int(), lens.int(), ring, state]


def _angles(s):
    """cos and sin [T, 1, R / 2] of the angles, taken in 64 bits."""
    a = s["positions"].double()[:, None] * s["inv_freq"].double()
    return a.cos().float()[:, None], a.sin().float()[:, None]


def _rotate(x, cos, sin, pairs):
    """The first R values of each row rotated; pairs: neighbours, else a value with the one R / 2 on."""
    R = 2 * cos.shape[-1]
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if pairs else (x[..., :R // 2], x[..., R // 2:R])
    c, d = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([c, d], -1).flatten(-2) if pairs else torch.cat([c, d], -1)
    return torch.cat([turned, x[..., R:]], -1)


def _plain_rope(s):
    cos, sin = _angles(s)
    out = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        x32 = x.float()
        y = x32 * torch.rsqrt(x32.square().mean(-1, keepdim=True) + EPS) * w.float()
        out.append(_rotate(y, cos, sin, s["pairs"]).to(x.dtype))
    return out


def _plain_rope_grad(s):
    cos, sin = _angles(s)
    rows, weights = [], []
    for dz, x, w in ((s["dq"], s["q"], s["wq"]), (s["dk"], s["k"], s["wk"])):
        x32 = x.float()
        r = torch.rsqrt(x32.square().mean(-1, keepdim=True) + EPS)
        dy = _rotate(dz.float(), cos, -sin, s["pairs"])
        n = x32 * r
        weights.append((dy * n).sum((0, 1)))
        dn = dy * w.float()
        rows.append((r * (dn - n * (dn * n).mean(-1, keepdim=True))).to(x.dtype))
    return rows + weights


def _values(codes, sf):
    """[..., D / 2] codes, [..., D / 32] exponents -> [..., D] fp32."""
    one = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    both = torch.stack([one.repeat(16), one.repeat_interleave(16)], -1)          # of a byte
    x = both[codes.int()].flatten(-2)
    return (x.unflatten(-1, (-1, BLOCK)) * torch.exp2(sf.float() - 127)[..., None]).flatten(-2)


def _plain_store(s):
    slots, page, out = s["slots"].long(), s["page"], []
    live = slots >= 0
    at = slots.clamp(min=0)
    for x, (codes, sf) in zip((s["k"], s["v"]), s["cache"]):
        c, e = _quantise(x.float())
        # tokens that are not stored go to a page of their own behind the others
        where = torch.where(live, at // page, codes.shape[0])
        for pool, new in ((codes, c), (sf, e)):
            longer = torch.cat([pool, pool[:1]])
            longer[where, :, at % page] = new
            pool.copy_(longer[:-1])
        rows = _values(codes[at // page, :, at % page], sf[at // page, :, at % page])
        out.append(torch.where(live[:, None, None], rows, 0.0).to(x.dtype))
    return out


def _plain_gather(pool, table):
    """[B, heads, table's tokens, D] fp32 values of the pages of a table."""
    x = _values(pool[0][table], pool[1][table])
    B, P, heads, page, D = x.shape
    return x.transpose(1, 2).reshape(B, heads, P * page, D)


def _plain_attention(s):
    q = s["q"].float()
    B, N, Hq, D = q.shape
    heads = s["H"]
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


# ---- the definitions in 64 bits --------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "rope": _exact_rope, "rope_grad": _exact_rope_grad, "store": _exact_store,
            "attn": _exact_attention}[case["op"]](s)


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _exact_plan(s):
    table, ring = s["table"].tolist(), s["ring"].tolist()
    page, P, (head, free) = s["page"], s["pages"], s["state"].tolist()
    ctx, add = s["context_lens"].tolist(), s["add_lens"].tolist()
    tail, wanted, taken, back, lens, rows = head + free, 0, 0, [], [], []
    for b, (c, a) in enumerate(zip(ctx, add)):
        held, after = -(-c // page), -(-max(c + a, 0) // page)
        wanted += max(after - held, 0)
        served = after <= held or wanted <= free
        if served:
            for j in range(held, after):
                table[b][j] = ring[(head + taken) % P]
                taken += 1
        back += table[b][after:held]
        lens.append(max(c + a, 0) if served else c)
        tokens = [(table[b][p // page] * page + p % page if served else -1, p) for p in range(c, c + max(a, 0))]
        rows += tokens + [(-1, 0)] * (s["N"] - len(tokens)) if s["N"] else tokens
    for i, p in enumerate(back):
        ring[(tail + i) % P] = p
    if not s["N"]:
        rows = rows[:s["rows"]] + [(-1, 0)] * (s["rows"] - len(rows))
    slots, positions = (_int32(x) for x in zip(*rows))
    if s["N"]:
        slots, positions = slots.view(s["B"], s["N"]), positions.view(s["B"], s["N"])
    return [_int32(table), slots, positions, _int32(lens), _int32(ring), _int32([(head + taken) % P, free - taken + len(back)])]


def _turns(s, D):
    """Each place's partner, and cosines and signed sines [T, 1, D]: z = y cos + y[partner] sin."""
    R = s["R"]
    partner, freq, sign = list(range(D)), [0.0] * D, [0.0] * D
    f = s["inv_freq"].double().tolist()
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if s["pairs"] else (i, i + R // 2)
        partner[a], partner[b], freq[a], freq[b], sign[a], sign[b] = b, a, f[i], f[i], -1.0, 1.0
    angle = s["positions"].double()[:, None] * torch.tensor(freq, dtype=torch.float64, device="cuda")
    sign = torch.tensor(sign, dtype=torch.float64, device="cuda")
    return partner, torch.cos(angle)[:, None], (torch.sin(angle) * sign)[:, None]


def _exact_rope(s):
    partner, cos, sin = _turns(s, s["D"])
    out = []
    for x, w in ((s["q"].double(), s["wq"].double()), (s["k"].double(), s["wk"].double())):
        y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / s["D"] + EPS) * w
        out.append(y * cos + y[..., partner] * sin)
    return out


def _exact_rope_grad(s):
    partner, cos, sin = _turns(s, s["D"])
    rows, weights = [], []
    for dz, x, w in ((s["dq"].double(), s["q"].double(), s["wq"].double()), (s["dk"].double(), s["k"].double(), s["wk"].double())):
        size = torch.sqrt((x * x).sum(-1, keepdim=True) / s["D"] + EPS)
        dy = dz * cos + (dz * sin)[..., partner]
        weights.append((dy * x / size).sum(1).sum(0))
        g = dy * w
        rows.append(g / size - x * (g * x).sum(-1, keepdim=True) / (s["D"] * size ** 3))
    return rows + weights


def _exact_store(s):
    grid, out = torch.tensor(E2M1, dtype=torch.float64, device="cuda"), []
    for x in (s["k"], s["v"]):
        b = x.double().unflatten(-1, (-1, BLOCK))
        most = b.abs().amax(-1, keepdim=True)
        scale = torch.exp2(torch.ceil(torch.log2(torch.where(most == 0, 6.0, most) / 6)))
        scale = torch.where(most > 6 * scale, 2 * scale, torch.where(most <= 3 * scale, scale / 2, scale))
        y = (b / torch.where(most == 0, 1.0, scale)).abs()
        hi = torch.searchsorted(grid, y.contiguous()).clamp(1, 7)
        up, down = grid[hi] - y, y - grid[hi - 1]
        near = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)
        rows = (torch.copysign(grid[near], b) * scale).flatten(-2)
        out.append(torch.where((s["slots"] >= 0)[:, None, None], rows, 0.0))
    return out


def _signed(codes, sf):
    grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    each = torch.stack([codes % 16, codes // 16], -1).flatten(-2)
    x = torch.where(each >= 8, -1.0, 1.0).double() * grid[(each % 8).long()]
    return x * torch.pow(2.0, sf.double() - 127).repeat_interleave(BLOCK, -1)


def _exact_attention(s):
    B, N, Hq, D = s["q"].shape
    heads, page = s["H"], s["page"]
    G = Hq // heads
    o = torch.zeros(B, N, Hq, D, device="cuda", dtype=torch.float64)
    lse = torch.full((B, N, Hq), -math.inf, device="cuda", dtype=torch.float64)
    for b in range(B):
        c, n = int(s["ctx_lens"][b]), int(s["tree_lens"][b])
        if n == 0:
            continue
        t = torch.arange(c + n, device="cuda")
        pg, off = s["table"][b].long()[t // page], t % page
        words = s["mask"][b, :, 0].tolist()
        tree = torch.tensor([[(words[i] >> j) & 1 for j in range(n)] for i in range(n)],
                            device="cuda", dtype=torch.bool).view(n, n)
        for h in range(heads):
            key, val = (_signed(codes[pg, h, off], sf[pg, h, off]) for codes, sf in s["cache"])
            for i in range(G):
                S = s["q"][b, :n, h * G + i].double() @ key.t() / math.sqrt(D)
                S[:, c:][~tree] = -math.inf
                l = torch.logsumexp(S, 1)
                lse[b, :n, h * G + i] = l
                o[b, :n, h * G + i] = torch.exp(S - l[:, None]) @ val
    return [o, lse]


# ---- what a pass cannot do without -------------------------------------------------------------

def work(case):
    size = {"bf16": 2, "f32": 4}
    if case["op"] == "plan":
        # lengths read and written; slots and positions; a page entry read and written for each page
        rows = case["rows"] or case["B"] * case["N"]
        return {"bytes": 12 * case["B"] + 8 * rows + 8 * -(-rows // case["page"]) + 16, "flops": 4 * rows}
    if case["op"] in ("rope", "rope_grad"):
        values = case["T"] * (case["Hq"] + case["H"]) * case["D"]
        if case["op"] == "rope":
            return {"bytes": 2 * values * size[case["dtype"]] + 4 * case["T"], "flops": 7 * values}
        return {"bytes": 3 * values * size[case["dtype"]] + 4 * case["T"] + 12 * case["D"], "flops": 14 * values}
    if case["op"] == "store":
        rows, D = 2 * case["T"] * case["H"], case["D"]
        live = rows * (1 - case["drop"])
        # rows read, codes written, codes read, rows written
        return {"bytes": rows * D * size[case["dtype"]] + live * D * size[case["dtype"]] + 2 * live * (D // 2 + D // BLOCK),
                "flops": 4 * rows * D}
    heads, D, Hq = case["H"], case["D"], case["H"] * case["G"]
    ctx, lens = _context_lens(case), _tree_lens(case)
    tokens = sum(c + n for c, n in zip(ctx, lens) if n)
    q = case["B"] * case["N"] * Hq
    return {"bytes": tokens * heads * 2 * (D // 2 + D // BLOCK) + q * (4 * D + 4) + 8 * case["B"] * case["N"]
            + 4 * tokens // case["page"],
            "flops": 4 * Hq * D * sum(n * (c + n) for c, n in zip(ctx, lens))}
