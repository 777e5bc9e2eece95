"""Measured cases of the serving operators around the verify step.

One target-model layer of a speculative decoding step does, before the verify
call: rotary positions for the new tokens' queries and keys and the write of
keys and values into the paged cache (``rope``), attention of the new tokens
over that cache (``attention``); and after it: the attention weight that each
cached key received from the accepted tokens, added up (``mass``), and the
eviction of the keys with the least of it (``evict``).

``listed()`` and ``draw(rng)`` give the cases, ``prepare`` the inputs, ``run``
one pass -- the plain form in elementary torch operations, or, with ``own``
set, the library's calls -- and ``exact`` the result in 64 bits.
"""
import math

import torch

own = False

GOLDEN = 0.6180339887498949
PAGE_SLACK = 3  # pages of the pool that belong to no sequence

TREES = {  # children per node, level by level
    "k21": (4, 2, 1),
    "w4": (4, 1, 1, 1),
    "b63": (2, 2, 2, 2, 2),
}
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f16": 2, "e4m3": 1}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one conversation, one token: the latency of a layer's write to the cache
        dict(name="rope_one_token", op="rope", B=1, T=1, Hq=32, Hkv=8, D=128, rotary=128, layout="half", scaling="none",
             ctx=777, page=16, order="nhd", dtype="bf16", kv="bf16", ragged=False),
        # a verify step of a serving batch: gamma = 4 drafted tokens and the last one, far positions, 8-bit cache
        dict(name="rope_verify_e4m3", op="rope", B=64, T=5, Hq=64, Hkv=8, D=128, rotary=128, layout="half",
             scaling="by_parts", ctx=1500, page=16, order="nhd", dtype="bf16", kv="e4m3", ragged=True),
        # prompts entering the cache, interleaved pairs on half of each head
        dict(name="rope_prompt", op="rope", B=8, T=2011, Hq=32, Hkv=8, D=128, rotary=64, layout="interleaved",
             scaling="linear", ctx=0, page=32, order="hnd", dtype="f16", kv="f16", ragged=True),
        # one conversation, one token: latency
        dict(name="attn_one_token", op="attention", B=1, T=1, Hq=32, Hkv=8, D=128, ctx=777, page=16, order="nhd",
             dtype="bf16", kv="bf16", tree="", ragged=False, lse=False),
        # plain decoding of a full batch, one new token each
        dict(name="attn_decode_batch", op="attention", B=64, T=1, Hq=32, Hkv=8, D=128, ctx=8191, page=16, order="nhd",
             dtype="bf16", kv="bf16", tree="", ragged=True, lse=False),
        # the verify step of the headline batch: gamma = 4, 64 query heads on 8 key heads, lse kept for the eviction
        dict(name="attn_verify_batch", op="attention", B=64, T=5, Hq=64, Hkv=8, D=128, ctx=8191, page=16, order="nhd",
             dtype="bf16", kv="bf16", tree="", ragged=True, lse=True),
        # the 21-node draft tree on a batch of 32
        dict(name="attn_tree_batch", op="attention", B=32, T=21, Hq=32, Hkv=8, D=128, ctx=4099, page=32, order="hnd",
             dtype="f16", kv="f16", tree="k21", ragged=True, lse=True),
        # two long documents, 8-bit cache, gamma = 7
        dict(name="attn_long_e4m3", op="attention", B=2, T=8, Hq=32, Hkv=8, D=128, ctx=131001, page=64, order="nhd",
             dtype="bf16", kv="e4m3", tree="", ragged=False, lse=False),
        # a small draft model's heads, one key head for each query head
        dict(name="attn_heads_64", op="attention", B=16, T=2, Hq=16, Hkv=16, D=64, ctx=2050, page=16, order="nhd",
             dtype="f16", kv="f16", tree="", ragged=True, lse=False),
        # the weight of every cached key after a verify step
        dict(name="mass_verify_batch", op="mass", B=64, T=5, Hq=64, Hkv=8, D=128, ctx=8191, page=16, order="nhd",
             dtype="bf16", kv="bf16", tree="", ragged=True),
        # after every step of one sequence: few keys leave
        dict(name="evict_step", op="evict", B=4, Hkv=8, D=128, ctx=2117, budget=2048, sinks=4, recent=256, page=16,
             order="nhd", kv="bf16", ragged=False),
        # a batch cut back to half
        dict(name="evict_half_batch", op="evict", B=32, Hkv=8, D=128, ctx=8191, budget=4096, sinks=4, recent=512, page=16,
             order="nhd", kv="bf16", ragged=False),
    ]


MOST_KV = 1.3e9      # bytes of the caches that the largest listed case reads
MOST_SCORES = 8e8    # scores of its plain form


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "attention", "attention", "mass", "evict"])
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    page = rng.choice([8, 16, 32, 64, 128])
    order = rng.choice(["nhd", "hnd"])
    dtype = rng.choice(["bf16", "f16"])
    kv = rng.choice([dtype, dtype, "e4m3"])
    if op == "rope":
        B, T = _log(rng, 1, 128), rng.choice([1, rng.randint(2, 33), _log(rng, 34, 4000)])
        while B * T * (G + 2) * Hkv * D > 8e7:
            B, T = max(1, B // 2), max(1, T * 3 // 4)
        return dict(op=op, B=B, T=T, Hq=G * Hkv, Hkv=Hkv, D=D, rotary=rng.choice([D, D, D // 2, D // 2 - 8]),
                    layout=rng.choice(["half", "interleaved"]), scaling=rng.choice(["none", "linear", "base", "by_parts"]),
                    ctx=_log(rng, 1, 2000), page=page, order=order, dtype=dtype, kv=kv, ragged=rng.random() < 0.5)
    if op == "evict":
        B, ctx = _log(rng, 1, 64), _log(rng, 40, 32000)
        while B * ctx * Hkv * D * 4.0 > MOST_KV:
            B, ctx = max(1, B // 2), max(40, ctx * 3 // 4)
        budget = max(8, int(ctx * rng.uniform(0.3, 0.99)))
        return dict(op=op, B=B, Hkv=Hkv, D=D, ctx=ctx, budget=budget, sinks=rng.choice([0, 1, 4]),
                    recent=int(budget * rng.uniform(0.0, 0.4)), page=page, order=order, kv=kv, ragged=rng.random() < 0.5)
    tree = rng.choice(["", "", "", "k21", "w4", "b63"])
    T = _nodes(tree) if tree else rng.choice([1, 1, rng.randint(2, 9), rng.randint(10, 33)])
    B, ctx = _log(rng, 1, 128), _log(rng, 1, 100000)
    while B * ctx * Hkv * D * 4.0 > MOST_KV or float(B) * T * G * Hkv * ctx > MOST_SCORES or B * T * G * Hkv * ctx * D > 3e10:
        B, ctx = max(1, B // 2), max(1, ctx * 3 // 4)
    c = dict(op=op, B=B, T=T, Hq=G * Hkv, Hkv=Hkv, D=D, ctx=ctx, page=page, order=order, dtype=dtype, kv=kv, tree=tree,
             ragged=rng.random() < 0.6)
    if op == "attention":
        c["lse"] = rng.random() < 0.5
    return c


def _nodes(tree):
    n, level = 1, 1
    for w in TREES[tree]:
        level *= w
        n += level
    return n


def _parents(tree):
    parent, level = [-1], [0]
    for w in TREES[tree]:
        nxt = []
        for u in level:
            for _ in range(w):
                nxt.append(len(parent))
                parent.append(u)
        level = nxt
    return parent


def _lens(case):
    """Cached lengths: all `ctx`, or spread over a quarter of it and the whole of it."""
    B, ctx = case["B"], case["ctx"]
    if not case["ragged"]:
        return [ctx] * B
    return [int(ctx * (0.25 + 0.75 * ((b + 1) * GOLDEN % 1.0))) for b in range(B)]


def _new(case):
    """New tokens of each sequence: all T, or fewer for every fifth sequence of a ragged batch."""
    T = case["T"]
    return [T - (b % T) // 2 if case["ragged"] and b % 5 == 4 else T for b in range(case["B"])]


def work(case):
    Hkv, D, e = case["Hkv"], case["D"], BYTES[case["kv"]]
    if case["op"] == "rope":
        n = sum(_new(case))
        read = n * (case["Hq"] + 2 * Hkv) * D * 2
        return {"bytes": read + n * (case["Hq"] * 2 + 2 * Hkv * e) * D, "flops": 3 * n * (case["Hq"] + Hkv) * case["rotary"]}
    if case["op"] == "evict":
        lens = _lens(case)
        kept = [min(n, case["budget"]) for n in lens]
        # a key at or above the budget stays with about the share that stays of all unprotected ones
        moved = sum(int((n - k) * max(0, k - case["recent"]) / n) + min(case["recent"], n - k) for n, k in zip(lens, kept))
        return {"bytes": Hkv * (8 * sum(lens) + 12 * sum(kept) + moved * 4 * D * e), "flops": Hkv * sum(lens)}
    L = sum(n + t for n, t in zip(_lens(case), _new(case)))
    rows = sum((n + t) * t for n, t in zip(_lens(case), _new(case))) * case["Hq"]
    n = sum(_new(case)) * case["Hq"]
    if case["op"] == "mass":
        return {"bytes": L * Hkv * (D * e + 8) + n * (2 * D + 4), "flops": 2 * rows * D // 2}
    return {"bytes": 2 * L * Hkv * D * e + n * (4 * D + (4 if case["lse"] else 0)), "flops": 4 * rows * D}


# ------------------------------------------------------------------ the inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _pools(case, gen, lens):
    """Page pools of K and V as [pages, page, heads, D] views, and each sequence's page table: as wide as the longest
    sequence of the case may need, -1 past each one's end."""
    page, Hkv, D = case["page"], case["Hkv"], case["D"]
    counts = [-(-n // page) for n in lens]
    pages, width = sum(counts) + PAGE_SLACK, -(-(case["ctx"] + case.get("T", 1)) // page)
    perm = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((case["B"], width), -1, dtype=torch.int32, device="cuda")
    count = torch.tensor(counts, device="cuda")
    held = torch.arange(width, device="cuda")[None] < count[:, None]
    table[held] = perm[: sum(counts)]
    pools = []
    for _ in range(2):
        shape = (pages, page, Hkv, D) if case["order"] == "nhd" else (pages, Hkv, page, D)
        pool = torch.empty(shape, dtype=DTYPES[case["kv"]], device="cuda")
        gain = 16.0 if case["kv"] == "e4m3" else 1.0
        step = max(1, (1 << 26) // pool[0].numel())
        for i in range(0, pages, step):  # in pieces: the fp32 draws of a large pool are large
            n = min(step, pages - i)
            pool[i : i + n] = (torch.randn((n,) + shape[1:], generator=gen, device="cuda") * gain).to(pool.dtype)
        pools.append(pool if case["order"] == "nhd" else pool.transpose(1, 2))
    scales = [None, None]
    if case["kv"] == "e4m3":
        scales = [(0.9 + 0.2 * torch.rand(Hkv, generator=gen, device="cuda")) / 16.0 for _ in range(2)]
    return pools, scales, table


def _frequencies(case):
    """Radians per position of each pair, in 64 bits."""
    r, base, factor = case["rotary"], 10000.0, 8.0
    if case["scaling"] == "base":
        base = base * factor ** (r / (r - 2.0))
    f = [base ** (-2.0 * i / r) for i in range(r // 2)]
    if case["scaling"] == "linear":
        f = [x / factor for x in f]
    if case["scaling"] == "by_parts":
        keep = [min(1.0, max(0.0, (8192.0 * x / (2.0 * math.pi) - 1.0) / 3.0)) for x in f]
        f = [k * x + (1.0 - k) * x / factor for k, x in zip(keep, f)]
    return f


def _turns(f):
    """Frequencies as 64-bit fractions of a turn per position (two's complement)."""
    n = [int(round(x / (2.0 * math.pi) * 2.0 ** 64)) % (1 << 64) for x in f]
    return [x - (1 << 64) if x >= 1 << 63 else x for x in n]


def prepare(case, seed):
    gen = _gen(seed)
    B, Hkv, D, dev = case["B"], case["Hkv"], case["D"], "cuda"
    if case["op"] == "evict":
        lens = _lens(case)
        (k, v), _, table = _pools(case, gen, lens)
        W = case["ctx"] + 1
        # weights of earlier steps: a few keys hold most of it, some got none
        mass = torch.exp(2.0 * torch.randn(B, Hkv, W, generator=gen, device=dev))
        mass[torch.rand(B, Hkv, W, generator=gen, device=dev) < 0.03] = 0.0
        # positions: an earlier eviction left gaps, and each head its own
        gaps = (torch.rand(B, Hkv, W, generator=gen, device=dev) < 0.1).to(torch.int32)
        pos = torch.arange(W, device=dev, dtype=torch.int32) + gaps.cumsum(-1).to(torch.int32)
        return dict(case=case, k=k, v=v, table=table, lens=torch.tensor(lens, dtype=torch.int32, device=dev), mass=mass, pos=pos,
                    out=dict(mass=torch.zeros(B, Hkv, case["budget"], device=dev),
                             pos=torch.full((B, Hkv, case["budget"]), -1, dtype=torch.int32, device=dev),
                             lens=torch.zeros(B, dtype=torch.int32, device=dev),
                             slot_src=torch.full((B, Hkv, case["budget"]), -1, dtype=torch.int32, device=dev)))
    T, Hq, dtype = case["T"], case["Hq"], DTYPES[case["dtype"]]
    ctx, new = _lens(case), _new(case)
    (k, v), scales, table = _pools(case, gen, [a + b for a, b in zip(ctx, new)])
    s = dict(case=case, k=k, v=v, k_scale=scales[0], v_scale=scales[1], table=table,
             ctx=torch.tensor(ctx, dtype=torch.int32, device=dev),
             new=torch.tensor(new, dtype=torch.int32, device=dev) if case["ragged"] else None)
    if case["op"] == "rope":
        # one projection's output holds q, k and v of a token side by side
        s["qkv"] = torch.randn(B, T, (Hq + 2 * Hkv) * D, generator=gen, device=dev).to(dtype)
        f = _frequencies(case)
        s["inv_freq"] = torch.tensor(f, dtype=torch.float64, device=dev)
        s["turns"] = torch.tensor(_turns(f), dtype=torch.int64, device=dev)
        # positions run ahead of the slots where an eviction has shortened the cache
        ahead = torch.randint(0, 60000, (B, 1), generator=gen, device=dev, dtype=torch.int32)
        s["positions"] = (s["ctx"][:, None] + torch.arange(T, device=dev, dtype=torch.int32) + ahead).contiguous()
        s["out"] = dict(q=torch.empty(B, T, Hq, D, dtype=dtype, device=dev))
        return s
    s["q"] = (2.0 * torch.randn(B, T, Hq, D, generator=gen, device=dev)).to(dtype)
    s["parent"] = None
    if case["tree"]:
        s["parent"] = torch.tensor(_parents(case["tree"]), dtype=torch.int32, device=dev).expand(B, T).contiguous()
    if case["op"] == "attention":
        s["out"] = dict(out=torch.empty(B, T, Hq, D, dtype=dtype, device=dev))
        if case["lse"]:
            s["out"]["lse"] = torch.empty(B, T, Hq, device=dev)
        return s
    # the verify step's outcome: each drafted token stands with probability 0.8
    W = case["ctx"] + T
    s["lse"] = _lse(_scores(s))
    if case["tree"]:
        path = [0]  # down the first children
        parent = _parents(case["tree"])
        while path[-1] in parent:
            path.append(parent.index(path[-1]))
        nodes = torch.full((B, T), -1, dtype=torch.int32, device=dev)
        nodes[:, : len(path) - 1] = torch.tensor(path[1:], dtype=torch.int32, device=dev)
        s["nodes"], depth = nodes, len(path) - 1
    else:
        s["nodes"], depth = None, T - 1
    stands = torch.rand(B, max(depth, 1), generator=gen, device=dev) < 0.8
    count = stands.to(torch.int32).cumprod(-1).sum(-1) if depth else torch.zeros(B, device=dev)
    here = torch.tensor(new, device=dev)
    last = (s["nodes"][:, :depth] < here[:, None]).sum(-1) if case["tree"] else here - 1
    s["accept"] = torch.minimum(count.to(torch.int32), last.to(torch.int32)).contiguous()
    if case["tree"]:
        s["nodes"] = torch.where(torch.arange(T, device=dev) < s["accept"][:, None], s["nodes"], -1).contiguous()
    s["mass_in"] = torch.rand(B, Hkv, W, generator=gen, device=dev)
    s["out"] = dict(mass=torch.zeros(B, Hkv, W, device=dev))
    return s


# ------------------------------------------------------------------ the plain forms

def _gather(pool, table, n):
    """Rows of the first n slots of each sequence: [B, n, heads, D]; page -1 reads page 0 (masked later)."""
    page = pool.shape[1]
    slot = torch.arange(n, device=pool.device)
    pages = table[:, slot // page].long().clamp(min=0)
    return pool[pages, slot % page]


def _span(s):
    """Slots that any sequence's new tokens can see."""
    return s["case"]["ctx"] + s["case"]["T"]


def _visible(s):
    """[B, T, n]: which slots each new token sees."""
    c, n, dev = s["case"], _span(s), s["q"].device
    T = c["T"]
    new = s["new"] if s["new"] is not None else torch.full((c["B"],), T, dtype=torch.int32, device=dev)
    if s["parent"] is None:
        sees = torch.ones(T, T, dtype=torch.bool, device=dev).tril().expand(c["B"], T, T)
    else:
        step = torch.zeros(c["B"], T, T, device=dev)
        step.scatter_(2, s["parent"].long().clamp(min=0)[:, :, None], 1.0)
        step[:, 0] = 0.0
        reach = torch.eye(T, device=dev) + step
        reach = (reach @ reach).clamp(max=1.0)  # ancestors up to 2, 4, ... 64 levels up
        reach = (reach @ reach).clamp(max=1.0)
        reach = (reach @ reach).clamp(max=1.0)
        reach = (reach @ reach).clamp(max=1.0)
        reach = (reach @ reach).clamp(max=1.0)
        sees = (reach @ reach) > 0
    slot = torch.arange(n, device=dev)
    node = slot[None] - s["ctx"][:, None]                                     # [B, n]
    drafted = torch.gather(sees, 2, node.clamp(0, T - 1)[:, None, :].expand(-1, T, -1))
    vis = (node < 0)[:, None, :] | (drafted & (node < new[:, None])[:, None, :])
    t = torch.arange(T, device=dev)
    return vis & (t[None] < new[:, None])[:, :, None]


def _scores(s):
    """Scaled scores [B, Hkv, T, G, n], minus infinity where a token does not see a slot."""
    c = s["case"]
    B, T, Hq, Hkv, D = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"]
    k = _gather(s["k"], s["table"], _span(s)).float().permute(0, 2, 3, 1)     # [B, Hkv, D, n]
    if s["k_scale"] is not None:
        k = k * s["k_scale"][None, :, None, None]
    q = s["q"].float().reshape(B, T, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    x = torch.matmul(q, k) * (1.0 / math.sqrt(D))
    x = x.reshape(B, Hkv, T, Hq // Hkv, -1)
    return x.masked_fill_(~_visible(s)[:, None, :, None, :], -math.inf)


def _lse(x):
    """log-sum-exp over the slots as [B, T, Hq]; minus infinity for a token that sees none."""
    m = x.amax(-1, keepdim=True)
    m0 = m.masked_fill(m == -math.inf, 0.0)
    z = torch.log(torch.exp(x - m0).sum(-1)) + m0.squeeze(-1)
    B, Hkv, T, G = z.shape
    return z.permute(0, 2, 1, 3).reshape(B, T, Hkv * G).contiguous()


def _plain_attention(s):
    c = s["case"]
    x = _scores(s)
    m = x.amax(-1, keepdim=True)
    x = torch.exp(x.sub_(m.masked_fill(m == -math.inf, 0.0)))
    z = x.sum(-1, keepdim=True)
    v = _gather(s["v"], s["table"], _span(s)).float().permute(0, 2, 1, 3)     # [B, Hkv, n, D]
    B, Hkv, T, G, n = x.shape
    # slots past a sequence's end hold anything
    end = s["ctx"] + (s["new"] if s["new"] is not None else T)
    v = v.masked_fill((torch.arange(n, device=v.device)[None] >= end[:, None])[:, None, :, None], 0.0)
    o = torch.matmul(x.reshape(B, Hkv, T * G, n), v).reshape(B, Hkv, T, G, -1)
    o = torch.where(z > 0, o / z, torch.zeros_like(o))
    if s["v_scale"] is not None:
        o = o * s["v_scale"][None, :, None, None, None]
    o = o.permute(0, 2, 1, 3, 4).reshape(B, T, Hkv * G, -1)
    out = {"out": o.to(s["q"].dtype)}
    if c["lse"]:
        m, z = m.squeeze(-1), z.squeeze(-1)
        lse = torch.log(z) + m.masked_fill(m == -math.inf, 0.0)
        out["lse"] = lse.permute(0, 2, 1, 3).reshape(B, T, Hkv * G)
    return out


def _counted(s):
    """[B, T]: the new tokens whose weights count: the first, and the accepted ones."""
    c = s["case"]
    t = torch.arange(c["T"], device=s["q"].device)
    if s["nodes"] is None:
        return t[None] <= s["accept"][:, None]
    on = torch.zeros(c["B"], c["T"] + 1, dtype=torch.bool, device=s["q"].device)
    taken = torch.where(t[None] < s["accept"][:, None], s["nodes"], c["T"]).long()
    on.scatter_(1, taken, True)
    on[:, 0] = s["accept"] >= 0
    return on[:, : c["T"]]


def _plain_mass(s):
    c = s["case"]
    x = _scores(s)
    B, Hkv, T, G, n = x.shape
    lse = s["lse"].reshape(B, T, Hkv, G).permute(0, 2, 1, 3)[..., None]
    w = torch.exp(x.sub_(lse.masked_fill(lse == -math.inf, 0.0)))
    w = (w * _counted(s)[:, None, :, None, None]).sum((2, 3))
    slot = torch.arange(n, device=w.device)[None, None]
    w = w + torch.where(slot < s["ctx"][:, None, None], s["mass_in"], torch.zeros_like(s["mass_in"]))
    end = (s["ctx"] + (s["new"] if s["new"] is not None else T))[:, None, None]
    out = s["out"]["mass"]
    out.copy_(torch.where(slot < end, w, out))
    return {"mass": out}


def _plain_rope(s):
    c, qkv = s["case"], s["qkv"]
    B, T, Hq, Hkv, D, r = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], c["rotary"]
    angle = s["positions"].double()[:, :, None] * s["inv_freq"]
    cos, sin = torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]
    x = qkv.float().reshape(B, T, Hq + 2 * Hkv, D)
    y = x.clone()
    turn = x[:, :, : Hq + Hkv, :r]
    if c["layout"] == "half":
        a, b = turn[..., : r // 2], turn[..., r // 2 :]
        y[:, :, : Hq + Hkv, : r // 2] = a * cos - b * sin
        y[:, :, : Hq + Hkv, r // 2 : r] = b * cos + a * sin
    else:
        a, b = turn[..., 0::2], turn[..., 1::2]
        y[:, :, : Hq + Hkv, 0:r:2] = a * cos - b * sin
        y[:, :, : Hq + Hkv, 1:r:2] = b * cos + a * sin
    t = torch.arange(T, device=qkv.device)[None]
    new = s["new"] if s["new"] is not None else torch.full((B,), T, dtype=torch.int32, device=qkv.device)
    live = t < new[:, None]
    slot = (s["ctx"][:, None] + t).long()
    q = torch.where(live[:, :, None, None], y[:, :, :Hq], 0.0).to(qkv.dtype)
    b, i = live.nonzero(as_tuple=True)
    at = slot[b, i]
    page = s["table"][b, at // c["page"]].long()
    for_k, for_v = y[b, i, Hq : Hq + Hkv], y[b, i, Hq + Hkv :]
    if s["k_scale"] is not None:
        for_k = (for_k / s["k_scale"][None, :, None]).clamp(-448.0, 448.0)
        for_v = (for_v / s["v_scale"][None, :, None]).clamp(-448.0, 448.0)
    s["k"][page, at % c["page"]] = for_k.to(s["k"].dtype)
    s["v"][page, at % c["page"]] = for_v.to(s["v"].dtype)
    return {"q": q, "k": s["k"], "v": s["v"]}


def _select(s):
    """slot_src [B, Hkv, budget]: the slot that each kept entry comes from, -1 past the new length; and the new lengths."""
    c, mass, pos = s["case"], s["mass"], s["pos"]
    W, budget, dev = mass.shape[-1], c["budget"], mass.device
    slot = torch.arange(W, device=dev)
    held = slot[None, None] < s["lens"][:, None, None]
    top = pos.masked_fill(~held, -1).amax(-1, keepdim=True)
    key = torch.where((pos < c["sinks"]) | (pos > top - c["recent"]), math.inf, mass.double())
    key = key.masked_fill(~held, -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :budget]
    kept = torch.zeros_like(held.expand_as(mass)).scatter(2, order, True) & held
    short = torch.clamp(s["lens"], max=budget)
    inside = slot[None, None] < short[:, None, None]
    hole = inside & ~kept
    mover = kept & ~inside
    source = torch.sort(torch.where(mover, slot, W), dim=-1).values             # movers first, in order
    rank = (hole.cumsum(-1) - 1).clamp(min=0)
    src = torch.where(hole, source.gather(2, rank), slot.expand_as(rank))
    src = torch.where(inside, src, -1)[..., :budget]
    if budget > W:
        src = torch.nn.functional.pad(src, (0, budget - W), value=-1)
    return src, short


def _plain_evict(s):
    c, out = s["case"], s["out"]
    src, short = _select(s)
    b, h, i = ((src >= 0) & (src != torch.arange(c["budget"], device=src.device))).nonzero(as_tuple=True)
    j = src[b, h, i]
    page = c["page"]
    p0, p1 = s["table"][b, j // page].long(), s["table"][b, i // page].long()
    s["k"][p1, i % page, h] = s["k"][p0, j % page, h]
    s["v"][p1, i % page, h] = s["v"][p0, j % page, h]
    at = src.clamp(min=0)
    live = src >= 0
    out["mass"].copy_(torch.where(live, s["mass"].gather(2, at), out["mass"]))
    out["pos"].copy_(torch.where(live, s["pos"].gather(2, at), out["pos"]))
    out["lens"].copy_(short)
    out["slot_src"].copy_(src)
    return {"k": s["k"], "v": s["v"], **out}


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    return {"rope": _plain_rope, "attention": _plain_attention, "mass": _plain_mass, "evict": _plain_evict}[op](state)


def _own(s, op):
    import speculative_decoding_token_spv_gb300 as spv

    c = s["case"]
    cache = spv.KVCache(s["k"], s["v"], s.get("k_scale"), s.get("v_scale"))
    if op == "rope":
        B, T, Hq, Hkv, D = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"]
        q, k, v = s["qkv"].view(B, T, Hq + 2 * Hkv, D).split([Hq, Hkv, Hkv], dim=2)
        got = spv.spv_rope_append(q, k, v, cache, s["table"], s["ctx"], s["turns"], interleaved=c["layout"] == "interleaved",
                                  positions=s["positions"], new_lens=s["new"], out=s["out"], want_status=False)
        return {"q": got["q"], "k": s["k"], "v": s["v"]}
    if op == "attention":
        if "workspace" not in s:
            s["workspace"] = spv.new_workspace(spv.spv_attention_workspace_bytes(c["B"], c["T"], c["Hq"], c["Hkv"], c["D"]),
                                               s["q"].device)
        return spv.spv_paged_attention(s["q"], cache, s["table"], s["ctx"], new_lens=s["new"], parent=s["parent"],
                                       workspace=s["workspace"], out=s["out"], want_lse=c["lse"], want_status=False)
    if op == "mass":
        return spv.spv_attention_mass(s["q"], s["lse"], cache, s["table"], s["ctx"], s["accept"], nodes=s["nodes"],
                                      new_lens=s["new"], parent=s["parent"], mass_in=s["mass_in"], out=s["out"],
                                      want_status=False)
    got = spv.spv_kv_evict(cache, s["table"], s["lens"], s["mass"], c["budget"], pos=s["pos"], sinks=c["sinks"],
                           recent=c["recent"], out=s["out"], want_status=False)
    return {"k": s["k"], "v": s["v"], **got}


# ------------------------------------------------------------------ the definition in 64 bits

def _rows64(pool, scale, table, b, n):
    """The first n rows of sequence b in 64 bits: [heads, n, D]."""
    page = pool.shape[1]
    slot = torch.arange(n, device=pool.device)
    x = pool[table[b].long()[slot // page], slot % page].double()
    if scale is not None:
        x = x * scale.double()[None, :, None]
    return x.transpose(0, 1)


def _probabilities64(s, b):
    """(keys in use, new tokens, probabilities [Hkv, T', G, n], lse [Hkv, T', G]) of sequence b."""
    c = s["case"]
    base, t = int(s["ctx"][b]), c["T"] if s["new"] is None else int(s["new"][b])
    n, Hkv, G = base + t, c["Hkv"], c["Hq"] // c["Hkv"]
    k = _rows64(s["k"], s["k_scale"], s["table"], b, n)
    q = s["q"][b, :t].double().reshape(t, Hkv, G, c["D"]).permute(1, 0, 2, 3)
    x = torch.einsum("htgd,hnd->htgn", q, k) / c["D"] ** 0.5
    sees = torch.zeros(t, n, dtype=torch.bool)
    sees[:, :base] = True
    up = [i - 1 for i in range(t)] if s["parent"] is None else s["parent"][b].tolist()
    for i in range(t):
        j = i
        while j >= 0:
            sees[i, base + j] = True
            j = up[j]
    x = x.masked_fill(~sees.to(x.device)[None, :, None, :], -math.inf)
    lse = torch.logsumexp(x, -1)
    return n, t, torch.softmax(x, -1), lse


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _rope64, "attention": _attention64, "mass": _mass64, "evict": _evict64}[case["op"]](s)


def _attention64(s):
    c = s["case"]
    out = torch.zeros(c["B"], c["T"], c["Hq"], c["D"], dtype=torch.float64, device=s["q"].device)
    lse = torch.full((c["B"], c["T"], c["Hq"]), -math.inf, dtype=torch.float64, device=s["q"].device)
    for b in range(c["B"]):
        n, t, p, z = _probabilities64(s, b)
        o = torch.einsum("htgn,hnd->thgd", p, _rows64(s["v"], s["v_scale"], s["table"], b, n))
        out[b, :t] = o.reshape(t, c["Hq"], c["D"])
        lse[b, :t] = z.transpose(0, 1).reshape(t, c["Hq"])
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}


def _mass64(s):
    c, mass = s["case"], s["out"]["mass"].double()
    for b in range(c["B"]):
        n, t, p, z = _probabilities64(s, b)
        k = int(s["accept"][b])
        rows = list(range(k + 1)) if s["nodes"] is None else [0] + s["nodes"][b, :k].tolist()
        w = p[:, rows].sum((1, 2))
        base = int(s["ctx"][b])
        w[:, :base] += s["mass_in"][b, :, :base].double()
        mass[b, :, :n] = w
    return {"mass": mass}


def _rope64(s):
    c = s["case"]
    B, T, Hq, Hkv, D, r = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], c["rotary"]
    x = s["qkv"].double().reshape(B, T, Hq + 2 * Hkv, D)
    pairs = x[..., :r].reshape(B, T, -1, 2, r // 2).transpose(-1, -2) if c["layout"] == "half" else x[..., :r].reshape(B, T, -1, r // 2, 2)
    z = torch.view_as_complex(pairs.contiguous())
    angle = s["positions"].double()[:, :, None, None] * s["inv_freq"]
    z = torch.view_as_real(z * torch.polar(torch.ones_like(angle), angle))
    z = z.transpose(-1, -2).reshape(B, T, -1, r) if c["layout"] == "half" else z.reshape(B, T, -1, r)
    x[:, :, : Hq + Hkv, :r] = z[:, :, : Hq + Hkv]
    q, k, v = x[:, :, :Hq].clone(), s["k"].double(), s["v"].double()
    for b in range(B):
        t = T if s["new"] is None else int(s["new"][b])
        q[b, t:] = 0.0
        slot = int(s["ctx"][b]) + torch.arange(t, device=x.device)
        page = s["table"][b].long()[slot // c["page"]]
        kb, vb = x[b, :t, Hq : Hq + Hkv], x[b, :t, Hq + Hkv :]
        if s["k_scale"] is not None:
            kb, vb = kb / s["k_scale"].double()[:, None], vb / s["v_scale"].double()[:, None]
        k[page, slot % c["page"]] = kb
        v[page, slot % c["page"]] = vb
    return {"q": q, "k": k, "v": v}


def _evict64(s):
    """The moved rows are copies and the weights too: their values in 64 bits, by a selection of its own on the host."""
    c, out = s["case"], s["out"]
    if c["B"] * c["Hkv"] * c["ctx"] > 3e6:
        return None
    mass, pos, lens = s["mass"].tolist(), s["pos"].tolist(), s["lens"].tolist()
    new = out["mass"].double()
    moves = [[], [], [], []]
    for b in range(c["B"]):
        n = lens[b]
        m = min(n, c["budget"])
        for h in range(c["Hkv"]):
            top = max(pos[b][h][:n], default=0)
            always = [p < c["sinks"] or p > top - c["recent"] for p in pos[b][h][:n]]
            best = sorted(range(n), key=lambda j: (not always[j], -mass[b][h][j] if not always[j] else 0.0, j))[:m]
            kept = set(best)
            movers = sorted(j for j in best if j >= m)
            src = [i if i in kept else movers.pop(0) for i in range(m)]
            new[b, h, :m] = s["mass"][b, h, src].double()
            for i, j in enumerate(src):
                if i != j:
                    for a, x in zip(moves, (b, h, i, j)):
                        a.append(x)
    b, h, i, j = (torch.tensor(a, dtype=torch.int64, device=s["k"].device) for a in moves)
    page = c["page"]
    pools = []
    for pool in (s["k"], s["v"]):
        x = pool.double()
        x[s["table"][b, i // page].long(), i % page, h] = pool[s["table"][b, j // page].long(), j % page, h].double()
        pools.append(x)
    return {"k": pools[0], "v": pools[1], "mass": new, "pos": None, "lens": None, "slot_src": None}
