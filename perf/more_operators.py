"""Measured cases of the attention layer of models whose attention is not plain.

Such a target model norms each head of q and k before the rotation, may rotate
by positions of several axes (time, height, width), caps its scores by a tanh,
takes a bias that grows with the distance off them, or sees no further than a
window, its document or a prefix.  The calls around a verify step in that form:
norms, rotation and the write to the paged cache in one pass (``norm_rope``),
attention of one token, a drafted chain or tree (``attention``), attention of
whole prompts (``prompt``), and the weight that each cached key received
(``mass``).

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
        # one conversation, one token: the latency of a layer's norms, rotation and write
        dict(name="norm_rope_one_token", op="norm_rope", B=1, T=1, Hq=32, Hkv=8, D=128, rotary=128, layout="half", axes=1,
             ctx=777, page=16, order="nhd", dtype="bf16", kv="bf16", ragged=False),
        # a verify step of a serving batch: gamma = 4 drafted tokens and the last one, 8-bit cache
        dict(name="norm_rope_verify_e4m3", op="norm_rope", B=64, T=5, Hq=64, Hkv=8, D=128, rotary=128, layout="half", axes=1,
             ctx=1500, page=16, order="nhd", dtype="bf16", kv="e4m3", ragged=True),
        # prompts with images and video entering the cache: time, height and width
        dict(name="norm_rope_video_prompt", op="norm_rope", B=8, T=2011, Hq=32, Hkv=8, D=128, rotary=128, layout="half",
             axes=3, ctx=0, page=32, order="hnd", dtype="f16", kv="f16", ragged=True),
        # one conversation, one token, capped scores: latency
        dict(name="attn_one_token_capped", op="attention", B=1, T=1, Hq=32, Hkv=8, D=128, ctx=777, page=16, order="nhd",
             dtype="bf16", kv="bf16", tree="", ragged=False, lse=False, cap=50.0, slopes=False, window=0, mask="",
             moved=False),
        # plain decoding of a full batch, capped, heads of 256, in a layer that sees the last 4,096 tokens
        dict(name="attn_decode_window", op="attention", B=64, T=1, Hq=16, Hkv=8, D=256, ctx=8191, page=16, order="nhd",
             dtype="bf16", kv="bf16", tree="", ragged=True, lse=False, cap=50.0, slopes=False, window=4096, mask="",
             moved=False),
        # the verify step of the headline batch with a distance bias, over caches that evictions have cut: each head
        # has positions of its own
        dict(name="attn_verify_bias", op="attention", B=64, T=5, Hq=64, Hkv=8, D=128, ctx=8191, page=16, order="nhd",
             dtype="bf16", kv="bf16", tree="", ragged=True, lse=True, cap=0.0, slopes=True, window=0, mask="", moved=True),
        # the 21-node draft tree on a batch of 32, capped; the sequences' caches begin with earlier documents
        dict(name="attn_tree_document", op="attention", B=32, T=21, Hq=32, Hkv=8, D=128, ctx=4099, page=32, order="hnd",
             dtype="f16", kv="f16", tree="k21", ragged=True, lse=True, cap=30.0, slopes=False, window=0, mask="documents",
             moved=False),
        # a piece of a prompt over a long 8-bit cache
        dict(name="prompt_piece_e4m3", op="prompt", B=1, T=251, Hq=32, Hkv=8, D=128, ctx=30011, page=64, order="nhd",
             dtype="bf16", kv="e4m3", ragged=False, lse=False, cap=0.0, slopes=True, window=0, mask="", moved=False),
        # whole prompts, capped scores
        dict(name="prompt_capped", op="prompt", B=2, T=5003, Hq=32, Hkv=8, D=128, ctx=0, page=16, order="nhd",
             dtype="bf16", kv="bf16", ragged=True, lse=False, cap=50.0, slopes=False, window=0, mask="", moved=False),
        # rows of packed documents, each with a prefix that sees itself whole
        dict(name="prompt_documents", op="prompt", B=2, T=8192, Hq=32, Hkv=8, D=128, ctx=0, page=32, order="hnd",
             dtype="f16", kv="f16", ragged=False, lse=True, cap=0.0, slopes=False, window=0, mask="prefixes", moved=False),
        # the weight of every cached key after a verify step, capped scores
        dict(name="mass_verify_capped", op="mass", B=64, T=5, Hq=64, Hkv=8, D=128, ctx=8191, page=16, order="nhd",
             dtype="bf16", kv="bf16", tree="", ragged=True, cap=50.0, slopes=False, window=0, mask="", moved=False),
        # the same of a small batch of trees with a distance bias over moved slots
        dict(name="mass_tree_bias", op="mass", B=4, T=17, Hq=32, Hkv=8, D=128, ctx=2111, page=16, order="nhd",
             dtype="f16", kv="f16", tree="w4", ragged=True, cap=0.0, slopes=True, window=0, mask="", moved=True),
    ]


MOST_KV = 1.3e9       # bytes of the caches that the largest listed case reads
MOST_SCORES = 8e8     # scores of its plain form, for calls of a few tokens
MOST_PROMPT = 1.6e9   # and for prompts


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "attention", "attention", "prompt", "prompt", "mass"])
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    page = rng.choice([8, 16, 32, 64, 128])
    order = rng.choice(["nhd", "hnd"])
    dtype = rng.choice(["bf16", "f16"])
    kv = rng.choice([dtype, dtype, "e4m3"])
    c = dict(op=op, Hq=G * Hkv, Hkv=Hkv, D=D, page=page, order=order, dtype=dtype, kv=kv)
    if op == "norm_rope":
        B, T = _log(rng, 1, 128), rng.choice([1, rng.randint(2, 33), _log(rng, 34, 4000)])
        while B * T * (G + 2) * Hkv * D > 8e7:
            B, T = max(1, B // 2), max(1, T * 3 // 4)
        return dict(c, B=B, T=T, rotary=rng.choice([D, D, D // 2]), layout=rng.choice(["half", "interleaved"]),
                    axes=rng.choice([1, 2, 3]), ctx=_log(rng, 1, 2000), ragged=rng.random() < 0.5)
    c.update(cap=rng.choice([0.0, 15.0, 30.0, 50.0]), slopes=rng.random() < 0.4, moved=rng.random() < 0.3)
    c["lse"] = op != "mass" and rng.random() < 0.5
    if op == "prompt":
        T, ctx, B = _log(rng, 65, 8000), rng.choice([0, 0, _log(rng, 1, 30000)]), _log(rng, 1, 16)
        while float(B) * T * G * Hkv * (ctx + T) > MOST_PROMPT or B * (ctx + T) * Hkv * D * 4.0 > MOST_KV \
                or float(B) * T * G * Hkv * (ctx + T) * D > 2.1e11:
            B, ctx, T = max(1, B // 2), ctx * 3 // 4, max(65, T * 7 // 8)
        mask = rng.choice(["", "", "documents", "prefixes"])
        tree = ""
    else:
        tree = rng.choice(["", "", "", "k21", "w4", "b63"])
        T = _nodes(tree) if tree else rng.choice([1, 1, rng.randint(2, 9), rng.randint(10, 33)])
        B, ctx = _log(rng, 1, 128), _log(rng, 1, 100000)
        while B * ctx * Hkv * D * 4.0 > MOST_KV or float(B) * T * G * Hkv * ctx > MOST_SCORES or B * T * G * Hkv * ctx * D > 3e10:
            B, ctx = max(1, B // 2), max(1, ctx * 3 // 4)
        mask = rng.choice(["", "", "documents"])
        c["tree"] = tree
    window = rng.choice([0, 0, _log(rng, 16, max(32, ctx + T))])
    return dict(c, B=B, T=T, ctx=ctx, window=window, mask=mask, ragged=rng.random() < 0.6)


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
    """New tokens of each sequence: all T; in a ragged batch of prompts between half and all of T, of a few tokens fewer
    for every fifth sequence."""
    B, T = case["B"], case["T"]
    if not case["ragged"]:
        return [T] * B
    if T > 64:
        return [T - int(T // 2 * ((b + 1) * GOLDEN % 1.0)) for b in range(B)]
    return [T - (b % T) // 2 if b % 5 == 4 else T for b in range(B)]


def _spans(case):
    """(first, last) of each sequence's new tokens as lists, or None: the slot where a token's document begins, and
    where the prefix ends that its document's tokens see whole."""
    if not case["mask"]:
        return None
    firsts, lasts, T = [], [], case["T"]
    for b, ctx in enumerate(_lens(case)):
        first, last = [], []
        if T <= 64:  # the present document began somewhere in the cache
            first = [int(ctx * ((b + 2) * GOLDEN % 1.0))] * T
        else:
            at, i = 0, b
            while at < T:  # the first document goes on from the cache
                n = min(T - at, max(1, int(T / 6 * (0.25 + 1.5 * ((i + 1) * GOLDEN % 1.0)))))
                start = 0 if at == 0 else ctx + at
                first += [start] * n
                last += [ctx + at + n // 3] * n
                at, i = at + n, i + 1
        firsts.append(first)
        lasts.append(last)
    return firsts, lasts if case["mask"] == "prefixes" else None


def _seen(case):
    """(keys read of all sequences, rows times keys seen of a query head), with positions taken for slots."""
    keys = rows = 0
    spans = _spans(case)
    tree = _parents(case["tree"]) if case.get("tree") else None
    depth = [0] * case["T"]
    for v in range(1, len(tree or [])):
        depth[v] = depth[tree[v]] + 1
    for b, (ctx, new) in enumerate(zip(_lens(case), _new(case))):
        lowest, total = ctx + new, ctx + new
        for t in range(new):
            lo = spans[0][b][t] if spans else 0
            if case["window"]:
                lo = max(lo, ctx + (depth[t] if tree else t) - case["window"] + 1)
            if tree:
                n = max(0, ctx - lo) + depth[t] + 1
            else:
                hi = ctx + t + 1
                if spans and spans[1]:
                    hi = max(hi, min(total, spans[1][b][t]))
                n = max(0, hi - lo)
            rows += n
            lowest = min(lowest, max(lo, 0))
        keys += total - lowest
    return keys, rows


def work(case):
    Hq, Hkv, D, e = case["Hq"], case["Hkv"], case["D"], BYTES[case["kv"]]
    n = sum(_new(case))
    if case["op"] == "norm_rope":
        read = n * (Hq + 2 * Hkv) * D * 2
        return {"bytes": read + n * (Hq * 2 + 2 * Hkv * e) * D + 8 * D, "flops": n * (Hq + Hkv) * (4 * D + 3 * case["rotary"])}
    keys, rows = _seen(case)
    flops = 4 * rows * Hq * D
    moved = 4 * keys * Hkv if case["moved"] else 0
    if case["op"] == "mass":
        L = sum(a + b for a, b in zip(_lens(case), _new(case)))
        return {"bytes": keys * Hkv * D * e + L * Hkv * 8 + moved + n * Hq * (2 * D + 4), "flops": flops // 4}
    return {"bytes": 2 * keys * Hkv * D * e + moved + n * Hq * (4 * D + (4 if case["lse"] else 0)), "flops": flops}


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
    pages, width = sum(counts) + PAGE_SLACK, -(-(case["ctx"] + case["T"]) // page)
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


def _sections(case):
    """The axis of each pair: the first pairs time's, then height's, then width's."""
    pairs, axes = case["rotary"] // 2, case["axes"]
    cuts = [pairs] if axes == 1 else [pairs // 2, pairs - pairs // 2] if axes == 2 else [pairs // 4, 3 * pairs // 8]
    if axes == 3:
        cuts.append(pairs - sum(cuts))
    return [a for a, n in enumerate(cuts) for _ in range(n)]


def _turns(f):
    """Frequencies as 64-bit fractions of a turn per position (two's complement)."""
    n = [int(round(x / (2.0 * math.pi) * 2.0 ** 64)) % (1 << 64) for x in f]
    return [x - (1 << 64) if x >= 1 << 63 else x for x in n]


def prepare(case, seed):
    gen = _gen(seed)
    B, T, Hq, Hkv, D, dev = case["B"], case["T"], case["Hq"], case["Hkv"], case["D"], "cuda"
    dtype, ctx, new = DTYPES[case["dtype"]], _lens(case), _new(case)
    (k, v), scales, table = _pools(case, gen, [a + b for a, b in zip(ctx, new)])
    s = dict(case=case, k=k, v=v, k_scale=scales[0], v_scale=scales[1], table=table,
             ctx=torch.tensor(ctx, dtype=torch.int32, device=dev),
             new=torch.tensor(new, dtype=torch.int32, device=dev) if case["ragged"] else None)
    if case["op"] == "norm_rope":
        # one projection's output holds q, k and v of a token side by side; its heads' sizes differ
        x = torch.randn(B, T, Hq + 2 * Hkv, D, generator=gen, device=dev)
        x *= torch.exp(0.5 * torch.randn(B, T, Hq + 2 * Hkv, 1, generator=gen, device=dev))
        s["qkv"] = x.to(dtype).reshape(B, T, -1)
        s["q_weight"], s["k_weight"] = (1.0 + 0.3 * torch.randn(D, generator=gen, device=dev) for _ in range(2))
        f = [10000.0 ** (-2.0 * i / case["rotary"]) for i in range(case["rotary"] // 2)]
        s["inv_freq"] = torch.tensor(f, dtype=torch.float64, device=dev)
        s["turns"] = torch.tensor(_turns(f), dtype=torch.int64, device=dev)
        s["axes"] = torch.tensor(_sections(case), dtype=torch.int32, device=dev) if case["axes"] > 1 else None
        if case["axes"] == 1:
            # positions run ahead of the slots where an eviction has shortened the cache
            ahead = torch.randint(0, 60000, (B, 1), generator=gen, device=dev, dtype=torch.int32)
            s["positions"] = (s["ctx"][:, None] + torch.arange(T, device=dev, dtype=torch.int32) + ahead).contiguous()
        else:
            # frames of 24 x 32 patches after the cached tokens
            t = torch.arange(T, device=dev, dtype=torch.int32)
            grid = torch.stack([t // 768, t % 768 // 32, t % 32][: case["axes"]], -1)
            s["positions"] = (s["ctx"][:, None, None] + grid).contiguous()
        s["out"] = dict(q=torch.empty(B, T, Hq, D, dtype=dtype, device=dev))
        return s
    # capped models have larger scores: the largest at a third of the cap or more
    gain = 4.0 if case["cap"] else 2.0
    s["q"] = (gain * torch.randn(B, T, Hq, D, generator=gen, device=dev)).to(dtype)
    s["parent"] = None
    if case.get("tree"):
        s["parent"] = torch.tensor(_parents(case["tree"]), dtype=torch.int32, device=dev).expand(B, T).contiguous()
    s["slopes"] = None
    if case["slopes"]:  # a geometric series over the heads
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, Hq + 1, device=dev, dtype=torch.float32) / Hq)
    s["first"] = s["last"] = None
    spans = _spans(case)
    if spans:
        s["first"] = torch.tensor(spans[0], dtype=torch.int32, device=dev)
        if spans[1]:
            s["last"] = torch.tensor(spans[1], dtype=torch.int32, device=dev)
    s["slot_pos"] = None
    if case["moved"]:
        # an earlier eviction has left gaps, each head its own; the new tokens follow at one position for all heads
        W = case["ctx"] + T
        gaps = (torch.rand(B, Hkv, W, generator=gen, device=dev) < 0.1).to(torch.int32)
        pos = torch.arange(W, device=dev, dtype=torch.int32) + gaps.cumsum(-1).to(torch.int32)
        ahead = pos[:, :, -1].amax(1)[:, None] + 1 + _depths(case, dev)               # [B, T]
        at = (s["ctx"][:, None] + torch.arange(T, device=dev)).long()[:, None, :].expand(-1, Hkv, -1)
        s["slot_pos"] = pos.scatter(2, at, ahead[:, None, :].expand(-1, Hkv, -1).to(torch.int32)).contiguous()
    if case["op"] != "mass":
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


def _depths(case, dev):
    """Levels of the new tokens below the first: 0, 1, 2, ... of a chain, those of the tree."""
    if not case.get("tree"):
        return torch.arange(case["T"], device=dev, dtype=torch.int32)
    depth, parent = [0], _parents(case["tree"])
    for v in range(1, len(parent)):
        depth.append(depth[parent[v]] + 1)
    return torch.tensor(depth, dtype=torch.int32, device=dev)


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


def _fresh(s):
    c = s["case"]
    return s["new"] if s["new"] is not None else torch.full((c["B"],), c["T"], dtype=torch.int32, device=s["table"].device)


def _distance(s):
    """Positions of the new tokens less those of the slots: [B, Hkv or 1, T, n]."""
    c, n, dev = s["case"], _span(s), s["q"].device
    if s["slot_pos"] is not None:
        pos = s["slot_pos"][:, :, :n]
        at = (s["ctx"][:, None] + torch.arange(c["T"], device=dev)).long()[:, None, :].expand(-1, c["Hkv"], -1)
        return pos.gather(2, at)[..., None] - pos[:, :, None, :]
    here = s["ctx"][:, None] + _depths(c, dev)                                # [B, T]
    slot = torch.arange(n, device=dev, dtype=torch.int32)
    node = (slot[None] - s["ctx"][:, None]).clamp(0, c["T"] - 1).long()
    there = torch.where(slot[None] < s["ctx"][:, None], slot[None].expand(c["B"], -1), here.gather(1, node))
    return (here[:, :, None] - there[:, None, :])[:, None]


def _visible(s):
    """[B, Hkv or 1, T, n]: which slots each new token sees."""
    c, n, dev = s["case"], _span(s), s["q"].device
    B, T, new = c["B"], c["T"], _fresh(s)
    slot, t = torch.arange(n, device=dev), torch.arange(T, device=dev)
    own_slot = s["ctx"][:, None] + t                                          # [B, T]
    if s["parent"] is None:
        vis = slot[None, None] <= own_slot[:, :, None]
        if s["last"] is not None:
            vis = vis | (slot[None, None] < s["last"][:, :, None])
    else:
        step = torch.zeros(B, T, T, device=dev)
        step.scatter_(2, s["parent"].long().clamp(min=0)[:, :, None], 1.0)
        step[:, 0] = 0.0
        reach = torch.eye(T, device=dev) + step
        reach = (reach @ reach).clamp(max=1.0)  # ancestors up to 2, 4, ... 64 levels up
        reach = (reach @ reach).clamp(max=1.0)
        reach = (reach @ reach).clamp(max=1.0)
        reach = (reach @ reach).clamp(max=1.0)
        reach = (reach @ reach).clamp(max=1.0)
        sees = (reach @ reach) > 0
        node = slot[None] - s["ctx"][:, None]
        drafted = torch.gather(sees, 2, node.clamp(0, T - 1)[:, None, :].expand(-1, T, -1))
        vis = (node < 0)[:, None, :] | (drafted & (node < T)[:, None, :])
    if s["first"] is not None:
        vis = vis & (slot[None, None] >= s["first"][:, :, None])
    vis = vis & (slot[None] < (s["ctx"] + new)[:, None])[:, None, :] & (t[None] < new[:, None])[:, :, None]
    if c["window"]:
        return vis[:, None] & (_distance(s) < c["window"])
    return vis[:, None]


def _scores(s):
    """Scores [B, Hkv, T, G, n], minus infinity where a token does not see a slot."""
    c = s["case"]
    B, T, Hq, Hkv, D = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"]
    k = _gather(s["k"], s["table"], _span(s)).float().permute(0, 2, 3, 1)     # [B, Hkv, D, n]
    if s["k_scale"] is not None:
        k = k * s["k_scale"][None, :, None, None]
    q = s["q"].float().reshape(B, T, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    x = torch.matmul(q, k).mul_(1.0 / math.sqrt(D))
    x = x.reshape(B, Hkv, T, Hq // Hkv, -1)
    if c["cap"]:
        x = x.mul_(1.0 / c["cap"]).tanh_().mul_(c["cap"])
    if s["slopes"] is not None:
        x = x.addcmul_(_distance(s).abs().float()[:, :, :, None, :], -s["slopes"].reshape(1, Hkv, 1, -1, 1))
    return x.masked_fill_(~_visible(s)[:, :, :, None, :], -math.inf)


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
    x = x.sub_(m.masked_fill(m == -math.inf, 0.0)).exp_()
    z = x.sum(-1, keepdim=True)
    v = _gather(s["v"], s["table"], _span(s)).float().permute(0, 2, 1, 3)     # [B, Hkv, n, D]
    B, Hkv, T, G, n = x.shape
    # slots past a sequence's end hold anything
    end = s["ctx"] + _fresh(s)
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
    x = _scores(s)
    B, Hkv, T, G, n = x.shape
    lse = s["lse"].reshape(B, T, Hkv, G).permute(0, 2, 1, 3)[..., None]
    w = x.sub_(lse.masked_fill(lse == -math.inf, 0.0)).exp_()
    w = (w * _counted(s)[:, None, :, None, None]).sum((2, 3))
    slot = torch.arange(n, device=w.device)[None, None]
    w = w + torch.where(slot < s["ctx"][:, None, None], s["mass_in"], torch.zeros_like(s["mass_in"]))
    end = (s["ctx"] + _fresh(s))[:, None, None]
    out = s["out"]["mass"]
    out.copy_(torch.where(slot < end, w, out))
    return {"mass": out}


def _plain_norm_rope(s):
    c, qkv = s["case"], s["qkv"]
    B, T, Hq, Hkv, D, r = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], c["rotary"]
    p = s["positions"].double()[..., None] if s["axes"] is None else s["positions"].double()[..., s["axes"].long()]
    angle = p * s["inv_freq"]                                                 # [B, T, r / 2]
    cos, sin = torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]
    x = qkv.float().reshape(B, T, Hq + 2 * Hkv, D)
    unit = torch.rsqrt((x * x).sum(-1, keepdim=True) / D + 1e-6)
    weight = torch.cat([s["q_weight"].expand(Hq, D), s["k_weight"].expand(Hkv, D)])
    x = torch.cat([x[:, :, : Hq + Hkv] * unit[:, :, : Hq + Hkv] * weight, x[:, :, Hq + Hkv :]], 2)
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
    live = t < _fresh(s)[:, None]
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


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    return {"norm_rope": _plain_norm_rope, "attention": _plain_attention, "prompt": _plain_attention, "mass": _plain_mass}[op](state)


def _own(s, op):
    import speculative_decoding_token_spv_gb300 as spv

    c = s["case"]
    B, T, Hq, Hkv, D = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"]
    cache = spv.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    if op == "norm_rope":
        q, k, v = s["qkv"].view(B, T, Hq + 2 * Hkv, D).split([Hq, Hkv, Hkv], dim=2)
        got = spv.spv_norm_rope_append(q, k, v, cache, s["table"], s["ctx"], s["turns"], q_weight=s["q_weight"],
                                       k_weight=s["k_weight"], eps=1e-6, axes=s["axes"], interleaved=c["layout"] == "interleaved",
                                       positions=s["positions"], new_lens=s["new"], out=s["out"], want_status=False)
        return {"q": got["q"], "k": s["k"], "v": s["v"]}
    scores = spv.Scores(cap=c["cap"], slopes=s["slopes"], window=c["window"], first=s["first"], last=s["last"],
                        slot_pos=s["slot_pos"])
    if op == "mass":
        return spv.spv_attention_mass_scored(s["q"], s["lse"], cache, s["table"], s["ctx"], s["accept"], scores,
                                             nodes=s["nodes"], new_lens=s["new"], parent=s["parent"], mass_in=s["mass_in"],
                                             out=s["out"], want_status=False)
    if op == "attention":
        if "workspace" not in s:
            s["workspace"] = spv.new_workspace(spv.spv_attention_workspace_bytes(B, T, Hq, Hkv, D), s["q"].device)
        return spv.spv_paged_attention_scored(s["q"], cache, s["table"], s["ctx"], scores, new_lens=s["new"],
                                              parent=s["parent"], workspace=s["workspace"], out=s["out"], want_lse=c["lse"],
                                              want_status=False)
    if "workspace" not in s:
        s["workspace"] = spv.new_workspace(spv.spv_prompt_workspace_bytes(B, T, Hq, Hkv, D), s["q"].device)
    return spv.spv_prompt_attention(s["q"], cache, s["table"], s["ctx"], scores, new_lens=s["new"], workspace=s["workspace"],
                                    out=s["out"], want_lse=c["lse"], want_status=False)


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm_rope": _norm_rope64, "attention": _attention64, "prompt": _attention64, "mass": _mass64}[case["op"]](s)


def _rows64(pool, scale, table, b, n):
    """The first n rows of sequence b in 64 bits: [heads, n, D]."""
    page = pool.shape[1]
    slot = torch.arange(n, device=pool.device)
    x = pool[table[b].long()[slot // page], slot % page].double()
    if scale is not None:
        x = x * scale.double()[None, :, None]
    return x.transpose(0, 1)


def _masks64(s, b, base, t):
    """(sees [t, n] without the window, level of each new token) of sequence b."""
    c, dev, n = s["case"], s["q"].device, base + t
    sees = torch.zeros(t, n, dtype=torch.bool, device=dev)
    sees[:, :base] = True
    if s["parent"] is None:
        sees[:, base:] = torch.ones(t, t, dtype=torch.bool, device=dev).tril()
        level = list(range(t))
        if s["last"] is not None:
            sees |= torch.arange(n, device=dev) < s["last"][b, :t, None]
    else:
        up, level = s["parent"][b].tolist(), []
        for i in range(t):
            j, path = i, []
            while j > 0:
                path.append(j)
                j = up[j]
            sees[i, [base + p for p in path] + [base]] = True
            level.append(len(path))
    if s["first"] is not None:
        sees &= torch.arange(n, device=dev) >= s["first"][b, :t, None]
    return sees, torch.tensor(level, device=dev, dtype=torch.long)


def _probabilities64(s, b):
    """For each key head h of sequence b: (h, probabilities [G, t, n], lse [G, t])."""
    c, dev = s["case"], s["q"].device
    base, t = int(s["ctx"][b]), c["T"] if s["new"] is None else int(s["new"][b])
    n, Hkv, G = base + t, c["Hkv"], c["Hq"] // c["Hkv"]
    sees, level = _masks64(s, b, base, t)
    k = _rows64(s["k"], s["k_scale"], s["table"], b, n)
    for h in range(Hkv):
        q = s["q"][b, :t, h * G : (h + 1) * G].double().permute(1, 0, 2)
        x = q @ k[h].T / c["D"] ** 0.5
        if c["cap"]:
            x = c["cap"] * torch.tanh(x / c["cap"])
        pos = s["slot_pos"][b, h, :n].long() if s["slot_pos"] is not None else torch.cat([torch.arange(base, device=dev), base + level])
        far = pos[base:, None] - pos[None]
        if s["slopes"] is not None:
            x = x - s["slopes"][h * G : (h + 1) * G].double()[:, None, None] * far.abs().double()
        see = sees & (far < c["window"]) if c["window"] else sees
        x = x.masked_fill(~see, -math.inf)
        lse = torch.logsumexp(x, -1)
        yield h, torch.exp(x - lse.masked_fill(lse == -math.inf, 0.0)[..., None]), lse


def _attention64(s):
    c = s["case"]
    G = c["Hq"] // c["Hkv"]
    out = torch.zeros(c["B"], c["T"], c["Hq"], c["D"], dtype=torch.float64, device=s["q"].device)
    lse = torch.full((c["B"], c["T"], c["Hq"]), -math.inf, dtype=torch.float64, device=s["q"].device)
    for b in range(c["B"]):
        t = c["T"] if s["new"] is None else int(s["new"][b])
        v = _rows64(s["v"], s["v_scale"], s["table"], b, int(s["ctx"][b]) + t)
        for h, p, z in _probabilities64(s, b):
            out[b, :t, h * G : (h + 1) * G] = (p @ v[h]).permute(1, 0, 2)
            lse[b, :t, h * G : (h + 1) * G] = z.T
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}


def _mass64(s):
    mass = s["out"]["mass"].double()
    for b in range(s["case"]["B"]):
        k, base = int(s["accept"][b]), int(s["ctx"][b])
        rows = list(range(k + 1)) if s["nodes"] is None else [0] + s["nodes"][b, :k].tolist()
        for h, p, z in _probabilities64(s, b):
            w = p[:, rows].sum((0, 1))
            w[:base] += s["mass_in"][b, h, :base].double()
            mass[b, h, : w.shape[0]] = w
    return {"mass": mass}


def _norm_rope64(s):
    c = s["case"]
    B, T, Hq, Hkv, D, r = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], c["rotary"]
    x = s["qkv"].double().reshape(B, T, Hq + 2 * Hkv, D)
    head = x[:, :, : Hq + Hkv]
    head = head / torch.sqrt(head.pow(2).mean(-1, keepdim=True) + 1e-6)
    head[:, :, :Hq] *= s["q_weight"].double()
    head[:, :, Hq:] *= s["k_weight"].double()
    turned = head[..., :r]
    pairs = turned.reshape(B, T, -1, 2, r // 2).transpose(-1, -2) if c["layout"] == "half" else turned.reshape(B, T, -1, r // 2, 2)
    z = torch.view_as_complex(pairs.contiguous())
    where = s["positions"].double()
    where = where[..., None] if c["axes"] == 1 else torch.stack([where[..., a] for a in _sections(c)], -1)
    angle = (where * s["inv_freq"])[:, :, None]
    z = torch.view_as_real(z * torch.polar(torch.ones_like(angle), angle))
    head[..., :r] = z.transpose(-1, -2).reshape(B, T, -1, r) if c["layout"] == "half" else z.reshape(B, T, -1, r)
    q, k, v = head[:, :, :Hq].clone(), s["k"].double(), s["v"].double()
    for b in range(B):
        t = T if s["new"] is None else int(s["new"][b])
        q[b, t:] = 0.0
        slot = int(s["ctx"][b]) + torch.arange(t, device=x.device)
        page = s["table"][b].long()[slot // c["page"]]
        for pool, rows, scale in ((k, head[b, :t, Hq:], s["k_scale"]), (v, x[b, :t, Hq + Hkv :], s["v_scale"])):
            pool[page, slot % c["page"]] = rows if scale is None else (rows / scale.double()[:, None]).clamp(-448.0, 448.0)
    return {"q": q, "k": k, "v": v}
