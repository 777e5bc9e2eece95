"""GPU tests of the calls with scores where they went wrong or nearly: pages that
were given back, pages outside the pool beside other items, masks near the ends
of 32 bits, rows of q next to nothing, trees of many short sequences."""
import pytest
import torch

import scored_reference as sr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def spv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import speculative_decoding_token_spv_gb300 as m
    return m


# ------------------------------------------------------------------ pages that were given back
def without_passed_pages(c, page):
    """The page table with every page that ends before the first slot that its sequence's tokens can see outside the pool."""
    table = c.table.clone()
    for b in range(c.B):
        if c.new[b] == 0:
            continue
        lowest = c.ctx[b] - c.window + 1 if c.window else 0
        if c.first is not None:
            lowest = max(lowest, int(c.first[b, : c.new[b]].min()))
        gone = max(0, min(lowest, c.ctx[b] + c.new[b] - 1)) // page
        table[b, :gone] = torch.tensor([-1, c.k.shape[0] + 5])[torch.arange(gone) % 2].to(torch.int32)
    return table


def check_without_passed_pages(c, page, prompt=False):
    table, whole = without_passed_pages(c, page), c.table
    assert (table != whole).any()
    c.table = table
    got = c.attend(prompt=prompt)
    c.table = whole
    c.check(got)


GONE = [((300, 5, 131, 448, 64), None, 64), ((1000, 777, 12), None, 100), ((700, 333), [[650, 651], [201, 333]], 0),
        ((700, 333), [[600, 702], [50, 0]], 77)]


@pytest.mark.parametrize("page", [1, 8, 16, 32])
@pytest.mark.parametrize("D,kv", [(64, "bf16"), (128, "f16"), (128, "e4m3"), (256, "bf16"), (256, "e4m3")])
@pytest.mark.parametrize("ctx,first,window", GONE, ids=["64", "100", "first", "both"])
def test_pages_before_the_first_slot_that_is_seen_few_rows(spv, ctx, first, window, D, kv, page):
    check_without_passed_pages(sr.Case(spv, 51, ctx, None, 2, 4, 2, D, page, "nhd", "f16" if kv == "f16" else "bf16", kv, first=first,
                                       window=window, cap=30.0), page)


@pytest.mark.parametrize("page", [1, 8, 16, 128])
@pytest.mark.parametrize("Hq,D,kv", [(2, 64, "bf16"), (4, 128, "f16"), (8, 128, "bf16"), (8, 128, "e4m3"), (4, 256, "bf16"), (4, 256, "e4m3")])
@pytest.mark.parametrize("first", [False, True])
def test_pages_before_the_first_slot_that_is_seen_many_rows(spv, first, Hq, D, kv, page):
    """20, 40 and 80 rows a key head: a row stands in tensor memory four times, twice, once."""
    ctx, T = (300, 5, 131, 1000, 517), 20 if D < 256 else 40
    begins = [[max(0, n - 40 + t) for t in range(T)] for n in ctx] if first else None
    check_without_passed_pages(sr.Case(spv, 52, ctx, None, T, Hq, 2, D, page, "nhd", "f16" if kv == "f16" else "bf16", kv,
                                       first=begins, window=0 if first else 64, slopes=True), page)


@pytest.mark.parametrize("page", [4, 16, 64])
@pytest.mark.parametrize("T,D,kv", [(1, 128, "bf16"), (70, 64, "f16"), (100, 128, "bf16"), (200, 128, "e4m3"), (70, 256, "bf16")])
@pytest.mark.parametrize("first", [False, True])
def test_pages_before_the_first_slot_that_is_seen_prompts(spv, first, T, D, kv, page):
    ctx = (300, 45, 1000, 517)
    begins = [[max(0, n - 31 + t // 2) for t in range(T)] for n in ctx] if first else None
    check_without_passed_pages(sr.Case(spv, 53, ctx, [T, 1, T - T // 3, T], T, 6, 2, D, page, "nhd", "f16" if kv == "f16" else "bf16", kv,
                                       first=begins, window=0 if first else 40), page, prompt=True)


@pytest.mark.parametrize("D", [64, 128])
def test_a_page_outside_the_pool_ends_with_its_item(spv, D):
    """The second tile of rows of the first sequence begins its document late: it is done before the page outside the pool,
    at the first's beginning, is asked for.  The items that its block goes on with have nothing to do with that page."""
    B, T, ctx, page = 2500, 256, 4000, 16
    gen = torch.Generator(device="cuda").manual_seed(54)
    q = torch.randn(B, T, 1, D, generator=gen, device="cuda").bfloat16()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    lens[0] = ctx
    pages = (ctx + T) // page
    k, v = (torch.randn(pages + B * 16, page, 1, D, generator=gen, device="cuda").bfloat16() for _ in range(2))
    table = torch.full((B, pages), -1, dtype=torch.int32, device="cuda")
    table[0] = torch.arange(pages, device="cuda")
    table[1:, :16] = pages + torch.arange((B - 1) * 16, device="cuda", dtype=torch.int32).reshape(B - 1, 16)
    first = torch.zeros(B, T, dtype=torch.int32, device="cuda")
    first[0, 128:] = ctx + 128
    scores = spv.Scores(first=first)
    want = spv.spv_prompt_attention(q, spv.KVCache(k, v), table, lens, scores, want_lse=True)
    table[0, 1] = -1
    got = spv.spv_prompt_attention(q, spv.KVCache(k, v), table, lens, scores, want_lse=True)
    assert want["row_status"].sum() == 0 and got["row_status"][0] == 4 and got["row_status"][1:].sum() == 0
    assert torch.isnan(got["out"][0, :128]).all()
    assert torch.equal(got["out"][1:], want["out"][1:]) and torch.equal(got["lse"][1:], want["lse"][1:])


# ------------------------------------------------------------------ masks near the ends of 32 bits
LEAST, MOST = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("T,D", [(3, 64), (30, 64), (30, 256)])
def test_documents_and_prefixes_at_the_ends_of_32_bits(spv, T, D):
    """`last` at its least is no prefix, `first` at its least the sequence's beginning; at their most, all and nothing."""
    ends = [LEAST, LEAST + 1, -1, 0, MOST]
    last = [[ends[(t + b) % 5] for t in range(T)] for b in range(2)]
    first = [[ends[(t + b) % 4] for t in range(T)] for b in range(2)]
    first[1][T - 1] = MOST
    c = sr.Case(spv, 55, [150, 70], None, T, 4, 2, D, 16, first=first, last=last)
    c.check(c.attend())


def test_weights_of_keys_of_documents_at_the_ends_of_32_bits(spv):
    T = 4
    c = sr.Case(spv, 56, [150, 70], None, T, 4, 2, 64, 16, first=[[LEAST, 0, 5, LEAST + 3]] * 2, last=[[LEAST, LEAST + 9, -1, MOST]] * 2)
    lse, W = c.attention()[1].float().cuda(), 160
    out = {"mass": torch.zeros(2, 2, W, device="cuda")}
    got = spv.spv_attention_mass_scored(c.q.cuda(), lse, c.cache(), c.table.cuda(), c.i32(c.ctx), c.i32([T - 1] * 2), c.scores(), out=out)
    want, bound = c.mass([list(range(T))] * 2, 1.0, torch.zeros(2, 2, W))
    there = ~torch.isnan(want)
    assert ((got["mass"].cpu().double() - want).abs() <= bound + 2.0 ** -24 * want.abs())[there].all()


@pytest.mark.parametrize("window", [MOST, MOST - 17, 2 ** 30])
@pytest.mark.parametrize("T,Hq,D,kv", [(3, 4, 64, "bf16"), (60, 4, 64, "bf16"), (60, 4, 128, "e4m3"), (33, 8, 256, "bf16")])
def test_trees_under_a_window_as_wide_as_32_bits(spv, T, Hq, D, kv, window):
    """Nodes next to the root that stand far behind it: a window that reaches further than any slot takes nothing away."""
    c = sr.Case(spv, 57, [64, 31, 500], None, T, Hq, 2, D, 16, "nhd", "bf16", kv, tree=True, window=window)
    c.parent[0, 1:] = 0
    c.seen = [c._seen(b) for b in range(c.B)]
    c.check(c.attend())


# ------------------------------------------------------------------ rows of q next to nothing
@pytest.mark.parametrize("prompt", [False, True])
@pytest.mark.parametrize("moved", [False, True])
@pytest.mark.parametrize("D,kv,size", [(128, "e4m3", 1e-33), (64, "e4m3", 1e-37), (256, "e4m3", 1e-33), (128, "bf16", 1e-33)])
def test_a_bias_beside_rows_of_q_next_to_nothing(spv, moved, prompt, D, kv, size):
    """All that tells keys apart is then the bias, and keys far away still count."""
    c = sr.Case(spv, 58, [700, 90], None, 66 if prompt else 40, 4, 2, D, 16, "nhd", "bf16", kv, slopes=True, moved=moved)
    c.slopes = torch.exp2(-6.0 - torch.arange(4.0))
    c.q[:, ::2] *= size
    c.check(c.attend(prompt=prompt))


@pytest.mark.parametrize("T", [2, 40])
@pytest.mark.parametrize("moved", [False, True])
def test_a_bias_beside_a_scale_next_to_nothing(spv, moved, T):
    c = sr.Case(spv, 59, [700, 90], None, T, 4, 2, 128, 16, slopes=True, moved=moved, scale=1e-39)
    c.slopes = torch.exp2(-6.0 - torch.arange(4.0))
    c.check(c.attend())


@pytest.mark.parametrize("T,Hq,D,kv", [(30, 2, 64, "f16"), (60, 2, 128, "bf16"), (60, 4, 128, "e4m3"), (40, 8, 256, "bf16"), (200, 4, 128, "bf16")])
def test_the_bias_of_near_keys_has_their_size(spv, T, Hq, D, kv):
    """Rows that see themselves or few keys before them, scores next to nothing: what is off is off by the bias of those
    keys, not of a tile's."""
    c = sr.Case(spv, 68, [191, 64, 500], None, T, Hq, 2, D, 16, "nhd", "f16" if kv == "f16" else "bf16", kv, window=1 + T % 7 // 3, slopes=True,
                spread=0.01)
    c.slopes = 1.0 - 0.11 * torch.rand(Hq, generator=c.gen)
    c.check(c.attend(prompt=T > 64))


# ------------------------------------------------------------------ trees of many short sequences
@pytest.mark.parametrize("T,Hq,D", [(64, 6, 128), (64, 6, 64), (40, 8, 256), (20, 4, 256)])
@pytest.mark.parametrize("seed", range(2))
def test_every_short_sequence_has_its_own_tree(spv, T, Hq, D, seed):
    """Items of a tile or two: the depths of the next items' trees are on their way while a row still needs its own."""
    ctx = [(17 * b) % 40 for b in range(160)]
    c = sr.Case(spv, 60 + seed, ctx, None, T, Hq, 2, D, 16, tree=True, slopes=True, cap=20.0, poison=False)
    a, b = c.attend(), c.attend()
    assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])
    c.check(a)




# ------------------------------------------------------------------ norms and rotation of many short sequences
@pytest.mark.parametrize("B,T,rotary,interleaved", [(4100, 1, 128, False), (2000, 2, 128, True), (1300, 3, 36, False), (950, 5, 64, False), (500, 9, 128, False)])
def test_many_short_sequences_are_appended_as_each_by_itself(spv, B, T, rotary, interleaved):
    """Whatever number of tokens a block takes: the same bits as from calls of a few sequences."""
    Hq, Hkv, D, page = 6, 2, 128, 4
    gen = torch.Generator(device="cuda").manual_seed(67)
    draw = lambda *shape: torch.randn(*shape, generator=gen, device="cuda").bfloat16()  # noqa: E731
    q, k, v = draw(B, T, Hq + 2 * Hkv, D).split([Hq, Hkv, Hkv], dim=2)
    per = (T + 8) // page + 1
    table = torch.randperm(B * per, generator=gen, device="cuda").to(torch.int32).reshape(B, per)
    ctx = torch.randint(0, 8, (B,), generator=gen, device="cuda", dtype=torch.int32)
    new = torch.randint(0, T + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
    qw, kw = (1 + torch.rand(D, generator=gen, device="cuda") for _ in range(2))
    freqs = spv.spv_rope_frequencies(rotary)
    got = []
    for step in (B, 100):
        cache = spv.KVCache(*(torch.zeros(B * per, page, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
        out = [spv.spv_norm_rope_append(q[i:i + step], k[i:i + step], v[i:i + step], cache, table[i:i + step], ctx[i:i + step], freqs, q_weight=qw,
                                        k_weight=kw, interleaved=interleaved, new_lens=new[i:i + step]) for i in range(0, B, step)]
        got.append((torch.cat([x["q"] for x in out]), torch.cat([x["row_status"] for x in out]), cache.k, cache.v))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert (got[0][1] == 0).all() and (got[0][0][new > 0][:, 0] != 0).any(-1).all()


# ------------------------------------------------------------------ few rows in tiles
@pytest.mark.parametrize("D,width", [(256, 600), (128, 32000)])
@pytest.mark.parametrize("T,Hq,tree,kw", [(1, 4, False, dict(cap=30.0)), (1, 16, False, dict(slopes=True)), (7, 4, True, dict(slopes=True)),
                                          (5, 6, False, dict(window=2 ** 30, cap=30.0, first=[[3 * t for t in range(5)]] * 4)),
                                          (8, 4, True, dict(moved=True, window=90, slopes=True))])
def test_few_rows_of_a_table_with_room_for_large_caches(spv, D, width, T, Hq, tree, kw):
    """How long the caches are only the page table's width tells the host: few rows go in tiles from 64 MB (heads of 256) or
    1 GB (heads of 128) of room on, whatever lies in them."""
    c = sr.Case(spv, 65, [300, 0, 41, 1000], [T, T, 0, T - T // 3], T, Hq, 2, D, 16, tree=tree, **kw)
    assert 4.0 * D * 2 * 4 * 16 * width > (64e6 if D == 256 else 1e9)
    table = torch.full((4, width), -1, dtype=torch.int32)
    table[:, : c.table.shape[1]] = c.table
    c.table = table
    ws = spv.new_workspace(spv.spv_attention_workspace_bytes(4, T, Hq, 2, D), "cuda")
    got = c.attend(workspace=ws)
    c.check(got)
    e = sr.Case(spv, 66, [300, 0, 41, 1000], [T, T, 0, T - T // 3], T, Hq, 2, D, 16, "nhd", "bf16", "e4m3", tree=tree, **kw)
    e.table = torch.cat([e.table, torch.full((4, width - e.table.shape[1]), -1, dtype=torch.int32)], 1)
    e.check(e.attend(workspace=ws))  # which stays where it was
