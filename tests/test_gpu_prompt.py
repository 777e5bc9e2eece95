"""GPU tests of spv_prompt_attention against plain 64-bit forms
(scored_reference): lengths from one token to long ones, odd sizes, masks that
leave rows empty, caches that are split over many blocks."""
import math

import pytest
import torch

import scored_reference as sr
from kv_reference import half_step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def spv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import speculative_decoding_token_spv_gb300 as m
    return m


def documents(T, ctx, lengths, prefix=None):
    """(first, last) of the tokens of documents of these lengths in turn; the first goes on from the cache."""
    first, last, at, i = [], [], 0, 0
    while at < T:
        n = min(T - at, lengths[i % len(lengths)])
        first += [0 if at == 0 else ctx + at] * n
        last += [ctx + at + (n // 2 if prefix is None else prefix)] * n
        at, i = at + n, i + 1
    return first, last


DOCS = [documents(200, 0, [1, 70, 13, 128]), documents(200, 37, [64, 5])]
CASES = [
    # ctx, new, T, Hq, Hkv, D, page, order, dtype, kv, options
    ([0], None, 1, 1, 1, 64, 16, "nhd", "bf16", "bf16", dict()),
    ([0], None, 1, 32, 8, 128, 16, "nhd", "bf16", "bf16", dict(cap=50.0)),
    ([129], None, 3, 5, 1, 128, 16, "nhd", "f16", "f16", dict(slopes=True)),
    ([0], None, 127, 1, 1, 128, 16, "nhd", "bf16", "bf16", dict()),
    ([0], None, 128, 1, 1, 128, 16, "nhd", "f16", "f16", dict()),
    ([0], None, 129, 1, 1, 128, 16, "nhd", "bf16", "bf16", dict()),
    ([0, 5], [300, 1], 300, 2, 2, 64, 16, "hnd", "bf16", "bf16", dict(cap=20.0)),
    ([0, 500, 3], [257, 0, 200], 257, 4, 2, 128, 16, "nhd", "bf16", "bf16", dict(cap=50.0)),
    ([0, 500, 3], [257, 0, 200], 257, 3, 1, 128, 8, "nhd", "f16", "f16", dict(slopes=True, cap=30.0)),
    ([0, 500], None, 190, 7, 1, 64, 4, "nhd", "bf16", "bf16", dict(window=33)),
    ([0, 500], None, 190, 7, 1, 64, 128, "hnd", "bf16", "bf16", dict(window=1, slopes=True)),
    ([1000, 20], None, 260, 4, 2, 128, 32, "nhd", "bf16", "bf16", dict(window=200, cap=50.0)),
    ([1000, 20], None, 70, 8, 2, 256, 16, "nhd", "bf16", "bf16", dict(window=200, cap=50.0)),
    ([1000, 0], [70, 33], 70, 6, 2, 256, 8, "nhd", "f16", "f16", dict(slopes=True)),
    ([700, 0], [150, 33], 150, 4, 2, 256, 64, "nhd", "bf16", "e4m3", dict(cap=15.0)),
    ([700, 0], [150, 133], 150, 4, 2, 128, 16, "nhd", "bf16", "e4m3", dict(slopes=True)),
    ([700, 0], [150, 133], 150, 8, 2, 128, 4, "hnd", "f16", "e4m3", dict(window=300, cap=30.0)),
    ([300, 0], None, 130, 6, 2, 64, 16, "nhd", "f16", "e4m3", dict()),
    ([300, 11], None, 130, 6, 2, 128, 16, "nhd", "f16", "f16", dict(slopes=True, moved=True)),
    ([300, 11], None, 130, 6, 2, 64, 16, "nhd", "bf16", "bf16", dict(slopes=True, moved=True, window=150, cap=30.0)),
    ([300, 11], None, 40, 3, 1, 128, 16, "nhd", "bf16", "bf16", dict(moved=True, window=100)),
    ([300, 11], None, 70, 4, 1, 256, 16, "nhd", "bf16", "bf16", dict(moved=True, window=100, slopes=True)),
    ([0, 37], None, 200, 4, 2, 128, 16, "nhd", "bf16", "bf16", dict(first=[DOCS[0][0], DOCS[1][0]])),
    ([0, 37], None, 200, 4, 2, 64, 16, "nhd", "f16", "f16", dict(first=[DOCS[0][0], DOCS[1][0]], last=[DOCS[0][1], DOCS[1][1]])),
    ([0, 37], [200, 77], 200, 8, 1, 128, 16, "nhd", "f16", "f16", dict(first=[DOCS[0][0], DOCS[1][0]], last=[DOCS[0][1], DOCS[1][1]], slopes=True, window=20, cap=9.0)),
    ([0, 37], [200, 77], 200, 2, 1, 256, 16, "nhd", "bf16", "bf16", dict(first=[DOCS[0][0], DOCS[1][0]], last=[DOCS[0][1], DOCS[1][1]])),
    ([5], None, 300, 1, 1, 128, 16, "nhd", "bf16", "bf16", dict(last=[[300] * 300])),
    ([5], None, 300, 1, 1, 64, 16, "nhd", "bf16", "bf16", dict(first=[[306 if t % 3 == 0 else t // 2 for t in range(300)]])),  # rows that see nothing
    ([5], None, 300, 2, 1, 128, 16, "nhd", "bf16", "bf16", dict(first=[[310] * 300])),  # none does
    ([64], None, 280, 1, 1, 128, 16, "nhd", "f16", "f16", dict(first=[[(t * 37) % 344 for t in range(280)]], last=[[(t * 91) % 400 for t in range(280)]])),
    ([50], None, 150, 4, 2, 64, 16, "nhd", "bf16", "bf16", dict(cap=20.0, scale=-0.3)),
    ([50], None, 150, 4, 2, 128, 16, "nhd", "bf16", "bf16", dict(scale=-0.3)),
    ([50], None, 150, 4, 2, 128, 16, "nhd", "f16", "f16", dict(scale=0.0, slopes=True)),
    ([50], None, 150, 4, 2, 128, 16, "nhd", "f16", "f16", dict(cap=3.0, spread=60.0)),
    ([0], None, 1000, 3, 1, 128, 16, "nhd", "bf16", "bf16", dict()),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).replace(" ", "") for x in c[2:10]) + "-" + "-".join(c[10]))
def test_prompt(spv, case):
    c = sr.Case(spv, 41, *case[:10], **case[10])
    c.check(c.attend(prompt=True))


def test_without_scores_it_is_causal(spv):
    c = sr.Case(spv, 42, [30, 0], [170, 90], 170, 4, 2, 128, 16)
    a = c.attend(prompt=True)
    b = spv.spv_prompt_attention(c.q.cuda(), c.cache(), c.table.cuda(), c.i32(c.ctx), new_lens=c.i32(c.new), want_lse=True)
    assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])
    c.check(b)


@pytest.mark.parametrize("D,kv", [(64, "bf16"), (128, "bf16"), (128, "e4m3"), (256, "bf16")])
def test_long_cache_in_pieces(spv, D, kv):
    """A few tokens over a long cache: each item lies in many blocks."""
    c = sr.Case(spv, 43, [9001], None, 66, 2, 1, D, 64, dtype="bf16", kv=kv, cap=30.0, slopes=True, poison=False)
    a, b = c.attend(prompt=True), c.attend(prompt=True)
    assert torch.equal(a["out"], b["out"])
    c.check(a)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_short_sequences(spv, D):
    """More items than blocks, most of one tile."""
    new = [(53 * i) % 97 for i in range(90)]
    c = sr.Case(spv, 44, [(29 * i) % 70 for i in range(90)], new, 97, 8, 4, D, 16, cap=50.0, window=60, poison=False)
    a, b = c.attend(prompt=True), c.attend(prompt=True)
    assert torch.equal(a["out"], b["out"])
    c.check(a)


@pytest.mark.parametrize("D,T", [(64, 150), (128, 150), (256, 100), (128, 30)])
def test_infinities_that_a_row_does_not_see(spv, D, T):
    """Infinities in V behind a token and before its document have no effect on it; those that it sees do."""
    half = T // 2
    c = sr.Case(spv, 45, [40], None, T, 4, 2, D, 16, first=[[0] * half + [40 + half] * (T - half)], poison=False)
    for j in (20, 40 + half - 1):  # cached; the last of the first document
        c.v[c.table[0, j // 16].long(), j % 16, 0, 5] = math.inf
        c.v[c.table[0, j // 16].long(), j % 16, 1, 7] = math.nan
    x = c.attend(prompt=True)["out"].cpu().float()
    bad = torch.zeros_like(x, dtype=torch.bool)
    bad[0, :half, :2, 5] = bad[0, :half, 2:, 7] = True
    assert (x[0, :half, :2, 5] == math.inf).all() and torch.isnan(x[0, :half, 2:, 7]).all()
    assert torch.isfinite(x[~bad]).all()
    c.v = torch.nan_to_num(c.v, nan=0.0, posinf=0.0)
    out, lse, bound, _ = c.attention()
    assert ((x.double() - out).abs() <= half_step(c.q.dtype) * (out.abs() + bound) + bound)[~bad].all()


def test_bad_pages_and_lengths(spv):
    c = sr.Case(spv, 46, [300, 300, 300, 5, 7], None, 100, 4, 2, 64, 16, window=64)
    table = c.table.clone()
    table[0, 2] = -1
    table[1, 17] = c.k.shape[0] + 3
    ctx = list(c.ctx)
    ctx[3], ctx[4] = 100000, -1
    got = spv.spv_prompt_attention(c.q.cuda(), c.cache(), table.cuda(), c.i32(ctx), c.scores(), want_lse=True)
    assert got["row_status"].tolist() == [0, 4, 0, 4, 4]
    x = got["out"].cpu()
    assert torch.isnan(x[1, :34]).all()  # the tokens whose window reaches slot 287
    assert torch.isnan(x[3:]).all() and torch.isnan(got["lse"][3:]).all()
    out, *_ = c.attention()
    assert ((x[[0, 2]].double() - out[[0, 2]]).abs() <= 0.03).all()


@pytest.mark.parametrize("block,item", [(0, 0), (40, 0), (151, 0)])
@pytest.mark.parametrize("D", [128, 256])
def test_a_wait_that_gives_up_leaves_nan_and_status(spv, D, block, item):
    c = sr.Case(spv, 47, [(100 * i) % 700 for i in range(12)], None, 150, 8, 4, D, 16, poison=False)
    ws = spv.new_workspace(spv.spv_prompt_workspace_bytes(12, 150, 8, 4, D), "cuda")
    good = c.attend(prompt=True, workspace=ws)
    spv.spv_selftest_give_up(block, item)
    try:
        got = c.attend(prompt=True, workspace=ws)
    finally:
        spv.spv_selftest_give_up(-1)
    status = got["row_status"].cpu()
    lost = torch.isnan(got["out"]).any(-1).cpu()
    assert (status == 5).any() and set(status.tolist()) <= {0, 5}
    assert lost.any() and not lost.all()
    assert torch.isnan(got["lse"]).cpu()[lost].all()
    assert torch.equal(got["out"].cpu()[~lost], good["out"].cpu()[~lost])
    assert spv.spv_workspace_status(ws) == spv.SPV_ERR_TIMEOUT
    ws.zero_()
    again = c.attend(prompt=True, workspace=ws)
    assert torch.equal(again["out"], good["out"])


def test_captured_and_replayed(spv):
    c = sr.Case(spv, 48, [100, 0], None, 150, 8, 2, 128, 16, cap=50.0, window=90)
    q, cache, table, ctx, scores = c.q.cuda(), c.cache(), c.table.cuda(), c.i32(c.ctx), c.scores()
    ws = spv.new_workspace(spv.spv_prompt_workspace_bytes(2, 150, 8, 2, 128), q.device)
    out = spv.spv_prompt_attention(q, cache, table, ctx, scores, workspace=ws, want_lse=True)
    want = {k: v.clone() for k, v in out.items()}
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        spv.spv_prompt_attention(q, cache, table, ctx, scores, workspace=ws, want_lse=True, out=out)
    for v in out.values():
        v.fill_(7)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[k], want[k]) for k in want)


def test_two_streams_with_their_own_workspaces(spv):
    c = sr.Case(spv, 49, [100, 0], None, 200, 8, 2, 64, 16, cap=50.0)
    want = c.attend(prompt=True)["out"]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [c.attend(prompt=True, stream=s)["out"] for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("D,T,B", [(64, 70, 90), (128, 66, 70), (256, 34, 40)])
def test_blocks_of_many_items_of_a_tile_or_two(spv, D, T, B, kv):
    """A block's copies run ahead of its rows by several whole items."""
    c = sr.Case(spv, 71, [(3 * b) % 7 for b in range(B)], None, T, 8 if D == 256 else 16, 4, D, 16, "nhd", "bf16", kv)
    c.check(c.attend(prompt=True))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_blocks_of_many_items_without_tiles(spv, D, kv):
    """Most rows are padding: items that see nothing lie between those that do, and behind them."""
    new = [(0, 1, 300, 0, 2, 70)[b % 6] for b in range(30)]
    c = sr.Case(spv, 72, [(11 * b) % 90 for b in range(30)], new, 300, 8, 2, D, 16, "nhd", "bf16", kv)
    c.check(c.attend(prompt=True))
