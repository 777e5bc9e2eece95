"""GPU tests of spv_norm_rope_append, spv_paged_attention_scored and
spv_attention_mass_scored against plain 64-bit forms (scored_reference), at the
sizes, masks and inputs where they can go wrong.  Tolerances: half a step of the
type plus the bounds that scored_reference derives."""
import math

import pytest
import torch

import kv_reference as ref
import scored_reference as sr
from kv_reference import DTYPES, half_step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def spv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import speculative_decoding_token_spv_gb300 as m
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ norms and rotation
NORM_CASES = [
    # ctx, new, T, Hq, Hkv, D, rotary, interleaved, axes, page, order, dtype, kv
    ([0], None, 1, 1, 1, 8, 8, False, 1, 16, "nhd", "bf16", "bf16"),
    ([777], None, 1, 32, 8, 128, 128, False, 1, 16, "nhd", "bf16", "bf16"),
    ([3, 60], None, 5, 8, 2, 128, 128, True, 3, 16, "hnd", "f16", "f16"),
    ([3, 60, 0], [5, 0, 2], 5, 10, 2, 64, 32, False, 2, 4, "nhd", "f16", "f16"),
    ([31, 1], None, 3, 6, 3, 256, 128, False, 1, 32, "nhd", "bf16", "bf16"),
    ([31, 1], None, 3, 6, 3, 256, 256, True, 3, 32, "nhd", "bf16", "e4m3"),
    ([100], None, 7, 4, 4, 96, 36, False, 2, 16, "nhd", "f16", "f16"),
    ([100], None, 7, 4, 4, 96, 36, True, 2, 16, "nhd", "bf16", "e4m3"),
    ([9, 2], None, 4, 5, 1, 80, 80, False, 1, 1, "nhd", "bf16", "bf16"),
    ([9, 2], None, 2, 3, 1, 48, 6, False, 1, 2, "nhd", "f16", "e4m3"),
    ([5], None, 2, 2, 2, 64, 0, False, 1, 8, "nhd", "bf16", "bf16"),
    ([17, 900], [700, 650], 700, 16, 4, 64, 64, False, 3, 16, "hnd", "bf16", "bf16"),
    ([0, 4000], None, 2500, 2, 1, 128, 64, False, 1, 64, "nhd", "f16", "f16"),
]


def norm_inputs(case, seed):
    ctx, new, T, Hq, Hkv, D, rotary, interleaved, axes, page, order, dtype, kv = case
    gen = torch.Generator().manual_seed(seed)
    B = len(ctx)
    lens = [c + n for c, n in zip(ctx, new or [T] * B)]
    k, v, ks, vs, table = ref.make_cache(gen, lens, page, Hkv, D, kv, order, garbage=False)
    x = (torch.randn(B, T, Hq + 2 * Hkv, D, generator=gen) * torch.exp(torch.randn(B, T, Hq + 2 * Hkv, 1, generator=gen))).to(DTYPES[dtype])
    weights = [1 + 0.3 * torch.randn(D, generator=gen) for _ in range(2)]
    inv = [10000.0 ** (-2.0 * i / rotary) for i in range(rotary // 2)]
    pos = torch.randint(0, 200000, (B, T, axes), generator=gen, dtype=torch.int32)
    ax = torch.randint(0, axes, (rotary // 2,), generator=gen, dtype=torch.int32) if axes > 1 else None
    return gen, k, v, ks, vs, table, x, weights, inv, pos, ax


def rope_tolerance(want, x, scale, dtype):
    """Half a step of the type, and in 32 bits: the head's norm and its products (8 roundings), the angle (2^-31) and its
    sine, of the size of the largest element of the pair's head."""
    step = torch.finfo(dtype).eps / 2
    least = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    size = want.abs().amax(-1, keepdim=True)
    return step * want.abs() + 2.0 ** -19 * size + least / 2


@pytest.mark.parametrize("case", NORM_CASES, ids=lambda c: "-".join(str(x).replace(" ", "") for x in c[2:]))
@pytest.mark.parametrize("normed", ["both", "q", "none"])
def test_norm_rope(spv, case, normed):
    ctx, new, T, Hq, Hkv, D, rotary, interleaved, axes, page, order, dtype, kv = case
    gen, k, v, ks, vs, table, x, weights, inv, pos, ax = norm_inputs(case, 11)
    B, fresh = len(ctx), new or [T] * len(ctx)
    to = lambda p: p.transpose(1, 2).contiguous().cuda().transpose(1, 2) if order == "hnd" else p.contiguous().cuda()  # noqa: E731
    cache = spv.KVCache(to(k), to(v), None if ks is None else ks.cuda(), None if vs is None else vs.cuda())
    qw = weights[0] if normed in ("both", "q") else None
    kw = weights[1] if normed == "both" else None
    freqs = spv.spv_rope_frequencies(rotary) if rotary else torch.empty(0, dtype=torch.int64, device="cuda")
    slot_pos = torch.full((B, Hkv, max(ctx) + T), -5, dtype=torch.int32, device="cuda")
    q, kk, vv = x.cuda().split([Hq, Hkv, Hkv], dim=2)
    got = spv.spv_norm_rope_append(q, kk, vv, cache, table.cuda(), i32(ctx), freqs, q_weight=None if qw is None else qw.cuda(),
                                   k_weight=None if kw is None else kw.cuda(), eps=1e-5, axes=None if ax is None else ax.cuda(),
                                   interleaved=interleaved, mscale=1.25, positions=(pos if axes > 1 else pos[..., 0]).cuda().contiguous(),
                                   new_lens=None if new is None else i32(new), slot_pos=slot_pos)
    torch.cuda.synchronize()
    assert (got["row_status"].cpu() == 0).all()
    want_q = sr.norm_rope(x[:, :, :Hq], qw, 1e-5, pos, ax, inv, interleaved, 1.25)
    want_k = sr.norm_rope(x[:, :, Hq:Hq + Hkv], kw, 1e-5, pos, ax, inv, interleaved, 1.25)
    gq, gk, gv = got["q"].cpu().double(), cache.k.cpu(), cache.v.cpu()
    before_k, before_v = ref.bits(k).clone(), ref.bits(v).clone()
    for b in range(B):
        n = fresh[b]
        assert ((gq[b, :n] - want_q[b, :n]).abs() <= rope_tolerance(want_q[b, :n], x, 1.0, DTYPES[dtype])).all()
        assert (gq[b, n:] == 0).all()
        rk, rv = ref.rows(gk, table[b], ctx[b] + n)[ctx[b]:], ref.rows(gv, table[b], ctx[b] + n)[ctx[b]:]
        wk, wv = want_k[b, :n], x[b, :n, Hq + Hkv:].double()
        if ks is not None:
            wk, wv = (wk / ks.double()[:, None]).clamp(-448, 448), (wv / vs.double()[:, None]).clamp(-448, 448)
            # a quotient of 32 bits next to the middle of two e4m3 values may round to either: half a step more of 2^-19
            assert ((rv - wv).abs() <= 2.0 ** -4 * wv.abs() * (1 + 2.0 ** -18) + 2.0 ** -10).all()
        else:
            assert torch.equal(rv, wv)
        assert ((rk - wk).abs() <= rope_tolerance(wk, x, 1.0, DTYPES[kv]) * (1 + 2.0 ** -18)).all()
        assert torch.equal(slot_pos[b, :, ctx[b]:ctx[b] + n].cpu(), pos[b, :n, 0].expand(Hkv, n))
        assert (slot_pos[b, :, ctx[b] + n:] == -5).all()
        used = torch.zeros(k.shape[:2], dtype=torch.bool)
    for b in range(B):
        for j in range(ctx[b], ctx[b] + fresh[b]):
            used[table[b, j // page].long(), j % page] = True
    assert torch.equal(ref.bits(gk)[~used], before_k[~used]) and torch.equal(ref.bits(gv)[~used], before_v[~used])


def test_norm_rope_in_place_and_default_positions(spv):
    gen = torch.Generator().manual_seed(5)
    B, T, Hq, Hkv, D = 2, 6, 4, 2, 128
    ctx = [13, 40]
    k, v, ks, vs, table = ref.make_cache(gen, [c + T for c in ctx], 16, Hkv, D, "bf16", garbage=False)
    q, kk, vv = (torch.randn(B, T, h, D, generator=gen).bfloat16().cuda() for h in (Hq, Hkv, Hkv))
    w = (1 + torch.rand(D, generator=gen)).cuda()
    freqs = spv.spv_rope_frequencies(D)
    results = []
    for where in ("apart", "in place"):
        cache = spv.KVCache(k.clone().cuda(), v.clone().cuda())
        mine = q.clone()
        got = spv.spv_norm_rope_append(mine, kk, vv, cache, table.cuda(), i32(ctx), freqs, q_weight=w, k_weight=w,
                                       positions=None if where == "apart" else (i32(ctx)[:, None] + torch.arange(T, device="cuda", dtype=torch.int32)).contiguous(),
                                       out={"q": mine} if where == "in place" else None)
        results.append((got["q"].clone(), cache.k, cache.v))
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_norm_rope_bad_sequences(spv):
    """A page outside the pool, and lengths beyond the table: nothing cached there, q as usual or 0, status set."""
    gen = torch.Generator().manual_seed(6)
    B, T, Hq, Hkv, D = 3, 2, 2, 1, 64
    ctx = [14, 5, 1000]
    k, v, ks, vs, table = ref.make_cache(gen, [16, 7, 2], 16, Hkv, D, "f16", garbage=False)
    table[0, 0] = k.shape[0]
    cache = spv.KVCache(k.cuda(), v.cuda())
    q, kk, vv = (torch.randn(B, T, h, D, generator=gen).half().cuda() for h in (Hq, Hkv, Hkv))
    w = torch.ones(D, device="cuda")
    got = spv.spv_norm_rope_append(q, kk, vv, cache, table.cuda(), i32(ctx), spv.spv_rope_frequencies(D), q_weight=w, k_weight=w)
    assert got["row_status"].tolist() == [4, 0, 4]
    assert (got["q"][0] != 0).any() and (got["q"][2] == 0).all()
    changed = (cache.k.cpu() != k).flatten(2).any(-1)
    assert changed.sum() == 2 and changed[table[1, 0].long(), 5:7].all()


# ------------------------------------------------------------------ attention
ATT_CASES = [
    # ctx, new, T, Hq, Hkv, D, page, order, dtype, kv, options
    ([0], None, 1, 1, 1, 64, 16, "nhd", "bf16", "bf16", dict(cap=50.0)),
    ([777], None, 1, 32, 8, 128, 16, "nhd", "bf16", "bf16", dict(cap=50.0)),
    ([777, 3], None, 1, 8, 2, 128, 1, "nhd", "f16", "f16", dict(cap=5.0, window=100)),
    ([63, 64, 65, 300, 1], None, 1, 4, 2, 64, 16, "hnd", "bf16", "bf16", dict(window=64)),
    ([500, 64], None, 4, 6, 2, 256, 16, "nhd", "bf16", "bf16", dict(cap=30.0, window=129, slopes=True)),
    ([500, 64], [4, 2], 4, 6, 2, 256, 16, "nhd", "bf16", "e4m3", dict(cap=30.0, slopes=True)),
    ([130, 700], [3, 0], 3, 8, 2, 128, 64, "nhd", "f16", "e4m3", dict(window=50)),
    ([130, 700], None, 5, 8, 2, 128, 32, "hnd", "f16", "f16", dict(slopes=True, moved=True)),
    ([130, 700], None, 5, 8, 2, 64, 8, "nhd", "bf16", "bf16", dict(slopes=True, moved=True, window=90, cap=20.0)),
    ([130, 70], None, 3, 3, 1, 128, 16, "nhd", "bf16", "bf16", dict(window=33, moved=True)),
    ([200, 90], None, 4, 4, 1, 128, 16, "nhd", "f16", "f16", dict(first=[[100, 150, 201, 204], [0, 91, 92, 93]])),
    ([200, 90], None, 4, 4, 2, 64, 16, "nhd", "bf16", "bf16", dict(last=[[204, 202, 0, -4], [91, 94, 1000, 92]])),
    ([200, 90], None, 4, 4, 2, 64, 16, "nhd", "bf16", "bf16", dict(first=[[0, 202, 203, 203], [95, 0, 50, 92]], last=[[204, 204, 203, 0], [94, 94, 94, 94]], window=3)),
    ([256, 31], None, 21, 8, 2, 128, 16, "nhd", "f16", "f16", dict(tree=True, cap=30.0, first=[[40] * 21, [7] * 21])),
    ([250, 31, 0], [21, 17, 1], 21, 32, 8, 128, 16, "hnd", "bf16", "bf16", dict(tree=True, slopes=True)),
    ([250, 31, 0], [21, 17, 1], 21, 8, 8, 64, 16, "nhd", "bf16", "bf16", dict(tree=True, slopes=True, window=4)),
    ([70, 129], None, 63, 10, 2, 128, 32, "nhd", "f16", "e4m3", dict(tree=True, window=5, cap=9.0)),
    ([100], None, 64, 16, 1, 64, 16, "nhd", "bf16", "bf16", dict(tree=True, moved=True, slopes=True)),
    ([70, 129], None, 40, 6, 2, 256, 16, "nhd", "bf16", "bf16", dict(slopes=True, window=60)),
    ([70, 129], None, 40, 6, 2, 256, 16, "nhd", "f16", "e4m3", dict(tree=True, cap=50.0)),
    ([40], None, 33, 64, 1, 128, 16, "nhd", "bf16", "bf16", dict(window=7)),
    ([3000, 2], None, 16, 8, 2, 128, 128, "nhd", "bf16", "bf16", dict(window=1000, cap=50.0)),
    ([3000, 2], None, 30, 4, 1, 128, 4, "nhd", "bf16", "bf16", dict(window=1000, slopes=True)),
    ([6000], None, 6, 5, 1, 128, 128, "nhd", "bf16", "bf16", dict(cap=1e5, slopes=True)),
    ([150], None, 2, 4, 2, 64, 16, "nhd", "bf16", "bf16", dict(cap=2.0, spread=40.0)),
    ([150], None, 2, 4, 2, 64, 16, "nhd", "bf16", "bf16", dict(cap=20.0, scale=-0.3)),
    ([150], None, 9, 4, 2, 64, 16, "nhd", "bf16", "bf16", dict(slopes=True, scale=0.0)),
    ([150], None, 20, 4, 2, 128, 16, "nhd", "f16", "f16", dict(cap=20.0, scale=-0.3)),
    ([150], None, 20, 4, 2, 64, 16, "nhd", "f16", "f16", dict()),
]


@pytest.mark.parametrize("case", ATT_CASES, ids=lambda c: "-".join(str(x).replace(" ", "") for x in c[2:10]) + "-" + "-".join(c[10]))
def test_attention(spv, case):
    c = sr.Case(spv, 21, *case[:10], **case[10])
    c.check(c.attend())


def test_neutral_scores_are_plain_attention(spv):
    """Without cap, bias and masks the call is spv_paged_attention's, to its rounding."""
    c = sr.Case(spv, 3, [300, 5], [5, 3], 5, 16, 2, 128, 16)
    got = c.attend()
    plain = spv.spv_paged_attention(c.q.cuda(), c.cache(), c.table.cuda(), c.i32(c.ctx), new_lens=c.i32(c.new), want_lse=True)
    c.check(got)
    c.check(plain)


@pytest.mark.parametrize("T,D", [(3, 128), (40, 128), (40, 64), (40, 256)])
def test_infinities_that_a_row_does_not_see(spv, T, D):
    """Infinities and NaN in V of slots that some rows see and others do not, at a window's edge and in a document before
    the row's own: only the rows that see them have them."""
    first = [[20] * (T // 2) + [150] * (T - T // 2)]
    c = sr.Case(spv, 8, [300], None, T, 4, 2, D, 16, first=first, poison=False)
    at = (c.table[0, 100 // 16].long(), 100 % 16)
    c.v[at][0, 5] = math.inf
    c.v[at][1, 7] = math.nan
    got = c.attend()
    x = got["out"].cpu().float()
    early, late = x[0, : T // 2], x[0, T // 2:]
    assert (early[:, :2, 5] == math.inf).all() and torch.isnan(early[:, 2:, 7]).all()
    assert torch.isfinite(late).all()
    bad = torch.zeros_like(x, dtype=torch.bool)
    bad[0, : T // 2, :2, 5] = bad[0, : T // 2, 2:, 7] = True
    assert torch.isfinite(x[~bad]).all()
    c.v[at][0, 5] = c.v[at][1, 7] = 0.0
    out, lse, bound, _ = c.attention()
    tol = half_step(c.q.dtype) * (out.abs() + bound) + bound
    assert ((x.double() - out).abs() <= tol)[~bad].all()


@pytest.mark.parametrize("T", [2, 24])
def test_bad_pages_and_lengths(spv, T):
    """A page outside the pool before the window does not matter; one that is seen makes its sequence bad."""
    c = sr.Case(spv, 9, [300, 300, 300, 5], None, T, 4, 2, 64, 16, window=64)
    table = c.table.clone()
    table[0, 2] = -1
    table[1, 17] = c.k.shape[0] + 3
    ctx = list(c.ctx)
    ctx[3] = 100000
    got = spv.spv_paged_attention_scored(c.q.cuda(), c.cache(), table.cuda(), c.i32(ctx), c.scores(), want_lse=True)
    assert got["row_status"].tolist() == [0, 4, 0, 4]
    x = got["out"].cpu()
    assert torch.isnan(x[1]).all() and torch.isnan(x[3]).all() and torch.isnan(got["lse"][3]).all()
    out, *_ = c.attention()
    assert ((x[[0, 2]].double() - out[[0, 2]]).abs() <= 0.02).all()


def test_short_slot_pos_makes_a_sequence_bad(spv):
    c = sr.Case(spv, 10, [20, 50], None, 2, 2, 1, 64, 16, slopes=True, moved=True)
    scores = c.scores()
    scores.slot_pos = scores.slot_pos[:, :, :40].contiguous()
    got = spv.spv_paged_attention_scored(c.q.cuda(), c.cache(), c.table.cuda(), c.i32(c.ctx), scores)
    assert got["row_status"].tolist() == [0, 4]
    assert torch.isfinite(got["out"][0]).all() and torch.isnan(got["out"][1]).all()


@pytest.mark.parametrize("T,Hq,kv", [(1, 8, "bf16"), (5, 16, "bf16"), (5, 16, "e4m3"), (30, 16, "bf16")])
def test_many_sequences_share_the_blocks(spv, T, Hq, kv):
    """More items than blocks and items in several pieces, with windows that skip most of the long ones; twice the same."""
    ctx = [(977 * i) % 2600 for i in range(40)]
    c = sr.Case(spv, 12, ctx, None, T, Hq, 4, 64, 16, dtype="bf16", kv=kv, window=500, cap=30.0, poison=False)
    got = c.attend()
    again = c.attend()
    assert torch.equal(got["out"], again["out"]) and torch.equal(got["lse"], again["lse"])
    c.check(got)


def test_long_cache(spv):
    """Few sequences over a long cache: an item in many pieces."""
    c = sr.Case(spv, 13, [30011], None, 2, 8, 2, 64, 64, cap=50.0, slopes=True, poison=False)
    c.check(c.attend())


def test_captured_and_replayed(spv):
    c = sr.Case(spv, 14, [100, 900], None, 5, 16, 2, 128, 16, cap=50.0, window=300, first=[[3] * 5, [700] * 5])
    q, cache, table, ctx, scores = c.q.cuda(), c.cache(), c.table.cuda(), c.i32(c.ctx), c.scores()
    ws = spv.new_workspace(spv.spv_attention_workspace_bytes(2, 5, 16, 2, 128), q.device)
    out = spv.spv_paged_attention_scored(q, cache, table, ctx, scores, workspace=ws, want_lse=True)
    want = {k: v.clone() for k, v in out.items()}
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        spv.spv_paged_attention_scored(q, cache, table, ctx, scores, workspace=ws, want_lse=True, out=out)
    for v in out.values():
        v.fill_(7)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[k], want[k]) for k in want)


# ------------------------------------------------------------------ weights of cached keys
MASS_CASES = [
    # ctx, new, T, Hq, Hkv, D, page, order, dtype, kv, accepted, options
    ([777], None, 1, 8, 2, 128, 16, "nhd", "bf16", "bf16", [0], dict(cap=50.0)),
    ([300, 5, 1200], None, 5, 16, 2, 128, 16, "nhd", "bf16", "bf16", [4, 0, 2], dict(cap=50.0)),
    ([300, 5, 1200], [5, 3, 4], 5, 16, 2, 64, 8, "hnd", "f16", "f16", [3, -1, 2], dict(window=200)),
    ([300, 5, 1200], None, 5, 16, 2, 128, 16, "nhd", "bf16", "bf16", [4, 0, 2], dict(slopes=True, moved=True)),
    ([300, 700], None, 4, 6, 2, 256, 16, "nhd", "bf16", "bf16", [3, 1], dict(slopes=True, cap=10.0, moved=True, window=150)),
    ([300, 700], None, 4, 6, 2, 256, 32, "nhd", "bf16", "e4m3", [3, 1], dict(cap=10.0, window=150)),
    ([300, 700], None, 6, 6, 2, 128, 16, "nhd", "f16", "e4m3", [5, 1], dict(slopes=True)),
    ([300, 700], None, 4, 6, 2, 64, 16, "nhd", "bf16", "bf16", [3, 3], dict(first=[[100, 301, 250, 305], [600] * 4], last=[[304] * 4, [0, 702, 701, 0]])),
    ([256, 31], None, 21, 8, 2, 128, 16, "nhd", "f16", "f16", "tree", dict(tree=True, slopes=True, cap=30.0)),
    ([256, 31], [21, 9], 21, 32, 4, 64, 16, "nhd", "bf16", "bf16", "tree", dict(tree=True, window=4, first=[[200] * 21, [0] * 21])),
    ([1500], None, 33, 8, 1, 128, 16, "nhd", "bf16", "bf16", [32], dict(window=700, cap=20.0)),
]


def accepted_of(c, accepted):
    """(accept_count, nodes or None, counted tokens of each sequence)."""
    if accepted != "tree":
        return accepted, None, [list(range(a + 1)) for a in accepted]
    counts, nodes, counted = [], [], []
    for b in range(c.B):
        path = [max((t for t in range(c.new[b])), key=lambda t: sr.depths(c.parent[b].tolist(), c.T)[t])]
        while path[-1] > 0:
            path.append(int(c.parent[b, path[-1]]))
        path = path[::-1][1:]
        counts.append(len(path))
        nodes.append(path + [-1] * (c.T - len(path)))
        counted.append([0] + path)
    return counts, nodes, counted


@pytest.mark.parametrize("case", MASS_CASES, ids=lambda c: "-".join(str(x).replace(" ", "") for x in c[2:10]) + "-" + "-".join(c[11]))
@pytest.mark.parametrize("decay", [1.0, 0.5])
def test_mass(spv, case, decay):
    c = sr.Case(spv, 31, *case[:10], **case[11])
    counts, nodes, counted = accepted_of(c, case[10])
    W = max(a + b for a, b in zip(c.ctx, c.new)) + 5
    mass_in = torch.rand(c.B, c.Hkv, W, generator=c.gen)
    lse = c.attention()[1].float()
    out = {"mass": torch.full((c.B, c.Hkv, W), -3.0, device="cuda")}
    got = spv.spv_attention_mass_scored(c.q.cuda(), lse.cuda(), c.cache(), c.table.cuda(), c.i32(c.ctx), c.i32(counts), c.scores(),
                                        nodes=None if nodes is None else i32(nodes), new_lens=c.i32(c.new) if c.ragged else None,
                                        parent=None if c.parent is None else c.parent.cuda(), scale=c.scale, decay=decay,
                                        mass_in=mass_in.cuda(), out=out)
    torch.cuda.synchronize()
    want, bound = c.mass(counted, decay, mass_in)
    x = got["mass"].cpu().double()
    written = ~torch.isnan(want)
    assert (x[~written] == -3.0).all()
    assert (got["row_status"].cpu() == 0).all()
    off = (x - want).abs()[written] - bound[written] - 2.0 ** -24 * want.abs()[written]
    assert off.max() <= 0, off.max()


def test_mass_of_a_batch_adds_up(spv):
    """Weights of one token over what it sees sum to 1 a query head, whatever the cap, bias and window."""
    ctx = [(379 * i) % 1500 for i in range(24)]
    c = sr.Case(spv, 33, ctx, None, 3, 8, 4, 64, 16, cap=30.0, window=222, slopes=True, poison=False)
    got = c.attend()
    mass = spv.spv_attention_mass_scored(c.q.cuda(), got["lse"], c.cache(), c.table.cuda(), c.i32(c.ctx), c.i32([2] * 24), c.scores(),
                                         scale=c.scale)["mass"]
    assert torch.allclose(mass.sum(-1).cpu(), torch.full((24, 4), 6.0), rtol=1e-4)


def test_mass_skips_what_no_token_sees(spv):
    """Pages before the window may be gone: their slots' weights are not written, the sequence is not bad."""
    c = sr.Case(spv, 34, [400], None, 2, 2, 1, 64, 16, window=50)
    table = c.table.clone()
    table[0, 3] = -1
    lse = c.attention()[1].float().cuda()
    out = {"mass": torch.full((1, 1, 420), -3.0, device="cuda")}
    got = spv.spv_attention_mass_scored(c.q.cuda(), lse, c.cache(), table.cuda(), c.i32(c.ctx), i32([1]), c.scores(), out=out,
                                        mass_in=torch.ones(1, 1, 420, device="cuda"))
    m = got["mass"][0, 0].cpu()
    assert got["row_status"].item() == 0
    assert (m[48:64] == -3.0).all() and (m[:48] == 1.0).all() and (m[64:340] == 1.0).all()
    assert (m[360:402] != 1.0).any() and (m[402:] == -3.0).all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_idle_sequences_in_tiles(spv, D, kv):
    """Sequences without new tokens, and short ones, between those of a batch whose rows go in tiles."""
    new = [(0, 9, 0, 1, 0, 0, 5, 0)[b % 8] for b in range(160)]
    c = sr.Case(spv, 73, [(13 * b) % 200 for b in range(160)], new, 9, 16, 2, D, 16, "nhd", "bf16", kv, cap=30.0)
    c.check(c.attend())
