"""GPU tests of the calls around the verify step where a plain computation in
fewer bits goes wrong -- scores and weights at the ends of their types -- and
on streams of their own."""
import math

import pytest
import torch

import kv_reference as ref
from kv_reference import DTYPES, half_step
from test_gpu_kv import Layer, i32, spv  # noqa: F401  (spv: the fixture)

pytestmark = pytest.mark.gpu

POWERS_OF_TWO = 0.6931472  # as a float32, times log2(e) it is 1: scores are powers of two, exactly


def _attend(spv, q, k, v, ctx, page, k_scale=None, v_scale=None, B=456):
    """The same sequence B times, on the same pages, so that each block has whole sequences and takes their keys one after
    another: q [T, Hq, D], k and v [slots, Hkv, D] on the GPU."""
    pages = -(-k.shape[0] // page)
    pools = []
    for x in (k, v):
        pool = torch.zeros(pages * page, *x.shape[1:], dtype=x.dtype, device="cuda")
        pool.view(torch.int8)[: x.shape[0]] = x.view(torch.int8)
        pools.append(pool.view(pages, page, *x.shape[1:]))
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(B, pages).contiguous()
    got = spv.spv_paged_attention(q.expand(B, *q.shape).contiguous(), spv.KVCache(*pools, k_scale, v_scale), table,
                                  i32([ctx] * B), scale=POWERS_OF_TWO, want_lse=True)
    torch.cuda.synchronize()
    assert (got["row_status"] == 0).all()
    return got["out"].cpu().double(), got["lse"].cpu().double()


# rows of a key head: the warp kernel, and each layout of the rows kernel
ROWS = [(1, 4), (5, 4), (12, 4), (24, 4), (40, 4)]


@pytest.mark.parametrize("T, G", ROWS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype, kv", [("f16", "f16"), ("bf16", "e4m3"), ("bf16", "bf16")])
def test_attention_scores_beyond_2_to_27(spv, T, G, D, dtype, kv):
    """Scores whose 32-bit neighbours are 16 powers of two apart: 2^27 + 16, then 2^27 + 32 for the later half.  The
    second ones have weight 1, the first 2^-16; every sum is exact but for the weights' rounding and the result's."""
    ctx = 600
    n = ctx + T
    late = (torch.arange(n, device="cuda") >= 300).float()
    q = torch.zeros(T, G, D, device="cuda")
    k = torch.zeros(n, 1, D, device="cuda")
    q[..., 0], q[..., 1] = 2.0 ** 15, 1.0
    ks = None
    if kv == "e4m3":  # 16 (2^15 2^8 + 1 or 2)
        k[:, 0, 0], k[:, 0, 1] = 2.0 ** 8, 1.0 + late
        ks = torch.full((1,), 16.0, device="cuda")
    else:             # 2^15 2^12 + 16 or 32
        k[:, 0, 0], k[:, 0, 1] = 2.0 ** 12, 16.0 + 16.0 * late
    v = torch.randn(n, 1, D, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(DTYPES[kv])
    vs = torch.ones(1, device="cuda") if ks is not None else None
    out, lse = _attend(spv, q.to(DTYPES[dtype]), k.to(DTYPES[kv]), v, ctx, 16, ks, vs)
    x = v[:, 0].float().cpu().double()
    w = torch.where(late.cpu() > 0, 1.0, 2.0 ** -16).double()
    for t in range(T):
        seen = w[: ctx + t + 1, None] / w[: ctx + t + 1].sum()
        want, size = (seen * x[: ctx + t + 1]).sum(0), (seen * x[: ctx + t + 1].abs()).sum(0)
        # weights equal to a power of two or its rounding; result rounded once
        tol = 2 * half_step(DTYPES[dtype]) * size + 2.0 ** -24
        assert ((out[:, t] - want).abs() <= tol).all()
        z = math.log(2.0) * (2.0 ** 27 + 32 + math.log2(w[: ctx + t + 1].sum().item()))
        assert ((lse[:, t] - z).abs() <= z * 2.0 ** -22).all()


@pytest.mark.parametrize("T, G", ROWS)
@pytest.mark.parametrize("dtype, kv", [("f16", "f16"), ("bf16", "e4m3"), ("f16", "e4m3"), ("bf16", "bf16")])
@pytest.mark.parametrize("peak", [0, 170_001, 262_143])
def test_attention_peak_over_a_long_flat_background(spv, T, G, dtype, kv, peak):
    """262,143 keys each 2^-25 of the largest: together 2^-7 of the result, though each is below what f16 holds."""
    ctx, D = 262_144, 64
    n = ctx + T
    q = torch.zeros(T, G, D, device="cuda")
    q[..., 0] = 1.0
    k = torch.full((n, 1, D), 0.0, device="cuda")
    k[:, 0, 0] = -12.0
    k[peak, 0, 0] = 13.0
    v = torch.full((n, 1, D), -1.0, device="cuda")
    v[peak] = 1.0
    one = torch.ones(1, device="cuda") if kv == "e4m3" else None
    out, lse = _attend(spv, q.to(DTYPES[dtype]), k.to(DTYPES[kv]), v.to(DTYPES[kv]), ctx, 64, one, one)
    for t in range(T):
        rest = (ctx + t) * 2.0 ** -25
        want = (1.0 - rest) / (1.0 + rest)
        # every product and sum of these powers of two is exact up to the 32-bit sums' roundings
        assert ((out[:, t] - want).abs() <= half_step(DTYPES[dtype]) + 2.0 ** -15).all()
        z = math.log(2.0) * (13.0 + math.log2(1.0 + rest))
        assert ((lse[:, t] - z).abs() <= z * 2.0 ** -20).all()


@pytest.mark.parametrize("T", [1, 12])
def test_calls_on_a_side_stream_have_buffers_of_their_own(spv, T):
    """Without workspace and outputs, while torch's current stream is far behind: nothing of the call waits there."""
    a = Layer(spv, 53, [5000, 700], None, T, 8, 2, 64, 16)
    b = Layer(spv, 54, [4000], None, T, 8, 2, 64, 16)
    inputs = [(x, x.q.cuda(), x.table.cuda(), i32(x.ctx), i32([T - 1] * x.B)) for x in (a, b)]

    def run(stream):
        res = []
        for x, q, table, ctx, acc in inputs:  # one after another: the second call may get the first one's memory
            got = spv.spv_paged_attention(q, x.cache, table, ctx, want_lse=True, stream=stream)
            mass = spv.spv_attention_mass(q, got["lse"], x.cache, table, ctx, acc, stream=stream)["mass"]
            keep = spv.spv_kv_evict(x.cache, table, ctx, mass, 8192, stream=stream)["mass"]
            res += [got["out"], got["lse"], mass, keep[:, :, : min(x.ctx)]]
            del got
        return res

    want = run(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda._sleep(200_000_000)  # about 0.1 s of the current stream
        got = run(side)
        side.synchronize()
        got = [x.cpu() for x in got]
        for x, y in zip(want, got):
            assert torch.equal(x.cpu(), y)
        torch.cuda.synchronize()


@pytest.mark.parametrize("W, budget", [(400, 64), (20_000, 9_000), (70_000, 30_000)])
def test_evict_lengths_in_place(spv, W, budget):
    """lens as its own output: every head of every sequence is cut as with lengths apart, also in a replayed graph."""
    B, Hkv, D, page = 5, 8, 64, 16
    lens = [W, budget + 1, budget, 3, W - 1]
    gen = torch.Generator(device="cuda").manual_seed(55)
    pages = -(-W // page)
    pool = lambda: torch.randn(pages * B, page, Hkv, D, generator=gen, device="cuda").bfloat16()  # noqa: E731
    k, v = pool(), pool()
    table = torch.arange(B * pages, dtype=torch.int32, device="cuda").reshape(B, pages)
    mass = torch.rand(B, Hkv, W, generator=gen, device="cuda")
    apart = spv.KVCache(k.clone(), v.clone())
    want = spv.spv_kv_evict(apart, table, i32(lens), mass, budget, sinks=2, recent=5)
    cache, at = spv.KVCache(k.clone(), v.clone()), i32(lens)
    out = {x: torch.empty_like(want[x]) for x in ("mass", "pos", "slot_src", "row_status")}

    def run():
        return spv.spv_kv_evict(cache, table, at, mass, budget, sinks=2, recent=5, out={**out, "lens": at})

    def check():
        torch.cuda.synchronize()
        assert at.tolist() == [min(n, budget) for n in lens] and out["row_status"].tolist() == [0] * B
        assert torch.equal(out["slot_src"], want["slot_src"])
        assert torch.equal(cache.k, apart.k) and torch.equal(cache.v, apart.v)
        for b, n in enumerate(at.tolist()):
            assert torch.equal(out["mass"][b, :, :n], want["mass"][b, :, :n])

    run()
    check()
    again = run()  # nothing is above the budget now
    torch.cuda.synchronize()
    assert again["lens"] is at and at.tolist() == [min(n, budget) for n in lens]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for _ in range(2):
        at.copy_(i32(lens))
        cache.k.copy_(k), cache.v.copy_(v)
        g.replay()
        check()


@pytest.mark.parametrize("inter, r", [(True, 26), (True, 6), (True, 60), (False, 26), (False, 48)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_rope_passes_elements_unchanged(spv, inter, r, dtype):
    """The elements from rotary_dim on keep their bits, whatever their neighbours are: infinities, NaN, signed zeros."""
    B, T, Hq, Hkv, D, page = 2, 3, 4, 2, 64, 16
    gen = torch.Generator().manual_seed(52)
    k, v, _, _, table = ref.make_cache(gen, [20] * B, page, Hkv, D, dtype, garbage=False)
    x = torch.randn(B, T, Hq + 2 * Hkv, D, generator=gen).to(DTYPES[dtype])
    odd = torch.tensor([math.inf, -0.0, -0.0, -1.0, math.nan, 2.0, -math.inf, 0.0, -0.0, math.inf])
    passing = odd.repeat(B * T * (Hq + Hkv) * D)[: B * T * (Hq + Hkv) * (D - r)].reshape(B, T, Hq + Hkv, D - r).to(DTYPES[dtype])
    x[:, :, : Hq + Hkv, r:] = passing
    cache = spv.KVCache(k.cuda(), v.cuda())
    q, kk, vv = x.cuda().split([Hq, Hkv, Hkv], dim=2)
    got = spv.spv_rope_append(q, kk, vv, cache, table.cuda(), i32([17] * B), spv.spv_rope_frequencies(r), interleaved=inter)
    torch.cuda.synchronize()
    bits = lambda y: y.contiguous().view(torch.int16).cpu()  # noqa: E731
    assert torch.equal(bits(got["q"][..., r:]), bits(x[:, :, :Hq, r:]))
    assert torch.isfinite(got["q"][..., :r]).all()
    for b in range(B):
        for t in range(T):
            at = (table[b, (17 + t) // page].long(), (17 + t) % page)
            assert torch.equal(bits(cache.k[at][:, r:]), bits(x[b, t, Hq: Hq + Hkv, r:]))
            assert torch.equal(bits(cache.v[at]), bits(x[b, t, Hq + Hkv:]))


@pytest.mark.parametrize("T, G", ROWS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_infinities_in_cached_v_are_seen(spv, T, G, D, dtype):
    """An infinity in a cached slot is every row's result in its column; infinities of both signs, or NaN, make NaN;
    the other columns keep every bit."""
    a = Layer(spv, 51, [700, 131], None, T, 2 * G, 2, D, 16, dtype=dtype)
    clean = a.attend()
    for b, slots in enumerate(((3, 130, 301, 699), (0, 64, 129, 130))):
        for i, j in enumerate(slots):
            at = (a.table[b, j // 16].long(), j % 16, 1)
            a.cache.v[at + (8 + i,)] = math.inf                        # one slot each
            a.cache.v[at + (40 + i,)] = -math.inf
            a.cache.v[at + (16,)] = math.inf                           # all four slots
            a.cache.v[at + (17,)] = math.inf if i % 2 else -math.inf   # both signs
            a.cache.v[at + (63,)] = math.nan if i == 2 else math.inf
    got = a.attend()
    want = clean["out"].clone()
    h = slice(G, 2 * G)
    want[:, :, h, 8:12] = math.inf
    want[:, :, h, 40:44] = -math.inf
    want[:, :, h, 16] = math.inf
    want[:, :, h, 17] = math.nan
    want[:, :, h, 63] = math.nan
    assert torch.equal(torch.isnan(got["out"]), torch.isnan(want))
    assert torch.equal(got["out"].nan_to_num(nan=0.5), want.nan_to_num(nan=0.5))
    assert torch.equal(got["lse"], clean["lse"])


@pytest.fixture
def gives_up(spv):
    yield spv.spv_selftest_give_up
    spv.spv_selftest_give_up(-1)


@pytest.mark.parametrize("T, G, kv", [(5, 4, "bf16"), (12, 4, "bf16"), (24, 4, "bf16"), (12, 4, "e4m3"), (24, 4, "e4m3")])
@pytest.mark.parametrize("page", [16, 2])
def test_attention_after_a_wait_gave_up(spv, gives_up, T, G, kv, page):
    """What a block still had to write is NaN, the pieces of items that it shares among them, the rest is as ever, and the
    workspace says so; nothing is left of what the outputs and the workspace held."""
    gen = torch.Generator().manual_seed(56)
    ctx = torch.randint(0, 500, (300,), generator=gen).tolist()
    ctx[20], ctx[250] = 6000, 3000
    a = Layer(spv, 57, ctx, None, T, 2 * G, 2, 64, page, dtype="bf16", kv=kv)
    ws = spv.new_workspace(spv.spv_attention_workspace_bytes(a.B, T, 2 * G, 2, 64), "cuda")
    q, table, at = a.q.cuda(), a.table.cuda(), i32(ctx)

    def run():
        out = {"out": torch.full_like(q, 7.0), "lse": torch.full((a.B, T, 2 * G), 7.0, device="cuda"),
               "row_status": torch.full((a.B,), 7, dtype=torch.int32, device="cuda")}
        spv.spv_paged_attention(q, a.cache, table, at, workspace=ws, out=out, want_lse=True)
        torch.cuda.synchronize()
        return out

    good = run()
    assert (good["row_status"] == 0).all() and torch.isfinite(good["out"]).all()
    for block, item in ((0, 0), (1, 1), (77, 0), (77, 2), (151, 1)):
        gives_up(block, item)
        got = run()
        gives_up(-1)
        gone = torch.isnan(got["lse"])
        assert gone.any() and not gone.all()
        assert spv.spv_workspace_status(ws) == spv.SPV_ERR_TIMEOUT
        assert torch.isnan(got["out"][gone]).all()
        assert torch.equal(got["out"][~gone], good["out"][~gone]) and torch.equal(got["lse"][~gone], good["lse"][~gone])
        assert torch.equal(got["row_status"] == spv.SPV_ERR_TIMEOUT, gone[:, 0, 0])
        assert ((got["row_status"] == 0) | (got["row_status"] == spv.SPV_ERR_TIMEOUT)).all()
        ws.zero_()
        again = run()
        assert spv.spv_workspace_status(ws) == spv.SPV_OK
        assert torch.equal(again["out"], good["out"]) and torch.equal(again["lse"], good["lse"])
        assert (again["row_status"] == 0).all()
    with pytest.raises(spv.SpvError):
        gives_up(-2)


@pytest.mark.parametrize("D, kv", [(64, "bf16"), (128, "bf16"), (256, "bf16"), (64, "e4m3"), (128, "e4m3"), (256, "e4m3")])
def test_mass_after_a_wait_gave_up(spv, gives_up, D, kv):
    """The weights that a block still had to write are NaN and their sequences' status says so; the rest is as ever."""
    gen = torch.Generator().manual_seed(58)
    ctx = torch.randint(0, 400, (200,), generator=gen).tolist()
    ctx[20], ctx[150] = 4000, 2000
    T, G = 6, 8
    a = Layer(spv, 59, ctx, None, T, 2 * G, 2, D, 16, dtype="bf16", kv=kv)
    q, table, at = a.q.cuda(), a.table.cuda(), i32(ctx)
    lse = spv.spv_paged_attention(q, a.cache, table, at, want_lse=True)["lse"]
    accept = torch.randint(-1, T, (a.B,), generator=gen).to(torch.int32).cuda()
    W = 4010
    old = torch.rand(a.B, 2, W, generator=gen).cuda()

    def run(status=True):
        out = {"mass": torch.full((a.B, 2, W), 7.0, device="cuda"), "row_status": torch.full((a.B,), 7, dtype=torch.int32, device="cuda")}
        spv.spv_attention_mass(q, lse, a.cache, table, at, accept, mass_in=old, out=out, want_status=status)
        torch.cuda.synchronize()
        return out

    good = run()
    assert (good["row_status"] == 0).all() and torch.isfinite(good["mass"]).all()
    for block, item in ((0, 0), (1, 1), (77, 0), (77, 2), (151, 0)):
        gives_up(block, item)
        got, silent = run(), run(status=False)
        gives_up(-1)
        for x in (got, silent):
            gone = torch.isnan(x["mass"])
            assert gone.any() and not gone.all()
            assert torch.equal(x["mass"][~gone], good["mass"][~gone])
        assert (silent["row_status"] == 7).all()
        lost = torch.isnan(got["mass"]).any(-1).any(-1)
        assert torch.equal(got["row_status"], torch.where(lost, spv.SPV_ERR_TIMEOUT, 0).to(torch.int32))
        again = run()
        assert torch.equal(again["mass"], good["mass"]) and (again["row_status"] == 0).all()
