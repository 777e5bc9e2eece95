"""GPU tests of the calls around the verify step against plain 64-bit forms
(kv_reference), at the sizes, masks and inputs where they can go wrong.

Tolerances: an element may be off by half a step of its type plus the bound
that kv_reference derives from the number of 32-bit roundings behind it."""
import math

import pytest
import torch

import kv_reference as ref
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


def to_gpu(pool, order="nhd"):
    if order == "hnd":
        return pool.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    return pool.contiguous().cuda()


class Layer:
    """Inputs of the attention calls, on the CPU and the GPU."""

    def __init__(self, spv, seed, ctx, new, T, Hq, Hkv, D, page, order="nhd", dtype="bf16", kv=None, tree=False,
                 spread=1.0):
        gen = torch.Generator().manual_seed(seed)
        self.B, self.T, self.Hq, self.Hkv, self.D = len(ctx), T, Hq, Hkv, D
        self.ctx, self.new = list(ctx), list(new) if new is not None else [T] * len(ctx)
        lens = [a + b for a, b in zip(self.ctx, self.new)]
        self.k, self.v, self.ks, self.vs, self.table = ref.make_cache(gen, lens, page, Hkv, D, kv or dtype, order)
        self.q = (torch.randn(self.B, T, Hq, D, generator=gen) * spread).to(DTYPES[dtype])
        self.parent = None
        if tree:
            self.parent = torch.tensor([ref.random_tree(gen, T) for _ in ctx], dtype=torch.int32)
        self.scale = 1.0 / math.sqrt(D)
        self.spv = spv
        self.order = order
        self.cache = spv.KVCache(to_gpu(self.k, order), to_gpu(self.v, order),
                                 self.ks.cuda() if self.ks is not None else None,
                                 self.vs.cuda() if self.vs is not None else None)
        self.gen = gen
        self.ragged = new is not None

    def args(self):
        return dict(new_lens=i32(self.new) if self.ragged else None,
                    parent=self.parent.cuda() if self.parent is not None else None)

    def attend(self, **kw):
        got = self.spv.spv_paged_attention(self.q.cuda(), self.cache, self.table.cuda(), i32(self.ctx), want_lse=True,
                                           **{**self.args(), **kw})
        torch.cuda.synchronize()
        return got

    def check(self, got):
        out, lse, bound, lse_bound = ref.attention(self.q, self.k, self.v, self.ks, self.vs, self.table, self.ctx,
                                                   self.new, self.parent, self.scale)
        x = got["out"].cpu().double()
        tol = half_step(self.q.dtype) * (out.abs() + bound) + bound + (2.0 ** -24 if self.q.dtype == torch.float16 else 0)
        assert torch.isfinite(x).all()
        worst = ((x - out).abs() - tol).max().item()
        assert worst <= 0, f"out: {worst} beyond the bound"
        z = got["lse"].cpu().double()
        assert torch.equal(torch.isinf(z), torch.isinf(lse))
        fine = torch.isfinite(lse)
        assert ((z - lse).abs() <= lse_bound)[fine].all(), ((z - lse).abs() / lse_bound)[fine].max()
        assert (got["row_status"].cpu() == 0).all()


CASES = [
    # ctx, new, T, Hq, Hkv, D, page, order, dtype, kv, tree
    ([0], None, 1, 1, 1, 64, 16, "nhd", "bf16", "bf16", False),
    ([1], None, 1, 8, 8, 128, 1, "nhd", "f16", "f16", False),
    ([777], None, 1, 32, 8, 128, 16, "nhd", "bf16", "bf16", False),
    ([63, 64, 65, 127, 0, 1], None, 1, 4, 2, 64, 16, "hnd", "bf16", "bf16", False),
    ([62, 63, 64, 200, 511], [2, 1, 0, 2, 2], 2, 6, 2, 64, 8, "nhd", "f16", "f16", False),
    ([300, 5, 1200], None, 5, 16, 2, 128, 16, "nhd", "bf16", "bf16", False),
    ([300, 5, 1200], [5, 3, 4], 5, 64, 8, 128, 32, "hnd", "f16", "f16", False),
    ([130, 700], None, 8, 8, 2, 128, 64, "nhd", "bf16", "e4m3", False),
    ([130, 701], None, 3, 8, 8, 64, 128, "hnd", "f16", "e4m3", False),
    ([99, 400], None, 1, 7, 1, 256, 16, "nhd", "bf16", "bf16", False),
    ([99, 400], [4, 2], 4, 20, 4, 256, 4, "nhd", "f16", "f16", False),
    ([50, 260], None, 2, 3, 1, 256, 16, "hnd", "bf16", "e4m3", False),
    ([256, 31], None, 21, 8, 2, 128, 16, "nhd", "f16", "f16", True),
    ([250, 31, 0], [21, 17, 1], 21, 32, 8, 128, 16, "hnd", "bf16", "bf16", True),
    ([100], None, 64, 16, 1, 64, 16, "nhd", "bf16", "bf16", True),
    ([70, 129], None, 63, 10, 2, 128, 32, "nhd", "f16", "e4m3", True),
    ([40], None, 33, 64, 1, 128, 16, "nhd", "bf16", "bf16", False),
    ([1000], None, 2, 64, 1, 64, 2, "nhd", "f16", "f16", False),
    ([5000, 3], None, 1, 16, 16, 64, 16, "nhd", "bf16", "bf16", False),
    ([9000], None, 6, 5, 1, 128, 128, "nhd", "bf16", "bf16", False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).replace(" ", "") for x in c[2:]))
def test_attention(spv, case):
    ctx, new, T, Hq, Hkv, D, page, order, dtype, kv, tree = case
    a = Layer(spv, 7, ctx, new, T, Hq, Hkv, D, page, order, dtype, kv, tree)
    a.check(a.attend())


@pytest.mark.parametrize("spread", [0.0, 8.0, 40.0])
@pytest.mark.parametrize("T", [1, 12])
def test_attention_flat_and_peaked_scores(spv, spread, T):
    """Equal scores, and scores whose largest leaves the others far behind, rising and falling along the cache."""
    a = Layer(spv, 3, [700, 333], None, T, 8, 2, 128, 16, dtype="bf16", spread=spread)
    a.check(a.attend())


@pytest.mark.parametrize("T", [1, 12])
@pytest.mark.parametrize("rising", [True, False])
def test_attention_monotone_scores(spv, rising, T):
    """The running maximum grows at every key, or never after the first."""
    a = Layer(spv, 4, [900], None, T, 8, 2, 64, 16, dtype="bf16")
    n = 900 + T
    for j in range(n):
        x = (j if rising else n - j) / n
        a.k[a.table[0, j // 16].long(), j % 16] = x * 16.0
    a.q = torch.full_like(a.q, 2.0)
    a.cache.k = to_gpu(a.k)
    a.check(a.attend())


@pytest.mark.parametrize("T, G", [(1, 4), (4, 4), (21, 4), (40, 3)])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_unseen_values_have_no_effect(spv, value, T, G):
    """Infinities and NaN in the K and V of new tokens that a row does not see, and past the end of the sequence."""
    a = Layer(spv, 5, [61, 130], None, T, 2 * G, 2, 128, 16, tree=T == 21)
    clean = a.attend()
    for b in range(2):  # the last token's K and V; no other token sees it
        j = a.ctx[b] + T - 1
        a.cache.k[a.table[b, j // 16].long(), j % 16] = value
        a.cache.v[a.table[b, j // 16].long(), j % 16] = value
    got = a.attend()
    assert torch.equal(got["out"][:, : T - 1], clean["out"][:, : T - 1])
    assert torch.equal(got["lse"][:, : T - 1], clean["lse"][:, : T - 1])
    assert torch.isnan(got["out"][:, T - 1]).all()


@pytest.mark.parametrize("T", [4, 20])
def test_unseen_infinite_v_only(spv, T):
    a = Layer(spv, 5, [61, 130], None, T, 8, 2, 64, 16, dtype="f16")
    clean = a.attend()
    for b in range(2):
        j = a.ctx[b] + T - 1
        a.cache.v[a.table[b, j // 16].long(), j % 16] = math.inf
    got = a.attend()
    assert torch.equal(got["out"][:, : T - 1], clean["out"][:, : T - 1])
    assert torch.equal(got["lse"], clean["lse"])
    assert not torch.isfinite(got["out"][:, T - 1]).any()


def test_seen_nan_stays(spv):
    a = Layer(spv, 6, [200, 200], None, 2, 4, 2, 64, 16)
    a.cache.k[a.table[0, 3].long(), 5, 0] = math.nan
    got = a.attend()
    G = 2
    assert torch.isnan(got["out"][0, :, :G]).all() and torch.isnan(got["lse"][0, :, :G]).all()
    assert torch.isfinite(got["out"][0, :, G:]).all() and torch.isfinite(got["out"][1]).all()


@pytest.mark.parametrize("T", [1, 12])
def test_scores_of_minus_infinity(spv, T):
    """Every score minus infinity: a row without a sum; the lowest finite value of the type: an ordinary score."""
    a = Layer(spv, 6, [40, 40], None, T, 2, 1, 64, 16)
    a.q = torch.ones_like(a.q)
    a.k[a.table[0].long()] = -math.inf
    a.k[a.table[1].long()] = torch.finfo(torch.bfloat16).min
    a.cache.k = to_gpu(a.k)
    got = a.attend()
    assert (got["out"][0] == 0).all() and (got["lse"][0] == -math.inf).all()
    # 64 times the lowest value is beyond 32 bits: minus infinity again
    assert (got["out"][1] == 0).all() and (got["lse"][1] == -math.inf).all()
    a.q = torch.zeros_like(a.q)
    a.q[..., 0] = 2.0 ** -60
    got = a.attend()
    assert torch.isnan(got["out"][0]).all()  # 0 * -inf
    for t in range(T):  # equal scores, however large: the mean
        v = ref.rows(a.v, a.table[1], 41 + t).mean(0)
        assert (got["out"][1, t].cpu().double() - v).abs().max() <= 2.0 ** -8 * (v.abs().max() + 1)


def test_bad_parents_empty_rows(spv):
    a = Layer(spv, 8, [90, 90], None, 6, 4, 2, 64, 16, tree=True)
    a.parent[0] = torch.tensor([-1, 0, 5, 2, 1, -3], dtype=torch.int32)   # 2 -> 5 ahead, 3 hangs from it, 5 negative
    a.parent[1] = torch.tensor([99, 0, 1, 3, 1, 2 ** 31 - 1], dtype=torch.int32)  # root ignored; 3 its own parent
    got = a.attend()
    a.check(got)
    for b, t in ((0, 2), (0, 3), (0, 5), (1, 3), (1, 5)):
        assert (got["out"][b, t] == 0).all() and (got["lse"][b, t] == -math.inf).all()


def test_bad_sequences(spv):
    """Lengths out of range and page ids out of the pool: NaN, a status, and the others as they are."""
    a = Layer(spv, 9, [100, 100, 100, 100, 100], None, 2, 4, 2, 64, 16)
    good = a.attend()
    width = a.table.shape[1]
    a.ctx[1], a.ctx[2] = -5, width * 16 - 1
    a.table[3, 2], a.table[4, 6] = a.k.shape[0], -1
    got = a.attend()
    assert got["row_status"].tolist() == [0, 4, 4, 4, 4]
    assert torch.equal(got["out"][0], good["out"][0]) and torch.equal(got["lse"][0], good["lse"][0])
    assert torch.isnan(got["out"][1:]).all() and torch.isnan(got["lse"][1:]).all()
    a.ctx = [100] * 5
    a.table[3, 2] = -(2 ** 31)
    new = i32([2, 3, -1, 0, 2])
    got = a.attend(new_lens=new)
    assert got["row_status"].tolist() == [0, 4, 4, 0, 4]
    assert (got["out"][3] == 0).all() and torch.isnan(got["out"][1]).all()


@pytest.mark.parametrize("T, dtype", [(1, "bf16"), (5, "f16"), (20, "bf16")])
def test_attention_repeats_bit_by_bit(spv, T, dtype):
    """Same call, one workspace, another call of other sizes between: the same bits, on another stream too."""
    a = Layer(spv, 10, [3000, 17, 801, 0], None, T, 16, 2, 128, 16, dtype=dtype)
    b = Layer(spv, 11, [100] * 9, None, 3, 8, 8, 128, 16, dtype=dtype)
    n = max(spv.spv_attention_workspace_bytes(x.B, x.T, x.Hq, x.Hkv, x.D) for x in (a, b))
    ws = spv.new_workspace(n, "cuda")
    one = a.attend(workspace=ws)
    b.check(b.attend(workspace=ws))
    two = a.attend(workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    three = a.attend(workspace=ws, stream=side)
    for other in (two, three):
        assert torch.equal(one["out"], other["out"]) and torch.equal(one["lse"], other["lse"])
    a.check(one)


def test_attention_in_a_graph_follows_the_lengths(spv):
    """A captured call reads the lengths at replay: the cache may grow between replays."""
    a = Layer(spv, 12, [500, 40], None, 2, 8, 2, 64, 16)
    q, table, ctx = a.q.cuda(), a.table.cuda(), i32(a.ctx)
    ws = spv.new_workspace(spv.spv_attention_workspace_bytes(2, 2, 8, 2, 64), "cuda")
    out = {"out": torch.empty_like(q), "lse": torch.empty(2, 2, 8, device="cuda"), "row_status": i32([0, 0])}
    run = lambda: spv.spv_paged_attention(q, a.cache, table, ctx, workspace=ws, out=out, want_lse=True)  # noqa: E731
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for ctx_now in ([500, 40], [100, 3], [0, 33]):
        a.ctx = ctx_now
        ctx.copy_(i32(ctx_now))
        g.replay()
        torch.cuda.synchronize()
        a.check(out)


def test_attention_many_sequences(spv):
    """More sequences than one warp scans at a time, most of them short."""
    gen = torch.Generator().manual_seed(1)
    ctx = torch.randint(0, 40, (300,), generator=gen).tolist()
    ctx[77], ctx[255] = 2000, 900
    a = Layer(spv, 13, ctx, None, 2, 4, 1, 64, 16)
    a.check(a.attend())


def test_joint_tensor_strides(spv):
    """K and V as slices of one [pages, 2, page, heads, D] tensor, heads 1..2 of 4."""
    a = Layer(spv, 14, [70, 300], None, 3, 8, 2, 64, 16)
    joint = torch.full((a.k.shape[0], 2, 16, 4, 64), math.nan, dtype=a.k.dtype, device="cuda")
    joint[:, 0, :, 1:3], joint[:, 1, :, 1:3] = a.k.cuda(), a.v.cuda()
    a.cache = spv.KVCache(joint[:, 0, :, 1:3], joint[:, 1, :, 1:3])
    a.check(a.attend())


def test_offsets_past_32_bits(spv):
    """Rows that lie more than 2^32 bytes and 2^31 elements into the pools, in every call."""
    pages, page, Hkv, D = 140_000, 16, 8, 128  # 2.3e9 elements, 4.6 GB a pool
    free = torch.cuda.mem_get_info()[0]
    if free < 16e9:
        pytest.skip("needs 16 GB of device memory")
    a = Layer(spv, 15, [60, 100], None, 2, 16, Hkv, D, page)
    far = spv.KVCache(*(torch.empty(pages, page, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    at = torch.arange(a.k.shape[0]) * 1000 + (pages - 1000 * a.k.shape[0])
    assert (at[-1] + 1) <= pages and at.min() >= 0
    far.k[at.cuda()], far.v[at.cuda()] = a.k.cuda(), a.v.cuda()
    near, table = a.cache, a.table.clone()
    got = a.attend()
    a.cache = far
    a.table = torch.where(table >= 0, at[table.clamp(min=0).long()].to(torch.int32), table)
    again = a.attend()
    assert torch.equal(got["out"], again["out"])
    acc = i32([1, 0])
    m = [spv.spv_attention_mass(a.q.cuda(), got["lse"], c, t.cuda(), i32(a.ctx), acc)["mass"] for c, t in
         ((near, table), (far, a.table))]
    assert torch.equal(*m)
    mass = torch.rand(2, Hkv, 102, device="cuda")
    for c, t in ((near, table), (far, a.table)):
        spv.spv_kv_evict(c, t.cuda(), i32([62, 102]), mass, 40, recent=8)
    assert torch.equal(far.k[at.cuda()].view(torch.int16), near.k.view(torch.int16))
    assert torch.equal(far.v[at.cuda()].view(torch.int16), near.v.view(torch.int16))
    del far
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ mass

def _mass_case(spv, seed, ctx, new, T, Hq, Hkv, D, page, order, dtype, kv, tree, accept, nodes=None, decay=1.0):
    a = Layer(spv, seed, ctx, new, T, Hq, Hkv, D, page, order, dtype, kv, tree)
    lse = ref.attention(a.q, a.k, a.v, a.ks, a.vs, a.table, a.ctx, a.new, a.parent, a.scale)[1].float()
    W = max(x + y for x, y in zip(a.ctx, a.new)) + 3
    mass_in = torch.rand(a.B, Hkv, W, generator=a.gen)
    counted = []
    for b in range(a.B):
        k = accept[b]
        counted.append([] if k < 0 else list(range(k + 1)) if nodes is None else sorted({0, *nodes[b][:k]}))
    want, bound = ref.attention_mass(a.q, a.k, a.ks, a.table, a.ctx, a.new, a.parent, a.scale, counted, decay, mass_in)
    out = torch.full((a.B, Hkv, W), -3.0, device="cuda")
    nd = None
    if nodes is not None:
        nd = torch.full((a.B, T), -1, dtype=torch.int32)
        for b, n in enumerate(nodes):
            nd[b, : len(n)] = torch.tensor(n, dtype=torch.int32)
    got = spv.spv_attention_mass(a.q.cuda(), lse.cuda(), a.cache, a.table.cuda(), i32(a.ctx), i32(accept),
                                 nodes=nd.cuda() if nd is not None else None, decay=decay, mass_in=mass_in.cuda(),
                                 out={"mass": out}, **a.args())
    torch.cuda.synchronize()
    assert (got["row_status"] == 0).all()
    x = got["mass"].cpu().double()
    written = ~torch.isnan(want)
    assert (x[~written] == -3.0).all()
    worst = ((x - want).abs() - bound)[written].max().item()
    assert worst <= 0, worst
    return a, got


@pytest.mark.parametrize("case", [
    ([0], None, 1, 1, 1, 64, 16, "nhd", "bf16", "bf16", False, [0]),
    ([777], None, 1, 32, 8, 128, 16, "nhd", "bf16", "bf16", False, [0]),
    ([300, 5, 1200, 64], None, 5, 16, 2, 128, 16, "hnd", "bf16", "bf16", False, [4, 0, 2, -1]),
    ([300, 5, 1200], [5, 3, 0], 5, 64, 8, 128, 32, "nhd", "f16", "f16", False, [4, 2, 0]),
    ([130, 700], None, 8, 8, 2, 128, 64, "nhd", "bf16", "e4m3", False, [7, 1]),
    ([99, 401], None, 3, 7, 1, 256, 1, "nhd", "f16", "f16", False, [2, 1]),
    ([129], None, 33, 64, 1, 64, 16, "nhd", "bf16", "e4m3", False, [32]),
], ids=lambda c: "-".join(str(x).replace(" ", "") for x in c[2:]))
def test_mass_chain(spv, case):
    *rest, accept = case
    _mass_case(spv, 21, *rest, accept, decay=0.75)


def test_mass_tree_nodes(spv):
    parent_free = [[1, 5, 13], [], [2]]
    _mass_case(spv, 22, [200, 31, 0], None, 21, 8, 2, 128, 16, "nhd", "f16", "f16", True, [3, 0, 1], parent_free)


def test_mass_sums_to_the_counted_rows(spv):
    a, got = _mass_case(spv, 23, [500, 90], None, 4, 8, 2, 64, 16, "nhd", "bf16", "bf16", False, [3, 1])
    fresh = spv.spv_attention_mass(a.q.cuda(), a.attend()["lse"], a.cache, a.table.cuda(), i32(a.ctx), i32([3, 1]))
    total = fresh["mass"].double().sum(-1).cpu()
    assert (total - torch.tensor([[16.0], [8.0]], dtype=torch.float64)).abs().max() < 16 * 2.0 ** -17


def test_mass_in_place_and_bad_sequences(spv):
    a = Layer(spv, 24, [100, 100, 100, 100], None, 3, 4, 2, 64, 16)
    lse = a.attend()["lse"]
    mass = torch.rand(4, 2, 110, device="cuda")
    apart = spv.spv_attention_mass(a.q.cuda(), lse, a.cache, a.table.cuda(), i32(a.ctx), i32([2, 1, 0, 2]),
                                   mass_in=mass, out={"mass": mass.clone()})
    kept = mass.clone()
    table = a.table.clone()
    table[3, 2] = 10 ** 6
    got = spv.spv_attention_mass(a.q.cuda(), lse, a.cache, table.cuda(), i32([100, 100, -1, 100]),
                                 i32([2, 3, 0, 2]), mass_in=mass, out={"mass": mass})
    torch.cuda.synchronize()
    assert got["row_status"].tolist() == [0, 4, 4, 4]
    assert torch.equal(mass[0], apart["mass"][0])
    assert torch.equal(mass[1:3], kept[1:3])
    assert torch.equal(mass[3, :, 32:48], kept[3, :, 32:48]) and torch.equal(mass[3, :, :32], apart["mass"][3, :, :32])
    nodes = i32([[1, 2, -1], [0, 3, -1], [-1] * 3, [1, -1, -1]])
    got = spv.spv_attention_mass(a.q.cuda(), lse, a.cache, a.table.cuda(), i32(a.ctx), i32([2, 2, 1, -2]), nodes=nodes)
    assert got["row_status"].tolist() == [0, 4, 4, 4]
    assert (got["mass"][1:] == 0).all()


def test_mass_rows_that_see_nothing_give_nothing(spv):
    a = Layer(spv, 25, [64], None, 3, 2, 1, 64, 16, tree=True)
    a.parent[0] = torch.tensor([-1, 2, 0], dtype=torch.int32)  # node 1 hangs from a later node
    lse = a.attend()["lse"]
    assert (lse[0, 1] == -math.inf).all()
    got = spv.spv_attention_mass(a.q.cuda(), lse, a.cache, a.table.cuda(), i32(a.ctx), i32([1]),
                                 nodes=i32([[1, -1, -1]]), parent=a.parent.cuda())
    only_root = spv.spv_attention_mass(a.q.cuda(), lse, a.cache, a.table.cuda(), i32(a.ctx), i32([0]),
                                       nodes=i32([[-1, -1, -1]]), parent=a.parent.cuda())
    assert torch.equal(got["mass"], only_root["mass"]) and torch.isfinite(got["mass"]).all()


# ------------------------------------------------------------------ evict

def _evict_case(spv, seed, lens, budget, sinks, recent, Hkv, D, page, order, kv, W=None, edit=None, in_place=False,
                use_pos=True):
    gen = torch.Generator().manual_seed(seed)
    B = len(lens)
    k, v, _, _, table = ref.make_cache(gen, lens, page, Hkv, D, kv, order, garbage=False)
    W = W or max(max(lens), 1)
    mass = torch.rand(B, Hkv, W, generator=gen)
    pos = torch.arange(W).expand(B, Hkv, W) + (torch.rand(B, Hkv, W, generator=gen) < 0.2).cumsum(-1)
    # an earlier eviction leaves the positions in any order
    pos = torch.stack([torch.stack([x[torch.randperm(W, generator=gen)] for x in row]) for row in pos]).to(torch.int32)
    if not use_pos:
        pos = torch.arange(W, dtype=torch.int32).expand(B, Hkv, W).contiguous()
    if edit:
        edit(mass, pos)
    want = ref.evict(mass, pos, lens, budget, sinks, recent)
    cache = spv.KVCache(to_gpu(k, order), to_gpu(v, order))
    m, p = mass.cuda(), pos.contiguous().cuda()
    out = {"mass": m, "pos": p} if in_place else None
    got = spv.spv_kv_evict(cache, table.cuda(), i32(lens), m, budget, pos=p if use_pos else None, sinks=sinks,
                           recent=recent, out=out)
    torch.cuda.synchronize()
    assert got["lens"].tolist() == [min(n, budget) for n in lens]
    assert (got["row_status"] == 0).all()
    src = got["slot_src"].cpu()
    k, v = ref.bits(k), ref.bits(v)
    k2, v2 = k.clone(), v.clone()
    for b, n in enumerate(lens):
        short = min(n, budget)
        for h in range(Hkv):
            assert src[b, h].tolist() == want[b][h] + [-1] * (budget - short), (b, h)
            s = torch.tensor(want[b][h], dtype=torch.long)
            assert torch.equal(got["mass"][b, h, :short].cpu().view(torch.int32), mass[b, h, s].view(torch.int32))
            assert torch.equal(got["pos"][b, h, :short].cpu(), pos[b, h, s])
            for i, j in enumerate(want[b][h]):
                if i != j:
                    for a, x in ((k, k2), (v, v2)):
                        x[table[b, i // page].long(), i % page, h] = a[table[b, j // page].long(), j % page, h]
    assert torch.equal(ref.bits(cache.k.cpu()), k2) and torch.equal(ref.bits(cache.v.cpu()), v2)
    return cache, got


@pytest.mark.parametrize("case", [
    ([40], 32, 0, 0, 1, 64, 16, "nhd", "bf16"),
    ([100, 33, 32, 31, 0, 64], 32, 4, 8, 2, 64, 16, "hnd", "bf16"),
    ([1000, 2000], 999, 4, 100, 3, 128, 8, "nhd", "f16"),
    ([1025, 3000], 1024, 0, 512, 2, 128, 64, "nhd", "e4m3"),
    ([5000, 1], 1, 0, 0, 1, 256, 16, "nhd", "bf16"),
    ([4097], 2048, 2048, 0, 2, 64, 16, "nhd", "bf16"),
    ([4097, 4096], 2049, 1, 2048, 2, 64, 1, "nhd", "bf16"),
    ([16384, 9000], 8191, 4, 100, 1, 64, 16, "nhd", "bf16"),
    ([20000], 12345, 4, 1000, 1, 64, 16, "nhd", "bf16"),
    ([70001], 65536, 4, 1000, 1, 64, 128, "nhd", "e4m3"),
], ids=lambda c: "-".join(str(x).replace(" ", "") for x in c))
@pytest.mark.parametrize("in_place", [False, True])
def test_evict(spv, case, in_place):
    _evict_case(spv, 31, *case, W=max(case[0]) + 5, in_place=in_place)


def test_evict_slots_as_positions(spv):
    _evict_case(spv, 32, [300, 100], 64, 4, 16, 2, 64, 16, "nhd", "bf16", use_pos=False)


def test_evict_ties_and_odd_weights(spv):
    """Equal weights keep the lower slots; -0 equals 0; NaN goes first; infinities, denormals and negative weights
    are ordered as numbers."""
    def all_equal(mass, pos):
        mass.fill_(0.25)

    def zeros(mass, pos):
        mass[:] = torch.where(torch.rand(mass.shape, generator=torch.Generator().manual_seed(1)) < 0.5, 0.0, -0.0)

    def odd(mass, pos):
        mass[..., ::7] = math.nan
        mass[..., 1::7] = math.inf
        mass[..., 2::7] = -math.inf
        mass[..., 3::7] = 1e-42
        mass[..., 4::7] = -1.0
        mass[..., 5::7] = 0.0

    for edit in (all_equal, zeros, odd):
        for budget in (33, 64, 150, 250):
            _evict_case(spv, 33, [300, 129], budget, 2, 16, 2, 64, 16, "nhd", "bf16", edit=edit)


def test_evict_bad_sequences(spv):
    gen = torch.Generator().manual_seed(3)
    lens = [100] * 5
    k, v, _, _, table = ref.make_cache(gen, lens, 16, 2, 64, "bf16", garbage=False)
    mass = torch.rand(5, 2, 100, generator=gen).cuda()
    for which in ("lens", "pages"):
        cache = spv.KVCache(k.clone().cuda(), v.clone().cuda())
        now, t = list(lens), table.clone()
        if which == "lens":
            now[1], now[2], now[3] = -1, 101, 2 ** 31 - 1
        else:
            t[1, 0], t[2, 6], t[3, 3] = -1, k.shape[0], 2 ** 31 - 1
        got = spv.spv_kv_evict(cache, t.cuda(), i32(now), mass, 48)
        torch.cuda.synchronize()
        assert got["row_status"].tolist() == [0, 4, 4, 4, 0]
        if which == "lens":
            assert got["lens"].tolist() == [48, -1, 101, 2 ** 31 - 1, 48]
            assert (got["slot_src"][1:4] == -1).all()
            for b in (1, 2, 3):
                assert torch.equal(cache.k[table[b].long().cuda()].cpu(), k[table[b].long()])
        else:
            assert got["lens"].tolist() == [48] * 5
            src = got["slot_src"]
            for b in (1, 2, 3):
                for h in range(2):
                    for i, j in enumerate(src[b, h].tolist()):
                        p = table[b, i // 16].long()
                        whole = 0 <= t[b, i // 16] < k.shape[0] and 0 <= t[b, j // 16] < k.shape[0]
                        q = table[b, (j if whole else i) // 16].long()
                        assert torch.equal(cache.k[p, i % 16, h].cpu(), k[q, (j if whole else i) % 16, h])


def test_evicted_cache_attends_as_the_kept_keys(spv):
    """Attention after an eviction equals attention over the kept keys in any order."""
    a = Layer(spv, 34, [300], None, 1, 4, 2, 64, 16)
    mass = torch.rand(1, 2, 301, generator=a.gen)
    got = spv.spv_kv_evict(a.cache, a.table.cuda(), i32([301]), mass.cuda(), 77, recent=8)
    src = got["slot_src"].cpu()
    k, v = a.k.clone(), a.v.clone()
    for h in range(2):
        for i, j in enumerate(src[0, h].tolist()):
            for x, y in ((k, a.k), (v, a.v)):
                x[a.table[0, i // 16].long(), i % 16, h] = y[a.table[0, j // 16].long(), j % 16, h]
    a.k, a.v, a.ctx = k, v, [76]
    a.check(a.attend())


# ------------------------------------------------------------------ rope

@pytest.mark.parametrize("case", [
    # B, T, Hq, Hkv, D, rotary, interleaved, dtype, kv, page, fused
    (1, 1, 32, 8, 128, 128, False, "bf16", "bf16", 16, True),
    (3, 5, 4, 2, 64, 64, True, "f16", "f16", 8, True),
    (2, 7, 8, 8, 128, 64, False, "bf16", "e4m3", 32, True),
    (2, 3, 6, 2, 64, 24, False, "f16", "f16", 1, False),
    (2, 3, 6, 2, 64, 26, False, "bf16", "e4m3", 16, True),
    (2, 3, 6, 2, 64, 26, True, "bf16", "bf16", 16, True),
    (1, 2, 3, 1, 256, 120, False, "f16", "e4m3", 16, False),
    (2, 40, 2, 1, 80, 80, False, "bf16", "bf16", 16, True),
    (1, 9, 2, 2, 512, 512, True, "f16", "f16", 64, True),
    (2, 2, 2, 2, 64, 0, False, "f16", "f16", 16, True),
    (1, 300, 4, 1, 64, 64, False, "bf16", "bf16", 16, True),
], ids=str)
@pytest.mark.parametrize("far", [False, True])
def test_rope(spv, case, far):
    B, T, Hq, Hkv, D, r, inter, dtype, kv, page, fused = case
    gen = torch.Generator().manual_seed(41)
    ctx = [5 + 13 * b for b in range(B)]
    new = [T - (b % 2) * (T // 2) for b in range(B)]
    k, v, ks, vs, table = ref.make_cache(gen, [a + b for a, b in zip(ctx, new)], page, Hkv, D, kv, garbage=False)
    x = torch.randn(B, T, Hq + 2 * Hkv, D, generator=gen).to(DTYPES[dtype])
    base = 10000.0
    inv = [base ** (-2.0 * i / r) for i in range(r // 2)]
    pos = torch.tensor(ctx)[:, None] + torch.arange(T)[None]
    if far:
        pos = pos + 10_000_019
    mscale = 1.25 if far else 1.0
    cache = spv.KVCache(k.clone().cuda(), v.clone().cuda(), ks.cuda() if ks is not None else None,
                        vs.cuda() if vs is not None else None)
    parts = x.cuda().split([Hq, Hkv, Hkv], dim=2)
    if not fused:
        parts = [p.contiguous() for p in parts]
    freqs = spv.spv_rope_frequencies(r, base) if r else torch.empty(0, dtype=torch.int64, device="cuda")
    W = max(ctx) + T + 2
    slot_pos = torch.full((B, Hkv, W), -5, dtype=torch.int32, device="cuda")
    in_place = not fused
    got = spv.spv_rope_append(*parts, cache, table.cuda(), i32(ctx), freqs, interleaved=inter, mscale=mscale,
                              positions=i32(pos.tolist()) if far else None, new_lens=i32(new), slot_pos=slot_pos,
                              out={"q": parts[0]} if in_place else None)
    torch.cuda.synchronize()
    assert (got["row_status"] == 0).all()
    want = ref.rope(x[:, :, : Hq + Hkv], pos, inv, inter, mscale)
    # the pair's size: what a 32-bit cosine (2^-22, angle and function) can be off, then half a step of the type
    size = mscale * 2 * x.double().abs().amax()
    u = half_step(DTYPES[dtype])
    q = got["q"].cpu().double()
    for b in range(B):
        assert (q[b, new[b]:] == 0).all()
        d = (q[b, : new[b]] - want[b, : new[b], :Hq]).abs()
        assert (d <= u * want[b, : new[b], :Hq].abs() + size * 2.0 ** -21).all()
    k2, v2 = k.clone(), v.clone()
    uc = half_step(DTYPES[kv])
    for pool, mine, scale, src in ((cache.k.cpu(), k2, ks, want[:, :, Hq:]), (cache.v.cpu(), v2, vs, x[:, :, Hq + Hkv:].double())):
        for b in range(B):
            for t in range(new[b]):
                at = (table[b, (ctx[b] + t) // page].long(), (ctx[b] + t) % page)
                w = src[b, t] if scale is None else src[b, t] / scale.double()[:, None]
                e = size * 2.0 ** -21 if scale is None else size * 2.0 ** -21 / scale.min().item()
                smallest = 2.0 ** -10 if kv == "e4m3" else 2.0 ** -25  # half of the smallest step
                got8 = ref.bits(pool)[at].view(pool.dtype).double()
                assert ((got8 - w).abs() <= uc * w.abs() + e + smallest).all()
                ref.bits(mine)[at] = ref.bits(pool)[at]
        assert torch.equal(ref.bits(pool), ref.bits(mine))  # nothing else was written
    sp = slot_pos.cpu()
    for b in range(B):
        inside = sp[b, :, ctx[b]: ctx[b] + new[b]]
        assert (inside == pos[b, : new[b]].to(torch.int32)).all()
        assert (sp[b, :, : ctx[b]] == -5).all() and (sp[b, :, ctx[b] + new[b]:] == -5).all()


def test_rope_saturates_e4m3(spv):
    gen = torch.Generator().manual_seed(42)
    k, v, _, _, table = ref.make_cache(gen, [1], 16, 1, 64, "e4m3", garbage=False)
    cache = spv.KVCache(k.cuda(), v.cuda())
    x = torch.full((1, 1, 1, 64), 60000.0, dtype=torch.float16, device="cuda")
    spv.spv_rope_append(x, x, -x, cache, table.cuda(), i32([0]), torch.empty(0, dtype=torch.int64, device="cuda"))
    at = table[0, 0].long().item()
    assert (cache.k[at, 0].float() == 448).all() and (cache.v[at, 0].float() == -448).all()


def test_rope_bad_sequences(spv):
    gen = torch.Generator().manual_seed(43)
    k, v, _, _, table = ref.make_cache(gen, [20] * 4, 16, 2, 64, "bf16", garbage=False)
    cache = spv.KVCache(k.clone().cuda(), v.clone().cuda())
    x = torch.randn(4, 4, 8, 64, generator=gen).bfloat16().cuda()
    q, kk, vv = x.split([4, 2, 2], dim=2)
    t = table.clone()
    t[3, 1] = 10 ** 9
    got = spv.spv_rope_append(q, kk, vv, cache, t.cuda(), i32([16, -1, 30, 14]), spv.spv_rope_frequencies(64))
    torch.cuda.synchronize()
    assert got["row_status"].tolist() == [0, 4, 4, 4]
    assert (got["q"][1:3] == 0).all() and (got["q"][0] != 0).any() and (got["q"][3] != 0).any()
    for b in (1, 2):
        assert torch.equal(cache.k[table[b].long().cuda()].cpu(), k[table[b].long()])
    assert torch.equal(cache.k[table[3, 1].long()].cpu(), k[table[3, 1].long()])
    assert not torch.equal(cache.k[table[3, 0].long()].cpu(), k[table[3, 0].long()])


@pytest.mark.parametrize("scale", [0.0, -0.25, 1.5])
@pytest.mark.parametrize("T, kv", [(2, "bf16"), (2, "e4m3"), (12, "bf16"), (12, "e4m3")])
def test_attention_scale(spv, scale, T, kv):
    """A scale of zero (every visible key alike), a negative one and a large one."""
    a = Layer(spv, 16, [300, 45], None, T, 8, 2, 64, 16, dtype="bf16", kv=kv)
    a.scale = scale
    a.check(a.attend(scale=scale))


@pytest.mark.parametrize("T, Hq, Hkv", [(24, 8, 2), (64, 6, 2), (17, 16, 2), (5, 8, 2)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_attention_growing_maximum(spv, T, Hq, Hkv, D, kv):
    """Scores that grow along the cache, more so in one half of every 128 slots: sums are rescaled on the way."""
    ctx, page = [900, 131, 0], 16
    a = Layer(spv, 21, ctx, None, T, Hq, Hkv, D, page, dtype="bf16", kv=kv)
    gain = torch.ones(a.k.shape[:2])
    for b, n in enumerate(ctx):
        for j in range(n + T):
            gain[a.table[b, j // page].long(), j % page] = (0.1 + 5.0 * j / 1000) * (1.4 if j % 128 >= 64 else 1.0)
    a.k = (a.k.float() * gain[:, :, None, None]).to(DTYPES[kv])
    a.cache.k.copy_(a.k)
    a.check(a.attend())
