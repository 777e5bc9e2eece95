"""GPU tests of forms of the calls around the verify step that only larger
calls take: rotary appends of several tokens a block, pages beyond a tile,
heads of 256, counted rows beyond one pass, evictions of long caches."""
import pytest
import torch

from test_gpu_kv import Layer, _evict_case, _mass_case, spv  # noqa: F401  (spv: the fixture)
from test_gpu_kv import test_rope as rope_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", [
    # B, T, Hq, Hkv, D, rotary, interleaved, dtype, kv, page, fused (else in place); 4,864 tokens or more, T and the
    # lengths of every second sequence of any remainder by four
    (3, 2001, 4, 2, 128, 128, False, "bf16", "bf16", 16, True),
    (3, 2003, 6, 2, 64, 64, True, "f16", "e4m3", 32, True),
    (3, 1998, 2, 1, 64, 24, False, "bf16", "bf16", 16, False),
    (3, 2003, 2, 1, 64, 24, False, "f16", "e4m3", 8, True),
    (3, 2001, 2, 2, 64, 26, True, "f16", "f16", 8, False),
    (3, 1998, 2, 2, 64, 26, True, "bf16", "e4m3", 8, True),
    (3, 2003, 3, 1, 128, 64, False, "f16", "e4m3", 64, False),
    (20, 251, 24, 2, 256, 256, True, "bf16", "bf16", 16, True),   # more heads than are read ahead
    (20, 253, 52, 2, 256, 256, False, "f16", "e4m3", 16, True),
], ids=str)
@pytest.mark.parametrize("far", [False, True])
def test_rope_of_many_tokens(spv, case, far):
    rope_case(spv, case, far)


@pytest.mark.parametrize("case", [
    # ctx, new, T, Hq, Hkv, D, page, order, dtype, kv, tree
    ([600, 1000, 255], None, 12, 8, 2, 128, 256, "nhd", "bf16", "bf16", False),
    ([600, 256, 257, 0], [12, 3, 1, 5], 12, 8, 2, 64, 256, "hnd", "f16", "f16", False),
    ([1500, 130], None, 40, 8, 2, 128, 1024, "nhd", "bf16", "bf16", True),
    ([700, 130], None, 5, 8, 2, 128, 512, "hnd", "f16", "f16", False),
    ([700, 130], None, 12, 8, 2, 128, 256, "nhd", "bf16", "e4m3", False),
    ([500, 1000], None, 1, 8, 2, 128, 256, "nhd", "f16", "f16", False),
    ([70, 300], None, 21, 8, 2, 256, 16, "nhd", "bf16", "bf16", True),
    ([70, 300, 0], [63, 20, 1], 63, 6, 2, 256, 32, "hnd", "f16", "f16", True),
    ([129, 40], None, 33, 8, 1, 256, 16, "nhd", "bf16", "e4m3", True),
    ([300, 5], [7, 5], 7, 64, 2, 256, 64, "hnd", "f16", "e4m3", False),
    ([300], None, 64, 8, 1, 128, 16, "nhd", "bf16", "bf16", True),    # four times 128 rows
    ([300, 17], None, 50, 6, 1, 64, 16, "hnd", "f16", "e4m3", True),
], ids=lambda c: "-".join(str(x).replace(" ", "") for x in c[2:]))
def test_attention_forms(spv, case):
    ctx, new, T, Hq, Hkv, D, page, order, dtype, kv, tree = case
    a = Layer(spv, 61, ctx, new, T, Hq, Hkv, D, page, order, dtype, kv, tree)
    a.check(a.attend())


@pytest.mark.parametrize("case", [
    # ctx, new, T, Hq, Hkv, D, page, order, dtype, kv, tree, accept
    ([99, 401], None, 3, 7, 1, 256, 16, "hnd", "bf16", "e4m3", False, [2, 1]),
    ([300, 40], None, 9, 8, 1, 256, 16, "nhd", "bf16", "e4m3", False, [8, 5]),      # 72 rows: three passes of 32
    ([300, 40, 129], [9, 2, 9], 9, 16, 2, 256, 32, "hnd", "f16", "f16", False, [8, 1, 4]),  # two of 64
    ([260, 40], None, 20, 16, 1, 128, 256, "nhd", "bf16", "bf16", False, [19, 3]),  # three of 128
    ([260, 40], None, 20, 16, 1, 64, 16, "nhd", "f16", "e4m3", False, [19, 7]),
], ids=lambda c: "-".join(str(x).replace(" ", "") for x in c[2:]))
def test_mass_of_many_rows(spv, case):
    *rest, accept = case
    _mass_case(spv, 62, *rest, accept, decay=0.5)


@pytest.mark.parametrize("D, kv", [(128, "e4m3"), (256, "e4m3"), (256, "bf16")])
def test_mass_tree_forms(spv, D, kv):
    _mass_case(spv, 63, [200, 31, 0], None, 21, 16, 2, D, 16, "nhd", "bf16", kv, True, [3, 0, 1], [[1, 5, 13], [], [2]])


@pytest.mark.parametrize("case", [
    ([50001, 49153, 10], 49000, 4, 1000, 1, 64, 16, "nhd", "bf16"),
    ([131073], 131000, 0, 50, 2, 64, 64, "hnd", "e4m3"),
    ([49152, 49151], 49100, 4, 0, 1, 64, 16, "nhd", "f16"),
], ids=lambda c: "-".join(str(x).replace(" ", "") for x in c))
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_long(spv, case, in_place):
    _evict_case(spv, 64, *case, W=max(case[0]) + 3, in_place=in_place)


def test_evict_long_ties(spv):
    def edit(mass, pos):
        mass.fill_(0.5)
        mass[..., 49000:] = 0.75

    _evict_case(spv, 65, [50001], 48990, 1, 16, 1, 64, 16, "nhd", "bf16", edit=edit)
