"""Host-side checks of the calls around the verify step that need no GPU:
refusals, workspace sizes and the frequency table."""
import ctypes
import math

import pytest

INV, UNS = 1, 3


@pytest.fixture(scope="module")
def spv():
    from speculative_decoding_token_spv_gb300 import build
    build.build_library()
    import speculative_decoding_token_spv_gb300 as m
    m.load_library()
    return m


def cache(spv, **kw):
    from speculative_decoding_token_spv_gb300 import kv
    a = dict(k=4096, v=8192, dtype=spv.SPV_BF16, num_pages=10, page_size=16, kv_heads=2, head_dim=128,
             k_page_stride=4096, k_slot_stride=256, k_head_stride=128, v_page_stride=4096, v_slot_stride=256,
             v_head_stride=128, k_scale=None, v_scale=None)
    a.update(kw)
    return kv._CacheStruct(*a.values())


P = ctypes.c_void_p
FAKE = P(4096)  # never dereferenced: the checks come first
F = ctypes.c_float

BAD_CACHES = [dict(k=None), dict(v=None), dict(k=4097), dict(v=4104), dict(dtype=0), dict(dtype=9), dict(num_pages=0),
              dict(page_size=0), dict(page_size=24), dict(kv_heads=0), dict(head_dim=0), dict(k_slot_stride=252),
              dict(v_page_stride=-8), dict(k_scale=4096)]


def attention(spv, **kw):
    a = dict(q=FAKE, dt=1, B=2, T=5, Hq=8, c=cache(spv), table=FAKE, pages=4, ctx=FAKE, new=None, parent=None,
             scale=0.1, out=FAKE, lse=None, st=None, ws=P(1 << 20), n=1 << 40)
    a.update(kw)
    c = ctypes.byref(a["c"]) if a["c"] is not None else None
    return spv.load_library().spv_paged_attention(
        a["q"], a["dt"], a["B"], a["T"], a["Hq"], c, a["table"], a["pages"], a["ctx"], a["new"], a["parent"],
        F(a["scale"]), a["out"], a["lse"], a["st"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw", [dict(q=None), dict(dt=0), dict(dt=3), dict(B=0), dict(T=0), dict(Hq=0), dict(Hq=7),
                                dict(table=None), dict(pages=0), dict(ctx=None), dict(out=None), dict(q=P(4104)),
                                dict(out=P(4100)), dict(scale=math.nan), dict(scale=math.inf), dict(ws=None),
                                dict(ws=P((1 << 20) + 8)), dict(n=1000), dict(dt=2), dict(c=None)])
def test_attention_refuses(spv, kw):
    assert attention(spv, **kw) == INV


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_attention_refuses_cache(spv, kw):
    assert attention(spv, c=cache(spv, **kw)) == INV


@pytest.mark.parametrize("kw", [dict(T=65), dict(Hq=130), dict(B=65536)])
def test_attention_unsupported_sizes(spv, kw):
    assert attention(spv, **kw) == UNS


def test_attention_unsupported_cache(spv):
    assert attention(spv, c=cache(spv, head_dim=96)) == UNS
    assert attention(spv, c=cache(spv, head_dim=100)) == UNS
    assert attention(spv, pages=1 << 27) == UNS


def test_attention_workspace(spv):
    f = spv.spv_attention_workspace_bytes
    assert f(1, 1, 32, 8, 128) >= 256
    assert f(64, 5, 64, 8, 128) >= f(1, 1, 32, 8, 128) - (1 << 20)
    for bad in ((0, 1, 8, 8, 128), (1, 0, 8, 8, 128), (1, 1, 7, 8, 128), (1, 65, 8, 8, 128), (1, 1, 8, 8, 80),
                (1, 1, 130, 1, 128)):
        assert f(*bad) == 0
    assert attention(spv, n=f(2, 5, 8, 2, 128) - 1) == INV


def mass(spv, **kw):
    a = dict(q=FAKE, dt=1, B=2, T=5, Hq=8, lse=FAKE, c=cache(spv), table=FAKE, pages=4, ctx=FAKE, scale=0.1,
             acc=FAKE, nodes=None, decay=1.0, min=None, mout=FAKE, stride=64)
    a.update(kw)
    return spv.load_library().spv_attention_mass(
        a["q"], a["dt"], a["B"], a["T"], a["Hq"], a["lse"], ctypes.byref(a["c"]), a["table"], a["pages"], a["ctx"],
        None, None, F(a["scale"]), a["acc"], a["nodes"], F(a["decay"]), a["min"], a["mout"], a["stride"], None, None)


@pytest.mark.parametrize("kw", [dict(q=None), dict(lse=None), dict(acc=None), dict(mout=None), dict(stride=0),
                                dict(decay=math.nan), dict(scale=math.inf), dict(ctx=None), dict(table=None),
                                dict(Hq=9)])
def test_mass_refuses(spv, kw):
    assert mass(spv, **kw) == INV


def test_mass_refuses_cache(spv):
    for kw in BAD_CACHES:
        assert mass(spv, c=cache(spv, **kw)) == INV, kw
    assert mass(spv, T=65) == UNS


def rope(spv, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, dt=1, strides=None, B=2, T=5, Hq=8, freqs=FAKE, r=128, inter=0, m=1.0, pos=None,
             ctx=FAKE, new=None, table=FAKE, pages=4, c=cache(spv), sp=None, ps=0, qo=P(16384))
    a.update(kw)
    s = (ctypes.c_int64 * 6)(*a["strides"]) if a["strides"] else None
    return spv.load_library().spv_rope_append(
        a["q"], a["k"], a["v"], a["dt"], s, a["B"], a["T"], a["Hq"], a["freqs"], a["r"], a["inter"], F(a["m"]),
        a["pos"], a["ctx"], a["new"], a["table"], a["pages"], ctypes.byref(a["c"]), a["sp"], a["ps"], a["qo"], None,
        None)


@pytest.mark.parametrize("kw", [dict(q=None), dict(k=None), dict(v=None), dict(qo=None), dict(freqs=None), dict(r=-2),
                                dict(r=3), dict(r=130), dict(m=math.nan), dict(k=P(4100)), dict(qo=P(8)),
                                dict(strides=[1024, 1024, 4, 256, 256, 256]), dict(strides=[-8, 8, 8, 8, 8, 8]),
                                dict(qo=FAKE, strides=[8192, 1536, 8192, 1536, 8192, 1536]), dict(sp=FAKE, ps=0),
                                dict(dt=0), dict(dt=2), dict(T=0), dict(ctx=None)])
def test_rope_refuses(spv, kw):
    assert rope(spv, **kw) == INV


def test_rope_refuses_cache(spv):
    for kw in BAD_CACHES:
        assert rope(spv, c=cache(spv, **kw)) == INV, kw
    assert rope(spv, c=cache(spv, head_dim=1024)) == UNS
    assert rope(spv, c=cache(spv, head_dim=24, dtype=spv.SPV_E4M3, k_slot_stride=256)) == UNS


def evict(spv, **kw):
    a = dict(c=cache(spv), table=FAKE, pages=4, B=2, lens=FAKE, budget=32, sinks=4, recent=8, mass=FAKE, pos=None,
             stride=64, mo=P(65536), po=None, os=32, nl=FAKE, src=FAKE)
    a.update(kw)
    return spv.load_library().spv_kv_evict(
        ctypes.byref(a["c"]), a["table"], a["pages"], a["B"], a["lens"], a["budget"], a["sinks"], a["recent"],
        a["mass"], a["pos"], a["stride"], a["mo"], a["po"], a["os"], a["nl"], a["src"], None, None)


@pytest.mark.parametrize("kw", [dict(table=None), dict(B=0), dict(lens=None), dict(budget=0), dict(sinks=-1),
                                dict(recent=-1), dict(sinks=20, recent=13), dict(sinks=2**31 - 1), dict(mass=None),
                                dict(mo=None), dict(os=31), dict(mo=FAKE, os=40), dict(pos=FAKE, po=FAKE, os=40),
                                dict(nl=None), dict(src=None), dict(stride=0)])
def test_evict_refuses(spv, kw):
    assert evict(spv, **kw) == INV


def test_evict_refuses_sizes(spv):
    for kw in BAD_CACHES:
        if "k_scale" not in kw:
            assert evict(spv, c=cache(spv, **kw)) == INV, kw
    assert evict(spv, stride=spv.SPV_MAX_EVICT_SLOTS + 1) == UNS
    assert evict(spv, budget=spv.SPV_MAX_EVICT_SLOTS + 1, os=1 << 20) == UNS
    assert evict(spv, B=40000) == UNS


def turns(spv, *a, **kw):
    return [x % (1 << 64) for x in spv.spv_rope_frequencies(*a, device="cpu", **kw).tolist()]


def test_frequencies(spv):
    def near(got, f):  # the table holds round(f / 2 pi 2^64); 2^12 covers the double's own rounding of f
        return all(abs(g - x / (2 * math.pi) * 2.0 ** 64) <= 2.0 ** 12 * max(1.0, x) for g, x in zip(got, f))

    plain = [10000.0 ** (-2.0 * i / 64) for i in range(32)]
    assert near(turns(spv, 64), plain)
    assert near(turns(spv, 64, scaling="linear", factor=8.0), [x / 8 for x in plain])
    b = 500000.0 * 4.0 ** (64 / 62)
    assert near(turns(spv, 64, 500000.0, scaling="base", factor=4.0), [b ** (-2.0 * i / 64) for i in range(32)])
    got = turns(spv, 64, scaling="by_parts", factor=8.0, low=1.0, high=4.0, original_len=8192)
    want = []
    for x in plain:
        n = 8192 * x / (2 * math.pi)
        g = min(1.0, max(0.0, (n - 1) / 3))
        want.append(g * x + (1 - g) * x / 8)
    assert near(got, want)
    # exact at far positions: position times entry, mod one turn, against integers
    p = 1_000_003
    for g, x in zip(turns(spv, 64), plain):
        angle = (p * g % (1 << 64)) / 2.0 ** 64 * 2 * math.pi
        assert abs(math.remainder(angle - p * x, 2 * math.pi)) < 1e-8


@pytest.mark.parametrize("a, kw", [((3,), {}), ((0,), {}), ((2048,), {}), ((64, 0.0), {}), ((64, math.inf), {}),
                                   ((64,), dict(scaling="linear", factor=0.0)), ((2,), dict(scaling="base", factor=2.0)),
                                   ((64,), dict(scaling="by_parts", low=4.0, high=4.0)),
                                   ((64,), dict(scaling="by_parts", original_len=0.0))])
def test_frequencies_refuse(spv, a, kw):
    with pytest.raises(spv.SpvError) as e:
        spv.spv_rope_frequencies(*a, device="cpu", **kw)
    assert e.value.status == INV


def test_frequencies_refuse_scaling_name(spv):
    with pytest.raises(ValueError):
        spv.spv_rope_frequencies(64, scaling="other", device="cpu")


def test_binding_refuses_cpu_tensors(spv):
    import torch
    x = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    c = spv.KVCache(x, x)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        spv.spv_paged_attention(torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16), c, i[None], i)
    with pytest.raises(ValueError):
        spv.spv_kv_evict(c, i[None], i, torch.zeros(1, 2, 64), 8)


def test_cache_struct_matches_header(spv):
    """The binding's struct is laid out as the header's (pointers, int32s, int64s in its order)."""
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = open(os.path.join(root, "include", "spv.h")).read()
    body = re.search(r"typedef struct \{(.*?)\} spv_kv_cache;", src, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    names = []
    for line in body.split(";"):
        line = re.sub(r"^\s*(const\s+)?(void|spv_dtype|int32_t|int64_t|float)\b", "", line.strip())
        names += [n.strip(" *\n") for n in line.split(",") if n.strip()]
    from speculative_decoding_token_spv_gb300 import kv
    assert names == [n for n, _ in kv._CacheStruct._fields_]
    assert ctypes.sizeof(kv._CacheStruct) == 8 * 2 + 4 * 5 + 4 + 8 * 6 + 8 * 2


def test_give_up_arguments(spv):
    f = spv.load_library().spv_selftest_give_up
    assert f(-2, 0) == INV and f(0, -1) == INV and f(-1, 0) == 0
