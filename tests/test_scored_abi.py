"""Host-side checks that need no GPU of the calls for attention that is not
plain and of prompts: refusals, workspace sizes, the layout of spv_scores."""
import ctypes
import math
import os
import re
import struct

import pytest

from test_kv_abi import BAD_CACHES, F, FAKE, INV, P, UNS, cache, spv  # noqa: F401  (spv is a fixture)


class ScoresStruct(ctypes.Structure):
    _fields_ = [("cap", ctypes.c_float), ("slopes", P), ("window", ctypes.c_int32), ("first", P), ("last", P), ("slot_pos", P),
                ("pos_stride", ctypes.c_int64)]


def scores(**kw):
    a = dict(cap=0.0, slopes=None, window=0, first=None, last=None, slot_pos=None, pos_stride=0)
    a.update(kw)
    return ctypes.byref(ScoresStruct(*a.values()))


BAD_SCORES = [dict(cap=-1.0), dict(cap=math.nan), dict(cap=math.inf), dict(cap=1e-35), dict(window=-1),
              dict(slot_pos=4096, pos_stride=0)]


def norm_rope(spv, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, dt=1, strides=None, B=2, T=5, Hq=8, qw=FAKE, kw=FAKE, eps=1e-6, freqs=FAKE, axes=None, n=1,
             r=128, inter=0, m=1.0, pos=None, ctx=FAKE, table=FAKE, pages=4, c=cache(spv), sp=None, ps=0, qo=P(16384))
    a.update(kw)
    s = (ctypes.c_int64 * 6)(*a["strides"]) if a["strides"] else None
    return spv.load_library().spv_norm_rope_append(
        a["q"], a["k"], a["v"], a["dt"], s, a["B"], a["T"], a["Hq"], a["qw"], a["kw"], F(a["eps"]), a["freqs"], a["axes"], a["n"],
        a["r"], a["inter"], F(a["m"]), a["pos"], a["ctx"], None, a["table"], a["pages"], ctypes.byref(a["c"]), a["sp"], a["ps"],
        a["qo"], None, None)


@pytest.mark.parametrize("kw", [dict(q=None), dict(k=None), dict(v=None), dict(qo=None), dict(freqs=None), dict(r=-2), dict(r=3),
                                dict(r=130), dict(m=math.nan), dict(k=P(4100)), dict(strides=[-8, 8, 8, 8, 8, 8]),
                                dict(qo=FAKE, strides=[8192, 1536, 8192, 1536, 8192, 1536]), dict(sp=FAKE, ps=0), dict(dt=0),
                                dict(T=0), dict(ctx=None), dict(eps=-1e-6), dict(eps=math.nan), dict(eps=math.inf), dict(n=0),
                                dict(n=9, pos=FAKE), dict(n=3)])
def test_norm_rope_refuses(spv, kw):  # noqa: F811
    assert norm_rope(spv, **kw) == INV


def test_norm_rope_refuses_cache(spv):  # noqa: F811
    for kw in BAD_CACHES:
        assert norm_rope(spv, c=cache(spv, **kw)) == INV, kw
    assert norm_rope(spv, c=cache(spv, head_dim=264, k_slot_stride=528, v_slot_stride=528)) == UNS


def attention(spv, **kw):
    a = dict(q=FAKE, dt=1, B=2, T=5, Hq=8, c=cache(spv), table=FAKE, pages=4, ctx=FAKE, parent=None, scale=0.1, s=scores(),
             out=FAKE, ws=P(1 << 20), n=1 << 40)
    a.update(kw)
    c = ctypes.byref(a["c"]) if a["c"] is not None else None
    return spv.load_library().spv_paged_attention_scored(
        a["q"], a["dt"], a["B"], a["T"], a["Hq"], c, a["table"], a["pages"], a["ctx"], None, a["parent"], F(a["scale"]), a["s"],
        a["out"], None, None, a["ws"], a["n"], None)


def prompt(spv, **kw):
    a = dict(q=FAKE, dt=1, B=2, T=500, Hq=8, c=cache(spv), table=FAKE, pages=40, ctx=FAKE, scale=0.1, s=scores(), out=FAKE,
             ws=P(1 << 20), n=1 << 40)
    a.update(kw)
    c = ctypes.byref(a["c"]) if a["c"] is not None else None
    return spv.load_library().spv_prompt_attention(
        a["q"], a["dt"], a["B"], a["T"], a["Hq"], c, a["table"], a["pages"], a["ctx"], None, F(a["scale"]), a["s"], a["out"], None,
        None, a["ws"], a["n"], None)


@pytest.mark.parametrize("call", [attention, prompt])
@pytest.mark.parametrize("kw", [dict(q=None), dict(dt=0), dict(dt=3), dict(B=0), dict(T=0), dict(Hq=0), dict(Hq=7),
                                dict(table=None), dict(pages=0), dict(ctx=None), dict(out=None), dict(q=P(4104)),
                                dict(out=P(4100)), dict(scale=math.nan), dict(scale=math.inf), dict(ws=None),
                                dict(ws=P((1 << 20) + 8)), dict(n=1000), dict(dt=2), dict(c=None)])
def test_attention_refuses(spv, call, kw):  # noqa: F811
    assert call(spv, **kw) == INV


@pytest.mark.parametrize("kw", BAD_SCORES)
def test_scores_are_refused(spv, kw):  # noqa: F811
    assert attention(spv, s=scores(**kw)) == INV
    assert prompt(spv, s=scores(**kw)) == INV
    assert mass(spv, s=scores(**kw)) == INV


def test_scores_and_trees(spv):  # noqa: F811
    assert attention(spv, s=None) == INV and mass(spv, s=None) == INV
    for call in (attention, mass):
        assert call(spv, s=scores(last=4096), parent=FAKE) == INV


@pytest.mark.parametrize("call", [attention, prompt])
def test_attention_refuses_cache(spv, call):  # noqa: F811
    for kw in BAD_CACHES:
        assert call(spv, c=cache(spv, **kw)) == INV, kw
    assert call(spv, c=cache(spv, head_dim=96)) == UNS
    assert call(spv, Hq=130) == UNS and call(spv, B=65536) == UNS
    assert call(spv, pages=1 << 27) == UNS


def test_lengths(spv):  # noqa: F811
    assert attention(spv, T=65) == UNS
    assert prompt(spv, T=(1 << 24) // 4 + 1) == UNS


def test_prompt_workspace(spv):  # noqa: F811
    f = spv.spv_prompt_workspace_bytes
    assert f(1, 1, 32, 8, 128) == f(64, 100000, 64, 8, 128) > 256
    for bad in ((0, 1, 8, 8, 128), (1, 0, 8, 8, 128), (1, 1, 7, 8, 128), (1, 1, 8, 8, 80), (1, 1, 130, 1, 128), (1, 1 << 24, 16, 8, 64)):
        assert f(*bad) == 0
    assert prompt(spv, n=f(2, 500, 8, 2, 128) - 1) == INV


def mass(spv, **kw):
    a = dict(q=FAKE, dt=1, B=2, T=5, Hq=8, lse=FAKE, c=cache(spv), table=FAKE, pages=4, ctx=FAKE, parent=None, scale=0.1, s=scores(),
             acc=FAKE, nodes=None, decay=1.0, mout=FAKE, stride=64)
    a.update(kw)
    return spv.load_library().spv_attention_mass_scored(
        a["q"], a["dt"], a["B"], a["T"], a["Hq"], a["lse"], ctypes.byref(a["c"]), a["table"], a["pages"], a["ctx"], None,
        a["parent"], F(a["scale"]), a["s"], a["acc"], a["nodes"], F(a["decay"]), None, a["mout"], a["stride"], None, None)


@pytest.mark.parametrize("kw", [dict(q=None), dict(lse=None), dict(acc=None), dict(mout=None), dict(stride=0),
                                dict(decay=math.nan), dict(scale=math.inf), dict(ctx=None), dict(table=None), dict(Hq=9)])
def test_mass_refuses(spv, kw):  # noqa: F811
    assert mass(spv, **kw) == INV


def test_scores_struct_matches_header(spv):  # noqa: F811
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = open(os.path.join(root, "include", "spv.h")).read()
    body = re.findall(r"typedef struct \{((?:(?!typedef).)*?)\} spv_scores;", src, re.S)[0]
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    names = []
    for line in body.split(";"):
        line = re.sub(r"^\s*(const\s+)?(int32_t|int64_t|float)\b", "", line.strip())
        names += [n.strip(" *\n") for n in line.split(",") if n.strip()]
    assert names == [n for n, _ in ScoresStruct._fields_]
    from speculative_decoding_token_spv_gb300 import kv
    want = bytes(ScoresStruct(1.5, 16, 7, 32, 48, 64, 9))
    got = kv._PACK_SCORES(1.5, 16, 7, 32, 48, 64, 9)
    assert len(got) == ctypes.sizeof(ScoresStruct)
    assert struct.unpack("@fPiPPPq", got) == struct.unpack("@fPiPPPq", want)


def test_binding_refuses(spv):  # noqa: F811
    import torch
    x = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    c = spv.KVCache(x, x)
    i = torch.zeros(1, dtype=torch.int32)
    q = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16)
    for call in (lambda: spv.spv_paged_attention_scored(q, c, i[None], i, spv.Scores()),
                 lambda: spv.spv_prompt_attention(q, c, i[None], i),
                 lambda: spv.spv_attention_mass_scored(q, torch.zeros(1, 1, 4), c, i[None], i, i, spv.Scores()),
                 lambda: spv.spv_norm_rope_append(q, q, q, c, i[None], i, torch.zeros(32, dtype=torch.int64))):
        with pytest.raises(ValueError):
            call()
    dev = torch.device("cpu")
    with pytest.raises(ValueError):
        spv.Scores(cap="a").packed(1, 1, 4, 2, dev)
    with pytest.raises(ValueError):
        spv.Scores(window=1 << 40).packed(1, 1, 4, 2, dev)
    with pytest.raises(ValueError):
        spv.Scores(slot_pos=i).packed(1, 1, 4, 2, dev)
    with pytest.raises(ValueError):  # slopes on the host
        spv.Scores(slopes=torch.zeros(3)).packed(1, 1, 4, 2, dev)
