"""Host-side checks that a call given a stream allocates and clears its own
buffers on that stream: the library and torch's stream context are fakes, no
GPU is needed."""
import contextlib
from types import SimpleNamespace

import pytest
import torch

import speculative_decoding_token_spv_gb300 as spv
from speculative_decoding_token_spv_gb300 import kv

I32 = torch.int32
STREAM = SimpleNamespace(cuda_stream=77)


class Library:
    """Every entry point succeeds; what it was called with, by name."""

    def __init__(self):
        self.calls = {}

    def __getattr__(self, name):
        def call(*args):
            self.calls[name] = args
            return 4096 if name.endswith("_workspace_bytes") else 0
        return call


@pytest.fixture
def world(monkeypatch):
    """Records the stream that is current at each allocation."""
    w = SimpleNamespace(lib=Library(), current="the caller's", made=[])

    @contextlib.contextmanager
    def stream(s):
        before, w.current = w.current, s
        yield
        w.current = before

    def recorded(make):
        def call(*args, **kw):
            w.made.append(w.current)
            return make(*args, **kw)
        return call

    monkeypatch.setattr(torch.cuda, "stream", stream)
    for m in (spv, kv):
        monkeypatch.setattr(m, "load_library", lambda: w.lib)
    monkeypatch.setattr(spv, "_cuda", lambda t, name, dtype=None: t)
    for name in ("empty", "zeros"):
        monkeypatch.setattr(torch, name, recorded(getattr(torch, name)))
    return w


def check(w, name, made):
    assert len(w.made) == made and all(s is STREAM for s in w.made), w.made
    assert 77 in w.lib.calls[name]
    assert w.current == "the caller's"


class Cache:
    def packed(self):
        return b"", torch.device("cpu"), (4, 16, 2, 64)


def test_attention_and_mass(world):
    q, table = torch.ones(1, 3, 4, 64, dtype=torch.bfloat16), torch.ones(1, 2, dtype=I32)
    one = torch.ones(1, dtype=I32)
    spv.spv_paged_attention(q, Cache(), table, one, want_lse=True, stream=STREAM)
    check(world, "spv_paged_attention", 4)  # the workspace, out, lse, row_status
    world.made.clear()
    spv.spv_attention_mass(q, torch.ones(1, 3, 4), Cache(), table, one, one, stream=STREAM)
    check(world, "spv_attention_mass", 2)


def test_rope_and_evict(world):
    q, k, table = torch.ones(1, 3, 4, 64).bfloat16(), torch.ones(1, 3, 2, 64).bfloat16(), torch.ones(1, 2, dtype=I32)
    one = torch.ones(1, dtype=I32)
    spv.spv_rope_append(q, k, k, Cache(), table, one, torch.ones(32, dtype=torch.int64), stream=STREAM)
    check(world, "spv_rope_append", 2)
    world.made.clear()
    spv.spv_kv_evict(Cache(), table, one, torch.ones(1, 2, 32), 8, stream=STREAM)
    check(world, "spv_kv_evict", 5)


LOGITS, DRAFT = torch.ones(1, 3, 8), torch.ones(1, 2, 8)
TOKENS, R, KEYS = torch.ones(1, 2, dtype=I32), torch.ones(1, 2), torch.ones(1, dtype=torch.int64)
CHAIN = (LOGITS, DRAFT, TOKENS, R, KEYS, 1.0)
TREE = (LOGITS, LOGITS, torch.ones(1, 3, dtype=I32), torch.ones(1, 3, dtype=I32), torch.ones(1, 3), KEYS, 1.0)
IDS = torch.ones(1, 6, dtype=I32)


@pytest.mark.parametrize("name, args, made", [  # the workspace, then the outputs
    ("spv_verify_chain", CHAIN, 5),
    ("spv_verify_chain_cached", (*CHAIN, IDS, [2, 2, 2]), 6),
    ("spv_verify_chain_saguaro", (*CHAIN, IDS, [2, 2, 2], 2.0), 6),
    ("spv_verify_chain_filtered", (*CHAIN, 4, 0.9), 5),
    ("spv_verify_tree", TREE, 5),
    ("spv_verify_greedy", (LOGITS, TOKENS), 4),
    ("spv_fanout_topk", (LOGITS, torch.ones(1, 3, dtype=I32), [2, 2, 2]), 3),
])
def test_verify_calls(world, name, args, made):
    getattr(spv, name)(*args, stream=STREAM)
    check(world, name, made)
