"""The calls around the verify step, run together as a serving loop makes them
(examples/decode_loop.py)."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def loop():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("decode_loop", os.path.join(ROOT, "examples", "decode_loop.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_greedy_speculation_decodes_what_one_by_one_does(loop):
    """At T = 0 the drafts change the number of steps, not the tokens."""
    model = loop.ToyModel()
    first = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    emitted, accepted = loop.speculative(model, first, 12)
    n = min(map(len, emitted))
    plain = loop.one_by_one(model, first, n)
    assert [e[:n] for e in emitted] == plain
    assert [len(e) for e in emitted] == (accepted + 1).sum(0).tolist()
    assert 0 < accepted.sum() < accepted.numel() * 4  # some drafts stood and some did not


@pytest.mark.parametrize("temperature", [0.0, 1.0])
def test_budget_holds(loop, temperature):
    """The caches stay within the budget, keep the newest positions, and their weights stay finite."""
    model = loop.ToyModel(layers=1)
    first = torch.tensor([5, 6], dtype=torch.int32, device="cuda")
    sessions = []
    original = loop.Session

    class Watched(original):
        def __init__(self, *a, **kw):
            super().__init__(*a, **kw)
            sessions.append(self)

    loop.Session = Watched
    try:
        emitted, accepted = loop.speculative(model, first, 60, temperature=temperature, budget=48)
    finally:
        loop.Session = original
    s = sessions[0]
    total = (accepted + 1).sum(0)
    assert (total > 48).all() and torch.equal(s.next, total.to(torch.int32))
    assert (s.ctx <= 48).all() and (s.ctx > 0).all()
    for b in range(2):
        n = int(s.ctx[b])
        pos = s.pos[0][b, :, :n]
        assert (pos.sort(-1).values.diff(dim=-1) > 0).all()          # distinct
        assert (pos.amax(-1) == total[b] - 1).all()                  # the newest
        assert (pos.sort(-1).values[:, :4] == torch.arange(4, device="cuda")).all()  # the sinks
        assert (pos.sort(-1).values[:, -32:] == torch.arange(int(total[b]) - 32, int(total[b]), device="cuda")).all()
        assert torch.isfinite(s.mass[0][b, :, :n]).all() and (s.mass[0][b, :, :n] > 0).any()
    assert all(0 <= t < model.vocab for e in emitted for t in e)
