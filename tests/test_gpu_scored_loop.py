"""The calls with scores, head norms and prompts, run together as a serving loop
makes them (examples/decode_loop.py): every call against its 64-bit form on what
the calls before it left."""
import importlib.util
import math
import os

import pytest
import torch

import kv_reference as ref
import scored_reference as sr

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


def case_of(session, layer, q, ctx, lens):
    """What an attention call of the session was given, as the 64-bit form takes it: the caches as they are now."""
    m, cache, scores = session.model, session.caches[layer], session.model.scores(layer, session.pos[layer])
    c = sr.Case.__new__(sr.Case)
    c.B, c.T, c.Hq, c.Hkv, c.D = *q.shape[:2], m.heads, m.kv_heads, m.head_dim
    c.ctx, c.new = ctx, lens
    c.k, c.v, c.ks, c.vs, c.table, c.q = cache.k.cpu(), cache.v.cpu(), None, None, session.table.cpu(), q.cpu()
    c.parent = c.first = c.last = None
    c.cap, c.window, c.slopes = scores.cap, scores.window, None if scores.slopes is None else scores.slopes.cpu()
    c.slot_pos, c.scale = session.pos[layer].cpu(), 1.0 / math.sqrt(m.head_dim)
    c.seen = [c._seen(b) for b in range(c.B)]
    return c


@pytest.mark.parametrize("head_dim", [64, 128])
def test_every_call_of_a_run(loop, head_dim):
    """A prompt, decode steps, weights, an eviction, and steps over the slots that it moved."""
    model = loop.ToyModel(layers=2, head_dim=head_dim, shaped=True)
    session = loop.Session(model, 3, 330, 4)
    gen = torch.Generator().manual_seed(5)
    seen = {"appended": 0, "attended": 0, "weighed": 0}
    attend = session.attend

    def checked(layer, q, k, v, positions, lens):
        ctx = session.ctx.tolist()
        new = [q.shape[1]] * 3 if lens is None else lens.tolist()
        got_q, out, lse = attend(layer, q, k, v, positions, lens)
        # q and K of the new tokens: the formula in 64 bits, off by 2^-20 of a head's size and half a step of bf16
        freqs = [2.0 * math.pi * f / 2.0 ** 64 for f in (int(x) % 2 ** 64 for x in model.freqs.tolist())]
        for x, weight, got in ((q, 0, got_q.cpu()), (k, 1, None)):
            want = sr.norm_rope(x.cpu(), model.norms[layer][weight].cpu(), 1e-6, positions.cpu()[..., None], None, freqs, False, 1.0)
            size = want.square().sum(-1, keepdim=True).sqrt()
            for b in range(3):
                for t in range(new[b]):
                    slot = ctx[b] + t
                    y = got[b, t] if got is not None else session.caches[layer].k[session.table[b, slot // 16].item(), slot % 16].cpu()
                    tol = ref.half_step(torch.bfloat16) * want[b, t].abs() + 2.0 ** -18 * size[b, t]
                    assert ((y.double() - want[b, t]).abs() <= tol).all()
        seen["appended"] += 1
        c = case_of(session, layer, got_q, ctx, new)
        c.check({"out": out, "lse": lse, "row_status": torch.zeros(3)})
        seen["attended"] += 1
        return got_q, out, lse

    session.attend = checked

    def step():
        fed = torch.randint(0, model.vocab, (3, 5), generator=gen, dtype=torch.int32).cuda()
        session.forward(fed)
        count = torch.randint(0, 5, (3,), generator=gen, dtype=torch.int32)
        before = [(c, m.cpu().clone()) for c, m in zip((case_of(session, i, session.kept[i][0], session.ctx.tolist(), [5] * 3)
                                                        for i in range(model.layers)), session.mass)]
        session.commit(count.cuda())
        for layer, (c, mass_in) in enumerate(before):
            want, bound = c.mass([list(range(k + 1)) for k in count.tolist()], 1.0, mass_in)
            there = ~torch.isnan(want)
            off = (session.mass[layer].cpu().double() - want).abs()[there] - bound[there] - 2.0 ** -24 * want.abs()[there]
            assert off.max() <= 0, off.max()
            seen["weighed"] += 1

    session.prefill([torch.randint(0, model.vocab, (n,), generator=gen).tolist() for n in (130, 71, 200)])
    for _ in range(2):
        step()
    session.evict(120)
    assert (session.ctx <= 120).all()
    for _ in range(2):
        step()
    assert seen == {"appended": 10, "attended": 10, "weighed": 8}


@pytest.mark.parametrize("temperature", [0.0, 1.0])
def test_shaped_run_within_its_budget(loop, temperature):
    model = loop.ToyModel(shaped=True)
    prompts = [list(range(100)), list(range(40, 110))]
    first = torch.tensor([5, 6], dtype=torch.int32, device="cuda")
    emitted, accepted = loop.speculative(model, first, 12, temperature=temperature, budget=80, prompts=prompts)
    assert [len(e) for e in emitted] == (accepted + 1).sum(0).tolist()
    assert all(0 <= t < model.vocab for e in emitted for t in e)


def test_a_prompt_in_pieces_decodes_the_same_keys(loop):
    """The first layer's keys of a prompt do not depend on how it is fed: whole, or five tokens a step."""
    model = loop.ToyModel(layers=1, shaped=True)
    tokens = [(11 * i) % model.vocab for i in range(75)]
    whole, pieces = (loop.Session(model, 1, 80, 4) for _ in range(2))
    whole.prefill([tokens])
    for i in range(0, 75, 5):
        pieces.forward(torch.tensor([tokens[i:i + 5]], dtype=torch.int32, device="cuda"))
        pieces.commit(torch.tensor([4], dtype=torch.int32, device="cuda"))
    for slot in range(75):
        a, b = (s.caches[0].k[s.table[0, slot // 16].item(), slot % 16].double() for s in (whole, pieces))
        # the projection's products may be summed in another order: two roundings apart before the norm, one after
        assert ((a - b).abs() <= 3 * 2.0 ** -8 * a.abs() + 2.0 ** -7 * a.square().mean(-1, keepdim=True).sqrt()).all()
        assert torch.equal(whole.pos[0][0, :, slot], pieces.pos[0][0, :, slot])


def test_a_step_captured_and_replayed(loop):
    """Append, attention and weights of a step in one graph: replayed after the lengths and the inputs have changed, it gives
    what the calls give."""
    spv, m = loop.spv, loop.ToyModel(layers=1, shaped=True)
    gen = torch.Generator(device="cuda").manual_seed(9)
    B, T, Hq, Hkv, D, pages = 3, 5, m.heads, m.kv_heads, m.head_dim, 20
    pools = [torch.randn(B * pages, 16, Hkv, D, generator=gen, device="cuda").bfloat16() for _ in range(2)]
    table = torch.arange(B * pages, dtype=torch.int32, device="cuda").reshape(B, pages)
    qkv = torch.empty(B, T, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device="cuda")
    ctx, accept = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
    pos = torch.arange(pages * 16, dtype=torch.int32, device="cuda").expand(B, Hkv, -1).contiguous()
    mass = torch.zeros(B, Hkv, pages * 16, device="cuda")
    workspace = spv.new_workspace(spv.spv_attention_workspace_bytes(B, T, Hq, Hkv, D), "cuda")
    outs = [dict(q=torch.empty(B, T, Hq, D, dtype=torch.bfloat16, device="cuda")),
            dict(out=torch.empty(B, T, Hq, D, dtype=torch.bfloat16, device="cuda"), lse=torch.empty(B, T, Hq, device="cuda")),
            dict(mass=mass)]

    def step():
        cache = spv.KVCache(*pools)
        q, k, v = qkv.split([Hq, Hkv, Hkv], dim=2)
        q = spv.spv_norm_rope_append(q, k, v, cache, table, ctx, m.freqs, q_weight=m.norms[0][0], k_weight=m.norms[0][1], slot_pos=pos,
                                     out=outs[0], want_status=False)["q"]
        scores = m.scores(1, pos)
        got = spv.spv_paged_attention_scored(q, cache, table, ctx, scores, workspace=workspace, out=outs[1], want_lse=True,
                                             want_status=False)
        spv.spv_attention_mass_scored(q, got["lse"], cache, table, ctx, accept, scores, mass_in=mass, out=outs[2], want_status=False)

    def state():
        return [x.clone() for x in (*pools, pos, mass)]

    def restore(saved):
        for x, y in zip((*pools, pos, mass), saved):
            x.copy_(y)

    qkv.normal_(generator=gen)
    step()  # as a user would before a capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens, counts in (([0, 17, 200], [0, 4, 2]), ([90, 300, 5], [4, 4, 0]), ([315, 64, 16], [1, 0, 3])):
        qkv.normal_(generator=gen)
        ctx.copy_(torch.tensor(lens, dtype=torch.int32))
        accept.copy_(torch.tensor(counts, dtype=torch.int32))
        before = state()
        step()
        want = [x.clone() for x in (*state(), outs[0]["q"], outs[1]["out"], outs[1]["lse"])]
        restore(before)
        for x in (outs[0]["q"], outs[1]["out"], outs[1]["lse"]):
            x.zero_()
        graph.replay()
        for a, b in zip((*state(), outs[0]["q"], outs[1]["out"], outs[1]["lse"]), want):
            assert torch.equal(a, b)
