"""Speculative decoding of a toy model with a paged, budgeted cache: every call
of the library around one verify step, in the order a serving loop makes them.

    python examples/decode_loop.py [--steps 40] [--budget 96]

Per step, for the last emitted token and gamma drafted ones of each sequence:
each layer projects q, k, v, `spv_rope_append` rotates them and writes the
cache, `spv_paged_attention` attends; `spv_verify_chain` decides how many drafts
stand; `spv_attention_mass` adds up what each cached key received from the
tokens that stand; and once a sequence's cache has outgrown its budget,
`spv_kv_evict` cuts it back.  Weights are random, the "draft model" is the
target's own embedding, so that some drafts stand and some do not.

With --shaped the model's heads are normed (`spv_norm_rope_append`), its layers
take turns at a sliding window and at a distance bias, both with capped scores
(`spv_paged_attention_scored`, `spv_attention_mass_scored`), and each sequence
begins with a prompt (`spv_prompt_attention`).
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_token_spv_gb300 as spv  # noqa: E402

PAGE = 16


class ToyModel:
    """A small decoder-only transformer with random bf16 weights."""

    def __init__(self, vocab=1024, layers=2, heads=8, kv_heads=2, head_dim=64, seed=0, device="cuda", shaped=False):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.vocab, self.heads, self.kv_heads, self.head_dim, self.device = vocab, heads, kv_heads, head_dim, device
        width = heads * head_dim
        draw = lambda *shape: torch.randn(*shape, generator=g, device=device).mul_(shape[0] ** -0.5).bfloat16()  # noqa: E731
        self.embed = draw(width, vocab).t().contiguous() * 8.0
        self.qkv = [draw(width, (heads + 2 * kv_heads) * head_dim) * 2.0 for _ in range(layers)]
        self.proj = [draw(width, width) for _ in range(layers)]
        self.shaped = shaped
        if shaped:
            self.norms = [(0.5 + torch.rand(2, head_dim, generator=g, device=device)) for _ in range(layers)]  # of q and of k
            self.slopes = torch.exp2(-8.0 * torch.arange(1, heads + 1, device=device) / heads)
        self.freqs = spv.spv_rope_frequencies(head_dim, scaling="by_parts", factor=4.0, original_len=2048, device=device)

    @property
    def layers(self):
        return len(self.qkv)

    def scores(self, layer, pos):
        """Scores of a shaped model's layer; pos: where its cached keys stood in the text."""
        if layer % 2 == 0:
            return spv.Scores(cap=30.0, window=64, slot_pos=pos)
        return spv.Scores(cap=30.0, slopes=self.slopes, slot_pos=pos)

    def draft(self, tokens):
        """Draft logits [B, vocab]: the next token from the last one alone."""
        return (self.embed[tokens.long()] @ self.embed.t()).float() * 0.05


def normed(x):
    return x * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6).to(x.dtype)


class Session:
    """The caches of a batch: per layer pages, weights and positions of the cached keys; one page table for all."""

    def __init__(self, model, batch, slots, gamma):
        m, dev = model, model.device
        self.model, self.batch, self.gamma = m, batch, gamma
        per = -(-slots // PAGE)
        self.table = torch.randperm(batch * per, device=dev).to(torch.int32).reshape(batch, per)
        pool = lambda: torch.zeros(batch * per, PAGE, m.kv_heads, m.head_dim, dtype=torch.bfloat16, device=dev)  # noqa: E731
        self.caches = [spv.KVCache(pool(), pool()) for _ in range(m.layers)]
        self.mass = [torch.zeros(batch, m.kv_heads, per * PAGE, device=dev) for _ in range(m.layers)]
        self.pos = [torch.zeros(batch, m.kv_heads, per * PAGE, dtype=torch.int32, device=dev) for _ in range(m.layers)]
        self.ctx = torch.zeros(batch, dtype=torch.int32, device=dev)    # cached slots
        self.next = torch.zeros(batch, dtype=torch.int32, device=dev)   # position of the next token fed
        self.slots = per * PAGE

    def forward(self, tokens, lens=None):
        """Logits [B, T, vocab] of the fed tokens (the first lens [B] of them), whose keys and values enter the cache;
        q and lse are kept for commit()."""
        m, (B, T) = self.model, tokens.shape
        x = m.embed[tokens.long()]
        positions = (self.next[:, None] + torch.arange(T, device=x.device, dtype=torch.int32)).contiguous()
        self.kept = []
        for layer in range(m.layers):
            heads = (normed(x) @ m.qkv[layer]).view(B, T, m.heads + 2 * m.kv_heads, m.head_dim)
            q, out, lse = self.attend(layer, *heads.split([m.heads, m.kv_heads, m.kv_heads], dim=2), positions, lens)
            self.kept.append((q, lse))
            x = x + out.reshape(B, T, -1) @ m.proj[layer]
        return (normed(x) @ m.embed.t()).float()

    def attend(self, layer, q, k, v, positions, lens):
        """q as it was attended with, what it took, and its log-sum-exp."""
        m, cache, T = self.model, self.caches[layer], q.shape[1]
        where = (cache, self.table, self.ctx)
        if not m.shaped:
            q = spv.spv_rope_append(q, k, v, *where, m.freqs, positions=positions, slot_pos=self.pos[layer], new_lens=lens)["q"]
            got = spv.spv_paged_attention(q, *where, new_lens=lens, workspace=self._workspace(T), want_lse=True)
            return q, got["out"], got["lse"]
        q_weight, k_weight = m.norms[layer]
        q = spv.spv_norm_rope_append(q, k, v, *where, m.freqs, q_weight=q_weight, k_weight=k_weight, positions=positions,
                                     slot_pos=self.pos[layer], new_lens=lens)["q"]
        call = spv.spv_paged_attention_scored if T <= 64 else spv.spv_prompt_attention
        got = call(q, *where, m.scores(layer, self.pos[layer]), new_lens=lens, workspace=self._workspace(T), want_lse=True)
        return q, got["out"], got["lse"]

    def prefill(self, prompts):
        """Logits [B, vocab] behind each prompt; prompts: a list of token lists."""
        lens = torch.tensor([len(x) for x in prompts], dtype=torch.int32, device=self.model.device)
        tokens = torch.zeros(len(prompts), int(lens.max()), dtype=torch.int32, device=lens.device)
        for b, x in enumerate(prompts):
            tokens[b, : len(x)] = torch.tensor(x, dtype=torch.int32)
        logits = self.forward(tokens, lens)
        self.ctx += lens
        self.next += lens
        return logits[torch.arange(len(prompts)), lens.long() - 1]

    def _workspace(self, T):
        m = self.model
        size = spv.spv_attention_workspace_bytes if T <= 64 else spv.spv_prompt_workspace_bytes
        need = size(self.batch, T, m.heads, m.kv_heads, m.head_dim)
        if getattr(self, "ws", None) is None or self.ws.numel() < need:
            self.ws = spv.new_workspace(need, m.device)
        return self.ws

    def commit(self, accept_count):
        """The last fed step stands up to accept_count drafts: weights of the cached keys, then the new lengths."""
        for layer, (q, lse) in enumerate(self.kept):
            args, to = (q, lse, self.caches[layer], self.table, self.ctx, accept_count), {"mass": self.mass[layer]}
            if self.model.shaped:
                spv.spv_attention_mass_scored(*args, self.model.scores(layer, self.pos[layer]), mass_in=self.mass[layer], out=to)
            else:
                spv.spv_attention_mass(*args, mass_in=self.mass[layer], out=to)
        self.ctx += accept_count + 1
        self.next += accept_count + 1

    def evict(self, budget, sinks=4, recent=32):
        for layer, cache in enumerate(self.caches):
            got = spv.spv_kv_evict(cache, self.table, self.ctx, self.mass[layer], budget, pos=self.pos[layer], sinks=sinks,
                                   recent=recent, out={"mass": self.mass[layer], "pos": self.pos[layer]})
        self.ctx = got["lens"]


def speculative(model, first, steps, gamma=4, temperature=0.0, budget=None, seed=1, prompts=None):
    """Decodes from the tokens `first` [B], behind `prompts` if there are any; returns each sequence's tokens and the accepted drafts of every step [steps, B]."""
    B, dev = first.shape[0], model.device
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    before = max(map(len, prompts)) if prompts else 0
    session = Session(model, B, max(budget, before) + gamma + 1 if budget else before + (steps + 1) * (gamma + 1), gamma)
    if prompts:
        session.prefill(prompts)
    last, emitted, accepted = first, [[] for _ in range(B)], []
    for _ in range(steps):
        fed, rows = [last], []
        for _ in range(gamma):
            rows.append(model.draft(fed[-1]))
            pick = rows[-1].argmax(-1) if temperature == 0 else torch.multinomial(
                torch.softmax(rows[-1] / temperature, -1), 1, generator=g).squeeze(1)
            fed.append(pick.to(torch.int32))
        fed = torch.stack(fed, 1).contiguous()
        target = session.forward(fed)
        r = 1.0 - torch.rand(B, gamma, generator=g, device=dev)
        keys = torch.randint(-2 ** 63, 2 ** 63 - 1, (B,), generator=g, device=dev)
        got = spv.spv_verify_chain(target, torch.stack(rows, 1).contiguous(), fed[:, 1:].contiguous(), r, keys, temperature)
        k = got["accept_count"]
        session.commit(k)
        if budget and bool((session.ctx > budget).any()):
            session.evict(budget)
        for b, row in enumerate(got["out_tokens"].tolist()):
            emitted[b] += [t for t in row if t >= 0]
        last = got["out_tokens"].gather(1, k.long()[:, None]).squeeze(1)
        accepted.append(k.clone())
    return emitted, torch.stack(accepted)


def one_by_one(model, first, tokens, prompts=None):
    """Greedy decoding without drafts: one token a step."""
    session = Session(model, first.shape[0], tokens + 1 + (max(map(len, prompts)) if prompts else 0), 0)
    if prompts:
        session.prefill(prompts)
    last, out = first, []
    none = torch.zeros_like(first)
    for _ in range(tokens):
        last = session.forward(last[:, None].contiguous())[:, 0].argmax(-1).to(torch.int32)
        session.commit(none)
        out.append(last)
    return torch.stack(out, 1).tolist()


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--budget", type=int, default=96)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--shaped", action="store_true", help="normed heads, windows, distance biases, capped scores and prompts")
    a = ap.parse_args()
    model = ToyModel(shaped=a.shaped)
    prompts = [[(7 * i + b) % model.vocab for i in range(90 + 40 * b)] for b in range(a.batch)] if a.shaped else None
    first = torch.arange(1, a.batch + 1, dtype=torch.int32, device=model.device)
    for temperature in (0.0, 1.0):
        emitted, accepted = speculative(model, first, a.steps, temperature=temperature, budget=a.budget, prompts=prompts)
        print(f"T = {temperature}: {sum(map(len, emitted))} tokens in {a.steps} steps of {a.batch} sequences, "
              f"{accepted.float().mean():.2f} of 4 drafts accepted a step, cache cut to {a.budget} slots")


if __name__ == "__main__":
    main()
