"""Plain 64-bit forms of the attention calls with scores and masks, of prompts
and of the head norms with rotation, on the CPU, and the inputs of their tests.
Shares no code with the kernels."""
import math

import torch

import kv_reference as ref
from kv_reference import DTYPES, half_step


def depths(parent, T):
    """Levels of the new tokens below the first (-1: the path to the root leaves the tree)."""
    if parent is None:
        return list(range(T))
    out = [0]
    for v in range(1, T):
        p = parent[v]
        out.append(-1 if p < 0 or p >= v or out[p] < 0 else out[p] + 1)
    return out


def visibility(ctx, new, T, parent, first, last, window, pos):
    """bool [new, ctx + new]; pos: positions of the slots [ctx + new] (own tokens at ctx + t)."""
    n = ctx + new
    slot = torch.arange(n)
    see = torch.zeros(new, n, dtype=torch.bool)
    for t in range(new):
        row = torch.zeros(n, dtype=torch.bool)
        if parent is None:
            row = slot <= ctx + t
            if last is not None:
                row |= slot < last[t]
        else:
            path, ok = [t], True
            while path[-1] != 0:
                p = parent[path[-1]]
                if p < 0 or p >= path[-1]:
                    ok = False
                    break
                path.append(p)
            if ok:
                row[:ctx] = True
                for u in path:
                    if ctx + u < n:
                        row[ctx + u] = True
        if first is not None:
            row &= slot >= first[t]
        if window:
            row &= pos[ctx + t] - pos < window
        see[t] = row
    return see


class Case:
    """Inputs of the calls, on the CPU and the GPU, and their 64-bit results."""

    def __init__(self, spv, seed, ctx, new, T, Hq, Hkv, D, page, order="nhd", dtype="bf16", kv=None, tree=False, cap=0.0,
                 slopes=False, window=0, first=None, last=None, moved=False, spread=2.0, scale=None, poison=True):
        gen = torch.Generator().manual_seed(seed)
        self.spv, self.gen = spv, gen
        self.B, self.T, self.Hq, self.Hkv, self.D = len(ctx), T, Hq, Hkv, D
        self.ctx, self.new = list(ctx), list(new) if new is not None else [T] * len(ctx)
        self.ragged = new is not None
        lens = [a + b for a, b in zip(self.ctx, self.new)]
        self.k, self.v, self.ks, self.vs, self.table = ref.make_cache(gen, lens, page, Hkv, D, kv or dtype, order)
        self.q = (torch.randn(self.B, T, Hq, D, generator=gen) * spread).to(DTYPES[dtype])
        self.parent = torch.tensor([ref.random_tree(gen, T) for _ in ctx], dtype=torch.int32) if tree else None
        self.cap, self.window = cap, window
        self.slopes = torch.exp2(-8.0 * torch.rand(Hq, generator=gen)) if slopes else None
        self.first = torch.tensor(first, dtype=torch.int32) if first is not None else None
        self.last = torch.tensor(last, dtype=torch.int32) if last is not None else None
        self.slot_pos = None
        if moved:
            W = max(lens) + 3
            steps = torch.randint(1, 4, (self.B, Hkv, W), generator=gen)
            pos = steps.cumsum(-1)
            for b in range(self.B):  # cached slots in any order, as evictions leave them
                perm = torch.randperm(self.ctx[b], generator=gen)
                pos[b, :, : self.ctx[b]] = pos[b][:, perm]
            self.slot_pos = pos.to(torch.int32)
        self.scale = 1.0 / math.sqrt(D) if scale is None else scale
        self.order = order
        self.seen = [self._seen(b) for b in range(self.B)]
        if poison:
            self._poison(page)

    def _positions(self, b, h):
        ctx, new = self.ctx[b], self.new[b]
        if self.slot_pos is not None:
            return self.slot_pos[b, h, : ctx + new].long()
        deep = depths(None if self.parent is None else self.parent[b].tolist(), self.T)
        return torch.cat([torch.arange(ctx), ctx + torch.tensor(deep[:new], dtype=torch.long)])

    def _seen(self, b):
        """[Hkv, new, n]"""
        return torch.stack([visibility(self.ctx[b], self.new[b], self.T, None if self.parent is None else self.parent[b].tolist(),
                                       None if self.first is None else self.first[b], None if self.last is None else self.last[b],
                                       self.window, self._positions(b, h)) for h in range(self.Hkv)])

    def _poison(self, page):
        """Slots that no token of their sequence and head sees hold NaN."""
        if self.k.element_size() == 1:
            return
        for b in range(self.B):
            for h in range(self.Hkv):
                for j in (~self.seen[b][h].any(0)).nonzero().flatten().tolist():
                    at = self.table[b, j // page].long(), j % page, h
                    self.k[at] = math.nan
                    self.v[at] = math.nan

    # ------------------------------------------------------------ calls
    def cache(self):
        if not hasattr(self, "_cache"):
            move = lambda x: (x.transpose(1, 2).contiguous().cuda().transpose(1, 2) if self.order == "hnd" else x.contiguous().cuda())  # noqa: E731
            self._cache = self.spv.KVCache(move(self.k), move(self.v), None if self.ks is None else self.ks.cuda(),
                                           None if self.vs is None else self.vs.cuda())
        return self._cache

    def scores(self):
        up = lambda x: None if x is None else x.cuda()  # noqa: E731
        return self.spv.Scores(cap=self.cap, slopes=up(self.slopes), window=self.window, first=up(self.first), last=up(self.last),
                               slot_pos=up(self.slot_pos))

    def i32(self, x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def attend(self, prompt=False, **kw):
        args = dict(new_lens=self.i32(self.new) if self.ragged else None, scale=self.scale, want_lse=True)
        if prompt:
            got = self.spv.spv_prompt_attention(self.q.cuda(), self.cache(), self.table.cuda(), self.i32(self.ctx), self.scores(),
                                                **{**args, **kw})
        else:
            got = self.spv.spv_paged_attention_scored(self.q.cuda(), self.cache(), self.table.cuda(), self.i32(self.ctx),
                                                      self.scores(), parent=None if self.parent is None else self.parent.cuda(),
                                                      **{**args, **kw})
        torch.cuda.synchronize()
        return got

    # ------------------------------------------------------------ 64 bits
    def weights(self, b, h):
        """(p [new, G, n], lse [new, G], ds [new, G, n]): weights in 64 bits, and how far a score may be off: D + 4
        roundings of 2^-24 of its terms' size; 2^-20 of a capped score (tanh: an exponential and a reciprocal of 2^-22,
        or the polynomial's 2^-22 and its roundings); 2^-22 of the bias and of the score (their products with log2 e,
        and the difference with the maximum)."""
        new, n, G = self.new[b], self.ctx[b] + self.new[b], self.Hq // self.Hkv
        K = ref.rows(self.k, self.table[b], n)[:, h]
        if self.ks is not None:
            K = K * self.ks[h].double()
        q = self.q[b, :new, h * G:(h + 1) * G].double()
        K = torch.nan_to_num(K)  # poisoned slots are seen by nobody
        x = self.scale * torch.einsum("tgd,nd->tgn", q, K)
        size = abs(self.scale) * torch.einsum("tgd,nd->tgn", q.abs(), K.abs())
        ds = (self.D + 4) * 2.0 ** -24 * size
        if self.cap:
            x = self.cap * torch.tanh(x / self.cap)
            ds = ds + 2.0 ** -20 * x.abs()
        if self.slopes is not None:
            pos = self._positions(b, h)
            far = (pos[self.ctx[b]:, None] - pos[None]).abs().double()[:, None]
            bias = self.slopes[h * G:(h + 1) * G].double()[None, :, None] * far
            x = x - bias
            ds = ds + 2.0 ** -22 * bias
        ds = ds + 2.0 ** -22 * x.abs()
        x = x.masked_fill(~self.seen[b][h][:, None], -math.inf)
        z = torch.logsumexp(x, -1)
        p = torch.exp(x - z.masked_fill(z == -math.inf, 0.0)[..., None])
        return p, z, ds

    def attention(self):
        """(out, lse, bound, lse_bound): `bound` what a kernel with 32-bit sums and weights rounded to 16 bits may be off
        besides the rounding of the result."""
        G, u = self.Hq // self.Hkv, half_step(self.q.dtype)
        out = torch.zeros(self.B, self.T, self.Hq, self.D, dtype=torch.float64)
        lse = torch.full((self.B, self.T, self.Hq), -math.inf, dtype=torch.float64)
        bound, lse_bound = torch.zeros_like(out), torch.zeros_like(lse)
        for b in range(self.B):
            new, n = self.new[b], self.ctx[b] + self.new[b]
            if new == 0:
                continue
            V = torch.nan_to_num(ref.rows(self.v, self.table[b], n))
            if self.vs is not None:
                V = V * self.vs.double()[:, None]
            for h in range(self.Hkv):
                p, z, ds = self.weights(b, h)
                mean = (p * ds).sum(-1, keepdim=True)
                # a weight: its own rounding, its score's and the sum's error, the exponential's 2^-21, sums of n terms
                # of mixed sign as sqrt(n) + 8 roundings; and the smallest step of a 16-bit weight of each key
                dp = p * (u + 2 * ds + 2 * mean + 2.0 ** -21 + (n ** 0.5 + 8) * 2.0 ** -23)
                top = p.amax(-1, keepdim=True)
                tiny = 2.0 ** -24 * top * self.seen[b][h][:, None].double()
                g = slice(h * G, (h + 1) * G)
                out[b, :new, g] = p @ V[:, h]
                bound[b, :new, g] = (dp + tiny) @ V[:, h].abs()
                lse[b, :new, g] = z
                lse_bound[b, :new, g] = 2 * mean.squeeze(-1) + 2.0 ** -20 + torch.nan_to_num(z.abs(), posinf=0.0) * 2.0 ** -22
        return out, lse, bound, lse_bound

    def check(self, got, status=0):
        out, lse, bound, lse_bound = self.attention()
        x = got["out"].cpu().double()
        tol = half_step(self.q.dtype) * (out.abs() + bound) + bound + (2.0 ** -24 if self.q.dtype == torch.float16 else 0)
        assert torch.isfinite(x).all(), f"{(~torch.isfinite(x)).sum()} not finite"
        worst = ((x - out).abs() - tol).max().item()
        assert worst <= 0, f"out: {worst} beyond the bound at {((x - out).abs() - tol).argmax().item()}"
        z = got["lse"].cpu().double()
        assert torch.equal(torch.isinf(z), torch.isinf(lse))
        fine = torch.isfinite(lse)
        assert ((z - lse).abs() <= lse_bound)[fine].all(), ((z - lse).abs() / lse_bound)[fine].max()
        assert (got["row_status"].cpu() == status).all()

    def mass(self, counted, decay, mass_in):
        """(mass [B, Hkv, W] with NaN where nothing is written, bound)."""
        W = mass_in.shape[2]
        mass = torch.full((self.B, self.Hkv, W), math.nan, dtype=torch.float64)
        bound = torch.zeros(self.B, self.Hkv, W, dtype=torch.float64)
        for b in range(self.B):
            n = self.ctx[b] + self.new[b]
            mass[b, :, :n] = 0
            mass[b, :, : self.ctx[b]] = decay * mass_in[b, :, : self.ctx[b]].double()
            bound[b, :, :n] = mass[b, :, :n].abs() * 2.0 ** -22
            rows = [t for t in counted[b] if t < self.new[b]]
            for h in range(self.Hkv):
                p, z, ds = self.weights(b, h)
                w, z, ds = p[rows], z[rows], ds[rows]
                z = torch.nan_to_num(z, neginf=0.0)
                mass[b, h, :n] += w.sum((0, 1))
                # the score's and lse's errors, lse's own rounding, the exponential's
                mean = (w * ds).sum(-1, keepdim=True)
                bound[b, h, :n] += (w * (2 * ds + 2 * mean + 2.0 ** -18 + z.abs()[..., None] * 2.0 ** -21)).sum((0, 1))
        return mass, bound


def norm_rope(x, weight, eps, positions, axes, inv_freq, interleaved, mscale):
    """float64: heads of x [B, T, H, D] normed by weight (None: not), then turned; positions [B, T, axes]; axes: the axis
    of each pair, or None."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps) * weight.double()
    x = x.clone()
    n = len(inv_freq)
    if n == 0:
        return x
    where = positions[..., list(axes) if axes is not None else [0] * n].double()
    angle = (where * torch.tensor(inv_freq, dtype=torch.float64))[:, :, None]
    c, s = mscale * torch.cos(angle), mscale * torch.sin(angle)
    a = (x[..., 0:2 * n:2] if interleaved else x[..., :n]).clone()
    b = (x[..., 1:2 * n:2] if interleaved else x[..., n:2 * n]).clone()
    if interleaved:
        x[..., 0:2 * n:2], x[..., 1:2 * n:2] = a * c - b * s, b * c + a * s
    else:
        x[..., :n], x[..., n:2 * n] = a * c - b * s, b * c + a * s
    return x
