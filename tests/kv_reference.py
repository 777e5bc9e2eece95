"""Plain 64-bit forms of the calls around the verify step, on the CPU, and the
random inputs of their tests.  Shares no code with the kernels."""
import math

import torch

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}


def half_step(dtype):
    """Largest relative error of one rounding to the type."""
    return torch.finfo(dtype).eps / 2


def make_cache(gen, lens, page, Hkv, D, kv, order="nhd", spare=2, width=None, garbage=True):
    """(k, v, k_scale, v_scale, table) on the CPU; slots past a sequence's end hold NaN where the type has one, and
    table entries past its pages are outside the pool."""
    counts = [-(-n // page) for n in lens]
    pages = sum(counts) + spare
    width = width or max(max(counts), 1)
    table = torch.full((len(lens), width), -7, dtype=torch.int32)
    perm = torch.randperm(pages, generator=gen).to(torch.int32)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = perm[at:at + c]
        at += c
    gain = 8.0 if kv == "e4m3" else 1.0
    pools = []
    for _ in range(2):
        x = (torch.randn(pages, page, Hkv, D, generator=gen) * gain).to(DTYPES[kv])
        if garbage:
            used = torch.zeros(pages, page, dtype=torch.bool)
            for b, n in enumerate(lens):
                for j in range(n):
                    used[table[b, j // page].long(), j % page] = True
            x = x.float()
            x[~used] = math.nan
            x = x.to(DTYPES[kv])
        pools.append(x if order == "nhd" else x.transpose(1, 2).contiguous().transpose(1, 2))
    scales = [0.05 + 0.1 * torch.rand(Hkv, generator=gen) if kv == "e4m3" else None for _ in range(2)]
    return pools[0], pools[1], scales[0], scales[1], table


def bits(pool):
    """The pool's elements as integers (8-bit floats cannot be indexed on the CPU)."""
    return pool.view(torch.int8 if pool.element_size() == 1 else torch.int16)


def rows(pool, table_row, n):
    """Slots 0..n-1 of a sequence as float64 [n, Hkv, D]."""
    page = pool.shape[1]
    j = torch.arange(n)
    return bits(pool)[table_row.long()[j // page], j % page].view(pool.dtype).double()


def visible(t, ctx, n, parent):
    """bool [n]: what token t sees (parent: list, or None for a chain)."""
    see = torch.zeros(n, dtype=torch.bool)
    path = [t]
    if parent is None:
        path = list(range(t + 1))
    else:
        while path[-1] != 0:
            p = parent[path[-1]]
            if p < 0 or p >= path[-1]:
                return see
            path.append(p)
    see[:ctx] = True
    for u in path:
        if ctx + u < n:
            see[ctx + u] = True
    return see


def attention(q, k, v, ks, vs, table, ctx, new, parent, scale):
    """float64 (out [B, T, Hq, D], lse [B, T, Hq], bound): `bound` holds what a kernel with 32-bit sums and
    probabilities rounded to q's type may be off, besides the rounding of the result."""
    B, T, Hq, D = q.shape
    Hkv = k.shape[2]
    G = Hq // Hkv
    out = torch.zeros(B, T, Hq, D, dtype=torch.float64)
    lse = torch.full((B, T, Hq), -math.inf, dtype=torch.float64)
    bound = torch.zeros_like(out)
    lse_bound = torch.zeros_like(lse)
    u = half_step(q.dtype)
    for b in range(B):
        n = ctx[b] + new[b]
        K, V = rows(k, table[b], n), rows(v, table[b], n)
        if ks is not None:
            K, V = K * ks.double()[:, None], V * vs.double()[:, None]
        for t in range(new[b]):
            see = visible(t, ctx[b], n, None if parent is None else parent[b].tolist())
            if not see.any():
                continue
            x = q[b, t].double().reshape(Hkv, G, D)
            Ks, Vs = K[see].transpose(0, 1), V[see].transpose(0, 1)  # [Hkv, n', D]
            s = scale * torch.einsum("hgd,hnd->hgn", x, Ks)
            size = abs(scale) * torch.einsum("hgd,hnd->hgn", x.abs(), Ks.abs()).amax(-1)
            z = torch.logsumexp(s, -1)
            p = torch.exp(s - z[..., None])
            out[b, t] = torch.einsum("hgn,hnd->hgd", p, Vs).reshape(Hq, D)
            lse[b, t] = z.reshape(Hq)
            # a score is off by at most D + 4 roundings of 2^-24 of its terms' size; a probability by twice the
            # worst score error, the exponential's 2^-21 and its own rounding; the sums by n roundings, taken as
            # sqrt(n) + 8 of them (they are of mixed sign), and the smallest step of a 16-bit probability
            ds = (D + 4) * 2.0 ** -24 * size
            dp = u + 2 * ds + 2.0 ** -21 + (see.sum().item() ** 0.5 + 8) * 2.0 ** -23
            mass = torch.einsum("hgn,hnd->hgd", p, Vs.abs())
            tiny = 2.0 ** -24 * Vs.abs().sum(1)[:, None, :] * torch.exp(s.amax(-1) - z)[..., None]
            bound[b, t] = (dp[..., None] * mass + tiny).reshape(Hq, D)
            lse_bound[b, t] = (2 * ds + 2.0 ** -20 + z.abs() * 2.0 ** -22).reshape(Hq)
    return out, lse, bound, lse_bound


def attention_mass(q, k, ks, table, ctx, new, parent, scale, counted, decay, mass_in):
    """float64 mass [B, Hkv, W] (NaN where nothing is written) and the bound of a 32-bit computation."""
    B, T, Hq, D = q.shape
    Hkv = k.shape[2]
    G = Hq // Hkv
    W = mass_in.shape[2]
    mass = torch.full((B, Hkv, W), math.nan, dtype=torch.float64)
    bound = torch.zeros(B, Hkv, W, dtype=torch.float64)
    for b in range(B):
        n = ctx[b] + new[b]
        K = rows(k, table[b], n)
        if ks is not None:
            K = K * ks.double()[:, None]
        mass[b, :, :n] = 0
        mass[b, :, :ctx[b]] = decay * mass_in[b, :, :ctx[b]].double()
        bound[b, :, :n] = mass[b, :, :n].abs() * 2.0 ** -22
        for t in counted[b]:
            if t >= new[b]:
                continue
            see = visible(t, ctx[b], n, None if parent is None else parent[b].tolist())
            if not see.any():
                continue
            x = q[b, t].double().reshape(Hkv, G, D)
            Ks = K[see].transpose(0, 1)
            s = scale * torch.einsum("hgd,hnd->hgn", x, Ks)
            size = abs(scale) * torch.einsum("hgd,hnd->hgn", x.abs(), Ks.abs()).amax(-1)
            z = torch.logsumexp(s, -1, keepdim=True)
            p = torch.exp(s - z)
            mass[b, :, :n][:, see] += p.sum(1)
            # score error, lse given in 32 bits and its own error, products of the logarithms, the exponential
            rel = 2 * (D + 4) * 2.0 ** -24 * size + 2.0 ** -18 + z.squeeze(-1).abs() * 2.0 ** -21
            bound[b, :, :n][:, see] += (p * rel[..., None]).sum(1)
    return mass, bound


def evict(mass, pos, lens, budget, sinks, recent):
    """slot_src as nested lists [B][Hkv] of the sources, by Python sorting."""
    out = []
    for b in range(mass.shape[0]):
        n, heads = lens[b], []
        m = min(n, budget)
        for h in range(mass.shape[1]):
            w, p = mass[b, h, :n].tolist(), pos[b, h, :n].tolist()
            top = max(p) if p else 0

            def key(j):
                if p[j] < sinks or p[j] > top - recent:
                    return (0, 0.0, j)
                if math.isnan(w[j]):
                    return (2, 0.0, j)
                return (1, -w[j], j)

            best = sorted(range(n), key=key)[:m]
            kept, movers = set(best), sorted(j for j in best if j >= m)
            heads.append([i if i in kept else movers.pop(0) for i in range(m)])
        out.append(heads)
    return out


def rope(x, positions, inv_freq, interleaved, mscale):
    """float64 rotation of x [B, T, H, D] at integer positions [B, T]."""
    x = x.double().clone()
    r = 2 * len(inv_freq)
    f = torch.tensor(inv_freq, dtype=torch.float64)
    angle = positions.double()[:, :, None, None] * f
    c, s = mscale * torch.cos(angle), mscale * torch.sin(angle)
    a = (x[..., 0:r:2] if interleaved else x[..., :r // 2]).clone()
    b = (x[..., 1:r:2] if interleaved else x[..., r // 2:r]).clone()
    if interleaved:
        x[..., 0:r:2], x[..., 1:r:2] = a * c - b * s, b * c + a * s
    else:
        x[..., :r // 2], x[..., r // 2:r] = a * c - b * s, b * c + a * s
    return x


def random_tree(gen, T):
    return [-1] + [int(torch.randint(0, v, (1,), generator=gen)) for v in range(1, T)]
