"""The target model's attention layer around a verify step: binding of
spv_rope_append, spv_paged_attention, spv_attention_mass and spv_kv_evict.

Like the verify calls: torch CUDA tensors in, work on torch's current stream
(or ``stream``), outputs allocated when the caller passes none in ``out``, no
CPU fallback.  A cache is two 4-D pools [pages, page_size, kv_heads, head_dim];
any strides will do as long as a row's elements are contiguous, so
``pool.transpose(1, 2)`` of a [pages, kv_heads, page_size, head_dim] tensor or
a slice of a joint K/V tensor can be passed.
"""
from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass

import torch

from . import SPV_BF16, SPV_E4M3, SPV_F16, _check, _cuda, _ptr, _stream, load_library, new_workspace

ROPE_SCALINGS = {"plain": 0, "linear": 1, "base": 2, "by_parts": 3}
_ACTIVATIONS = {torch.bfloat16: SPV_BF16, torch.float16: SPV_F16}
_CACHES = {**_ACTIVATIONS, torch.float8_e4m3fn: SPV_E4M3}


class _CacheStruct(ctypes.Structure):
    _fields_ = ([("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int)]
                + [(n, ctypes.c_int32) for n in ("num_pages", "page_size", "kv_heads", "head_dim")]
                + [(f"{p}_{n}_stride", ctypes.c_int64) for p in "kv" for n in ("page", "slot", "head")]
                + [("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)])


@dataclass
class KVCache:
    """A paged cache: pools k, v [pages, page_size, kv_heads, head_dim] of one
    dtype (bfloat16, float16 or float8_e4m3fn) and, for float8, what an element
    stands for: [kv_heads] float32 scales (None: 1)."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor | None = None
    v_scale: torch.Tensor | None = None

    def struct(self) -> _CacheStruct:
        k, v = self.k, self.v
        for name, t in (("cache.k", k), ("cache.v", v)):
            if not isinstance(t, torch.Tensor) or not t.is_cuda:
                raise ValueError(f"{name} must be a CUDA tensor")
            if t.dim() != 4 or (t.shape[3] > 1 and t.stride(3) != 1):
                raise ValueError(f"{name} must be [pages, page_size, kv_heads, head_dim] with contiguous rows")
            if t.dtype not in _CACHES:
                raise TypeError(f"{name} must be bfloat16, float16 or float8_e4m3fn, got {t.dtype}")
        if k.shape != v.shape or k.dtype != v.dtype or k.device != v.device:
            raise ValueError("cache.k and cache.v must have the same shape, dtype and device")
        for name, s in (("k_scale", self.k_scale), ("v_scale", self.v_scale)):
            if s is not None:
                _on(_cuda(s, name, torch.float32), name, k.device)
                if tuple(s.shape) != (k.shape[2],):
                    raise ValueError(f"{name} must be [kv_heads]")
        # a dimension of one entry may carry any stride: it is never stepped over
        strides = [t.stride(i) if t.shape[i] > 1 else 0 for t in (k, v) for i in (0, 1, 2)]
        return _CacheStruct(_ptr(k), _ptr(v), _CACHES[k.dtype], *k.shape, *strides, _ptr(self.k_scale),
                            _ptr(self.v_scale))


def _on(t, name, device):
    if t is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    return t


def _ints(t, name, shape, device):
    """An optional int32 tensor of the given shape."""
    if t is None:
        return None
    _on(_cuda(t, name, torch.int32), name, device)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return t


def _floats(t, name, shape, device):
    if t is None:
        return None
    _on(_cuda(t, name, torch.float32), name, device)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return t


def _output(out, key, shape, dtype, device):
    """The caller's output tensor `key`, checked, or a new one."""
    t = out.get(key)
    if t is None:
        t = out[key] = torch.empty(shape, dtype=dtype, device=device)
        return t
    _on(_cuda(t, f"out[{key!r}]", dtype), f"out[{key!r}]", device)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"out[{key!r}] must be {list(shape)}, got {list(t.shape)}")
    return t


def _table(page_table, B, device):
    _on(_cuda(page_table, "page_table", torch.int32), "page_table", device)
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError("page_table must be [B, max_pages]")
    return page_table


def _queries(q, cache):
    """Checks q [B, T, q_heads, head_dim] against the cache: its sizes, dtype code and the cache struct."""
    c = cache.struct()
    q = _on(_cuda(q, "q"), "q", cache.k.device)
    if q.dim() != 4 or q.shape[3] != c.head_dim:
        raise ValueError("q must be [B, T, q_heads, head_dim]")
    if q.dtype not in _ACTIVATIONS:
        raise TypeError(f"q must be bfloat16 or float16, got {q.dtype}")
    return c, *q.shape[:3], _ACTIVATIONS[q.dtype]


def spv_rope_frequencies(rotary_dim: int, base: float = 10000.0, *, scaling: str = "plain", factor: float = 1.0,
                         low: float = 1.0, high: float = 4.0, original_len: float = 8192.0,
                         device="cuda") -> torch.Tensor:
    """The frequency table of :func:`spv_rope_append` (see spv_rope_frequencies
    in spv.h): int64 [rotary_dim / 2] holding uint64 bit patterns, on `device`.
    scaling: one of ROPE_SCALINGS."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}")
    host = torch.empty(max(int(rotary_dim) // 2, 0), dtype=torch.int64)
    _check(load_library().spv_rope_frequencies(int(rotary_dim), float(base), ROPE_SCALINGS[scaling], float(factor),
                                               float(low), float(high), float(original_len), host.data_ptr()),
           "spv_rope_frequencies")
    return host.to(device)


def spv_rope_append(q, k, v, cache: KVCache, page_table, ctx_lens, freqs, *, interleaved: bool = False,
                    mscale: float = 1.0, positions=None, new_lens=None, slot_pos=None, out=None,
                    want_status: bool = True, stream=None) -> dict:
    """Rotary positions for q [B, T, q_heads, D] and k [B, T, kv_heads, D], and
    k, v into the cache's slots ctx_lens[b] + t (see spv_rope_append in spv.h).

    q, k and v may be views of one projection's output: heads contiguous, any
    batch and token strides.  freqs: :func:`spv_rope_frequencies` of the
    rotary_dim.  Returns dict(q, and row_status when requested); out["q"] may
    be q itself."""
    c = cache.struct()
    dev = cache.k.device
    if not isinstance(q, torch.Tensor) or q.dim() != 4 or q.shape[3] != c.head_dim:
        raise ValueError("q must be [B, T, q_heads, head_dim]")
    B, T, Hq, D = q.shape
    if q.dtype not in _ACTIVATIONS:
        raise TypeError(f"q must be bfloat16 or float16, got {q.dtype}")
    strides = []
    for name, t, heads in (("q", q, Hq), ("k", k, c.kv_heads), ("v", v, c.kv_heads)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        _on(t, name, dev)
        if t.dtype != q.dtype:
            raise TypeError(f"{name} must be {q.dtype}, got {t.dtype}")
        if tuple(t.shape) != (B, T, heads, D):
            raise ValueError(f"{name} must be [B, T, {heads}, {D}]")
        if t.stride(3) != 1 or (heads > 1 and t.stride(2) != D):
            raise ValueError(f"{name}: the heads of a token must be contiguous")
        strides += [t.stride(0) if B > 1 else 0, t.stride(1) if T > 1 else 0]
    if strides[0] == 0:  # one sequence: the packed stride, so that q can be its own output
        strides[0] = T * Hq * D
    if strides[1] == 0:
        strides[1] = Hq * D
    freqs = _on(_cuda(freqs, "freqs", torch.int64), "freqs", dev)
    if freqs.dim() != 1 or 2 * freqs.numel() > D:
        raise ValueError("freqs must be [rotary_dim / 2], rotary_dim <= head_dim")
    page_table = _table(page_table, B, dev)
    ctx_lens = _ints(ctx_lens, "ctx_lens", (B,), dev)
    new_lens = _ints(new_lens, "new_lens", (B,), dev)
    positions = _ints(positions, "positions", (B, T), dev)
    if slot_pos is not None:
        _on(_cuda(slot_pos, "slot_pos", torch.int32), "slot_pos", dev)
        if slot_pos.dim() != 3 or tuple(slot_pos.shape[:2]) != (B, c.kv_heads):
            raise ValueError("slot_pos must be [B, kv_heads, slots]")
    out = dict(out) if out else {}
    _output(out, "q", (B, T, Hq, D), q.dtype, dev)
    if want_status:
        _output(out, "row_status", (B,), torch.int32, dev)
    st = load_library().spv_rope_append(
        _ptr(q), _ptr(k), _ptr(v), _ACTIVATIONS[q.dtype], (ctypes.c_int64 * 6)(*strides), B, T, Hq, _ptr(freqs),
        2 * freqs.numel(), int(bool(interleaved)), float(mscale), _ptr(positions), _ptr(ctx_lens), _ptr(new_lens),
        _ptr(page_table), page_table.shape[1], ctypes.byref(c), _ptr(slot_pos),
        slot_pos.shape[2] if slot_pos is not None else 0, _ptr(out["q"]), _ptr(out.get("row_status")),
        _stream(stream, dev))
    _check(st, "spv_rope_append")
    return out


def spv_attention_workspace_bytes(B: int, T: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    return load_library().spv_attention_workspace_bytes(B, T, q_heads, kv_heads, head_dim)


def spv_paged_attention(q, cache: KVCache, page_table, ctx_lens, *, new_lens=None, parent=None, scale=None,
                        workspace=None, out=None, want_lse: bool = False, want_status: bool = True,
                        stream=None) -> dict:
    """Attention of the new tokens q [B, T, q_heads, D] (rotated, their keys and
    values already in the cache) over the paged cache: a chain, or with
    ``parent`` [B, T] a draft tree (see spv_paged_attention in spv.h).  scale
    defaults to 1 / sqrt(D).  Returns dict(out [B, T, q_heads, D], and lse [B,
    T, q_heads] / row_status when requested)."""
    c, B, T, Hq, dt = _queries(q, cache)
    dev = q.device
    page_table = _table(page_table, B, dev)
    ctx_lens = _ints(ctx_lens, "ctx_lens", (B,), dev)
    new_lens = _ints(new_lens, "new_lens", (B,), dev)
    parent = _ints(parent, "parent", (B, T), dev)
    lib = load_library()
    if workspace is None:
        workspace = new_workspace(lib.spv_attention_workspace_bytes(B, T, Hq, c.kv_heads, c.head_dim), dev)
    _on(_cuda(workspace, "workspace"), "workspace", dev)
    out = dict(out) if out else {}
    _output(out, "out", tuple(q.shape), q.dtype, dev)
    if want_lse:
        _output(out, "lse", (B, T, Hq), torch.float32, dev)
    if want_status:
        _output(out, "row_status", (B,), torch.int32, dev)
    st = lib.spv_paged_attention(
        _ptr(q), dt, B, T, Hq, ctypes.byref(c), _ptr(page_table), page_table.shape[1], _ptr(ctx_lens), _ptr(new_lens),
        _ptr(parent), 1.0 / math.sqrt(c.head_dim) if scale is None else float(scale), _ptr(out["out"]),
        _ptr(out.get("lse")), _ptr(out.get("row_status")), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream, dev))
    _check(st, "spv_paged_attention")
    return out


def spv_attention_mass(q, lse, cache: KVCache, page_table, ctx_lens, accept_count, *, nodes=None, new_lens=None,
                       parent=None, scale=None, decay: float = 1.0, mass_in=None, out=None,
                       want_status: bool = True, stream=None) -> dict:
    """What each cached key received from the tokens that stand after the
    verify step (see spv_attention_mass in spv.h): out["mass"] [B, kv_heads,
    slots] float32 = decay * mass_in + the sum of the weights.  q, lse and the
    other arguments as in the :func:`spv_paged_attention` call; accept_count
    (and, for a tree, nodes: out_nodes) from the verify call.  Without
    ``mass_in`` and ``out`` a zero-filled mass as wide as the page table is
    made."""
    c, B, T, Hq, dt = _queries(q, cache)
    dev = q.device
    lse = _floats(lse, "lse", (B, T, Hq), dev)
    page_table = _table(page_table, B, dev)
    ctx_lens = _ints(ctx_lens, "ctx_lens", (B,), dev)
    accept_count = _ints(accept_count, "accept_count", (B,), dev)
    nodes = _ints(nodes, "nodes", (B, T), dev)
    new_lens = _ints(new_lens, "new_lens", (B,), dev)
    parent = _ints(parent, "parent", (B, T), dev)
    out = dict(out) if out else {}
    mass = out.get("mass")
    if mass is None:
        slots = mass_in.shape[2] if mass_in is not None else page_table.shape[1] * c.page_size
        mass = out["mass"] = torch.zeros(B, c.kv_heads, slots, dtype=torch.float32, device=dev)
    if mass.dim() != 3:
        raise ValueError("out['mass'] must be [B, kv_heads, slots]")
    slots = mass.shape[2]
    _floats(mass, "out['mass']", (B, c.kv_heads, slots), dev)
    mass_in = _floats(mass_in, "mass_in", (B, c.kv_heads, slots), dev)
    if want_status:
        _output(out, "row_status", (B,), torch.int32, dev)
    st = load_library().spv_attention_mass(
        _ptr(q), dt, B, T, Hq, _ptr(lse), ctypes.byref(c), _ptr(page_table), page_table.shape[1], _ptr(ctx_lens),
        _ptr(new_lens), _ptr(parent), 1.0 / math.sqrt(c.head_dim) if scale is None else float(scale),
        _ptr(accept_count), _ptr(nodes), float(decay), _ptr(mass_in), _ptr(mass), slots, _ptr(out.get("row_status")),
        _stream(stream, dev))
    _check(st, "spv_attention_mass")
    return out


def spv_kv_evict(cache: KVCache, page_table, lens, mass, budget: int, *, pos=None, sinks: int = 0, recent: int = 0,
                 out=None, want_status: bool = True, stream=None) -> dict:
    """Cuts every sequence of more than ``budget`` slots back to it, in place
    and per key head, by the accumulated weight ``mass`` [B, kv_heads, slots]
    (see spv_kv_evict in spv.h).  Returns dict(mass, pos [B, kv_heads, >=
    budget], lens [B], slot_src [B, kv_heads, budget], and row_status when
    requested); pass ``mass`` and ``pos`` themselves in ``out`` to update them
    in place."""
    c = cache.struct()
    dev = cache.k.device
    mass = _on(_cuda(mass, "mass", torch.float32), "mass", dev)
    if mass.dim() != 3 or mass.shape[1] != c.kv_heads:
        raise ValueError("mass must be [B, kv_heads, slots]")
    B, Hkv, slots = mass.shape
    page_table = _table(page_table, B, dev)
    lens = _ints(lens, "lens", (B,), dev)
    pos = _ints(pos, "pos", tuple(mass.shape), dev)
    budget = int(budget)
    out = dict(out) if out else {}
    width = max(out["mass"].shape[-1] if out.get("mass") is not None else min(budget, slots), 0)
    _output(out, "mass", (B, Hkv, width), torch.float32, dev)
    _output(out, "pos", (B, Hkv, width), torch.int32, dev)
    _output(out, "lens", (B,), torch.int32, dev)
    _output(out, "slot_src", (B, Hkv, max(budget, 0)), torch.int32, dev)
    if want_status:
        _output(out, "row_status", (B,), torch.int32, dev)
    st = load_library().spv_kv_evict(
        ctypes.byref(c), _ptr(page_table), page_table.shape[1], B, _ptr(lens), budget, int(sinks), int(recent),
        _ptr(mass), _ptr(pos), slots, _ptr(out["mass"]), _ptr(out["pos"]), width, _ptr(out["lens"]),
        _ptr(out["slot_src"]), _ptr(out.get("row_status")), _stream(stream, dev))
    _check(st, "spv_kv_evict")
    return out
