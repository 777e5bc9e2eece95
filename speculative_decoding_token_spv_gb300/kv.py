"""The target model's attention layer around a verify step: binding of
spv_rope_append, spv_paged_attention, spv_attention_mass and spv_kv_evict.

Like the verify calls: torch CUDA tensors in, work on torch's current stream
(or ``stream``), outputs allocated when the caller passes none in ``out``, no
CPU fallback.  What a call with ``stream`` allocates belongs to that stream, as
under ``torch.cuda.stream(stream)``; tensors that come from another one are in
order only if the caller has made them so.  A cache is two 4-D pools [pages, page_size, kv_heads, head_dim];
any strides will do as long as a row's elements are contiguous, so
``pool.transpose(1, 2)`` of a [pages, kv_heads, page_size, head_dim] tensor or
a slice of a joint K/V tensor can be passed.
"""
from __future__ import annotations

import ctypes
import math
import struct
from dataclasses import dataclass

import torch

from . import SPV_BF16, SPV_E4M3, SPV_F16, SpvError, _check, _stream, load_library, new_workspace

ROPE_SCALINGS = {"plain": 0, "linear": 1, "base": 2, "by_parts": 3}
_ACTIVATIONS = {torch.bfloat16: SPV_BF16, torch.float16: SPV_F16}
_CACHES = {**_ACTIVATIONS, torch.float8_e4m3fn: SPV_E4M3}
_F32, _I32, _I64, _U8 = torch.float32, torch.int32, torch.int64, torch.uint8


class _CacheStruct(ctypes.Structure):
    """spv_kv_cache of spv.h."""
    _fields_ = ([("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int)]
                + [(n, ctypes.c_int32) for n in ("num_pages", "page_size", "kv_heads", "head_dim")]
                + [(f"{p}_{n}_stride", ctypes.c_int64) for p in "kv" for n in ("page", "slot", "head")]
                + [("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)])


# These calls take a few microseconds on the GPU, so the checks below are written to cost little: the struct is packed
# as bytes (the layout of _CacheStruct), and a tensor's properties are compared at once and looked at one by one only
# to say what is wrong.
_PACK = struct.Struct("@PPiiiii4xqqqqqqPP").pack
_PACK_STRIDES = struct.Struct("@6q").pack


@dataclass
class KVCache:
    """A paged cache: pools k, v [pages, page_size, kv_heads, head_dim] of one
    dtype (bfloat16, float16 or float8_e4m3fn) and, for float8, what an element
    stands for: [kv_heads] float32 scales (None: 1)."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor | None = None
    v_scale: torch.Tensor | None = None

    def packed(self):
        """(spv_kv_cache as bytes, device, its shape [pages, page_size, kv_heads, head_dim])."""
        k, v = self.k, self.v
        try:
            shape, dtype, dev = k.shape, k.dtype, k.device
            ks, vs = k.stride(), v.stride()
            if not k.is_cuda or len(shape) != 4 or dtype not in _CACHES or v.shape != shape or v.dtype != dtype \
                    or v.device != dev or (shape[3] > 1 and (ks[3] != 1 or vs[3] != 1)):
                self._complain()
        except AttributeError:
            raise ValueError("cache.k and cache.v must be CUDA tensors") from None
        heads = (shape[2],)
        sk = 0 if self.k_scale is None else _arg(self.k_scale, "k_scale", _F32, heads, dev)
        sv = 0 if self.v_scale is None else _arg(self.v_scale, "v_scale", _F32, heads, dev)
        if 1 in shape:  # a dimension of one entry may carry any stride: it is never stepped over
            ks = [x if n > 1 else 0 for x, n in zip(ks, shape)]
            vs = [x if n > 1 else 0 for x, n in zip(vs, shape)]
        try:
            return (_PACK(k.data_ptr(), v.data_ptr(), _CACHES[dtype], *shape, ks[0], ks[1], ks[2], vs[0], vs[1], vs[2],
                          sk, sv), dev, shape)
        except struct.error:
            raise ValueError("the cache's sizes do not fit 32 bits") from None

    def _complain(self):
        k, v = self.k, self.v
        for name, t in (("cache.k", k), ("cache.v", v)):
            if not t.is_cuda:
                raise ValueError(f"{name} must be a CUDA tensor")
            if t.dim() != 4 or (t.shape[3] > 1 and t.stride(3) != 1):
                raise ValueError(f"{name} must be [pages, page_size, kv_heads, head_dim] with contiguous rows")
            if t.dtype not in _CACHES:
                raise TypeError(f"{name} must be bfloat16, float16 or float8_e4m3fn, got {t.dtype}")
        raise ValueError("cache.k and cache.v must have the same shape, dtype and device")


def _arg(t, name, dtype, shape, dev):
    """Address of a contiguous tensor of this dtype, shape and device."""
    try:
        if t.dtype is dtype and t.shape == shape and t.device == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _opt(t, name, dtype, shape, dev):
    return None if t is None else _arg(t, name, dtype, shape, dev)


def _made(stream, make, *args, **kw):
    """make(...) with the call's stream as torch's current one: what is made belongs to it, in order with its kernels."""
    if stream is None:
        return make(*args, **kw)
    with torch.cuda.stream(stream):
        return make(*args, **kw)


def _output(out, key, shape, dtype, dev, stream):
    """Address of the caller's output tensor `key`, checked, or of a new one."""
    t = out.get(key)
    if t is None:
        t = out[key] = _made(stream, torch.empty, shape, dtype=dtype, device=dev)
        return t.data_ptr()
    return _arg(t, key, dtype, shape, dev)


def _table(page_table, B, dev):
    try:
        shape = page_table.shape
    except AttributeError:
        raise ValueError("page_table must be a CUDA tensor") from None
    if len(shape) != 2 or shape[0] != B:
        raise ValueError("page_table must be [B, max_pages]")
    return _arg(page_table, "page_table", _I32, shape, dev), shape[1]


def _queries(q, head_dim, dev):
    """q [B, T, q_heads, head_dim]: its sizes, dtype code and address."""
    try:
        shape, code = q.shape, _ACTIVATIONS.get(q.dtype)
    except AttributeError:
        raise ValueError("q must be a CUDA tensor") from None
    if len(shape) != 4 or shape[3] != head_dim:
        raise ValueError("q must be [B, T, q_heads, head_dim]")
    if code is None:
        raise TypeError(f"q must be bfloat16 or float16, got {q.dtype}")
    return shape, code, _arg(q, "q", q.dtype, shape, dev)


def _complain_qkv(tensors, shape, kv_shape, dtype, dev):
    for name, t, want in zip("qkv", tensors, (shape, kv_shape, kv_shape)):
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.shape != want:
            raise ValueError(f"{name} must be {list(want)}, got {list(t.shape)}")
        if t.device != dev:
            raise ValueError(f"{name} must be on {dev}, got {t.device}")
        if t.stride(3) != 1 or (want[2] > 1 and t.stride(2) != want[3]):
            raise ValueError(f"{name}: the heads of a token must be contiguous")


_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _on_stream(stream, dev):
    """The stream's handle: torch's current one unless the caller names another."""
    if stream is None and _current_raw_stream is not None and dev.index is not None:
        return _current_raw_stream(dev.index)
    return _stream(stream, dev)


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
    pack, dev, (_, _, Hkv, D) = cache.packed()
    try:
        shape, dtype = q.shape, q.dtype
        code = _ACTIVATIONS.get(dtype)
        if len(shape) != 4 or shape[3] != D:
            raise ValueError("q must be [B, T, q_heads, head_dim]")
        if code is None:
            raise TypeError(f"q must be bfloat16 or float16, got {dtype}")
        B, T, Hq, _ = shape
        kv_shape = (B, T, Hkv, D)
        sq, sk, sv = q.stride(), k.stride(), v.stride()
        if k.shape != kv_shape or v.shape != kv_shape or k.dtype is not dtype or v.dtype is not dtype or q.device != dev \
                or k.device != dev or v.device != dev or sq[3] != 1 or sk[3] != 1 or sv[3] != 1 \
                or (Hq > 1 and sq[2] != D) or (Hkv > 1 and (sk[2] != D or sv[2] != D)):
            _complain_qkv((q, k, v), shape, kv_shape, dtype, dev)
        pairs = freqs.shape[0] if freqs.dim() == 1 else D
    except AttributeError:
        raise ValueError("q, k, v and freqs must be CUDA tensors") from None
    if B == 1 or T == 1:
        # a dimension of one entry may carry any stride: its packed one, so that q can be its own output
        sq, sk, sv = (((T * (s[1] if T > 1 else h * D) if B == 1 else s[0]), s[1] if T > 1 else h * D)
                      for s, h in ((sq, Hq), (sk, Hkv), (sv, Hkv)))
    if 2 * pairs > D:
        raise ValueError("freqs must be [rotary_dim / 2], rotary_dim <= head_dim")
    table, pages = _table(page_table, B, dev)
    slots = 0
    if slot_pos is not None:
        if slot_pos.dim() != 3:
            raise ValueError("slot_pos must be [B, kv_heads, slots]")
        slots = slot_pos.shape[2]
    out = dict(out) if out else {}
    st = load_library().spv_rope_append(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), code, _PACK_STRIDES(sq[0], sq[1], sk[0], sk[1], sv[0], sv[1]), B, T, Hq,
        _arg(freqs, "freqs", _I64, (pairs,), dev), 2 * pairs, int(bool(interleaved)), mscale,
        _opt(positions, "positions", _I32, (B, T), dev),
        _arg(ctx_lens, "ctx_lens", _I32, (B,), dev), _opt(new_lens, "new_lens", _I32, (B,), dev), table, pages, pack,
        _opt(slot_pos, "slot_pos", _I32, (B, Hkv, slots), dev), slots, _output(out, "q", (B, T, Hq, D), dtype, dev, stream),
        _output(out, "row_status", (B,), _I32, dev, stream) if want_status else None, _on_stream(stream, dev))
    if st:
        raise SpvError(st, "spv_rope_append")
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
    pack, dev, (_, _, Hkv, D) = cache.packed()
    shape, code, address = _queries(q, D, dev)
    B, T, Hq, _ = shape
    table, pages = _table(page_table, B, dev)
    lib = load_library()
    if workspace is None:
        workspace = _made(stream, new_workspace, lib.spv_attention_workspace_bytes(B, T, Hq, Hkv, D), dev)
    out = dict(out) if out else {}
    st = lib.spv_paged_attention(
        address, code, B, T, Hq, pack, table, pages, _arg(ctx_lens, "ctx_lens", _I32, (B,), dev),
        _opt(new_lens, "new_lens", _I32, (B,), dev), _opt(parent, "parent", _I32, (B, T), dev),
        1.0 / math.sqrt(D) if scale is None else scale, _output(out, "out", shape, q.dtype, dev, stream),
        _output(out, "lse", (B, T, Hq), _F32, dev, stream) if want_lse else None,
        _output(out, "row_status", (B,), _I32, dev, stream) if want_status else None,
        _arg(workspace, "workspace", _U8, (workspace.numel(),), dev), workspace.numel(), _on_stream(stream, dev))
    if st:
        raise SpvError(st, "spv_paged_attention")
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
    pack, dev, (_, page_size, Hkv, D) = cache.packed()
    shape, code, address = _queries(q, D, dev)
    B, T, Hq, _ = shape
    table, pages = _table(page_table, B, dev)
    out = dict(out) if out else {}
    mass = out.get("mass")
    if mass is None:
        slots = mass_in.shape[2] if mass_in is not None and mass_in.dim() == 3 else pages * page_size
        mass = out["mass"] = _made(stream, torch.zeros, B, Hkv, slots, dtype=_F32, device=dev)
    if mass.dim() != 3:
        raise ValueError("out['mass'] must be [B, kv_heads, slots]")
    full = (B, Hkv, mass.shape[2])
    st = load_library().spv_attention_mass(
        address, code, B, T, Hq, _arg(lse, "lse", _F32, (B, T, Hq), dev), pack, table, pages,
        _arg(ctx_lens, "ctx_lens", _I32, (B,), dev), _opt(new_lens, "new_lens", _I32, (B,), dev),
        _opt(parent, "parent", _I32, (B, T), dev), 1.0 / math.sqrt(D) if scale is None else scale,
        _arg(accept_count, "accept_count", _I32, (B,), dev), _opt(nodes, "nodes", _I32, (B, T), dev), decay,
        _opt(mass_in, "mass_in", _F32, full, dev), _arg(mass, "out['mass']", _F32, full, dev), full[2],
        _output(out, "row_status", (B,), _I32, dev, stream) if want_status else None, _on_stream(stream, dev))
    if st:
        raise SpvError(st, "spv_attention_mass")
    return out


def spv_kv_evict(cache: KVCache, page_table, lens, mass, budget: int, *, pos=None, sinks: int = 0, recent: int = 0,
                 out=None, want_status: bool = True, stream=None) -> dict:
    """Cuts every sequence of more than ``budget`` slots back to it, in place
    and per key head, by the accumulated weight ``mass`` [B, kv_heads, slots]
    (see spv_kv_evict in spv.h).  Returns dict(mass, pos [B, kv_heads, >=
    budget], lens [B], slot_src [B, kv_heads, budget], and row_status when
    requested); pass ``mass``, ``pos`` and ``lens`` themselves in ``out`` to
    update them in place."""
    pack, dev, (_, _, Hkv, _) = cache.packed()
    try:
        full = mass.shape
    except AttributeError:
        raise ValueError("mass must be a CUDA tensor") from None
    if len(full) != 3 or full[1] != Hkv:
        raise ValueError("mass must be [B, kv_heads, slots]")
    B, _, slots = full
    table, pages = _table(page_table, B, dev)
    budget = int(budget)
    out = dict(out) if out else {}
    kept = out.get("mass")
    width = kept.shape[-1] if kept is not None else max(min(budget, slots), 0)
    st = load_library().spv_kv_evict(
        pack, table, pages, B, _arg(lens, "lens", _I32, (B,), dev), budget, int(sinks), int(recent),
        _arg(mass, "mass", _F32, full, dev), _opt(pos, "pos", _I32, full, dev), slots,
        _output(out, "mass", (B, Hkv, width), _F32, dev, stream), _output(out, "pos", (B, Hkv, width), _I32, dev, stream), width,
        _output(out, "lens", (B,), _I32, dev, stream), _output(out, "slot_src", (B, Hkv, max(budget, 0)), _I32, dev, stream),
        _output(out, "row_status", (B,), _I32, dev, stream) if want_status else None, _on_stream(stream, dev))
    if st:
        raise SpvError(st, "spv_kv_evict")
    return out
