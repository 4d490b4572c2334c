"""Attention between two linears: the binding of the head norm, cache and attention calls.

A transformer layer whose projections are svdq_linear calls runs

    qkv = svdq_linear(w_qkv, x)                            # rows q | k | v
    q, k, v = qkv.view(T, -1, D).split([H, Hkv, Hkv], 1)   # strided views, no copy

and then, for image tokens or a prompt without a cache,

    svdq_qk_norm_rope(q, k, positions, rope, q_weight, k_weight, q_out=q, k_out=k)
    o = svdq_attention_prompt(q, k, v, cu_q, cu_k, causal=True)

or, for a decode step over a paged cache,

    q = svdq_kv_append(k_cache, v_cache, k, v, slots, positions, rope, k_weight, q=q, q_weight=q_weight)
    o = svdq_attention_decode(q, k_cache, v_cache, page_table, kv_len)

before svdq_linear(w_out, o.view(T, -1)). AttentionStep holds such a sequence as one
step of svdq_linear_chain.

Heads are tensors [tokens, heads, head_dim] with unit stride along head_dim. Inputs in
another layout are copied; outputs and caches in another layout are refused. Calls run on
the current stream of the tensors' device and raise ValueError for wrong arguments.
Mistakes that only the device sees (a slot or page outside the cache, lengths beyond
the page table) are recorded in the status word (svdq_check_status).
"""

from __future__ import annotations

import contextlib
import ctypes
import math
from dataclasses import dataclass
from typing import Optional, Tuple

import torch

from . import (LinearWorkspace, SvdqHeads, SvdqKvCache, SvdqRope, _check, _dt, _ptr, _require_cuda, c_sz,
               load_library)


@dataclass
class Rope:
    """Rotary positions: pair j of a head turns by 2 pi * position * turns[j].

    turns        fp64 [rot_dim / 2] on the GPU, in turns per position
    interleaved  pairs (2j, 2j + 1) instead of (j, j + rot_dim / 2)
    amplitude    multiplies cosine and sine (the attention factor of a scaled context)
    """
    turns: torch.Tensor
    interleaved: bool = False
    amplitude: float = 1.0

    @property
    def rot_dim(self) -> int:
        return 2 * self.turns.numel()

    @classmethod
    def make(cls, rot_dim: int, base: float = 10000.0, interleaved: bool = False, factor: float = 1.0,
             trained_len: Optional[int] = None, fast: float = 32.0, slow: float = 1.0, device="cuda") -> "Rope":
        """base^(-2j / rot_dim) / (2 pi) turns per position, scaled for contexts `factor`
        times as long: every pair by 1 / factor (position interpolation), or, with
        trained_len, only the pairs that turn less than `slow` times over the trained
        length, those that turn more than `fast` times not at all, with a linear ramp
        between and the amplitude 1 + 0.1 ln(factor) ("YaRN: Efficient Context Window
        Extension of Large Language Models", NTK-by-parts)."""
        if isinstance(rot_dim, bool) or not isinstance(rot_dim, int) or rot_dim < 2 or rot_dim % 2:
            raise ValueError("rot_dim must be a positive even int")
        if not (base > 0 and factor >= 1 and fast > slow >= 0):
            raise ValueError("base must be positive, factor >= 1 and fast > slow >= 0")
        j = torch.arange(0, rot_dim, 2, dtype=torch.float64)
        turns = base ** (-j / rot_dim) / (2 * math.pi)
        amplitude = 1.0
        if trained_len is None:
            turns = turns / factor
        else:
            keep = ((turns * trained_len - slow) / (fast - slow)).clamp(0, 1)
            turns = turns * (keep + (1 - keep) / factor)
            amplitude = 1.0 + 0.1 * math.log(factor)
        return cls(turns.to(device), interleaved, amplitude)


_NO_HEADS = SvdqHeads(None, 0, 0, 0)


def _on(device):
    """Work on the tensors' device, whatever the current one is."""
    if device.index is None or device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def _same_device(first, **others):
    _require_cuda(first, *others.values())
    for name, t in others.items():
        if t is not None and t.device != first.device:
            raise ValueError(f"{name} lives on another device")
    return first.device


def _strides(t: torch.Tensor):
    """Strides of all axes but the last; those of axes of one element (which torch leaves
    free) as a dense tensor has them."""
    s = [t.stride(i) for i in range(t.dim() - 1)]
    dense = -(-t.shape[-1] // 8) * 8
    for i in range(t.dim() - 2, -1, -1):
        if t.shape[i] <= 1:
            s[i] = dense
        dense = max(dense, s[i] * t.shape[i])
    return s


def _usable(t: torch.Tensor) -> bool:
    es = t.element_size()
    return (t.stride(-1) == 1 or t.shape[-1] == 1) and t.data_ptr() % 16 == 0 and \
        all(s * es % 16 == 0 and s >= t.shape[-1] for s in _strides(t))


def _check_3d(t, name, dtype, shape=None):
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim]")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, not {tuple(t.shape)}")


def _heads(t: torch.Tensor):
    """(descriptor, the tensor it points to) of an input; a copy where the layout needs one."""
    if not _usable(t):
        t = t.contiguous() if t.data_ptr() % 16 == 0 or not t.is_contiguous() else t.clone()
    s = _strides(t)
    return SvdqHeads(t.data_ptr(), s[0], s[1], t.shape[1]), t


def _out_heads(t: torch.Tensor, name: str):
    if not _usable(t):
        raise ValueError(f"{name} needs unit stride along head_dim, 16-byte aligned rows and no broadcast axis")
    s = _strides(t)
    return SvdqHeads(t.data_ptr(), s[0], s[1], t.shape[1])


def _vector(t, name, dtype, n):
    if t is None:
        return None
    if t.dtype != dtype or t.dim() != 1 or t.shape[0] != n:
        raise ValueError(f"{name} must be {dtype} [{n}]")
    return t.contiguous()


def _weights(q_weight, k_weight, dim):
    given = [w for w in (q_weight, k_weight) if w is not None]
    for w in given:
        if tuple(w.shape) != (dim,):
            raise ValueError(f"a norm weight must be [{dim}]")
    if len({w.dtype for w in given}) > 1:
        raise ValueError("the norm weights must have one type")
    dt = _dt(given[0]) if given else _dt(torch.empty(0, dtype=torch.bfloat16))

    def ready(w):
        if w is None:
            return None
        w = w.contiguous()
        return w if w.data_ptr() % 16 == 0 else w.clone()
    return ready(q_weight), ready(k_weight), dt


def _rope(rope: Optional[Rope], positions, tokens: int, dim: int):
    """(descriptor, positions, tensors to keep until the launch)."""
    if rope is None or rope.turns.numel() == 0:
        return SvdqRope(None, 0, 0, 1.0), None, None
    if positions is None:
        raise ValueError("a rotation needs positions")
    positions = _vector(positions, "positions", torch.int64, tokens)
    if rope.turns.dtype != torch.float64 or rope.turns.dim() != 1:
        raise ValueError("turns must be float64 [rot_dim / 2]")
    if rope.rot_dim > dim:
        raise ValueError("rot_dim must not exceed head_dim")
    turns = rope.turns.contiguous()
    return SvdqRope(turns.data_ptr(), 2 * turns.numel(), int(bool(rope.interleaved)), float(rope.amplitude)), \
        positions, turns


def _cache(k_cache, v_cache):
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if t.dim() != 4 or t.dtype != torch.bfloat16:
            raise ValueError(f"{name} must be bfloat16 [pages, page_size, heads, head_dim]")
    if k_cache.shape != v_cache.shape or _strides(k_cache) != _strides(v_cache):
        raise ValueError("k_cache and v_cache must have one shape and layout")
    if not _usable(k_cache) or not _usable(v_cache):
        raise ValueError("a cache needs unit stride along head_dim and 16-byte aligned rows")
    if k_cache.numel() == 0:
        raise ValueError("the cache is empty")
    pages, page_size, heads, dim = k_cache.shape
    page_ld, slot_ld, head_ld = _strides(k_cache)
    return SvdqKvCache(k_cache.data_ptr(), v_cache.data_ptr(), pages, page_ld, slot_ld, head_ld, page_size, heads, dim)


def _stream_of(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def svdq_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: Optional[torch.Tensor] = None,
                      rope: Optional[Rope] = None, q_weight: Optional[torch.Tensor] = None,
                      k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                      q_out: Optional[torch.Tensor] = None,
                      k_out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """RMS norm (with a weight) and rotation (with a rope) of query and key heads, one pass.

    q [T, H, D], k [T, Hkv, D], bf16 or fp32; positions int64 [T]; weights [D] bf16 or
    fp32. q_out=q, k_out=k work in place. Returns (q_out, k_out).
    """
    lib = load_library()
    dev = _same_device(q, k=k, positions=positions, q_weight=q_weight, k_weight=k_weight, q_out=q_out, k_out=k_out,
                       turns=rope.turns if rope is not None else None)
    _check_3d(q, "q", q.dtype)
    _check_3d(k, "k", q.dtype, (q.shape[0], k.shape[1] if k.dim() == 3 else 0, q.shape[2]))
    dt = _dt(q)
    T, _, D = q.shape
    if q_out is not None:
        _check_3d(q_out, "q_out", q.dtype, q.shape)
    if k_out is not None:
        _check_3d(k_out, "k_out", q.dtype, k.shape)
    with _on(dev):
        qw, kw, wdt = _weights(q_weight, k_weight, D)
        r, pos, _turns = _rope(rope, positions, T, D)
        q_out = torch.empty(q.shape, dtype=q.dtype, device=dev) if q_out is None else q_out
        k_out = torch.empty(k.shape, dtype=k.dtype, device=dev) if k_out is None else k_out
        if T == 0:
            return q_out, k_out
        qd, q = _heads(q) if q.shape[1] else (_NO_HEADS, q)
        kd, k = _heads(k) if k.shape[1] else (_NO_HEADS, k)
        qo = _out_heads(q_out, "q_out") if q.shape[1] else _NO_HEADS
        ko = _out_heads(k_out, "k_out") if k.shape[1] else _NO_HEADS
        _check(lib.svdq_qk_norm_rope(qd, kd, dt, T, D, _ptr(pos), r, _ptr(qw), _ptr(kw), wdt, float(eps), qo, ko,
                                     _stream_of(dev)), "svdq_qk_norm_rope")
    return q_out, k_out


def svdq_kv_append(k_cache: torch.Tensor, v_cache: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                   slots: torch.Tensor, positions: Optional[torch.Tensor] = None, rope: Optional[Rope] = None,
                   k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, q: Optional[torch.Tensor] = None,
                   q_weight: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                   k_out: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """Append keys (normed and rotated as in svdq_qk_norm_rope) and values to a paged cache.

    Caches [pages, page_size, Hkv, D] bf16 (any order of the outer axes in memory); k, v
    [T, Hkv, D]; slots int64 [T]: page * page_size + row, negative for padding, no slot
    twice. q [T, H, D] is normed and rotated in the same pass. k_out receives the
    finished keys too (k_out=k: in place). Returns q_out (None without q).
    """
    lib = load_library()
    dev = _same_device(k_cache, v_cache=v_cache, k=k, v=v, slots=slots, positions=positions, k_weight=k_weight, q=q,
                       q_weight=q_weight, q_out=q_out, k_out=k_out, turns=rope.turns if rope is not None else None)
    c = _cache(k_cache, v_cache)
    bf16 = torch.bfloat16
    _check_3d(k, "k", bf16, (k.shape[0], c.heads, c.head_dim))
    _check_3d(v, "v", bf16, k.shape)
    T, D = k.shape[0], c.head_dim
    if q is not None:
        _check_3d(q, "q", bf16, (T, q.shape[1] if q.dim() == 3 else 0, D))
        if q.shape[1] == 0:
            raise ValueError("q has no heads")
        if q_out is not None:
            _check_3d(q_out, "q_out", bf16, q.shape)
    elif q_out is not None or q_weight is not None:
        raise ValueError("q_out and q_weight need q")
    if k_out is not None:
        _check_3d(k_out, "k_out", bf16, k.shape)
    with _on(dev):
        qw, kw, wdt = _weights(q_weight, k_weight, D)
        r, pos, _turns = _rope(rope, positions, T, D)
        slots = _vector(slots, "slots", torch.int64, T)
        if q is not None and q_out is None:
            q_out = torch.empty(q.shape, dtype=bf16, device=dev)
        if T == 0:
            return q_out
        kd, k = _heads(k)
        vd, v = _heads(v)
        qd, q = _heads(q) if q is not None else (_NO_HEADS, None)
        qo = _out_heads(q_out, "q_out") if q is not None else _NO_HEADS
        ko = _out_heads(k_out, "k_out") if k_out is not None else _NO_HEADS
        _check(lib.svdq_kv_append(ctypes.byref(c), kd, vd, _ptr(slots), T, _ptr(pos), r, _ptr(kw), wdt, float(eps),
                                  qd, _ptr(qw), qo, ko, _stream_of(dev)), "svdq_kv_append")
    return q_out


def _scale(scale: Optional[float], dim: int) -> float:
    return 1.0 / math.sqrt(dim) if scale is None else float(scale)


def svdq_attention_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: Optional[torch.Tensor] = None,
                          cu_k: Optional[torch.Tensor] = None, causal: bool = True,
                          scale: Optional[float] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention over packed sequences: q [Tq, H, D], k and v [Tk, Hkv, D], bf16.

    cu_q, cu_k int32 [batch + 1]: sequence s owns rows cu[s] .. cu[s + 1] - 1 (None: one
    sequence of all rows). causal: rows and keys of a sequence end together, and a row
    sees no key behind its own place; a row that sees none becomes zero. Rows of no
    sequence are left as they were in `out`, and mean nothing in an output allocated here.
    Returns [Tq, H, D].
    """
    lib = load_library()
    dev = _same_device(q, k=k, v=v, cu_q=cu_q, cu_k=cu_k, out=out)
    bf16 = torch.bfloat16
    _check_3d(q, "q", bf16)
    T, H, D = q.shape
    _check_3d(k, "k", bf16, (k.shape[0], k.shape[1] if k.dim() == 3 else 0, D))
    _check_3d(v, "v", bf16, k.shape)
    if H == 0 or k.shape[1] == 0 or H % k.shape[1]:
        raise ValueError("the query heads must be a multiple of the key heads")
    for name, cu in (("cu_q", cu_q), ("cu_k", cu_k)):
        if cu is not None and (cu.dtype != torch.int32 or cu.dim() != 1 or cu.shape[0] < 1):
            raise ValueError(f"{name} must be int32 [batch + 1]")
    sizes = [cu.shape[0] - 1 if cu is not None else 1 for cu in (cu_q, cu_k)]
    if sizes[0] != sizes[1]:
        raise ValueError("cu_q and cu_k must have one length")
    if out is not None:
        _check_3d(out, "out", bf16, q.shape)
    with _on(dev):
        out = torch.empty(q.shape, dtype=bf16, device=dev) if out is None else out
        if T == 0:
            return out
        qd, q = _heads(q)
        kd, k = _heads(k)
        vd, v = _heads(v)
        cu_q = cu_q.contiguous() if cu_q is not None else None
        cu_k = cu_k.contiguous() if cu_k is not None else None
        _check(lib.svdq_attention_prompt(qd, kd, vd, _ptr(cu_q), _ptr(cu_k), sizes[0], T, k.shape[0], D,
                                         int(bool(causal)), _scale(scale, D), _out_heads(out, "out"), _stream_of(dev)),
               "svdq_attention_prompt")
    return out


def svdq_attention_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                          kv_len: torch.Tensor, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                          workspace: Optional[LinearWorkspace] = None) -> torch.Tensor:
    """Attention of one token per sequence over a paged cache: q [B, H, D] bf16.

    Caches as in svdq_kv_append; page_table int32 [B, pages per sequence], kv_len int32
    [B] (0: a zero row). The scratch is allocated per call unless a workspace is given
    (one per stream in flight). Returns [B, H, D].
    """
    lib = load_library()
    dev = _same_device(q, k_cache=k_cache, v_cache=v_cache, page_table=page_table, kv_len=kv_len, out=out)
    bf16 = torch.bfloat16
    c = _cache(k_cache, v_cache)
    _check_3d(q, "q", bf16, (q.shape[0], q.shape[1] if q.dim() == 3 else 0, c.head_dim))
    B, H, D = q.shape
    if H == 0 or H % c.heads:
        raise ValueError("the query heads must be a multiple of the key heads")
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError(f"page_table must be int32 [{B}, pages]")
    kv_len = _vector(kv_len, "kv_len", torch.int32, B)
    if out is not None:
        _check_3d(out, "out", bf16, q.shape)
    with _on(dev):
        out = torch.empty(q.shape, dtype=bf16, device=dev) if out is None else out
        if B == 0:
            return out
        page_table = page_table.contiguous()
        size = c_sz()
        _check(lib.svdq_attention_decode_workspace_size(B, H, c.heads, D, ctypes.byref(size)), "workspace")
        ws = workspace.get(size.value, dev) if workspace is not None else \
            torch.empty(size.value, dtype=torch.uint8, device=dev)
        qd, q = _heads(q)
        _check(lib.svdq_attention_decode(qd, ctypes.byref(c), _ptr(page_table), page_table.shape[1], _ptr(kv_len), B,
                                         _scale(scale, D), _out_heads(out, "out"), _ptr(ws), ws.numel(),
                                         _stream_of(dev)), "svdq_attention_decode")
    return out


@dataclass
class AttentionStep:
    """What lies between the qkv and the output projection, as a step of svdq_linear_chain.

    Called with the projection's rows q | k | v, bf16 [T, (heads + 2 kv_heads) * head_dim],
    it returns [T, heads * head_dim]. The queries and keys are normed and rotated in place,
    in those rows.

    Without a cache, or with k_cache, v_cache and slots: attention over packed prompts
    (cu_seqlens as in svdq_attention_prompt, None: one sequence; rows behind the last
    sequence come out zero), the finished keys and the values being appended to the cache
    if there is one. With page_table and kv_len
    too: one token per sequence, attention over the cache after appending (kv_len counts
    the new token).
    """
    heads: int
    kv_heads: int
    head_dim: int
    positions: Optional[torch.Tensor] = None
    rope: Optional[Rope] = None
    q_weight: Optional[torch.Tensor] = None
    k_weight: Optional[torch.Tensor] = None
    eps: float = 1e-6
    scale: Optional[float] = None
    cu_seqlens: Optional[torch.Tensor] = None
    causal: bool = True
    k_cache: Optional[torch.Tensor] = None
    v_cache: Optional[torch.Tensor] = None
    slots: Optional[torch.Tensor] = None
    page_table: Optional[torch.Tensor] = None
    kv_len: Optional[torch.Tensor] = None
    workspace: Optional[LinearWorkspace] = None

    def __call__(self, qkv: torch.Tensor) -> torch.Tensor:
        H, Hkv, D = self.heads, self.kv_heads, self.head_dim
        if qkv.dim() != 2 or qkv.shape[1] != (H + 2 * Hkv) * D:
            raise ValueError(f"the projection's rows must be [tokens, {(H + 2 * Hkv) * D}]")
        cached = self.k_cache is not None
        if cached != (self.v_cache is not None) or cached != (self.slots is not None):
            raise ValueError("k_cache, v_cache and slots belong together")
        decode = self.page_table is not None
        if decode != (self.kv_len is not None) or (decode and not cached):
            raise ValueError("page_table and kv_len belong together, with a cache")
        T = qkv.shape[0]
        q, k, v = qkv.view(T, H + 2 * Hkv, D).split([H, Hkv, Hkv], 1)
        if cached:
            svdq_kv_append(self.k_cache, self.v_cache, k, v, self.slots, self.positions, self.rope, self.k_weight,
                           self.eps, q=q, q_weight=self.q_weight, q_out=q, k_out=None if decode else k)
        elif self.rope is not None or self.q_weight is not None or self.k_weight is not None:
            svdq_qk_norm_rope(q, k, self.positions, self.rope, self.q_weight, self.k_weight, self.eps, q_out=q, k_out=k)
        if decode:
            o = svdq_attention_decode(q, self.k_cache, self.v_cache, self.page_table, self.kv_len, self.scale,
                                      workspace=self.workspace)
        else:
            # rows of no sequence must not reach the next projection: its scale is the maximum over all rows
            o = torch.zeros((T, H, D), dtype=qkv.dtype, device=qkv.device) if self.cu_seqlens is not None else None
            o = svdq_attention_prompt(q, k, v, self.cu_seqlens, self.cu_seqlens, self.causal, self.scale, out=o)
        return o.view(T, H * D)
