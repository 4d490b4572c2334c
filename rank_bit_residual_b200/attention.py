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

import ctypes
import functools
import importlib.util
import math
import os
import warnings
from dataclasses import dataclass
from importlib.machinery import ExtensionFileLoader
from typing import Optional, Tuple

import torch

from . import (SVDQ_BF16, SVDQ_F32, LinearWorkspace, SvdqHeads, SvdqKvCache, SvdqRope, _check, c_sz, load_library)

_BF16 = torch.bfloat16
_TYPES = {torch.bfloat16: SVDQ_BF16, torch.float32: SVDQ_F32}


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
_NO_ROPE = SvdqRope(None, 0, 0, 1.0)

# A decode step calls these functions between kernels of a few microseconds, so their host
# work counts. The usual call goes through _calls.*.so (csrc/attention_calls.cpp), which reads
# the tensors directly: 5 us. What it does not take - a copy to make, another device than the
# current one, a mistake to name - comes back as None and goes the long way below: 15 us.

_calls = None
_calls_lib = None


def _load_calls():
    """The module built for this Python and this torch, and no other."""
    from . import build
    path = build.calls_path()
    if not os.path.exists(path):
        raise ImportError(f"{path} not built; run python -m rank_bit_residual_b200.build")
    loader = ExtensionFileLoader("rank_bit_residual_b200._calls", path)
    module = importlib.util.module_from_spec(importlib.util.spec_from_file_location(loader.name, path, loader=loader))
    loader.exec_module(module)
    return module


def _quick():
    """The module of quick calls, bound to the loaded library; None, after one warning, where it
    is not there (built without torch's headers, say): all goes the long way then."""
    global _calls, _calls_lib
    lib = load_library()
    if _calls_lib is not lib:
        try:
            module = _load_calls()
            module.bind(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in (
                "svdq_qk_norm_rope", "svdq_kv_append", "svdq_attention_prompt", "svdq_attention_prompt_workspace_size",
                "svdq_attention_decode", "svdq_attention_decode_workspace_size")))
        except ImportError as e:
            warnings.warn(f"attention calls without the quick way, some 10 us of host work slower: {e}", RuntimeWarning,
                          stacklevel=3)
            module = None
        _calls, _calls_lib = module, lib
    return _calls


def _device(first, *others) -> int:
    """The index of the one CUDA device that all the tensors live on."""
    dev = first.get_device()
    if dev < 0:
        raise ValueError("tensors must live on a CUDA device")
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError("all tensors must live on one CUDA device")
    return dev


def _raw_stream(dev: int) -> int:
    """torch.cuda.current_stream(dev).cuda_stream without the stream object (1 us less)."""
    return torch._C._cuda_getCurrentRawStream(dev)


def _on_device(call):
    """Run `call` with the tensors' device current, whatever the caller's current device is
    (the first argument, a tensor, names it)."""
    @functools.wraps(call)
    def run(first, *args, **kwargs):
        dev = first.get_device()
        if dev < 0 or dev == torch._C._cuda_getDevice():
            return call(first, *args, **kwargs)
        with torch.cuda.device(dev):
            return call(first, *args, **kwargs)
    return run


@functools.lru_cache(maxsize=4096)
def _layout(shape, stride, size: int):
    """The strides of all axes but the last, as the library takes them, or None where it
    cannot: unit stride along the last axis, 16-byte steps along the others, no broadcast.
    Strides of axes of one element, which torch leaves free, are those of a dense tensor."""
    dim = shape[-1]
    if stride[-1] != 1 and dim > 1:
        return None
    out = list(stride[:-1])
    dense = -(-dim // 8) * 8
    for i in range(len(out) - 1, -1, -1):
        if shape[i] <= 1:
            out[i] = dense
        if out[i] * size % 16 or out[i] < dim:
            return None
        dense = max(dense, out[i] * shape[i])
    return tuple(out)


def _heads(t: torch.Tensor, shape):
    """(descriptor, the tensor it points to) of an input; a copy where the layout needs one."""
    s, p = _layout(shape, t.stride(), t.element_size()), t.data_ptr()
    if s is None or p & 15:
        t = t.clone(memory_format=torch.contiguous_format)
        s, p = _layout(shape, t.stride(), t.element_size()), t.data_ptr()
        if s is None:
            raise ValueError(f"rows of {shape[-1]} elements are not a multiple of 16 bytes")
    return SvdqHeads(p, s[0], s[1], shape[1]), t


def _out_heads(t: Optional[torch.Tensor], name: str, like: torch.Tensor, shape):
    """(descriptor, tensor) of an output of the shape and type of `like`: the given one, or
    a dense new one."""
    if t is None:
        t = torch.empty_like(like, memory_format=torch.contiguous_format)
        return SvdqHeads(t.data_ptr(), shape[1] * shape[2], shape[2], shape[1]), t
    if t.shape != shape or t.dtype != like.dtype:
        raise ValueError(f"{name} must be {like.dtype} {tuple(shape)}")
    s, p = _layout(shape, t.stride(), t.element_size()), t.data_ptr()
    if s is None or p & 15:
        raise ValueError(f"{name} needs unit stride along head_dim, 16-byte aligned rows and no broadcast axis")
    return SvdqHeads(p, s[0], s[1], shape[1]), t


def _shape3(t: torch.Tensor, name: str, dtype):
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim]")
    return shape


def _vector(t, name: str, dtype, n: int):
    if t.dtype != dtype or t.numel() != n or t.dim() != 1:
        raise ValueError(f"{name} must be {dtype} [{n}]")
    return t if t.is_contiguous() else t.contiguous()


def _weight(w, dim: int):
    """(norm weight, its type) as the library takes it."""
    t = _TYPES.get(w.dtype)
    if t is None or w.numel() != dim or w.dim() != 1:
        raise ValueError(f"a norm weight must be bfloat16 or float32 [{dim}]")
    if not w.is_contiguous() or w.data_ptr() & 15:
        w = w.clone(memory_format=torch.contiguous_format)
    return w, t


def _weights(q_weight, k_weight, dim: int):
    """(the weights, their pointers, their type) as the library takes them."""
    q_p = k_p = None
    t = qt = kt = SVDQ_BF16
    if q_weight is not None:
        q_weight, qt = _weight(q_weight, dim)
        q_p, t = q_weight.data_ptr(), qt
    if k_weight is not None:
        k_weight, kt = _weight(k_weight, dim)
        k_p, t = k_weight.data_ptr(), kt
        if q_p is not None and qt != kt:
            raise ValueError("the norm weights must have one type")
    return q_weight, k_weight, q_p, k_p, t


def _rotation(rope: Optional[Rope], positions, tokens: int, dim: int):
    """(descriptor, pointer to the positions, tensors to keep until the launch)."""
    if rope is None:
        return _NO_ROPE, None, None
    turns = rope.turns
    n = turns.numel()
    if n == 0:
        return _NO_ROPE, None, None
    if positions is None:
        raise ValueError("a rotation needs positions")
    positions = _vector(positions, "positions", torch.int64, tokens)
    if turns.dtype != torch.float64 or turns.dim() != 1:
        raise ValueError("turns must be float64 [rot_dim / 2]")
    if 2 * n > dim:
        raise ValueError("rot_dim must not exceed head_dim")
    turns = turns.contiguous()
    return (SvdqRope(turns.data_ptr(), 2 * n, 1 if rope.interleaved else 0, rope.amplitude), positions.data_ptr(),
            (positions, turns))


def _cache(k_cache, v_cache):
    shape, stride = k_cache.shape, k_cache.stride()
    if len(shape) != 4 or k_cache.dtype != _BF16 or v_cache.dtype != _BF16:
        raise ValueError("a cache must be bfloat16 [pages, page_size, heads, head_dim]")
    if v_cache.shape != shape or (v_cache.stride() != stride and _layout(shape, v_cache.stride(), 2) !=
                                  _layout(shape, stride, 2)):
        raise ValueError("k_cache and v_cache must have one shape and layout")
    if 0 in shape:
        raise ValueError("the cache is empty")
    s, k, v = _layout(shape, stride, 2), k_cache.data_ptr(), v_cache.data_ptr()
    if s is None or k & 15 or v & 15:
        raise ValueError("a cache needs unit stride along head_dim and 16-byte aligned rows")
    return SvdqKvCache(k, v, shape[0], s[0], s[1], s[2], shape[1], shape[2], shape[3])


def svdq_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: Optional[torch.Tensor] = None,
                      rope: Optional[Rope] = None, q_weight: Optional[torch.Tensor] = None,
                      k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                      q_out: Optional[torch.Tensor] = None,
                      k_out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """RMS norm (with a weight) and rotation (with a rope) of query and key heads, one pass.

    q [T, H, D], k [T, Hkv, D], bf16 or fp32; positions int64 [T]; weights [D] bf16 or
    fp32. q_out=q, k_out=k work in place. Returns (q_out, k_out).
    """
    turns, inter, amp = (None, False, 1.0) if rope is None else (rope.turns, rope.interleaved, rope.amplitude)
    quick = _quick()
    if quick is not None:
        done = quick.norm_rope(q, k, positions, turns, inter, amp, q_weight, k_weight, eps, q_out, k_out)
        if done is not None:
            return done
    return _qk_norm_rope(q, k, positions, rope, q_weight, k_weight, eps, q_out, k_out)


@_on_device
def _qk_norm_rope(q, k, positions, rope, q_weight, k_weight, eps, q_out, k_out):
    dev = _device(q, k, positions, q_weight, k_weight, q_out, k_out, None if rope is None else rope.turns)
    dt = _TYPES.get(q.dtype)
    if dt is None:
        raise ValueError(f"unsupported dtype {q.dtype}")
    qs, ks = _shape3(q, "q", q.dtype), _shape3(k, "k", q.dtype)
    T, H, D = qs
    if ks[0] != T or ks[2] != D:
        raise ValueError(f"k must be [{T}, heads, {D}]")
    qw, kw, qw_p, kw_p, wdt = _weights(q_weight, k_weight, D)
    r, pos, _keep = _rotation(rope, positions, T, D)
    if T == 0 or H == 0 or ks[1] == 0:   # nothing of q or of k
        q_out = q.new_empty(qs) if q_out is None else q_out
        k_out = k.new_empty(ks) if k_out is None else k_out
        if T == 0:
            return q_out, k_out
    qd, q = _heads(q, qs) if H else (_NO_HEADS, q)
    kd, k = _heads(k, ks) if ks[1] else (_NO_HEADS, k)
    qo, q_out = _out_heads(q_out, "q_out", q, qs) if H else (_NO_HEADS, q_out)
    ko, k_out = _out_heads(k_out, "k_out", k, ks) if ks[1] else (_NO_HEADS, k_out)
    st = load_library().svdq_qk_norm_rope(qd, kd, dt, T, D, pos, r, qw_p, kw_p, wdt, eps, qo, ko, _raw_stream(dev))
    if st:
        _check(st, "svdq_qk_norm_rope")
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
    quick = _quick() if q is not None else None
    if quick is not None:
        turns, inter, amp = (None, False, 1.0) if rope is None else (rope.turns, rope.interleaved, rope.amplitude)
        done = quick.append(k_cache, v_cache, k, v, slots, positions, turns, inter, amp, k_weight, eps, q, q_weight,
                            q_out, k_out)
        if done is not None:
            return done
    return _kv_append(k_cache, v_cache, k, v, slots, positions, rope, k_weight, eps, q, q_weight, q_out, k_out)


@_on_device
def _kv_append(k_cache, v_cache, k, v, slots, positions, rope, k_weight, eps, q, q_weight, q_out, k_out):
    dev = _device(k_cache, v_cache, k, v, slots, positions, k_weight, q, q_weight, q_out, k_out,
                  None if rope is None else rope.turns)
    c = _cache(k_cache, v_cache)
    D = c.head_dim
    ks, vs = _shape3(k, "k", _BF16), _shape3(v, "v", _BF16)
    T = ks[0]
    if ks != (T, c.heads, D) or vs != ks:
        raise ValueError(f"k and v must be [tokens, {c.heads}, {D}]")
    if q is not None:
        qs = _shape3(q, "q", _BF16)
        if qs[0] != T or qs[2] != D or qs[1] == 0:
            raise ValueError(f"q must be [{T}, heads, {D}]")
    elif q_out is not None or q_weight is not None:
        raise ValueError("q_out and q_weight need q")
    qw, kw, qw_p, kw_p, wdt = _weights(q_weight, k_weight, D)
    r, pos, _keep = _rotation(rope, positions, T, D)
    slots = _vector(slots, "slots", torch.int64, T)
    if T == 0:
        return q_out if q is None or q_out is not None else q.new_empty(qs)
    kd, k_in = _heads(k, ks)
    vd, v = _heads(v, vs)
    qd = qo = ko = _NO_HEADS
    if q is not None:
        qd, q = _heads(q, qs)
        qo, q_out = _out_heads(q_out, "q_out", q, qs)
    if k_out is not None:
        ko, k_out = _out_heads(k_out, "k_out", k, ks)
    st = load_library().svdq_kv_append(c, kd, vd, slots.data_ptr(), T, pos, r, kw_p, wdt, eps, qd, qw_p, qo, ko,
                                       _raw_stream(dev))
    if st:
        _check(st, "svdq_kv_append")
    return q_out


@functools.lru_cache(maxsize=4096)
def _prompt_scratch(dev: int, heads: int, kv_heads: int, dim: int, batch: int, q_tokens: int, k_tokens: int) -> int:
    size = c_sz()
    _check(load_library().svdq_attention_prompt_workspace_size(heads, kv_heads, dim, batch, q_tokens, k_tokens,
                                                               ctypes.byref(size)),
           "svdq_attention_prompt_workspace_size")
    return size.value


def svdq_attention_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: Optional[torch.Tensor] = None,
                          cu_k: Optional[torch.Tensor] = None, causal: bool = True,
                          scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                          workspace: Optional[LinearWorkspace] = None) -> torch.Tensor:
    """Attention over packed sequences: q [Tq, H, D], k and v [Tk, Hkv, D], bf16.

    cu_q, cu_k int32 [batch + 1]: sequence s owns rows cu[s] .. cu[s + 1] - 1 (None: one
    sequence of all rows). causal: rows and keys of a sequence end together, and a row
    sees no key behind its own place; a row that sees none becomes zero. Rows of no
    sequence are left as they were in `out`, and mean nothing in an output allocated here.
    Scratch (few rows over many keys need some) is allocated per call unless a workspace
    is given (one per stream in flight). Returns [Tq, H, D].
    """
    quick = _quick() if workspace is None else None
    if quick is not None:
        done = quick.prompt(q, k, v, cu_q, cu_k, causal, scale, out)
        if done is not None:
            return done
    return _attention_prompt(q, k, v, cu_q, cu_k, causal, scale, out, workspace)


@_on_device
def _attention_prompt(q, k, v, cu_q, cu_k, causal, scale, out, workspace):
    dev = _device(q, k, v, cu_q, cu_k, out)
    qs, ks, vs = _shape3(q, "q", _BF16), _shape3(k, "k", _BF16), _shape3(v, "v", _BF16)
    T, H, D = qs
    if ks[2] != D or vs != ks:
        raise ValueError(f"k and v must be of one size [keys, heads, {D}]")
    if H == 0 or ks[1] == 0 or H % ks[1]:
        raise ValueError("the query heads must be a multiple of the key heads")
    batch = -1
    for name, cu in (("cu_q", cu_q), ("cu_k", cu_k)):
        n = 1
        if cu is not None:
            if cu.dtype != torch.int32 or cu.dim() != 1 or cu.numel() < 1:
                raise ValueError(f"{name} must be int32 [batch + 1]")
            n = cu.numel() - 1
        if batch not in (-1, n):
            raise ValueError("cu_q and cu_k must have one length")
        batch = n
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    qo, out = _out_heads(out, "out", q, qs)
    if T == 0:
        return out
    qd, q = _heads(q, qs)
    kd, k = _heads(k, ks)
    vd, v = _heads(v, vs)
    cu_q = None if cu_q is None else cu_q.contiguous()
    cu_k = None if cu_k is None else cu_k.contiguous()
    size, ws = _prompt_scratch(dev, H, ks[1], D, batch, T, ks[0]), None
    if size:
        ws = q.new_empty(size, dtype=torch.uint8) if workspace is None else workspace.get(size, q.device)
    st = load_library().svdq_attention_prompt(
        qd, kd, vd, None if cu_q is None else cu_q.data_ptr(), None if cu_k is None else cu_k.data_ptr(), batch, T,
        ks[0], D, 1 if causal else 0, scale, qo, None if ws is None else ws.data_ptr(), size, _raw_stream(dev))
    if st:
        _check(st, "svdq_attention_prompt")
    return out


@functools.lru_cache(maxsize=4096)
def _decode_scratch(dev: int, batch: int, heads: int, kv_heads: int, dim: int) -> int:
    size = c_sz()
    _check(load_library().svdq_attention_decode_workspace_size(batch, heads, kv_heads, dim, ctypes.byref(size)),
           "svdq_attention_decode_workspace_size")
    return size.value


def svdq_attention_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                          kv_len: torch.Tensor, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                          workspace: Optional[LinearWorkspace] = None) -> torch.Tensor:
    """Attention of one token per sequence over a paged cache: q [B, H, D] bf16.

    Caches as in svdq_kv_append; page_table int32 [B, pages per sequence], kv_len int32
    [B] (0: a zero row). The scratch is allocated per call unless a workspace is given
    (one per stream in flight). Returns [B, H, D].
    """
    quick = _quick() if workspace is None else None
    if quick is not None:
        done = quick.decode(q, k_cache, v_cache, page_table, kv_len, scale, out)
        if done is not None:
            return done
    return _attention_decode(q, k_cache, v_cache, page_table, kv_len, scale, out, workspace)


@_on_device
def _attention_decode(q, k_cache, v_cache, page_table, kv_len, scale, out, workspace):
    dev = _device(q, k_cache, v_cache, page_table, kv_len, out)
    c = _cache(k_cache, v_cache)
    qs = _shape3(q, "q", _BF16)
    B, H, D = qs
    if D != c.head_dim:
        raise ValueError(f"q must be [batch, heads, {c.head_dim}]")
    if H == 0 or H % c.heads:
        raise ValueError("the query heads must be a multiple of the key heads")
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError(f"page_table must be int32 [{B}, pages]")
    kv_len = _vector(kv_len, "kv_len", torch.int32, B)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    qo, out = _out_heads(out, "out", q, qs)
    if B == 0:
        return out
    page_table = page_table.contiguous()
    size = _decode_scratch(dev, B, H, c.heads, D)
    ws = q.new_empty(size, dtype=torch.uint8) if workspace is None else workspace.get(size, q.device)
    qd, q = _heads(q, qs)
    st = load_library().svdq_attention_decode(qd, c, page_table.data_ptr(), page_table.shape[1], kv_len.data_ptr(), B,
                                              scale, qo, ws.data_ptr(), ws.numel(), _raw_stream(dev))
    if st:
        _check(st, "svdq_attention_decode")
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
            o = svdq_attention_prompt(q, k, v, self.cu_seqlens, self.cu_seqlens, self.causal, self.scale, out=o,
                                      workspace=self.workspace)
        return o.view(T, H * D)
