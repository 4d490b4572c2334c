"""Refusals of the attention operators: argument checks on the host, before anything
touches the device (the pointers here are never dereferenced)."""

import ctypes

import pytest
import torch

import rank_bit_residual_b200 as rb
from rank_bit_residual_b200 import build as rbuild

P = 0x10000          # an aligned, never dereferenced address
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    rbuild.build()
    return rb.load_library()


def heads(n=4, dim=64, data=P, tokens_first=True, **kw):
    d = dict(data=data, token_ld=n * dim, head_ld=dim, heads=n)
    d.update(kw)
    return rb.SvdqHeads(**d)


NONE = rb.SvdqHeads(None, 0, 0, 0)
ROPE = dict(turns=P, rot_dim=64, interleaved=0, amplitude=1.0)


def norm_rope(lib, q=None, k=None, dtype=1, tokens=3, dim=64, positions=P, rope=None, qw=P, kw=P, wdt=1, eps=1e-6,
              qo=None, ko=None):
    q = heads() if q is None else q
    k = heads(2) if k is None else k
    return lib.svdq_qk_norm_rope(q, k, dtype, tokens, dim, positions, rb.SvdqRope(**{**ROPE, **(rope or {})}), qw, kw,
                                 wdt, eps, heads(data=2 * P) if qo is None else qo,
                                 heads(2, data=2 * P) if ko is None else ko, None)


@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(tokens=-1), dict(dim=0), dict(positions=None), dict(rope=dict(turns=None)),
    dict(rope=dict(rot_dim=66)), dict(rope=dict(rot_dim=7)), dict(rope=dict(rot_dim=-2)),
    dict(rope=dict(interleaved=2)), dict(rope=dict(amplitude=float("nan"))), dict(wdt=7), dict(eps=-1.0),
    dict(eps=float("inf")), dict(eps=float("nan")), dict(q=heads(data=None)), dict(q=heads(token_ld=32)),
    dict(q=heads(head_ld=32)), dict(q=heads(n=0)), dict(qo=heads(3, data=2 * P)), dict(qo=NONE), dict(k=NONE),
    dict(qo=heads(data=P, token_ld=512)),     # in place with other strides
])
def test_norm_rope_invalid(lib, kw):
    assert norm_rope(lib, **kw) == rb.SVDQ_EINVAL


@pytest.mark.parametrize("kw", [
    dict(dim=60), dict(dim=264), dict(tokens=BIG), dict(q=heads(data=P + 8)), dict(q=heads(token_ld=257)),
    dict(q=heads(head_ld=65)), dict(qo=heads(data=2 * P + 2)), dict(qw=P + 2), dict(kw=P + 4),
])
def test_norm_rope_unsupported(lib, kw):
    assert norm_rope(lib, **kw) == rb.SVDQ_EUNSUPPORTED


def test_nothing_to_do_is_ok(lib):
    assert norm_rope(lib, tokens=0) == rb.SVDQ_OK
    assert norm_rope(lib, q=NONE, k=NONE, qo=NONE, ko=NONE) == rb.SVDQ_OK
    assert prompt(lib, q_tokens=0) == rb.SVDQ_OK
    assert prompt(lib, batch=0) == rb.SVDQ_OK
    assert decode(lib, batch=0) == rb.SVDQ_OK
    assert append(lib, tokens=0) == rb.SVDQ_OK


def cache(**kw):
    d = dict(k=P, v=P, pages=10, page_ld=16 * 2 * 64, slot_ld=2 * 64, head_ld=64, page_size=16, heads=2, head_dim=64)
    d.update(kw)
    return rb.SvdqKvCache(**d)


def append(lib, c=None, k=None, v=None, slots=P, tokens=3, positions=P, rope=None, kw=P, wdt=1, eps=1e-6, q=None,
           qw=P, qo=None, ko=NONE):
    c = cache() if c is None else c
    return lib.svdq_kv_append(ctypes.byref(c) if c != "none" else None, heads(2) if k is None else k,
                              heads(2) if v is None else v, slots, tokens, positions,
                              rb.SvdqRope(**{**ROPE, **(rope or {})}), kw, wdt, eps, heads() if q is None else q, qw,
                              heads(data=2 * P) if qo is None else qo, ko, None)


@pytest.mark.parametrize("kw", [
    dict(c="none"), dict(c=cache(k=None)), dict(c=cache(v=None)), dict(c=cache(pages=0)), dict(c=cache(page_size=0)),
    dict(c=cache(heads=0)), dict(c=cache(head_dim=0)), dict(c=cache(slot_ld=32)), dict(c=cache(head_ld=8)),
    dict(c=cache(page_ld=8)), dict(slots=None), dict(tokens=-1), dict(k=heads(3)), dict(v=heads(3)),
    dict(k=heads(2, data=None)), dict(v=NONE), dict(q=NONE), dict(qo=NONE), dict(ko=heads(3)), dict(positions=None),
    dict(rope=dict(rot_dim=128)), dict(eps=-1.0), dict(wdt=3),
])
def test_append_invalid(lib, kw):
    assert append(lib, **kw) == rb.SVDQ_EINVAL


@pytest.mark.parametrize("kw", [
    dict(c=cache(k=P + 8)), dict(c=cache(page_ld=16 * 128 + 4)), dict(c=cache(slot_ld=132)), dict(c=cache(head_ld=68)),
    dict(c=cache(head_dim=60)), dict(c=cache(head_dim=264, slot_ld=528, head_ld=264)), dict(tokens=BIG),
    dict(k=heads(2, data=P + 2)), dict(v=heads(2, token_ld=129)), dict(ko=heads(2, data=P + 2)), dict(kw=P + 2),
])
def test_append_unsupported(lib, kw):
    assert append(lib, **kw) == rb.SVDQ_EUNSUPPORTED


def prompt(lib, q=None, k=None, v=None, cu_q=P, cu_k=P, batch=2, q_tokens=5, k_tokens=5, dim=64, causal=1, scale=0.1,
           out=None, ws=None, ws_bytes=0):
    return lib.svdq_attention_prompt(heads() if q is None else q, heads(2) if k is None else k,
                                     heads(2) if v is None else v, cu_q, cu_k, batch, q_tokens, k_tokens, dim, causal,
                                     scale, heads(data=2 * P) if out is None else out, ws, ws_bytes, None)


@pytest.mark.parametrize("kw", [
    dict(batch=-1), dict(q_tokens=-1), dict(k_tokens=-1), dict(causal=2), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(scale=3e38), dict(cu_q=None), dict(cu_k=None), dict(q=NONE), dict(q=heads(3)), dict(v=heads(4)),
    dict(k=heads(2, data=None)), dict(k=heads(0), v=heads(0)), dict(out=heads()), dict(out=heads(2, data=2 * P)),
    dict(dim=0),
])
def test_prompt_invalid(lib, kw):
    assert prompt(lib, **kw) == rb.SVDQ_EINVAL


@pytest.mark.parametrize("kw", [
    dict(dim=60), dict(dim=136), dict(q_tokens=1 << 25), dict(k_tokens=1 << 25), dict(q=heads(data=P + 2)),
    dict(k=heads(2, token_ld=130)), dict(out=heads(data=2 * P + 8)),
    dict(q=heads(1 << 15), out=heads(1 << 15, data=2 * P), q_tokens=1 << 24),
])
def test_prompt_unsupported(lib, kw):
    if kw.get("dim") == 136:
        kw = dict(kw, q=heads(dim=136), k=heads(2, dim=136), v=heads(2, dim=136), out=heads(dim=136, data=2 * P))
    assert prompt(lib, **kw) == rb.SVDQ_EUNSUPPORTED


def test_prompt_workspace(lib):
    n = ctypes.c_size_t(7)
    size = lib.svdq_attention_prompt_workspace_size
    assert size(32, 8, 128, 1, 8192, 8192, ctypes.byref(n)) == rb.SVDQ_OK and n.value == 0
    assert size(4, 2, 64, 0, 0, 0, ctypes.byref(n)) == rb.SVDQ_OK and n.value == 0
    assert size(4, 2, 64, 1, 100, 8192, ctypes.byref(n)) == rb.SVDQ_OK and n.value > 0   # few rows, many keys
    few = dict(batch=1, q_tokens=100, k_tokens=8192)
    assert prompt(lib, **few) == rb.SVDQ_EWORKSPACE
    assert prompt(lib, ws=P, ws_bytes=n.value - 1, **few) == rb.SVDQ_EWORKSPACE
    assert prompt(lib, ws=P + 8, ws_bytes=n.value, **few) == rb.SVDQ_EUNSUPPORTED
    assert size(4, 3, 64, 1, 100, 8192, ctypes.byref(n)) == rb.SVDQ_EINVAL
    assert size(4, 2, 60, 1, 100, 8192, ctypes.byref(n)) == rb.SVDQ_EUNSUPPORTED
    assert size(4, 2, 64, 1, 100, 8192, None) == rb.SVDQ_EINVAL


def decode(lib, q=None, c=None, table=P, table_ld=4, kv_len=P, batch=3, scale=0.1, out=None, ws=P, ws_bytes=1 << 30):
    c = cache() if c is None else c
    return lib.svdq_attention_decode(heads() if q is None else q, ctypes.byref(c) if c != "none" else None, table,
                                     table_ld, kv_len, batch, scale, heads(data=2 * P) if out is None else out, ws,
                                     ws_bytes, None)


@pytest.mark.parametrize("kw", [
    dict(c="none"), dict(c=cache(pages=0)), dict(q=heads(3)), dict(q=NONE), dict(table=None), dict(table_ld=-1),
    dict(kv_len=None), dict(batch=-1), dict(scale=float("nan")), dict(scale=-3e38), dict(out=heads()), dict(out=heads(2, data=2 * P)),
])
def test_decode_invalid(lib, kw):
    assert decode(lib, **kw) == rb.SVDQ_EINVAL


@pytest.mark.parametrize("kw", [
    dict(c=cache(head_dim=136, slot_ld=272, head_ld=136)), dict(c=cache(v=P + 2)), dict(q=heads(data=P + 2)),
    dict(ws=P + 8), dict(batch=1 << 30),
])
def test_decode_unsupported(lib, kw):
    assert decode(lib, **kw) == rb.SVDQ_EUNSUPPORTED


def test_decode_workspace(lib):
    n = ctypes.c_size_t()
    assert lib.svdq_attention_decode_workspace_size(3, 4, 2, 64, ctypes.byref(n)) == rb.SVDQ_OK and n.value > 0
    assert decode(lib, ws_bytes=n.value - 1) == rb.SVDQ_EWORKSPACE
    assert decode(lib, ws=None) == rb.SVDQ_EWORKSPACE
    assert lib.svdq_attention_decode_workspace_size(3, 4, 3, 64, ctypes.byref(n)) == rb.SVDQ_EINVAL
    assert lib.svdq_attention_decode_workspace_size(3, 4, 2, 136, ctypes.byref(n)) == rb.SVDQ_EUNSUPPORTED
    assert lib.svdq_attention_decode_workspace_size(3, 4, 2, 64, None) == rb.SVDQ_EINVAL


def test_binding_refuses_host_tensors():
    """No CPU path: host tensors raise."""
    t = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    c = torch.zeros((3, 16, 4, 64), dtype=torch.bfloat16)
    i32, i64 = torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int64)
    for call in (lambda: rb.svdq_qk_norm_rope(t, t), lambda: rb.svdq_kv_append(c, c, t, t, i64),
                 lambda: rb.svdq_attention_prompt(t, t, t),
                 lambda: rb.svdq_attention_decode(t, c, c, i32.view(2, 1), i32)):
        with pytest.raises(ValueError):
            call()


def test_rope_make_refuses():
    for kw in (dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=8.0), dict(rot_dim=True), dict(rot_dim=8, base=0.0),
               dict(rot_dim=8, factor=0.5), dict(rot_dim=8, fast=1.0, slow=1.0)):
        with pytest.raises(ValueError):
            rb.Rope.make(device="cpu", **kw)


def test_rope_make_scales():
    plain = rb.Rope.make(64, device="cpu")
    assert plain.rot_dim == 64 and plain.turns.dtype == torch.float64
    assert abs(float(plain.turns[0]) * 2 * 3.141592653589793 - 1) < 1e-15
    assert torch.equal(rb.Rope.make(64, factor=4.0, device="cpu").turns, plain.turns / 4)
    part = rb.Rope.make(64, factor=8.0, trained_len=4096, device="cpu")
    ratio = part.turns / plain.turns
    assert float(ratio[0]) == 1.0 and float(ratio[-1]) == 0.125      # fast pairs kept, slow ones interpolated
    assert bool((ratio[1:] <= ratio[:-1]).all()) and abs(part.amplitude - 1.2079441541679836) < 1e-12


def test_attention_step_refuses():
    x = torch.zeros((3, 8 * 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        rb.AttentionStep(heads=4, kv_heads=3, head_dim=64)(x)                  # row length
    with pytest.raises(ValueError):
        rb.AttentionStep(heads=4, kv_heads=2, head_dim=64, k_cache=x)(x)       # half a cache
    with pytest.raises(ValueError):
        rb.AttentionStep(heads=4, kv_heads=2, head_dim=64, kv_len=x)(x)        # lengths without a table


def test_chain_steps_take_no_bias_or_output():
    class Step:
        def __call__(self, y):
            return y + 1
    x = torch.zeros(2, 4)
    assert torch.equal(rb.svdq_linear_chain([Step(), Step()], x), x + 2)
    with pytest.raises(ValueError):
        rb.svdq_linear_chain([Step()], x, biases=[x])
    with pytest.raises(ValueError):
        rb.svdq_linear_chain([Step()], x, outs=[x])
