"""svdq_qk_norm_rope and svdq_kv_append against the float64 definition: every lane layout of
the head, both rotation layouts, parts of the head, far positions, strides, padding."""

import numpy as np
import pytest
import torch

import rank_bit_residual_b200 as rb
from oracle import attention as oa
from tests.gpu_util import device

pytestmark = pytest.mark.gpu


def draw(seed, *shape, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).to(device())


def f64(t):
    return t.detach().double().cpu().numpy()


def want(x, weight, positions, rope, eps):
    y = oa.norm(f64(x), None if weight is None else f64(weight), eps)
    if rope is None:
        return y, np.abs(y)
    return oa.rotate(y, positions.cpu().numpy(), rope.turns.cpu().numpy(), rope.interleaved, rope.amplitude)


def check(got, x, weight, positions, rope, eps, what):
    y, mag = want(x, weight, positions, rope, eps)
    err = np.abs(f64(got) - y)
    tol = oa.norm_rope_tolerance(y, mag, torch.finfo(x.dtype).eps)
    assert np.all(err <= tol), f"{what}: {np.max(err / np.maximum(tol, 1e-300)):.3f} of the tolerance"


# tokens, heads, kv heads, head_dim, rot_dim, interleaved
SHAPES = [
    (1, 1, 1, 8, 8, False), (1, 32, 8, 128, 128, False), (3, 5, 1, 64, 64, True), (7, 3, 3, 80, 40, False),
    (5, 4, 2, 96, 96, False), (2, 6, 2, 256, 256, False), (9, 2, 1, 248, 62, False), (4, 3, 1, 120, 2, True),
    (1201, 12, 4, 128, 64, False), (2500, 4, 4, 64, 32, True), (13, 40, 8, 72, 36, False), (2, 1, 7, 16, 0, False),
]


@pytest.mark.parametrize("T,H,K,D,rot,inter", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("normed", [True, False])
def test_norm_rope(T, H, K, D, rot, inter, dtype, normed):
    row = draw(T + D, T, (H + 2 * K) * D, dtype=dtype)
    q, k, _ = row.view(T, -1, D).split([H, K, K], 1)
    pos = torch.randint(-1000, 200000, (T,), generator=torch.Generator().manual_seed(D)).to(device())
    rope = rb.Rope.make(rot, interleaved=inter, factor=4.0, trained_len=2048) if rot else None
    qw = draw(1, D, dtype=torch.float32) if normed else None
    kw = draw(2, D, dtype=torch.float32) if normed else None
    before = row.clone()
    qo, ko = rb.svdq_qk_norm_rope(q, k, pos, rope, qw, kw, 1e-5)
    assert rb.svdq_check_status() == rb.SVDQ_OK
    assert torch.equal(row, before)
    check(qo, q, qw, pos, rope, 1e-5, "q")
    check(ko, k, kw, pos, rope, 1e-5, "k")
    # in place: the same bits, the values untouched
    v = row.view(T, -1, D)[:, H + K:].clone()
    rb.svdq_qk_norm_rope(q, k, pos, rope, qw, kw, 1e-5, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(row.view(T, -1, D)[:, H + K:], v)


def test_weights_of_one_side_and_bf16():
    T, H, K, D = 33, 4, 2, 128
    q, k = draw(1, T, H, D), draw(2, T, K, D)
    w = draw(3, D)
    qo, ko = rb.svdq_qk_norm_rope(q, k, q_weight=w)
    check(qo, q, w, None, None, 1e-6, "q")
    assert torch.equal(ko, k)


def test_far_positions_lose_nothing():
    """fp32 angles would be off by whole turns at these positions."""
    T, D = 4, 128
    q, k = draw(1, T, 2, D, dtype=torch.float32), draw(2, T, 1, D, dtype=torch.float32)
    pos = torch.tensor([2 ** 31 + 5, 10 ** 9 + 7, -(2 ** 30) - 1, 16777217], device=device())
    rope = rb.Rope.make(D)
    qo, ko = rb.svdq_qk_norm_rope(q, k, pos, rope)
    # the product position * turns is rounded in fp64 on both sides: 2^31 / (2 pi) turns
    # times 2^-53 is 2^-24.6 of a turn, 4 half steps of fp32 in the angle at most
    for got, x in ((qo, q), (ko, k)):
        y, mag = want(x, None, pos, rope, 0.0)
        err = np.abs(f64(got) - y)
        assert np.all(err <= oa.norm_rope_tolerance(y, mag, 2.0 ** -23) + 2 * 4 * 2.0 ** -24 * mag)


def test_zero_rows_large_and_small_values():
    D = 128
    q = torch.zeros((4, 1, D), device=device(), dtype=torch.float32)
    q[1] = 1e-30
    q[2] = 1e15
    q[3, 0, 5] = float("inf")
    w = torch.ones(D, device=device())
    qo, _ = rb.svdq_qk_norm_rope(q, q[:, :0], q_weight=w)
    assert torch.all(qo[0] == 0) and torch.all(qo[1].abs() <= 1.001e-27)
    assert torch.allclose(qo[2], torch.ones_like(qo[2]), rtol=1e-5)
    assert torch.isnan(qo[3, 0, 5]) and torch.all(qo[3, 0, :5] == 0)


def test_transposed_and_unaligned_inputs():
    T, H, D = 11, 3, 64
    q = draw(5, H, T, D).transpose(0, 1)                  # heads first in memory
    flat = draw(6, T * H * D + 3)
    k = flat[3:].view(T, H, D)                            # 6 bytes off a 16-byte boundary
    pos = torch.arange(T, device=device())
    rope = rb.Rope.make(D)
    qo, ko = rb.svdq_qk_norm_rope(q, k, pos, rope)
    check(qo, q, None, pos, rope, 0.0, "transposed")
    check(ko, k, None, pos, rope, 0.0, "unaligned")
    with pytest.raises(ValueError):
        rb.svdq_qk_norm_rope(q, q, pos, rope, k_out=k)    # outputs are not copied
    with pytest.raises(ValueError):
        rb.svdq_qk_norm_rope(q, q, pos, rope, q_out=torch.empty((1, H, D), device=device(), dtype=q.dtype).expand(T, H, D))
    expanded = draw(7, T, 1, D).expand(T, H, D)           # a broadcast input is copied
    eo, _ = rb.svdq_qk_norm_rope(expanded, q, pos, rope)
    check(eo, expanded, None, pos, rope, 0.0, "broadcast")


def test_wrong_arguments_raise():
    q = draw(1, 4, 2, 64)
    rope = rb.Rope.make(64)
    pos = torch.arange(4, device=device())
    for kw in (dict(positions=None, rope=rope), dict(positions=pos.int(), rope=rope), dict(positions=pos[:3], rope=rope),
               dict(positions=pos, rope=rb.Rope.make(128)), dict(q_weight=draw(1, 32)), dict(eps=-1.0),
               dict(q_weight=draw(1, 64), k_weight=draw(1, 64).float()), dict(q_weight=draw(1, 64).half()),
               dict(positions=pos, rope=rb.Rope(rope.turns.float())), dict(positions=pos.cpu(), rope=rope),
               dict(q_out=q[:3]), dict(q_out=q.float())):
        with pytest.raises(ValueError):
            rb.svdq_qk_norm_rope(q, q, **kw)
    with pytest.raises(ValueError):
        rb.svdq_qk_norm_rope(q, q.float())
    with pytest.raises(ValueError):
        rb.svdq_qk_norm_rope(q.half(), q.half())
    with pytest.raises(ValueError):
        rb.svdq_qk_norm_rope(q[0], q)


# ------------------------------------------------------------------ appending to a cache
def make_cache(pages, page, K, D, heads_first, seed=3):
    if heads_first:
        k, v = draw(seed, pages, K, page, D).transpose(1, 2), draw(seed + 1, pages, K, page, D).transpose(1, 2)
    else:
        k, v = draw(seed, pages, page, K, D), draw(seed + 1, pages, page, K, D)
    return k, v


def run_append(T, H, K, D, page, heads_first, padded=0, with_q=True, with_k_out=True, inter=False, normed=True):
    row = draw(T, T, (H + 2 * K) * D)
    q, k, v = row.view(T, -1, D).split([H, K, K], 1)
    pages = 2 + 2 * T // page
    kc, vc = make_cache(pages, page, K, D, heads_first)
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(T))[:T].to(device())
    if padded:
        slots[::padded] = -1 - torch.arange(len(slots[::padded]), device=device())
    pos = torch.arange(T, device=device()) + 77
    rope = rb.Rope.make(D, interleaved=inter)
    qw, kw = (draw(8, D), draw(9, D)) if normed else (None, None)
    k0, v0 = f64(kc), f64(vc)
    vbits = vc.clone()
    ko = torch.empty((T, K, D), dtype=torch.bfloat16, device=device()) if with_k_out else None
    qo = rb.svdq_kv_append(kc, vc, k, v, slots, pos, rope, kw, q=q if with_q else None, q_weight=qw if with_q else None,
                           k_out=ko)
    assert rb.svdq_check_status() == rb.SVDQ_OK
    if with_q:
        check(qo, q, qw, pos, rope, 1e-6, "q")
    else:
        assert qo is None
    y, mag = want(k, kw, pos, rope, 1e-6)
    tol = oa.norm_rope_tolerance(y, mag, torch.finfo(torch.bfloat16).eps)
    s = slots.cpu().numpy()
    assert np.all(np.abs(f64(kc) - oa.append(k0, y, s)) <= oa.append(np.zeros_like(k0), tol, s))   # others: no change
    assert np.array_equal(f64(vc), oa.append(v0, f64(v), s))
    if with_k_out:
        check(ko, k, kw, pos, rope, 1e-6, "k_out")
        live = slots >= 0
        assert torch.equal(kc[slots[live] // page, slots[live] % page], ko[live])
    del vbits


@pytest.mark.parametrize("T,H,K,D,page", [(1, 32, 8, 128, 16), (5, 4, 2, 64, 7), (300, 6, 3, 96, 32), (2049, 8, 8, 128, 64),
                                          (3, 2, 1, 256, 1)])
@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("padded", [0, 1, 3])
def test_append(T, H, K, D, page, heads_first, padded):
    run_append(T, H, K, D, page, heads_first, padded)


@pytest.mark.parametrize("with_q,with_k_out,inter,normed", [(False, False, False, True), (False, True, True, False),
                                                            (True, False, True, True)])
def test_append_parts(with_q, with_k_out, inter, normed):
    run_append(37, 4, 2, 128, 16, False, 5, with_q, with_k_out, inter, normed)


def test_append_in_place_keys():
    T, K, D = 20, 2, 64
    k, v = draw(1, T, K, D), draw(2, T, K, D)
    kc, vc = make_cache(3, 16, K, D, False)
    slots = torch.arange(T, device=device())
    pos = slots + 5
    rope = rb.Rope.make(D)
    kept = k.clone()
    rb.svdq_kv_append(kc, vc, k, v, slots, pos, rope, k_out=k)
    check(k, kept, None, pos, rope, 0.0, "k in place")
    assert torch.equal(kc.view(-1, K, D)[:T], k)


def test_slots_outside_the_cache_are_recorded_and_write_nothing():
    T, K, D = 6, 2, 64
    k, v = draw(1, T, K, D), draw(2, T, K, D)
    kc, vc = make_cache(2, 8, K, D, False)
    k0, v0 = kc.clone(), vc.clone()
    slots = torch.tensor([3, 16, -1, 2 ** 40, 15, -(2 ** 50)], device=device())
    rb.svdq_kv_append(kc, vc, k, v, slots)
    assert rb.svdq_check_status() == rb.SVDQ_EINVAL
    assert rb.svdq_check_status() == rb.SVDQ_OK
    for cache, old, new in ((kc, k0, k), (vc, v0, v)):
        old = old.clone()
        old.view(-1, K, D)[3], old.view(-1, K, D)[15] = new[0], new[4]
        assert torch.equal(cache, old)


def test_append_wrong_arguments_raise():
    k = draw(1, 4, 2, 64)
    kc, vc = make_cache(2, 8, 2, 64, False)
    s = torch.arange(4, device=device())
    bad = [
        lambda: rb.svdq_kv_append(kc, vc[:1], k, k, s), lambda: rb.svdq_kv_append(kc.float(), vc.float(), k, k, s),
        lambda: rb.svdq_kv_append(kc, vc, k[:, :1], k, s), lambda: rb.svdq_kv_append(kc, vc, k, k[:3], s),
        lambda: rb.svdq_kv_append(kc, vc, k, k, s.int()), lambda: rb.svdq_kv_append(kc, vc, k, k, s[:3]),
        lambda: rb.svdq_kv_append(kc, vc, k.float(), k.float(), s), lambda: rb.svdq_kv_append(kc, vc, k, k, s, q_weight=k),
        lambda: rb.svdq_kv_append(kc, vc.transpose(1, 2).contiguous().transpose(1, 2), k, k, s),
        lambda: rb.svdq_kv_append(kc[:0], vc[:0], k, k, s), lambda: rb.svdq_kv_append(kc, vc, k, k, s, q=k[:, :0]),
        lambda: rb.svdq_kv_append(kc, vc, k, k, s.cpu()),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()


def test_nothing_to_append():
    kc, vc = make_cache(2, 8, 2, 64, False)
    e = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=device())
    out = rb.svdq_kv_append(kc, vc, e, e, torch.empty(0, dtype=torch.int64, device=device()), q=e)
    assert out.shape == (0, 2, 64)
    a, b = rb.svdq_qk_norm_rope(e, e)
    assert a.shape == b.shape == (0, 2, 64)
