"""svdq_attention_prompt and svdq_attention_decode against the float64 definition."""

import ctypes
import math

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


def ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=device())


def close(got, out, spread, reach, dim, keys, what):
    err = np.abs(f64(got) - out)
    tol = oa.attention_tolerance(out, spread, reach, dim, keys)
    assert np.all(err <= tol), f"{what}: {np.max(err / np.maximum(tol, 1e-300)):.3f} of the tolerance"


def run_prompt(q_lens, k_lens, H, K, D, causal, seed=0, scale=None, q_gain=1.0):
    Tq, Tk = sum(q_lens), sum(k_lens)
    q = draw(seed, Tq, H, D) * q_gain
    kv = draw(seed + 1, Tk, 2 * K * D)
    k, v = kv.view(Tk, 2, K, D).unbind(1)
    cu_q, cu_k = np.cumsum([0] + q_lens), np.cumsum([0] + k_lens)
    got = rb.svdq_attention_prompt(q, k, v, ints(cu_q), ints(cu_k), causal=causal, scale=scale)
    assert rb.svdq_check_status() == rb.SVDQ_OK
    sc = 1 / math.sqrt(D) if scale is None else scale
    out, spread, reach = oa.prompt(f64(q), f64(k), f64(v), cu_q, cu_k, sc, causal)
    close(got, out, spread, reach, D, max(k_lens + [1]), f"{q_lens} {k_lens}")
    return q, k, v, got


@pytest.mark.parametrize("q_lens,k_lens", [
    ([1], [1]), ([64], [64]), ([65], [65]), ([128], [128]), ([127], [129]), ([256], [256]), ([257], [257]),
    ([1, 2, 3], [1, 2, 3]), ([130, 1, 300, 63], [130, 1, 300, 63]), ([5], [700]), ([300], [7]), ([100, 40], [0, 40]),
    ([0, 33, 0, 129], [5, 33, 0, 140]), ([513], [1025]),
])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt(q_lens, k_lens, D, causal):
    run_prompt(q_lens, k_lens, 4, 2, D, causal, seed=len(q_lens) + D)


@pytest.mark.parametrize("D", [8, 24, 40, 72, 80, 96, 120])
def test_prompt_head_dims(D):
    run_prompt([150, 20], [150, 20], 2, 1, D, True, seed=D)


@pytest.mark.parametrize("H,K", [(1, 1), (8, 1), (5, 5), (12, 4), (32, 8)])
def test_prompt_head_groups(H, K):
    run_prompt([200], [333], H, K, 128, True, seed=H)


@pytest.mark.parametrize("H,K", [(4, 1), (6, 1), (16, 2), (16, 1), (32, 1), (64, 1), (48, 2)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_heads_side_by_side(H, K, D, causal):
    """Groups of every power of two (and with another factor), sequences that end inside a tile."""
    run_prompt([1, 31, 33, 0, 70, 9], [1, 40, 33, 5, 66, 130], H, K, D, causal, seed=H + K + D)


@pytest.mark.parametrize("H,K", [(4, 1), (32, 1)])
def test_prompt_heads_side_by_side_few_rows_many_keys(H, K):
    run_prompt([9, 3], [5000, 4100], H, K, 128, True, seed=H)
    run_prompt([70], [6000], H, K, 64, False, seed=H)


@pytest.mark.parametrize("H", [4, 8])
def test_prompt_heads_side_by_side_in_heads_major_tensors(H):
    """Strides of heads larger than those of tokens; rows around the sequences stay."""
    T, D = 90, 64
    q = draw(1, H, T, D).transpose(0, 1)
    k, v = draw(2, T, 1, D), draw(3, T, 1, D)
    out = torch.full((H, T, D), 7.0, dtype=torch.bfloat16, device=device()).transpose(0, 1)
    cu = [5, 20, 20, 77]
    rb.svdq_attention_prompt(q, k, v, ints(cu), ints(cu), out=out)
    want, spread, reach = oa.prompt(f64(q), f64(k), f64(v), cu, cu, 0.125, True)
    close(out[5:77], want[5:77], spread[5:77], reach, D, 57, "heads major")
    assert torch.all(out[:5] == 7) and torch.all(out[77:] == 7)


def test_prompt_heads_side_by_side_values_without_end():
    """A row and all its heads see the infinity at their own key and no later one."""
    T, H, D = 50, 8, 128
    q, k, v = draw(1, T, H, D), draw(2, T, 1, D), draw(3, T, 1, D)
    clean = rb.svdq_attention_prompt(q, k, v)
    v[20, 0, 3] = float("inf")
    v[30, 0, 5] = float("nan")
    got = rb.svdq_attention_prompt(q, k, v)
    assert torch.equal(got[:20], clean[:20])
    assert torch.isinf(got[20:30, :, 3]).all() and torch.isfinite(got[20:30, :, 4:]).all()
    assert torch.isnan(got[30:, :, 5]).all() and torch.isinf(got[30:, :, 3]).all()


@pytest.mark.parametrize("D", [8, 24, 64, 72, 120])
@pytest.mark.parametrize("T,K,H", [(150, 150, 2), (40, 9000, 4), (300, 300, 1)])
def test_prompt_values_without_end(T, K, H, D):
    """One infinity in V: its column is infinite for the rows that see it, all else is as without it."""
    q, k, v = draw(1, T, H, D), draw(2, K, 1, D), draw(3, K, 1, D)
    clean = rb.svdq_attention_prompt(q, k, v)
    first, col = T - 30, D - 3               # the first row that sees it
    v[K - T + first, 0, col] = float("-inf")
    got = rb.svdq_attention_prompt(q, k, v)
    assert torch.all(got[first:, :, col] == float("-inf"))
    got[first:, :, col] = clean[first:, :, col]
    assert torch.equal(got, clean)


def test_prompt_large_scores_and_scales():
    run_prompt([300], [300], 2, 2, 128, True, q_gain=8.0)          # scores up to hundreds: one key wins
    run_prompt([300], [300], 2, 2, 64, False, scale=0.0)           # the plain mean
    run_prompt([200], [200], 2, 1, 64, True, scale=-0.25)


def test_prompt_growing_scores():
    """Every tile of keys beats the one before, so that each renews the maximum."""
    T, D = 1024, 128
    q = torch.ones((T, 1, D), dtype=torch.bfloat16, device=device())
    k = (torch.arange(T, device=device())[:, None, None] / 64).expand(T, 1, D).to(torch.bfloat16)
    v = draw(3, T, 1, D)
    for causal in (True, False):
        got = rb.svdq_attention_prompt(q, k, v, causal=causal)
        out, spread, reach = oa.prompt(f64(q), f64(k), f64(v), [0, T], [0, T], D ** -0.5, causal)
        close(got, out, spread, reach, D, T, "growing")
        got = rb.svdq_attention_prompt(q, -k, v, causal=causal)
        out, spread, reach = oa.prompt(f64(q), f64(-k), f64(v), [0, T], [0, T], D ** -0.5, causal)
        close(got, out, spread, reach, D, T, "falling")


def test_prompt_long():
    run_prompt([2500, 700], [2500, 700], 2, 1, 128, True, seed=9)
    run_prompt([1500], [4000], 1, 1, 64, False, seed=10)


@pytest.mark.parametrize("q_lens,k_lens,H,K", [
    ([37], [5000], 4, 2), ([1], [9000], 3, 1), ([300], [7501], 6, 2), ([5, 130], [6000, 2500], 4, 4),
    ([200, 40], [0, 8200], 2, 2), ([2100], [2100], 1, 1),
])
@pytest.mark.parametrize("D", [64, 128, 80])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_few_rows_many_keys(q_lens, k_lens, H, K, D, causal):
    """The keys are divided among blocks and the shares joined."""
    n = ctypes.c_size_t()
    lib = rb.load_library()
    lib.svdq_attention_prompt_workspace_size(H, K, D, len(q_lens), sum(q_lens), sum(k_lens), ctypes.byref(n))
    assert n.value > 0
    q, k, v, got = run_prompt(q_lens, k_lens, H, K, D, causal, seed=H + D)
    cu_q, cu_k = ints(np.cumsum([0] + q_lens)), ints(np.cumsum([0] + k_lens))
    work = rb.LinearWorkspace()
    for _ in range(3):                           # the same bits, whatever the scratch holds
        again = rb.svdq_attention_prompt(q, k, v, cu_q, cu_k, causal=causal, workspace=work)
        assert torch.equal(again, got)
        work.buf.fill_(255)


def test_prompt_shares_nan_behind_the_mask():
    q, k, v = draw(1, 100, 2, 64), draw(2, 5000, 1, 64), draw(3, 5000, 1, 64)
    want = rb.svdq_attention_prompt(q, k, v)
    k2, v2 = k.clone(), v.clone()
    k2[4960:], v2[4960:] = float("inf"), float("nan")
    got = rb.svdq_attention_prompt(q, k2, v2)
    assert torch.equal(got[:60], want[:60]) and torch.isnan(got[60:]).all()


def test_prompt_projection_row_and_outputs():
    """Views of one projection row, a given output with a pitch, transposed inputs."""
    T, H, K, D = 301, 6, 2, 64
    row = draw(4, T, (H + 2 * K) * D)
    q, k, v = row.view(T, -1, D).split([H, K, K], 1)
    want = rb.svdq_attention_prompt(q.contiguous(), k.contiguous(), v.contiguous())
    assert torch.equal(rb.svdq_attention_prompt(q, k, v), want)
    wide = torch.full((T, H + 1, D), 7.0, dtype=torch.bfloat16, device=device())
    out = rb.svdq_attention_prompt(q, k, v, out=wide[:, :H])
    assert torch.equal(out, want) and torch.all(wide[:, H] == 7)
    hf = q.transpose(0, 1).contiguous().transpose(0, 1)            # heads first in memory
    assert torch.equal(rb.svdq_attention_prompt(hf, k, v), want)
    flat = torch.empty(T * K * D + 1, dtype=torch.bfloat16, device=device())
    off = flat[1:].view(T, K, D)
    off.copy_(k)                                                   # not on a 16-byte boundary
    assert torch.equal(rb.svdq_attention_prompt(q, off, v), want)


def test_prompt_rows_of_no_sequence_stay():
    q, k, v = draw(1, 200, 2, 64), draw(2, 200, 2, 64), draw(3, 200, 2, 64)
    out = torch.full_like(q, 5.0)
    cu = ints([10, 80, 80, 150])
    rb.svdq_attention_prompt(q, k, v, cu, cu, out=out)
    want, spread, reach = oa.prompt(f64(q), f64(k), f64(v), [10, 80, 80, 150], [10, 80, 80, 150], 0.125)
    close(out[10:150], want[10:150], spread[10:150], reach, 64, 70, "middle")
    assert torch.all(out[:10] == 5) and torch.all(out[150:] == 5)


def test_prompt_nan_outside_what_a_row_sees():
    """Infinities and NaN behind the mask, in other sequences and in rows of none."""
    T, D = 300, 128
    q, k, v = draw(1, T, 2, D), draw(2, T, 1, D), draw(3, T, 1, D)
    cu = ints([0, 130, 250])
    want = rb.svdq_attention_prompt(q, k, v, cu, cu)
    k2, v2, q2 = k.clone(), v.clone(), q.clone()
    for t in (k2, v2, q2):
        t[250:] = float("nan")
    k2[100:130] = float("inf")
    v2[100:130] = float("nan")
    got = rb.svdq_attention_prompt(q2, k2, v2, cu, cu)
    assert torch.equal(got[:100], want[:100]) and torch.equal(got[130:250], want[130:250])
    assert torch.isnan(got[129]).all()


def test_prompt_bad_lists_are_recorded():
    q, k, v = draw(1, 50, 2, 64), draw(2, 50, 1, 64), draw(3, 50, 1, 64)
    for cu in ([0, 60], [-3, 50], [0, 30, 20]):
        rb.svdq_attention_prompt(q, k, v, ints(cu), ints(cu))
        assert rb.svdq_check_status() == rb.SVDQ_EINVAL
    rb.svdq_attention_prompt(q, k, v, ints([0, 50]), ints([0, 51]))
    assert rb.svdq_check_status() == rb.SVDQ_EINVAL
    assert rb.svdq_check_status() == rb.SVDQ_OK


@pytest.mark.parametrize("place", [31, 32, 69])
def test_prompt_bad_lists_are_recorded_in_long_batches(place):
    cu = [2 * i for i in range(71)]
    q, k, v = draw(1, 140, 2, 64), draw(2, 140, 1, 64), draw(3, 140, 1, 64)
    good = rb.svdq_attention_prompt(q, k, v, ints(cu), ints(cu))
    assert rb.svdq_check_status() == rb.SVDQ_OK
    cu[place] += 3                           # beyond the next one
    for lists in ((cu, [2 * i for i in range(71)]), ([2 * i for i in range(71)], cu)):
        got = rb.svdq_attention_prompt(q, k, v, *map(ints, lists))
        assert rb.svdq_check_status() == rb.SVDQ_EINVAL
        assert torch.equal(got[:2 * place - 2], good[:2 * place - 2])


@pytest.mark.parametrize("lens", [[1, 700, 129, 0, 384, 385], [260] * 5, [1] * 31 + [2000], [0] * 40 + [300, 0, 9]])
@pytest.mark.parametrize("heads, kv_heads", [(4, 2), (3, 1)])
def test_prompt_every_range_of_every_sequence_has_its_turn(lens, heads, kv_heads):
    """One key per sequence: each row is a copy of its sequence's value."""
    n, total = len(lens), sum(lens)
    q, k, v = draw(1, total, heads, 64), draw(2, n, kv_heads, 64), draw(3, n, kv_heads, 64)
    cu = [sum(lens[:i]) for i in range(n + 1)]
    got = rb.svdq_attention_prompt(q, k, v, ints(cu), ints(range(n + 1)), causal=False)
    of = torch.repeat_interleave(torch.arange(n), torch.tensor(lens)).to(got.device)
    assert torch.equal(got, v[of].repeat_interleave(heads // kv_heads, 1))


def test_prompt_no_keys_and_no_rows():
    q = draw(1, 40, 2, 64)
    e = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=device())
    assert torch.all(rb.svdq_attention_prompt(q, e, e, causal=False) == 0)
    assert rb.svdq_attention_prompt(e, q, q).shape == (0, 2, 64)
    assert torch.all(rb.svdq_attention_prompt(q, q, q, ints([0, 40]), ints([7, 7])) == 0)


def test_prompt_many_sequences():
    """More sequences than a block has threads."""
    lens = [1 + (i * 7) % 5 for i in range(700)]
    run_prompt(lens, lens, 1, 1, 64, True, seed=12)


def test_prompt_wrong_arguments_raise():
    q = draw(1, 8, 4, 64)
    cu = ints([0, 8])
    bad = [lambda: rb.svdq_attention_prompt(q, q[:, :3], q[:, :3]), lambda: rb.svdq_attention_prompt(q, q, q[:7]),
           lambda: rb.svdq_attention_prompt(q.float(), q.float(), q.float()),
           lambda: rb.svdq_attention_prompt(q, q, q, cu.long(), cu), lambda: rb.svdq_attention_prompt(q, q, q, cu, ints([0, 4, 8])),
           lambda: rb.svdq_attention_prompt(q, q, q, ints([0, 4, 8])), lambda: rb.svdq_attention_prompt(q, q, q, out=q[:7]),
           lambda: rb.svdq_attention_prompt(q, q, q, scale=float("nan")), lambda: rb.svdq_attention_prompt(q, q, q, out=q),
           lambda: rb.svdq_attention_prompt(q, q.cpu(), q), lambda: rb.svdq_attention_prompt(q[0], q, q)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(rb.SvdqError):
        rb.svdq_attention_prompt(draw(1, 4, 1, 136), draw(1, 4, 1, 136), draw(1, 4, 1, 136))


# ------------------------------------------------------------------ decode
def make_paged(lens, K, D, page, seed=0, heads_first=False, spare=2):
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    shape = (pages, K, page, D) if heads_first else (pages, page, K, D)
    kc, vc = draw(seed, *shape), draw(seed + 1, *shape)
    if heads_first:
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    order = np.random.default_rng(seed).permutation(pages)
    table = np.full((len(lens), max(need + [1])), -1, np.int32)    # entries past the end are never read
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    return kc, vc, table


def run_decode(lens, H, K, D, page, seed=0, heads_first=False, scale=None, q_gain=1.0):
    kc, vc, table = make_paged(lens, K, D, page, seed, heads_first)
    q = draw(seed + 2, len(lens), H, D) * q_gain
    got = rb.svdq_attention_decode(q, kc, vc, ints(table), ints(lens), scale=scale)
    assert rb.svdq_check_status() == rb.SVDQ_OK
    out, spread, reach = oa.decode(f64(q), f64(kc), f64(vc), table, lens, 1 / math.sqrt(D) if scale is None else scale)
    close(got, out, spread, reach, D, max(lens + [1]), f"{lens[:8]}")
    return q, kc, vc, table, got


@pytest.mark.parametrize("lens", [[1], [15], [16], [17], [64], [1000], [5000], [0], [0, 3, 0, 129, 1],
                                  [700, 1, 64, 63, 65, 0, 2, 333]])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page,heads_first", [(16, False), (64, True), (7, False), (1, False)])
def test_decode(lens, D, page, heads_first):
    run_decode(lens, 8, 2, D, page, seed=len(lens) + D, heads_first=heads_first)


@pytest.mark.parametrize("D", [8, 24, 40, 72, 80, 96, 120])
def test_decode_head_dims(D):
    run_decode([100, 33], 4, 2, D, 16, seed=D)


@pytest.mark.parametrize("H,K", [(1, 1), (8, 1), (9, 1), (16, 1), (17, 1), (40, 1), (7, 7), (24, 3), (32, 8)])
def test_decode_head_groups(H, K):
    run_decode([300, 1, 77], H, K, 128, 16, seed=H)
    run_decode([300, 1, 77], H, K, 64, 16, seed=H)


def test_decode_scores_and_scales():
    run_decode([700, 40], 4, 2, 128, 16, q_gain=8.0)
    run_decode([700, 40], 4, 2, 64, 16, scale=0.0)
    run_decode([700, 40], 4, 2, 64, 16, scale=-0.25)


def test_decode_growing_scores():
    n, D, page = 4096, 128, 16
    kc = (torch.arange(n, device=device()).view(-1, page, 1, 1) / 256).expand(-1, page, 1, D).to(torch.bfloat16).contiguous()
    vc = draw(1, n // page, page, 1, D)
    table = np.arange(n // page, dtype=np.int32)[None]
    q = torch.ones((1, 4, D), dtype=torch.bfloat16, device=device())
    for sign in (1, -1):
        got = rb.svdq_attention_decode(sign * q, kc, vc, ints(table), ints([n]))
        out, spread, reach = oa.decode(f64(sign * q), f64(kc), f64(vc), table, [n], D ** -0.5)
        close(got, out, spread, reach, D, n, "growing")


def test_decode_many_sequences():
    rng = np.random.default_rng(0)
    run_decode([int(n) for n in rng.integers(0, 90, 600)], 2, 1, 64, 16, seed=4)


def test_decode_long_sequence_over_all_blocks():
    run_decode([40000], 4, 1, 64, 64, seed=5)


def test_decode_nan_behind_the_last_key():
    """Slots behind a sequence's end in its last page, and pages it does not name."""
    lens, page = [37, 100], 16
    kc, vc, table = make_paged(lens, 2, 128, page, seed=3)
    q = draw(9, 2, 8, 128)
    want = rb.svdq_attention_decode(q, kc, vc, ints(table), ints(lens))
    for s, n in enumerate(lens):
        kc[table[s, n // page], n % page:] = float("nan")
        vc[table[s, n // page], n % page:] = float("inf")
    used = set(table[table >= 0].tolist())
    for p in set(range(kc.shape[0])) - used:
        kc[p] = float("nan")
    assert torch.equal(rb.svdq_attention_decode(q, kc, vc, ints(table), ints(lens)), want)


def test_decode_nan_inside_reaches_the_row():
    kc, vc, table = make_paged([50, 50], 1, 64, 16, seed=3)
    kc[table[0, 1], 3] = float("nan")
    got = rb.svdq_attention_decode(draw(9, 2, 2, 64), kc, vc, ints(table), ints([50, 50]))
    assert torch.isnan(got[0]).all() and not torch.isnan(got[1]).any()


def test_decode_bad_pages_and_lengths_are_recorded():
    lens = [40, 40]
    kc, vc, table = make_paged(lens, 2, 64, 16, seed=1)
    q = draw(2, 2, 4, 64)
    good = rb.svdq_attention_decode(q, kc, vc, ints(table), ints(lens))
    for page in (-1, kc.shape[0], 2 ** 31 - 1):
        bad = table.copy()
        bad[0, 1] = page
        got = rb.svdq_attention_decode(q, kc, vc, ints(bad), ints(lens))
        assert rb.svdq_check_status() == rb.SVDQ_EINVAL
        assert torch.equal(got[1], good[1])
        # the page's keys are left out
        rest = [t for t in range(40) if t // 16 != 1]
        k = np.stack([f64(kc)[table[0, t // 16], t % 16] for t in rest])
        v = np.stack([f64(vc)[table[0, t // 16], t % 16] for t in rest])
        for h in range(4):
            o, sp, r = oa.attend(f64(q)[0, h][None], k[:, h // 2], v[:, h // 2], 0.125)
            close(got[0, h][None], o, sp, r, 64, 40, "left out")
    for bad_len, same in ((-5, 0), (49, 48), (2 ** 31 - 1, 48)):
        kc2, vc2, table2 = make_paged([48, 40], 2, 64, 16, seed=1)
        got = rb.svdq_attention_decode(q, kc2, vc2, ints(table2), ints([bad_len, 40]))
        assert rb.svdq_check_status() == rb.SVDQ_EINVAL
        assert torch.equal(got, rb.svdq_attention_decode(q, kc2, vc2, ints(table2), ints([same, 40])))
    assert rb.svdq_check_status() == rb.SVDQ_OK


def test_decode_shared_pages_and_repeats():
    """Two sequences over the same pages; the same call gives the same bits."""
    kc, vc, table = make_paged([3000], 2, 128, 16, seed=6)
    both = np.concatenate([table, table])
    q = draw(1, 1, 8, 128).expand(2, 8, 128).contiguous()
    first = rb.svdq_attention_decode(q, kc, vc, ints(both), ints([3000, 3000]))
    work = rb.LinearWorkspace()
    for _ in range(5):
        assert torch.equal(rb.svdq_attention_decode(q, kc, vc, ints(both), ints([3000, 3000]), workspace=work), first)


def test_decode_far_offsets():
    """Cache offsets that pass 2^31 elements."""
    K, D, page = 1, 128, 64
    pages = (2 ** 31) // (page * K * D) + 4
    kc = torch.zeros((pages, page, K, D), dtype=torch.bfloat16, device=device())
    vc = torch.zeros_like(kc)
    table = np.array([[pages - 1, 0, pages - 3]], np.int32)
    n = 2 * page + 9
    small = draw(1, 3, page, K, D), draw(2, 3, page, K, D)
    for i, p in enumerate(table[0]):
        kc[int(p)], vc[int(p)] = small[0][i], small[1][i]
    q = draw(3, 1, 4, D)
    got = rb.svdq_attention_decode(q, kc, vc, ints(table), ints([n]))
    want = rb.svdq_attention_decode(q, small[0], small[1], ints([[0, 1, 2]]), ints([n]))
    assert torch.equal(got, want)
    # and the append reaches them
    t = draw(4, 1, K, D)
    rb.svdq_kv_append(kc, vc, t, t, ints([pages * page - 1], torch.int64))
    assert torch.equal(kc[pages - 1, page - 1], t[0]) and rb.svdq_check_status() == rb.SVDQ_OK


def test_decode_strided_rows():
    kc, vc, table = make_paged([90, 20], 2, 64, 16)
    wide = draw(1, 2, 12, 64)
    q = wide[:, 4:8]
    out = torch.full((2, 6, 64), 3.0, dtype=torch.bfloat16, device=device())
    rb.svdq_attention_decode(q, kc, vc, ints(table), ints([90, 20]), out=out[:, 1:5])
    want = rb.svdq_attention_decode(q.contiguous(), kc, vc, ints(table), ints([90, 20]))
    assert torch.equal(out[:, 1:5], want) and torch.all(out[:, 0] == 3) and torch.all(out[:, 5] == 3)


def test_decode_wrong_arguments_raise():
    kc, vc, table = make_paged([20], 2, 64, 16)
    q, t, n = draw(1, 1, 4, 64), ints(table), ints([20])
    bad = [lambda: rb.svdq_attention_decode(q[:, :3], kc, vc, t, n), lambda: rb.svdq_attention_decode(q, kc, vc[:1], t, n),
           lambda: rb.svdq_attention_decode(q.float(), kc, vc, t, n), lambda: rb.svdq_attention_decode(q, kc, vc, t.long(), n),
           lambda: rb.svdq_attention_decode(q, kc, vc, t, n.long()), lambda: rb.svdq_attention_decode(q, kc, vc, t[0], n),
           lambda: rb.svdq_attention_decode(q, kc, vc, t, ints([1, 2])), lambda: rb.svdq_attention_decode(q, kc, vc, t, n, out=q),
           lambda: rb.svdq_attention_decode(q, kc, vc, t.cpu(), n), lambda: rb.svdq_attention_decode(q[:, :, :32], kc, vc, t, n)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
