"""Every key counts once: with q = 0 all weights are equal, and a value that is the number of
keys at one key and zero at all others comes out as 1 if that key was counted, and as 0
(or 2) if not. A column of the head takes one key, so that a call tries 64 or 128 of them. (With
random values one key among thousands is far inside the rounding of the result.)

The value is rounded to bf16 (2^-8 of it) and so is the result: 1 comes out between
1 - 2^-6 and 1 + 2^-6."""

import numpy as np
import pytest
import torch

import rank_bit_residual_b200 as rb
from tests.gpu_util import device

pytestmark = pytest.mark.gpu

ONE = 2.0 ** -6


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device=device())


@pytest.mark.parametrize("lens", [[40000], [5000, 1, 0, 777, 16, 12345], [64, 4097] * 9])
@pytest.mark.parametrize("H,K,D,page", [(4, 1, 64, 64), (16, 8, 64, 16), (12, 4, 128, 16), (40, 2, 128, 7)])
def test_decode_counts_every_key_once(lens, H, K, D, page):
    need = [-(-n // page) for n in lens]
    order = np.random.default_rng(0).permutation(sum(need) + 1)
    table = np.zeros((len(lens), max(need)), np.int32)
    for s, n in enumerate(need):
        table[s, :n] = order[sum(need[:s]):sum(need[:s]) + n]
    kc = torch.randn((len(order), page, K, D), device=device()).to(torch.bfloat16)
    vc = torch.zeros_like(kc)
    q = torch.zeros((len(lens), H, D), dtype=torch.bfloat16, device=device())
    pages, length = ints(table), ints(lens)
    column = torch.arange(D, device=device())
    wrong = []
    for first in range(0, max(lens), D):
        vc.zero_()
        key = first + column
        want = torch.zeros((len(lens), 1, D), device=device())
        for s, n in enumerate(lens):
            on = key < n
            vc[pages[s, key[on] // page].long(), key[on] % page, :, column[on]] = float(n)
            want[s, 0, on] = 1.0
        got = rb.svdq_attention_decode(q, kc, vc, pages, length).float()
        if not torch.all((got - want).abs() <= ONE * want):
            wrong.append(first)
    assert not wrong and rb.svdq_check_status() == rb.SVDQ_OK


# one share; the shares of few rows over many keys; several sequences; all tiles with heads side by side
@pytest.mark.parametrize("q_lens,k_lens,H,K", [
    ([300], [2000], 2, 1), ([301], [7501], 6, 2), ([1], [9000], 3, 1), ([5, 130, 0, 64], [6000, 2500, 7, 1], 4, 4),
    ([37], [5000], 32, 1), ([700], [700], 8, 2),
])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_counts_every_key_once(q_lens, k_lens, H, K, D, causal):
    cu_q, cu_k = np.cumsum([0] + q_lens), np.cumsum([0] + k_lens)
    q = torch.zeros((sum(q_lens), H, D), dtype=torch.bfloat16, device=device())
    k = torch.randn((sum(k_lens), K, D), device=device()).to(torch.bfloat16)
    v = torch.zeros_like(k)
    lists = ints(cu_q), ints(cu_k)
    column = torch.arange(D, device=device())
    wrong = []
    for first in range(0, max(k_lens), D):
        v.zero_()
        key = first + column
        want = torch.zeros((sum(q_lens), 1, D), device=device())
        for s, (n, m) in enumerate(zip(q_lens, k_lens)):
            on = key < m
            v[cu_k[s] + key[on], :, column[on]] = float(m)
            rows = torch.arange(n, device=device())
            seen = m - n + 1 + rows if causal else torch.full_like(rows, m)
            want[cu_q[s]:cu_q[s + 1], 0] = torch.where(on & (key < seen[:, None]), m / seen.clamp(min=1)[:, None], 0.0)
        got = rb.svdq_attention_prompt(q, k, v, *lists, causal=causal).float()
        if not torch.all((got - want).abs() <= ONE * want):
            wrong.append(first)
    assert not wrong and rb.svdq_check_status() == rb.SVDQ_OK
