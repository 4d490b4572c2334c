"""Prompt attention: what lies outside a sequence - the rows packed behind it, the rows of no
sequence - changes no bit of the rows inside."""

import pytest
import torch

import rank_bit_residual_b200 as rb
from tests.gpu_util import device

pytestmark = pytest.mark.gpu


def draw(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(torch.bfloat16).to(device())


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device=device())


# 1000 keys are one block's work, 9000 are divided among several and joined
@pytest.mark.parametrize("keys", [1000, 9000])
@pytest.mark.parametrize("H,K", [(2, 2), (4, 1)])
@pytest.mark.parametrize("D", [64, 72, 128])
@pytest.mark.parametrize("causal", [False, True])
def test_rows_behind_a_sequence_change_no_bit_of_it(keys, H, K, D, causal):
    n, more = 100, 150                       # the sequence ends inside a warp's 32 rows
    q, k, v = draw(1, n + more, H, D), draw(2, keys + more, K, D), draw(3, keys + more, K, D)
    for lists in (([0, n], [0, keys]), ([0, n, n + more], [0, keys, keys + more])):
        cu_q, cu_k = map(ints, lists)
        want = rb.svdq_attention_prompt(q, k, v, cu_q, cu_k, causal=causal)
        for fill in (float("nan"), float("inf"), 1e30, 8.0, 0.0, None):
            other = q.clone()
            if fill is None:
                other[n:] *= 4               # scores that pass each row's maximum now and then
            else:
                other[n:] = fill
            got = rb.svdq_attention_prompt(other, k, v, cu_q, cu_k, causal=causal)
            assert torch.equal(got[:n], want[:n]), (lists, fill)
    assert rb.svdq_check_status() == rb.SVDQ_OK


@pytest.mark.parametrize("D", [64, 128])
def test_a_sequence_has_the_same_bits_in_every_batch(D):
    """Alone, first, last and in the middle, with neighbours of any kind."""
    n, keys, H = 77, 900, 2
    q, k, v = draw(1, n, H, D), draw(2, keys, H, D), draw(3, keys, H, D)
    want = rb.svdq_attention_prompt(q, k, v, causal=False)
    for front, behind in ((0, 5), (13, 0), (300, 41)):
        Q = torch.cat([draw(4, front, H, D) * 9, q, draw(5, behind, H, D) * 9])
        KV = [torch.cat([draw(6, front, H, D), t, draw(7, behind, H, D)]) for t in (k, v)]
        cu_q = ints([0, front, front + n, front + n + behind])
        cu_k = ints([0, front, front + keys, front + keys + behind])
        got = rb.svdq_attention_prompt(Q, *KV, cu_q, cu_k, causal=False)
        assert torch.equal(got[front:front + n], want), (front, behind)
    assert rb.svdq_check_status() == rb.SVDQ_OK
