"""The binding's two ways into the attention kernels - the quick calls and the checked Python
behind them - hand the library the same numbers."""

import ctypes
import math

import pytest
import torch

import rank_bit_residual_b200 as rb
import rank_bit_residual_b200.attention as rba
from rank_bit_residual_b200 import build as rbuild
from tests.gpu_util import device

pytestmark = pytest.mark.gpu

DIMS = range(8, 129, 8)


def draw(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(torch.bfloat16).to(device())


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device=device())


@pytest.fixture
def scales():
    """The scales that the quick calls hand to the library, which refuses the calls."""
    seen = []
    names = ("svdq_qk_norm_rope", "svdq_kv_append", "svdq_attention_prompt", "svdq_attention_prompt_workspace_size",
             "svdq_attention_decode", "svdq_attention_decode_workspace_size")

    def note(at):
        def call(*args):
            seen.append(args[at])
            return rb.SVDQ_EINVAL
        return call

    lib, quick = rb.load_library(), rba._quick()
    at = {"svdq_attention_prompt": 10, "svdq_attention_decode": 6}
    stand_in = {n: ctypes.CFUNCTYPE(ctypes.c_int32, *rb._SIGS[n][1])(note(at[n])) for n in at}
    quick.bind(*(ctypes.cast(stand_in.get(n, getattr(lib, n)), ctypes.c_void_p).value for n in names))
    yield seen
    quick.bind(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in names))


def test_the_quick_default_scale_is_the_rounded_one(scales):
    quick = rba._quick()
    for D in DIMS:
        q, kv = draw(1, 3, 2, D), draw(2, 3, 2, D)
        cache = draw(3, 1, 4, 2, D)
        assert quick.prompt(q, kv, kv, None, None, True, None, None) is None
        assert quick.decode(q[:1], cache, cache, ints([[0]]), ints([3]), None, None) is None
        want = ctypes.c_float(1.0 / math.sqrt(D)).value
        assert scales[-2:] == [want, want], D
    assert len(scales) == 2 * len(DIMS)


@pytest.mark.parametrize("D", [24, 64, 72, 96, 112])
def test_a_workspace_or_a_copy_changes_no_bit(D):
    """Scores in the hundreds, where a scale one step off shows."""
    T, H, K = 400, 4, 2
    q, k, v = draw(1, T, H, D) * 100, draw(2, T, K, D), draw(3, T, K, D)
    shifted = torch.empty(T * K * D + 1, dtype=torch.bfloat16, device=device())[1:].view(T, K, D)
    shifted.copy_(k)                         # not on a 16-byte boundary: the binding copies it
    quick = rb.svdq_attention_prompt(q, k, v)
    assert torch.equal(rb.svdq_attention_prompt(q, k, v, workspace=rb.LinearWorkspace()), quick)
    assert torch.equal(rb.svdq_attention_prompt(q, shifted, v), quick)
    assert torch.equal(rb.svdq_attention_prompt(q, k, v, scale=1.0 / math.sqrt(D)), quick)
    kc, vc = draw(4, 30, 16, K, D), draw(5, 30, 16, K, D)
    table, lens = ints([[30 - 1 - i for i in range(25)]] * 50), ints([400 - i for i in range(50)])
    dq = q[:50]
    quick = rb.svdq_attention_decode(dq, kc, vc, table, lens)
    shifted = torch.empty(50 * H * D + 1, dtype=torch.bfloat16, device=device())[1:].view(50, H, D)
    shifted.copy_(dq)
    assert torch.equal(rb.svdq_attention_decode(dq, kc, vc, table, lens, workspace=rb.LinearWorkspace()), quick)
    assert torch.equal(rb.svdq_attention_decode(shifted, kc, vc, table, lens), quick)
    assert torch.equal(rb.svdq_attention_decode(dq, kc, vc, table, lens, scale=1.0 / math.sqrt(D)), quick)
    assert rb.svdq_check_status() == rb.SVDQ_OK


def test_all_calls_without_the_quick_calls(monkeypatch, tmp_path):
    """The library alone is enough: the same bits, after a warning."""
    T, H, K, D = 40, 4, 2, 64
    row = draw(1, T, (H + 2 * K) * D)
    q, k, v = row.view(T, -1, D).split([H, K, K], 1)
    w, pos, rope = draw(2, D), torch.arange(T, device=device()), rb.Rope.make(D)

    def all_four():
        kc, vc = (torch.zeros((4, 16, K, D), dtype=torch.bfloat16, device=device()) for _ in range(2))
        a, b = rb.svdq_qk_norm_rope(q, k, pos, rope, w, w)
        c = rb.svdq_kv_append(kc, vc, k, v, pos, pos, rope, w, q=q, q_weight=w)
        o = rb.svdq_attention_prompt(a, b, v)
        d = rb.svdq_attention_decode(a[-1:], kc, vc, ints([[0, 1, 2]]), ints([T]))
        return a, b, c, kc, vc, o, d

    want = all_four()
    monkeypatch.setattr(rbuild, "calls_path", lambda: str(tmp_path / "none.so"))
    monkeypatch.setattr(rba, "_calls_lib", None)
    monkeypatch.setattr(rba, "_calls", None)
    with pytest.warns(RuntimeWarning, match="quick way"):
        got = all_four()
    assert rba._quick() is None
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    assert rb.svdq_check_status() == rb.SVDQ_OK
