"""The attention operators together, as a layer uses them: through svdq_linear_chain, with a
cache filled by a prompt and read by decode steps, in CUDA graphs and on side streams."""

import numpy as np
import pytest
import torch

import rank_bit_residual_b200 as rb
import rank_bit_residual_b200.attention as rba
from oracle import attention as oa
from tests.gpu_util import SyntheticWeight, device

pytestmark = pytest.mark.gpu

H, K, D, PAGE = 8, 2, 64, 16
M = H * D


def draw(seed, *shape, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).to(device())


def f64(t):
    return t.detach().double().cpu().numpy()


def ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=device())


def weights():
    return SyntheticWeight(M, (H + 2 * K) * D, 16, "int4", seed=1).w, SyntheticWeight(M, M, 16, "int4", seed=2).w


def settings():
    return dict(heads=H, kv_heads=K, head_dim=D, rope=rb.Rope.make(D), q_weight=draw(3, D).abs() + 0.5,
                k_weight=draw(4, D).abs() + 0.5)


def paged(pages=40):
    return torch.zeros((pages, PAGE, K, D), dtype=torch.bfloat16, device=device()), \
        torch.zeros((pages, PAGE, K, D), dtype=torch.bfloat16, device=device())


def slots_of(table, seq, first, n):
    t = np.arange(first, first + n)
    return table[seq, t // PAGE].astype(np.int64) * PAGE + t % PAGE


def oracle_layer(qkv, positions, st, cu):
    """Norm, rotation (rounded to bf16 as stored) and attention of one projection row."""
    x = f64(qkv).reshape(qkv.shape[0], -1, D)
    turn = lambda t, w: torch.from_numpy(oa.rotate(oa.norm(t, f64(w)), positions, f64(st["rope"].turns))[0]).bfloat16().double().numpy()  # noqa: E731
    q, k, v = turn(x[:, :H], st["q_weight"]), turn(x[:, H:H + K], st["k_weight"]), x[:, H + K:]
    return (q, k, v) + oa.prompt(q, k, v, cu, cu, D ** -0.5)


def test_chain_with_a_step_equals_separate_calls_and_the_definition():
    wq, wo = weights()
    T = 150
    x, st, pos = draw(5, T, M), settings(), torch.arange(T, device=device())
    cu = ints([0, 100, 140])
    step = rb.AttentionStep(positions=pos, cu_seqlens=cu, **st)
    got = rb.svdq_linear_chain([wq, step, wo], x)
    assert rb.svdq_check_status() == rb.SVDQ_OK
    qkv = rb.svdq_linear(wq, x)
    _, _, _, out, spread, reach = oracle_layer(qkv, pos.cpu().numpy(), st, [0, 100, 140])
    q, k, v = qkv.view(T, -1, D).split([H, K, K], 1)
    q, k = rb.svdq_qk_norm_rope(q, k, pos, st["rope"], st["q_weight"], st["k_weight"])
    o = torch.zeros((T, H, D), dtype=torch.bfloat16, device=device())
    rb.svdq_attention_prompt(q, k, v, cu, cu, out=o)
    assert torch.equal(got, rb.svdq_linear(wo, o.view(T, M)))
    assert torch.equal(got, rb.svdq_linear_chain([wq, step, wo], x, pdl=False))
    # The definition: q and k there are rounded to bf16 from float64 and here from fp32, so
    # single elements may differ by one step (2^-7 of the value): a score by 2 * 2^-7 of its
    # reach at the very most, and p by that, once in p and once in the total.
    err = np.abs(f64(o)[:140] - out[:140])
    tol = oa.attention_tolerance(out, spread, reach, D, 100)[:140] + 2 * 2 * 2.0 ** -7 * reach * spread[:140]
    assert np.all(err <= tol)
    assert np.sqrt(np.mean(err ** 2)) <= 2.0 ** -8 * np.sqrt(np.mean(spread[:140] ** 2))
    assert torch.all(o[140:] == 0)


@pytest.mark.parametrize("fmt", ["int4", "nvfp4"])
def test_prompt_then_decode_steps_over_the_cache(fmt):
    """A prompt fills the cache, decode steps extend it; each step's row equals the row that
    attention over the whole text gives."""
    wq = SyntheticWeight(M, (H + 2 * K) * D, 16, fmt, seed=1).w
    st = settings()
    lens, steps = [45, 1, 16], 4
    table = np.random.default_rng(0).permutation(40)[:3 * 6].reshape(3, 6).astype(np.int32)
    kc, vc = paged()
    texts = [draw(10 + s, n + steps, M) for s, n in enumerate(lens)]
    cu = np.cumsum([0] + lens)
    pos = ints(np.concatenate([np.arange(n) for n in lens]), torch.int64)
    slots = ints(np.concatenate([slots_of(table, s, 0, n) for s, n in enumerate(lens)]), torch.int64)
    rows = torch.cat([t[:n] for t, n in zip(texts, lens)])
    qkv_rows = [rb.svdq_linear(wq, rows)]
    prompt = rb.AttentionStep(positions=pos, cu_seqlens=ints(cu), k_cache=kc, v_cache=vc, slots=slots, **st)
    outs = [prompt(qkv_rows[0].clone())]
    for i in range(steps):
        x = torch.stack([t[n + i] for t, n in zip(texts, lens)])
        qkv_rows.append(rb.svdq_linear(wq, x))
        step = rb.AttentionStep(
            positions=ints([n + i for n in lens], torch.int64), k_cache=kc, v_cache=vc,
            slots=ints(np.concatenate([slots_of(table, s, n + i, 1) for s, n in enumerate(lens)]), torch.int64),
            page_table=ints(table), kv_len=ints([n + i + 1 for n in lens]), **st)
        outs.append(step(qkv_rows[-1].clone()))
    assert rb.svdq_check_status() == rb.SVDQ_OK
    for s, n in enumerate(lens):
        qkv = torch.cat([qkv_rows[0][cu[s]:cu[s + 1]]] + [r[s:s + 1] for r in qkv_rows[1:]])
        got = torch.cat([outs[0][cu[s]:cu[s + 1]]] + [o[s:s + 1] for o in outs[1:]]).view(n + steps, H, D)
        _, _, _, out, spread, reach = oracle_layer(qkv, np.arange(n + steps), st, [0, n + steps])
        err = np.abs(f64(got) - out)
        tol = oa.attention_tolerance(out, spread, reach, D, n + steps) + 2 * 2 * 2.0 ** -7 * reach * spread
        assert np.all(err <= tol)
        # a wrong page, position or head would be off by the size of the values themselves
        assert np.sqrt(np.mean(err ** 2)) <= 2.0 ** -8 * np.sqrt(np.mean(spread ** 2))


def test_decode_steps_in_a_graph():
    """One captured decode step, replayed while the lengths, slots and positions move on."""
    wq, wo = weights()
    st = settings()
    B, steps = 3, 5
    table = np.arange(B * 4, dtype=np.int32).reshape(B, 4)
    first = [20, 0, 15]
    caches = [paged(), paged()]
    for kc, vc in caches:
        kc.copy_(draw(1, *kc.shape)), vc.copy_(draw(2, *vc.shape))
    x = torch.empty((B, M), dtype=torch.bfloat16, device=device())
    pos, slots, lens = (torch.zeros(B, dtype=t, device=device()) for t in (torch.int64, torch.int64, torch.int32))

    def load(i):
        x.copy_(draw(50 + i, B, M))
        pos.copy_(ints([n + i for n in first], torch.int64))
        slots.copy_(ints(np.concatenate([slots_of(table, s, n + i, 1) for s, n in enumerate(first)]), torch.int64))
        lens.copy_(ints([n + i + 1 for n in first]))

    def chain(cache):
        step = rb.AttentionStep(positions=pos, k_cache=cache[0], v_cache=cache[1], slots=slots, page_table=ints(table),
                                kv_len=lens, **st)
        work = rb.LinearWorkspace()
        return lambda: rb.svdq_linear_chain([wq, step, wo], x, workspace=work)

    eager, captured = chain(caches[0]), chain(caches[1])
    want = []
    for i in range(steps):
        load(i)
        want.append(eager().clone())
    load(0)
    slots.fill_(-1)
    captured()                                   # sizes the workspace; nothing is appended
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = captured()
    for i in range(steps):
        load(i)
        g.replay()
        assert torch.equal(y, want[i]), i
    assert rb.svdq_check_status() == rb.SVDQ_OK
    assert torch.equal(caches[0][0], caches[1][0]) and torch.equal(caches[0][1], caches[1][1])


def test_the_quick_and_the_long_way_agree():
    """The binding's quick calls and the checked ones behind them, on the same arguments."""
    T = 40
    row = draw(1, T, (H + 2 * K) * D)
    q, k, v = row.view(T, -1, D).split([H, K, K], 1)
    pos, st = torch.arange(T, device=device()), settings()
    args = (pos, st["rope"], st["q_weight"], st["k_weight"], 1e-6)
    quick, calls = rba._quick(), []

    class Spy:
        def __getattr__(self, name):
            def call(*a):
                calls.append((name, getattr(quick, name)(*a)))
                return calls[-1][1]
            return call

    saved = rba._calls
    rba._calls = Spy()
    try:
        a = rb.svdq_qk_norm_rope(q, k, *args)
        kc, vc = paged(4)
        slots = torch.arange(T, device=device())
        qa = rb.svdq_kv_append(kc, vc, k, v, slots, pos, st["rope"], st["k_weight"], q=q, q_weight=st["q_weight"])
        cu = ints([0, 13, T])
        o = rb.svdq_attention_prompt(a[0], a[1], v, cu, cu)
        table, lens = ints([[0, 1, 2]]), ints([T])
        d = rb.svdq_attention_decode(a[0][:1], kc, vc, table, lens)
    finally:
        rba._calls = saved
    assert [n for n, _ in calls] == ["norm_rope", "append", "prompt", "decode"]
    assert all(r is not None for _, r in calls)                 # none of them was sent the long way
    b = rba._qk_norm_rope(q, k, *args, None, None)
    kc2, vc2 = paged(4)
    qb = rba._kv_append(kc2, vc2, k, v, slots, pos, st["rope"], st["k_weight"], 1e-6, q, st["q_weight"], None, None)
    ob = rba._attention_prompt(a[0], a[1], v, cu, cu, True, None, None, None)
    db = rba._attention_decode(a[0][:1], kc2, vc2, table, lens, None, None, None)
    for x, y in ((a[0], b[0]), (a[1], b[1]), (qa, qb), (kc, kc2), (vc, vc2), (o, ob), (d, db)):
        assert torch.equal(x, y) and x.stride() == y.stride()


def test_quick_calls_send_the_unusual_on():
    """What needs a copy or a message is not taken, and nothing is launched for it."""
    quick = rba._quick()
    q, k = draw(1, 4, H, D), draw(2, 4, K, D)
    pos, turns = torch.arange(4, device=device()), rb.Rope.make(D).turns
    usual = dict(q=q, k=k, positions=pos, turns=turns, inter=False, amp=1.0, qw=None, kw=None, eps=1e-6, qo=None, ko=None)
    assert quick.norm_rope(*usual.values()) is not None
    flat = torch.empty(4 * H * D + 1, dtype=torch.bfloat16, device=device())
    for change in (dict(q=q.half()), dict(q=q.float()), dict(q=q.cpu()), dict(q=q[0]), dict(q=flat[1:].view(4, H, D)),
                   dict(q=q[:, :, ::2]), dict(k=k[:3]), dict(positions=None), dict(positions=pos.int()),
                   dict(positions=pos[:3]), dict(turns=turns.float()), dict(turns=torch.cat([turns, turns])),
                   dict(amp="x"), dict(eps=None), dict(eps=-1.0), dict(qw=draw(3, 8)), dict(qw=draw(3, D).half()),
                   dict(qw=draw(3, D), kw=draw(3, D).float()), dict(qo=k), dict(ko=k.float()), dict(q=None), dict(q=1),
                   dict(q=q[:0], k=k[:0], positions=pos[:0]), dict(q=q[:, :0])):
        assert quick.norm_rope(*{**usual, **change}.values()) is None, change
    assert quick.norm_rope(q, k) is None and quick.decode(q) is None
    assert rb.svdq_check_status() == rb.SVDQ_OK


def test_captured_behind_a_memset_a_copy_and_two_streams():
    """The kernels start behind the work before them: also where that is no kernel, or is
    on two streams."""
    T = 64
    src = draw(1, T, (H + 2 * K) * D)
    row = torch.zeros_like(src)
    q, k, v = row.view(T, -1, D).split([H, K, K], 1)
    pos = torch.arange(T, device=device())
    rope = rb.Rope.make(D)
    kc, vc = paged(8)
    table, lens = ints([[0, 1, 2, 3]]), ints([T])

    def work():
        a, b = rb.svdq_qk_norm_rope(q, k, pos, rope)
        rb.svdq_kv_append(kc, vc, b, v, pos, q=a, k_out=b)
        return rb.svdq_attention_prompt(a, b, v), rb.svdq_attention_decode(a[-1:], kc, vc, table, lens)

    row.copy_(src)
    want = [t.clone() for t in work()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for kind in ("copy", "memset", "streams"):
        row.zero_(), kc.zero_(), vc.zero_()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            if kind == "streams":
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(side):
                    row[T // 2:].copy_(src[T // 2:])
                row[:T // 2].copy_(src[:T // 2])
                torch.cuda.current_stream().wait_stream(side)
            else:
                row.copy_(src)
                if kind == "memset":
                    kc.zero_()
            got = work()
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y), kind
    assert rb.svdq_check_status() == rb.SVDQ_OK


def test_calls_of_two_threads():
    """Two host threads, each on its own stream."""
    import threading
    kc, vc = draw(1, 300, PAGE, K, D), draw(2, 300, PAGE, K, D)
    table, lens = ints(np.arange(300, dtype=np.int32).reshape(2, 150)), ints([2400, 2001])
    qs = [draw(3, 2, H, D), draw(4, 2, H, D)]
    row = draw(5, 300, (H + 2 * K) * D)
    pq, pk, pv = row.view(300, -1, D).split([H, K, K], 1)
    want = [rb.svdq_attention_decode(q, kc, vc, table, lens) for q in qs]
    prompt = rb.svdq_attention_prompt(pq, pk, pv)
    torch.cuda.synchronize()
    bad = []

    def run(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                if not torch.equal(rb.svdq_attention_decode(qs[i], kc, vc, table, lens), want[i]):
                    bad.append(("decode", i))
                if not torch.equal(rb.svdq_attention_prompt(pq, pk, pv), prompt):
                    bad.append(("prompt", i))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad and rb.svdq_check_status() == rb.SVDQ_OK


def test_two_graphs_replayed_on_two_streams():
    """Each captured decode call has its own scratch: replays may overlap."""
    kc, vc = draw(1, 600, PAGE, K, D), draw(2, 600, PAGE, K, D)
    table = ints(np.arange(600, dtype=np.int32).reshape(2, 300))
    lens = ints([4799, 4001])
    qs = [draw(3, 2, H, D), draw(4, 2, H, D)]
    want = [rb.svdq_attention_decode(q, kc, vc, table, lens) for q in qs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for q in qs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(rb.svdq_attention_decode(q, kc, vc, table, lens))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_calls_on_a_side_stream():
    T = 64
    q, k, v = draw(1, T, H, D), draw(2, T, K, D), draw(3, T, K, D)
    pos = torch.arange(T, device=device())
    rope = rb.Rope.make(D)
    want = rb.svdq_attention_prompt(*rb.svdq_qk_norm_rope(q, k, pos, rope), v)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(2000000)               # the inputs below are made behind this
        q2, k2, v2 = q * 1, k * 1, v * 1
        got = rb.svdq_attention_prompt(*rb.svdq_qk_norm_rope(q2, k2, pos, rope), v2)
    s.synchronize()
    assert torch.equal(got, want)


def test_prompt_in_a_graph():
    T = 300
    row = draw(1, T, (H + 2 * K) * D)
    q, k, v = row.view(T, -1, D).split([H, K, K], 1)
    cu = ints([0, 100, 300])
    rb.svdq_attention_prompt(q, k, v, cu, cu)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = rb.svdq_attention_prompt(q, k, v, cu, cu)
    row.copy_(draw(2, T, (H + 2 * K) * D))
    cu.copy_(ints([0, 37, 300]))                 # the lengths are read when the graph runs
    g.replay()
    assert torch.equal(out, rb.svdq_attention_prompt(q, k, v, cu, cu))
