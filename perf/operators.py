"""Cases of the attention operators between two quantised linears, and their plain forms.

A transformer layer whose projections are svdq_linear calls has four steps between
the qkv projection and the output projection:

  norm_rope  an RMS norm of every query and key head and the rotation by position
  append     the same for a step that keeps a paged cache: keys (normed, rotated) and
             values go to their slots, queries come back
  prompt     attention over packed sequences, causal or full, with grouped heads
  decode     attention of one new token per sequence over the paged cache

The heads are views of one projection row [q | k | v], as svdq_linear writes it.
`run` computes a case in elementary torch operations in 32 bits (angles in 64), or,
with `own`, through this framework's calls. `exact` is the definition in 64 bits.
"""

import math
import random

import torch

own = False

NORM_EPS = 1e-6


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one prompt of 8192 tokens, 32 query and 8 key heads: the pass between projection and attention
        dict(name="norm_rope_prompt", op="norm_rope", tokens=8192, heads=32, kv_heads=8, head_dim=128, rot_dim=128,
             interleaved=False, norm=True, dtype="bf16", scaled=False, first=0),
        # image tokens in fp32 between bf16 layers: interleaved pairs, part of the head turned, odd count
        dict(name="norm_rope_partial_f32", op="norm_rope", tokens=1237, heads=16, kv_heads=16, head_dim=64, rot_dim=32,
             interleaved=True, norm=True, dtype="f32", scaled=False, first=0),
        # one decode step of 16 sequences far into a scaled context: latency
        dict(name="append_step", op="append", tokens=16, heads=32, kv_heads=8, head_dim=128, rot_dim=128,
             interleaved=False, norm=True, dtype="bf16", scaled=True, first=100000, page=16, pages=256, padded=0),
        # a padded batch of prompts written to the cache; every fifteenth row is padding
        dict(name="append_prompt", op="append", tokens=6007, heads=32, kv_heads=8, head_dim=128, rot_dim=128,
             interleaved=False, norm=False, dtype="bf16", scaled=False, first=0, page=64, pages=128, padded=15),
        # a prompt of one sequence, the longest here: compute bound
        dict(name="prompt_long", op="prompt", batch=1, q_len=8192, k_len=8192, ragged=False, causal=True, heads=32,
             kv_heads=8, head_dim=128, lens_seed=1),
        # prompts of different lengths packed into one batch, down to one token
        dict(name="prompt_ragged", op="prompt", batch=9, q_len=1700, k_len=1700, ragged=True, causal=True, heads=32,
             kv_heads=8, head_dim=128, lens_seed=2),
        # image tokens that all see one another (no causal order), narrow heads
        dict(name="prompt_full_64", op="prompt", batch=2, q_len=2048, k_len=2048, ragged=False, causal=False, heads=32,
             kv_heads=32, head_dim=64, lens_seed=3),
        # the last part of a prompt whose keys are there already: few rows, many keys
        dict(name="prompt_tail", op="prompt", batch=1, q_len=301, k_len=7501, ragged=False, causal=True, heads=32,
             kv_heads=8, head_dim=128, lens_seed=4),
        # one sequence, one token: latency of a long cache
        dict(name="decode_single", op="decode", batch=1, k_len=8191, ragged=False, heads=32, kv_heads=8, head_dim=128,
             page=16, lens_seed=5),
        # a serving batch of sequences of all lengths: memory bound
        dict(name="decode_batch", op="decode", batch=128, k_len=6000, ragged=True, heads=32, kv_heads=8, head_dim=128,
             page=16, lens_seed=6),
        # long contexts, every query head with its own key head, larger pages
        dict(name="decode_long_64", op="decode", batch=8, k_len=30001, ragged=False, heads=32, kv_heads=32, head_dim=64,
             page=64, lens_seed=7),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "prompt", "decode"])
    head_dim = rng.choice([64, 96, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([g for g in (1, 2, 4, 5, 8) if g * kv_heads <= 32])
    case = dict(op=op, heads=heads, kv_heads=kv_heads, head_dim=head_dim)
    if op in ("norm_rope", "append"):
        case.update(tokens=_log_uniform(rng, 1, 8192), rot_dim=rng.choice([head_dim, head_dim, head_dim // 2, 16]),
                    interleaved=rng.random() < 0.4, norm=rng.random() < 0.7,
                    dtype="f32" if op == "norm_rope" and rng.random() < 0.3 else "bf16", scaled=rng.random() < 0.3,
                    first=rng.choice([0, _log_uniform(rng, 1, 1000000)]))
    if op == "append":
        page = rng.choice([16, 32, 64])
        case.update(page=page, pages=2 + 2 * case["tokens"] // page, padded=rng.choice([0, 0, 7, 15]))
    if op == "prompt":
        causal, ragged = rng.random() < 0.7, rng.random() < 0.5
        batch = _log_uniform(rng, 1, 8) if not ragged else rng.randint(2, 12)
        most = (8192 if causal else 5600) // batch
        q_len = _log_uniform(rng, 1, most)
        k_len = q_len if rng.random() < 0.7 else _log_uniform(rng, 1, most)
        case.update(batch=batch, q_len=q_len, k_len=k_len, ragged=ragged, causal=causal, lens_seed=rng.randint(0, 1 << 20))
    if op == "decode":
        batch = _log_uniform(rng, 1, 128)
        case.update(batch=batch, k_len=_log_uniform(rng, 1, min(32768, 400000 // batch)), ragged=rng.random() < 0.6,
                    page=rng.choice([16, 32, 64]), lens_seed=rng.randint(0, 1 << 20))
    return case


def _lens(case, which):
    """The lengths of a case's sequences; a ragged batch has all lengths up to the largest, one token among them."""
    most, batch = case[which], case["batch"]
    if not case["ragged"]:
        return [most] * batch
    rng = random.Random(case["lens_seed"])
    return [most, 1] + [rng.randint(1, most) for _ in range(batch - 2)] if batch > 1 else [most]


# ------------------------------------------------------------------ the inputs
def _turns(case, device):
    """The rotation of each pair per position, in turns: base 10000, and for a scaled context
    the slow pairs slowed by 8 with a ramp between (first trained on 4096 positions)."""
    dim = case["rot_dim"]
    i = torch.arange(0, dim, 2, dtype=torch.float64, device=device)
    turns = 10000.0 ** (-i / dim) / (2 * math.pi)
    if case["scaled"]:
        rounds = turns * 4096
        keep = ((rounds - 1) / (32 - 1)).clamp(0, 1)
        turns = turns * (keep + (1 - keep) / 8)
    return turns


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev)
    gen.manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)

    heads, kv_heads, dim = case["heads"], case["kv_heads"], case["head_dim"]
    st = dict(case=case)
    if case["op"] in ("norm_rope", "append"):
        tokens = case["tokens"]
        dtype = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        row = normal(tokens, (heads + 2 * kv_heads) * dim, dtype=dtype)
        # a few channels far above the others, as projections have them
        row[:, torch.randperm(row.shape[1], generator=gen, device=dev)[:row.shape[1] // 100 + 1]] *= 8
        st["q"], st["k"], st["v"] = _split(row, heads, kv_heads, dim)
        st["positions"] = case["first"] + torch.arange(tokens, device=dev)
        if tokens > 1 and case["first"]:    # a step of many sequences, each somewhere else
            st["positions"] = torch.randint(0, 2 * case["first"], (tokens,), generator=gen, device=dev)
        st["q_weight"] = (1 + 0.2 * normal(dim).float()).to(torch.bfloat16) if case["norm"] else None
        st["k_weight"] = (1 + 0.2 * normal(dim).float()).to(torch.bfloat16) if case["norm"] else None
        st["turns"] = _turns(case, dev)
        st["amplitude"] = 1.0 + 0.1 * math.log(8) if case["scaled"] else 1.0
    if case["op"] == "append":
        pages, page = case["pages"], case["page"]
        st["k_cache"], st["v_cache"] = normal(pages, page, kv_heads, dim), normal(pages, page, kv_heads, dim)
        slots = torch.randperm(pages * page, generator=gen, device=dev)[:case["tokens"]]
        if case["padded"]:
            slots[case["padded"] - 1::case["padded"]] = -1
        st["slots"] = slots
    if case["op"] == "prompt":
        q_lens, k_lens = _lens(case, "q_len"), _lens(case, "k_len")
        if q_lens == k_lens:
            row = normal(sum(q_lens), (heads + 2 * kv_heads) * dim)
            st["q"], st["k"], st["v"] = _split(row, heads, kv_heads, dim)
        else:
            st["q"] = normal(sum(q_lens), heads, dim)
            row = normal(sum(k_lens), 2 * kv_heads * dim)
            st["k"], st["v"] = row.view(-1, 2, kv_heads, dim).unbind(1)
        st["cu_q"], st["cu_k"] = _sums(q_lens, dev), _sums(k_lens, dev)
    if case["op"] == "decode":
        lens, page = _lens(case, "k_len"), case["page"]
        need = [-(-n // page) for n in lens]
        pages = sum(need) + 3
        st["k_cache"], st["v_cache"] = normal(pages, page, kv_heads, dim), normal(pages, page, kv_heads, dim)
        order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
        # the pages of all sequences one behind the other, cut where a sequence ends
        column = torch.arange(max(need), device=dev)
        first = _sums(need, dev)[:-1, None]
        used = column[None, :] < torch.tensor(need, device=dev)[:, None]
        st["page_table"] = torch.where(used, order[(first + column).clamp(max=pages - 1)], torch.zeros_like(order[:1]))
        st["kv_len"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        st["q"] = normal(case["batch"], heads, dim)
    return st


def _split(row, heads, kv_heads, dim):
    """Views of the query, key and value heads of a projection row."""
    return row.view(row.shape[0], -1, dim).split([heads, kv_heads, kv_heads], dim=1)


def _sums(lens, device):
    return torch.tensor([0] + lens, device=device).cumsum(0).to(torch.int32)


# ------------------------------------------------------------------ one pass
def run(st):
    op = st["case"]["op"]
    if own:
        import rank_bit_residual_b200 as rb
        if op == "prompt":
            return rb.svdq_attention_prompt(st["q"], st["k"], st["v"], st["cu_q"], st["cu_k"], causal=st["case"]["causal"])
        if op == "decode":
            return rb.svdq_attention_decode(st["q"], st["k_cache"], st["v_cache"], st["page_table"], st["kv_len"])
        rope = rb.Rope(st["turns"], interleaved=st["case"]["interleaved"], amplitude=st["amplitude"])
        if op == "norm_rope":
            return rb.svdq_qk_norm_rope(st["q"], st["k"], st["positions"], rope, q_weight=st["q_weight"],
                                        k_weight=st["k_weight"], eps=NORM_EPS)
        q = rb.svdq_kv_append(st["k_cache"], st["v_cache"], st["k"], st["v"], st["slots"], st["positions"], rope,
                              k_weight=st["k_weight"], eps=NORM_EPS, q=st["q"], q_weight=st["q_weight"])
        return q, st["k_cache"], st["v_cache"]
    if op == "prompt":
        return _prompt(st)
    if op == "decode":
        return _decode(st)
    q = _norm_rope(st["q"], st["q_weight"], st)
    k = _norm_rope(st["k"], st["k_weight"], st)
    if op == "norm_rope":
        return q, k
    kept = st["slots"] >= 0
    for cache, rows in ((st["k_cache"], k), (st["v_cache"], st["v"])):
        cache.view(-1, *cache.shape[2:])[st["slots"][kept]] = rows[kept]
    return q, st["k_cache"], st["v_cache"]


def _norm_rope(x, weight, st):
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + NORM_EPS) * weight.float()
    angle = 2 * math.pi * st["positions"].double()[:, None] * st["turns"]
    cos = (st["amplitude"] * angle.cos()).float()[:, None, :]
    sin = (st["amplitude"] * angle.sin()).float()[:, None, :]
    rot = 2 * st["turns"].numel()
    turned, rest = y[..., :rot], y[..., rot:]
    if st["case"]["interleaved"]:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = turned.chunk(2, -1)
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, rest), -1).to(x.dtype)


def _softmax_product(scores, keep, v):
    """softmax over the kept scores times v; a row that keeps none is zero."""
    scores = scores.masked_fill(~keep, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - top.masked_fill(top == -math.inf, 0.0))
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / total.masked_fill(total == 0, 1.0)


def _prompt(st):
    q, k, v = (st[n].float().transpose(0, 1) for n in ("q", "k", "v"))
    heads, rows, dim = q.shape
    kv_heads, keys = k.shape[:2]
    cu_q, cu_k = st["cu_q"].long(), st["cu_k"].long()
    # every row's sequence, and its place counted from that sequence's end
    row = torch.arange(rows, device=q.device)
    key = torch.arange(keys, device=q.device)
    row_seq = torch.searchsorted(cu_q, row, right=True) - 1
    key_seq = torch.searchsorted(cu_k, key, right=True) - 1
    keep = row_seq[:, None] == key_seq[None, :]
    if st["case"]["causal"]:
        keep &= (cu_k[key_seq + 1] - key)[None, :] >= (cu_q[row_seq + 1] - row)[:, None]
    group = heads // kv_heads
    scores = torch.matmul(q.reshape(kv_heads, group * rows, dim) / math.sqrt(dim), k.transpose(1, 2))
    out = _softmax_product(scores.view(kv_heads, group, rows, keys), keep, v[:, None])
    return out.reshape(heads, rows, dim).transpose(0, 1).to(st["q"].dtype).contiguous()


def _decode(st):
    q = st["q"].float()
    batch, heads, dim = q.shape
    kv_heads = st["k_cache"].shape[2]
    table = st["page_table"].long()
    k, v = (st[n][table].flatten(1, 2).transpose(1, 2).float() for n in ("k_cache", "v_cache"))
    scores = torch.matmul(q.view(batch, kv_heads, heads // kv_heads, dim) / math.sqrt(dim), k.transpose(2, 3))
    keep = torch.arange(k.shape[2], device=q.device) < st["kv_len"][:, None, None, None]
    return _softmax_product(scores, keep, v).reshape(batch, heads, dim).to(st["q"].dtype)


# ------------------------------------------------------------------ what a pass needs
def work(case):
    heads, kv_heads, dim = case["heads"], case["kv_heads"], case["head_dim"]
    if case["op"] in ("norm_rope", "append"):
        size = 4 if case["dtype"] == "f32" else 2
        values = case["tokens"] * (heads + kv_heads) * dim
        moved = 2 * size * values + 8 * case["tokens"] + 4 * case["rot_dim"]
        if case["op"] == "append":
            moved += 2 * size * case["tokens"] * kv_heads * dim + 8 * case["tokens"]
        turned = 3 * case["tokens"] * (heads + kv_heads) * case["rot_dim"]
        return {"bytes": moved, "flops": turned + (4 * values if case["norm"] else 0)}
    k_lens = _lens(case, "k_len")
    if case["op"] == "decode":
        tokens = sum(k_lens)
        return {"bytes": 4 * tokens * kv_heads * dim + 4 * case["batch"] * heads * dim + 4 * sum(-(-n // case["page"]) for n in k_lens),
                "flops": 4 * tokens * heads * dim}
    q_lens = _lens(case, "q_len")
    pairs = 0
    for nq, nk in zip(q_lens, k_lens):
        # row i of a causal sequence sees nk - nq + i + 1 keys, none where that is not positive
        seen = min(nq, nk)
        pairs += seen * nk - seen * (seen - 1) // 2 if case["causal"] else nq * nk
    return {"bytes": 4 * dim * (sum(q_lens) * heads + sum(k_lens) * kv_heads), "flops": 4 * dim * heads * pairs}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "prompt":
        return _exact_prompt(st)
    if case["op"] == "decode":
        return _exact_decode(st)
    q, k = (_exact_turned(st[n].double(), st[n + "_weight"], st) for n in ("q", "k"))
    if case["op"] == "norm_rope":
        return q, k
    k_cache, v_cache = st["k_cache"].double(), st["v_cache"].double()
    token = torch.nonzero(st["slots"] >= 0).flatten()
    place, within = st["slots"][token] // case["page"], st["slots"][token] % case["page"]
    k_cache[place, within] = k[token]
    v_cache[place, within] = st["v"][token].double()
    return q, k_cache, v_cache


def _exact_turned(x, weight, st):
    """The pairs as complex numbers, multiplied by amplitude * exp(i angle)."""
    if weight is not None:
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + NORM_EPS) * weight.double()
    half = st["turns"].numel()
    around = torch.outer(st["positions"].double(), st["turns"])
    around = 2 * math.pi * (around - around.floor())
    factor = torch.polar(torch.full_like(around, st["amplitude"]), around)[:, None]
    pairs = x[..., :2 * half]
    pairs = pairs.unflatten(-1, (half, 2)) if st["case"]["interleaved"] else pairs.unflatten(-1, (2, half)).transpose(-1, -2)
    turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * factor)
    if not st["case"]["interleaved"]:
        turned = turned.transpose(-1, -2)
    out = x.clone()
    out[..., :2 * half] = turned.flatten(-2)
    return out


def _weighted(q, k, v, seen=None):
    """One head's rows over their keys; `seen` is the number of keys that each row sees."""
    logits = q @ k.T * q.shape[-1] ** -0.5
    if seen is not None:
        logits[torch.arange(k.shape[0], device=q.device)[None] >= seen[:, None]] = -math.inf
    out = torch.softmax(logits, -1) @ v
    if seen is not None:
        out[seen <= 0] = 0
    return out


def _exact_prompt(st):
    case = st["case"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    group = case["heads"] // case["kv_heads"]
    q0 = k0 = 0
    for nq, nk in zip(_lens(case, "q_len"), _lens(case, "k_len")):
        seen = torch.arange(nk - nq + 1, nk + 1, device=out.device) if case["causal"] else None
        for h in range(case["heads"]):
            out[q0:q0 + nq, h] = _weighted(st["q"][q0:q0 + nq, h].double(), st["k"][k0:k0 + nk, h // group].double(),
                                           st["v"][k0:k0 + nk, h // group].double(), seen)
        q0, k0 = q0 + nq, k0 + nk
    return out


def _exact_decode(st):
    case = st["case"]
    out = torch.empty(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    group = case["heads"] // case["kv_heads"]
    for s, n in enumerate(_lens(case, "k_len")):
        at = torch.arange(n, device=out.device)
        where = st["page_table"][s].long()[at // case["page"]], at % case["page"]
        k, v = st["k_cache"][where].double(), st["v_cache"][where].double()
        for j in range(case["kv_heads"]):
            out[s, j * group:(j + 1) * group] = _weighted(st["q"][s, j * group:(j + 1) * group].double(), k[:, j], v[:, j])
    return out
