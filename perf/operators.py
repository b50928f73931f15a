"""The full-attention operators of a hybrid model's step: what is measured.

A hybrid model answers with gated delta-rule layers (ReplayStore) and, every few
layers, with softmax attention over a paged key-value cache. The operators here
are those of the attention layers: attention over whole prompts, attention of
new tokens over the cache's pages, rotary positions fused with the append of
keys and values, and the fork and compaction of pages.

`run` computes an operator with elementary torch operations in 32 bits
(own = False) or through KVCache's calls (own = True).
"""
import math
import random
from types import SimpleNamespace

import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
KEYS_MOST = 0.9e9    # bytes of keys and values that a drawn decode pass reads


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a chat turn of one user: latency counts, the tile is mostly empty
        dict(name="prompt_one_short", op="prompt", dtype="bf16", B=1, low=37, high=37, HQ=8,
             HKV=8, D=64, past=0, lens=1),
        # a step of continuous batching: prompts of very different lengths, wide heads
        dict(name="prompt_ragged", op="prompt", dtype="bf16", B=8, low=64, high=4096, HQ=16,
             HKV=4, D=256, past=0, lens=2),
        # one long document
        dict(name="prompt_long", op="prompt", dtype="bf16", B=1, low=14336, high=14336, HQ=16,
             HKV=4, D=128, past=0, lens=3),
        # the same layer kept in 32 bits: chunks of prompts whose first part was seen before
        dict(name="prompt_f32_past", op="prompt", dtype="f32", B=5, low=33, high=700, HQ=8,
             HKV=2, D=64, past=257, lens=4),
        # one user, a short answer so far: latency counts
        dict(name="decode_one_short", op="decode", dtype="bf16", B=1, null=0, T=1, low=131,
             high=131, HQ=16, HKV=4, D=128, page=16, lens=5),
        # the serving batch: 64 rows of which 8 are null, lengths spread over a decade
        dict(name="decode_batch", op="decode", dtype="bf16", B=64, null=8, T=1, low=1024,
             high=8192, HQ=16, HKV=4, D=256, page=64, lens=6),
        # few rows, long contexts: the split over the length
        dict(name="decode_long", op="decode", dtype="f16", B=2, null=0, T=1, low=100001,
             high=131072, HQ=32, HKV=8, D=128, page=64, lens=7),
        # speculative verify: 8 draft tokens a row at batch 128
        dict(name="verify_window", op="decode", dtype="bf16", B=128, null=3, T=8, low=300,
             high=3000, HQ=16, HKV=4, D=128, page=32, lens=8),
        # a decode step's new keys and values
        dict(name="append_decode", op="append", dtype="bf16", B=64, null=8, T=1, HQ=16, HKV=4,
             D=256, rot=64, axes=1, page=64, lens=9),
        # the prompts of a step with images: positions of three axes, heads of 128
        dict(name="append_prompt_axes", op="append", dtype="bf16", B=8, null=0, T=2021, HQ=32,
             HKV=8, D=128, rot=128, axes=3, page=64, lens=10),
        # parallel samples from one prompt each: full pages shared, the last one copied
        dict(name="fork_samples", op="fork", dtype="bf16", B=96, src=24, low=200, high=4000,
             HKV=4, D=128, layers=8, page=64, lens=11),
        # a pool after many requests have ended: pages in use move to its front
        dict(name="compact_pool", op="compact", dtype="bf16", slots=192, keep=0.5, low=200,
             high=1500, HKV=4, D=128, layers=8, page=32, lens=12),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("prompt", "prompt", "decode", "decode", "append", "fork", "compact"))
    lens = rng.randrange(1, 10**6)
    D = rng.choice((64, 128, 256))
    HKV = rng.choice((1, 2, 4, 8))
    G = rng.choice((1, 2, 3, 4, 5, 6, 8))
    page = rng.choice((16, 32, 64, 128))
    if op == "prompt":
        dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
        high = _log(rng, 16, 2048 if dtype == "f32" else 8192)
        low = max(1, int(high * rng.choice((0.02, 0.3, 1.0))))
        past = rng.choice((0, 0, _log(rng, 1, 1024)))
        B = _log(rng, 1, 32)
        most = 2e8 if dtype == "f32" else 1.5e9
        while B > 1 and B * HKV * G * high * (high + past) > most:
            B //= 2
        while HKV * G * high * (high + past) > most:
            high = high * 2 // 3
            low = min(low, high)
        return dict(op=op, dtype=dtype, B=B, low=low, high=high, HQ=HKV * G, HKV=HKV, D=D,
                    past=past, lens=lens)
    if op == "decode":
        dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
        T = rng.choice((1, 1, 1, 2, 3, 5, 8, 16))
        high = _log(rng, 16, 65536)
        low = max(1, int(high * rng.choice((0.02, 0.5, 1.0))))
        B = _log(rng, 1, 256)
        while B > 1 and (B * high * HKV * D * 2 * SIZE[dtype] > KEYS_MOST
                         or B * high * HKV * G * T > 3e8):
            B //= 2
        null = rng.choice((0, B // 8))
        return dict(op=op, dtype=dtype, B=B, null=null, T=T, low=low, high=high, HQ=HKV * G,
                    HKV=HKV, D=D, page=page, lens=lens)
    if op == "append":
        dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
        B, T = _log(rng, 1, 128), _log(rng, 1, 2000)
        while B > 1 and B * T * (2 * G + 4) * HKV * D * SIZE[dtype] > 8e8:
            B //= 2
        return dict(op=op, dtype=dtype, B=B, null=rng.choice((0, B // 8)), T=T, HQ=HKV * G,
                    HKV=HKV, D=D, rot=rng.choice((D, D // 2)), axes=rng.choice((1, 2, 3)),
                    page=page, lens=lens)
    dtype = rng.choice(("bf16", "f32"))
    layers = rng.choice((1, 3, 8))
    if op == "fork":
        src = _log(rng, 1, 32)
        B = src * rng.choice((1, 2, 4))
        high = _log(rng, 8, 3000)
        while B > src and B * page * HKV * D * SIZE[dtype] * 2 * layers > 2e8:
            B -= src
        return dict(op=op, dtype=dtype, B=B, src=src, low=max(1, high // 5), high=high, HKV=HKV,
                    D=D, layers=layers, page=page, lens=lens)
    slots, high = _log(rng, 2, 192), _log(rng, 50, 1500)
    while slots > 2 and slots * high * HKV * D * SIZE[dtype] * 2 * layers > 1e9:
        slots //= 2
    return dict(op=op, dtype=dtype, slots=slots, keep=rng.choice((0.3, 0.5, 0.8)),
                low=max(1, high // 5), high=high, HKV=HKV, D=D, layers=layers, page=page,
                lens=lens)


def _lengths(case, n):
    """n lengths of the case, spread over the logarithm of [low, high]; the first is high."""
    r = random.Random(case["lens"])
    return [case["high"] if i == 0 else _log(r, case["low"], case["high"]) for i in range(n)]


# ------------------------------------------------------------------ inputs
def _gen(case, seed):
    return torch.Generator("cuda").manual_seed(seed * 1000003 + case["lens"])


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _normal(shape, dtype, gen, by=1.0):
    """N(0, by^2) in the type, drawn in slices of the first axis (a pool is large)."""
    x = torch.empty(shape, dtype=DTYPE[dtype], device="cuda")
    for i in range(x.shape[0]):
        x[i].normal_(0.0, by, generator=gen)
    return x


def _cache(case, layers, slots, pages, max_pages):
    """A program's cache: KVCache, or the same buffers where it is not to be had."""
    shape = (layers, pages, case["HKV"], case["page"], case["D"])
    if own:
        from linear_attention_state_rssm_gb300.store import KVCache
        c = KVCache(layers, slots, case.get("HQ", case["HKV"]), case["HKV"], case["D"],
                    n_pages=pages, page_size=case["page"], max_pages=max_pages,
                    dtype=case["dtype"])
    else:
        z = dict(dtype=torch.int32, device="cuda")
        c = SimpleNamespace(
            k_pages=torch.empty(shape, dtype=DTYPE[case["dtype"]], device="cuda"),
            v_pages=torch.empty(shape, dtype=DTYPE[case["dtype"]], device="cuda"),
            table=torch.full((slots, max_pages), -1, **z), held=torch.zeros(slots, **z),
            length=torch.zeros(slots, **z), refs=torch.zeros(pages, **z))
    return c


def _fill(c, gen, by):
    for pool in (c.k_pages, c.v_pages):
        for layer in range(pool.shape[0]):
            pool[layer].normal_(0.0, by, generator=gen)


def _hand_out(c, counts, gen):
    """Gives slot i counts[i] pages, in a random order of the pool."""
    pages, most = c.refs.shape[0], c.table.shape[1]
    order = torch.randperm(pages, generator=gen, device="cuda").int()
    n = torch.tensor(counts, device="cuda")
    start = torch.cumsum(n, 0) - n
    at = torch.arange(most, device="cuda")
    take = (start[:, None] + at).clamp(max=pages - 1)
    c.table[:len(counts)] = torch.where(at < n[:, None], order[take], torch.full_like(order[take], -1))
    c.held[:len(counts)] = n.int()
    c.refs.zero_()
    c.refs[order[:sum(counts)].long()] = 1


def _pages(tokens, page):
    return -(-tokens // page)


def prepare(case, seed):
    gen = _gen(case, seed)
    return {"prompt": _prepare_prompt, "decode": _prepare_decode, "append": _prepare_append,
            "fork": _prepare_fork, "compact": _prepare_compact}[case["op"]](case, seed, gen)


def _prepare_prompt(case, seed, gen):
    """Packed prompts: q, k and v are views of one projection's output (token stride over
    all heads) unless keys of earlier chunks come before this chunk's."""
    HQ, HKV, D, B = case["HQ"], case["HKV"], case["D"], case["B"]
    lens = _lengths(case, B)
    klens = [n + case["past"] for n in lens]
    N, M = sum(lens), sum(klens)
    s = SimpleNamespace(case=case, B=B)
    if case["past"] == 0:
        qkv = _normal((N, HQ + 2 * HKV, D), case["dtype"], gen) if N < 64 else \
            _normal((1, N, HQ + 2 * HKV, D), case["dtype"], gen)[0]
        qkv[:, :HQ] *= 1.5
        s.q, s.k, s.v = qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]
    else:
        s.q = _normal((1, N, HQ, D), case["dtype"], gen, 1.5)[0]
        s.k = _normal((1, M, HKV, D), case["dtype"], gen)[0]
        s.v = _normal((1, M, HKV, D), case["dtype"], gen)[0]
    s.cu = _ints([0] + [sum(lens[:i + 1]) for i in range(B)])
    s.cu_k = _ints([0] + [sum(klens[:i + 1]) for i in range(B)]) if case["past"] else None
    s.most, s.most_k = max(lens), max(klens)
    s.o = torch.zeros((N, HQ, D), dtype=DTYPE[case["dtype"]], device="cuda")
    s.slot = torch.arange(B, dtype=torch.int32, device="cuda")
    s.scale = D ** -0.5
    if own:
        c = SimpleNamespace(**case)
        from linear_attention_state_rssm_gb300.store import KVCache
        s.cache = KVCache(1, B, c.HQ, c.HKV, c.D, n_pages=1, page_size=16, max_pages=1,
                          dtype=c.dtype)
    return s


def _rows(case):
    """Slots of a batch: row r has slot r but each (B // null)-th, which is null."""
    B, null = case["B"], case["null"]
    slot = list(range(B))
    for i in range(null):
        slot[i * (B // null)] = -1
    return slot


def _prepare_decode(case, seed, gen):
    HQ, D, B, T, page = case["HQ"], case["D"], case["B"], case["T"], case["page"]
    lens = _lengths(case, B)
    counts = [_pages(n + T, page) for n in lens]
    s = SimpleNamespace(case=case)
    s.cache = _cache(case, 1, B, sum(counts) + 3, max(counts))
    _fill(s.cache, gen, 1.0)
    _hand_out(s.cache, counts, gen)
    s.cache.length.copy_(_ints(lens))
    s.slot = _ints(_rows(case))
    s.q = _normal((1, B * T, HQ, D), case["dtype"], gen, 1.5)[0]
    s.o = torch.zeros_like(s.q)
    s.most, s.scale = max(lens) + T, D ** -0.5
    return s


def _prepare_append(case, seed, gen):
    HQ, HKV, D, B, T = case["HQ"], case["HKV"], case["D"], case["B"], case["T"]
    r = random.Random(case["lens"])
    lens = [r.randrange(0, 3000) for _ in range(B)]
    counts = [_pages(n + T, case["page"]) for n in lens]
    s = SimpleNamespace(case=case)
    s.cache = _cache(case, 1, B, sum(counts) + 2, max(counts))
    _fill(s.cache, gen, 1.0)
    _hand_out(s.cache, counts, gen)
    s.cache.length.copy_(_ints(lens))
    s.slot = _ints(_rows(case))
    qkv = _normal((1, B * T, HQ + 2 * HKV, D), case["dtype"], gen, 1.5)[0]
    s.q, s.k, s.v = qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]
    s.q_out = torch.zeros((B * T, HQ, D), dtype=DTYPE[case["dtype"]], device="cuda")
    P, A = case["rot"] // 2, case["axes"]
    most = 8192
    s.sections = [P - (A - 1) * (P // A)] + [P // A] * (A - 1)
    angle = torch.arange(most, dtype=torch.float64, device="cuda")[:, None] * \
        1e6 ** (-torch.arange(P, dtype=torch.float64, device="cuda") / P)
    s.table = torch.stack((angle.cos(), angle.sin()), 1).float().contiguous()
    s.positions = torch.randint(0, most, (A, B * T), generator=gen, device="cuda",
                                dtype=torch.int32)
    if own:
        from linear_attention_state_rssm_gb300.store import RotaryTable
        s.rope = RotaryTable(s.table, s.sections)
    return s


def _prepare_fork(case, seed, gen):
    """`src` slots with prompts; each is forked into B / src others."""
    n, B, page = case["src"], case["B"], case["page"]
    lens = _lengths(case, n)
    counts = [_pages(t, page) for t in lens]
    s = SimpleNamespace(case=case)
    s.cache = _cache(case, case["layers"], n + B, sum(counts) + B + 5, max(counts))
    _fill(s.cache, gen, 1.0)
    _hand_out(s.cache, counts, gen)
    s.cache.length[:n].copy_(_ints(lens))
    s.src = _ints([i % n for i in range(B)])
    s.dst = _ints([n + i for i in range(B)])
    return s


def _prepare_compact(case, seed, gen):
    """A pool whose slots ended at random but for a share `keep`; a snapshot of the page
    tables is kept, from which each pass begins (the pages' contents stand in both)."""
    lens = _lengths(case, case["slots"])
    counts = [_pages(t, case["page"]) for t in lens]
    r = random.Random(case["lens"] + 1)
    left = [i for i in range(case["slots"]) if r.random() < case["keep"]] or [0]
    s = SimpleNamespace(case=case)
    c = s.cache = _cache(case, case["layers"], case["slots"], sum(counts), max(counts))
    _fill(c, gen, 1.0)
    _hand_out(c, counts, gen)
    gone = torch.ones(case["slots"], dtype=torch.bool, device="cuda")
    gone[torch.tensor(left, device="cuda")] = False
    dead = c.table[gone]
    c.refs[dead[dead >= 0].long()] = 0
    c.table[gone] = -1
    c.held[gone] = 0
    c.length.copy_(torch.where(gone, torch.zeros_like(c.length), _ints(lens)))
    s.was = (c.table.clone(), c.refs.clone())
    return s


# --------------------------------------------------------------------- run
def run(state):
    return {"prompt": _run_prompt, "decode": _run_decode, "append": _run_append,
            "fork": _run_fork, "compact": _run_compact}[state.case["op"]](state)


def _softmax(scores, keep):
    """exp(s - max) / sum over the last axis where `keep`; zeros where it keeps nothing."""
    scores = torch.where(keep, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.where(keep, torch.exp(scores - torch.where(top > -math.inf, top, 0.0)), 0.0)
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total > 0, total, 1.0)


def _run_prompt(s):
    if own:
        s.cache.rssm_attn_prefill(s.q, s.k, s.v, s.cu, s.slot, s.o, cu_keys=s.cu_k)
        return s.o
    N, HQ, D = s.q.shape
    HKV, B = s.k.shape[1], s.B
    G = HQ // HKV
    cu, cu_k = s.cu.long(), (s.cu if s.cu_k is None else s.cu_k).long()
    lq, lk = cu[1:] - cu[:-1], cu_k[1:] - cu_k[:-1]
    iq, ik = torch.arange(s.most, device="cuda"), torch.arange(s.most_k, device="cuda")
    at = (cu[:-1, None] + iq).clamp(max=N - 1)
    at_k = (cu_k[:-1, None] + ik).clamp(max=s.k.shape[0] - 1)
    q = s.q[at].float().view(B, s.most, HKV, G, D).permute(0, 2, 3, 1, 4).flatten(2, 3)
    k = s.k[at_k].float().permute(0, 2, 3, 1)
    v = s.v[at_k].float().permute(0, 2, 1, 3)
    last = iq + (lk - lq)[:, None]
    keep = (ik <= last[:, :, None]) & (ik < lk[:, None, None])
    scores = (torch.matmul(q, k) * s.scale).unflatten(2, (G, s.most))
    p = _softmax(scores, keep[:, None, None]).flatten(2, 3)
    o = torch.matmul(p, v).unflatten(2, (G, s.most)).permute(0, 3, 1, 2, 4)
    o = o.reshape(B, s.most, HQ, D)
    token = torch.arange(N, device="cuda")
    of = torch.bucketize(token, cu[1:], right=True)
    return o[of, token - cu[of]].to(s.o.dtype)


def _run_decode(s):
    T, page = s.case["T"], s.case["page"]
    if own:
        s.cache.rssm_attn_decode(0, s.q, s.slot, T, s.o)
        return s.o
    B, HKV, D = s.case["B"], s.case["HKV"], s.case["D"]
    G = s.case["HQ"] // HKV
    live, slot = s.slot >= 0, s.slot.clamp(min=0).long()
    at = torch.arange(s.most, device="cuda")
    ids = s.cache.table[slot][:, at // page].clamp(min=0).long()
    k = s.cache.k_pages[0][ids, :, at % page].float().permute(0, 2, 3, 1)
    q = s.q.float().view(B, T, HKV, G, D).permute(0, 2, 3, 1, 4).flatten(2, 3)
    scores = (torch.matmul(q, k) * s.scale).unflatten(2, (G, T))
    del k
    last = s.cache.length[slot][:, None] + torch.arange(T, device="cuda")
    p = _softmax(scores, (at <= last[:, :, None])[:, None, None]).flatten(2, 3)
    v = s.cache.v_pages[0][ids, :, at % page].float().permute(0, 2, 1, 3)
    o = torch.matmul(p, v).unflatten(2, (G, T)).permute(0, 3, 1, 2, 4)
    o = o.reshape(B, T, HKV * G, D)
    o = torch.where(live[:, None, None, None], o, 0.0)
    return o.reshape(B * T, HKV * G, D).to(s.o.dtype)


def _axes(P, sections):
    """Axis of each pair: the first sections[0] pairs take axis 0, the next sections[1] axis 1."""
    ends = torch.tensor(sections, device="cuda").cumsum(0)
    return torch.bucketize(torch.arange(P, device="cuda"), ends, right=True)


def _rotate(x, cos, sin):
    x = x.float()
    P = cos.shape[-1]
    a, b = x[..., :P], x[..., P:2 * P]
    cos, sin = cos[:, None], sin[:, None]
    return torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., 2 * P:]), -1)


def _run_append(s):
    T, page = s.case["T"], s.case["page"]
    c = s.cache
    if own:
        c.rssm_kv_append(0, s.q, s.k, s.v, s.slot, T, s.q_out, rope=s.rope,
                         positions=s.positions)
        return s.q_out, c.k_pages, c.v_pages
    P = s.table.shape[-1]
    row = s.table[s.positions.long()[_axes(P, s.sections)].t(), :, torch.arange(P, device="cuda")]
    cos, sin = row[..., 0], row[..., 1]
    q, k = _rotate(s.q, cos, sin), _rotate(s.k, cos, sin)
    live = (s.slot >= 0).repeat_interleave(T)
    slot = s.slot.clamp(min=0).long().repeat_interleave(T)
    at = c.length[slot].long() + torch.arange(T, device="cuda").repeat(s.slot.shape[0])
    ids = c.table[slot, at // page].long()[live]
    off = (at % page)[live]
    c.k_pages[0, ids, :, off] = k[live].to(c.k_pages.dtype)
    c.v_pages[0, ids, :, off] = s.v[live]
    s.q_out.copy_(torch.where(live[:, None, None], q.to(s.q_out.dtype), s.q_out))
    return s.q_out, c.k_pages, c.v_pages


def _run_fork(s):
    c, page = s.cache, s.case["page"]
    if own:
        c.rssm_kv_fork(s.src, s.dst)
        return c.table, c.held, c.length, c.refs, c.k_pages, c.v_pages
    src, dst = s.src.long(), s.dst.long()
    old = c.table[dst]
    c.refs -= torch.bincount(old[old >= 0].long(), minlength=c.refs.shape[0]).int()
    n = c.length[src]
    whole, part = n // page, n % page > 0
    at = torch.arange(c.table.shape[1], device="cuda")
    rows = torch.where(at < whole[:, None], c.table[src], -1)
    c.refs += torch.bincount(rows[rows >= 0].long(), minlength=c.refs.shape[0]).int()
    free = torch.nonzero(c.refs == 0)[:, 0]
    new = free[:int(part.sum())]
    tail = c.table[src[part], whole[part].long()].long()
    c.refs[new] = 1
    rows[part, whole[part].long()] = new.int()
    c.table[dst] = rows
    c.held[dst] = whole + part.int()
    c.length[dst] = n
    c.k_pages[:, new] = c.k_pages[:, tail]
    c.v_pages[:, new] = c.v_pages[:, tail]
    return c.table, c.held, c.length, c.refs, c.k_pages, c.v_pages


def _run_compact(s):
    c = s.cache
    c.table.copy_(s.was[0])
    c.refs.copy_(s.was[1])
    if own:
        c.rssm_kv_compact()
        return c.table, c.refs, c.k_pages, c.v_pages
    used = c.refs > 0
    n = int(used.sum())
    src = torch.nonzero(used[n:])[:, 0] + n
    dst = torch.nonzero(~used[:n])[:, 0]
    to = torch.arange(c.refs.shape[0], device="cuda", dtype=torch.int32)
    to[src] = dst.int()
    c.table.copy_(torch.where(c.table >= 0, to[c.table.clamp(min=0).long()], c.table))
    c.refs[dst] = c.refs[src]
    c.refs[src] = 0
    c.k_pages[:, dst] = c.k_pages[:, src]
    c.v_pages[:, dst] = c.v_pages[:, src]
    return c.table, c.refs, c.k_pages, c.v_pages


# -------------------------------------------------------------------- work
def work(case):
    size, D, HKV = SIZE[case["dtype"]], case["D"], case["HKV"]
    if case["op"] == "prompt":
        lens = _lengths(case, case["B"])
        past, HQ = case["past"], case["HQ"]
        pairs = sum(n * past + n * (n + 1) // 2 for n in lens)
        N, M = sum(lens), sum(lens) + past * len(lens)
        return {"bytes": (2 * N * HQ + 2 * M * HKV) * D * size, "flops": 4 * D * HQ * pairs}
    if case["op"] == "decode":
        T, HQ = case["T"], case["HQ"]
        lens = [n for n, s in zip(_lengths(case, case["B"]), _rows(case)) if s >= 0]
        keys = sum(n + T for n in lens)
        pairs = sum(n * T + T * (T + 1) // 2 for n in lens)
        return {"bytes": (2 * keys * HKV + 2 * len(lens) * T * HQ) * D * size
                + 4 * sum(_pages(n + T, case["page"]) for n in lens), "flops": 4 * D * HQ * pairs}
    if case["op"] == "append":
        N = (case["B"] - case["null"]) * case["T"]
        return {"bytes": N * ((2 * case["HQ"] + 4 * HKV) * D * size + 4 * case["axes"]
                              + 4 * case["rot"]), "flops": 3 * N * (case["HQ"] + HKV) * case["rot"]}
    one = HKV * D * case["page"] * size * 2 * case["layers"]
    if case["op"] == "fork":
        lens = _lengths(case, case["src"])
        tails = sum(lens[i % case["src"]] % case["page"] > 0 for i in range(case["B"]))
        held = sum(_pages(lens[i % case["src"]], case["page"]) for i in range(case["B"]))
        # a source's last page is read once, however many copies are made of it
        read = len({i % case["src"] for i in range(case["B"])
                    if lens[i % case["src"]] % case["page"]})
        return {"bytes": (read + tails) * one + 8 * held, "flops": 0}
    moved, held = _moves(case)
    return {"bytes": 2 * moved * one + 8 * held, "flops": 0}


def _moves(case):
    """Pages that a compaction moves, about (the pages' order is drawn on the device): those
    in use behind the front, at the share of pages in use; and pages held."""
    counts = [_pages(t, case["page"]) for t in _lengths(case, case["slots"])]
    r = random.Random(case["lens"] + 1)
    left = [i for i in range(case["slots"]) if r.random() < case["keep"]] or [0]
    held = sum(counts[i] for i in left)
    return held * (sum(counts) - held) // sum(counts), held


# ------------------------------------------------------------------- exact
def exact(case, seed):
    """The attention's and the rotation's outputs in 64 bits, row by row from the formulas;
    whole-number state and copied pages have no such value."""
    s = prepare(case, seed)
    if case["op"] == "prompt":
        return _exact_prompt(case, s)
    if case["op"] == "decode":
        return _exact_decode(case, s)
    if case["op"] == "append":
        return _exact_append(case, s), None, None
    return None


def _attend(q, k, v, scale, past):
    """One head in 64 bits: query i sees keys 0 .. past + i."""
    s = q.double() @ k.double().t() * scale
    i = torch.arange(s.shape[0], device=s.device)[:, None]
    s.masked_fill_(torch.arange(s.shape[1], device=s.device) > past + i, -math.inf)
    return torch.softmax(s, -1) @ v.double()


def _exact_prompt(case, s):
    G, o = case["HQ"] // case["HKV"], torch.zeros(s.o.shape, dtype=torch.float64, device="cuda")
    a = b = 0
    for n in _lengths(case, case["B"]):
        m = n + case["past"]
        for h in range(case["HQ"]):
            o[a:a + n, h] = _attend(s.q[a:a + n, h], s.k[b:b + m, h // G], s.v[b:b + m, h // G],
                                    s.scale, case["past"])
        a, b = a + n, b + m
    return o


def _exact_decode(case, s):
    T, G = case["T"], case["HQ"] // case["HKV"]
    o = torch.zeros(s.o.shape, dtype=torch.float64, device="cuda")
    table = s.cache.table.cpu()
    for r, (n, slot) in enumerate(zip(_lengths(case, case["B"]), _rows(case))):
        if slot < 0:
            continue
        ids = table[slot, :_pages(n + T, case["page"])].long().cuda()
        # [pages, HKV, page, D] -> [HKV, tokens, D]
        k, v = (p[0, ids].transpose(0, 1).flatten(1, 2)[:, :n + T]
                for p in (s.cache.k_pages, s.cache.v_pages))
        for h in range(case["HKV"]):
            for g in range(G):
                at = (slice(r * T, r * T + T), h * G + g)
                o[at] = _attend(s.q[at], k[h], v[h], s.scale, n)
    return o


def _exact_append(case, s):
    P, A = case["rot"] // 2, case["axes"]
    freq = 1e6 ** (-torch.arange(P, dtype=torch.float64) / P)
    axis = torch.tensor([a for a in range(A) for _ in range(s.sections[a])])
    angle = s.positions.cpu().double()[axis].t() * freq
    z = torch.polar(torch.ones_like(angle), angle).cuda()[:, None]
    x = s.q.double()
    y = torch.complex(x[..., :P], x[..., P:2 * P]) * z
    out = torch.cat((y.real, y.imag, x[..., 2 * P:]), -1)
    live = (s.slot >= 0).repeat_interleave(case["T"])
    return torch.where(live[:, None, None], out, 0.0)
