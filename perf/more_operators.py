"""More of a hybrid model's full-attention layers: what is measured.

Norms of queries and keys for each head with the rotary append, a cache whose
pages are quantised as they are written (e4m3 values, a power of two for each
token and head) and read back by the attention of new tokens and in a row, and
attention for a batch whose slots share the pages of a long prefix.

`run` computes an operator with elementary torch operations in 32 bits
(own = False) or through KVCache's calls (own = True).
"""
import math
import random
from types import SimpleNamespace

import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}
EPS = 1e-6
KEYS_MOST = 6e8      # bytes of keys and values that a drawn pass reads


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step's new tokens, 8 of 64 rows null, a quarter of each head turned
        dict(name="append_norm_decode", op="append", dtype="bf16", pages="bf16", B=64, null=8,
             T=1, ragged=False, HQ=16, HKV=4, D=256, rot=64, axes=1, page=64, lens=21),
        # packed prompts of very different lengths, positions of three axes
        dict(name="append_norm_prompt", op="append", dtype="bf16", pages="bf16", B=8, null=0,
             T=2021, ragged=True, HQ=32, HKV=8, D=128, rot=128, axes=3, page=64, lens=22),
        # a speculative window, quantised as it is written
        dict(name="append_e4m3_window", op="append", dtype="f16", pages="e4m3", B=33, null=4,
             T=5, ragged=False, HQ=8, HKV=8, D=64, rot=64, axes=1, page=16, lens=23),
        # prompts into a quantised cache
        dict(name="append_e4m3_prompt", op="append", dtype="bf16", pages="e4m3", B=9, null=1,
             T=1777, ragged=False, HQ=16, HKV=4, D=256, rot=64, axes=1, page=64, lens=24),
        # one user, a short answer so far: latency counts
        dict(name="decode_e4m3_short", op="decode", dtype="bf16", pages="e4m3", B=1, null=0, T=1,
             low=131, high=131, HQ=16, HKV=4, D=128, page=16, lens=25),
        # the serving batch: lengths spread over a decade
        dict(name="decode_e4m3_batch", op="decode", dtype="bf16", pages="e4m3", B=64, null=8, T=1,
             low=1024, high=8192, HQ=16, HKV=4, D=256, page=64, lens=26),
        # few rows, long contexts: the split over the length
        dict(name="decode_e4m3_long", op="decode", dtype="f16", pages="e4m3", B=2, null=0, T=1,
             low=100001, high=131072, HQ=32, HKV=8, D=128, page=64, lens=27),
        # speculative verify at batch 128
        dict(name="verify_e4m3_window", op="decode", dtype="bf16", pages="e4m3", B=128, null=3,
             T=8, low=300, high=3000, HQ=16, HKV=4, D=128, page=32, lens=28),
        # the cached first parts of a step's prompts, in a row for their attention
        dict(name="gather_e4m3_prefix", op="gather", dtype="bf16", pages="e4m3", B=12, null=1,
             low=500, high=16000, first=0, HKV=8, D=128, page=64, lens=29),
        # a window of the last tokens of short chats: latency counts
        dict(name="gather_window", op="gather", dtype="bf16", pages="bf16", B=5, null=0, low=60,
             high=255, first=301, HKV=4, D=64, page=32, lens=30),
        # samples drawn from one long prompt
        dict(name="shared_one_prompt", op="shared", dtype="bf16", pages="bf16", groups=1,
             members=64, T=1, low=8200, high=8200, own=300, HQ=16, HKV=4, D=128, page=64,
             layers=4, lens=31),
        # a few samples from each of many prompts, windows of two tokens, quantised pages
        dict(name="shared_e4m3_groups", op="shared", dtype="bf16", pages="e4m3", groups=20,
             members=4, T=2, low=700, high=5000, own=150, HQ=16, HKV=4, D=128, page=32,
             layers=4, lens=32),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("append", "append", "decode", "decode", "gather", "shared", "shared"))
    lens = rng.randrange(1, 10**6)
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    pages = dtype if dtype == "f32" or (op != "decode" and rng.random() < 0.5) else "e4m3"
    if op == "decode" and dtype == "f32":
        dtype, pages = "f16", "e4m3"
    D = rng.choice((64, 128, 256))
    HKV = rng.choice((1, 2, 4, 8))
    G = rng.choice((1, 2, 3, 4, 5, 6, 8))
    page = rng.choice((16, 32, 64, 128))
    both = dict(dtype=dtype, pages=pages, HKV=HKV, D=D, page=page, lens=lens)
    if op == "append":
        B, T = _log(rng, 1, 128), _log(rng, 1, 2000)
        while B > 1 and B * T * (2 * G + 6) * HKV * D * SIZE[dtype] > 4e8:
            B //= 2
        return dict(op=op, B=B, null=rng.choice((0, B // 8)), T=T, ragged=rng.random() < 0.4,
                    HQ=HKV * G, rot=rng.choice((D, D // 2)), axes=rng.choice((1, 2, 3)), **both)
    if op == "decode":
        T = rng.choice((1, 1, 1, 2, 3, 5, 8, 16))
        high = _log(rng, 16, 65536)
        low = max(1, int(high * rng.choice((0.02, 0.5, 1.0))))
        B = _log(rng, 1, 256)
        while B > 1 and (B * high * HKV * D * 2 > KEYS_MOST / 2 or B * high * HKV * G * T > 2e8):
            B //= 2
        return dict(op=op, B=B, null=rng.choice((0, B // 8)), T=T, low=low, high=high,
                    HQ=HKV * G, **both)
    if op == "gather":
        high = _log(rng, 16, 16000)
        low = max(1, int(high * rng.choice((0.02, 0.5, 1.0))))
        B = _log(rng, 1, 64)
        while B > 1 and B * high * HKV * D * 4 > 3e8:
            B //= 2
        return dict(op=op, B=B, null=rng.choice((0, B // 8)), low=low, high=high,
                    first=rng.choice((0, 0, _log(rng, 1, 500))), **both)
    groups, members = _log(rng, 1, 24), _log(rng, 1, 64)
    T = rng.choice((1, 1, 1, 2, 4, 8))
    high = _log(rng, 40, 16000)
    layers = rng.choice((1, 2, 4))
    most = 3e8 if dtype == "f32" else KEYS_MOST
    while members > 1 and groups * members * layers * high * HKV * D * 4 > most:
        members //= 2
    while groups > 1 and groups * members * layers * high * HKV * D * 4 > most:
        groups //= 2
    return dict(op=op, groups=groups, members=members, T=T, low=max(1, int(high * 0.3)),
                high=high, own=_log(rng, 1, 400), HQ=HKV * G, layers=layers, **both)


def _lengths(case, n):
    """n lengths of the case, spread over the logarithm of [low, high]; the first is high."""
    r = random.Random(case["lens"])
    return [case["high"] if i == 0 else _log(r, case["low"], case["high"]) for i in range(n)]


def _windows(case):
    """New tokens of each row of an append."""
    r = random.Random(case["lens"] + 7)
    T = case["T"]
    return [T if i == 0 or not case["ragged"] else _log(r, 1, T) for i in range(case["B"])]


def _rows(case):
    """Slots of a batch: row r has slot r but each (B // null)-th, which is null."""
    B, null = case["B"], case["null"]
    slot = list(range(B))
    for i in range(null):
        slot[i * (B // null)] = -1
    return slot


def _shared_lengths(case):
    """(shared prefix, all committed tokens) of each row; a group's rows are side by side."""
    r = random.Random(case["lens"] + 3)
    got = []
    for n in _lengths(case, case["groups"]):
        got += [(n, n + r.randrange(0, case["own"] + 1)) for _ in range(case["members"])]
    return got


# ------------------------------------------------------------------ inputs
def _gen(case, seed):
    return torch.Generator("cuda").manual_seed(seed * 1000003 + case["lens"])


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _ends(lens):
    return _ints([0] + [sum(lens[:i + 1]) for i in range(len(lens))])


def _normal(shape, dtype, gen, by=1.0):
    """N(0, by^2) in the type, drawn in slices of the first axis (a pool is large)."""
    x = torch.empty(shape, dtype=DTYPE[dtype], device="cuda")
    for i in range(x.shape[0]):
        x[i].normal_(0.0, by, generator=gen)
    return x


def _power(e):
    """2^e in fp32 for whole e in [-126, 127]."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantise(x):
    """e4m3 values and the power of two (its exponent + 127, a byte) of fp32 [..., D]."""
    top = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)
    m, k = torch.frexp(top)
    e = torch.where(m <= 0.875, k - 9, k - 8).clamp(-64, 63)  # top <= 448 2^e
    e = torch.where(top > 0, e, -64)
    y = (x * _power(-e)[..., None]).clamp(-448.0, 448.0)
    y = torch.where(torch.isinf(x), math.nan, y)
    return y.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _value(codes, scale):
    """What codes (bytes) stand for, in fp32."""
    return codes.view(torch.float8_e4m3fn).float() * _power(scale.int() - 127)[..., None]


def _cache(case, layers, slots, pages, max_pages):
    """A program's cache: KVCache, or the same buffers where it is not to be had."""
    shape = (layers, pages, case["HKV"], case["page"], case["D"])
    e4m3 = case["pages"] == "e4m3"
    if own:
        from linear_attention_state_rssm_gb300.store import KVCache
        return KVCache(layers, slots, case.get("HQ", case["HKV"]), case["HKV"], case["D"],
                       n_pages=pages, page_size=case["page"], max_pages=max_pages,
                       dtype=case["dtype"], page_dtype="e4m3" if e4m3 else None)
    z = dict(dtype=torch.int32, device="cuda")
    kind = torch.float8_e4m3fn if e4m3 else DTYPE[case["dtype"]]
    return SimpleNamespace(
        k_pages=torch.empty(shape, dtype=kind, device="cuda"),
        v_pages=torch.empty(shape, dtype=kind, device="cuda"),
        page_scales=torch.empty(shape[:4] + (2,), dtype=torch.uint8, device="cuda")
        if e4m3 else None,
        table=torch.full((slots, max_pages), -1, **z), held=torch.zeros(slots, **z),
        length=torch.zeros(slots, **z), refs=torch.zeros(pages, **z))


def _fill(case, c, gen):
    """Pages full of keys and values; those of e4m3 pages have sizes of their own per token."""
    for which, pool in enumerate((c.k_pages, c.v_pages)):
        for layer in range(pool.shape[0]):
            if case["pages"] != "e4m3":
                pool[layer].normal_(0.0, 1.0, generator=gen)
                continue
            for a in range(0, pool.shape[1], 512):
                part = pool[layer, a:a + 512]
                x = torch.empty(part.shape, device="cuda").normal_(0.0, 1.0, generator=gen)
                by = torch.empty(part.shape[:3], device="cuda").uniform_(0.5, 2.0, generator=gen)
                codes, scale = _quantise(x * by[..., None])
                part.view(torch.uint8).copy_(codes.view(torch.uint8))
                c.page_scales[layer, a:a + 512, ..., which] = scale


def _hand_out(c, counts, gen):
    """Gives slot i counts[i] pages, in a random order of the pool; the pages left over."""
    order = torch.randperm(c.refs.shape[0], generator=gen, device="cuda").int()
    most, n = c.table.shape[1], torch.tensor(counts, device="cuda")
    start = torch.cumsum(n, 0) - n
    at = torch.arange(most, device="cuda")
    take = (start[:, None] + at).clamp(max=c.refs.shape[0] - 1)
    c.table[:len(counts)] = torch.where(at < n[:, None], order[take], -1)
    c.held[:len(counts)] = n.int()
    c.refs.zero_()
    c.refs[order[:sum(counts)].long()] = 1


def _pages(tokens, page):
    return -(-tokens // page)


def prepare(case, seed):
    gen = _gen(case, seed)
    return {"append": _prepare_append, "decode": _prepare_decode, "gather": _prepare_gather,
            "shared": _prepare_shared}[case["op"]](case, gen)


def _prepare_append(case, gen):
    """q, k and v are views of one projection's output."""
    HQ, HKV, D, B = case["HQ"], case["HKV"], case["D"], case["B"]
    r = random.Random(case["lens"])
    new, slot = _windows(case), _rows(case)
    lens = [r.randrange(0, 3000) for _ in range(B)]
    counts = [_pages(n + t, case["page"]) for n, t in zip(lens, new)]
    s = SimpleNamespace(case=case, N=sum(new))
    s.cache = _cache(case, 1, B, sum(counts) + 2, max(counts))
    if case["pages"] != "e4m3":  # these are returned whole
        _fill(case, s.cache, gen)
    _hand_out(s.cache, counts, gen)
    s.cache.length.copy_(_ints(lens))
    s.slot, s.new = _ints(slot), _ints(new)
    s.cu = _ends(new) if case["ragged"] else None
    qkv = _normal((1, s.N, HQ + 2 * HKV, D), case["dtype"], gen, 1.5)[0]
    s.q, s.k, s.v = qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]
    s.q_out = torch.zeros((s.N, HQ, D), dtype=DTYPE[case["dtype"]], device="cuda")
    s.k_out = s.v_out = None
    if case["pages"] == "e4m3":
        s.k_out = torch.zeros((s.N, HKV, D), dtype=DTYPE[case["dtype"]], device="cuda")
        s.v_out = torch.zeros_like(s.k_out)
    s.q_weight, s.k_weight = (1.0 + 0.2 * _normal((1, D), "f32", gen)[0] for _ in range(2))
    P, A, most = case["rot"] // 2, case["axes"], 8192
    s.sections = [P - (A - 1) * (P // A)] + [P // A] * (A - 1)
    angle = torch.arange(most, dtype=torch.float64, device="cuda")[:, None] * \
        1e6 ** (-torch.arange(P, dtype=torch.float64, device="cuda") / P)
    s.table = torch.stack((angle.cos(), angle.sin()), 1).float().contiguous()
    s.positions = torch.randint(0, most, (A, s.N), generator=gen, device="cuda",
                                dtype=torch.int32)
    if own:
        from linear_attention_state_rssm_gb300.store import HeadNorm, RotaryTable
        s.rope = RotaryTable(s.table, s.sections)
        s.norm = HeadNorm(s.q_weight, s.k_weight, EPS)
    return s


def _prepare_decode(case, gen):
    B, T, page = case["B"], case["T"], case["page"]
    lens = _lengths(case, B)
    counts = [_pages(n + T, page) for n in lens]
    s = SimpleNamespace(case=case)
    s.cache = _cache(case, 1, B, sum(counts) + 3, max(counts))
    _fill(case, s.cache, gen)
    _hand_out(s.cache, counts, gen)
    s.cache.length.copy_(_ints(lens))
    s.slot = _ints(_rows(case))
    s.q = _normal((1, B * T, case["HQ"], case["D"]), case["dtype"], gen, 1.5)
    s.o = torch.zeros_like(s.q)
    s.most, s.scale = max(lens) + T, case["D"] ** -0.5
    return s


def _prepare_gather(case, gen):
    """Row r's tokens from `first` on (some of the rows' later tokens stay where they are)."""
    B, page = case["B"], case["page"]
    lens, slot = _lengths(case, B), _rows(case)
    counts = [_pages(case["first"] + n + i % 3, page) for i, n in enumerate(lens)]
    s = SimpleNamespace(case=case, N=sum(lens))
    s.cache = _cache(case, 1, B, sum(counts) + 3, max(counts))
    _fill(case, s.cache, gen)
    _hand_out(s.cache, counts, gen)
    s.cache.length.copy_(_ints([case["first"] + n for n in lens]))
    s.slot, s.cu = _ints(slot), _ends(lens)
    s.first = _ints([case["first"]] * B) if case["first"] else None
    s.k_out = torch.zeros((s.N, case["HKV"], case["D"]), dtype=DTYPE[case["dtype"]],
                          device="cuda")
    s.v_out = torch.zeros_like(s.k_out)
    return s


def _prepare_shared(case, gen):
    """Slots as a fork leaves them: the prefix's full pages are named by all of a group's
    tables, its partly filled last page by copies of each slot's own."""
    B, T, page = case["groups"] * case["members"], case["T"], case["page"]
    lens = _shared_lengths(case)
    counts = [_pages(n + T, page) for _, n in lens]
    s = SimpleNamespace(case=case)
    shared = [n // page for n, _ in lens]
    extra = sum(k for i, k in enumerate(shared) if i % case["members"])
    s.cache = _cache(case, case["layers"], B, sum(counts) - extra + 3, max(counts))
    _fill(case, s.cache, gen)
    free = iter(torch.randperm(s.cache.refs.shape[0], generator=gen, device="cuda").tolist())
    table, refs = [], [0] * s.cache.refs.shape[0]
    for i in range(B):
        lead = table[i - i % case["members"]] if i % case["members"] else []
        row = lead[:shared[i]] + [next(free) for _ in range(counts[i] - len(lead[:shared[i]]))]
        for x in row:
            refs[x] += 1
        table.append(row)
    s.cache.table.copy_(_ints([row + [-1] * (max(counts) - len(row)) for row in table]))
    s.cache.held.copy_(_ints(counts))
    s.cache.refs.copy_(_ints(refs))
    s.cache.length.copy_(_ints([n for _, n in lens]))
    s.slot = torch.arange(B, dtype=torch.int32, device="cuda")
    s.q = _normal((case["layers"], B * T, case["HQ"], case["D"]), case["dtype"], gen, 1.5)
    s.o = torch.zeros_like(s.q)
    s.most, s.scale = max(n for _, n in lens) + T, case["D"] ** -0.5
    if own:
        s.share = s.cache.new_share(B, T)
    return s


# --------------------------------------------------------------------- run
def run(state):
    return {"append": _run_append, "decode": _run_decode, "gather": _run_gather,
            "shared": _run_shared}[state.case["op"]](state)


def _axes(P, sections):
    """Axis of each pair: the first sections[0] pairs take axis 0, the next sections[1] axis 1."""
    ends = torch.tensor(sections, device="cuda").cumsum(0)
    return torch.bucketize(torch.arange(P, device="cuda"), ends, right=True)


def _norm(x, weight):
    x = x.float()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight


def _rotate(x, cos, sin):
    P = cos.shape[-1]
    a, b = x[..., :P], x[..., P:2 * P]
    cos, sin = cos[:, None], sin[:, None]
    return torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., 2 * P:]), -1)


def _run_append(s):
    c, T, page = s.cache, s.case["T"], s.case["page"]
    e4m3 = s.case["pages"] == "e4m3"
    if own:
        c.rssm_kv_append(0, s.q, s.k, s.v, s.slot, T, s.q_out, rope=s.rope,
                         positions=s.positions, cu_seqlens=s.cu, k_out=s.k_out, norm=s.norm,
                         v_out=s.v_out)
        return (s.q_out, s.k_out, s.v_out) if e4m3 else (s.q_out, c.k_pages, c.v_pages)
    P = s.table.shape[-1]
    row = s.table[s.positions.long()[_axes(P, s.sections)].t(), :, torch.arange(P, device="cuda")]
    cos, sin = row[..., 0], row[..., 1]
    q = _rotate(_norm(s.q, s.q_weight), cos, sin)
    k = _rotate(_norm(s.k, s.k_weight), cos, sin)
    of = torch.repeat_interleave(torch.arange(s.slot.shape[0], device="cuda"), s.new.long(),
                                 output_size=s.N)
    start = torch.cumsum(s.new.long(), 0) - s.new
    live = s.slot[of] >= 0
    slot = s.slot[of].clamp(min=0).long()
    at = c.length[slot].long() + torch.arange(s.N, device="cuda") - start[of]
    ids = c.table[slot, at // page].long()[live]
    off = (at % page)[live]
    s.q_out.copy_(torch.where(live[:, None, None], q.to(s.q_out.dtype), s.q_out))
    if not e4m3:
        c.k_pages[0, ids, :, off] = k[live].to(c.k_pages.dtype)
        c.v_pages[0, ids, :, off] = s.v[live]
        return s.q_out, c.k_pages, c.v_pages
    (kc, ks), (vc, vs) = _quantise(k), _quantise(s.v.float())
    kc, vc = kc.view(torch.uint8), vc.view(torch.uint8)
    c.k_pages.view(torch.uint8)[0, ids, :, off] = kc[live]
    c.v_pages.view(torch.uint8)[0, ids, :, off] = vc[live]
    c.page_scales[0, ids, :, off] = torch.stack((ks, vs), -1)[live]
    live = live[:, None, None]
    s.k_out.copy_(torch.where(live, _value(kc, ks).to(s.k_out.dtype), s.k_out))
    s.v_out.copy_(torch.where(live, _value(vc, vs).to(s.v_out.dtype), s.v_out))
    return s.q_out, s.k_out, s.v_out


def _paged(c, which, layer, ids, off):
    """Keys (which 0) or values of tokens, fp32, from pages `ids` and places `off` in them."""
    pool = (c.k_pages, c.v_pages)[which][layer]
    if c.page_scales is None:
        return pool[ids, :, off].float()
    return _value(pool.view(torch.uint8)[ids, :, off], c.page_scales[layer][ids, :, off, which])


def _softmax(scores, keep):
    """exp(s - max) / sum over the last axis where `keep`."""
    scores = torch.where(keep, scores, -math.inf)
    p = torch.exp(scores - scores.amax(-1, keepdim=True))
    return p / p.sum(-1, keepdim=True)


def _window(s, layer):
    """Attention of T new tokens of every row over its own pages."""
    c, T, page, HKV, D = s.cache, s.case["T"], s.case["page"], s.case["HKV"], s.case["D"]
    B, G = s.slot.shape[0], s.case["HQ"] // HKV
    live, slot = s.slot >= 0, s.slot.clamp(min=0).long()
    at = torch.arange(s.most, device="cuda")
    ids, off = c.table[slot][:, at // page].clamp(min=0).long(), at % page
    k = _paged(c, 0, layer, ids, off).permute(0, 2, 3, 1)
    q = s.q[layer].float().view(B, T, HKV, G, D).permute(0, 2, 3, 1, 4).flatten(2, 3)
    scores = (torch.matmul(q, k) * s.scale).unflatten(2, (G, T))
    del k
    last = c.length[slot][:, None] + torch.arange(T, device="cuda")
    p = _softmax(scores, (at <= last[:, :, None])[:, None, None]).flatten(2, 3)
    v = _paged(c, 1, layer, ids, off).permute(0, 2, 1, 3)
    o = torch.matmul(p, v).unflatten(2, (G, T)).permute(0, 3, 1, 2, 4)
    o = o.reshape(B, T, HKV * G, D)
    o = torch.where(live[:, None, None, None], o, 0.0)
    return o.reshape(B * T, HKV * G, D).to(s.o.dtype)


def _run_decode(s):
    if own:
        s.cache.rssm_attn_decode(0, s.q[0], s.slot, s.case["T"], s.o[0])
        return s.o[0]
    return _window(s, 0)


def _run_gather(s):
    c, page = s.cache, s.case["page"]
    if own:
        c.rssm_kv_gather(0, s.slot, s.k_out, s.v_out, cu_seqlens=s.cu, first=s.first)
        return s.k_out, s.v_out
    token = torch.arange(s.N, device="cuda")
    of = torch.bucketize(token, s.cu[1:].long(), right=True)
    live = (s.slot[of] >= 0)[:, None, None]
    slot = s.slot[of].clamp(min=0).long()
    at = token - s.cu[of] + (0 if s.first is None else s.first[of])
    ids, off = c.table[slot, at // page].long(), at % page
    k, v = _paged(c, 0, 0, ids, off), _paged(c, 1, 0, ids, off)
    s.k_out.copy_(torch.where(live, k.to(s.k_out.dtype), s.k_out))
    s.v_out.copy_(torch.where(live, v.to(s.v_out.dtype), s.v_out))
    return s.k_out, s.v_out


def _run_shared(s):
    """A step: the groups are found once, then each layer's attention."""
    c, T, layers = s.cache, s.case["T"], s.case["layers"]
    if own:
        c.rssm_kv_share(s.slot, T, s.share)
        for i in range(layers):
            c.rssm_attn_decode_shared(i, s.q[i], s.slot, T, s.share, s.o[i])
        return s.o
    return torch.stack([_window(s, i) for i in range(layers)])


# -------------------------------------------------------------------- work
def work(case):
    size, psize, D, HKV = SIZE[case["dtype"]], SIZE[case["pages"]], case["D"], case["HKV"]
    # a token's keys and values of all heads, as the pages hold them
    token = 2 * HKV * (D * psize + (case["pages"] == "e4m3"))
    if case["op"] == "append":
        N = sum(t for t, s in zip(_windows(case), _rows(case)) if s >= 0)
        out = 2 * HKV * D * size if case["pages"] == "e4m3" else 0
        return {"bytes": N * ((2 * case["HQ"] + 2 * HKV) * D * size + token + out
                              + 4 * case["axes"] + 4 * case["rot"]),
                "flops": N * (case["HQ"] + HKV) * (4 * D + 3 * case["rot"])}
    if case["op"] == "gather":
        N = sum(n for n, s in zip(_lengths(case, case["B"]), _rows(case)) if s >= 0)
        return {"bytes": N * (token + 2 * HKV * D * size), "flops": 0}
    T, HQ = case["T"], case["HQ"]
    if case["op"] == "decode":
        lens = [n for n, s in zip(_lengths(case, case["B"]), _rows(case)) if s >= 0]
        keys = sum(n + T for n in lens)
        layers, pages = 1, sum(_pages(n + T, case["page"]) for n in lens)
    else:
        both = _shared_lengths(case)
        whole = [n // case["page"] * case["page"] for n, _ in both]
        lens = [n for _, n in both]
        keys = sum(n + T for n in lens) - sum(w for i, w in enumerate(whole)
                                              if i % case["members"])
        layers, pages = case["layers"], keys // case["page"] + len(lens)
    pairs = sum(n * T + T * (T + 1) // 2 for n in lens)
    return {"bytes": layers * (keys * token + 2 * len(lens) * T * HQ * D * size + 4 * pages),
            "flops": layers * 4 * D * HQ * pairs}


# ------------------------------------------------------------------- exact
def exact(case, seed):
    """Outputs in 64 bits, row by row from the formulas; copied 16- and 32-bit pages have no
    such value."""
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, s)
    if case["op"] == "gather":
        return _exact_gather(case, s) if case["pages"] == "e4m3" else None
    if case["op"] == "decode":
        return _exact_window(case, s, 0, _lengths(case, case["B"]), _rows(case))
    lens = [n for _, n in _shared_lengths(case)]
    return torch.stack([_exact_window(case, s, i, lens, range(len(lens)))
                        for i in range(case["layers"])])


def _e4m3_table():
    """The 256 values: sign, four bits of exponent (bias 7), three of mantissa."""
    got = []
    for b in range(256):
        e, m = b >> 3 & 15, b & 7
        x = math.nan if b & 127 == 127 else \
            (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        got.append(-x if b & 128 else x)
    return torch.tensor(got, dtype=torch.float64, device="cuda")


def _exact_quantised(x):
    """The multiples of 2^e that the pages hold for finite 64-bit x [..., D]."""
    top = x.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -200)
    e = torch.ceil(torch.log2(top / 448)).clamp(-64, 63)
    y = x / 2.0 ** e
    step = 2.0 ** (torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(y / step) * step).clamp(-448, 448) * 2.0 ** e


def _exact_append(case, s):
    P, A = case["rot"] // 2, case["axes"]
    freq = 1e6 ** (-torch.arange(P, dtype=torch.float64) / P)
    axis = torch.tensor([a for a in range(A) for _ in range(s.sections[a])])
    angle = s.positions.cpu().double()[axis].t() * freq
    z = torch.polar(torch.ones_like(angle), angle).cuda()[:, None]
    live = (s.slot >= 0).repeat_interleave(s.new.long())[:, None, None]

    def turned(x, weight):
        x = x.double()
        x = x * weight.double() / torch.sqrt((x * x).sum(-1, keepdim=True) / case["D"] + EPS)
        y = torch.complex(x[..., :P], x[..., P:2 * P]) * z
        return torch.cat((y.real, y.imag, x[..., 2 * P:]), -1)

    q = torch.where(live, turned(s.q, s.q_weight), 0.0)
    if case["pages"] != "e4m3":
        return q, None, None
    return (q, torch.where(live, _exact_quantised(turned(s.k, s.k_weight)), 0.0),
            torch.where(live, _exact_quantised(s.v.double()), 0.0))


def _exact_row(case, c, which, layer, slot, n):
    """Keys or values of a slot's first n tokens, [HKV, n, D] in 64 bits."""
    ids = c.table[slot, :_pages(n, case["page"])].long()
    x = (c.k_pages, c.v_pages)[which][layer]
    if case["pages"] != "e4m3":
        return x[ids].transpose(0, 1).flatten(1, 2)[:, :n].double()
    codes = x.view(torch.uint8)[ids].transpose(0, 1).flatten(1, 2)[:, :n]
    scale = c.page_scales[layer][ids][..., which].transpose(0, 1).flatten(1, 2)[:, :n]
    return _e4m3_table()[codes.long()] * 2.0 ** (scale.double() - 127)[..., None]


def _exact_gather(case, s):
    got = [torch.zeros(s.k_out.shape, dtype=torch.float64, device="cuda") for _ in range(2)]
    at = 0
    for r, (n, slot) in enumerate(zip(_lengths(case, case["B"]), _rows(case))):
        for which in range(2 if slot >= 0 else 0):
            x = _exact_row(case, s.cache, which, 0, slot, case["first"] + n)
            got[which][at:at + n] = x[:, case["first"]:].transpose(0, 1)
        at += n
    return got


def _exact_window(case, s, layer, lens, slots):
    T, HKV, D = case["T"], case["HKV"], case["D"]
    o = torch.zeros(s.o.shape[1:], dtype=torch.float64, device="cuda")
    for r, (n, slot) in enumerate(zip(lens, slots)):
        if slot < 0:
            continue
        k, v = (_exact_row(case, s.cache, i, layer, slot, n + T) for i in range(2))
        q = s.q[layer, r * T:r * T + T].double().unflatten(1, (HKV, -1)).permute(1, 2, 0, 3)
        x = q @ k[:, None].transpose(-1, -2) * s.scale          # [HKV, G, T, keys]
        seen = torch.arange(n + T, device="cuda") <= n + torch.arange(T, device="cuda")[:, None]
        x.masked_fill_(~seen, -math.inf)
        y = torch.softmax(x, -1) @ v[:, None]
        o[r * T:r * T + T] = y.permute(2, 0, 1, 3).reshape(T, -1, D)
    return o
