"""Attention of new tokens over prefixes that rows share, against the fp64 oracle.

Tolerances are those of the attention that reads every row for itself: the weights
are rounded to the input type (2^-8, 2^-11; over quantised pages to fp16), the
output once more; fp32 sums, the exponential and the two parts' common reference
add below 1e-4 of the mass sum_j p_j |v_j| (fp32 inputs, nothing rounded: 6e-5).
"""
import numpy as np
import pytest
import torch

from oracle import attention as ref
from oracle import quant

pytestmark = pytest.mark.gpu
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
REL = {"bf16": 2 * 2.0 ** -8 + 1e-4, "f16": 2 * 2.0 ** -11 + 2e-4, "f32": 6e-5}
LSE = 5e-5
SENTINEL = 7.0
KINDS = [("bf16", None), ("f16", None), ("f32", None), ("bf16", "e4m3"), ("f16", "e4m3")]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_attention_state_rssm_gb300 import build
    build.build()


def ints(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def draw(rng, shape, dtype, by=1.0):
    t = torch.from_numpy(by * rng.standard_normal(shape)).to(TORCH[dtype])
    return t.cuda(), t.double().numpy()


class Batch:
    """Slots by groups: (prefix tokens, own tokens of each member); a member's table begins
    with the pages that the prefix fills. Pages hold random tokens everywhere."""

    def __init__(self, rng, groups, T, HQ, HKV, D, dtype, pages, page, scale=None, powers=(-2, 2),
                 key_powers=(0, 0)):
        from linear_attention_state_rssm_gb300.store import KVCache
        self.T, self.dtype = T, dtype
        self.lens, self.tables, used = [], [], 0
        for prefix, owns in groups:
            whole = prefix // page
            shared = list(range(used, used + whole))
            used += whole
            for own in owns:
                n = -(-(prefix + own + T) // page) - whole
                self.tables.append(shared + list(range(used, used + n)))
                used += n
                self.lens.append(prefix + own)
        n_pages = used + 2
        order = rng.permutation(n_pages)
        self.tables = [[int(order[i]) for i in t] for t in self.tables]
        most = max(len(t) for t in self.tables) + 1
        c = self.c = KVCache(n_layers=2, n_slots=len(self.lens), HQ=HQ, HKV=HKV, D=D,
                             n_pages=n_pages, page_size=page, max_pages=most, dtype=dtype,
                             page_dtype=pages, scale=scale)
        for s, t in enumerate(self.tables):
            c.table[s, :len(t)] = ints(t)
            c.held[s], c.length[s] = len(t), self.lens[s]
            for i in t:
                c.refs[i] += 1
        self.values = []
        for which, pool in enumerate((c.k_pages, c.v_pages)):
            x = 1.2 * rng.standard_normal((n_pages, HKV, page, D))
            if pages is None:
                t = torch.from_numpy(x).to(TORCH[dtype])
                pool[1] = t.cuda()
                self.values.append(t.double().numpy())
            else:
                lo, hi = powers if which else key_powers
                x = x * 2.0 ** rng.uniform(lo, hi, x.shape[:3])[..., None]
                codes, scale_ = quant.quantise(x)
                pool[1].view(torch.uint8).copy_(torch.from_numpy(codes))
                c.page_scales[1, ..., which] = torch.from_numpy(scale_).cuda()
                self.values.append(quant.value(codes, scale_))

    def tokens(self, s):
        n = self.lens[s] + self.T
        return tuple(v[self.tables[s]].transpose(0, 2, 1, 3).reshape(-1, *v.shape[1:2],
                                                                      v.shape[3])[:n]
                     for v in self.values)

    def want(self, qd, slots):
        return ref.window(qd, [None if s < 0 else self.tokens(s) for s in slots],
                          [self.lens[s] for s in slots], self.T, self.c.scale)


def check(got, want, mass, dtype):
    got = got.double().cpu().numpy()
    floor = 1e-7 if dtype == "f32" else {"f16": 2.0 ** -24, "bf16": 2.0 ** -126}[dtype]
    off, lim = np.abs(got - want), REL[dtype] * mass + floor   # the types' smallest steps
    assert np.all(off <= lim), (off / lim).max()


def run(kind, groups, T, HQ, HKV, D, page, seed, null=(), shuffle=True, strided=False, by=1.2, **kw):
    dtype, pages = kind
    rng = np.random.default_rng([seed, D, T, HQ])
    b = Batch(rng, groups, T, HQ, HKV, D, dtype, pages, page, **kw)
    B = len(b.lens)
    q, qd = draw(rng, (B * T, HQ + (2 if strided else 0), D), dtype, by)
    q, qd = q[:, :HQ], qd[:, :HQ]
    perm = rng.permutation(B) if shuffle else np.arange(B)
    slots = [-1 if r in null else int(perm[r]) for r in range(B)]
    o = torch.full((B * T, HQ, D), SENTINEL, dtype=TORCH[dtype], device="cuda")
    lse = torch.full((B * T, HQ), SENTINEL, device="cuda")
    share = b.c.new_share(B, T)
    b.c.rssm_kv_share(ints(slots), T, share)
    b.c.rssm_attn_decode_shared(1, q, ints(slots), T, share, o, lse=lse)
    assert b.c.rssm_kv_get_device_error() == 0
    want, wlse, mass = b.want(qd, slots)
    on = np.repeat(np.array(slots) >= 0, T)
    off = torch.from_numpy(~on)
    assert (o[off] == SENTINEL).all() and (lse[off] == SENTINEL).all()
    check(o[~off], want[on], mass[on], dtype)
    gl = lse.double().cpu().numpy()[on]
    assert np.all(np.abs(gl - wlse[on]) <= LSE + 1e-6 * np.abs(wlse[on]))
    for _ in range(2):   # the same sums whatever the order of arrival, or of a plan's members
        again = torch.empty_like(o)
        b.c.rssm_kv_share(ints(slots), T, share)
        b.c.rssm_attn_decode_shared(1, q, ints(slots), T, share, again)
        assert torch.equal(again[~off], o[~off])
    assert int(b.c.work[:1216].sum()) == 0
    return b, share


def plan(share, B):
    """n groups and every row's prefix, as the plan has them."""
    x = share.buffer.view(torch.int32).cpu().numpy()
    up = -(-4 * B // 256) * 64
    return int(x[2]), x[64:64 + B].tolist(), x[64 + up:64 + up + B].tolist()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,HQ,HKV", [(1, 4, 1), (1, 3, 3), (3, 8, 2), (16, 4, 1), (1, 40, 2)])
def test_groups_of_many_shapes(kind, D, T, HQ, HKV):
    groups = [(64, [0, 1, 17, 200]), (33, [5, 0]), (1000, [3, 40, 15]), (0, [50]), (15, [3, 4]),
              (16, [0, 0, 0]), (500, [90])]
    b, share = run(kind, groups, T, HQ, HKV, D, 16, 41, null=(4,))
    assert plan(share, len(b.lens))[0] in (3, 4)   # the null row may empty a pair


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("kind", [("bf16", None), ("bf16", "e4m3")])
def test_page_sizes(page, kind):
    groups = [(page, [0, 1]), (5 * page + 3, [page, 2, 9]), (page - 1, [4, 5]),
              (2 * page, [0, 3 * page])]
    b, share = run(kind, groups, 2, 8, 2, 128, page, 42, shuffle=False)
    n, prefix, _ = plan(share, len(b.lens))
    assert n == 3 and prefix == [page] * 2 + [5 * page] * 3 + [0] * 2 + [2 * page] * 2


@pytest.mark.parametrize("kind,D", [(("bf16", None), 128), (("f16", None), 256),
                                    (("f32", None), 64), (("bf16", "e4m3"), 128),
                                    (("f16", "e4m3"), 64)])
def test_long_prefixes_are_split_and_joined(kind, D):
    run(kind, [(20000, [3, 0, 700]), (64, [9000])], 1, 4, 1, D, 64, 43)


@pytest.mark.parametrize("kind", [("bf16", None), ("bf16", "e4m3"), ("f32", None)])
def test_groups_of_many_rows(kind):
    """More query rows than a block has, and more rows than the plan has threads."""
    run(kind, [(300, list(range(70)))], 3, 4, 1, 64, 32, 44)
    rng = np.random.default_rng(45)
    groups = [(int(n), [int(x) for x in rng.integers(0, 30, m)])
              for n, m in zip(rng.integers(0, 90, 300), rng.integers(1, 8, 300))]
    run(kind, groups, 1, 2, 1, 64, 16, 46, null=(0, 7, 1000))


@pytest.mark.parametrize("powers", [(-60, -45), (-12, 12), (-25, 25), (30, 50)])
def test_quantised_values_of_very_different_sizes(powers):
    """Powers of two far apart within a step of a prefix, and from step to step."""
    run(("bf16", "e4m3"), [(700, [0, 40, 3]), (300, [5, 60])], 2, 4, 2, 64, 16, 58, powers=powers)


@pytest.mark.parametrize("by,keys", [(1e-20, (40, 60)), (1e20, (-75, -65)), (0.3, (-9, 3)),
                                     (0.0, (0, 0))])
def test_quantised_keys_and_queries_of_very_different_sizes(by, keys):
    run(("bf16", "e4m3"), [(700, [0, 40, 3]), (300, [5, 60])], 2, 4, 2, 128, 16, 59, by=by,
        key_powers=keys)


def test_nothing_shared_and_one_row():
    b, share = run(("bf16", None), [(100, [0]), (64, [1]), (0, [0])], 1, 4, 2, 64, 16, 47)
    assert plan(share, 3)[0] == 0
    run(("bf16", "e4m3"), [(300, [2])], 1, 4, 2, 64, 16, 48, strided=True)
    run(("bf16", None), [(64, [0, 0])], 1, 4, 2, 64, 16, 49, null=(0, 1))


def test_a_slot_named_twice():
    rng = np.random.default_rng(50)
    b = Batch(rng, [(100, [5]), (40, [3])], 1, 4, 2, 64, "bf16", None, 16)
    q, qd = draw(rng, (4, 4, 64), "bf16")
    slots = [0, 1, 0, 0]
    share, o = b.c.new_share(4), torch.zeros_like(q)
    b.c.rssm_kv_share(ints(slots), 1, share)
    n, prefix, group = plan(share, 4)
    assert n == 1 and prefix == [96, 0, 96, 96] and [group[i] for i in (0, 2, 3)] == [0, 0, 0]
    b.c.rssm_attn_decode_shared(1, q, ints(slots), 1, share, o)
    want, _, mass = b.want(qd, slots)
    check(o, want, mass, "bf16")


@pytest.mark.parametrize("pages", [None, "e4m3"])
def test_forks_growth_and_compaction_under_one_plan(pages):
    """Slots forked (and forked again) from prompts; the plan stays true while they grow and
    while pages move, and results stay those of the unshared attention."""
    from linear_attention_state_rssm_gb300.store import KVCache
    rng = np.random.default_rng(51)
    HQ, HKV, D, page = 4, 2, 64, 16
    c = KVCache(n_slots=12, HQ=HQ, HKV=HKV, D=D, n_pages=200, page_size=page, max_pages=20,
                page_dtype=pages)

    def new(slots, T):
        k, v = (draw(rng, (len(slots) * T, HKV, D), "bf16")[0] for _ in range(2))
        c.rssm_kv_reserve(ints(slots), T)
        c.rssm_kv_append(0, None, k, v, ints(slots), T)
    new([0, 1], 75)
    c.rssm_kv_commit(ints([0, 1]), 75)
    c.rssm_kv_fork(ints([0, 0, 0, 1, 1]), ints([2, 3, 4, 5, 6]))
    new([2], 40)
    c.rssm_kv_commit(ints([2]), 40)
    c.rssm_kv_fork(ints([2, 2]), ints([7, 8]))
    c.rssm_kv_release(ints([1]))
    rows = [8, 5, 0, 3, 6, 7, 4, 2]
    share = c.new_share(8, 2)
    for step in range(6):
        new(rows, 2)
        if step == 0:
            c.rssm_kv_share(ints(rows), 2, share)
            n, prefix, _ = plan(share, 8)
            assert n == 2 and prefix == [64] * 8
        if step == 3:
            c.rssm_kv_release(ints([9, 10]))
            c.rssm_kv_compact()
        q = draw(rng, (16, HQ, D), "bf16")[0]
        a, b = torch.zeros_like(q), torch.zeros_like(q)
        c.rssm_attn_decode_shared(0, q, ints(rows), 2, share, a)
        c.rssm_attn_decode(0, q, ints(rows), 2, b)
        assert c.rssm_kv_get_device_error() == 0
        assert (a.float() - b.float()).abs().max() <= 2 * REL["bf16"] * 6.0
        c.rssm_kv_commit(ints(rows), 2)


def test_plans_that_no_longer_hold_skip_their_rows():
    from linear_attention_state_rssm_gb300 import _lib as lib
    rng = np.random.default_rng(52)
    b = Batch(rng, [(64, [0, 5, 20]), (32, [1, 2])], 1, 4, 2, 64, "bf16", None, 16)
    c, B = b.c, 5
    q, qd = draw(rng, (B, 4, 64), "bf16")
    slot = ints(range(B))
    want, _, mass = b.want(qd, list(range(B)))
    share = c.new_share(B)

    def call(slots=None, buffer=None):
        o = torch.full_like(q, SENTINEL)
        c.rssm_attn_decode_shared(1, q, slot if slots is None else ints(slots), 1, share, o)
        left = (o == SENTINEL).all(-1).all(-1)
        fine = (~left).cpu()
        check(o[fine], want[fine.numpy()], mass[fine.numpy()], "bf16")
        return c.rssm_kv_get_device_error(), left.tolist()

    assert call() == (lib.DEVERR["pages"], [True] * B)     # no plan yet
    c.rssm_kv_share(slot, 1, share)
    assert call() == (0, [False] * B)
    was = c.table[1].clone()
    c.table[1, 2] = 99 % c.n_pages if int(was[2]) != 99 % c.n_pages else 0
    err, left = call()                                     # another page in the middle
    assert err == lib.DEVERR["pages"] and left == [False, True, False, False, False]
    c.table[1] = was
    n = int(c.length[2])
    c.length[2] = 63                                       # shorter than the prefix
    err, left = call()
    assert err == lib.DEVERR["pages"] and left == [False, False, True, False, False]
    c.length[2] = n
    err, left = call([0, -1, 2, -1, 4])                    # rows that ended
    assert err == 0 and left == [False, True, False, True, False]
    assert call([-1, 1, 2, 3, 4]) == (0, [True, False, False, False, False])   # the first one
    assert call([-1, -1, -1, 3, 4]) == (0, [True, True, True, False, False])   # a whole group
    assert call([-1] * 5) == (0, [True] * 5)
    c.rssm_kv_share(ints([-1, 1, 2, 3, 4]), 1, share)
    assert call([-1, 1, 2, 3, 4]) == (0, [True, False, False, False, False])
    # a buffer of another plan's sizes, past the Python layer's check
    other = c.new_share(B, 2)
    o = torch.full_like(q, SENTINEL)
    c.rssm_kv_share(slot, 2, other)
    assert c.rssm_kv_get_device_error() == 0
    lib.rssm_attn_decode_shared(c.handle, 1, q, 256, slot, B, 1, other.buffer, o, None)
    assert c.rssm_kv_get_device_error() == lib.DEVERR["pages"] and (o == SENTINEL).all()


def test_refusals():
    from linear_attention_state_rssm_gb300 import _lib as lib
    rng = np.random.default_rng(53)
    b = Batch(rng, [(64, [0, 5])], 1, 4, 2, 64, "bf16", None, 16)
    c, slot = b.c, ints([0, 1])
    q = draw(rng, (2, 4, 64), "bf16")[0]
    share, o = c.new_share(2), torch.zeros_like(q)
    for bad in (c.new_share(3), c.new_share(2, 2)):
        with pytest.raises(ValueError):
            c.rssm_kv_share(slot, 1, bad)
        with pytest.raises(ValueError):
            c.rssm_attn_decode_shared(1, q, slot, 1, bad, o)
    b2 = Batch(rng, [(64, [0, 5])], 1, 4, 2, 64, "bf16", None, 16)
    with pytest.raises(ValueError):
        c.rssm_kv_share(slot, 1, b2.c.new_share(2))
    with pytest.raises(ValueError):
        c.rssm_attn_decode_shared(1, q[:1], slot, 1, share, o)
    with pytest.raises(lib.RssmError):
        c.rssm_attn_decode_shared(2, q, slot, 1, share, o)
    with pytest.raises(lib.RssmError):
        c.new_share(2, 65)
    with pytest.raises(lib.RssmError):
        lib.rssm_kv_share(c.handle, slot, 2, 1, share.buffer[8:])
    with pytest.raises(lib.RssmError):
        lib.rssm_attn_decode_shared(c.handle, 1, q, 256, slot, 2, 1, None, o, None)
    # slots that are refused: left out by the plan, told by the attention
    bad = ints([0, 9])
    c.rssm_kv_share(bad, 1, share)
    assert c.rssm_kv_get_device_error() == 0
    o.fill_(SENTINEL)
    c.rssm_attn_decode_shared(1, q, bad, 1, share, o)
    assert c.rssm_kv_get_device_error() == lib.DEVERR["slot"]
    assert (o[1] == SENTINEL).all() and (o[0] != SENTINEL).any()
    empty = c.new_share(0)
    c.rssm_kv_share(ints([]), 1, empty)
    c.rssm_attn_decode_shared(1, q[:0], ints([]), 1, empty, o[:0])


@pytest.mark.parametrize("kind", [("bf16", None), ("f32", None), ("bf16", "e4m3")])
def test_poison_reaches_only_those_who_see_it(kind):
    """A NaN in a row's own tokens, and one in a group's prefix."""
    dtype, pages = kind
    rng = np.random.default_rng(54)
    T = 4
    b = Batch(rng, [(64, [0, 5, 20]), (48, [1, 2])], T, 4, 2, 64, dtype, pages, 16)
    c, slot = b.c, ints(range(5))
    q = draw(rng, (5 * T, 4, 64), dtype)[0]
    share = c.new_share(5, T)
    c.rssm_kv_share(slot, T, share)
    clean, dirty = torch.zeros_like(q), torch.zeros_like(q)
    c.rssm_attn_decode_shared(1, q, slot, T, share, clean)

    def poison(s, at):
        pg = b.tables[s][at // 16]
        for pool in (c.k_pages, c.v_pages):
            if pages:
                pool.view(torch.uint8)[1, pg, :, at % 16] = 127
            else:
                pool[1, pg, :, at % 16] = float("nan")
    poison(1, b.lens[1] + 2)                      # a rejected draft of row 1
    poison(3, 17)                                 # in the second group's prefix
    c.rssm_attn_decode_shared(1, q, slot, T, share, dirty)
    rows = dirty.view(5, T, -1).float()
    fine = torch.isfinite(rows).all(-1)
    want = torch.ones(5, T, dtype=torch.bool, device="cuda")
    want[1, 2:], want[3:] = False, False
    assert torch.equal(fine, want)
    ref_rows = clean.view(5, T, -1).float()
    assert (rows[want] - ref_rows[want]).abs().max() <= 2 * REL[dtype] * 24.0
    assert torch.equal(rows[[0, 2]], ref_rows[[0, 2]])


@pytest.mark.parametrize("kind", [("bf16", None), ("bf16", "e4m3")])
def test_waits_that_run_out(kind):
    """What is stored is right; a prefix that was lost keeps its rows out until the next
    plan; the call after is right."""
    from linear_attention_state_rssm_gb300 import _lib as lib
    rng = np.random.default_rng(55)
    b = Batch(rng, [(6400, [0, 300]), (0, [3000])], 1, 4, 1, 128, *kind, 64)
    c, slot = b.c, ints([0, 1, 2])
    q, qd = draw(rng, (3, 4, 128), "bf16")
    want, _, mass = b.want(qd, [0, 1, 2])
    share = c.new_share(3)
    c.rssm_kv_share(slot, 1, share)

    def call():
        o = torch.full_like(q, SENTINEL)
        c.rssm_attn_decode_shared(1, q, slot, 1, share, o)
        left = (o == SENTINEL).all(-1).all(-1).cpu().numpy()
        check(o[torch.from_numpy(~left)], want[~left], mass[~left], "bf16")
        return c.rssm_kv_get_device_error(), left
    for cta, unit in ((0, 0), (1, 1)):
        c.rssm_kv_debug_withhold(cta, unit)
        err, left = call()
        assert err == lib.DEVERR["timeout"] and left[:2].all()
        c.rssm_kv_debug_withhold(-1)
        err, left = call()                        # still the lost plan
        assert err == lib.DEVERR["timeout"] and left.tolist() == [True, True, False]
        c.rssm_kv_share(slot, 1, share)
        err, left = call()
        assert err == 0 and not left.any()


def test_in_a_graph_and_on_a_stream():
    """Two captured graphs with plans of their own over one cache, replayed in turn as the
    slots grow; the plan is part of one of them."""
    rng = np.random.default_rng(56)
    b = Batch(rng, [(64, [0, 5, 20]), (200, [1, 2])], 2, 4, 2, 128, "bf16", "e4m3", 16)
    c = b.c
    c.length.sub_(2)                              # room for what they grow by
    sets = []
    for rows in ([0, 1, 2, 3, 4], [4, 3, 1, 0]):
        n = len(rows)
        q = draw(rng, (2 * n, 4, 128), "bf16")[0]
        sets.append((ints(rows), q, torch.zeros_like(q), c.new_share(n, 2)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for i, (slot, q, o, share) in enumerate(sets):
            c.rssm_kv_share(slot, 2, share)
            c.rssm_attn_decode_shared(1, q, slot, 2, share, o)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                if i == 0:
                    c.rssm_kv_share(slot, 2, share)
                c.rssm_attn_decode_shared(1, q, slot, 2, share, o)
            graphs.append(g)
    torch.cuda.current_stream().wait_stream(side)
    for step in range(3):
        for g, (slot, q, o, share) in zip(graphs, sets):
            q.copy_(draw(rng, q.shape, "bf16")[0])
            o.zero_()
            g.replay()
            plain = torch.zeros_like(o)
            c.rssm_attn_decode(1, q, slot, 2, plain)
            assert (o.float() - plain.float()).abs().max() <= 2 * REL["bf16"] * 24.0
            assert c.rssm_kv_get_device_error() == 0
        c.length.add_(1)                          # other lengths than when captured


def test_a_step_of_all_together():
    """Prompts with normed and turned keys into quantised pages, attended over in a row;
    forks; a shared step; a second chunk of a prompt whose first part is gathered."""
    from linear_attention_state_rssm_gb300.store import HeadNorm, KVCache, RotaryTable
    rng = np.random.default_rng(57)
    HQ, HKV, D, page, eps = 4, 2, 64, 16, 1e-6
    c = KVCache(n_slots=6, HQ=HQ, HKV=HKV, D=D, n_pages=80, page_size=page, max_pages=16,
                page_dtype="e4m3")
    (qw, qwd), (kw, kwd) = (draw(rng, D, "f32") for _ in range(2))
    norm, rope = HeadNorm(qw, kw, eps), RotaryTable.from_base(256, 32)
    freq = 1e4 ** (-np.arange(32) / 32)
    cached = {}                                   # slot -> (k, v) in 64 bits, as the pages hold

    def turned(x, w, at):
        return ref.rotate(quant.norm(x, w, eps), np.asarray(at, float)[None], freq,
                          np.zeros(32, int))

    def append(slots, T, starts):
        (x, xd) = draw(rng, (len(slots) * T, HQ + 2 * HKV, D), "bf16")
        q_out = torch.zeros(len(slots) * T, HQ, D, device="cuda").bfloat16()
        k_out, v_out = (torch.zeros(len(slots) * T, HKV, D, device="cuda").bfloat16()
                        for _ in range(2))
        c.rssm_kv_reserve(ints(slots), T)
        c.rssm_kv_append(0, x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], ints(slots), T, q_out,
                         rope=rope, norm=norm, k_out=k_out, v_out=v_out)
        at = np.concatenate([n + np.arange(T) for n in starts])
        want = turned(xd[:, :HQ], qwd, at)
        assert np.abs(q_out.double().cpu().numpy() - want).max() <= 2.0 ** -7 * np.abs(want).max()
        want = turned(xd[:, HQ:HQ + HKV], kwd, at)
        got = k_out.double().cpu().numpy()
        # half a step of e4m3, and of bf16 on what it stands for
        assert np.all(np.abs(got - want) <= 2.0 ** -4 * np.abs(want)
                      + 2.0 ** -9 * np.abs(want).max(-1, keepdims=True))
        return q_out, k_out, v_out

    def grow(s, k, v):
        old = cached.get(s)
        k, v = k.double().cpu().numpy(), v.double().cpu().numpy()
        cached[s] = (k, v) if old is None else tuple(np.concatenate(x) for x in zip(old, (k, v)))

    n = 70
    q, k, v = append([0, 1], n, [0, 0])
    o = torch.zeros_like(q)
    c.rssm_attn_prefill(q, k, v, ints([0, n, 2 * n]), None, o)
    c.rssm_kv_commit(ints([0, 1]), n)
    for r in range(2):
        grow(r, k[r * n:r * n + n], v[r * n:r * n + n])
    cu = np.array([0, n, 2 * n])
    want, _, mass = ref.prompt(q.double().cpu().numpy(), k.double().cpu().numpy(),
                               v.double().cpu().numpy(), cu, cu, c.scale)
    check(o, want, mass, "bf16")
    # parallel samples
    c.rssm_kv_fork(ints([0, 0, 1]), ints([2, 3, 4]))
    for d, s in ((2, 0), (3, 0), (4, 1)):
        cached[d] = cached[s]
    rows, T = [0, 2, 3, 1, 4], 2
    share = c.new_share(5, T)
    for step in range(3):
        q, k, v = append(rows, T, [len(cached[s][0]) for s in rows])
        if step == 0:
            c.rssm_kv_share(ints(rows), T, share)
        o = torch.zeros_like(q)
        c.rssm_attn_decode_shared(0, q, ints(rows), T, share, o)
        c.rssm_kv_commit(ints(rows), T)
        lens = [len(cached[s][0]) for s in rows]
        for r, s in enumerate(rows):
            grow(s, k[r * T:r * T + T], v[r * T:r * T + T])
        want, _, mass = ref.window(q.double().cpu().numpy(), [cached[s] for s in rows], lens, T,
                                   c.scale)
        check(o, want, mass, "bf16")
    # slot 3's next 30 tokens as a prompt after what the cache holds
    m = len(cached[3][0])
    keys, vals = (torch.zeros(m + 30, HKV, D, device="cuda").bfloat16() for _ in range(2))
    q, k, v = append([3], 30, [m])
    c.rssm_kv_gather(0, ints([3]), keys, vals, T=m + 30)
    assert torch.equal(keys[m:], k) and torch.equal(vals[m:], v)
    o = torch.zeros_like(q)
    c.rssm_attn_prefill(q, keys, vals, ints([0, 30]), None, o, cu_keys=ints([0, m + 30]))
    grow(3, k, v)
    assert np.array_equal(keys.double().cpu().numpy(), cached[3][0])
    want, _, mass = ref.prompt(q.double().cpu().numpy(), *cached[3], np.array([0, 30]),
                               np.array([0, m + 30]), c.scale)
    check(o, want, mass, "bf16")
    assert c.rssm_kv_get_device_error() == 0


def test_plans_of_another_cache_are_refused():
    """The same rows and tokens, other heads, sizes of heads or pages: every row is skipped,
    and none of the plan's places is used."""
    from linear_attention_state_rssm_gb300 import _lib as lib
    rng = np.random.default_rng(60)
    sizes = [(4, 2, 64, 16), (8, 2, 64, 16), (8, 1, 64, 16), (4, 2, 128, 16), (4, 2, 64, 32)]
    caches = [Batch(rng, [(64, [0, 5, 20])], 2, HQ, HKV, D, "bf16", None, page).c
              for HQ, HKV, D, page in sizes]
    most = max(lib.rssm_kv_share_bytes(c.cfg, 3, 2) for c in caches)
    slot = ints(range(3))
    for of in caches:
        buffer = torch.zeros(most, dtype=torch.uint8, device="cuda")
        lib.rssm_kv_share(of.handle, slot, 3, 2, buffer)
        for c in caches:
            q = draw(rng, (6, c.HQ, c.D), "bf16")[0]
            o = torch.full_like(q, SENTINEL)
            lib.rssm_attn_decode_shared(c.handle, 1, q, c.HQ * c.D, slot, 3, 2, buffer, o, None)
            err = c.rssm_kv_get_device_error()
            if c is of:
                assert err == 0 and not (o == SENTINEL).all(-1).any()
            else:
                assert err == lib.DEVERR["pages"] and (o == SENTINEL).all()


@pytest.mark.parametrize("kind", [("bf16", None), ("f16", "e4m3"), ("f32", None)])
def test_the_longest_windows_with_the_most_heads(kind):
    run(kind, [(64, [0, 3]), (16, [1])], 64, 64, 1, 64, 16, 61)


@pytest.mark.parametrize("kind", [("bf16", None), ("bf16", "e4m3"), ("f32", None)])
def test_pools_past_32_bit_offsets(kind):
    from linear_attention_state_rssm_gb300.store import KVCache
    dtype, pages = kind
    D, HKV, page = 256, 4, 256
    n = (1 << 32) // (HKV * page * D) + 40        # past 2^32 values, and bytes
    c = KVCache(n_slots=2, HQ=2 * HKV, HKV=HKV, D=D, n_pages=n, page_size=page, max_pages=3,
                dtype=dtype, page_dtype=pages)
    for s in range(2):
        c.table[s] = ints([n - 1, n - 3, n - 5 - s])
    c.held[:] = 3
    rng = np.random.default_rng(62)
    (k, kd), (v, vd) = (draw(rng, (2 * 600, HKV, D), dtype) for _ in range(2))
    q, qd = draw(rng, (2, 2 * HKV, D), dtype)
    c.rssm_kv_append(0, None, k[:600], v[:600], ints([0]), cu_seqlens=ints([0, 600]))
    c.length[1] = 512
    c.rssm_kv_append(0, None, k[1112:], v[1112:], ints([1]), cu_seqlens=ints([0, 88]))
    c.length[:] = 599
    share, o = c.new_share(2), torch.zeros_like(q)
    c.rssm_kv_share(ints([0, 1]), 1, share)
    assert plan(share, 2)[:2] == (1, [512, 512])
    c.rssm_attn_decode_shared(0, q, ints([0, 1]), 1, share, o)
    assert c.rssm_kv_get_device_error() == 0
    kv = [quant.value(*quant.quantise(x)) if pages else x for x in (kd, vd)]
    rows = [tuple(x[:600] for x in kv), tuple(np.concatenate([x[:512], x[1112:]]) for x in kv)]
    want, _, mass = ref.window(qd, rows, [599, 599], 1, c.scale)
    check(o, want, mass, dtype)


@pytest.mark.parametrize("kind,own", [(("bf16", None), [3, 40, 0]), (("bf16", "e4m3"), [700, 1500, 3]),
                                      (("f32", None), [3, 40, 0])])
def test_calls_that_follow_one_another_closely(kind, own):
    """Layers that use one plan's room in turn, with nothing between them: each answers as
    it does alone, bit for bit."""
    rng = np.random.default_rng(63)
    b = Batch(rng, [(2000, own), (64, [0, 1]), (0, [30])], 1, 8, 2, 128, kind[0], kind[1], 16)
    B = len(b.lens)
    slot, share = ints(range(B)), b.c.new_share(B)
    b.c.rssm_kv_share(slot, 1, share)
    qs = [draw(rng, (B, 8, 128), kind[0])[0] for _ in range(5)]
    alone = []
    for q in qs:
        alone.append(torch.empty_like(q))
        torch.cuda.synchronize()
        b.c.rssm_attn_decode_shared(1, q, slot, 1, share, alone[-1])
        torch.cuda.synchronize()
    close = [torch.empty_like(qs[0]) for _ in range(60)]
    for i, o in enumerate(close):
        b.c.rssm_attn_decode_shared(1, qs[i % 5], slot, 1, share, o)
    g, replayed = torch.cuda.CUDAGraph(), [torch.empty_like(q) for q in qs]
    with torch.cuda.graph(g):
        for q, o in zip(qs, replayed):
            b.c.rssm_attn_decode_shared(1, q, slot, 1, share, o)
    g.replay()
    g.replay()
    for i, o in enumerate(close):
        assert torch.equal(o, alone[i % 5])
    assert all(torch.equal(x, y) for x, y in zip(replayed, alone))
    assert b.c.rssm_kv_get_device_error() == 0
