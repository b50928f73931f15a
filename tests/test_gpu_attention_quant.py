"""Attention of new tokens over quantised pages against the fp64 oracle on the
values that the codes stand for.

Tolerances. Queries pass into fp16 whole (scaled by a power of two a row), codes
are fp16 values, so scores are off by their fp32 sums alone. The weights are
rounded to fp16 (2^-11 of each; those under 2^-28 of the largest by 2^-39 of it)
and the output once to its type (2^-8 or 2^-11); fp32 sums of up to some ten
thousand terms and the base-2 exponential add below 1e-4 of the mass sum_j p_j
|v_j|.
"""
import numpy as np
import pytest
import torch

from oracle import attention as ref
from oracle import quant

pytestmark = pytest.mark.gpu
TORCH = {"bf16": torch.bfloat16, "f16": torch.float16}
REL = {"bf16": 2.0 ** -8 + 2.0 ** -11 + 1e-4, "f16": 2 * 2.0 ** -11 + 1e-4}
FLOOR = {"bf16": 2.0 ** -126, "f16": 2.0 ** -24}   # the types' smallest steps
LSE = 5e-5
SENTINEL = 7.0


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


def filled(rng, lens, T, HQ, HKV, D, dtype, page, extra=2, powers=(-3, 3), sized=None, **kw):
    """A cache whose slots hold random quantised tokens in shuffled pages, each token and
    head with a size of its own; places that hold no token have the code NaN and a power
    that no token has. sized(which, slot) -> factors of the tokens."""
    from linear_attention_state_rssm_gb300.store import KVCache
    counts = [-(-(n + T) // page) for n in lens]
    c = KVCache(n_layers=2, n_slots=len(lens), HQ=HQ, HKV=HKV, D=D, n_pages=sum(counts) + extra,
                page_size=page, max_pages=max(counts) + 1, dtype=dtype, page_dtype="e4m3", **kw)
    c.k_pages.view(torch.uint8).fill_(127)
    c.v_pages.view(torch.uint8).fill_(127)
    c.page_scales.fill_(255)
    order = rng.permutation(sum(counts) + extra)
    tokens, at = [], 0
    pools = (c.k_pages.view(torch.uint8), c.v_pages.view(torch.uint8))
    for s, n in enumerate(lens):
        ids = order[at:at + counts[s]]
        at += counts[s]
        c.table[s, :counts[s]] = ints(ids)
        c.held[s], c.length[s] = counts[s], n
        c.refs[torch.from_numpy(ids).cuda()] = 1
        pair = []
        for which in range(2):
            x = rng.standard_normal((n + T, HKV, D))
            # keys differ by less than values: scores of some ten thousand would leave one key
            x *= 2.0 ** rng.uniform(*((-1, 1) if which == 0 else powers), x.shape[:2])[..., None]
            if sized is not None:
                x *= sized(which, s)[:, None, None]
            codes, scale = quant.quantise(x)
            pair.append(quant.value(codes, scale))
            full = counts[s] * page
            pad = np.full((full, HKV, D), 127, np.uint8)
            pad[:n + T] = codes
            spad = np.full((full, HKV), 255, np.uint8)
            spad[:n + T] = scale
            i = torch.from_numpy(ids).cuda()
            pools[which][1, i] = torch.from_numpy(pad).cuda().view(
                counts[s], page, HKV, D).transpose(1, 2)
            c.page_scales[1, i, :, :, which] = torch.from_numpy(spad).cuda().view(
                counts[s], page, HKV).transpose(1, 2)
        tokens.append(tuple(pair))
    return c, tokens


def check(got, want, mass, dtype):
    got = got.double().cpu().numpy()
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    off, lim = np.abs(got - want)[fine], (REL[dtype] * mass + FLOOR[dtype])[fine]
    assert np.all(off <= lim), (off / lim).max()


def run(dtype, HQ, HKV, D, T, lens, page, seed, null=(), strided=False, by=1.2, **kw):
    rng = np.random.default_rng([seed, D, T, HQ])
    c, tokens = filled(rng, lens, T, HQ, HKV, D, dtype, page, **kw)
    B = len(lens)
    q, qd = draw(rng, (B * T, HQ + (3 if strided else 0), D), dtype, by)
    q, qd = q[:, :HQ], qd[:, :HQ]
    perm = rng.permutation(B)
    slots = [-1 if r in null else int(perm[r]) for r in range(B)]
    o = torch.full((B * T, HQ, D), SENTINEL, dtype=TORCH[dtype], device="cuda")
    lse = torch.full((B * T, HQ), SENTINEL, device="cuda")
    c.rssm_attn_decode(1, q, ints(slots), T, o, lse=lse)
    assert c.rssm_kv_get_device_error() == 0
    want, wlse, mass = ref.window(qd, [None if s < 0 else tokens[s] for s in slots],
                                  [lens[s] for s in slots], T, c.scale)
    on = np.repeat(np.array(slots) >= 0, T)
    off = torch.from_numpy(~on)
    assert (o[off] == SENTINEL).all() and (lse[off] == SENTINEL).all()
    check(o[~off], want[on], mass[on], dtype)
    gl = lse.double().cpu().numpy()[on]
    assert np.all(np.abs(gl - wlse[on]) <= LSE + 1e-6 * np.abs(wlse[on]))
    again = torch.empty_like(o)
    c.rssm_attn_decode(1, q, ints(slots), T, again)
    assert torch.equal(again[~off], o[~off])
    assert int(c.work[:1216].sum()) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,HQ,HKV", [(1, 4, 1), (1, 3, 3), (1, 40, 2), (3, 8, 2), (16, 4, 1),
                                      (8, 12, 2)])
def test_rows_of_many_lengths(dtype, D, T, HQ, HKV):
    run(dtype, HQ, HKV, D, T, [0, 1, 15, 16, 17, 31, 32, 33, 127, 128, 500, 1111, 64], 16, 11,
        null=(3,))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_page_sizes(page, D):
    run("bf16", 8, 2, D, 2, [0, page - 1, page, page + 1, 5 * page + 3], page, 12)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 256), ("bf16", 64)])
def test_one_long_row_is_split_and_joined(dtype, D):
    run(dtype, 4, 1, D, 1, [30011], 64, 13)
    run(dtype, 2, 1, D, 5, [9000, 3], 64, 14, strided=True)


def test_many_rows():
    lens = [int(x) for x in np.random.default_rng(15).integers(0, 300, 700)]
    run("bf16", 4, 2, 64, 1, lens, 32, 15, null=(0, 5, 699))


@pytest.mark.parametrize("powers", [(-70, -50), (-30, 30), (40, 60)])
def test_values_of_very_different_sizes(powers):
    """bf16 outputs of the size of the values, whatever the powers of two are."""
    run("bf16", 4, 2, 128, 2, [0, 5, 70, 900], 16, 16, powers=powers)


@pytest.mark.parametrize("by,size", [(1e-20, 1e15), (1e20, 1e-20), (1e-30, 1.0), (0.0, 1.0)])
def test_queries_and_keys_of_very_different_sizes(by, size):
    def sized(which, slot):
        return np.full(1, size if which == 0 else 1.0)
    run("bf16", 4, 2, 64, 1, [0, 40, 300], 16, 17, by=by, sized=sized)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_many_small_weights_beside_a_large_one(dtype):
    """Thirty thousand keys of a weight of 2^-23 beside one of weight one: their sum is
    a part of the answer that fp16 weights relative to one would lose."""
    rng = np.random.default_rng(18)
    n, D = 30000, 64
    c, _ = filled(rng, [n], 1, 1, 1, D, dtype, 256, powers=(0, 0), scale=1.0)
    k = np.zeros((n + 1, 1, D))
    k[77, 0, 0] = 17.0                                   # e4m3 holds 16 and 18
    v = np.full((n + 1, 1, D), 448.0)
    v[77] = 1.0
    (kc, ks), (vc, vs) = quant.quantise(k), quant.quantise(v)
    ids = c.table[0, :int(c.held[0])].long()
    pad = -(n + 1) % 256
    for which, (pool, codes, scale) in enumerate(((c.k_pages, kc, ks), (c.v_pages, vc, vs))):
        x = np.concatenate([codes, np.zeros((pad, 1, D), np.uint8)])
        pool.view(torch.uint8)[1, ids] = torch.from_numpy(x).cuda().view(-1, 256, 1, D).transpose(
            1, 2)
        x = np.concatenate([scale, np.zeros((pad, 1), np.uint8)])
        c.page_scales[1, ids, :, :, which] = torch.from_numpy(x).cuda().view(-1, 256, 1).transpose(
            1, 2)
    q = torch.zeros(1, 1, D, dtype=TORCH[dtype], device="cuda")
    q[0, 0, 0] = 1.0
    o = torch.zeros_like(q)
    c.rssm_attn_decode(1, q, ints([0]), 1, o)
    want, _, mass = ref.window(q.double().cpu().numpy(),
                               [(quant.value(kc, ks), quant.value(vc, vs))], [n], 1, 1.0)
    check(o, want, mass, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bad", [127, 255])
def test_rejected_drafts_do_not_reach_earlier_tokens(dtype, D, bad):
    """NaN codes under a power that no token has, in the window's last tokens: the others
    are bit for bit what they are without."""
    rng = np.random.default_rng([19, D])
    lens, T, page = [40, 13, 200], 8, 16
    c, _ = filled(rng, lens, T, 8, 2, D, dtype, page)
    q = draw(rng, (3 * T, 8, D), dtype)[0]
    clean, dirty = torch.empty_like(q), torch.empty_like(q)
    slot = ints([0, 1, 2])
    c.rssm_attn_decode(1, q, slot, T, clean)
    for s, n in enumerate(lens):
        for at in range(n + 5, n + T):
            pg = int(c.table[s, at // page])
            c.k_pages.view(torch.uint8)[1, pg, :, at % page] = bad
            c.v_pages.view(torch.uint8)[1, pg, :, at % page] = bad
            c.page_scales[1, pg, :, at % page] = 255
    c.rssm_attn_decode(1, q, slot, T, dirty)
    a, b = (x.view(3, T, 8, D)[:, :5].float() for x in (dirty, clean))
    assert torch.isfinite(a).all()
    mass = 24.0   # |v| <= 8 |N(0, 1)|, rounded
    assert (a - b).abs().max() <= 2 * REL[dtype] * mass
    assert not torch.isfinite(dirty.view(3, T, 8, D)[:, 5:].float()).all()


def test_a_nan_that_is_seen_is_answered():
    rng = np.random.default_rng(20)
    c, _ = filled(rng, [20, 20, 20], 1, 2, 1, 64, "bf16", 16)
    q = draw(rng, (3, 2, 64), "bf16")[0]
    c.k_pages.view(torch.uint8)[1, int(c.table[0, 0]), 0, 3, 5] = 127
    c.v_pages.view(torch.uint8)[1, int(c.table[1, 0]), 0, 3, 5] = 255
    o = torch.zeros_like(q)
    c.rssm_attn_decode(1, q, ints([0, 1, 2]), 1, o)
    assert o[0].isnan().all()
    assert o[1, :, 5].isnan().all() and torch.isfinite(o[1, :, 6:].float()).all()
    assert torch.isfinite(o[2].float()).all()
    q[2, 1, 9] = float("inf")
    c.rssm_attn_decode(1, q, ints([0, 1, 2]), 1, o)
    assert o[2, 1].isnan().all() and torch.isfinite(o[2, 0].float()).all()


def test_refused_rows():
    from linear_attention_state_rssm_gb300 import _lib as lib
    c, _ = filled(np.random.default_rng(21), [20, 30, 40], 1, 2, 1, 64, "bf16", 16)
    q = draw(np.random.default_rng(22), (3, 2, 64), "bf16")[0]
    o = torch.full_like(q, SENTINEL)
    c.rssm_attn_decode(1, q, ints([0, 3, 2]), 1, o)
    assert c.rssm_kv_get_device_error() == lib.DEVERR["slot"] and (o[1] == SENTINEL).all()
    c.length[1] = 33
    o.fill_(SENTINEL)
    c.rssm_attn_decode(1, q, ints([0, 1, 2]), 1, o)
    assert c.rssm_kv_get_device_error() == lib.DEVERR["pages"]
    assert (o[1] == SENTINEL).all() and (o[0] != SENTINEL).any()
    c.length[1] = 30
    c.table[1, 0] = 99
    c.rssm_attn_decode(1, q[:1], ints([1]), 1, o[:1])
    assert c.rssm_kv_get_device_error() == lib.DEVERR["pages"]
    with pytest.raises(lib.RssmError):
        c.rssm_attn_decode(1, q.new_zeros(195, 2, 64), ints([0, 1, 2]), 65, q.new_zeros(195, 2, 64))


@pytest.mark.parametrize("D,lens", [(64, [300]), (128, [40, 20000]), (256, [40, 20000])])
def test_waits_that_run_out_and_the_call_after(D, lens):
    """No output is wrong, the bit is set, and the next call is right."""
    from linear_attention_state_rssm_gb300 import _lib as lib
    rng = np.random.default_rng(23)
    c, tokens = filled(rng, lens, 1, 4, 1, D, "bf16", 64)
    B = len(lens)
    q, qd = draw(rng, (B, 4, D), "bf16")
    slot = ints(range(B))
    want, _, mass = ref.window(qd, tokens, lens, 1, c.scale)
    for cta, unit in ((0, 0), (1 if B > 1 else 0, 1)):
        o = torch.full_like(q, SENTINEL)
        c.rssm_kv_debug_withhold(cta, unit)
        c.rssm_attn_decode(1, q, slot, 1, o)
        c.rssm_kv_debug_withhold(-1)
        assert c.rssm_kv_get_device_error() == lib.DEVERR["timeout"]
        left = (o == SENTINEL).all(-1).all(-1).cpu().numpy()
        assert left.any()
        check(o[torch.from_numpy(~left)], want[~left], mass[~left], "bf16")
        c.rssm_attn_decode(1, q, slot, 1, o)
        assert c.rssm_kv_get_device_error() == 0
        check(o, want, mass, "bf16")


def test_pools_past_32_bit_offsets():
    from linear_attention_state_rssm_gb300.store import KVCache
    D, HKV, page = 256, 4, 256
    n = (1 << 32) // (HKV * page * D) + 40
    c = KVCache(HQ=HKV, HKV=HKV, D=D, n_pages=n, page_size=page, max_pages=2, page_dtype="e4m3")
    c.table[0, 0], c.table[0, 1] = n - 1, n - 3
    c.held[0] = 2
    rng = np.random.default_rng(24)
    (k, kd), (v, vd) = (draw(rng, (300, HKV, D), "bf16") for _ in range(2))
    q, qd = draw(rng, (1, HKV, D), "bf16")
    c.rssm_kv_append(0, None, k, v, ints([0]), 300)
    c.rssm_kv_commit(ints([0]), 299)
    o = torch.zeros_like(q)
    c.rssm_attn_decode(0, q, ints([0]), 1, o)
    assert c.rssm_kv_get_device_error() == 0
    kv = [quant.value(*quant.quantise(x)) for x in (kd, vd)]
    want, _, mass = ref.window(qd, [kv], [299], 1, c.scale)
    check(o, want, mass, "bf16")
