"""Attention over pages and shared prefixes where sizes lie far apart: powers of two of
quantised tokens, weights far below the largest, queries near the ends of their type;
and what calls leave behind.

Tolerances are those of the two modules whose batches are used here: a weight is rounded
to the type of the products (2^-8; fp16, quantised pages too: 2^-11), the output to its
own, fp32 sums and the exponential add 1e-4 of the mass sum_j p_j |v_j|.
"""
import numpy as np
import pytest
import torch

import test_gpu_attention_shared as shared
from oracle import attention as ref
from oracle import quant
from test_gpu_attention_shared import SENTINEL, TORCH, Batch, draw, ints

pytestmark = pytest.mark.gpu
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
FLOOR = {"bf16": 2.0 ** -126, "f16": 2.0 ** -24}   # the types' smallest steps
LSE = 5e-5
ARRIVALS = 4 * 3 * 152    # bytes of the work buffer that count parts


def rel(dtype, pages):
    return HALF[dtype] + HALF["f16" if pages else dtype] + 1e-4


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_attention_state_rssm_gb300 import build
    build.build()


def put(b, which, s, x):
    """x [n, HKV, D]: slot s's first n keys (0) or values (1), in the pool and the oracle."""
    c, page = b.c, b.c.page_size
    pool = (c.k_pages, c.v_pages)[which]
    for i, pg in enumerate(b.tables[s]):
        part = x[i * page:(i + 1) * page].transpose(1, 0, 2)
        n = part.shape[1]
        if n == 0:
            break
        if c.page_scales is None:
            t = torch.from_numpy(part.copy()).to(TORCH[b.dtype])
            pool[1, pg, :, :n] = t.cuda()
            b.values[which][pg, :, :n] = t.double().numpy()
        else:
            codes, scale = quant.quantise(part)
            pool.view(torch.uint8)[1, pg, :, :n] = torch.from_numpy(codes).cuda()
            c.page_scales[1, pg, :, :n, which] = torch.from_numpy(scale).cuda()
            b.values[which][pg, :, :n] = quant.value(codes, scale)


def close(got, want, mass, dtype, pages):
    got = got.double().cpu().numpy()
    off, lim = np.abs(got - want), rel(dtype, pages) * mass + FLOOR[dtype]
    assert np.all(off <= lim), (off / lim).max()


def both(b, q, pages):
    """The batch by the shared attention and row by row, against the oracle."""
    c, B, T = b.c, len(b.lens), b.T
    want, wlse, mass = b.want(q.double().cpu().numpy(), list(range(B)))
    slot, share = ints(range(B)), c.new_share(B, T)
    c.rssm_kv_share(slot, T, share)
    for call in (lambda *a, **k: c.rssm_attn_decode_shared(1, q, slot, T, share, *a, **k),
                 lambda *a, **k: c.rssm_attn_decode(1, q, slot, T, *a, **k)):
        o = torch.full_like(q, SENTINEL)
        lse = torch.full(q.shape[:2], SENTINEL, device="cuda")
        call(o, lse=lse)
        assert c.rssm_kv_get_device_error() == 0
        close(o, want, mass, b.dtype, pages)
        assert np.all(np.abs(lse.double().cpu().numpy() - wlse) <= LSE + 1e-6 * np.abs(wlse))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("by", [2.0 ** -75, 2.0 ** -110])
def test_small_queries_on_keys_of_zeros(D, by):
    """Every score is 0, in a last step that is not whole too: the answer is the mean."""
    rng = np.random.default_rng([70, D])
    b = Batch(rng, [(100, [0, 30]), (200, [3, 1])], 1, 4, 2, D, "bf16", "e4m3", 16)
    for s in range(4):
        put(b, 0, s, np.zeros((b.lens[s] + 1, 2, D)))
    both(b, draw(rng, (4, 4, D), "bf16", by)[0], "e4m3")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("gap", [5, 20, 27, 45])
def test_a_large_value_of_no_weight_beside_small_ones(dtype, D, gap):
    """Tokens of values 2^gap times the others' and a weight of 2^-80: the answer is the
    others', in the large tokens' step, behind it and in the rows' own keys."""
    rng = np.random.default_rng([71, D, gap])
    b = Batch(rng, [(1000, [0, 40, 9]), (300, [5, 60])], 2, 4, 2, D, dtype, "e4m3", 16, scale=1.0)
    for s, n in enumerate(b.lens):
        k, v = 0.3 * rng.standard_normal((n + 2, 2, D)), rng.standard_normal((n + 2, 2, D))
        k[..., 0] = 0.0
        for at in (7, 140, n - 3):
            k[at] = 0.0
            k[at, :, 0] = -56.0                     # 2^-80.8 beside scores of 0
            v[at] *= 2.0 ** gap
        put(b, 0, s, k)
        put(b, 1, s, v)
    q = draw(rng, (2 * len(b.lens), 4, D), dtype, 0.1)[0]
    q[..., 0] = 1.0
    both(b, q, "e4m3")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("gap", [13, 16, 27, 50])
def test_a_large_key_without_a_score_beside_small_ones(dtype, D, gap):
    """Keys 2^gap times the others', orthogonal to every query."""
    rng = np.random.default_rng([72, D, gap])
    b = Batch(rng, [(1000, [0, 40, 9]), (300, [5, 60])], 2, 4, 2, D, dtype, "e4m3", 16)
    for s, n in enumerate(b.lens):
        k = 1.2 * rng.standard_normal((n + 2, 2, D))
        k[..., 1] = 0.0
        for at in (7, 140, n - 3):
            k[at] = 0.0
            k[at, :, 1] = 2.0 ** gap
        put(b, 0, s, k)
    q = draw(rng, (2 * len(b.lens), 4, D), dtype, 1.2)[0]
    q[..., 1] = 0.0
    both(b, q, "e4m3")


@pytest.mark.parametrize("D", [64, 128, 256])
def test_large_queries_beside_large_keys_without_a_score(D):
    """2^110 in a query and 2^60 in a key, in dimensions that the other has not: a score of
    0, whatever the product of their powers is."""
    rng = np.random.default_rng([73, D])
    b = Batch(rng, [(200, [0, 40, 9]), (0, [50])], 1, 4, 2, D, "bf16", "e4m3", 16)
    for s, n in enumerate(b.lens):
        k = np.zeros((n + 1, 2, D))
        k[::3, :, 1] = 2.0 ** 60
        put(b, 0, s, k)
    q = torch.zeros(4, 4, D, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 2.0 ** 110
    both(b, q, "e4m3")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("first", [True, False])
def test_values_of_zeros_beside_the_largest(D, first):
    """Powers of two at both ends of their range under scores that are all alike: tokens
    without a value count in the sum as the others do."""
    rng = np.random.default_rng([74, D])
    b = Batch(rng, [(640, [0, 300, 9]), (0, [3000]), (0, [9000])], 1, 4, 2, D, "bf16", "e4m3", 16)
    for s, n in enumerate(b.lens):
        v = 2.0 ** 71 * rng.choice((-1.0, 1.0), (n + 1, 2, D)) * rng.uniform(0.9, 1.7, (n + 1, 2, D))
        none = np.arange(n + 1) < n // 2
        v[none if first else ~none] = 0.0
        put(b, 1, s, v)
    both(b, torch.zeros(len(b.lens), 4, D, dtype=torch.bfloat16, device="cuda"), "e4m3")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("pages", [None, "e4m3"])
@pytest.mark.parametrize("low", [16.0, 18.0])
@pytest.mark.parametrize("top", [1.0, 14.0])
def test_many_small_weights_in_fp16(D, pages, low, top):
    """Thousands of keys of a weight of 2^-23 or 2^-26 beside one of weight one, and values
    448 or 32 times its: weights relative to one would lose them in fp16, or round them by
    half."""
    rng = np.random.default_rng([75, D])
    b = Batch(rng, [(20000, [0, 40]), (0, [9000])], 1, 4, 2, D, "f16", pages, 64, scale=1.0)
    for s, n in enumerate(b.lens):
        k, v = np.zeros((n + 1, 2, D)), np.full((n + 1, 2, D), 448.0)
        k[77, :, 0], v[77] = low, top
        put(b, 0, s, k)
        put(b, 1, s, v)
    q = torch.zeros(3, 4, D, dtype=torch.float16, device="cuda")
    q[..., 0] = 1.0
    both(b, q, pages)


@pytest.mark.parametrize("D,G", [(64, 1), (128, 4), (256, 2), (256, 4)])
@pytest.mark.parametrize("low", [16.0, 18.0])
def test_many_small_weights_in_fp16_prompts(D, G, low):
    from linear_attention_state_rssm_gb300.store import KVCache
    HKV, n, m = 2, 100, 20000
    c = KVCache(HQ=HKV * G, HKV=HKV, D=D, dtype="f16", scale=1.0)
    k = torch.zeros(m, HKV, D, dtype=torch.float16, device="cuda")
    v = torch.full((m, HKV, D), 448.0, dtype=torch.float16, device="cuda")
    k[77, :, 0], v[77] = low, 1.0
    q = torch.zeros(n, HKV * G, D, dtype=torch.float16, device="cuda")
    q[..., 0] = 1.0
    o, lse = torch.empty_like(q), torch.empty(n, HKV * G, device="cuda")
    c.rssm_attn_prefill(q, k, v, ints([0, n]), None, o, cu_keys=ints([0, m]), lse=lse)
    assert c.rssm_kv_get_device_error() == 0
    want, wlse, mass = ref.prompt(*(x.double().cpu().numpy() for x in (q, k, v)),
                                  np.array([0, n]), np.array([0, m]), 1.0)
    close(o, want, mass, "f16", None)
    assert np.all(np.abs(lse.double().cpu().numpy() - wlse) <= LSE + 1e-6 * np.abs(wlse))


def test_rows_that_wait_long_for_their_prefix():
    """A prefix of 2^28 keys (one page, named again and again) takes longer than a wait's
    limit. The rows' launch, whose rings are full by then, does not count that as its own."""
    from linear_attention_state_rssm_gb300.store import KVCache
    rng = np.random.default_rng(76)
    HQ, D, T, page, own = 64, 64, 64, 256, 17
    most = 1 << 20
    c = KVCache(n_slots=5, HQ=HQ, HKV=1, D=D, n_pages=1 + 5 * own, page_size=page, max_pages=most)
    for pool in (c.k_pages, c.v_pages):
        pool[0] = torch.from_numpy(rng.standard_normal(pool[0].shape)).to(pool)
    lens, prefix = [], most - own - 1
    for s in range(5):
        ids = 1 + own * s + np.arange(own)
        held = own if s == 4 else prefix + own
        c.table[s, :held - own] = 0
        c.table[s, held - own:held] = ints(ids)
        c.held[s], c.length[s] = held, held * page - T
        lens.append(held * page - T)
    q, qd = draw(rng, (5 * T, HQ, D), "bf16")
    slot, share, o = ints(range(5)), c.new_share(5, T), torch.full_like(q, SENTINEL)
    c.rssm_kv_share(slot, T, share)
    n, keys, _ = shared.plan(share, 5)
    assert n == 1 and keys == [prefix * page] * 4 + [0]
    t = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    t[0].record()
    c.rssm_attn_decode_shared(0, q, slot, T, share, o)
    t[1].record()
    assert c.rssm_kv_get_device_error() == 0
    assert t[0].elapsed_time(t[1]) > 500            # else nothing was waited for
    assert not (o == SENTINEL).all(-1).any() and torch.isfinite(o.float()).all()
    kv = [x[0, 1 + 4 * own:].transpose(1, 2).reshape(-1, 1, D).double().cpu().numpy()
          for x in (c.k_pages, c.v_pages)]
    want, _, mass = ref.window(qd[4 * T:], [kv], [lens[4]], T, c.scale)
    close(o[4 * T:], want, mass, "bf16", None)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,HQ,HKV", [(1, 4, 1), (3, 8, 2), (16, 4, 1)])
def test_quantised_groups_to_the_rounding_of_their_weights(dtype, D, T, HQ, HKV, monkeypatch):
    """Over quantised pages weights are rounded to fp16 whatever the type: the shapes of the
    other module again, with that tolerance, and every count of arrivals is zero after."""
    monkeypatch.setitem(shared.REL, dtype, rel(dtype, "e4m3"))
    b, _ = shared.run((dtype, "e4m3"), [(64, [0, 1, 17, 200]), (1000, [3, 40, 15]), (0, [50]),
                                        (16, [0, 0, 0]), (500, [90])], T, HQ, HKV, D, 16, 77)
    assert not b.c.work[:ARRIVALS].any()


@pytest.mark.parametrize("kind", [("bf16", None), ("f32", None), ("bf16", "e4m3")])
def test_every_arrival_is_counted_off(kind):
    """Heads of 64 have three CTAs an SM: rows that are split over all of them."""
    dtype, pages = kind
    rng = np.random.default_rng(78)
    b = Batch(rng, [(0, [9000] * 24), (64, [5000, 4000])], 1, 8, 2, 64, dtype, pages, 256)
    q = draw(rng, (26, 8, 64), dtype)[0]
    slot, share = ints(range(26)), b.c.new_share(26)
    b.c.rssm_kv_share(slot, 1, share)
    for _ in range(2):
        b.c.rssm_attn_decode(1, q, slot, 1, torch.empty_like(q))
        b.c.rssm_attn_decode_shared(1, q, slot, 1, share, torch.empty_like(q))
    assert b.c.rssm_kv_get_device_error() == 0
    assert not b.c.work[:ARRIVALS].any()
