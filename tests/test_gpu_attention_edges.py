"""The full-attention layers' operators where their parts meet: streams of a tile
without work, waits that run out, sums of page plans near their limits, rows
with refused offsets. Tolerances are those of test_gpu_attention.py unless a
test derives its own."""
import time

import numpy as np
import pytest
import torch

from linear_attention_state_rssm_gb300._lib import DEVERR
from oracle import attention as ref
from test_gpu_attention import REL, SENTINEL, cache, draw, filled, ints, rng_of, run_prompt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_attention_state_rssm_gb300 import build
    build.build()


# ------------------------------------------- a stream of a tile without a key
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("HQ,HKV,lq,lk", [
    (2, 2, 256, 100),      # 128 tokens to a stream: the first sees nothing, the second does
    (3, 1, 84, 40),        # 42 tokens
    (64, 1, 4, 1),         # two tokens
    (4, 2, 300, 3)])       # tiles of which both, one and no stream sees nothing
def test_prompt_stream_without_any_key(dtype, D, HQ, HKV, lq, lk):
    """Rows that see no key are 0 and -inf whichever part of a tile they fill, every time."""
    o, lse = run_prompt(dtype, HQ, HKV, D, [lq], [lk], 51)
    none = lq - lk
    assert (o[:none] == 0).all() and torch.isneginf(lse[:none]).all()
    # many tiles at once, many times: a load of queries that lands late would show in these rows
    B = 40
    rng = rng_of(52, D)
    q, k, v = (draw(rng, (B * n, h, D), dtype)[0] for n, h in ((lq, HQ), (lk, HKV), (lk, HKV)))
    c = cache(n_slots=B, HQ=HQ, HKV=HKV, D=D, page_size=16, dtype=dtype)
    cu, cuk = ints(range(0, B * lq + 1, lq)), ints(range(0, B * lk + 1, lk))
    first = None
    for _ in range(20):
        o = torch.full_like(q, SENTINEL)
        lse = torch.full((B * lq, HQ), SENTINEL, device="cuda")
        c.rssm_attn_prefill(q, k, v, cu, None, o, cu_keys=cuk, lse=lse)
        assert (o.view(B, lq, HQ, D)[:, :none] == 0).all()
        assert torch.isneginf(lse.view(B, lq, HQ)[:, :none]).all()
        first = o if first is None else first
        assert torch.equal(o, first)
    assert c.rssm_kv_get_device_error() == 0


# ------------------------------------------------------------ host-side tensors
def test_lse_in_host_memory_is_refused():
    c = cache(n_slots=2, HQ=2, HKV=1, D=64, n_pages=2, page_size=16)
    q, o = (torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k, slot, lse = q[:, :1], ints([0, 1]), torch.zeros(2, 2)
    with pytest.raises(ValueError):
        c.rssm_attn_decode(0, q, slot, 1, o, lse=lse)
    with pytest.raises(ValueError):
        c.rssm_attn_prefill(q, k, k, ints([0, 1, 2]), slot, o, lse=lse)


# ---------------------------------------------------------- waits that run out
def timed(call):
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    call()
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 30.0


@pytest.mark.parametrize("dtype,D,HQ,T", [("bf16", 128, 4, 1), ("f16", 64, 4, 1),
                                          ("bf16", 256, 4, 1), ("f32", 64, 2, 1),
                                          ("bf16", 128, 4, 8), ("bf16", 128, 1, 64),
                                          ("f16", 256, 1, 48)])
@pytest.mark.parametrize("unit", [0, 1, 3, 8])
def test_decode_wait_that_runs_out_leaves_the_row_alone(dtype, D, HQ, T, unit):
    """Three rows of one length, a CTA each. One copy of the second is promised more than it
    brings: the call returns, says so, leaves that row as it is, and the others and the next
    call are what they are without (every copy has landed: nothing faults)."""
    c, _ = filled(rng_of(61, D), [400 - T] * 3, T, HQ, 1, D, dtype, 16)
    q, slot = draw(rng_of(62), (3 * T, HQ, D), dtype)[0], ints([0, 1, 2])

    def decode():
        o = torch.full_like(q, SENTINEL)
        lse = torch.full((3 * T, HQ), SENTINEL, device="cuda")
        timed(lambda: c.rssm_attn_decode(1, q, slot, T, o, lse=lse))
        return o.view(3, T, HQ, D), lse.view(3, T, HQ)

    clean = decode()
    assert c.rssm_kv_get_device_error() == 0
    c.rssm_kv_debug_withhold(1, unit)
    late = decode()
    assert c.rssm_kv_get_device_error() == DEVERR["timeout"]
    c.rssm_kv_debug_withhold(-1)
    for got, want in zip(late, clean):
        assert torch.equal(got[[0, 2]], want[[0, 2]])
        assert (got[1] == SENTINEL).all()
    for got, want in zip(decode(), clean):
        assert torch.equal(got, want)
    assert c.rssm_kv_get_device_error() == 0


@pytest.mark.parametrize("dtype,D,HQ,HKV,T", [("bf16", 128, 4, 1, 1), ("f16", 64, 8, 2, 5),
                                              ("bf16", 256, 6, 2, 9), ("f32", 128, 4, 1, 1)])
@pytest.mark.parametrize("cta", [0, 1, 7, 39])  # 39: the end of a row and the begin of the next
@pytest.mark.parametrize("unit", [0, 2])
def test_decode_wait_that_runs_out_in_a_split_row(dtype, D, HQ, HKV, T, cta, unit):
    """Rows cut over many CTAs, of which one loses a copy: each row and key head is either
    complete or as it was, arrivals are back at zero, and the next call is right."""
    lens = [30011, 700, 12345, 3]
    c, _ = filled(rng_of(63, D), lens, T, HQ, HKV, D, dtype, 64)
    q, slot = draw(rng_of(64), (4 * T, HQ, D), dtype)[0], ints([0, 1, 2, 3])
    G = HQ // HKV

    def decode():
        o = torch.full_like(q, SENTINEL)
        lse = torch.full((4 * T, HQ), SENTINEL, device="cuda")
        timed(lambda: c.rssm_attn_decode(1, q, slot, T, o, lse=lse))
        # one block of T G query rows per row and key head (of 16 or more rows: in one piece)
        return (o.view(4, T, HKV, G, D).transpose(1, 2).flatten(2),
                lse.view(4, T, HKV, G).transpose(1, 2).flatten(2))

    clean = decode()
    assert c.rssm_kv_get_device_error() == 0
    c.rssm_kv_debug_withhold(cta, unit)
    late = decode()
    assert c.rssm_kv_get_device_error() == DEVERR["timeout"]
    c.rssm_kv_debug_withhold(-1)
    kept = [(got == SENTINEL).all(-1) for got in late]
    right = [(got == want).all(-1) for got, want in zip(late, clean)]
    assert torch.equal(kept[0], kept[1])
    assert kept[0].any() and torch.equal(right[0], ~kept[0]) and torch.equal(right[1], ~kept[1])
    assert (c.work[:4 * 456] == 0).all()            # the arrival counters of every CTA
    for _ in range(2):
        for got, want in zip(decode(), clean):
            assert torch.equal(got, want)
    assert c.rssm_kv_get_device_error() == 0


@pytest.mark.parametrize("dtype,D,HQ,HKV", [("bf16", 64, 4, 4), ("f16", 64, 6, 2),
                                            ("bf16", 128, 4, 4), ("f16", 128, 40, 2),
                                            ("bf16", 256, 4, 4), ("f16", 256, 96, 32)])
@pytest.mark.parametrize("unit", [0, 1, 2, "queries"])
def test_prompt_wait_that_runs_out_leaves_rows_alone(dtype, D, HQ, HKV, unit):
    """One CTA's keys, values or queries are promised more than they bring: each row and head
    is either complete or as it was, and the next call is right."""
    late_prompt(dtype, D, HQ, HKV, unit, {64: 8, 128: 5, 256: 5}[D])


def late_prompt(dtype, D, HQ, HKV, unit, places):
    cu = ints([0, 400, 430, 900])
    q, k, v = (draw(rng_of(65, D), (900, h, D), dtype)[0] for h in (HQ, HKV, HKV))
    c = cache(n_slots=3, HQ=HQ, HKV=HKV, D=D, page_size=16, dtype=dtype)

    def prompt():
        o = torch.full_like(q, SENTINEL)
        lse = torch.full((900, HQ), SENTINEL, device="cuda")
        timed(lambda: c.rssm_attn_prefill(q, k, v, cu, None, o, lse=lse))
        return o, lse[..., None]

    clean = prompt()
    assert c.rssm_kv_get_device_error() == 0
    c.rssm_kv_debug_withhold(0, places if unit == "queries" else unit)
    late = prompt()
    assert c.rssm_kv_get_device_error() == DEVERR["timeout"]
    c.rssm_kv_debug_withhold(-1)
    kept = [(got == SENTINEL).all(-1) for got in late]
    assert kept[0].any() and not kept[0].all() and torch.equal(kept[0], kept[1])
    for got, want, left in zip(late, clean, kept):
        assert torch.equal((got == want).all(-1), ~left)
    for got, want in zip(prompt(), clean):
        assert torch.equal(got, want)
    assert c.rssm_kv_get_device_error() == 0


def test_arguments_of_the_waits_hook_are_checked():
    from linear_attention_state_rssm_gb300 import RssmError
    c = cache(n_slots=1, HQ=1, HKV=1, D=64, page_size=16)
    for bad in ((-2, 0), (0, -1)):
        with pytest.raises(RssmError):
            c.rssm_kv_debug_withhold(*bad)
    c.rssm_kv_debug_withhold(-1)


# --------------------------------------------------------- sums of page plans
def test_page_plans_whose_needs_are_past_two_to_the_thirty():
    """2048 rows that want 2^20 pages each, of a pool with five free ones: every row is
    refused and nothing else changes."""
    n, pages = 2048, 1 << 20
    c = cache(n_slots=n + 1, HQ=1, HKV=1, D=64, n_pages=pages + 5, page_size=16,
              max_pages=pages, dtype="f16")
    c.table[0] = torch.arange(pages, dtype=torch.int32, device="cuda")
    c.refs[:pages] = 1
    c.held[0], c.length[0] = pages, 16 * pages
    refs = c.refs.clone()
    rest = ints(range(1, n + 1))
    c.rssm_kv_fork(torch.zeros_like(rest), rest, deep=True)
    assert c.rssm_kv_get_device_error() == DEVERR["pages"]
    assert torch.equal(c.refs, refs) and not c.held[1:].any() and not c.length[1:].any()
    c.length[1:] = 16 * pages - 1
    c.rssm_kv_reserve(rest, 1)
    assert c.rssm_kv_get_device_error() == DEVERR["pages"]
    assert torch.equal(c.refs, refs) and not c.held[1:].any()
    assert (c.table[1:] == -1).all()
    c.length[1:] = 0
    c.rssm_kv_reserve(rest[:6], 1)                  # five rows get the five pages
    assert c.rssm_kv_get_device_error() == DEVERR["pages"]
    assert c.held[1:].tolist() == [1] * 5 + [0] * (n - 5)


# --------------------------------------------------- rows with refused offsets
@pytest.mark.parametrize("cu,live", [([0, 4, 9], [0]), ([-2, 4, 6], [1]), ([0, 4, 2], [0])])
def test_append_skips_rows_whose_offsets_are_refused(cu, live):
    c, _ = filled(rng_of(71), [0, 0], 16, 2, 1, 64, "f32", 16)
    q, k, v = (draw(rng_of(72), (6, h, 64), "f32")[0] for h in (2, 1, 1))
    out, kout = torch.full_like(q, SENTINEL), torch.full_like(k, SENTINEL)
    pages = [int(c.table[s, 0]) for s in range(2)]
    before = c.k_pages.clone()
    c.rssm_kv_append(0, q, k, v, ints([0, 1]), q_out=out, cu_seqlens=ints(cu), k_out=kout)
    assert c.rssm_kv_get_device_error() == DEVERR["seqlen"]
    for r in range(2):
        a, b = max(cu[r], 0), min(cu[r + 1], 6)
        if r in live:
            assert torch.equal(out[a:b], q[a:b]) and torch.equal(kout[a:b], k[a:b])
            assert torch.equal(c.k_pages[0, pages[r], 0, :b - a], k[a:b, 0])
        else:
            assert torch.equal(c.k_pages[0, pages[r]].isnan(), before[0, pages[r]].isnan())
            if b > a:
                assert (out[a:b] == SENTINEL).all() and (kout[a:b] == SENTINEL).all()


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("f16", 128), ("bf16", 256), ("f32", 64)])
def test_prompt_reports_tiles_that_it_has_no_room_for(dtype, D):
    """Offsets that go back at a null row, so that two sequences share tokens: more tiles than
    N tokens in order can make are not dropped silently."""
    q, k, v = (draw(rng_of(73), (1300, h, D), dtype)[0] for h in (1, 1, 1))
    c = cache(n_slots=4, HQ=1, HKV=1, D=D, page_size=16, dtype=dtype)
    o = torch.empty_like(q)
    c.rssm_attn_prefill(q, k, v, ints([0, 1000, 1, 1000, 1300]), ints([0, -1, 2, 3]), o)
    assert c.rssm_kv_get_device_error() == DEVERR["seqlen"]
    c.rssm_attn_prefill(q, k, v, ints([0, 1000, 1000, 1000, 1300]), ints([0, -1, 2, 3]), o)
    assert c.rssm_kv_get_device_error() == 0


# ------------------------------------------------------------ closer tolerances
def test_decode_leaves_every_arrival_counter_at_zero():
    """Three CTAs per SM (16-bit heads of 64) and rows that all of them share."""
    c, _ = filled(rng_of(81), [4000] * 24, 1, 4, 4, 64, "bf16", 64)
    q = draw(rng_of(82), (24, 4, 64), "bf16")[0]
    o, first = torch.empty_like(q), None
    for _ in range(3):
        c.rssm_attn_decode(1, q, ints(range(24)), 1, o)
        assert (c.work[:4 * 456] == 0).all()
        first = o.clone() if first is None else first
        assert torch.equal(o, first)
    assert c.rssm_kv_get_device_error() == 0


# fp32 sums of D products in a row: partial sums of size 1.7 sqrt(k) round by 2^-24 of
# themselves each, about 1.1e-5 (D = 256) of standard deviation, times scale 1/16 = 7e-7;
# six of those, and the rounding of x c (2^-24 of at most 15), leave the exponent within
# 5e-6. Weights and their sum are off by that each: 1e-5 of the mass, and the sum over the
# keys and the base-2 exponential (2 ulp) add 2e-6.
CLOSE32 = 1.2e-5


def close32(got, want, mass):
    off = np.abs(got.double().cpu().numpy() - want)
    assert np.all(off <= CLOSE32 * mass + 1e-8), (off / mass).max()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_fp32_attention_keeps_fp32_accuracy(D):
    rng = rng_of(83, D)
    lq, lk = [300, 1, 77], [900, 700, 77]
    cu, cuk = np.cumsum([0] + lq), np.cumsum([0] + lk)
    (q, qd), (k, kd), (v, vd) = (draw(rng, (n, h, D), "f32", 1.3)
                                 for n, h in ((cu[-1], 4), (cuk[-1], 2), (cuk[-1], 2)))
    c = cache(n_slots=3, HQ=4, HKV=2, D=D, page_size=16, dtype="f32")
    o = torch.empty_like(q)
    c.rssm_attn_prefill(q, k, v, ints(cu), None, o, cu_keys=ints(cuk))
    want, _, mass = ref.prompt(qd, kd, vd, cu, cuk, c.scale)
    close32(o, want, mass)
    lens, T = [0, 1500, 4001, 63], 3
    c, tokens = filled(rng, lens, T, 4, 2, D, "f32", 32)
    q, qd = draw(rng, (4 * T, 4, D), "f32", 1.2)
    o = torch.empty_like(q)
    c.rssm_attn_decode(1, q, ints(range(4)), T, o)
    want, _, mass = ref.window(qd, tokens, lens, T, c.scale)
    close32(o, want, mass)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_prompt_rows_before_a_poisoned_token(dtype, D, bad):
    """Token 600 of 700 and its neighbours' ends are poisoned. Rows of tiles that end before
    its keys are bitwise what they are without; the rows right before it, computed again,
    are within their own mass of rounding."""
    rng = rng_of(84, D)
    (q, qd), (k, kd), (v, vd) = (draw(rng, (740, h, D), dtype) for h in (2, 1, 1))
    cu = [0, 700, 740]
    c = cache(n_slots=2, HQ=2, HKV=1, D=D, page_size=16, dtype=dtype)
    want, _, mass = ref.prompt(qd, kd, vd, cu, cu, c.scale)
    clean, dirty = torch.empty_like(q), torch.empty_like(q)
    c.rssm_attn_prefill(q, k, v, ints(cu), None, clean)
    k[600], v[600] = bad, bad
    c.rssm_attn_prefill(q, k, v, ints(cu), None, dirty)
    assert torch.equal(dirty[:512], clean[:512]) and torch.equal(dirty[700:], clean[700:])
    off = np.abs(dirty[512:600].double().cpu().numpy() - want[512:600])
    assert np.all(off <= REL[dtype] * mass[512:600] + 1e-7)
    assert not torch.isfinite(dirty[600:700].float()).any()


# --------------------------------------------------- large pools, other streams
def test_pages_past_32_bit_offsets():
    """Pools of 13 G values (26 GB) each: append, decode, fork and compaction at their far end
    give what a small pool gives."""
    HQ, HKV, D, page, T, n = 8, 4, 128, 64, 3, 200
    pages = 400_000
    lens = [n, 64]
    results = []
    for total, ids in ((16, [5, 9, 7, 2, 11, 12]),
                       (pages, [pages - 1, pages - 9, pages - 2, 131072, pages - 3, pages - 5])):
        rng = rng_of(91)
        c = cache(n_layers=1, n_slots=3, HQ=HQ, HKV=HKV, D=D, n_pages=total, page_size=page,
                  max_pages=8, dtype="bf16")
        c.table[0, :4], c.table[1, :2] = ints(ids[:4]), ints(ids[4:])
        c.held[:2], c.refs[ids] = ints([4, 2]), 1
        cu = ints([0, n, n + 64])
        k, v = (draw(rng, (n + 64, HKV, D), "bf16")[0] for _ in range(2))
        c.rssm_kv_append(0, None, k, v, ints([0, 1]), cu_seqlens=cu)
        c.rssm_kv_commit(ints([0, 1]), cu_seqlens=cu)
        out = []

        def decode(slot):
            B = slot.numel()
            q, k, v = (draw(rng, (B * T, h, D), "bf16")[0] for h in (HQ, HKV, HKV))
            c.rssm_kv_reserve(slot, T)
            c.rssm_kv_append(0, None, k, v, slot, T)
            o = torch.empty_like(q)
            c.rssm_attn_decode(0, q, slot, T, o)
            out.append(o)

        decode(ints([0, 1]))
        c.rssm_kv_fork(ints([0]), ints([2]), deep=True)
        decode(ints([2, 0]))
        c.rssm_kv_compact()
        decode(ints([1, 2, 0]))
        assert c.rssm_kv_get_device_error() == 0
        assert sorted(c.refs.nonzero().flatten().tolist()) == list(range(int((c.refs > 0).sum())))
        results.append(out)
        del c
        torch.cuda.empty_cache()
    for got, want in zip(*results):
        assert torch.equal(got, want)


def test_page_calls_in_a_graph_on_another_stream():
    from linear_attention_state_rssm_gb300.store import KVCache
    a, b = (KVCache(2, 6, 2, 1, 64, n_pages=40, page_size=16, max_pages=8, dtype="f32")
            for _ in range(2))
    for c in (a, b):
        c.k_pages.copy_(torch.arange(c.k_pages.numel(), device="cuda").view_as(c.k_pages))
        c.v_pages.copy_(c.k_pages).neg_()
    slots, n = ints([0, 1, 2]), ints([40, 3, 100])
    src, dst, gone = ints([0, 2]), ints([3, 4]), ints([1, 2])

    def calls(c):
        c.rssm_kv_reserve(slots, 110)
        c.rssm_kv_commit(slots, 110, accept_len=n)
        c.rssm_kv_fork(src, dst)
        c.rssm_kv_release(gone)
        c.rssm_kv_compact()
        c.rssm_kv_fork(dst, ints_5, deep=True)
        c.rssm_kv_release(slots)
        c.rssm_kv_compact()

    ints_5 = ints([5, 1])
    calls(a)
    st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=st):
        calls(b)
    with torch.cuda.stream(st):
        graph.replay()
    st.synchronize()
    for name in ("table", "held", "length", "refs", "k_pages", "v_pages"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name
    assert a.rssm_kv_get_device_error() == b.rssm_kv_get_device_error() == 0
    assert a.held.tolist()[3:] == [3, 7, 3]
