"""The full-attention layers' operators against the fp64 oracle.

Tolerances. The weights p enter the product with v rounded to the input type
(unit roundoff u = 2^-8 for bf16 with its 8 significant bits, 2^-11 for f16 with
11) and the output is rounded once more, so a value is off by at most
2 u sum_j p_j |v_j|; fp32 sums of up to a few thousand terms and the base-2
exponential add below 1e-4 of the same mass. f16 weights under 2^-14 lose up to
2^-25 each: below 2e-4 of |v| at the lengths used. fp32 has room for products
split in two tf32 parts (2^-21 per operand: scores of D = 256 off by less than
2e-5, outputs by less than 6e-5 of the mass); the kernels' fp32 FMAs stay well
inside.
"""
import numpy as np
import pytest
import torch

import synth
from oracle import attention as ref

pytestmark = pytest.mark.gpu
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
REL = {"bf16": 2 * 2.0 ** -8 + 1e-4, "f16": 2 * 2.0 ** -11 + 2e-4, "f32": 6e-5}
LSE = 5e-5  # fp32 scores of size ~10 and the logarithm
SENTINEL = 7.0


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_attention_state_rssm_gb300 import build
    build.build()


def cache(**kw):
    from linear_attention_state_rssm_gb300.store import KVCache
    return KVCache(**kw)


def rng_of(*key):
    return np.random.default_rng(list(key))


def draw(rng, shape, dtype, by=1.0):
    """Values of the type on the device and the same values in 64 bits."""
    t = torch.from_numpy(by * rng.standard_normal(shape)).to(TORCH[dtype])
    return t.cuda(), t.double().numpy()


def ints(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def check(got, want, mass, dtype):
    got = got.double().cpu().numpy()
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    off = np.abs(got - want)[fine]
    lim = (REL[dtype] * mass + 1e-7)[fine]
    assert np.all(off <= lim), (off / lim).max()


# ------------------------------------------------------------------- prompts
def run_prompt(dtype, HQ, HKV, D, lq, lk, seed, live=None, strided=False, scale=None):
    rng = rng_of(seed, D, HQ)
    cu = np.concatenate([[0], np.cumsum(lq)])
    cuk = np.concatenate([[0], np.cumsum(lk)])
    N, M = int(cu[-1]), int(cuk[-1])
    c = cache(n_slots=len(lq), HQ=HQ, HKV=HKV, D=D, page_size=16, dtype=dtype, scale=scale)
    if strided:
        x, xd = draw(rng, (N, HQ + 2 * HKV, D), dtype, 1.3)
        q, k, v = x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:]
        qd, kd, vd = xd[:, :HQ], xd[:, HQ:HQ + HKV], xd[:, HQ + HKV:]
    else:
        (q, qd), (k, kd), (v, vd) = (draw(rng, (n, h, D), dtype, 1.3)
                                     for n, h in ((N, HQ), (M, HKV), (M, HKV)))
    o = torch.full((N, HQ, D), SENTINEL, dtype=TORCH[dtype], device="cuda")
    lse = torch.full((N, HQ), SENTINEL, device="cuda")
    slot = None if live is None else ints(i if x else -1 for i, x in enumerate(live))
    c.rssm_attn_prefill(q, k, v, ints(cu), slot, o, cu_keys=None if strided else ints(cuk),
                        lse=lse)
    want, wlse, mass = ref.prompt(qd, kd, vd, cu, cuk, c.scale, live)
    on = np.ones(N, bool)
    if live is not None:
        on = np.repeat(np.array(live), lq)
        assert (o[~torch.from_numpy(on)] == SENTINEL).all()
        assert (lse[~torch.from_numpy(on)] == SENTINEL).all()
    check(o[torch.from_numpy(on)], want[on], mass[on], dtype)
    got = lse.double().cpu().numpy()[on]
    none = np.isneginf(wlse[on])
    assert np.array_equal(np.isneginf(got), none)
    assert np.abs(got[~none] - wlse[on][~none]).max(initial=0) <= LSE
    assert c.rssm_kv_get_device_error() == 0
    return o, lse


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("HQ,HKV", [(1, 1), (4, 2), (8, 1), (3, 1), (14, 2)])
def test_prompts_of_many_lengths(dtype, D, HQ, HKV):
    lq = [1, 130, 0, 257, 63, 2, 128]
    run_prompt(dtype, HQ, HKV, D, lq, lq, 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_prompts_with_keys_before_and_rows_without_any(dtype, D):
    lq = [5, 40, 33, 1, 17]
    lk = [133, 40, 20, 300, 0]       # chunk after a prefix; Lk < Lq; a lone token; no key at all
    o, lse = run_prompt(dtype, 6, 2, D, lq, lk, 2)
    assert (o[45:58] == 0).all() and torch.isneginf(lse[45:58]).all()   # 13 rows of the third
    assert (o[-17:] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_prompt_views_of_one_projection_and_null_rows(dtype):
    lq = [9, 140, 31]
    run_prompt(dtype, 4, 2, 128, lq, lq, 3, strided=True)
    run_prompt(dtype, 4, 2, 64, lq, lq, 4, live=[True, False, True])


@pytest.mark.parametrize("HQ,HKV", [(64, 1), (40, 1), (5, 5), (33, 1)])
def test_prompt_wide_groups(HQ, HKV):
    lq = [37, 3]
    run_prompt("bf16", HQ, HKV, 64, lq, lq, 5)


def test_prompt_long_and_large_scores():
    lq = [1500, 700]
    run_prompt("bf16", 2, 1, 128, lq, lq, 6, scale=0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_prompt_values_a_row_does_not_see_do_not_reach_it(dtype, D, bad):
    """Poisoned tokens in the middle and behind: rows before them, and the other
    sequences, are bitwise what they are without."""
    lq = [70, 150, 20]
    N, HQ, HKV = sum(lq), 4, 2
    rng = rng_of(7, D)
    q, k, v = (draw(rng, (N, h, D), dtype)[0] for h in (HQ, HKV, HKV))
    cu = ints([0, 70, 220, 240])
    c = cache(n_slots=3, HQ=HQ, HKV=HKV, D=D, page_size=16, dtype=dtype)
    clean, dirty = torch.empty_like(q), torch.empty_like(q)
    c.rssm_attn_prefill(q, k, v, cu, None, clean)
    for x in (k, v):
        x[70 + 61] = bad
        x[220 + 7, :, ::3] = bad
    c.rssm_attn_prefill(q, k, v, cu, None, dirty)
    safe = [i for i in range(N) if not (131 <= i < 220 or i >= 227)]
    got, want = dirty[safe].float(), clean[safe].float()
    assert torch.isfinite(got).all()
    assert (got - want).abs().max() <= 2 * REL[dtype] * 4.5   # mass <= max |v|
    assert not torch.isfinite(dirty[131:220].float()).all()


def test_prompt_bad_offsets_skip_the_sequence():
    from linear_attention_state_rssm_gb300 import _lib as lib
    c = cache(n_slots=3, HQ=2, HKV=1, D=64, page_size=16, dtype="bf16")
    q, k, v = (draw(rng_of(8), (64, h, 64), "bf16")[0] for h in (2, 1, 1))
    o = torch.full_like(q, SENTINEL)
    c.rssm_attn_prefill(q, k, v, ints([0, 10, 5, 90]), None, o)
    assert c.rssm_kv_get_device_error() == lib.DEVERR["seqlen"]
    assert (o[10:] == SENTINEL).all() and (o[:10] != SENTINEL).any()
    assert c.rssm_kv_get_device_error() == 0
    c.rssm_attn_prefill(q, k, v, ints([0, 10, 20, 64]), ints([0, 3, -1]), o)
    assert c.rssm_kv_get_device_error() == lib.DEVERR["slot"]


# -------------------------------------------------------------------- decode
def filled(rng, lens, T, HQ, HKV, D, dtype, page, extra=2):
    """A cache whose slots hold random tokens in shuffled pages; the places that
    hold no token are NaN."""
    counts = [-(-(n + T) // page) for n in lens]
    c = cache(n_layers=2, n_slots=len(lens), HQ=HQ, HKV=HKV, D=D, n_pages=sum(counts) + extra,
              page_size=page, max_pages=max(counts) + 1, dtype=dtype)
    c.k_pages.fill_(float("nan"))
    c.v_pages.fill_(float("nan"))
    order = rng.permutation(sum(counts) + extra)
    tokens, at = [], 0
    for s, n in enumerate(lens):
        (k, kd), (v, vd) = (draw(rng, (n + T, HKV, D), dtype, 1.2) for _ in range(2))
        tokens.append((kd, vd))
        ids = order[at:at + counts[s]]
        at += counts[s]
        c.table[s, :counts[s]] = ints(ids)
        c.held[s], c.length[s] = counts[s], n
        c.refs[torch.from_numpy(ids).cuda()] = 1
        for i, pg in enumerate(ids):
            w = slice(i * page, min((i + 1) * page, n + T))
            m = w.stop - w.start
            c.k_pages[1, pg, :, :m] = k[w].transpose(0, 1)
            c.v_pages[1, pg, :, :m] = v[w].transpose(0, 1)
    return c, tokens


def run_decode(dtype, HQ, HKV, D, T, lens, page, seed, null=(), strided=False):
    rng = rng_of(seed, D, T, HQ)
    c, tokens = filled(rng, lens, T, HQ, HKV, D, dtype, page)
    B = len(lens)
    q, qd = draw(rng, (B * T, HQ + (3 if strided else 0), D), dtype, 1.2)
    q, qd = q[:, :HQ], qd[:, :HQ]
    perm = rng.permutation(B)                       # rows are not in the slots' order
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
    assert np.abs(lse.double().cpu().numpy()[on] - wlse[on]).max(initial=0) <= LSE
    again = torch.empty_like(o)
    c.rssm_attn_decode(1, q, ints(slots), T, again)
    assert torch.equal(again[~off], o[~off])        # same sums whatever the order of arrival
    assert int(c.work[:1216].sum()) == 0            # arrivals are back at zero


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,HQ,HKV", [(1, 4, 1), (1, 3, 3), (1, 40, 2), (3, 8, 2), (16, 4, 1),
                                      (8, 12, 2)])
def test_decode_rows_of_many_lengths(dtype, D, T, HQ, HKV):
    run_decode(dtype, HQ, HKV, D, T, [0, 1, 15, 16, 17, 127, 128, 500, 1111, 64], 16, 11,
               null=(3,))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_decode_page_sizes(page):
    run_decode("bf16", 8, 2, 128, 2, [0, page - 1, page, page + 1, 5 * page + 3], page, 12)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 256), ("f32", 64)])
def test_decode_one_long_row_is_split_and_joined(dtype, D):
    run_decode(dtype, 4, 1, D, 1, [30011], 64, 13)
    run_decode(dtype, 2, 1, D, 5, [9000, 3], 64, 14, strided=True)


def test_decode_many_rows():
    lens = list(rng_of(15).integers(0, 300, 700))
    run_decode("bf16", 4, 2, 64, 1, [int(x) for x in lens], 32, 15, null=(0, 5, 699))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_decode_rejected_drafts_do_not_reach_earlier_tokens(dtype, D, bad):
    rng = rng_of(16, D)
    lens, T, page = [40, 13, 200], 8, 16
    c, _ = filled(rng, lens, T, 8, 2, D, dtype, page)
    q = draw(rng, (3 * T, 8, D), dtype)[0]
    clean, dirty = torch.empty_like(q), torch.empty_like(q)
    slot = ints([0, 1, 2])
    c.rssm_attn_decode(1, q, slot, T, clean)
    for s, n in enumerate(lens):                    # tokens 5.. of each window are rejected
        for at in range(n + 5, n + T):
            pg = int(c.table[s, at // page])
            c.k_pages[1, pg, :, at % page] = bad
            c.v_pages[1, pg, :, at % page] = bad
    c.rssm_attn_decode(1, q, slot, T, dirty)
    a, b = (x.view(3, T, 8, D)[:, :5].float() for x in (dirty, clean))
    assert torch.isfinite(a).all()
    assert (a - b).abs().max() <= 2 * REL[dtype] * 6.0
    assert not torch.isfinite(dirty.view(3, T, 8, D)[:, 5:].float()).all()


def test_decode_refused_rows():
    from linear_attention_state_rssm_gb300 import _lib as lib
    c, _ = filled(rng_of(17), [20, 30, 40], 1, 2, 1, 64, "bf16", 16)
    q = draw(rng_of(18), (3, 2, 64), "bf16")[0]
    o = torch.full_like(q, SENTINEL)
    c.rssm_attn_decode(0, q, ints([0, 3, 2]), 1, o)
    assert c.rssm_kv_get_device_error() == lib.DEVERR["slot"]
    assert (o[1] == SENTINEL).all()
    c.length[1] = 33                                 # two pages hold 32 tokens
    o.fill_(SENTINEL)
    c.rssm_attn_decode(1, q, ints([0, 1, 2]), 1, o)
    assert c.rssm_kv_get_device_error() == lib.DEVERR["pages"]
    assert (o[1] == SENTINEL).all() and (o[0] != SENTINEL).any()
    c.length[1] = -2
    c.rssm_attn_decode(1, q, ints([0, 1, 2]), 1, o)
    assert c.rssm_kv_get_device_error() == lib.DEVERR["cursor"]
    c.length[1] = 30
    c.table[1, 0] = 99                               # outside the pool: skipped, not read
    c.rssm_attn_decode(1, q[:1], ints([1]), 1, o[:1])
    assert c.rssm_kv_get_device_error() == lib.DEVERR["pages"]


# -------------------------------------------------------------------- append
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D,pairs,sections,inter", [
    (64, 32, [32], False), (128, 64, [24, 20, 20], False), (128, 64, [24, 20, 20], True),
    (256, 32, [12, 20], True), (256, 128, [128], False), (64, 8, [2, 3, 3], False)])
def test_append_rotates_and_writes_the_pages(dtype, D, pairs, sections, inter):
    from linear_attention_state_rssm_gb300.store import RotaryTable
    rng = rng_of(21, D, pairs)
    HQ, HKV, T, page, most = 6, 2, 5, 16, 5000
    lens = [0, 14, 16, 29]
    c, _ = filled(rng, lens, T, HQ, HKV, D, dtype, page)
    x, xd = draw(rng, (4 * T, HQ + 2 * HKV, D), dtype)
    axes = len(sections)
    pos = rng.integers(0, most, (axes, 4 * T))
    rope = RotaryTable.from_base(most, pairs, 1e4, sections, inter)
    out = torch.full((4 * T, HQ, D), SENTINEL, dtype=TORCH[dtype], device="cuda")
    kout = torch.full((4 * T, HKV, D), SENTINEL, dtype=TORCH[dtype], device="cuda")
    before = c.k_pages.clone()
    slots = [2, -1, 0, 3]
    c.rssm_kv_append(1, x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], ints(slots), T, out,
                     rope=rope, positions=torch.from_numpy(pos).int().cuda(), k_out=kout)
    assert c.rssm_kv_get_device_error() == 0
    freq = 1e4 ** (-np.arange(pairs) / pairs)
    y = ref.rotate(xd[:, :HQ + HKV], pos.astype(float), freq,
                   ref.pair_axes(pairs, sections, inter))
    # one rounding of the output, fp32 products and a table rounded to fp32
    u = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 0.0}[dtype] + 3e-7
    amp = np.abs(xd[:, :HQ + HKV]).max()
    live = np.repeat(np.array(slots) >= 0, T)
    off = np.abs(out.double().cpu().numpy()[live] - y[live, :HQ]).max()
    assert off <= 1.5 * u * amp
    assert (out[torch.from_numpy(~live)] == SENTINEL).all()
    assert (kout[torch.from_numpy(~live)] == SENTINEL).all()
    written = torch.zeros(c.k_pages.shape[1], page, dtype=torch.bool)
    for r, s in enumerate(slots):
        for i in range(T if s >= 0 else 0):
            at = lens[s] + i
            pg = int(c.table[s, at // page])
            written[pg, at % page] = True
            k = c.k_pages[1, pg, :, at % page].double().cpu().numpy()
            v = c.v_pages[1, pg, :, at % page].double().cpu().numpy()
            assert np.abs(k - y[r * T + i, HQ:]).max() <= 1.5 * u * amp
            assert np.array_equal(kout[r * T + i].double().cpu().numpy(), k)
            assert np.array_equal(v, xd[r * T + i, HQ + HKV:])
    same = (c.k_pages[1] == before[1]) | (c.k_pages[1].isnan() & before[1].isnan())
    assert same.transpose(1, 2)[~written].all()
    assert ((c.k_pages[0] == before[0]) | before[0].isnan()).all()


def test_append_ragged_in_place_and_default_positions():
    from linear_attention_state_rssm_gb300.store import RotaryTable
    rng = rng_of(22)
    HQ, HKV, D, page = 4, 2, 64, 16
    lens, cu = [3, 0, 30, 8], [0, 7, 7, 8, 20]
    c, _ = filled(rng, lens, 16, HQ, HKV, D, "f32", page)
    (q, qd), (k, kd), (v, _) = (draw(rng, (20, h, D), "f32") for h in (HQ, HKV, HKV))
    rope = RotaryTable.from_base(100, 32, 1e4)
    c.rssm_kv_append(0, q, k, v, ints([0, 1, 2, 3]), q_out=q, rope=rope, cu_seqlens=ints(cu))
    pos = np.concatenate([lens[r] + np.arange(cu[r + 1] - cu[r]) for r in range(4)])
    freq = 1e4 ** (-np.arange(32) / 32)
    y = ref.rotate(qd, pos[None].astype(float), freq, np.zeros(32, int))
    assert np.abs(q.double().cpu().numpy() - y).max() <= 1e-6 * np.abs(qd).max() * 2
    yk = ref.rotate(kd, pos[None].astype(float), freq, np.zeros(32, int))
    got = c.k_pages[0, int(c.table[3, 1]), :, 2].double().cpu().numpy()   # token 18 of slot 3
    assert np.abs(got - yk[18]).max() <= 1e-5
    c.rssm_kv_append(0, None, k, v, ints([0, 1, 2, 3]), cu_seqlens=ints(cu))   # no rotation
    assert torch.equal(c.k_pages[0, int(c.table[3, 1]), :, 2], k[18])
    assert c.rssm_kv_get_device_error() == 0


def test_append_refused_tokens():
    from linear_attention_state_rssm_gb300 import _lib as lib
    from linear_attention_state_rssm_gb300.store import RotaryTable
    rng = rng_of(23)
    c, _ = filled(rng, [14, 15], 1, 2, 1, 64, "bf16", 16)
    q, k, v = (draw(rng, (6, h, 64), "bf16")[0] for h in (2, 1, 1))
    c.rssm_kv_append(0, None, k, v, ints([0, 1]), 3)       # one page each: tokens 16, 17 do not fit
    assert c.rssm_kv_get_device_error() == lib.DEVERR["pages"]
    assert torch.equal(c.k_pages[0, int(c.table[0, 0]), :, 15], k[1])
    rope = RotaryTable.from_base(10, 32)
    c.rssm_kv_append(0, q[:2], k[:2], v[:2], ints([0, 1]), 1, torch.empty_like(q[:2]), rope=rope,
                     positions=ints([9, 10]))
    assert c.rssm_kv_get_device_error() == lib.DEVERR["position"]
    c.rssm_kv_append(0, None, k, v, ints([0, 1]), cu_seqlens=ints([0, 4, 2]))
    assert c.rssm_kv_get_device_error() & lib.DEVERR["seqlen"]
    c.rssm_kv_append(0, None, k[:2], v[:2], ints([0, 2]), 1)
    assert c.rssm_kv_get_device_error() == lib.DEVERR["slot"]


# --------------------------------------------------------------------- pages
def same_state(c, m):
    table = c.table.cpu().tolist()
    held = c.held.cpu().tolist()
    assert held == [len(t) for t in m.table]
    for row, t in zip(table, m.table):
        assert row == t + [-1] * (len(row) - len(t))
    assert c.length.cpu().tolist() == m.length
    assert c.refs.cpu().tolist() == m.refs
    assert c.k_pages[:, :, 0, 0, 0].long().cpu().tolist()[-1] == m.data
    flat = c.v_pages.flatten(2)
    assert torch.equal(flat, flat[:, :, :1].expand_as(flat))
    assert torch.equal(flat[0, :, 0], -flat[-1, :, 0])


def marked(n_slots, n_pages, page, max_pages, dtype="f32"):
    """Every page filled with its own number (layer 0: negated in v)."""
    c = cache(n_layers=3, n_slots=n_slots, HQ=2, HKV=2, D=64, n_pages=n_pages, page_size=page,
              max_pages=max_pages, dtype=dtype)
    ids = torch.arange(n_pages, device="cuda").to(TORCH[dtype]).view(-1, 1, 1, 1)
    c.k_pages.copy_(ids.expand(3, n_pages, 2, page, 64))
    c.v_pages.copy_(ids.expand(3, n_pages, 2, page, 64))
    c.v_pages[0].neg_()
    return c, ref.Pages(n_slots, n_pages, page, max_pages)


def test_pages_random_walk():
    """Reserve, commit, fork, release and compact in random order, the pool often
    empty, against the lists."""
    from linear_attention_state_rssm_gb300 import _lib as lib
    rng = rng_of(31)
    n_slots, n_pages, page, max_pages = 12, 60, 16, 9
    c, m = marked(n_slots, n_pages, page, max_pages)
    for step in range(150):
        what = rng.choice(["reserve", "reserve", "commit", "fork", "deep", "release", "compact"])
        rows = [int(s) for s in rng.permutation(n_slots)[:rng.integers(1, 6)]]
        if rng.random() < 0.3:
            rows[0] = -1
        m.failed = False
        if what == "reserve":
            n = [int(x) for x in rng.integers(0, 70, len(rows))]
            cu = ints(np.concatenate([[0], np.cumsum(n)]))
            c.rssm_kv_reserve(ints(rows), cu_seqlens=cu)
            m.reserve(rows, n)
        elif what == "commit":
            rows = [s for s in rows if s >= 0]
            room = [len(m.table[s]) * page - m.length[s] for s in rows]
            a = [int(rng.integers(0, r + 1)) for r in room]
            c.rssm_kv_commit(ints(rows), 200, accept_len=ints(a))
            for s, x in zip(rows, a):
                m.length[s] += x
        elif what in ("fork", "deep"):
            k = max(1, len(rows) // 2)
            dst = rows[:k]
            src = [int(x) for x in rng.choice([s for s in range(n_slots) if s not in dst], k)]
            c.rssm_kv_fork(ints(src), ints(dst), deep=what == "deep")
            m.fork(src, dst, what == "deep")
        elif what == "release":
            c.rssm_kv_release(ints(rows))
            m.release(rows)
        else:
            c.rssm_kv_compact()
            m.compact()
        want = lib.DEVERR["pages"] if m.failed else 0
        assert c.rssm_kv_get_device_error() == want, (step, what)
        same_state(c, m)


def test_pages_many_rows_and_a_large_pool():
    n = 1500
    c, m = marked(2 * n, 9000, 16, 4, "f32")
    slots = list(range(n))
    tokens = [int(x) for x in rng_of(32).integers(0, 64, n)]
    cu = ints(np.concatenate([[0], np.cumsum(tokens)]))
    c.rssm_kv_reserve(ints(slots), cu_seqlens=cu)
    c.rssm_kv_commit(ints(slots), cu_seqlens=cu)
    m.reserve(slots, tokens)
    m.length[:n] = tokens
    same_state(c, m)
    dst = [n + i for i in range(n)]
    c.rssm_kv_fork(ints(slots), ints(dst))
    m.fork(slots, dst)
    same_state(c, m)
    c.rssm_kv_release(ints(slots[::3] + dst[::2]))
    m.release(slots[::3] + dst[::2])
    c.rssm_kv_compact()
    m.compact()
    same_state(c, m)
    assert c.rssm_kv_get_device_error() == 0


def test_pages_refusals():
    from linear_attention_state_rssm_gb300 import _lib as lib
    c, _ = marked(3, 8, 16, 4)
    c.rssm_kv_reserve(ints([0, 7]), 20)
    assert c.rssm_kv_get_device_error() == lib.DEVERR["slot"]
    assert c.held.tolist() == [2, 0, 0]
    c.rssm_kv_reserve(ints([1]), 65)                      # five pages, table of four
    assert c.rssm_kv_get_device_error() == lib.DEVERR["pages"]
    c.rssm_kv_commit(ints([0]), 33)                       # past its pages
    assert c.rssm_kv_get_device_error() == lib.DEVERR["pages"]
    c.rssm_kv_commit(ints([0]), 4, accept_len=ints([5]))
    assert c.rssm_kv_get_device_error() == lib.DEVERR["accept"]
    c.rssm_kv_reserve(ints([0, 1]), cu_seqlens=ints([0, 5, 3]))
    assert c.rssm_kv_get_device_error() == lib.DEVERR["seqlen"]
    c.rssm_kv_fork(ints([0]), ints([0]))
    assert c.rssm_kv_get_device_error() == lib.DEVERR["slot"]
    c.rssm_kv_fork(ints([0]), ints([3]))
    assert c.rssm_kv_get_device_error() == lib.DEVERR["slot"]
    assert c.length.tolist() == [0, 0, 0] and c.held.tolist() == [2, 0, 0]


def test_index_tensors_that_the_kernels_would_misread_are_refused():
    from linear_attention_state_rssm_gb300.store import RotaryTable
    c, slot = cache(n_slots=4, HQ=2, HKV=1, D=64, n_pages=8, page_size=16), ints([0, 1])
    q, o = (torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k, cu, rope = q[:, :1], ints([0, 1, 2]), RotaryTable.from_base(64, 32)
    good = dict(slot=slot, cu=cu, cu_keys=None, accept=None, pos=None, q=q)

    def calls(slot, cu, cu_keys, accept, pos, q):
        return {"reserve": lambda: c.rssm_kv_reserve(slot, cu_seqlens=cu),
                "append": lambda: c.rssm_kv_append(0, q, k, k, slot, 1, o, rope, pos, cu),
                "decode": lambda: c.rssm_attn_decode(0, q, slot, 1, o),
                "prefill": lambda: c.rssm_attn_prefill(q, k, k, cu, slot, o, cu_keys=cu_keys),
                "commit": lambda: c.rssm_kv_commit(slot, 1, accept, cu),
                "fork": lambda: c.rssm_kv_fork(slot, ints([2, 3])),
                "release": lambda: c.rssm_kv_release(slot)}

    takes_slot = tuple(calls(**good))
    bad = [(dict(slot=s), takes_slot) for s in (slot.long(), slot.cpu(), ints([0, 9, 1, 9])[::2])]
    bad += [(dict(slot=ints([0])), ("reserve", "append", "decode", "prefill", "commit", "fork"))]
    bad += [(dict(cu=x), ("reserve", "append", "prefill", "commit"))
            for x in (cu[:2], cu.long(), cu.cpu())]
    bad += [(dict(cu_keys=cu[:2]), ("prefill",)), (dict(accept=ints([1])), ("commit",)),
            (dict(accept=ints([1, 1]).long()), ("commit",)), (dict(pos=ints([0])), ("append",)),
            (dict(q=q.cpu()), ("append", "decode", "prefill"))]
    for change, names in bad:
        for name in names:
            with pytest.raises(ValueError):
                calls(**{**good, **change})[name]()
    assert c.held.tolist() == [0] * 4
    for call in calls(**good).values():
        call()
    assert c.rssm_kv_get_device_error() == 0


# ------------------------------------------------------------------ together
def test_a_cache_through_a_conversation():
    """Prompt, draft windows with rejections, a fork and decode steps, captured
    in a graph and on another stream than the tensors' own."""
    rng = rng_of(41)
    HQ, HKV, D, page, dtype, T = 4, 2, 64, 16, "bf16", 4
    c = cache(n_layers=1, n_slots=4, HQ=HQ, HKV=HKV, D=D, n_pages=40, page_size=page,
              max_pages=12, dtype=dtype)
    lq = [21, 50]
    cu = [0, 21, 71]
    hist = [[], []]
    st = torch.cuda.Stream()
    slot = ints([0, 1])
    (q, qd), (k, kd), (v, vd) = (draw(rng, (71, h, D), dtype) for h in (HQ, HKV, HKV))
    o = torch.empty_like(q)
    cu_t = ints(cu)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        c.rssm_kv_reserve(slot, cu_seqlens=cu_t)
        c.rssm_kv_append(0, None, k, v, slot, cu_seqlens=cu_t)
        c.rssm_attn_prefill(q, k, v, cu_t, slot, o)
        c.rssm_kv_commit(slot, cu_seqlens=cu_t)
    st.synchronize()
    want, _, mass = ref.prompt(qd, kd, vd, cu, cu, c.scale)
    check(o, want, mass, dtype)
    for r in range(2):
        hist[r] = [kd[cu[r]:cu[r + 1]], vd[cu[r]:cu[r + 1]]]
    bufs = [torch.empty((2 * T, h, D), dtype=TORCH[dtype], device="cuda")
            for h in (HQ, HKV, HKV, HQ)]
    acc = ints([0, 0])

    def step():
        c.rssm_kv_reserve(slot, T)
        c.rssm_kv_append(0, None, bufs[1], bufs[2], slot, T)
        c.rssm_attn_decode(0, bufs[0], slot, T, bufs[3])
        c.rssm_kv_commit(slot, T, accept_len=acc)

    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(6):
        data = [draw(rng, (2 * T, h, D), dtype) for h in (HQ, HKV, HKV)]
        for b, (x, _) in zip(bufs, data):
            b.copy_(x)
        a = rng.integers(0, T + 1, 2)
        acc.copy_(ints(a))
        g.replay()
        torch.cuda.synchronize()
        tokens = [[np.concatenate([hist[r][j], data[1 + j][1][r * T:r * T + T]])
                   for j in range(2)] for r in range(2)]
        want, _, mass = ref.window(data[0][1], tokens, [len(h[0]) for h in hist], T, c.scale)
        check(bufs[3], want, mass, dtype)
        for r in range(2):
            hist[r] = [x[:len(x) - T + a[r]] for x in tokens[r]]
        assert c.length[:2].tolist() == [len(h[0]) for h in hist]
    c.rssm_kv_fork(ints([1]), ints([2]))
    slot = ints([1, 2])
    for _ in range(3):      # both go on from the same tokens, each with its own
        data = [draw(rng, (2, h, D), dtype) for h in (HQ, HKV, HKV)]
        hist = hist if len(hist) == 3 else [hist[0], hist[1], list(hist[1])]
        c.rssm_kv_reserve(slot, 1)
        c.rssm_kv_append(0, None, data[1][0], data[2][0], slot, 1)
        o = torch.empty_like(data[0][0])
        c.rssm_attn_decode(0, data[0][0], slot, 1, o)
        c.rssm_kv_commit(slot, 1)
        lens = [len(hist[r + 1][0]) for r in range(2)]
        for r in range(2):
            hist[r + 1] = [np.concatenate([hist[r + 1][j], data[1 + j][1][r:r + 1]])
                           for j in range(2)]
        want, _, mass = ref.window(data[0][1], hist[1:], lens, 1, c.scale)
        check(o, want, mass, dtype)
    assert c.rssm_kv_get_device_error() == 0
