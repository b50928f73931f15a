"""Norms in the append, quantised pages and pages read in a row, against the fp64
oracle.

Tolerances. A norm takes an fp32 sum of at most 256 squares (a tree of at most 16
+ 5 steps: 21 x 2^-24), a root of 2 ulp and two products, the rotation two
products and a table rounded to fp32: below 40 x 2^-24 = 2.4e-6 of the head's
largest value, and the output is rounded once, by u = 2^-8 / 2^-11 / 2^-24 of
itself at most. An e4m3 page holds a value to half a step, 2^-4 of it or 2^-10
2^e where that is more; what is quantised without a norm and a rotation is
exact, code by code, and so is whatever is read back.
"""
import numpy as np
import pytest
import torch

from oracle import attention as ref
from oracle import quant

pytestmark = pytest.mark.gpu
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
FP32 = 2.4e-6
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


def draw(rng, shape, dtype, by=1.0):
    t = torch.from_numpy(by * rng.standard_normal(shape)).to(TORCH[dtype])
    return t.cuda(), t.double().numpy()


def ints(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def laid_out(rng, lens, T, page, **kw):
    """A cache whose slots hold lens tokens and room for T more, in shuffled pages."""
    counts = [-(-(n + T) // page) for n in lens]
    c = cache(n_slots=len(lens), n_pages=sum(counts) + 2, page_size=page,
              max_pages=max(counts) + 1, **kw)
    order = rng.permutation(sum(counts) + 2)
    at = 0
    for s, n in enumerate(lens):
        c.table[s, :counts[s]] = ints(order[at:at + counts[s]])
        at += counts[s]
        c.held[s], c.length[s] = counts[s], n
    return c


def codes_of(pages):
    return pages.view(torch.uint8).cpu().numpy()


def put(c, layer, rng, dtype):
    """Random pages of a layer; the values they stand for, [n_pages, HKV, page, D] each."""
    out = []
    for which, pool in enumerate((c.k_pages, c.v_pages)):
        x = rng.standard_normal(pool.shape[1:])
        if c.page_scales is None:
            t = torch.from_numpy(x).to(TORCH[dtype])
            pool[layer] = t.cuda()
            out.append(t.double().numpy())
        else:
            x = x * 2.0 ** rng.uniform(-8, 8, x.shape[:-1])[..., None]
            codes, scale = quant.quantise(x)
            pool[layer].view(torch.uint8).copy_(torch.from_numpy(codes))
            c.page_scales[layer, ..., which] = torch.from_numpy(scale).cuda()
            out.append(quant.value(codes, scale))
    return out


# -------------------------------------------------------------------- append
def near(got, want, amp, dtype):
    off = np.abs(got - want)
    lim = U[dtype] * np.abs(want) + FP32 * amp + 2.0 ** -25 * (dtype == "f16")
    assert np.all(off <= lim), (off / lim).max()


@pytest.mark.parametrize("dtype,pages", [("bf16", None), ("f16", None), ("f32", None),
                                         ("bf16", "e4m3"), ("f16", "e4m3")])
@pytest.mark.parametrize("D,pairs,sections,inter", [
    (64, 32, [32], False), (128, 64, [24, 20, 20], True), (256, 32, [32], False),
    (256, 128, [100, 28], False), (128, 0, None, False)])
def test_append_with_norms(dtype, pages, D, pairs, sections, inter):
    from linear_attention_state_rssm_gb300.store import HeadNorm, RotaryTable
    rng = np.random.default_rng([D, pairs])
    HQ, HKV, T, page, most = 6, 2, 5, 16, 5000
    lens = [0, 14, 16, 29]
    c = laid_out(rng, lens, T, page, n_layers=2, HQ=HQ, HKV=HKV, D=D, dtype=dtype,
                 page_dtype=pages)
    x, xd = draw(rng, (4 * T, HQ + 2 * HKV, D), dtype, 1.7)
    (qw, qwd), (kw, kwd) = (draw(rng, D, "f32") for _ in range(2))
    eps = 1e-5
    rope = pos = None
    if pairs:
        pos = rng.integers(0, most, (len(sections), 4 * T))
        rope = RotaryTable.from_base(most, pairs, 1e4, sections, inter)
    out = torch.full((4 * T, HQ, D), SENTINEL, dtype=TORCH[dtype], device="cuda")
    kout = torch.full((4 * T, HKV, D), SENTINEL, dtype=TORCH[dtype], device="cuda")
    vout = kout.clone()
    slots = [2, -1, 0, 3]
    c.rssm_kv_append(1, x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], ints(slots), T, out,
                     rope=rope, positions=None if pos is None else torch.from_numpy(pos).int().cuda(),
                     k_out=kout, norm=HeadNorm(qw, kw, eps), v_out=vout)
    assert c.rssm_kv_get_device_error() == 0
    y = np.concatenate([quant.norm(xd[:, :HQ], qwd, eps),
                        quant.norm(xd[:, HQ:HQ + HKV], kwd, eps)], 1)
    if pairs:
        freq = 1e4 ** (-np.arange(pairs) / pairs)
        y = ref.rotate(y, pos.astype(float), freq, ref.pair_axes(pairs, sections, inter))
    amp = np.abs(y).max(-1, keepdims=True)
    live = np.repeat(np.array(slots) >= 0, T)
    dead = torch.from_numpy(~live)
    for t in (out, kout, vout):
        assert (t[dead] == SENTINEL).all()
    near(out.double().cpu().numpy()[live], y[live, :HQ], amp[live, :HQ], dtype)
    kp, vp = (codes_of(p) if pages else p.double().cpu().numpy() for p in (c.k_pages, c.v_pages))
    sc = c.page_scales.cpu().numpy() if pages else None
    written = np.zeros((c.n_pages, page), bool)
    for r, s in enumerate(slots):
        for i in range(T if s >= 0 else 0):
            n, at = r * T + i, lens[s] + i
            pg, o = int(c.table[s, at // page]), at % page
            written[pg, o] = True
            k, v = kp[1, pg, :, o], vp[1, pg, :, o]
            if pages:
                ks, vs = sc[1, pg, :, o, 0], sc[1, pg, :, o, 1]
                vc, ve = quant.quantise(xd[n, HQ + HKV:])
                assert np.array_equal(v, vc) and np.array_equal(vs, ve)
                top = np.abs(y[n, HQ:]).max(-1)
                for h in range(HKV):   # the power is the oracle's but at the very border
                    assert int(ks[h]) - 127 in (quant.exponent(top[h] * (1 - 1e-5)),
                                                quant.exponent(top[h] * (1 + 1e-5)))
                k, v = quant.value(k, ks), quant.value(v, vs)
                e = ks.astype(float)[:, None] - 127
                step = np.maximum(2.0 ** -4 * np.abs(y[n, HQ:]), 2.0 ** -10 * 2.0 ** e)
                assert np.all(np.abs(k - y[n, HQ:]) <= step + 1.1 * FP32 * amp[n, HQ:])
            else:
                near(k, y[n, HQ:], amp[n, HQ:], dtype)
                assert np.array_equal(v, xd[n, HQ + HKV:])
            assert np.array_equal(kout[n].double().cpu().numpy(), k)
            assert np.array_equal(vout[n].double().cpu().numpy(), v)
    assert not kp[0].any() and not vp[0].any()
    assert not kp[1].transpose(0, 2, 1, 3)[~written].any()
    if pages:
        assert not sc[0].any() and not sc[1].transpose(0, 2, 1, 3)[~written].any()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_one_norm_alone_and_the_call_without(dtype):
    """A null weight leaves its heads bit for bit as the plain append has them."""
    from linear_attention_state_rssm_gb300.store import HeadNorm, RotaryTable
    rng = np.random.default_rng(5)
    HQ, HKV, D, T = 4, 2, 64, 3
    x = draw(rng, (2 * T, HQ + 2 * HKV, D), dtype)[0]
    w = torch.full((D,), 1.5, device="cuda")
    rope = RotaryTable.from_base(100, 32)
    got = {}
    for name, norm in (("none", None), ("null", HeadNorm()), ("q", HeadNorm(w)),
                       ("k", HeadNorm(None, w))):
        c = laid_out(np.random.default_rng(6), [3, 20], T, 16, HQ=HQ, HKV=HKV, D=D, dtype=dtype)
        out = torch.zeros((2 * T, HQ, D), dtype=TORCH[dtype], device="cuda")
        vout = torch.zeros((2 * T, HKV, D), dtype=TORCH[dtype], device="cuda")
        c.rssm_kv_append(0, x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], ints([0, 1]), T, out,
                         rope=rope, norm=norm, v_out=vout)
        assert torch.equal(vout, x[:, HQ + HKV:])
        got[name] = out, c.k_pages
        if name == "none":
            c.rssm_kv_append(0, x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], ints([0, 1]), T,
                             out, rope=rope)
            got["plain"] = out, c.k_pages
    for name, q_same, k_same in (("none", 1, 1), ("null", 1, 1), ("q", 0, 1), ("k", 1, 0)):
        assert torch.equal(got[name][0], got["plain"][0]) == bool(q_same)
        assert torch.equal(got[name][1], got["plain"][1]) == bool(k_same)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_of_large_small_and_zero_heads(dtype):
    """Squares past fp32's range, squares below it, zeros, and heads with an infinity or a
    NaN, which become NaN there and zeros elsewhere (infinity) or NaN throughout."""
    from linear_attention_state_rssm_gb300.store import HeadNorm
    rng = np.random.default_rng(8)
    D, eps = 128, 1e-6
    size = np.array([1e30, 3e38 / 8, 1e19, 1e-25, 0.0, 1.0, 1.0])
    x = rng.uniform(-1, 1, (7, 1, D)) * size[:, None, None]
    x[5, 0, 3], x[6, 0, 4] = np.inf, np.nan
    q = torch.from_numpy(x).to(TORCH[dtype]).cuda()
    qd = q.double().cpu().numpy()
    c = cache(n_slots=1, HQ=1, HKV=1, D=D, n_pages=1, page_size=16, dtype=dtype)
    c.table[0, 0], c.held[0] = 0, 1
    out, kv = torch.zeros_like(q), torch.zeros_like(q)
    w, wd = draw(rng, D, "f32")
    c.rssm_kv_append(0, q, kv, kv, ints([0]), 7, out, norm=HeadNorm(w, w, eps))
    got = out.double().cpu().numpy()
    want = quant.norm(qd[:5], wd, eps)
    near(got[:5], want, np.abs(want).max(-1, keepdims=True), dtype)
    assert np.isnan(got[5, 0, 3]) and not got[5, 0, 4:].any()
    assert np.isnan(got[6]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_quantised_codes_of_every_kind_of_value(dtype, D):
    """Borders of the powers of two, ties, subnormals, signed zeros, infinities, NaN,
    saturation: code by code, in the pages, k_out and v_out, and read back."""
    rng = np.random.default_rng(D)
    n = 40
    x = rng.standard_normal((n, 2, D)) * 2.0 ** rng.integers(-12, 9, (n, 2, 1))
    x[0], x[1] = 0.0, -0.0
    x[2, :, 0], x[3, :, 0] = 448.0, 449.0 if dtype == "f16" else 450.0
    x[2, :, 1:], x[3, :, 1:] = rng.choice([17, 18, 19, 27, 0.5, 2 ** -10, 3 * 2.0 ** -10, -2 ** -9],
                                          (2, D - 1))
    x[4, 0, 5], x[5, 1, 6], x[6, 0, 7] = np.inf, -np.inf, np.nan
    x[7] = np.nan
    x[8] = 2.0 ** -24
    if dtype == "bf16":
        x[9], x[10], x[11] = 1e30, -3e38, 1e-38
        x[12, :, ::2] = 1e-30
    v = torch.from_numpy(x).to(TORCH[dtype]).cuda()
    vd = v.double().cpu().numpy()
    c = laid_out(rng, [7], n, 16, HQ=2, HKV=2, D=D, dtype=dtype, page_dtype="e4m3")
    k = v.flip(0).contiguous()
    kd = k.double().cpu().numpy()
    kout, vout = torch.zeros_like(v), torch.zeros_like(v)
    c.rssm_kv_append(0, None, k, v, ints([0]), n, k_out=kout, v_out=vout)
    back = [torch.zeros_like(v) for _ in range(2)]
    c.rssm_kv_gather(0, ints([0]), *back, T=n, first=ints([7]))
    assert c.rssm_kv_get_device_error() == 0
    for which, (xd, pages, row, again) in enumerate(((kd, c.k_pages, kout, back[0]),
                                                     (vd, c.v_pages, vout, back[1]))):
        codes, scale = quant.quantise(xd)
        want = torch.from_numpy(quant.value(codes, scale)).to(TORCH[dtype])
        got_c, got_s = codes_of(pages), c.page_scales.cpu().numpy()
        for i in range(n):
            pg, o = int(c.table[0, (7 + i) // 16]), (7 + i) % 16
            nan = codes[i] & 127 == 127
            assert np.array_equal(got_c[0, pg, :, o][~nan], codes[i][~nan])
            assert (got_c[0, pg, :, o][nan] & 127 == 127).all()
            assert np.array_equal(got_s[0, pg, :, o, which], scale[i])
        for t in (row, again):
            assert torch.equal(torch.nan_to_num(t.cpu(), nan=SENTINEL),
                               torch.nan_to_num(want, nan=SENTINEL))


def test_quantised_append_in_place():
    """k_out and v_out may be k and v themselves."""
    rng = np.random.default_rng(3)
    c = laid_out(rng, [0, 5], 9, 16, HQ=2, HKV=2, D=64, dtype="bf16", page_dtype="e4m3")
    (k, kd), (v, vd) = (draw(rng, (18, 2, 64), "bf16") for _ in range(2))
    c.rssm_kv_append(0, None, k, v, ints([0, 1]), 9, k_out=k, v_out=v)
    for t, d in ((k, kd), (v, vd)):
        assert np.array_equal(t.double().cpu().numpy(), quant.value(*quant.quantise(d)))


def test_append_refuses_bad_norms():
    from linear_attention_state_rssm_gb300 import _lib as lib
    from linear_attention_state_rssm_gb300.store import HeadNorm
    c = laid_out(np.random.default_rng(1), [0], 2, 16, HQ=2, HKV=1, D=64)
    q, k = torch.zeros(2, 2, 64).bfloat16().cuda(), torch.zeros(2, 1, 64).bfloat16().cuda()
    w = torch.ones(68, device="cuda")

    def call(norm, **kw):
        c.rssm_kv_append(0, q, k, k, ints([0]), 2, q.clone(), norm=norm, **kw)
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(lib.RssmError):
            call(HeadNorm(w[:64], None, eps))
    with pytest.raises(lib.RssmError):
        call(HeadNorm(w[1:65]))                       # not 16-byte aligned
    with pytest.raises(ValueError):
        call(HeadNorm(torch.ones(128, device="cuda")))
    for bad in (w[:64].double(), w[::2], w.view(4, 17), w[:64].cpu()):
        with pytest.raises(ValueError):
            HeadNorm(bad)
    with pytest.raises(ValueError):
        HeadNorm(w[:64], w[:68])
    with pytest.raises(ValueError):
        call(None, v_out=torch.zeros(2, 2, 64).bfloat16().cuda())


# -------------------------------------------------------------------- gather
@pytest.mark.parametrize("dtype,pages", [("bf16", None), ("f16", None), ("f32", None),
                                         ("bf16", "e4m3"), ("f16", "e4m3")])
@pytest.mark.parametrize("D,HKV,page", [(64, 1, 16), (128, 3, 64), (256, 2, 256), (64, 8, 32)])
def test_gather_rows_of_many_lengths(dtype, pages, D, HKV, page):
    rng = np.random.default_rng([D, HKV])
    lens = [0, 1, page - 1, page, page + 1, 333, 5, 40]
    c = laid_out(rng, lens, 3, page, n_layers=2, HQ=HKV, HKV=HKV, D=D, dtype=dtype,
                 page_dtype=pages)
    kd, vd = put(c, 1, rng, dtype)
    first = [0, 0, 3, page // 2, 0, 100, 6, 0]
    # up to what the pages hold, committed or not; a slot twice
    slots = [0, 1, 2, 3, 4, 5, -1, 5]
    lq = [3, 4, page - 1, page // 2 + 1, 2, 233, 9, 336]
    cu = np.concatenate([[0], np.cumsum(lq)])
    N = int(cu[-1])
    k, v = (torch.full((N, HKV, D), SENTINEL, dtype=TORCH[dtype], device="cuda")
            for _ in range(2))
    c.rssm_kv_gather(1, ints(slots), k, v, cu_seqlens=ints(cu), first=ints(first))
    assert c.rssm_kv_get_device_error() == 0
    for r, s in enumerate(slots):
        a, b = cu[r], cu[r + 1]
        if s < 0:
            assert (k[a:b] == SENTINEL).all() and (v[a:b] == SENTINEL).all()
            continue
        at = first[r] + np.arange(lq[r])
        pg = c.table[s].cpu().numpy()[at // page]
        for t, d in ((k, kd), (v, vd)):
            want = torch.from_numpy(d[pg, :, at % page]).to(TORCH[dtype])
            assert torch.equal(t[a:b].cpu(), want)
    # windows of one length from the beginning, keys alone
    one = torch.zeros(16, HKV, D, dtype=TORCH[dtype], device="cuda")
    c.rssm_kv_gather(1, ints([5, 7]), one, None, T=8)
    for r, s in enumerate((5, 7)):
        pg = int(c.table[s, 0])
        want = torch.from_numpy(kd[pg, :, :8].transpose(1, 0, 2)).to(TORCH[dtype])
        assert torch.equal(one[8 * r:8 * r + 8].cpu(), want)


@pytest.mark.parametrize("pages", [None, "e4m3"])
def test_gather_skips_what_is_not_there(pages):
    from linear_attention_state_rssm_gb300 import _lib as lib
    rng = np.random.default_rng(4)
    c = laid_out(rng, [10, 20], 1, 16, HQ=1, HKV=1, D=64, page_dtype=pages)
    kd, _ = put(c, 0, rng, "bf16")

    def call(slot, first, T=8, cu=None, n=None):
        k, v = (torch.full((n or len(slot) * T, 1, 64), SENTINEL, device="cuda").bfloat16()
                for _ in range(2))
        c.rssm_kv_gather(0, ints(slot), k, v, T=T, first=ints(first),
                         cu_seqlens=None if cu is None else ints(cu))
        return k, c.rssm_kv_get_device_error()

    k, err = call([0, 1], [12, 30])                  # 16 and 32 tokens have room
    assert err == lib.DEVERR["pages"]
    assert (k[4:8] == SENTINEL).all() and (k[10:] == SENTINEL).all()
    want = torch.from_numpy(kd[int(c.table[0, 0]), 0, 12:]).bfloat16()
    assert torch.equal(k[:4, 0].cpu(), want)
    k, err = call([0, 1], [-1, 2**31 - 4])
    assert err == lib.DEVERR["pages"] and (k == SENTINEL).all()
    k, err = call([2, -5], [0, 0])
    assert err == lib.DEVERR["slot"] and (k == SENTINEL).all()
    c.table[0, 0] = 999
    k, err = call([0, 1], [0, 0])
    assert err == lib.DEVERR["pages"] and (k[:8] == SENTINEL).all() and (k[8:] != SENTINEL).any()
    k, err = call([0, 1], [0, 0], cu=[0, 9, 4], n=12)
    assert err & lib.DEVERR["seqlen"]
    k, err = call([1, 1], [0, 0], cu=[0, 5, 99], n=12)
    assert err == lib.DEVERR["seqlen"] and (k[5:] == SENTINEL).all()
    with pytest.raises(lib.RssmError):
        c.rssm_kv_gather(1, ints([0]), k[:1], None)
    with pytest.raises(ValueError):
        c.rssm_kv_gather(0, ints([0, 1]), k[:3], None, T=2)
    with pytest.raises(ValueError):
        c.rssm_kv_gather(0, ints([0, 1]), k, None, T=6, first=ints([0]))
    with pytest.raises(ValueError):
        c.rssm_kv_gather(0, ints([0, 1]).long(), k, None, T=6)
    c.rssm_kv_gather(0, ints([0, 1]), None, None, T=6)
    c.rssm_kv_gather(0, ints([]), k[:0], k[:0], T=6)
    assert c.rssm_kv_get_device_error() == 0


@pytest.mark.parametrize("pages", [None, "e4m3"])
def test_append_and_gather_past_32_bit_offsets(pages):
    """A pool of more than 2^32 bytes of keys: its last pages are written and read."""
    D, HKV, page = 256, 4, 256
    n = (1 << 32) // (HKV * page * D) * (1 if pages else 1) + 40
    c = cache(HQ=HKV, HKV=HKV, D=D, n_pages=n, page_size=page, max_pages=2, dtype="bf16",
              page_dtype=pages)
    c.table[0, 0], c.table[0, 1] = n - 1, n - 3
    c.held[0], c.length[0] = 2, 250
    rng = np.random.default_rng(2)
    (k, kd), (v, vd) = (draw(rng, (20, HKV, D), "bf16") for _ in range(2))
    c.rssm_kv_append(0, None, k, v, ints([0]), 20)
    a, b = torch.zeros_like(k), torch.zeros_like(k)
    c.rssm_kv_gather(0, ints([0]), a, b, T=20, first=ints([250]))
    assert c.rssm_kv_get_device_error() == 0
    for t, d in ((a, kd), (b, vd)):
        want = quant.value(*quant.quantise(d)) if pages else d
        assert np.array_equal(t.double().cpu().numpy(), want)
    assert (c.k_pages[0, n - 3, :, 13].view(torch.uint8) != 0).any()


# --------------------------------------------------------------------- pages
def test_quantised_pages_move_with_their_scales():
    """Fork (shallow and deep), release and compaction against the lists: every page's
    codes and scales are its own number's."""
    rng = np.random.default_rng(31)
    n_slots, n_pages, page, max_pages = 10, 50, 16, 9
    c = cache(n_layers=3, n_slots=n_slots, HQ=2, HKV=2, D=64, n_pages=n_pages, page_size=page,
              max_pages=max_pages, dtype="bf16", page_dtype="e4m3")
    m = ref.Pages(n_slots, n_pages, page, max_pages)
    ids = torch.arange(n_pages, device="cuda", dtype=torch.uint8).view(-1, 1, 1, 1)
    c.k_pages.view(torch.uint8).copy_(ids.expand(3, n_pages, 2, page, 64))
    c.v_pages.view(torch.uint8).copy_(100 + ids.expand(3, n_pages, 2, page, 64))
    c.page_scales.copy_(50 + ids[None].expand(3, n_pages, 2, page, 2))
    c.page_scales[1, ..., 1] += 7
    for step in range(60):
        what = rng.choice(["reserve", "reserve", "commit", "fork", "deep", "release", "compact"])
        rows = [int(s) for s in rng.permutation(n_slots)[:rng.integers(1, 6)]]
        if what == "reserve":
            T = int(rng.integers(1, 50))
            c.rssm_kv_reserve(ints(rows), T)
            m.reserve(rows, [T] * len(rows))
        elif what == "commit":
            acc = [int(rng.integers(0, len(m.table[s]) * page - m.length[s] + 1)) for s in rows]
            c.rssm_kv_commit(ints(rows), 200, accept_len=ints(acc))
            for s, a in zip(rows, acc):
                m.length[s] += a
        elif what in ("fork", "deep"):
            dst = [int(s) for s in rng.permutation(n_slots) if s not in rows][:len(rows)]
            rows = rows[:len(dst)]
            c.rssm_kv_fork(ints(rows), ints(dst), deep=what == "deep")
            m.fork(rows, dst, what == "deep")
        elif what == "release":
            c.rssm_kv_release(ints(rows[:2]))
            m.release(rows[:2])
        else:
            c.rssm_kv_compact()
            m.compact()
        assert c.refs.cpu().tolist() == m.refs and c.length.cpu().tolist() == m.length
        want = torch.tensor(m.data, dtype=torch.uint8, device="cuda").view(-1, 1, 1, 1)
        assert torch.equal(c.k_pages.view(torch.uint8), want.expand(3, n_pages, 2, page, 64))
        assert torch.equal(c.v_pages.view(torch.uint8), 100 + want.expand(3, n_pages, 2, page, 64))
        sc = (50 + want[None].expand(3, n_pages, 2, page, 2)).clone()
        sc[1, ..., 1] += 7
        assert torch.equal(c.page_scales, sc)


# ------------------------------------------------------------ streams, graphs
@pytest.mark.parametrize("pages", [None, "e4m3"])
def test_append_and_gather_on_a_stream_and_in_a_graph(pages):
    """New inputs in the same buffers: the replay writes and reads what they hold then."""
    from linear_attention_state_rssm_gb300.store import HeadNorm, RotaryTable
    rng = np.random.default_rng(12)
    c = laid_out(rng, [3, 30], 4, 16, HQ=2, HKV=2, D=128, page_dtype=pages)
    x = draw(rng, (8, 6, 128), "bf16")[0]
    w = draw(rng, 128, "f32")[0]
    norm, rope, slot = HeadNorm(w, w), RotaryTable.from_base(64, 64), ints([0, 1])
    q_out, k_out, v_out = (torch.zeros(8, 2, 128, device="cuda").bfloat16() for _ in range(3))
    back = [torch.zeros_like(k_out) for _ in range(2)]

    def step():
        c.rssm_kv_append(0, x[:, :2], x[:, 2:4], x[:, 4:], slot, 4, q_out, rope=rope, norm=norm,
                         k_out=k_out, v_out=v_out)
        c.rssm_kv_gather(0, slot, *back, T=4, first=c.length)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    x.copy_(draw(rng, (8, 6, 128), "bf16")[0])
    graph.replay()
    got = [t.clone() for t in (q_out, k_out, v_out, *back)]
    step()
    for a, b in zip(got, (q_out, k_out, v_out, *back)):
        assert torch.equal(a, b)
    assert torch.equal(back[0], k_out) and torch.equal(back[1], v_out)
