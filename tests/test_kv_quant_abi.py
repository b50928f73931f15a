"""Host-side checks of quantised caches, norms in the append and pages read in a
row (no GPU): what is refused before anything is launched."""
import ctypes
from types import SimpleNamespace

import pytest
import torch

from linear_attention_state_rssm_gb300 import _lib, build
from linear_attention_state_rssm_gb300.store import HeadNorm, KVCache


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def config(**kw):
    base = dict(n_layers=3, n_slots=5, HQ=16, HKV=4, D=128, n_pages=100, page_size=32, max_pages=7,
                dtype="bf16")
    return _lib.make_kv_config(**{**base, **kw})


def test_required_bytes(lib):
    s, scales = _lib.rssm_kv_quant_required_bytes(config())
    rows = 3 * 100 * 4 * 32
    assert s.k_pages == s.v_pages == rows * 128 and scales == rows * 2
    plain = _lib.rssm_kv_required_bytes(config())
    assert (s.table, s.held, s.length, s.refs, s.work) == \
        (plain.table, plain.held, plain.length, plain.refs, plain.work)


@pytest.mark.parametrize("kw,status", [(dict(dtype="f32"), 2), (dict(D=96), 2), (dict(HQ=6), 1),
                                       (dict(page_size=8), 2), (dict(scale=-1.0), 1)])
def test_configuration_refusals(lib, kw, status):
    with pytest.raises(_lib.RssmError) as e:
        _lib.rssm_kv_quant_required_bytes(config(**kw))
    assert e.value.status == status


@pytest.mark.parametrize("scales", [None, 0x9008])
def test_alloc_refuses_bad_scales_before_touching_the_device(lib, scales):
    bufs = _lib.rssm_kv_buffers(*(0x1000 * (i + 1) for i in range(8)))
    with pytest.raises(_lib.RssmError) as e:
        _lib.rssm_kv_quant_alloc(config(), bufs, scales)
    assert e.value.status == 1


def test_null_arguments_are_refused(lib):
    for call in (lambda: _lib.rssm_kv_gather(None, 0, None, None, None, 1, 1, 1, None, None,
                                             stream=0),
                 lambda: _lib.rssm_kv_append_norm(None, 0, None, None, None, 0, 0, 0, None, None,
                                                  None, None, None, 1, 1, 1, None, stream=0)):
        with pytest.raises(_lib.RssmError) as e:
            call()
        assert e.value.status == 1
    cfg = config()
    assert lib.rssm_kv_quant_required_bytes(ctypes.byref(cfg), None, None) == 1


def test_page_types_that_are_not_built_are_refused():
    for kind in ("e5m2", "int8", "f32"):
        with pytest.raises(ValueError):
            KVCache(dtype="bf16", page_dtype=kind)


def test_norm_weights_off_the_device_are_refused():
    with pytest.raises(ValueError):
        HeadNorm(torch.ones(64))
    assert HeadNorm().D is None


def like(shape, dtype=torch.bfloat16, is_cuda=True, contiguous=True):
    t = torch.zeros(shape, dtype=dtype)
    return SimpleNamespace(dtype=dtype, shape=t.shape, is_cuda=is_cuda, numel=t.numel,
                           stride=t.stride, is_contiguous=lambda: contiguous)


@pytest.mark.parametrize("kw", [dict(is_cuda=False), dict(dtype=torch.float32),
                                dict(shape=(3, 2, 64)), dict(contiguous=False)])
def test_rows_that_the_kernels_cannot_write_are_refused(kw):
    kv = SimpleNamespace(HKV=2, D=64, _torch_dtype=torch.bfloat16)
    KVCache._row(kv, "v_out", like((4, 2, 64)), 4)
    with pytest.raises(ValueError):
        KVCache._row(kv, "v_out", like(**{"shape": (4, 2, 64), **kw}), 4)


def test_share_buffers(lib):
    cfg = config()
    n = _lib.rssm_kv_share_bytes(cfg, 64, 2)
    # outputs of every query row, of 2 x 152 stretches of 128 rows, lists of the rows
    out = (64 * 2 * 16 + 2 * 152 * 128) * (128 + 2) * 4
    segs = 152 + 4 * (64 * 2 * 4 // 128 + 64 // 2 + 1)
    assert out + 32 * segs <= n <= out + 32 * segs + 12 * 64 * 4 + 16 * 256
    small = (2 * 16 + 2 * 152 * 8) * (128 + 2) * 4     # eight rows of a key head in all
    assert small <= _lib.rssm_kv_share_bytes(cfg, 2, 1) <= small + 32 * 160 + 17 * 256
    assert _lib.rssm_kv_share_bytes(cfg, 0, 1) >= 16
    for B, T, status in ((-1, 1, 1), (65536, 1, 1), (4, 0, 1), (4, 65, 2)):
        with pytest.raises(_lib.RssmError) as e:
            _lib.rssm_kv_share_bytes(cfg, B, T)
        assert e.value.status == status
    for call in (lambda: _lib.rssm_kv_share(None, None, 1, 1, 0x1000, stream=0),
                 lambda: _lib.rssm_attn_decode_shared(None, 0, None, 0, None, 1, 1, 0x1000, None,
                                                      None, stream=0)):
        with pytest.raises(_lib.RssmError) as e:
            call()
        assert e.value.status == 1


def test_plans_of_other_batches_are_refused():
    kv = SimpleNamespace()
    share = SimpleNamespace(cache=kv, B=4, T=2)
    KVCache._shared(kv, share, 4, 2)
    for args in ((kv, share, 3, 2), (kv, share, 4, 1), (SimpleNamespace(), share, 4, 2)):
        with pytest.raises(ValueError):
            KVCache._shared(*args)
