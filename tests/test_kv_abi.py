"""Host-side checks of the key-value cache's and its attention's entry points
(no GPU): configurations, buffers and arguments that are refused before
anything is launched."""
import numpy as np
import pytest

from linear_attention_state_rssm_gb300 import _lib, build
from oracle import attention as ref


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_required_bytes_matches_layouts(lib):
    s = _lib.rssm_kv_required_bytes(_lib.make_kv_config(3, 5, 16, 4, 128, 100, 32, 7, "bf16"))
    assert s.k_pages == s.v_pages == 3 * 100 * 4 * 32 * 128 * 2
    assert s.table == 5 * 7 * 4 and s.held == s.length == 20 and s.refs == 400
    assert s.err_word == 4
    assert s.work >= 2 * 304 * 4096 * 4 + 3 * 400


@pytest.mark.parametrize("kw,status", [
    (dict(D=96), 2), (dict(D=0), 1), (dict(page_size=8), 2), (dict(page_size=48), 2),
    (dict(page_size=512), 2), (dict(HQ=6, HKV=4), 1), (dict(HQ=65, HKV=1), 2),
    (dict(n_pages=0), 1), (dict(max_pages=0), 1), (dict(n_slots=0), 1), (dict(n_layers=0), 1),
    (dict(max_pages=(1 << 20) + 1), 2), (dict(scale=0.0), 1), (dict(scale=-1.0), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
])
def test_configuration_refusals(lib, kw, status):
    base = dict(n_layers=1, n_slots=2, HQ=8, HKV=2, D=64, n_pages=4, page_size=16, max_pages=4,
                dtype="bf16", scale=1.0)
    base.update(kw)
    with pytest.raises(_lib.RssmError) as e:
        _lib.rssm_kv_required_bytes(_lib.make_kv_config(**base))
    assert e.value.status == status


def test_unknown_dtype_is_refused(lib):
    cfg = _lib.make_kv_config(1, 1, 1, 1, 64, 1, 16, 1, "f32")
    cfg.dtype = 3
    with pytest.raises(_lib.RssmError) as e:
        _lib.rssm_kv_required_bytes(cfg)
    assert e.value.status == 1


@pytest.mark.parametrize("at,value", [(0, 0), (0, 0x1008), (1, 0x2004), (2, 0), (3, 0x4002),
                                      (6, 0x7008), (7, 0)])
def test_alloc_refuses_bad_buffers_before_touching_the_device(lib, at, value):
    cfg = _lib.make_kv_config(1, 1, 1, 1, 64, 1, 16, 1, "f32")
    addr = [0x1000 * (i + 1) for i in range(8)]
    addr[at] = value
    with pytest.raises(_lib.RssmError) as e:
        _lib.rssm_kv_alloc(cfg, _lib.rssm_kv_buffers(*addr))
    assert e.value.status == 1


def test_null_handles_are_refused(lib):
    for call in (lambda: _lib.rssm_kv_reserve(None, None, None, 1, 1, stream=0),
                 lambda: _lib.rssm_kv_commit(None, None, None, None, 1, 1, stream=0),
                 lambda: _lib.rssm_kv_fork(None, None, None, 1, False, stream=0),
                 lambda: _lib.rssm_kv_release(None, None, 1, stream=0),
                 lambda: _lib.rssm_kv_compact(None, stream=0),
                 lambda: _lib.rssm_kv_append(None, 0, None, None, None, 0, 0, 0, None, None,
                                             None, None, 1, 1, 1, None, stream=0),
                 lambda: _lib.rssm_attn_decode(None, 0, None, 0, None, 1, 1, None, None,
                                               stream=0),
                 lambda: _lib.rssm_attn_prefill(None, None, None, None, 0, 0, 0, None, None,
                                                None, 1, 1, 1, None, None, stream=0)):
        with pytest.raises(_lib.RssmError) as e:
            call()
        assert e.value.status == 1


def test_reference_attention_is_the_plain_softmax():
    """The oracle's rows against the written-out formula, and its empty rows."""
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((4, 3)), rng.standard_normal((6, 3)), rng.standard_normal((6, 2))
    o, lse, _ = ref.attend(q, k, v, [0, 1, 4, 6], 0.7)
    assert np.all(o[0] == 0) and np.isneginf(lse[0])
    np.testing.assert_allclose(o[1], v[0])
    w = np.exp(0.7 * q[2] @ k[:4].T)
    np.testing.assert_allclose(o[2], (w / w.sum()) @ v[:4])
    np.testing.assert_allclose(lse[2], np.log(w.sum()))
    k[4:], v[4:] = np.nan, np.inf
    np.testing.assert_array_equal(ref.attend(q, k, v, [0, 1, 4, 4], 0.7)[0][:3], o[:3])


def test_reference_rotation_turns_pairs():
    x = np.random.default_rng(1).standard_normal((5, 2, 8))
    freq = 10.0 ** -np.arange(3)
    pos = np.array([[3.0, 0, 1, 2, 9], [1.0, 0, 5, 7, 2]])
    axis = ref.pair_axes(3, [2, 1], False)
    assert axis.tolist() == [0, 0, 1]
    y = ref.rotate(x, pos, freq, axis)
    for n in range(5):
        for i in range(3):
            a = pos[axis[i], n] * freq[i]
            m = np.array([[np.cos(a), -np.sin(a)], [np.sin(a), np.cos(a)]])
            np.testing.assert_allclose(y[n, :, [i, i + 3]], m @ x[n][:, [i, i + 3]].T, atol=1e-12)
    np.testing.assert_array_equal(y[..., 6:], x[..., 6:])
    assert ref.pair_axes(8, [4, 2, 2], True).tolist() == [0, 1, 2, 0, 1, 2, 0, 0]


def test_reference_pages_by_hand():
    m = ref.Pages(3, 6, 4, 5)
    m.reserve([0, 1], [9, 4])
    assert m.table[:2] == [[0, 1, 2], [3]] and m.refs == [1, 1, 1, 1, 0, 0]
    m.length[0] = 6
    m.fork([0], [2])
    assert m.table[2] == [0, 4] and m.refs == [2, 1, 1, 1, 1, 0] and m.data[4] == 1
    m.release([0])
    assert m.refs == [1, 0, 0, 1, 1, 0]
    m.compact()
    assert m.refs == [1, 1, 1, 0, 0, 0] and m.table == [[], [1], [0, 2]]
    assert m.data[:3] == [0, 3, 1]


def test_index_tensors_off_the_device_are_refused():
    import torch
    from linear_attention_state_rssm_gb300.store import KVCache, RotaryTable
    assert KVCache._index(None, 3) == 0
    with pytest.raises(ValueError):
        KVCache._index(torch.zeros(3, dtype=torch.int32), 3)
    with pytest.raises(ValueError):
        RotaryTable(torch.zeros(4, 2, 32))
