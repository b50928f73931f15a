"""Arguments of KVCache's calls that are refused on the host (no GPU)."""
from types import SimpleNamespace

import pytest
import torch

from linear_attention_state_rssm_gb300 import _lib, build
from linear_attention_state_rssm_gb300.store import KVCache


def tensor_like(shape, dtype, is_cuda=True, contiguous=True):
    """What the checks ask of a tensor, on whichever device it says it is."""
    t = torch.zeros(shape, dtype=dtype)
    return SimpleNamespace(dtype=dtype, shape=t.shape, is_cuda=is_cuda, numel=t.numel,
                           stride=t.stride, is_contiguous=lambda: contiguous)


@pytest.mark.parametrize("kw", [dict(is_cuda=False), dict(dtype=torch.float16),
                                dict(shape=(3, 2)), dict(contiguous=False)])
def test_lse_that_the_kernels_cannot_write_is_refused(kw):
    kv = SimpleNamespace(HQ=2, D=64, _torch_dtype=torch.bfloat16)
    o = tensor_like((4, 2, 64), torch.bfloat16)
    base = dict(shape=(4, 2), dtype=torch.float32)
    KVCache._output(kv, o, 4, tensor_like(**base))
    KVCache._output(kv, o, 4)
    with pytest.raises(ValueError):
        KVCache._output(kv, o, 4, tensor_like(**{**base, **kw}))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_work_buffer_holds_the_largest_parts_and_little_else(D):
    build.build()
    sms, pages = 152, 100
    # CTAs per SM and rows of a block that the decode kernel has at most, 16-bit types
    ctas, rows = {64: (3, 64), 128: (2, 64), 256: (1, 48)}[D]
    parts = 2 * ctas * sms * rows * (D + 2) * 4
    work = _lib.rssm_kv_required_bytes(
        _lib.make_kv_config(1, 1, 1, 1, D, pages, 16, 1, "bf16")).work
    lists = 4 * (456 + 3 * pages + 65536)
    assert parts + lists <= work <= 2 * 2 * sms * 64 * 130 * 4 + lists + 4096
