"""Arguments of KVCache's calls that are refused on the host (no GPU)."""
from types import SimpleNamespace

import pytest
import torch

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
