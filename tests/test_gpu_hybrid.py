"""A hybrid stack end to end (examples/hybrid_step.py): the same tokens as one
prompt, and as prompt, draft windows with rejections, a fork and single tokens
in a CUDA graph.

Tolerances on the hidden states, relative to the largest: fp32 layers each add
about 1e-6 (chunked and replayed forms of the recurrence sum in other orders),
amplified by at most the norms' and projections' factor of a few per layer: 1e-4
over four layers. bf16 hidden states are rounded eight times on the way
(2^-8 each, of values up to the largest), and intermediate q, k, v once each:
0.06."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "hybrid_step.py")


@pytest.mark.parametrize("dtype,tol", [("f32", 1e-4), ("bf16", 0.06)])
def test_tokens_give_the_same_states_whichever_way_they_come(dtype, tol):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_attention_state_rssm_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("hybrid_step", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    assert mod.run(dtype) <= tol
