"""Arguments that no field of the C structs can hold, and heads without elements."""
import pytest
import torch

import transposed_conv_implicit_gb300 as cg
from tests.test_gpu_attention import DEV

pytestmark = pytest.mark.gpu


def _zeros(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16, device=DEV)


@pytest.mark.parametrize("scale", [1e39, -1e200, "one"])
def test_scales_past_fp32(scale):
    q, k = _zeros(1, 3, 2, 64), _zeros(1, 5, 2, 64)
    with pytest.raises(cg.ConvError) as e:
        cg.cross_attention_fwd(q, k, k, torch.empty_like(q), scale=scale)
    assert e.value.status == cg.CONV_ERR_INVALID_VALUE


def test_eps_past_fp32():
    q, w = _zeros(1, 3, 2, 64), _zeros(64)
    with pytest.raises(cg.ConvError) as e:
        cg.qk_norm_rope_fwd(q, None, w, None, torch.empty_like(q), None, eps=1e39)
    assert e.value.status == cg.CONV_ERR_INVALID_VALUE


def test_heads_without_elements():
    q, k = _zeros(1, 3, 2, 0), _zeros(1, 5, 2, 0)
    with pytest.raises(cg.ConvError) as e:
        cg.cross_attention_fwd(q, k, k, torch.empty_like(q))
    assert e.value.status == cg.CONV_ERR_INVALID_VALUE
