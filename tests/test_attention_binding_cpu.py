"""Numbers that the C structs cannot hold are refused as any other argument is."""
import pytest

import transposed_conv_implicit_gb300 as cg
from transposed_conv_implicit_gb300 import attention, build


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.mark.parametrize("sizes", [(1 << 31, 1, 1, 1, 1, 64), (1, 1, 1, 1 << 40, 1, 64), (1, 1, 1, 1, 1, -(1 << 31) - 1)])
def test_sizes_past_31_bits(sizes):
    with pytest.raises(cg.ConvError) as e:
        cg.cross_attention_workspace_size(*sizes)
    assert e.value.status == cg.CONV_ERR_INVALID_VALUE


def test_a_factor_that_is_no_number():
    with pytest.raises(cg.ConvError) as e:
        attention._pack(attention._NORM_HEAD, 0, 1, 64, 0, 0, 0, "small", 0, 0)
    assert e.value.status == cg.CONV_ERR_INVALID_VALUE
