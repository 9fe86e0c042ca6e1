"""How much workspace the layer norm's backward pass asks for (validation, without a GPU)."""
import pytest

from tests.test_decoder_abi_cpu import WS, _norm, lib  # noqa: F401  (a fixture)
from transposed_conv_implicit_gb300 import _lib

TOO_SMALL = _lib.CONV_ERR_WORKSPACE_TOO_SMALL


@pytest.mark.parametrize("channels", [1, 64, 16384])
def test_without_weights_the_status_region_does(lib, channels):  # noqa: F811
    row = (64 * channels, channels)
    call = _norm(channels=channels, dweight=0, dbias=0, batch=0, x_stride=row, dy_stride=row, dx_stride=row)
    assert lib.layer_norm_bwd(call, WS, _lib.CONV_STATUS_BYTES - 1, None) == TOO_SMALL
    assert lib.layer_norm_bwd(call, WS, _lib.CONV_STATUS_BYTES, None) != TOO_SMALL
