"""The decoder operators' workspaces: no more than a call needs, and no more cleared than has to be."""
import pytest
import torch

import transposed_conv_implicit_gb300 as cg
from tests.test_gpu_layer_norm import DEV, _gen, _rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("c", [8, 321, 4096, 9001])
def test_gradients_of_the_rows_alone(c):
    """Without dweight and dbias a status region is workspace enough; with either it is refused."""
    x, dy = _rows(_gen(c), 300, c, torch.bfloat16), _rows(_gen(c + 1), 300, c, torch.bfloat16)
    y, dx, dx2 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(300, device=DEV), torch.empty(300, device=DEV)
    dw = torch.empty(c, device=DEV)
    cg.layer_norm_fwd(x, None, None, y, mean=mean, rstd=rstd)
    cg.layer_norm_bwd(dy, x, None, mean, rstd, dx, dw, None)
    ws = torch.zeros(cg.CONV_STATUS_BYTES + 256, dtype=torch.uint8, device=DEV)
    ws[cg.CONV_STATUS_BYTES:] = 0x5A
    cg.layer_norm_bwd(dy, x, None, mean, rstd, dx2, None, None, workspace=ws[:cg.CONV_STATUS_BYTES])
    assert torch.equal(dx, dx2) and (ws[cg.CONV_STATUS_BYTES:] == 0x5A).all()
    for weights in ((dw, None), (None, dw)):
        with pytest.raises(cg.ConvError) as e:
            cg.layer_norm_bwd(dy, x, None, mean, rstd, dx2, *weights, workspace=ws[:cg.CONV_STATUS_BYTES])
        assert e.value.status == cg.CONV_ERR_WORKSPACE_TOO_SMALL
