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


def _left(size, call):
    """Bytes of a default workspace of this size, as the call leaves them where they were 0x5A: the
    allocator hands out the block that was freed last."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = torch.full((size,), 0x5A, dtype=torch.uint8, device=DEV)
    at = old.data_ptr()
    del old
    call()
    again = torch.empty(size, dtype=torch.uint8, device=DEV)
    assert again.data_ptr() == at
    return again


def test_a_default_workspace_is_not_cleared_as_a_whole():
    c = 16384
    x = torch.randn((1, c), device=DEV).bfloat16()
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd, dw = torch.empty(1, device=DEV), torch.empty(1, device=DEV), torch.empty(c, device=DEV)
    cg.layer_norm_fwd(x, None, None, y, mean=mean, rstd=rstd)
    size = cg.layer_norm_workspace_size(c)
    left = _left(size, lambda: cg.layer_norm_bwd(x, x, None, mean, rstd, dx, dw, None))
    assert not left[:cg.CONV_STATUS_BYTES].any() and (left[size // 2:] == 0x5A).all()

    cache = torch.zeros((2, 64, 1, 64), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    scales = torch.full((2, 1, 64, 2), 127, dtype=torch.uint8, device=DEV)
    table = torch.tensor([[0, 1, 1, 1]], dtype=torch.int32, device=DEV)
    n = torch.tensor([100], dtype=torch.int32, device=DEV)
    for t in (1, 100):
        q = torch.randn((1, t, 1, 64), device=DEV).bfloat16()
        out = torch.empty_like(q)
        size = cg.tree_attention_workspace_size(1, 1, 1, t, 256, 64)
        left = _left(size, lambda: cg.tree_attention_fwd(q, cache, cache, scales, table, n, out))
        assert not left[:cg.CONV_STATUS_BYTES].any() and (left[cg.CONV_STATUS_BYTES:] == 0x5A).any()
        assert not out.any()
