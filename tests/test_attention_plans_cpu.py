"""How the attention entry points share a call's work and their workspaces, without a GPU."""
import ctypes

import pytest

from tests.test_attention_abi_cpu import _attn, _norm
from transposed_conv_implicit_gb300 import _lib, build

SMS = 152


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.lib()


def _blocks(lib, backward, batch, q, k, d, rot):
    """(blocks of q, of k, rows of partial sums in the workspace); q and k are (length, heads)."""
    out = (ctypes.c_int * 3)()
    args = _norm(backward, batch=batch, head_dim=d, rot_dim=rot, table_rows=5000,
                 q_length=q[0], q_heads=q[1], k_length=k[0], k_heads=k[1])
    assert lib.conv_testing_qk_norm_rope_blocks(args, int(backward), SMS, out) == 0
    return tuple(out)


FULL = [  # batch, q, k, head_dim: the rows of both tensors just fill the SMs, or nearly
    (1, (607, 16), (609, 16), 128),
    (1, (1215, 16), (1, 16), 128),
    (2, (1139, 8), (77, 8), 128),
    (1, (1, 16), (1215, 16), 128),
]


@pytest.mark.parametrize("case", FULL, ids=str)
def test_partial_sums_of_the_norm_fit_their_workspace(lib, case):
    batch, q, k, d = case
    a, b, rows = _blocks(lib, True, batch, q, k, d, d)
    assert rows == 4 * SMS and a > 0 and b > 0 and a + b <= rows


@pytest.mark.parametrize("backward", [False, True])
def test_the_grid_of_the_norm_fills_the_gpu_at_most_once(lib, backward):
    """Every split of the tokens around the size where a warp for each unit no longer fits."""
    for total in range(1200, 1232):
        for lq in (0, 1, 2, 3, 77, 300, 607, 608, 609, 1000, total - 3, total - 2, total - 1, total):
            lk = total - lq
            scale = 1 if backward else 2      # (a unit holds twice the rows in the forward pass)
            a, b, rows = _blocks(lib, backward, 1, (scale * lq, 16), (scale * lk, 16), 128, 128)
            assert a + b <= rows, (lq, lk)
            assert (a > 0) == (lq > 0) and (b > 0) == (lk > 0), (lq, lk)


def test_small_calls_of_the_norm_get_a_warp_for_each_unit(lib):
    # 8 tokens x 32 heads x 128: 16 lanes hold 8 elements twice, so a warp takes 4 rows.
    a, b, _ = _blocks(lib, False, 8, (1, 32), (1, 8), 128, 128)
    rows = 4 * 4
    assert a == -(-(-(-8 * 32 // rows)) // 4) and b == -(-(-(-8 * 8 // rows)) // 4)


@pytest.mark.parametrize("kv_len", [1, 16, 40, 64, 77, 80, 96, 100, 112, 128])
@pytest.mark.parametrize("head_dim", [8, 16, 24, 32, 40, 48, 64])
def test_one_tile_of_keys_runs_in_one_round(lib, head_dim, kv_len):
    """Persistent thread blocks with equal shares of the row tiles: no more than an SM holds at once
    (228 KB of shared memory, 1 KB of it taken for each block; 512 columns of tensor memory)."""
    out = (ctypes.c_int * 3)()
    args = _attn(batch=16, heads=8, kv_heads=8, q_len=4096, kv_len=kv_len, head_dim=head_dim, mask=0)
    assert lib.conv_testing_cross_attention_plan(args, SMS, out) == 0
    schedule, grid, smem = out
    columns = 128 if -(-kv_len // 16) * 16 + -(-head_dim // 16) * 16 <= 128 else 256
    assert schedule == 2 and grid % SMS == 0
    assert grid == SMS * min(512 // columns, 228 * 1024 // (smem + 1024))


def test_few_rows_take_a_block_each(lib):
    out = (ctypes.c_int * 3)()
    args = _attn(batch=2, heads=3, kv_heads=3, q_len=200, kv_len=77, head_dim=64, mask=0)
    assert lib.conv_testing_cross_attention_plan(args, SMS, out) == 0
    assert list(out)[:2] == [2, 2 * 3 * 2]
