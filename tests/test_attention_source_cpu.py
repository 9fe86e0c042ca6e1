"""Orders in the kernels' source that a run cannot be relied on to show."""
import os
import re

import pytest

from transposed_conv_implicit_gb300 import build


def _kernels():
    """(file, name, body) of every kernel."""
    for name in sorted(os.listdir(build.CSRC)):
        if not name.endswith((".cu", ".cuh")):
            continue
        with open(os.path.join(build.CSRC, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        parts = re.split(r"__global__", text)[1:]
        for part in parts:
            head = re.search(r"(\w+_kernel)\s*\(", part)
            if head:
                yield name, head.group(1), part


TMEM = [(f, n, body) for f, n, body in _kernels() if "tmem_alloc(" in body]


def test_the_kernels_that_hold_tensor_memory_are_seen():
    assert {n for _, n, _ in TMEM} >= {"attn_fwd_kernel", "attn_dq_kernel", "attn_dkv_kernel",
                                       "attn_one_kernel", "attn_short_bwd_kernel", "conv_igemm_kernel"}


@pytest.mark.parametrize("kernel", TMEM, ids=lambda k: k[1])
def test_dependents_are_released_once_tensor_memory_is_held(kernel):
    """A block of the next kernel that took the columns first would hold them until this grid ends,
    which waits for them: the release comes after a barrier behind the allocation."""
    body = kernel[2]
    alloc, release = body.index("tmem_alloc("), body.index("grid_launch_dependents()")
    assert "__syncthreads()" in body[alloc:release]


MEET = [("attn_short_bwd_kernel", "barrier_all(1 + quarter, 64, ok)"),
        ("attn_dkv_kernel", "if (kMask) ok = barrier_all(1, 32 * kSoftWarps, ok)"),
        ("attn_dq_kernel", "if (kOne) ok = barrier_all(1 + quarter, 128, ok)")]


@pytest.mark.parametrize("name,barrier", MEET, ids=[m[0] for m in MEET])
def test_warps_that_meet_at_barriers_leave_an_item_together(name, barrier):
    """A wait that runs out in one warp alone must not leave others at a named barrier, which has no
    limit: after the wait that ends an item, and before anything can leave it, they agree."""
    body = next(b for _, n, b in TMEM if n == name)
    wait = "ok = ok && wait(&bars.acc_done, items & 1u, kAttnSoftmaxTimeout);"
    after = body[body.index(wait) + len(wait):]
    assert after.lstrip().startswith(barrier) or after.lstrip().startswith("ok = " + barrier)
    # From the item's last step to that wait nothing leaves the item but what all warps do together.
    loop = body[:body.index(wait)]
    assert not loop.rstrip().endswith("break;")
