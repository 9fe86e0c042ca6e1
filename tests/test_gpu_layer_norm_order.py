"""Layer norm of rows of several lengths, in orders that a process may meet them in."""
import subprocess
import sys

import pytest

from tests.conftest import ROOT

pytestmark = pytest.mark.gpu

PROGRAM = """
import sys
import torch
import transposed_conv_implicit_gb300 as cg
for c in map(int, sys.argv[1:]):
    x = torch.randn((3, c), device="cuda").bfloat16()
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
    dw, db = torch.empty(c, device="cuda"), torch.empty(c, device="cuda")
    cg.layer_norm_fwd(x, None, None, y, mean=mean, rstd=rstd)
    cg.layer_norm_bwd(x, x, None, mean, rstd, dx, dw, db)
    want = torch.nn.functional.layer_norm(x.double(), (c,))
    assert (y.double() - want).abs().max() < 0.03, c
print("fine")
"""


@pytest.mark.parametrize("lengths", [(16384, 4096, 10240), (4096, 16384, 8192, 12288), (8185, 2001, 4099, 8001)], ids=str)
def test_a_process_that_starts_with(lengths):
    run = subprocess.run([sys.executable, "-c", PROGRAM] + [str(c) for c in lengths], cwd=ROOT, capture_output=True,
                         text=True, timeout=300)
    assert run.returncode == 0 and run.stdout.strip() == "fine", run.stdout + run.stderr
