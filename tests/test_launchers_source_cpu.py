"""What a launcher remembers of its kernel (the shared-memory limit that is set) is of one kernel: two
instances of a launcher for one kernel would each remember a limit of their own, and the second could
lower what the first takes for set."""
import os
import re

import pytest

from transposed_conv_implicit_gb300 import build


def _launchers():
    for name in sorted(os.listdir(build.CSRC)):
        if not name.endswith((".cu", ".cuh")):
            continue
        with open(os.path.join(build.CSRC, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for call in re.finditer(r"raise_smem\(\s*([\w:]+(?:<[^>]*>)?)\s*,", text):
            if text[:call.start()].rstrip().endswith("cudaError_t"):   # its definition
                continue
            heads = list(re.finditer(r"template <([^>]*)>\s*\n\s*(?:cudaError_t|conv_status_t) (\w+)\(", text[:call.start()]))
            kernel = call.group(1)
            body = text[heads[-1].start():call.start()] if heads else ""
            if "<" not in kernel:
                kernel = re.search(r"const auto %s = (\w+<[^;]*>);" % kernel, body).group(1)
            yield name, heads[-1].group(2), heads[-1].group(1), kernel


FOUND = list(_launchers())


def test_the_launchers_are_seen():
    assert {n for _, n, _, _ in FOUND} >= {"launch_dq", "launch_masked", "few_launch", "many_launch", "ln_launch_bwd"}


@pytest.mark.parametrize("launcher", FOUND, ids=lambda f: f[1])
def test_a_launcher_has_its_kernels_parameters(launcher):
    _, _, params, kernel = launcher
    names = [p.split("=")[0].split()[-1] for p in params.split(",")]
    args = set(re.findall(r"\w+", kernel[kernel.index("<"):]))
    assert not [n for n in names if n not in args], (names, kernel)
