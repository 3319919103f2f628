"""What no run can show without a wait that gives up: a kernel of the gated linear recurrence whose
waits ran out still waits for its own copies, and for the maps that other CTAs send it,
before it ends."""
import os
import re

import selective_state_space_fwd_gb300 as S


def test_every_kernel_waits_for_what_is_on_its_way():
    path = os.path.join(os.path.dirname(S.__file__), "csrc", "kernel_recur_tma.cu")
    with open(path) as f:
        kernels = re.split(r"(?=__global__ )", f.read())[1:]
    assert len(kernels) == 2
    for kernel in kernels:
        assert "cluster.send(" in kernel and "ring.load(" in kernel
        failed = re.search(r"  if \(bad\) \{\n(.*?)\n  \}\n", kernel, re.S).group(1)
        assert "ring.drain(" in failed and "cluster.drain(" in failed
