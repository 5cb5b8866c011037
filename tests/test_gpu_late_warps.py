"""Waits of the differential attention kernels when one warp is far behind the others.

The debug build of the library can make one warp of every block late to each of its waits.  Whatever a block's other
warps, copies and products have done meanwhile, the late warp must find what it waits for, and every result must have
the bits that it has without the delay.  The cases have more items than a device has SMs, so that a block goes from one
item to the next, whose copies run ahead.
"""
import os
import re
import subprocess
import sys

import numpy as np
import pytest
import torch

import ulysses_dit_attention_gb300 as uaa
from helpers import bits

HERE = os.path.dirname(os.path.abspath(__file__))
DEV = "cuda"


def test_other_builds_have_no_late_warps():
    if not uaa.debug_build():
        with pytest.raises(uaa.UAAError, match="debug build"):
            uaa.debug_late_warp(3, 1000)
    with pytest.raises(uaa.UAAError, match="ns"):
        uaa.debug_late_warp(-1, 1000001)
    uaa.debug_late_warp()


@pytest.mark.gpu
@pytest.mark.parametrize("B,Sq,Sk,D,masked", [(4, 260, 300, 128, False), (4, 260, 700, 64, False), (4, 260, 700, 128, True),
                                              (4, 300, 100, 64, False)])
def test_a_late_warp_changes_nothing(B, Sq, Sk, D, masked):
    if not uaa.debug_build():
        pytest.skip("runs in the child process that loads the debug build")
    H = 24
    g = torch.Generator(DEV).manual_seed(60)
    q, do = (torch.randn(B, Sq, H, D, generator=g, device=DEV).bfloat16() for _ in range(2))
    k, v = (torch.randn(B, Sk, H, D, generator=g, device=DEV).bfloat16() for _ in range(2))
    lam = torch.rand(H, generator=g, device=DEV)
    mask = torch.arange(Sk, device=DEV) < torch.tensor([Sk, 1, Sk // 2, 0], device=DEV)[:, None] if masked else None

    def step():
        out, out2, lse = uaa.diff_attn_fwd(q, k, v, lam, mask)
        return (out, out2, lse) + uaa.diff_attn_bwd(q, k, v, lam, out, out2, do, lse, mask)

    want = step()
    uaa.check_device_status()
    for warp in range(18):
        uaa.debug_late_warp(warp, 20000)
        try:
            got = step()
        finally:
            uaa.debug_late_warp()
        uaa.check_device_status()
        for name, a, w in zip(("out", "out2", "lse", "dq", "dk", "dv", "dlam"), got, want):
            assert np.array_equal(bits(a), bits(w)), (warp, name)


@pytest.mark.gpu
def test_late_warps_under_the_debug_build():
    if uaa.debug_build():
        pytest.skip("this is the child process")
    from ulysses_dit_attention_gb300 import build

    build.build(debug=True)
    cmd = [sys.executable, "-m", "pytest", "-x", "-q", "-p", "no:cacheprovider", "-m", "gpu", "-k", "changes_nothing",
           "tests/test_gpu_late_warps.py"]
    r = subprocess.run(cmd, cwd=os.path.dirname(HERE), env=dict(os.environ, UAA_DEBUG="1"), capture_output=True, text=True,
                       timeout=900)
    tail = "\n".join((r.stdout + r.stderr).strip().splitlines()[-30:])
    assert r.returncode == 0, tail
    m = re.search(r"(\d+) passed", tail)
    assert m and int(m.group(1)) == 4 and " skipped" not in tail, tail
