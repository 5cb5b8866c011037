"""Rotary positions, 8-bit checkpoints and differential attention under the debug build of the library, whose kernels
check every tensor-core operand and every output store before they make it: the operators' GPU tests once more, in a
child process that loads it."""
import os
import re
import subprocess
import sys

import pytest

import ulysses_dit_attention_gb300 as uaa

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SELECTION = ["tests/test_gpu_debug_build.py::test_loaded_library_is_the_debug_build", "tests/test_rotary.py",
             "tests/test_act8.py", "tests/test_diff_attention.py", "tests/test_diff_attention_not_finite.py",
             "tests/test_operator_guard_bands.py"]


def test_the_operators_pass_the_debug_build_checks():
    if uaa.debug_build():
        pytest.skip("this is the child process")
    from ulysses_dit_attention_gb300 import build

    build.build(debug=True)
    cmd = [sys.executable, "-m", "pytest", "-x", "-q", "-p", "no:cacheprovider", "-m", "gpu", *SELECTION]
    r = subprocess.run(cmd, cwd=ROOT, env=dict(os.environ, UAA_DEBUG="1"), capture_output=True, text=True, timeout=1800)
    tail = "\n".join((r.stdout + r.stderr).strip().splitlines()[-30:])
    assert r.returncode == 0, tail
    m = re.search(r"(\d+) passed", tail)
    assert m and int(m.group(1)) >= 250 and " skipped" not in tail, tail
