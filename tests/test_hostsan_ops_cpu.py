"""The training-step operators' CPU tests against the library whose host code is under
AddressSanitizer and UndefinedBehaviorSanitizer, as test_hostsan_cpu.py runs the others."""
import os
import subprocess
import sys

import pytest

from matrix_orthogonalising_optimizer_02_amd import build as BUILD
from test_hostsan_cpu import CHILD, ROOT, sanitized_lib  # noqa: F401


def test_operator_cpu_tests_under_host_sanitizers(sanitized_lib):  # noqa: F811
    try:
        runtime = BUILD.sanitizer_runtime()
    except RuntimeError as e:
        pytest.skip(str(e))
    env = dict(os.environ, MUON_ROCM_LIBRARY=sanitized_lib, LD_PRELOAD=runtime,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    child = CHILD.format(root=ROOT, lib=sanitized_lib).replace('"tests/test_abi_cpu.py", "tests/test_plan_cpu.py"',
                                                               '"tests/test_norm_cpu.py", "tests/test_multi_cpu.py"')
    res = subprocess.run([sys.executable, "-c", child], cwd=ROOT, env=env, stdout=subprocess.PIPE,
                         stderr=subprocess.STDOUT, text=True, timeout=600)
    out = res.stdout
    assert res.returncode == 0, out[-4000:]
    assert "AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
    assert " passed" in out and "test_norm_cpu" in child, out[-2000:]
