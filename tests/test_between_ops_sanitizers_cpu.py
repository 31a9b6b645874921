"""The host code of the operators between blocks (descriptor checks, workspace layout) under
AddressSanitizer and UndefinedBehaviorSanitizer, as test_sanitizers_cpu does for the rest."""
import os
import subprocess
import sys

import pytest

from fno_spectral_convolution_amd import build as B
from tests.test_sanitizers_cpu import ROOT, _sanitized_library


def test_between_ops_host_code_clean_under_sanitizers():
    import torch
    if torch.cuda.device_count() > 0:
        pytest.skip("CPU-only check")
    env = dict(os.environ)
    env.update({
        "FNO_LIBRARY": _sanitized_library(),
        "LD_PRELOAD": B.sanitizer_runtime(),
        "ASAN_OPTIONS": "detect_leaks=0:halt_on_error=1:abort_on_error=0",
        "UBSAN_OPTIONS": "halt_on_error=1:print_stacktrace=1",
    })
    res = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-p", "no:cacheprovider",
                          "tests/test_between_ops_cpu.py"], cwd=ROOT, env=env,
                         capture_output=True, text=True, timeout=900)
    out = res.stdout + res.stderr
    assert res.returncode == 0, out[-3000:]
    assert "Sanitizer" not in out and "runtime error" not in out, out[-3000:]
    assert " passed" in out
