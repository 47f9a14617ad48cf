"""The host code of the rotation, the attention of several new tokens and the
verification of drafted tokens under AddressSanitizer and UndefinedBehaviorSanitizer,
on the CPU: tests/test_tokens_abi_cpu.py run against the sanitized build of the
library."""

import os
import subprocess
import sys

import pytest

from gguf_block_quant_dequant_amd import build
from tests.test_host_sanitizers import ROOT, _asan_runtime


@pytest.mark.skipif(not os.path.exists(build.HIPCC) or _asan_runtime() is None,
                    reason="hipcc or the clang sanitizer runtime is not installed")
def test_token_validation_clean_under_asan_and_ubsan():
    lib = build.build_library(sanitize=True)
    env = dict(os.environ)
    env.update({"LD_PRELOAD": _asan_runtime(), "GGUF_QK_LIBRARY": lib,
                "ASAN_OPTIONS": "detect_leaks=0:halt_on_error=1:abort_on_error=0",
                "UBSAN_OPTIONS": "print_stacktrace=1:halt_on_error=1"})
    res = subprocess.run([sys.executable, "-m", "pytest", "tests/test_tokens_abi_cpu.py", "-q", "-m", "not gpu",
                          "-p", "no:cacheprovider"],
                         cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = res.stdout + res.stderr
    assert "AddressSanitizer" not in out and "runtime error:" not in out, out[-4000:]
    assert res.returncode == 0, out[-4000:]
    assert " passed" in out and " skipped" not in out, out[-2000:]
