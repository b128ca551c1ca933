"""The host-side argument checks of the calls on a 4-bit cache from plain C under AddressSanitizer and
UndefinedBehaviorSanitizer (tests/c_abi/fp4_validate.c): every status as documented, no launch
behind a refused or empty call, and neither sanitizer reports. Host code only; no GPU is needed."""
import importlib.util
import os
import subprocess

import pytest

HERE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "c_abi")


def test_fp4_validation_under_sanitizers():
    script = os.path.join(HERE, "build_fp4.py")
    if not os.path.exists("/opt/rocm/llvm/bin/clang") or not os.path.exists(script):
        pytest.skip("the ROCm compiler or the sanitizer build script is not available")
    spec = importlib.util.spec_from_file_location("kvx_build_fp4", script)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([mod.build()], capture_output=True, text=True, timeout=120, env=env)
    assert r.returncode == 0, r.stdout + r.stderr
    assert ", 0 mismatches" in r.stdout, r.stdout
    assert "runtime error" not in r.stderr and "Sanitizer" not in r.stderr, r.stderr
