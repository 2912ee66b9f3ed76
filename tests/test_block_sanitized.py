"""The argument checks of the operators around the projections under
AddressSanitizer and UndefinedBehaviorSanitizer: the host code of the library
built with both, and tests/test_block_abi.py run against it in a child Python
process with the sanitizer runtime preloaded."""

import os
import subprocess
import sys

import pytest

from tests.test_sanitized_abi import ROOT, _runtime


def test_block_checks_clean_under_asan_ubsan(tmp_path):
    from int4_quantized_gemm_amd import build_lib
    asan = _runtime("libasan.so")
    if asan is None:
        pytest.skip("g++ with AddressSanitizer is not available")
    try:
        lib = build_lib.build_sanitized_api(str(tmp_path))
    except FileNotFoundError as e:
        pytest.skip(str(e))
    code = (
        f"import sys; sys.path.insert(0, {ROOT!r})\n"
        "import int4_quantized_gemm_amd._lib as L\n"
        f"L.LIB_PATH = {lib!r}\n"
        "import pytest\n"
        f"sys.exit(pytest.main([{os.path.join(ROOT, 'tests', 'test_block_abi.py')!r}, '-q', '-x', '-p', "
        "'no:cacheprovider']))\n"
    )
    env = dict(os.environ, LD_PRELOAD=asan, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, env=env, cwd=ROOT, timeout=600)
    out = r.stdout + r.stderr
    assert "ERROR: AddressSanitizer" not in out and "runtime error:" not in out, out[-4000:]
    assert r.returncode == 0, out[-4000:]
    assert " passed" in out
