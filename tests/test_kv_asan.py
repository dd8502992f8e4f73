"""The host code of the paged cache's and the attention's entry points under
AddressSanitizer (CPU only): their refusals and size queries run against the
sanitized build, as test_capi_asan.py does for the linears."""
import os
import subprocess
import sys

import pytest

from w4a4_block_scaled_amd import build as B

HERE = os.path.dirname(os.path.abspath(__file__))


def sanitized() -> str:
    """The sanitized library, built unless it is newer than every source."""
    sources = [os.path.join(d, f) for d in (B.CSRC, B.INCLUDE) for f in os.listdir(d)] + [B.__file__]
    if os.path.exists(B.ASAN_LIB) and os.path.getmtime(B.ASAN_LIB) > max(os.path.getmtime(f) for f in sources):
        return B.ASAN_LIB
    return B.build_asan(jobs=8)


def test_kv_validation_under_address_sanitizer():
    try:
        runtime = B.asan_runtime()
    except RuntimeError as e:
        pytest.skip(str(e))
    env = dict(os.environ, LD_PRELOAD=runtime, W4A4_LIBRARY=sanitized(), ASAN_OPTIONS="detect_leaks=0:halt_on_error=1")
    res = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider",
                          *[os.path.join(HERE, f) for f in ("test_kv_refusals.py", "test_kv_limits.py", "test_kv_binding.py")]],
                         env=env, capture_output=True, text=True, timeout=900)
    out = res.stdout[-4000:] + res.stderr[-4000:]
    assert res.returncode == 0, out
    assert "ERROR: AddressSanitizer" not in res.stderr, out
    assert " passed" in res.stdout and "skipped" not in res.stdout
