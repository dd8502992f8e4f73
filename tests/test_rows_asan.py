"""The host code of rotary positions, rows and the 4-bit cache under
AddressSanitizer (CPU only), as test_kv_asan.py does for the cache."""
import os
import subprocess
import sys

import pytest

from test_kv_asan import B, HERE, sanitized


def test_rows_validation_under_address_sanitizer():
    try:
        runtime = B.asan_runtime()
    except RuntimeError as e:
        pytest.skip(str(e))
    env = dict(os.environ, LD_PRELOAD=runtime, W4A4_LIBRARY=sanitized(), ASAN_OPTIONS="detect_leaks=0:halt_on_error=1")
    res = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider",
                          os.path.join(HERE, "test_rows_refusals.py")], env=env, capture_output=True, text=True, timeout=900)
    out = res.stdout[-4000:] + res.stderr[-4000:]
    assert res.returncode == 0, out
    assert "ERROR: AddressSanitizer" not in res.stderr, out
    assert " passed" in res.stdout and "skipped" not in res.stdout
