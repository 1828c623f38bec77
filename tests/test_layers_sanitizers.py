"""kdlayers.h's host code under the address and undefined-behaviour sanitizers
(tests/host/layers_driver.cpp), on the CPU: no case reaches a HIP call."""
import os
import subprocess

import pytest

from chunked_kl_loss_logit_amd import build as B


def test_layers_host_code_is_clean_under_sanitizers():
    try:
        driver = B.build_host_sanitizer_driver("layers_driver")
    except RuntimeError as e:  # pragma: no cover - toolchain problems are reported, not hidden
        pytest.fail(str(e))
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:halt_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([driver], capture_output=True, text=True, env=env, timeout=300)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "ok: 0 failure(s)" in r.stdout
    assert "ERROR: AddressSanitizer" not in out and "runtime error" not in out
