"""Where the integer product's tiles read (csrc/kd_int8_place.h), on the CPU: what its kernel reads past an array, its
results do not show."""
import os
import subprocess

from chunked_kl_loss_logit_amd import build as B


def test_no_address_of_the_tiles_leaves_its_array():
    r = subprocess.run([B.build_host_sanitizer_driver("int8_place_driver")], capture_output=True, text=True,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"), timeout=300)
    assert r.returncode == 0 and "ok: 0 failure(s)" in r.stdout, (r.stdout + r.stderr)[-4000:]
