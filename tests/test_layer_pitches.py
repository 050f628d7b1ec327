"""Pitches that pass 64 bits in bytes, at the decoder-layer entry points, under
AddressSanitizer and UndefinedBehaviorSanitizer (host code with recording stubs for the
launchers, built with g++; CPU only)."""
import os
import shutil

import pytest

from test_sanitizers import HERE, ROOT, SAN, _run


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="g++ or the HIP headers not available")
def test_pitches_past_64_bits_are_refused(tmp_path):
    exe = str(tmp_path / "layer_pitch")
    csrc = os.path.join(ROOT, "microscaling_block_scaled_amd", "csrc")
    _run(["g++", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"),
          "-I" + csrc, os.path.join(HERE, "helpers", "layer_pitch_main.cpp"), os.path.join(csrc, "mx_layer_api.cpp"),
          "-o", exe])
    r = _run([exe], env=dict(os.environ, ASAN_OPTIONS="detect_leaks=1"))
    assert "all checks passed" in r.stdout
