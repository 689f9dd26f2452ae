"""What the host decides for a batch of attention from its sizes alone, on the CPU:
tests/sanitize/attend_sizes_check.cpp."""
import os
import subprocess

import pytest

from test_sanitizers import BUILD, HIPCC, ROOT, SAN, SAN_ENV, _build


def test_sizes_of_batches():
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    csrc = os.path.join(ROOT, "lora_adapter_application_amd", "csrc")
    src = os.path.join(SAN, "attend_sizes_check.cpp")
    out = os.path.join(BUILD, "attend_sizes_check")
    cmd = [HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17",
           "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
           "-I", os.path.join(ROOT, "include"), src, "-o", out]
    _build(out, cmd, [src, os.path.join(ROOT, "include", "lora_mi355x.h")] +
           [os.path.join(csrc, h) for h in ("lora_internal.h", "lora_layer.h", "lora_attend.h")])
    res = subprocess.run([out], capture_output=True, text=True, timeout=300,
                         env=dict(SAN_ENV, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1"))
    print(res.stdout)
    assert res.returncode == 0, res.stdout + res.stderr
    assert "failures: 0" in res.stdout
    assert "runtime error" not in res.stderr
