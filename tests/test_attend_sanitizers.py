"""The host side of the cache and attention under AddressSanitizer and
UndefinedBehaviorSanitizer, on the CPU: tests/sanitize/attend_check.cpp over the plans of many
batches, proper and out of order, the cache's order, and the refusals that need no device."""
import os
import subprocess

import pytest

from test_sanitizers import BUILD, HIPCC, ROOT, SAN, SAN_ENV, _build


def test_attend_host_under_asan_ubsan():
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    csrc = os.path.join(ROOT, "lora_adapter_application_amd", "csrc")
    srcs = [os.path.join(csrc, "lora_runtime.cpp"), os.path.join(csrc, "lora_attend.cpp"),
            os.path.join(SAN, "attend_check.cpp")]
    out = os.path.join(BUILD, "attend_check")
    cmd = [HIPCC, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17",
           "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
           "-I", os.path.join(ROOT, "include"), *srcs, "-o", out]
    _build(out, cmd, srcs + [os.path.join(ROOT, "include", "lora_mi355x.h")] +
           [os.path.join(csrc, h) for h in ("lora_internal.h", "lora_layer.h", "lora_ctx.h", "lora_attend.h")])
    # the HIP runtime keeps allocations to process exit: no leak report
    res = subprocess.run([out], capture_output=True, text=True, timeout=300,
                         env=dict(SAN_ENV, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1"))
    print(res.stdout)
    assert res.returncode == 0, res.stdout + res.stderr
    assert "failures: 0" in res.stdout
    assert "runtime error" not in res.stderr
