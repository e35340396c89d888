"""The FP8 product's plans and the storage sizes (csrc/mx/mx_plan.cpp) under AddressSanitizer and
UndefinedBehaviorSanitizer, by a seeded fuzz of 100000 descriptors and of sizes up to the largest; plan.cpp holds the
error messages."""
import os
import shutil

import pytest

from test_sanitize_host import HERE, ROOT, _build_and_run


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_fp8_plan_under_asan_ubsan(tmp_path):
    csrc = os.path.join(ROOT, "gemm_epilogue_persistent_amd", "csrc")
    out = _build_and_run(tmp_path, "g++", [os.path.join(csrc, "mx", "mx_plan.cpp"), os.path.join(csrc, "plan.cpp"),
                                           os.path.join(HERE, "fp8_plan_fuzz.cpp")], ["-std=c++17"], "fp8_plan_fuzz")
    assert "fp8 plans accepted" in out
