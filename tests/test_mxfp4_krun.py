"""How groups of waves share out K in the MXFP4 products with 16-bit activations
(csrc/mxfp4_krun.h), checked on the CPU over every K (tests/sanitize/mxfp4_krun_driver.cpp): a
group without a run once read before its buffers."""
import os
import shutil
import tempfile

import pytest

from tests.test_host_sanitizers import ROOT, SAN, _run


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="g++ or the HIP headers not available")
def test_every_group_of_waves_has_a_run():
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "mxfp4_krun_driver")
        _run(["g++", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
              "-I" + os.path.join(ROOT, "quantized_unpack_q4_amd", "csrc"), "-o", exe,
              os.path.join(ROOT, "tests", "sanitize", "mxfp4_krun_driver.cpp")], d)
        assert "all checks passed" in _run([exe], d)
