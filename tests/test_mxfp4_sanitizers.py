"""The C ABI layer of the MXFP4 operators (csrc/mxfp4_api.cpp) under AddressSanitizer and
UndefinedBehaviorSanitizer, CPU only: counting stand-ins for the device launchers, every
refusal and the largest accepted sizes (tests/sanitize/mxfp4_driver.cpp)."""
import os
import shutil
import tempfile

import pytest

from tests.test_host_sanitizers import ROOT, SAN, _run


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="g++ or the HIP headers not available")
def test_mxfp4_abi_layer_under_asan_ubsan():
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "mxfp4_driver")
        csrc = os.path.join(ROOT, "quantized_unpack_q4_amd", "csrc")
        inc = ["-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"),
               "-I" + csrc]
        _run(["g++", "-std=c++17", *SAN, *inc, "-o", exe,
              os.path.join(ROOT, "tests", "sanitize", "mxfp4_driver.cpp"),
              os.path.join(csrc, "mxfp4_api.cpp"), "-L/opt/rocm/lib", "-lamdhip64",
              "-Wl,-rpath,/opt/rocm/lib"], d)
        assert "all checks passed" in _run([exe], d)
