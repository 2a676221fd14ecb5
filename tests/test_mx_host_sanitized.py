"""The host half of the MXFP4 operators and of the expert routing (argument
checks, the packer, the jobs that sequences record) under AddressSanitizer and
UndefinedBehaviorSanitizer: rebuilt with g++ beside the rest of the host
library, kernel launches replaced by stubs, and test_mx_abi.py run against it
in a child process."""
import os
import shutil
import subprocess
import sys

import pytest

from block_scaled_fp4_04_amd import build as nvbuild
from test_host_sanitized import HERE, ROCM, ROOT, STUBS, _runtime

MX_STUBS = r"""
#include "nvfp4_mx_internal.h"
namespace nvfp4 {
hipError_t launch_mx_quantize(const MxQuantArgs&, hipStream_t) { return hipErrorInvalidValue; }
hipError_t launch_mx_dequantize(const MxQuantArgs&, hipStream_t) { return hipErrorInvalidValue; }
hipError_t launch_mx_gemm(const MxGemmArgs&, hipStream_t) { return hipErrorInvalidValue; }
bool mx_gemm_fits(const MxGemmArgs&) { return true; }
hipError_t launch_moe_sort(const MoeArgs&, hipStream_t) { return hipErrorInvalidValue; }
hipError_t launch_moe_gather(const MoeArgs&, hipStream_t) { return hipErrorInvalidValue; }
hipError_t launch_moe_combine(const MoeArgs&, hipStream_t) { return hipErrorInvalidValue; }
hipError_t launch_moe_combine_grad(const MoeArgs&, hipStream_t) { return hipErrorInvalidValue; }
}
"""

CHILD = r"""
import sys
sys.path.insert(0, {root!r}); sys.path.insert(0, {here!r})
import block_scaled_fp4_04_amd as nv
nv.LIB_PATH = {lib!r}
import pytest
sys.exit(pytest.main(["-q", "-p", "no:cacheprovider", "-m", "not gpu", {abi!r}]))
"""


@pytest.mark.skipif(shutil.which("g++") is None or shutil.which("gcc") is None, reason="needs gcc and g++")
def test_host_library_under_sanitizers(tmp_path):
    asan, ubsan = _runtime("libasan.so"), _runtime("libubsan.so")
    if not asan or not ubsan or not os.path.exists(os.path.join(ROCM, "lib", "libamdhip64.so")):
        pytest.skip("sanitizer runtimes or the HIP runtime not installed")
    stubs = tmp_path / "device_stubs.cpp"
    stubs.write_text(STUBS + MX_STUBS)
    lib = str(tmp_path / "libnvfp4_mx_host_sanitized.so")
    host = [s for s in nvbuild.SOURCES if s.endswith(".cpp")]
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fPIC", "-shared", "-fsanitize=address,undefined",
                        "-fno-sanitize-recover=undefined", "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__",
                        f"-DNVFP4_BUILD_ID=\"{nvbuild.build_id()}\"", "-I", os.path.join(ROCM, "include"),
                        "-I", nvbuild.INCLUDE, "-I", nvbuild.CSRC, *host, str(stubs), "-o", lib,
                        "-L", os.path.join(ROCM, "lib"), "-lamdhip64"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, LD_PRELOAD=f"{asan} {ubsan}", ASAN_OPTIONS="detect_leaks=0:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    child = CHILD.format(root=ROOT, here=HERE, lib=lib, abi=os.path.join(HERE, "test_mx_abi.py"))
    r = subprocess.run([sys.executable, "-c", child], capture_output=True, text=True, env=env, timeout=600, cwd=ROOT)
    tail = (r.stdout + r.stderr)[-3000:]
    assert r.returncode == 0, tail
    assert " passed" in r.stdout and "failed" not in r.stdout, tail
