"""Recording a call when memory runs out: the host library built with g++, kernel
launches replaced by stubs, in a program whose operator new fails when told to."""
import os
import shutil
import subprocess

import pytest

from block_scaled_fp4_04_amd import build as nvbuild
from test_host_sanitized import ROCM, STUBS
from test_layer_host_sanitized import LAYER_STUBS
from test_mx_host_sanitized import MX_STUBS

MAIN = r"""
#include <cstdio>
#include <cstdlib>
#include <new>
#include "nvfp4.h"
#include "nvfp4_layer.h"
static int countdown = -1;  // allocations until one fails
void* operator new(size_t n) {
    if (countdown == 0) throw std::bad_alloc();
    if (countdown > 0) --countdown;
    if (void* p = std::malloc(n)) return p;
    throw std::bad_alloc();
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, size_t) noexcept { std::free(p); }
#define CHECK(x) do { if (!(x)) { std::printf("%s:%d: %s\n", __FILE__, __LINE__, #x); return 1; } } while (0)

int main() {
    void* const P = reinterpret_cast<void*>(0x100000);
    nvfp4_mx_experts l{};
    l.experts = 8;
    l.hidden = 64;
    l.inner = 96;
    l.up_packed = l.up_scales = l.down_packed = l.down_scales = P;
    auto moe = [&](nvfp4_sequence_t s, int64_t tokens) {
        return nvfp4_sequence_add_mx_moe(s, &l, P, NVFP4_TYPE_BF16, 64, P, NVFP4_INDEX_I32, nullptr, tokens, 2, P,
                                         NVFP4_TYPE_BF16, P, (size_t)1 << 40);
    };
    int failed = 0;
    for (int n = 0; n < 8; ++n) {
        nvfp4_sequence_t s = nullptr;
        CHECK(nvfp4_sequence_create(&s) == NVFP4_OK);
        countdown = n;
        const int st = moe(s, 500);
        countdown = -1;
        CHECK(st == NVFP4_OK || st == NVFP4_ERR_ALLOC);
        if (st != NVFP4_OK) {
            ++failed;
            CHECK(nvfp4_sequence_finalize(s) == NVFP4_ERR_INVALID_VALUE);  // (nothing is recorded)
        }
        CHECK(nvfp4_sequence_destroy(s) == NVFP4_OK);
    }
    CHECK(failed > 0);
    CHECK(moe(nullptr, 500) == NVFP4_ERR_INVALID_VALUE);
    std::printf("ok\n");
    return 0;
}
"""


def build_and_run(tmp_path, main):
    if shutil.which("g++") is None or not os.path.exists(os.path.join(ROCM, "lib", "libamdhip64.so")):
        pytest.skip("needs g++ and the HIP runtime")
    source, exe = tmp_path / "main.cpp", str(tmp_path / "main")
    source.write_text(STUBS + MX_STUBS + LAYER_STUBS + main)
    host = [s for s in nvbuild.SOURCES + nvbuild.LAYER_SOURCES if s.endswith(".cpp")]
    lib = os.path.join(ROCM, "lib")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-D__HIP_PLATFORM_AMD__", "-DNVFP4_BUILD_ID=\"test\"",
                        "-I", os.path.join(ROCM, "include"), "-I", nvbuild.INCLUDE, "-I", nvbuild.CSRC, *host, str(source),
                        "-o", exe, "-L", lib, f"-Wl,-rpath,{lib}", "-lamdhip64"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "ok" in r.stdout, r.stdout + r.stderr


def test_a_layer_of_experts_is_recorded_whole_or_not_at_all(tmp_path):
    build_and_run(tmp_path, MAIN)


def test_recording_without_memory_is_an_error(tmp_path):
    """Every call that records reports it: no exception leaves the library."""
    body = r"""
    for (int which = 0; which < 6; ++which) {
        nvfp4_sequence_t s = nullptr;
        CHECK(nvfp4_sequence_create(&s) == NVFP4_OK);
        countdown = 0;
        const int32_t* const off = static_cast<const int32_t*>(P);
        const int st = which == 0 ? nvfp4_sequence_add_gemm(s, P, P, P, P, 1.0f, P, 16, 64, 128)
                     : which == 1 ? nvfp4_sequence_add_grouped_gemm(s, P, P, P, P, off, 2, 1.0f, P, 16, 64, 128)
                     : which == 2 ? nvfp4_sequence_add_quantize(s, static_cast<const float*>(P), 16, 128, 128, P, P)
                     : which == 3 ? nvfp4_sequence_add_gemm_quantized(s, P, 1, 128, P, P, 1.0f, P, 1, 64, 128)
                     : which == 4 ? nvfp4_sequence_add_quantize_bf16(s, P, 16, 128, 128, P, P) : moe(s, 4);
        countdown = -1;
        CHECK(st == NVFP4_ERR_ALLOC);
        CHECK(nvfp4_sequence_finalize(s) == NVFP4_ERR_INVALID_VALUE);
        CHECK(nvfp4_sequence_destroy(s) == NVFP4_OK);
    }
    std::printf("ok\n");
    return 0;
}
"""
    build_and_run(tmp_path, MAIN[:MAIN.index("    int failed = 0;")] + body)
