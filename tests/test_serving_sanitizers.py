"""The serving operators' host code (csrc/serving_abi.hip: argument checks,
spans, overlap and overflow arithmetic) under AddressSanitizer and
UndefinedBehaviorSanitizer on the CPU: a host-only build with the launchers
replaced by stubs that abort if ever reached, against which the ABI and binding
tests run.  Skipped where a GPU is visible (valid calls would reach the stubs)."""
import os
import shutil
import subprocess

import pytest
import torch

from test_sanitizers import CSRC, ROOT, STUBS, _child

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="host-only builds; a GPU is visible")

SERVING_STUBS = """#include <cstdlib>
#include "serving.hpp"
namespace mpdt {
int64_t attn_workspace(const AttnArgs& a) { return (int64_t)a.sv.width * a.kv.page_size > 1024 ? 4096 : 0; }
hipError_t launch_paged_attention(const AttnArgs&, hipStream_t) { std::abort(); }
hipError_t launch_paged_append(const AppendArgs&, hipStream_t) { std::abort(); }
int64_t pages_workspace(int64_t pages, int64_t rows) { return (16 + 2 * pages + rows) * 4; }
hipError_t launch_cache_fork(const PagesArgs&, hipStream_t) { std::abort(); }
hipError_t launch_cache_extend(const PagesArgs&, hipStream_t) { std::abort(); }
hipError_t launch_cache_free(const PagesArgs&, hipStream_t) { std::abort(); }
hipError_t launch_cache_compact(const PagesArgs&, hipStream_t) { std::abort(); }
bool logprob_fits(int, int64_t rows, int64_t vocab) { return rows * ((vocab + 8191) / 8192) <= 0x7fffffff; }
int64_t logprob_workspace(int, int64_t rows, int64_t vocab, int top) {
    return vocab > 8192 ? rows * (16 + 8 * top) : rows * (vocab > 4096 ? 2 * (16 + 8 * top) : 0);
}
hipError_t launch_token_logprobs(const LogprobArgs&, hipStream_t) { std::abort(); }
hipError_t launch_token_logprobs_backward(const LogprobArgs&, hipStream_t) { std::abort(); }
}  // namespace mpdt
"""


def test_serving_host_code_under_asan_ubsan(tmp_path):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    stubs = tmp_path / "stubs.hip"
    stubs.write_text(STUBS + SERVING_STUBS)
    lib = str(tmp_path / "libmpdt_serving_san.so")
    # host-only build: every sanitizer flag is for the host compiler
    subprocess.run([hipcc, "--offload-arch=gfx950", "--offload-host-only", "-O1", "-g", "-fPIC", "-std=c++17",
                    "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
                    "-Xarch_host", "-fno-sanitize-recover=all", "-shared-libsan",
                    "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-shared", os.path.join(CSRC, "abi.hip"),
                    os.path.join(CSRC, "serving_abi.hip"), str(stubs), "-o", lib], check=True)
    rt = subprocess.run([hipcc, "--print-file-name=libclang_rt.asan-x86_64.so"], capture_output=True,
                        text=True).stdout.strip()
    if not os.path.isabs(rt) or not os.path.exists(rt):
        pytest.skip("clang's ASan runtime not found")
    _child({"MPDT_LIB_PATH": lib, "LD_PRELOAD": rt}, ["tests/test_serving_binding.py"], tmp_path)
