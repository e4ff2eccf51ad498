"""The host code of a decoder layer's operators at its limits, under AddressSanitizer and
UndefinedBehaviorSanitizer on the CPU: a host-only build whose workspaces and limits are the
library's own (csrc/layer_sizes.hpp) and whose launchers are stubs that abort if ever reached,
against which the tests of both sides of each limit run.  Skipped where a GPU is visible."""
import os
import shutil
import subprocess

import pytest
import torch

from test_sanitizers import CSRC, ROOT, STUBS, _child
from test_serving_sanitizers import SERVING_STUBS

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="host-only builds; a GPU is visible")

LAUNCHERS = """#include <cstdlib>
#include "layer_sizes.hpp"
namespace mpdt {
hipError_t launch_rms_norm(const NormArgs&, hipStream_t) { std::abort(); }
int64_t rms_norm_backward_ws(int64_t rows, int64_t dim) { return grad_sums_bytes(rows, dim); }
hipError_t launch_rms_norm_backward(const NormGradArgs&, hipStream_t) { std::abort(); }
hipError_t launch_paged_append_rope(const RopeArgs&, hipStream_t) { std::abort(); }
bool grouped_fits(int mode, const GroupedArgs& a) { return tiles_fit(mode, a); }
hipError_t launch_grouped(GroupedType, int, const GroupedArgs&, hipStream_t) { std::abort(); }
}  // namespace mpdt
"""


def test_limits_under_asan_ubsan(tmp_path):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    stubs = tmp_path / "stubs.hip"
    stubs.write_text(STUBS + SERVING_STUBS + LAUNCHERS)
    lib = str(tmp_path / "libmpdt_limits_san.so")
    # host-only build: every sanitizer flag is for the host compiler
    subprocess.run([hipcc, "--offload-arch=gfx950", "--offload-host-only", "-O1", "-g", "-fPIC", "-std=c++17",
                    "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
                    "-Xarch_host", "-fno-sanitize-recover=all", "-shared-libsan",
                    "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-shared", os.path.join(CSRC, "abi.hip"),
                    os.path.join(CSRC, "serving_abi.hip"), os.path.join(CSRC, "layers_abi.hip"), str(stubs), "-o",
                    lib], check=True)
    rt = subprocess.run([hipcc, "--print-file-name=libclang_rt.asan-x86_64.so"], capture_output=True,
                        text=True).stdout.strip()
    if not os.path.isabs(rt) or not os.path.exists(rt):
        pytest.skip("clang's ASan runtime not found")
    _child({"MPDT_LIB_PATH": lib, "LD_PRELOAD": rt}, ["tests/test_layers_limits.py", "tests/test_layers_binding.py"],
           tmp_path)
