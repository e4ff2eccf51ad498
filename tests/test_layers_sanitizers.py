"""The host code of a decoder layer's operators (csrc/layers_abi.hip: argument
checks, spans, overlap and overflow arithmetic) under AddressSanitizer and
UndefinedBehaviorSanitizer on the CPU: a host-only build with the launchers
replaced by stubs that abort if ever reached, against which the ABI and binding
tests run.  Skipped where a GPU is visible (valid calls would reach the stubs)."""
import os
import shutil
import subprocess

import pytest
import torch

from test_sanitizers import CSRC, ROOT, STUBS, _child
from test_serving_sanitizers import SERVING_STUBS

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="host-only builds; a GPU is visible")

LAYER_STUBS = """#include <cstdlib>
#include "layers.hpp"
namespace mpdt {
hipError_t launch_rms_norm(const NormArgs&, hipStream_t) { std::abort(); }
int64_t rms_norm_backward_ws(int64_t rows, int64_t dim) {
    return rows > 1 ? 4 * (rows < 512 ? rows : 512) * dim : 0;
}
hipError_t launch_rms_norm_backward(const NormGradArgs&, hipStream_t) { std::abort(); }
hipError_t launch_paged_append_rope(const RopeArgs&, hipStream_t) { std::abort(); }
bool grouped_fits(int mode, const GroupedArgs& a) {
    const int64_t rows = mode == GROUPED_TN ? (a.M + 127) / 128 * (int64_t)a.groups
                                            : a.rows / 128 + (a.rows < a.groups ? a.rows : a.groups);
    return rows * ((a.N + 127) / 128) <= MAX_GROUPS;
}
hipError_t launch_grouped(GroupedType, int, const GroupedArgs&, hipStream_t) { std::abort(); }
}  // namespace mpdt
"""


def test_layers_host_code_under_asan_ubsan(tmp_path):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    stubs = tmp_path / "stubs.hip"
    stubs.write_text(STUBS + SERVING_STUBS + LAYER_STUBS)
    lib = str(tmp_path / "libmpdt_layers_san.so")
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
    _child({"MPDT_LIB_PATH": lib, "LD_PRELOAD": rt}, ["tests/test_layers_binding.py"], tmp_path)
