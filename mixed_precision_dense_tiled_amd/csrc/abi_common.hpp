// abi_common.hpp -- what the sources of the C ABI share: the error record and
// the device check (defined in abi.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "mpdt.h"

#define MPDT_EXPORT extern "C" __attribute__((visibility("default")))

namespace mpdt {

// Records "fn: what" for mpdt_last_error() and returns s.
mpdt_status abi_fail(mpdt_status s, const char* fn, const char* what);
// The current device is a gfx950.
mpdt_status abi_check_device(const char* fn);
// A launch's error as a status.
mpdt_status abi_launched(hipError_t e, const char* fn);

}  // namespace mpdt
