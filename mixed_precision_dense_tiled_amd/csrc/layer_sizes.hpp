// layer_sizes.hpp -- how many workgroups the launches of a decoder layer's operators make
// of a call's sizes: what their kernels, their workspaces and their limits go by.
#pragma once

#include <stdint.h>

#include "layers.hpp"

namespace mpdt {

// Workgroups of a norm's gradient.  Each (each wave, for rows of up to 1024 elements) walks
// rows of its own and keeps its columns' sums of grad * h * rstd in registers; a second launch
// adds the workgroups' sums in their order.  Few workgroups leave loads waiting, many have that
// many sums to write and read again (us at workgroups: 500 x 5120 FP16 20 at 500, 14.4 at
// 250, 15.5 at 128 of 512 threads; 16000 x 1000 53 at 512, 27 at 1024 of four rows; 2000 x 16384 60 at
// 512, 46 at 256).
inline int grad_groups(int64_t rows, int64_t dim) {
    const int64_t n = dim <= 1024 ? (rows + 3) / 4 : rows;     // (rows of a workgroup at a time)
    const int64_t most = dim <= 2048 ? 1024 : dim <= 8192 ? 512 : 256;
    const int64_t few = n < 128 ? n : n < 384 ? 128 : n / 3;
    return (int)(few < most ? few : most);
}
// Bytes of their sums; one workgroup writes the result.
inline int64_t grad_sums_bytes(int64_t rows, int64_t dim) {
    const int g = grad_groups(rows, dim);
    return g > 1 ? 4 * g * dim : 0;
}

// The most row tiles of bm rows that the groups of a grouped product can have.
inline int64_t most_row_tiles(const GroupedArgs& a, int64_t bm) {
    return a.rows / bm + (a.rows < a.groups ? a.rows : a.groups);
}
inline int64_t grouped_tiles(int mode, const GroupedArgs& a, int64_t bm, int64_t bn) {
    const int64_t tn = (a.N + bn - 1) / bn;
    return tn * (mode == GROUPED_TN ? (a.M + bm - 1) / bm * a.groups : most_row_tiles(a, bm));
}
// Whether its launches hold them (and what the XCDs' shares round up).
inline bool tiles_fit(int mode, const GroupedArgs& a) {
    constexpr int64_t xcds = 8;
    return grouped_tiles(mode, a, 128, 128) <= MAX_GROUPS - xcds;
}

}  // namespace mpdt
