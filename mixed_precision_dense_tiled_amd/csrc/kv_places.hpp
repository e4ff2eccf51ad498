// kv_places.hpp -- where a new token belongs in a paged cache, and the conversions
// of what is written there; shared by the kernels that append.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"
#include "serving.hpp"

namespace mpdt {

__device__ __forceinline__ float widen(uint16_t x, bool bf16) {
    return bf16 ? __uint_as_float((uint32_t)x << 16) : (float)__builtin_bit_cast(_Float16, x);
}

// x / scale, cut to the format's range (NaN stays), rounded to nearest even.
__device__ __forceinline__ float cut448(float x) { return x > 448.0f ? 448.0f : x < -448.0f ? -448.0f : x; }

struct Place {
    int64_t off;    // byte offset of the token's slot in K and V, -1: it has none
    int pos;        // position in its sequence
    bool in;        // it belongs to a sequence
};

// Places of the N <= 64 tokens from t0 on, one to a lane, by one whole wave: a
// token's sequence is the last that starts at or before it, found among up to 64 in
// one look (a lane each), else by halves.
template <int N>
__device__ __forceinline__ Place place_of(const PagedKV& kv, const SeqView& sv, int t0, int lane) {
    const int t = t0 + lane;
    int seq = 0;
    if (sv.seqs <= 64) {
        const int start = lane < sv.seqs ? sv.cu_q[lane] : 0x7fffffff;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int upto = __popcll(__ballot(start <= t0 + k));
            if (lane == k) seq = upto > 0 ? upto - 1 : 0;
        }
    } else if (lane < N) {
        int hi = sv.seqs;
        while (hi - seq > 1) {
            const int mid = (seq + hi) / 2;
            if (sv.cu_q[mid] <= t) seq = mid;
            else hi = mid;
        }
    }
    Place p{-1, 0, false};
    if (lane < N) {
        const Seq s = seq_of(sv, kv.page_size, seq);
        p.pos = s.n - (s.start + s.nq - t);
        p.in = t >= s.start && t < s.start + s.nq;
        if (p.in && p.pos >= 0) {
            const int pi = kv.page_of(p.pos);
            const int pg = sv.table[(int64_t)seq * sv.ld_table + pi];
            if (pg >= 0 && pg < kv.pages) p.off = pg * kv.page_b + (p.pos - pi * kv.page_size) * kv.slot_b;
        }
    }
    return p;
}

}  // namespace mpdt
