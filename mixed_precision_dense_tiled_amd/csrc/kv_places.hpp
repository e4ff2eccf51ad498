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
    int seq, pos;   // its sequence, and its position there
    bool in;        // it belongs to a sequence
};

// Where the N <= 64 tokens from t0 on stand, one to a lane, by one whole wave: a token's
// sequence is the last that starts at or before it.  Among up to 64 it is found in one
// look, a lane having read each; else by halves.  (The lanes' own reads of their sequences after
// the look made paged_kv_append of 8800 tokens 13.8 us, 13.4 so; 64 single tokens 4.8 and 4.7.)
template <int N>
__device__ __forceinline__ Place place_of(const PagedKV& kv, const SeqView& sv, int t0, int lane) {
    const int t = t0 + lane;
    int seq = 0;
    Seq s;
    if (sv.seqs <= 64) {
        const int b = min(lane, sv.seqs - 1);
        const int start = lane < sv.seqs ? sv.cu_q[lane] : 0x7fffffff;
        const Seq own = seq_of(sv, kv.page_size, b);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int upto = __popcll(__ballot(start <= t0 + k));
            if (lane == k) seq = upto > 0 ? upto - 1 : 0;
        }
        s.start = __shfl(own.start, seq);
        s.nq = __shfl(own.nq, seq);
        s.n = __shfl(own.n, seq);
    } else {
        if (lane < N) {
            int hi = sv.seqs;
            while (hi - seq > 1) {
                const int mid = (seq + hi) / 2;
                if (sv.cu_q[mid] <= t) seq = mid;
                else hi = mid;
            }
        }
        s = seq_of(sv, kv.page_size, seq);
    }
    return Place{seq, s.n - (s.start + s.nq - t), t >= s.start && t < s.start + s.nq};
}

// Byte offset of its slot in K and V; -1: it has none.
__device__ __forceinline__ int64_t slot_of(const PagedKV& kv, const SeqView& sv, const Place& p) {
    if (!p.in || p.pos < 0) return -1;
    const int pi = kv.page_of(p.pos);
    const int pg = sv.table[(int64_t)p.seq * sv.ld_table + pi];
    return pg >= 0 && pg < kv.pages ? pg * kv.page_b + (p.pos - pi * kv.page_size) * kv.slot_b : -1;
}

}  // namespace mpdt
