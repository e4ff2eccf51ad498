// rotary.hip -- new keys and values into a paged cache, the keys rotated by their
// positions on the way, and the queries beside them.
//
//   a' = a cos t - b sin t,  b' = b cos t + a sin t,  t = position * inv_freq[pair]
//
// Bound by the bytes that it moves.  A workgroup takes a few tokens: one wave finds
// where they belong, all threads then form the tokens' angles (each once, for every
// head) into LDS, and the rows go through registers once.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"
#include "kv_places.hpp"
#include "layers.hpp"

namespace mpdt {
namespace {

// cos and sin of p * f.  The angle in turns is p * f / 2 pi; FP64 holds it to 2^-52 of
// itself (p < 2^31: 1e-7 of a turn at the very end, 1e-10 below 10^6).  Whole quarters
// come off there; what is left, at most pi / 4, goes through the Taylor series of
// sine (to x^9 / 9!, next term 2e-9) and cosine (to x^10 / 10!, next term 1.2e-10).
__device__ __forceinline__ float2 cos_sin(int p, float f) {
    const double turns = (double)p * (double)f * 0.15915494309189533577;
    const double quarters = __builtin_rint(turns * 4.0);
    const float x = (float)((turns - quarters * 0.25) * 6.283185307179586477);
    const float z = x * x;
    float s = 1.0f / 362880.0f, c = -1.0f / 3628800.0f;
    s = fmaf(s, z, -1.0f / 5040.0f);
    s = fmaf(s, z, 1.0f / 120.0f);
    s = fmaf(s, z, -1.0f / 6.0f);
    s = fmaf(s * z, x, x);
    c = fmaf(c, z, 1.0f / 40320.0f);
    c = fmaf(c, z, -1.0f / 720.0f);
    c = fmaf(c, z, 1.0f / 24.0f);
    c = fmaf(c, z, -0.5f);
    c = fmaf(c, z, 1.0f);
    const int q = (int)(int64_t)quarters & 3;
    const float cc = q & 1 ? s : c, ss = q & 1 ? c : s;
    return float2{q == 1 || q == 2 ? -cc : cc, q & 2 ? -ss : ss};
}

__device__ __forceinline__ uint16_t narrow(float x, bool bf16) { return bf16 ? f32_to_bf16_bits(x) : f32_to_f16_bits(x); }

__device__ __forceinline__ uint8_t to_e4m3(float x) {
    return (uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(x, 0.0f, 0, false) & 0xff);
}

constexpr int ROPE_TOKENS = 8;

template <bool TO8>
__global__ __launch_bounds__(256) void append_rope_kernel(RopeArgs r) {
    const AppendArgs& a = r.ap;
    __shared__ int64_t dst[ROPE_TOKENS];
    __shared__ int pos[ROPE_TOKENS], in[ROPE_TOKENS];
    __shared__ float2 turn[ROPE_TOKENS][64];
    const int t0 = blockIdx.x * ROPE_TOKENS;
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x;
        const Place p = place_of<ROPE_TOKENS>(a.kv, a.sv, t0, lane);
        if (lane < ROPE_TOKENS) {
            dst[lane] = p.off;
            pos[lane] = p.pos;
            in[lane] = p.in;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < ROPE_TOKENS * r.pairs; i += 256) {
        const int k = i / r.pairs, j = i - k * r.pairs;
        if (in[k]) turn[k][j] = cos_sin(pos[k], r.inv_freq[j]);
    }
    __syncthreads();
    const bool bf16 = a.type == DT_BF16;
    const int dim = a.kv.dim, heads = r.heads + 2 * a.kv.kv_heads;
    // one pair (or one element that is not rotated, or of V) at a time
    const int items = ROPE_TOKENS * heads * dim;
    for (int i = threadIdx.x; i < items; i += 256) {
        const int k = i / (heads * dim), rest = i - k * heads * dim, hh = rest / dim, d = rest - hh * dim;
        if (!in[k]) continue;
        const bool is_q = hh < r.heads, is_v = hh >= r.heads + a.kv.kv_heads;
        const int h = is_q ? hh : is_v ? hh - r.heads - a.kv.kv_heads : hh - r.heads;
        if (!is_q && dst[k] < 0) continue;
        const int64_t t = t0 + k;
        const char* src = is_q ? r.q + t * r.q_tok_b + h * r.q_head_b
                          : is_v ? a.v_new + t * a.v_tok_b + h * a.v_head_b : a.k_new + t * a.k_tok_b + h * a.k_head_b;
        char* to = is_q ? r.q_out + t * r.qo_tok_b + h * r.qo_head_b
                        : (is_v ? a.kv.v : a.kv.k) + dst[k] + h * a.kv.head_b;
        const uint16_t* x = reinterpret_cast<const uint16_t*>(src);
        const bool turned = !is_v && d < 2 * r.pairs;
        // the second of a pair is done with the first
        if (turned && (r.interleaved ? d & 1 : d >= r.pairs)) continue;
        const int d2 = r.interleaved ? d + 1 : d + r.pairs;
        float y = widen(x[d], bf16), y2 = 0;
        if (turned) {
            const float2 cs = turn[k][r.interleaved ? d >> 1 : d];
            const float p = y, q = widen(x[d2], bf16);
            y = p * cs.x - q * cs.y;
            y2 = q * cs.x + p * cs.y;
        }
        if (TO8 && !is_q) {
            const float scale = (is_v ? a.kv.v_scale : a.kv.k_scale)[h];
            to[d] = (char)to_e4m3(cut448(y / scale));
            if (turned) to[d2] = (char)to_e4m3(cut448(y2 / scale));
        } else {
            reinterpret_cast<uint16_t*>(to)[d] = turned ? narrow(y, bf16) : x[d];
            if (turned) reinterpret_cast<uint16_t*>(to)[d2] = narrow(y2, bf16);
        }
    }
}

}  // namespace

hipError_t launch_paged_append_rope(const RopeArgs& r, hipStream_t stream) {
    const dim3 grid((unsigned)((r.ap.sv.tokens + ROPE_TOKENS - 1) / ROPE_TOKENS));
    if (r.ap.kv.type == DT_E4M3) append_rope_kernel<true><<<grid, dim3(256), 0, stream>>>(r);
    else append_rope_kernel<false><<<grid, dim3(256), 0, stream>>>(r);
    return hipGetLastError();
}

}  // namespace mpdt
