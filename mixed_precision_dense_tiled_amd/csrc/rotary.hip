// rotary.hip -- new keys and values into a paged cache, the keys rotated by their
// positions on the way, and the queries beside them.
//
//   a' = a cos t - b sin t,  b' = b cos t + a sin t,  t = position * inv_freq[pair]
//
// Bound by the bytes that it moves.  A workgroup takes a few tokens: one wave finds
// where they belong, all threads then form the tokens' angles (each once, for every
// head) into LDS, and the rows go through registers once.  8800 tokens of 32 + 8 heads of
// 128, BF16: 42 us, 5.2 TB/s, what a large copy reaches; 64 tokens 4.9 us, the way from a
// token to its sequence, page and angles; 4801 tokens of 16 + 4 heads of 80 into E4M3 14.2
// us, 2.4 TB/s: the codes' arithmetic.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device_common.hpp"
#include "kv_places.hpp"
#include "layers.hpp"
#include "quotient.hpp"

namespace mpdt {
namespace {

// cos and sin of p * f.  The angle in turns is p * f / 2 pi; FP64 holds it to 2^-52 of
// itself (p < 2^31: 1e-7 of a turn at the very end, 1e-10 below 10^6).  Whole quarters
// come off there; what is left, at most pi / 4, goes through the Taylor series of
// sine (to x^11 / 11!, next term 7e-12) and cosine (to x^12 / 12!, next term 4e-13) in FP64
// and is rounded once: half a step of FP32 off.  (Series in FP32 are up to 7e-8 off
// instead of 3e-8, which shows where a cos t and b sin t cancel, and no faster: 8800 tokens 44 us
// either way, inside a graph.)
__device__ __forceinline__ float2 cos_sin(int p, float f) {
    const double turns = (double)p * (double)f * 0.15915494309189533577;
    const double quarters = __builtin_rint(turns * 4.0);
    const double x = (turns - quarters * 0.25) * 6.283185307179586477, z = x * x;
    double sd = -1.0 / 39916800.0, cd = 1.0 / 479001600.0;
    cd = fma(cd, z, -1.0 / 3628800.0);
    sd = fma(sd, z, 1.0 / 362880.0);
    cd = fma(cd, z, 1.0 / 40320.0);
    sd = fma(sd, z, -1.0 / 5040.0);
    cd = fma(cd, z, -1.0 / 720.0);
    sd = fma(sd, z, 1.0 / 120.0);
    cd = fma(cd, z, 1.0 / 24.0);
    sd = fma(sd, z, -1.0 / 6.0);
    cd = fma(cd, z, -0.5);
    const float s = (float)fma(sd * z, x, x), c = (float)fma(cd, z, 1.0);
    const int q = (int)(int64_t)quarters & 3;
    const float cc = q & 1 ? s : c, ss = q & 1 ? c : s;
    return float2{q == 1 || q == 2 ? -cc : cc, q & 2 ? -ss : ss};
}

__device__ __forceinline__ uint16_t narrow(float x, bool bf16) { return bf16 ? f32_to_bf16_bits(x) : f32_to_f16_bits(x); }

__device__ __forceinline__ uint8_t to_e4m3(float x) {
    return (uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(x, 0.0f, 0, false) & 0xff);
}

// What a workgroup's tokens need: where they belong, and their angles.
template <int N>
struct Tokens {
    int64_t dst[N];
    int pos[N], in[N];
    float2 turn[N][64];
};
// (a workgroup of 256 threads)
template <int N>
__device__ __forceinline__ void find_tokens(const RopeArgs& r, int t0, Tokens<N>& to) {
    Place p{};
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x;
        p = place_of<N>(r.ap.kv, r.ap.sv, t0, lane);
        if (lane < N) {
            to.pos[lane] = p.pos;
            to.in[lane] = p.in;
        }
    }
    // half (a quarter, ..) of the threads to a token
    constexpr int PER = 256 / N;
    const int k = threadIdx.x / PER, j = threadIdx.x % PER;
    const float f = j < r.pairs ? r.inv_freq[j] : 0.0f;
    __syncthreads();
    // (the page's number is on its way while the angles are worked out)
    int64_t dst = -1;
    if (threadIdx.x < N) dst = slot_of(r.ap.kv, r.ap.sv, p);
    if (to.in[k]) {
        if (j < r.pairs) to.turn[k][j] = cos_sin(to.pos[k], f);
        if constexpr (PER < 64)
            for (int i = j + PER; i < r.pairs; i += PER) to.turn[k][i] = cos_sin(to.pos[k], r.inv_freq[i]);
    }
    if (threadIdx.x < N) to.dst[threadIdx.x] = dst;
    __syncthreads();
}

// 8 elements to E4M3, as the division by the scale gives them.  (What is past the range of
// E4M3 keeps the product with the reciprocal, which is past it too.)
__device__ __forceinline__ u32x2 to_e4m3_8(const float (&x)[8], float scale) {
    float q[8];
    if (divides(scale)) {
        const float r = 1.0f / scale;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float p = x[i] * r;
            q[i] = fabsf(p) <= 1000.0f ? quotient(x[i], scale, r) : p;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = x[i] / scale;
    }
    u32x2 w;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        int c = __builtin_amdgcn_cvt_pk_fp8_f32(cut448(q[4 * j]), cut448(q[4 * j + 1]), 0, false);
        w[j] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(cut448(q[4 * j + 2]), cut448(q[4 * j + 3]), c, true);
    }
    return w;
}

// Rows in pieces of 16 bytes: a thread takes two pieces of a head that turn together (or
// that lie beside each other, where nothing turns), four such at a time.  The first
// four are under way before the workgroup looks its tokens up.  Wants pairs that fill
// pieces, or neighbouring pairs, which always do.
template <bool BF16, bool TO8, bool NEAR, int N>
__global__ __launch_bounds__(256) void append_rope_kernel(RopeArgs r) {
    const AppendArgs& a = r.ap;
    __shared__ Tokens<N> tok;
    const int t0 = blockIdx.x * N;
    const int per = a.kv.dim / 16, j = threadIdx.x % per, first = threadIdx.x / per, step = 256 / per;
    const int heads = r.heads + 2 * a.kv.kv_heads, rows = first < step ? N * heads : 0;
    const int turned = NEAR ? per : r.pairs / 8;        // of q's and K's items
    constexpr int U = 4;
    u32x4 x[U][2];
    // row i: all of q's, then K's, then V's (a wave then has rows of one kind); of each kind
    // one token's heads after the other's
    struct Row {
        int kind, k, h;     // 0 q, 1 K, 2 V
    };
    auto row_at = [&](int i) {
        Row w{0, 0, i};
        int n = r.heads;
        if (i >= N * r.heads) {
            n = a.kv.kv_heads;
            w.h -= N * r.heads;
            w.kind = w.h >= N * n ? 2 : 1;
            w.h -= (w.kind - 1) * N * n;
        }
        w.k = N == 1 ? 0 : w.h / n;
        w.h -= w.k * n;
        return w;
    };
    auto load = [&](int i0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const Row w = row_at(min(i0 + u * step, N * heads - 1));
            const int64_t t = min(t0 + w.k, a.sv.tokens - 1);   // (a row that is there)
            const char* p = w.kind == 0 ? r.q + t * r.q_tok_b + w.h * r.q_head_b
                            : w.kind == 1 ? a.k_new + t * a.k_tok_b + w.h * a.k_head_b
                                          : a.v_new + t * a.v_tok_b + w.h * a.v_head_b;
            const bool apart = !NEAR && w.kind < 2 && j < turned;
            const int c0 = apart ? j : 2 * j, c1 = apart ? j + turned : 2 * j + 1;
            x[u][0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p + 16 * c0));
            x[u][1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p + 16 * c1));
        }
    };
    if (rows) load(first);
    find_tokens<N>(r, t0, tok);
    for (int i0 = first; i0 < rows; i0 += U * step) {
        if (i0 != first) load(i0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * step;
            if (i >= rows) break;
            const auto [kind, k, h] = row_at(i);
            const int64_t dst = tok.dst[k];
            if (kind == 0 ? !tok.in[k] : dst < 0) continue;
            const bool apart = !NEAR && kind < 2 && j < turned;
            const int c0 = apart ? j : 2 * j, c1 = apart ? j + turned : 2 * j + 1;
            const bool turns = NEAR ? kind < 2 && 8 * j < r.pairs : apart;
            const bool to8 = TO8 && kind > 0;
            float y[2][8];
            if (turns || to8) {
#pragma unroll
                for (int e = 0; e < 16; ++e) y[e >> 3][e & 7] = widen((uint16_t)(x[u][e >> 3][(e & 7) >> 1] >> (16 * (e & 1))), BF16);
            }
            if (turns) {
                const float2* cs = tok.turn[k] + 8 * j;
                if constexpr (NEAR) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (8 * j + e < r.pairs) {
                            const float2 t = cs[e];
                            const float p = y[e >> 2][2 * (e & 3)], q = y[e >> 2][2 * (e & 3) + 1];
                            y[e >> 2][2 * (e & 3)] = p * t.x - q * t.y;
                            y[e >> 2][2 * (e & 3) + 1] = q * t.x + p * t.y;
                        }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 t = cs[e];
                        const float p = y[0][e], q = y[1][e];
                        y[0][e] = p * t.x - q * t.y;
                        y[1][e] = q * t.x + p * t.y;
                    }
                }
                if (!to8) {
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int w = 0; w < 4; ++w)
                            x[u][c][w] = narrow(y[c][2 * w], BF16) | (uint32_t)narrow(y[c][2 * w + 1], BF16) << 16;
                }
            }
            if (kind == 0) {
                char* to = r.q_out + (int64_t)(t0 + k) * r.qo_tok_b + h * r.qo_head_b;
                *reinterpret_cast<u32x4*>(to + 16 * c0) = x[u][0];
                *reinterpret_cast<u32x4*>(to + 16 * c1) = x[u][1];
                continue;
            }
            char* to = (kind == 1 ? a.kv.k : a.kv.v) + dst + h * a.kv.head_b;
            if constexpr (TO8) {
                const float scale = (kind == 1 ? a.kv.k_scale : a.kv.v_scale)[h];
                *reinterpret_cast<u32x2*>(to + 8 * c0) = to_e4m3_8(y[0], scale);
                *reinterpret_cast<u32x2*>(to + 8 * c1) = to_e4m3_8(y[1], scale);
            } else {
                *reinterpret_cast<u32x4*>(to + 16 * c0) = x[u][0];
                *reinterpret_cast<u32x4*>(to + 16 * c1) = x[u][1];
            }
        }
    }
}

// Pairs that fill no pieces: one pair, or one element that does not turn, at a time.  Bound by
// that: 8800 tokens of 32 + 8 heads of 96 with 12 pairs, FP16, 163 us, where 16 pairs take 40.
constexpr int ROPE_TOKENS = 8;

template <bool TO8>
__global__ __launch_bounds__(256) void append_rope_any_kernel(RopeArgs r) {
    const AppendArgs& a = r.ap;
    __shared__ Tokens<ROPE_TOKENS> tok;
    const int t0 = blockIdx.x * ROPE_TOKENS;
    find_tokens<ROPE_TOKENS>(r, t0, tok);
    const bool bf16 = a.type == DT_BF16;
    const int dim = a.kv.dim, heads = r.heads + 2 * a.kv.kv_heads;
    // one pair (or one element that is not rotated, or of V) at a time
    const int items = ROPE_TOKENS * heads * dim;
    for (int i = threadIdx.x; i < items; i += 256) {
        const int k = i / (heads * dim), rest = i - k * heads * dim, hh = rest / dim, d = rest - hh * dim;
        if (!tok.in[k]) continue;
        const bool is_q = hh < r.heads, is_v = hh >= r.heads + a.kv.kv_heads;
        const int h = is_q ? hh : is_v ? hh - r.heads - a.kv.kv_heads : hh - r.heads;
        if (!is_q && tok.dst[k] < 0) continue;
        const int64_t t = t0 + k;
        const char* src = is_q ? r.q + t * r.q_tok_b + h * r.q_head_b
                          : is_v ? a.v_new + t * a.v_tok_b + h * a.v_head_b : a.k_new + t * a.k_tok_b + h * a.k_head_b;
        char* to = is_q ? r.q_out + t * r.qo_tok_b + h * r.qo_head_b
                        : (is_v ? a.kv.v : a.kv.k) + tok.dst[k] + h * a.kv.head_b;
        const uint16_t* x = reinterpret_cast<const uint16_t*>(src);
        const bool turned = !is_v && d < 2 * r.pairs;
        // the second of a pair is done with the first
        if (turned && (d >= r.pairs)) continue;
        const int d2 = d + r.pairs;
        float y = widen(x[d], bf16), y2 = 0;
        if (turned) {
            const float2 cs = tok.turn[k][d];
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
    const AppendArgs& a = r.ap;
    const bool to8 = a.kv.type == DT_E4M3, bf16 = a.type == DT_BF16;
    if (!r.interleaved && r.pairs % 8) {
        const dim3 grid((unsigned)((a.sv.tokens + ROPE_TOKENS - 1) / ROPE_TOKENS));
        if (to8) append_rope_any_kernel<true><<<grid, dim3(256), 0, stream>>>(r);
        else append_rope_any_kernel<false><<<grid, dim3(256), 0, stream>>>(r);
        return hipGetLastError();
    }
    // Tokens of a workgroup: enough rows for three rounds of its threads, and one where the
    // tokens are too few for two workgroups to a CU
    const int step = 256 / (a.kv.dim / 16), heads = r.heads + 2 * a.kv.kv_heads;
    int n = 1;
    while (n < 8 && n * heads < 3 * step && a.sv.tokens / (2 * n) >= 512) n *= 2;
    const auto go = [&](auto BF16, auto TO8, auto NEAR, auto N) {
        constexpr int tokens = decltype(N)::value;
        append_rope_kernel<decltype(BF16)::value, decltype(TO8)::value, decltype(NEAR)::value, tokens>
            <<<dim3((unsigned)((a.sv.tokens + tokens - 1) / tokens)), dim3(256), 0, stream>>>(r);
    };
    const auto yes = std::true_type{};
    const auto no = std::false_type{};
    const auto with_n = [&](auto BF16, auto TO8, auto NEAR) {
        using std::integral_constant;
        if (n == 1) go(BF16, TO8, NEAR, integral_constant<int, 1>{});
        else if (n == 2) go(BF16, TO8, NEAR, integral_constant<int, 2>{});
        else if (n == 4) go(BF16, TO8, NEAR, integral_constant<int, 4>{});
        else go(BF16, TO8, NEAR, integral_constant<int, 8>{});
    };
    const auto with_near = [&](auto BF16, auto TO8) {
        if (r.interleaved) with_n(BF16, TO8, yes);
        else with_n(BF16, TO8, no);
    };
    if (bf16) to8 ? with_near(yes, yes) : with_near(yes, no);
    else to8 ? with_near(no, yes) : with_near(no, no);
    return hipGetLastError();
}

}  // namespace mpdt
