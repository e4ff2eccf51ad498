// logprobs.hip -- log probabilities of given tokens, entropy, the most likely
// alternatives, and the gradient.
//
// For a row x of logits and its target t:
//     lse = log sum_j exp(x_j),  logprob = x_t - lse,  p_j = exp(x_j - lse),
//     entropy H = -sum_j p_j log p_j = lse - sum_j p_j x_j,
// and with gradients gl (of logprob) and ge (of entropy)
//     dx_j = gl * ([j = t] - p_j) - ge * p_j * (log p_j + H).
//
// A row is cut into segments, one workgroup each: its values are loaded once
// into registers and give the segment's maximum m, sum e^(x-m), sum e^(x-m)(x-m)
// and its largest `top` values; a second launch joins a row's segments in
// order.  Bound by the bytes of the logits in 16-bit types; the arithmetic (an
// exponential and half a dozen FP32 operations a value) lies close below.
//
// The largest values of a segment: the k-th largest of a wave's 64 lane
// maxima cannot be larger than the k-th largest value, so few values lie at or
// above the best such bound; these are gathered and each counts how many beat
// it (larger, or equal at a lower index).  Where too many tie, or a value is no
// number, k passes over the registers find them one by one.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "device_common.hpp"
#include "serving.hpp"

namespace mpdt {
namespace {

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr int NO_INDEX = 0x7fffffff;
constexpr int NT = 256, WAVES = NT / 64;
constexpr int CAND = 1024;            // gathered values of a workgroup

#define NEG_INF (-__builtin_inff())

template <int TYPE>
struct Elem {
    static constexpr int BYTES = TYPE == DT_F32 ? 4 : 2, PER16 = 16 / BYTES;
    // element j of a 16-byte piece
    static __device__ __forceinline__ float get(const u32x4& v, int j) {
        if constexpr (TYPE == DT_F32) return __uint_as_float(v[j]);
        const uint32_t h = (v[j >> 1] >> (16 * (j & 1))) & 0xffffu;
        if constexpr (TYPE == DT_BF16) return __uint_as_float(h << 16);
        return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
    }
    static __device__ __forceinline__ float at(const char* row, int i) {
        if constexpr (TYPE == DT_F32) return reinterpret_cast<const float*>(row)[i];
        const uint16_t h = reinterpret_cast<const uint16_t*>(row)[i];
        if constexpr (TYPE == DT_BF16) return __uint_as_float((uint32_t)h << 16);
        return (float)__builtin_bit_cast(_Float16, h);
    }
    static __device__ __forceinline__ void put(char* row, int i, float x) {
        if constexpr (TYPE == DT_F32) reinterpret_cast<float*>(row)[i] = x;
        else reinterpret_cast<uint16_t*>(row)[i] = TYPE == DT_BF16 ? f32_to_bf16_bits(x) : f32_to_f16_bits(x);
    }
    static __device__ __forceinline__ u32x4 pack(const float* x) {
        u32x4 r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (TYPE == DT_F32) r[i] = __float_as_uint(x[i]);
            else if constexpr (TYPE == DT_BF16)
                r[i] = f32_to_bf16_bits(x[2 * i]) | ((uint32_t)f32_to_bf16_bits(x[2 * i + 1]) << 16);
            else
                r[i] = f32_to_f16_bits(x[2 * i]) | ((uint32_t)f32_to_f16_bits(x[2 * i + 1]) << 16);
        }
        return r;
    }
};

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v = fmaxf(v, __shfl_xor(v, d));
    return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
    return v;
}

// The k-th largest (k from 0) of the 64 lanes' values: a bitonic sort.
__device__ __forceinline__ float wave_kth(float v, int k) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int size = 2; size <= 64; size <<= 1) {
#pragma unroll
        for (int d = size >> 1; d > 0; d >>= 1) {
            const float o = __shfl_xor(v, d);
            const bool low = (lane & d) == 0, down = (lane & size) == 0 || size == 64;
            v = low == down ? fmaxf(v, o) : fminf(v, o);
        }
    }
    return __shfl(v, k);
}

// Order of (value, index): larger first, NaN above all, then the lower index.
__device__ __forceinline__ uint64_t order_key(float x, int index) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    const uint32_t k = x != x ? 0xffffffffu : (b >> 31) ? ~b : b | 0x80000000u;
    return ((uint64_t)k << 32) | (uint32_t)~index;
}

struct TopShared {
    float bound[WAVES];
    float value[CAND];
    int index[CAND];
    uint64_t best[WAVES];
    int count;
};

// The k largest of the workgroup's values, in order, to (out_v, out_i).
// value(i) / index(i): this thread's N values; mine: their maximum; odd: a
// value is no number.  All threads call it.
template <int N, class V, class I>
__device__ __forceinline__ void block_top(TopShared& sh, int k, float mine, bool odd, V value, I index, float* out_v,
                                          int* out_i) {
    const int tid = threadIdx.x, wave = tid >> 6;
    const float kth = wave_kth(mine, k - 1);
    if ((tid & 63) == 0) sh.bound[wave] = kth;
    if (tid == 0) sh.count = 0;
    __syncthreads();
    float bound = sh.bound[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) bound = fmaxf(bound, sh.bound[w]);
    if (mine >= bound && !odd) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float x = value(i);
            if (x >= bound) {
                const int ix = index(i);
                if (ix != NO_INDEX) {
                    const int at = atomicAdd(&sh.count, 1);
                    if (at < CAND) {
                        sh.value[at] = x;
                        sh.index[at] = ix;
                    }
                }
            }
        }
    }
    __syncthreads();
    const int count = sh.count;
    if (!odd && count >= k && count <= CAND) {
        for (int c = tid; c < count; c += NT) {
            const float x = sh.value[c];
            const int ix = sh.index[c];
            int rank = 0;
            for (int j = 0; j < count; ++j) {
                const float y = sh.value[j];
                rank += y > x || (y == x && sh.index[j] < ix);
            }
            if (rank < k) {
                out_v[rank] = x;
                out_i[rank] = ix;
            }
        }
    } else {
        uint64_t last = ~0ull;      // above every key: no index is -1
        for (int r = 0; r < k; ++r) {
            uint64_t best = 0;
            float bx = NEG_INF;
            int bi = NO_INDEX;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint64_t key = order_key(value(i), index(i));
                if (key < last && key > best) {
                    best = key;
                    bx = value(i);
                    bi = index(i);
                }
            }
            uint64_t all = best;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const uint64_t o = ((uint64_t)(uint32_t)__shfl_xor((int)(all >> 32), d) << 32) |
                                   (uint32_t)__shfl_xor((int)(uint32_t)all, d);
                all = o > all ? o : all;
            }
            if ((tid & 63) == 0) sh.best[wave] = all;
            __syncthreads();
            all = sh.best[0];
#pragma unroll
            for (int w = 1; w < WAVES; ++w) all = sh.best[w] > all ? sh.best[w] : all;
            if (all == 0) {             // fewer than k values
                if (tid == 0) {
                    out_v[r] = NEG_INF;
                    out_i[r] = NO_INDEX;
                }
            } else if (best == all) {
                // padding of several threads has one key: any of them writes the same
                out_v[r] = bx;
                out_i[r] = bi;
            }
            last = all == 0 ? 1 : all;
            __syncthreads();
        }
    }
}

// Per segment in the workspace: maximum, sum, weighted sum, then `top` values
// and indices.
struct SegWs {
    float* stat;    // [rows][segments][4]
    float* value;   // [rows][segments][top]
    int* index;
};
__host__ __device__ inline SegWs seg_ws(char* ws, int64_t rows, int64_t segments, int top) {
    SegWs w;
    w.stat = (float*)ws;
    w.value = (float*)(ws + rows * segments * 16);
    w.index = (int*)(ws + rows * segments * (16 + 4 * (int64_t)top));
    return w;
}

// C: 16-byte pieces a thread.  Pieces are read on 16-byte boundaries of
// memory whatever the row's alignment (a piece that holds a value of the row
// lies in mapped memory); elements before and past the row count as -inf.
template <int TYPE, int C, bool TOP>
__global__ __launch_bounds__(NT) void logprob_segment_kernel(LogprobArgs a) {
    using E = Elem<TYPE>;
    constexpr int P = E::PER16, N = C * P;
    __shared__ TopShared sh;
    __shared__ float red[3][WAVES];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int row = blockIdx.x / a.segments, seg = blockIdx.x % a.segments;
    const char* base = a.logits + (int64_t)row * a.ld_b;
    const int skip = (int)((uintptr_t)base & 15) / E::BYTES;
    const char* aligned = base - skip * E::BYTES;
    const int first = seg * (NT * N) - skip;         // index of the segment's first element
    const bool inner = first >= 0 && first + NT * N <= a.vocab;
    u32x4 v[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int i = first + (c * NT + tid) * P;
        v[c] = u32x4{0, 0, 0, 0};
        if (inner || (i + P > 0 && i < a.vocab))
            v[c] = *reinterpret_cast<const u32x4*>(aligned + ((int64_t)seg * (NT * C) + c * NT + tid) * 16);
    }
    float x[N];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < P; ++j) x[c * P + j] = E::get(v[c], j);
    if (!inner) {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const int i = first + (c * NT + tid) * P + j;
                if (i < 0 || i >= a.vocab) x[c * P + j] = NEG_INF;
            }
    }
    float mine = x[0];
#pragma unroll
    for (int i = 1; i < N; ++i) mine = fmaxf(mine, x[i]);
    const float wm = wave_max(mine);
    if (lane == 0) red[0][wave] = wm;
    __syncthreads();
    float m = red[0][0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) m = fmaxf(m, red[0][w]);
    // y = (x - m) log2(e), the difference first: a mask of the type's lowest
    // value would leave the range times log2(e).  m counts as 0 where every
    // value is -inf.
    const float from = m == NEG_INF ? 0.0f : m;
    float s = 0.0f, t = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float y = (x[i] - from) * LOG2E;
        const float e = __builtin_amdgcn_exp2f(y);                 // no number where x is none, or +inf
        s += e;
        t = fmaf(e, fmaxf(y, -1e30f), t);                          // e = 0 times a finite y where x = -inf
    }
    s = wave_sum(s);
    t = wave_sum(t);
    if (lane == 0) {
        red[1][wave] = s;
        red[2][wave] = t;
    }
    __syncthreads();
    s = red[1][0];
    t = red[2][0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) {
        s += red[1][w];
        t += red[2][w];
    }
    const SegWs ws = seg_ws(a.ws, a.rows, a.segments, a.top);
    const int64_t at = (int64_t)row * a.segments + seg;
    if (tid == 0) *reinterpret_cast<f32x4*>(ws.stat + at * 4) = f32x4{m, s, t, 0.0f};
    if constexpr (TOP) {
        block_top<N>(
            sh, a.top, mine, s != s, [&](int i) { return x[i]; },
            [&](int i) {
                const int ix = first + ((i / P) * NT + tid) * P + i % P;
                return ix < 0 || ix >= a.vocab ? NO_INDEX : ix;
            },
            ws.value + at * a.top, ws.index + at * a.top);
    }
}

// A row's segments joined, in order.
template <int TYPE>
__global__ __launch_bounds__(NT) void logprob_join_kernel(LogprobArgs a) {
    using E = Elem<TYPE>;
    __shared__ TopShared sh;
    __shared__ float red[WAVES];
    __shared__ float out_v[LOGPROB_MAX_TOP];
    __shared__ int out_i[LOGPROB_MAX_TOP];
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 63;
    const SegWs ws = seg_ws(a.ws, a.rows, a.segments, a.top);
    const f32x4* stat = reinterpret_cast<const f32x4*>(ws.stat) + (int64_t)row * a.segments;
    // every wave joins the statistics: 64 segments at a time
    float m = NEG_INF;
    for (int g = lane; g < a.segments; g += 64) m = fmaxf(m, stat[g][0]);
    m = wave_max(m);
    const float from = m == NEG_INF ? 0.0f : m;
    float s = 0.0f, t = 0.0f;
    for (int g = lane; g < a.segments; g += 64) {
        const f32x4 q = stat[g];
        const float d = (q[0] - from) * LOG2E, f = q[0] == NEG_INF ? 0.0f : __builtin_amdgcn_exp2f(d);
        s += q[1] != q[1] ? q[1] : f * q[1];
        t += f == 0.0f ? 0.0f : f * fmaf(d, q[1], q[2]);
    }
    s = wave_sum(s);
    t = wave_sum(t);
    const bool nan = s != s, none = !nan && m == NEG_INF;
    const float l2 = __builtin_amdgcn_logf(s);
    const float lse = none ? NEG_INF : fmaf(l2, LN2, m);
    if (tid == 0) {
        const int64_t tg = a.targets[row];
        const bool has = tg >= 0 && tg < a.vocab;
        float lp = 0.0f;
        if (has) {
            const float x = E::at(a.logits + (int64_t)row * a.ld_b, (int)tg);
            lp = none ? NEG_INF : x - lse;
        }
        a.logprob[row] = lp;
        a.lse[row] = lse;
        a.entropy[row] = none ? 0.0f : (l2 - t / s) * LN2;
    }
    if (a.top == 0) return;
    const int n = a.segments * a.top;
    const float* val = ws.value + (int64_t)row * n;
    const int* idx = ws.index + (int64_t)row * n;
    // the k-th largest of the segments' own maxima bounds the k-th largest value
    const int k = a.top;
    float mine = NEG_INF;
    for (int g = tid; g < a.segments; g += NT) mine = fmaxf(mine, val[(int64_t)g * k]);
    const float kth = wave_kth(mine, k - 1);
    if (lane == 0) red[tid >> 6] = kth;
    if (tid == 0) sh.count = 0;
    __syncthreads();
    float bound = red[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) bound = fmaxf(bound, red[w]);
    if (!nan) {
        for (int i = tid; i < n; i += NT) {
            const float x = val[i];
            if (x >= bound && idx[i] != NO_INDEX) {
                const int at = atomicAdd(&sh.count, 1);
                if (at < CAND) {
                    sh.value[at] = x;
                    sh.index[at] = idx[i];
                }
            }
        }
    }
    __syncthreads();
    const int count = sh.count;
    if (!nan && count >= k && count <= CAND) {
        for (int c = tid; c < count; c += NT) {
            const float x = sh.value[c];
            const int ix = sh.index[c];
            int rank = 0;
            for (int j = 0; j < count; ++j) {
                const float y = sh.value[j];
                rank += y > x || (y == x && sh.index[j] < ix);
            }
            if (rank < k) {
                out_v[rank] = x;
                out_i[rank] = ix;
            }
        }
    } else {
        // one by one; every list is in order, so its next value is its best
        uint64_t last = ~0ull;
        for (int r = 0; r < k; ++r) {
            uint64_t best = 0;
            int bi = 0;
            for (int i = tid; i < n; i += NT) {
                const uint64_t key = idx[i] == NO_INDEX ? 0 : order_key(val[i], idx[i]);
                if (key < last && key > best) {
                    best = key;
                    bi = i;
                }
            }
            uint64_t all = best;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const uint64_t o = ((uint64_t)(uint32_t)__shfl_xor((int)(all >> 32), d) << 32) |
                                   (uint32_t)__shfl_xor((int)(uint32_t)all, d);
                all = o > all ? o : all;
            }
            if (lane == 0) sh.best[tid >> 6] = all;
            __syncthreads();
            all = sh.best[0];
#pragma unroll
            for (int w = 1; w < WAVES; ++w) all = sh.best[w] > all ? sh.best[w] : all;
            if (best == all && all != 0) {
                out_v[r] = val[bi];
                out_i[r] = idx[bi];
            }
            last = all;
            __syncthreads();
        }
    }
    __syncthreads();
    if (tid < k) {
        a.top_logprob[(int64_t)row * k + tid] = nan ? __builtin_nanf("") : none ? NEG_INF : out_v[tid] - lse;
        a.top_index[(int64_t)row * k + tid] = out_i[tid];
    }
}

// The gradient, piece by piece.  Rows run from the last to the first: the
// logits that a forward pass has read last are the ones that the cache still
// holds.
template <int TYPE, int C>
__global__ __launch_bounds__(NT) void logprob_grad_kernel(LogprobArgs a) {
    using E = Elem<TYPE>;
    constexpr int P = E::PER16, N = C * P;
    const int tid = threadIdx.x;
    const int row = a.rows - 1 - (int)(blockIdx.x / a.segments), seg = blockIdx.x % a.segments;
    const char* base = a.logits + (int64_t)row * a.ld_b;
    char* grad = a.grad + (int64_t)row * a.ld_grad_b;
    const int skip = (int)((uintptr_t)base & 15) / E::BYTES;
    const bool same = (((uintptr_t)base ^ (uintptr_t)grad) & 15) == 0;
    const char* aligned = base - skip * E::BYTES;
    const int first = seg * (NT * N) - skip;
    u32x4 v[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int i = first + (c * NT + tid) * P;
        v[c] = u32x4{0, 0, 0, 0};
        if (i + P > 0 && i < a.vocab)
            v[c] = *reinterpret_cast<const u32x4*>(aligned + ((int64_t)seg * (NT * C) + c * NT + tid) * 16);
    }
    const int64_t tg = a.targets[row];
    const bool has = tg >= 0 && tg < a.vocab;
    const int target = has ? (int)tg : -1;
    const float gl = has && a.g_logprob ? a.g_logprob[row] : 0.0f;
    const float ge = a.g_entropy ? a.g_entropy[row] : 0.0f;
    const float lse = a.lse[row];
    const bool none = lse == NEG_INF;        // no token is possible: no gradient
    const float shift = none ? 0.0f : lse;
    const float c0 = -gl - ge * a.entropy[row];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int i = first + (c * NT + tid) * P;
        if (i + P <= 0 || i >= a.vocab) continue;
        float d[P];
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const float z = fmaxf(E::get(v[c], j) - shift, -1e30f);       // log p, finite where p = 0
            const float p = __builtin_amdgcn_exp2f(z * LOG2E);
            float g = p * fmaf(-ge, z, c0);
            if (i + j == target) g += gl;
            d[j] = none ? 0.0f : g;
        }
        if (same && i >= 0 && i + P <= a.vocab) {
            *reinterpret_cast<u32x4*>(grad + (int64_t)i * E::BYTES) = E::pack(d);
        } else {
#pragma unroll
            for (int j = 0; j < P; ++j)
                if (i + j >= 0 && i + j < a.vocab) E::put(grad, i + j, d[j]);
        }
    }
}

// 16-byte pieces a thread: 4 where that still gives every CU several
// workgroups, else 1.
int pieces(int type, int64_t rows, int64_t vocab) {
    const int per16 = type == DT_F32 ? 4 : 8;
    return rows * vocab >= (int64_t)1024 * NT * per16 * 4 ? 4 : 1;
}

template <int TYPE, int C>
hipError_t forward_as(const LogprobArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)((int64_t)a.rows * a.segments));
    if (a.top > 0) {
        hipLaunchKernelGGL((logprob_segment_kernel<TYPE, C, true>), grid, dim3(NT), 0, stream, a);
    } else {
        hipLaunchKernelGGL((logprob_segment_kernel<TYPE, C, false>), grid, dim3(NT), 0, stream, a);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(logprob_join_kernel<TYPE>, dim3((unsigned)a.rows), dim3(NT), 0, stream, a);
    return hipGetLastError();
}

template <int TYPE, int C>
hipError_t backward_as(const LogprobArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL((logprob_grad_kernel<TYPE, C>), dim3((unsigned)((int64_t)a.rows * a.segments)), dim3(NT), 0,
                       stream, a);
    return hipGetLastError();
}

template <int TYPE>
hipError_t forward(const LogprobArgs& a, hipStream_t stream) {
    return pieces(TYPE, a.rows, a.vocab) == 4 ? forward_as<TYPE, 4>(a, stream) : forward_as<TYPE, 1>(a, stream);
}
template <int TYPE>
hipError_t backward(const LogprobArgs& a, hipStream_t stream) {
    return pieces(TYPE, a.rows, a.vocab) == 4 ? backward_as<TYPE, 4>(a, stream) : backward_as<TYPE, 1>(a, stream);
}

}  // namespace

// Segments of a row; a row that does not start on a 16-byte boundary may
// reach one piece further.
int logprob_segments(int type, int64_t rows, int64_t vocab) {
    const int64_t per16 = type == DT_F32 ? 4 : 8, seg = NT * per16 * pieces(type, rows, vocab);
    return (int)((vocab + per16 - 1 + seg - 1) / seg);
}

int64_t logprob_workspace(int type, int64_t rows, int64_t vocab, int top) {
    return rows * logprob_segments(type, rows, vocab) * (16 + 8 * (int64_t)top);
}

hipError_t launch_token_logprobs(const LogprobArgs& a, hipStream_t stream) {
    switch (a.type) {
        case DT_F32: return forward<DT_F32>(a, stream);
        case DT_BF16: return forward<DT_BF16>(a, stream);
        default: return forward<DT_F16>(a, stream);
    }
}

hipError_t launch_token_logprobs_backward(const LogprobArgs& a, hipStream_t stream) {
    switch (a.type) {
        case DT_F32: return backward<DT_F32>(a, stream);
        case DT_BF16: return backward<DT_BF16>(a, stream);
        default: return backward<DT_F16>(a, stream);
    }
}

}  // namespace mpdt
