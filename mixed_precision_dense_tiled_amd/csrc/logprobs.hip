// logprobs.hip -- log probabilities of given tokens, entropy, the most likely
// alternatives, and the gradient.
//
// For a row x of logits and its target t:
//     lse = log sum_j exp(x_j),  logprob = x_t - lse,  p_j = exp(x_j - lse),
//     entropy H = -sum_j p_j log p_j = lse - sum_j p_j x_j,
// and with gradients gl (of logprob) and ge (of entropy)
//     dx_j = gl * ([j = t] - p_j) - ge * p_j * (log p_j + H).
//
// A workgroup walks a segment of a row in chunks that it holds in registers,
// the next chunk's loads in flight.  Each thread keeps a running maximum m,
// sum e^(x-m) and sum e^(x-m)(x-m) of its own; they are joined once at the end.
// Where there are enough rows a segment is a whole row and the workgroup writes
// the results itself; else a second launch joins a row's segments in order.
// Bound by the bytes of the logits; the arithmetic (an exponential and seven
// FP32 operations a value) lies close below in 16-bit types.
//
// The largest values: the k-th largest of a wave's 64 lane maxima cannot be
// larger than the k-th largest value, so of the first chunk only values at or
// above the best such bound are gathered; each counts how many beat it (larger,
// or equal at a lower index), and the k-th largest becomes the bound of the
// chunks that follow.  Where too many tie, or a value is no number, k passes
// over the registers find a chunk's largest one by one.
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
constexpr int CAND = 1024;            // room for gathered values
constexpr int PRUNE = 192;            // more of them are cut to the k largest

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

// A wave's maximum and sum by DPP (rows of 16 lanes, then across them): the
// last lane's value, to all.
template <int CTRL>
__device__ __forceinline__ float dpp(float old, float v) {
    return __int_as_float(
        __builtin_amdgcn_update_dpp(__float_as_int(old), __float_as_int(v), CTRL, 0xf, 0xf, false));
}
__device__ __forceinline__ float last_lane(float v) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ float wave_max(float v) {
    v = fmaxf(v, dpp<0x111>(v, v));     // row_shr 1, 2, 4, 8
    v = fmaxf(v, dpp<0x112>(v, v));
    v = fmaxf(v, dpp<0x114>(v, v));
    v = fmaxf(v, dpp<0x118>(v, v));
    v = fmaxf(v, dpp<0x142>(v, v));     // row_bcast 15, 31
    v = fmaxf(v, dpp<0x143>(v, v));
    return last_lane(v);
}
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp<0x111>(0.0f, v);
    v += dpp<0x112>(0.0f, v);
    v += dpp<0x114>(0.0f, v);
    v += dpp<0x118>(0.0f, v);
    v += dpp<0x142>(0.0f, v);
    v += dpp<0x143>(0.0f, v);
    return last_lane(v);
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
    int odd;             // a value is no number
};

// The best such bound over the workgroup's values.  mine: this thread's
// largest.  All threads call it.
__device__ __forceinline__ float top_bound(TopShared& sh, int k, float mine) {
    const float kth = wave_kth(mine, k - 1);
    if ((threadIdx.x & 63) == 0) sh.bound[threadIdx.x >> 6] = kth;
    __syncthreads();
    float bound = sh.bound[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) bound = fmaxf(bound, sh.bound[w]);
    return bound;
}

__device__ __forceinline__ void top_gather(TopShared& sh, float x, int index) {
    const int at = atomicAdd(&sh.count, 1);
    if (at < CAND) {
        sh.value[at] = x;
        sh.index[at] = index;
    }
}

// The k best of the `count` gathered values to the front of the list, in
// order.  (Gathered in any order: the result is the same.)  All threads call it.
__device__ __forceinline__ void top_sort(TopShared& sh, int k, int count) {
    constexpr int EACH = CAND / NT;
    float x[EACH];
    int ix[EACH], rank[EACH];
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
        const int c = threadIdx.x + e * NT;
        rank[e] = k;
        if (c >= count) continue;
        x[e] = sh.value[c];
        ix[e] = sh.index[c];
        const uint64_t key = order_key(x[e], ix[e]);
        int r = 0;
#pragma unroll 1
        for (int j = 0; j < count; ++j) r += order_key(sh.value[j], sh.index[j]) > key;
        rank[e] = r;
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < EACH; ++e)
        if (rank[e] < k) {
            sh.value[rank[e]] = x[e];
            sh.index[rank[e]] = ix[e];
        }
    if (threadIdx.x == 0) sh.count = min(count, k);
    __syncthreads();
}

// One of k passes for the largest of the workgroup's N values a thread below
// `last`; 0 where there is none.  All threads call it.
template <class V, class I>
__device__ __forceinline__ uint64_t top_next(TopShared& sh, int n, uint64_t last, V value, I index, float& bx,
                                             int& bi, bool& mine) {
    uint64_t best = 0;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        const int ix = index(i);
        const uint64_t key = ix == NO_INDEX ? 0 : order_key(value(i), ix);
        if (key < last && key > best) {
            best = key;
            bx = value(i);
            bi = ix;
        }
    }
    uint64_t all = best;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint64_t o = ((uint64_t)(uint32_t)__shfl_xor((int)(all >> 32), d) << 32) |
                           (uint32_t)__shfl_xor((int)(uint32_t)all, d);
        all = o > all ? o : all;
    }
    if ((threadIdx.x & 63) == 0) sh.best[threadIdx.x >> 6] = all;
    __syncthreads();
    all = sh.best[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) all = sh.best[w] > all ? sh.best[w] : all;
    __syncthreads();
    mine = all != 0 && best == all;
    return all;
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

// A row's results from its maximum m, s = sum e^(x-m), t = sum of e^y y with
// y = (x - m) log2(e).
struct RowResult {
    float lse, entropy;
    bool nan, none;
};
__device__ __forceinline__ RowResult row_result(float m, float s, float t) {
    RowResult r;
    r.nan = s != s;
    r.none = !r.nan && m == NEG_INF;
    const float l2 = __builtin_amdgcn_logf(s);
    r.lse = r.none ? NEG_INF : fmaf(l2, LN2, m);
    r.entropy = r.none ? 0.0f : (l2 - t / s) * LN2;
    return r;
}
template <class E>
__device__ __forceinline__ void write_row(const LogprobArgs& a, int row, const RowResult& r) {
    const int64_t tg = a.targets[row];
    float lp = 0.0f;
    if (tg >= 0 && tg < a.vocab)
        lp = r.none ? NEG_INF : E::at(a.logits + (int64_t)row * a.ld_b, (int)tg) - r.lse;
    a.logprob[row] = lp;
    a.lse[row] = r.lse;
    a.entropy[row] = r.entropy;
}
__device__ __forceinline__ void write_top(const LogprobArgs& a, int row, const RowResult& r, const TopShared& sh) {
    if ((int)threadIdx.x < a.top) {
        const int64_t at = (int64_t)row * a.top + threadIdx.x;
        a.top_logprob[at] = r.nan ? __builtin_nanf("") : r.none ? NEG_INF : sh.value[threadIdx.x] - r.lse;
        a.top_index[at] = sh.index[threadIdx.x];
    }
}

// C: 16-byte pieces a thread and chunk.  Pieces are read on 16-byte boundaries
// of memory whatever the row's alignment (a piece that holds a value of the
// row lies in mapped memory); elements before and past the row count as -inf.
template <int TYPE, int C, bool TOP>
__global__ __launch_bounds__(NT) void logprob_segment_kernel(LogprobArgs a) {
    using E = Elem<TYPE>;
    constexpr int P = E::PER16, N = C * P;
    __shared__ TopShared sh;
    __shared__ float red[3][WAVES];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, k = a.top;
    const int row = blockIdx.x / a.segments, seg = blockIdx.x % a.segments;
    const char* base = a.logits + (int64_t)row * a.ld_b;
    const int skip = (int)((uintptr_t)base & 15) / E::BYTES;
    const char* aligned = base - skip * E::BYTES;
    const int chunk0 = seg * a.chunks, chunk1 = min(chunk0 + a.chunks, (a.vocab + skip + NT * N - 1) / (NT * N));
    auto first_of = [&](int chunk) { return chunk * (NT * N) - skip; };      // index of a chunk's first element
    auto fetch = [&](int chunk, u32x4 (&v)[C]) {
        const int first = first_of(chunk);
        const bool inner = first >= 0 && first + NT * N <= a.vocab;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = first + (c * NT + tid) * P;
            if (inner || (i + P > 0 && i < a.vocab))
                v[c] = *reinterpret_cast<const u32x4*>(aligned + ((int64_t)chunk * (NT * C) + c * NT + tid) * 16);
        }
    };
    float m = NEG_INF, s = 0.0f, t = 0.0f, bound = NEG_INF;
    int kept = 0;        // gathered values of the chunks so far
    if constexpr (TOP) {
        if (tid == 0) sh.count = sh.odd = 0;
    }
    u32x4 v[C];
#pragma unroll
    for (int c = 0; c < C; ++c) v[c] = u32x4{0, 0, 0, 0};
    if (chunk0 < chunk1) fetch(chunk0, v);
    for (int chunk = chunk0; chunk < chunk1; ++chunk) {
        const int first = first_of(chunk);
        float x[N];
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < P; ++j) x[c * P + j] = E::get(v[c], j);
        if (chunk + 1 < chunk1) fetch(chunk + 1, v);
        if (first < 0 || first + NT * N > a.vocab) {
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
        // y = (x - m) log2(e), the difference first: a mask of the type's lowest
        // value would leave the range times log2(e).  Nothing but -inf so far: m
        // counts as 0.
        const float to = fmaxf(m, mine), from = to == NEG_INF ? 0.0f : to;
        const float d = fmaxf((m - from) * LOG2E, -1e30f), f = __builtin_amdgcn_exp2f(d);
        t = f * fmaf(d, s, t);
        s *= f;
        m = to;
        float s1 = 0.0f, t1 = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float y = (x[i] - from) * LOG2E;
            const float e = __builtin_amdgcn_exp2f(y);                 // no number where x is none, or +inf
            s1 += e;
            t1 = fmaf(e, fmaxf(y, -1e30f), t1);                        // e = 0 times a finite y where x = -inf
        }
        s += s1;
        t += t1;
        if constexpr (TOP) {
            if (chunk == chunk0) bound = top_bound(sh, k, mine);
            if (s1 != s1) sh.odd = 1;
            if (mine >= bound) {
                // (few threads after the first chunk; read again, as the values'
                // registers are worth more to the loop above)
#pragma unroll 1
                for (int c = 0; c < C; ++c) {
                    const int i = first + (c * NT + tid) * P;
                    if (i + P <= 0 || i >= a.vocab) continue;
                    const u32x4 w = *reinterpret_cast<const u32x4*>(
                        aligned + ((int64_t)chunk * (NT * C) + c * NT + tid) * 16);
#pragma unroll
                    for (int j = 0; j < P; ++j)
                        if (E::get(w, j) >= bound && i + j >= 0 && i + j < a.vocab) top_gather(sh, E::get(w, j), i + j);
                }
            }
            __syncthreads();
            const int count = sh.count, odd = sh.odd;
            __syncthreads();
            if (odd || count > CAND) {
                // one by one, in the place of what this chunk has gathered (read
                // again: the rare path takes no registers from the others)
                const int c0 = max(first, 0) + tid, c1 = min(first + NT * N, a.vocab);
                uint64_t last = ~0ull;
                int at = kept;
#pragma unroll 1
                for (int r = 0; r < k; ++r) {
                    float bx = 0.0f;
                    int bi = 0;
                    bool mine_it = false;
                    const uint64_t all =
                        top_next(sh, (c1 - c0 + NT - 1) / NT, last, [&](int i) { return E::at(base, c0 + i * NT); },
                                 [&](int i) { return c0 + i * NT; }, bx, bi, mine_it);
                    if (all == 0) break;
                    if (mine_it) {
                        sh.value[at] = bx;
                        sh.index[at] = bi;
                    }
                    ++at;
                    last = all;
                }
                if (tid == 0) {
                    sh.count = at;
                    sh.odd = 0;
                }
                kept = at;
                __syncthreads();
            } else {
                kept = count;
            }
            if (kept > (chunk == chunk0 ? k : PRUNE)) {
                top_sort(sh, k, kept);
                kept = k;
                const float kth = sh.value[k - 1];
                bound = kth == kth ? kth : bound;
            }
        }
    }
    // the threads' running sums joined
    const float wm = wave_max(m);
    if (lane == 0) red[0][wave] = wm;
    __syncthreads();
    float all = red[0][0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) all = fmaxf(all, red[0][w]);
    const float from = all == NEG_INF ? 0.0f : all;
    const float d = fmaxf((m - from) * LOG2E, -1e30f), f = __builtin_amdgcn_exp2f(d);
    t = wave_sum(f * fmaf(d, s, t));
    s = wave_sum(f * s);
    if (lane == 0) {
        red[1][wave] = s;
        red[2][wave] = t;
    }
    if constexpr (TOP) top_sort(sh, k, kept);
    __syncthreads();
    s = red[1][0];
    t = red[2][0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) {
        s += red[1][w];
        t += red[2][w];
    }
    if (a.segments == 1) {
        const RowResult r = row_result(all, s, t);
        if (tid == 0) write_row<E>(a, row, r);
        if constexpr (TOP) write_top(a, row, r, sh);
        return;
    }
    const SegWs ws = seg_ws(a.ws, a.rows, a.segments, k);
    const int64_t at = (int64_t)row * a.segments + seg;
    if (tid == 0) *reinterpret_cast<f32x4*>(ws.stat + at * 4) = f32x4{all, s, t, 0.0f};
    if constexpr (TOP) {
        const int have = sh.count;
        if (tid < k) {
            ws.value[at * k + tid] = tid < have ? sh.value[tid] : NEG_INF;
            ws.index[at * k + tid] = tid < have ? sh.index[tid] : NO_INDEX;
        }
    }
}

// A row's segments joined, in order.
template <int TYPE>
__global__ __launch_bounds__(NT) void logprob_join_kernel(LogprobArgs a) {
    using E = Elem<TYPE>;
    __shared__ TopShared sh;
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 63, k = a.top;
    const SegWs ws = seg_ws(a.ws, a.rows, a.segments, k);
    const f32x4* stat = reinterpret_cast<const f32x4*>(ws.stat) + (int64_t)row * a.segments;
    const int n = a.segments * k;
    const float* val = ws.value + (int64_t)row * n;
    const int* idx = ws.index + (int64_t)row * n;
    if (tid == 0) sh.count = 0;
    // every wave joins the statistics: 64 segments at a time
    float m = NEG_INF;
    for (int g = lane; g < a.segments; g += 64) m = fmaxf(m, stat[g][0]);
    m = wave_max(m);
    const float from = m == NEG_INF ? 0.0f : m;
    float s = 0.0f, t = 0.0f;
    for (int g = lane; g < a.segments; g += 64) {
        const f32x4 q = stat[g];
        const float d = fmaxf((q[0] - from) * LOG2E, -1e30f), f = __builtin_amdgcn_exp2f(d);
        s += f * q[1];
        t += f * fmaf(d, q[1], q[2]);
    }
    s = wave_sum(s);
    t = wave_sum(t);
    const RowResult r = row_result(m, s, t);
    if (tid == 0) write_row<E>(a, row, r);
    if (k == 0) return;
    // the k-th largest of the segments' own maxima bounds the k-th largest value
    float mine = NEG_INF;
    for (int g = tid; g < a.segments; g += NT) mine = fmaxf(mine, val[(int64_t)g * k]);
    const float bound = top_bound(sh, k, mine);
    if (!r.nan) {
        for (int i = tid; i < n; i += NT) {
            const float x = val[i];
            const int ix = idx[i];
            if (x >= bound && ix != NO_INDEX) top_gather(sh, x, ix);
        }
    }
    __syncthreads();
    const int count = sh.count;
    __syncthreads();
    if (!r.nan && count <= CAND) {
        top_sort(sh, k, count);
    } else {
        uint64_t last = ~0ull;
        for (int i = 0; i < k; ++i) {
            float bx = 0.0f;
            int bi = 0;
            bool mine_it = false;
            last = top_next(sh, (n - tid + NT - 1) / NT, last, [&](int e) { return val[tid + e * NT]; },
                            [&](int e) { return idx[tid + e * NT]; }, bx, bi, mine_it);
            if (mine_it) {
                sh.value[i] = bx;
                sh.index[i] = bi;
            }
        }
        __syncthreads();
    }
    write_top(a, row, r, sh);
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

// Pieces of 16 bytes a thread and chunk, chunks of a row, and how many
// workgroups share a row in the forward pass: with 256 workgroups or more at
// work a whole row each saves the second launch; below, a row is cut so that
// about 256 run.
struct Cut {
    int pieces, chunks, segments, per_segment;
};
Cut cut_of(int type, int64_t rows, int64_t vocab) {
    const int64_t per16 = type == DT_F32 ? 4 : 8;
    Cut c;
    c.pieces = rows * vocab >= (int64_t)256 * NT * per16 * 4 ? 4 : 1;
    const int64_t len = NT * per16 * c.pieces;
    c.chunks = (int)((vocab + per16 - 1 + len - 1) / len);     // (a row off 16 bytes may reach one piece further)
    const int64_t want = std::max<int64_t>(1, 256 / rows);
    c.per_segment = (int)((c.chunks + want - 1) / want);
    c.segments = (c.chunks + c.per_segment - 1) / c.per_segment;
    return c;
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
    if (e != hipSuccess || a.segments == 1) return e;
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
hipError_t forward(LogprobArgs a, hipStream_t stream) {
    const Cut c = cut_of(TYPE, a.rows, a.vocab);
    a.segments = c.segments;
    a.chunks = c.per_segment;
    return c.pieces == 4 ? forward_as<TYPE, 4>(a, stream) : forward_as<TYPE, 1>(a, stream);
}
template <int TYPE>
hipError_t backward(LogprobArgs a, hipStream_t stream) {
    const Cut c = cut_of(TYPE, a.rows, a.vocab);
    a.segments = c.chunks;
    return c.pieces == 4 ? backward_as<TYPE, 4>(a, stream) : backward_as<TYPE, 1>(a, stream);
}

}  // namespace

bool logprob_fits(int type, int64_t rows, int64_t vocab) {
    return rows * cut_of(type, rows, vocab).chunks <= 0x7fffffff;
}

int64_t logprob_workspace(int type, int64_t rows, int64_t vocab, int top) {
    const Cut c = rows > 0 ? cut_of(type, rows, vocab) : Cut{};
    return c.segments > 1 ? rows * c.segments * (16 + 8 * (int64_t)top) : 0;
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
