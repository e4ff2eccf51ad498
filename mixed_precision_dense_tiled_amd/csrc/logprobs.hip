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
// FP32 operations a value) lies close below in 16-bit types.  2048 x 131072 BF16
// (537 MB): 103 us without alternatives (5.2 TB/s), 136 with the 5 largest, 152
// with 20.
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

// Maxima that pass a NaN over, without the extra operation that makes a
// signalling one quiet first (fmaxf's).
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}
__device__ __forceinline__ float max2(float a, float b) {
    float r;
    asm("v_max_f32 %0, %1, %2" : "=v"(r) : "s"(b), "v"(a));
    return r;
}

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

// The 64 lanes' values, largest first: a bitonic sort.
__device__ __forceinline__ float lane_xor(float v, int lane, int d) {
    return __int_as_float(__builtin_amdgcn_ds_bpermute((lane ^ d) << 2, __float_as_int(v)));
}
__device__ __forceinline__ float wave_sorted(float v, int lane) {
#pragma unroll
    for (int size = 2; size <= 64; size <<= 1) {
#pragma unroll
        for (int d = size >> 1; d > 0; d >>= 1) {
            const float o = lane_xor(v, lane, d);
            const bool low = (lane & d) == 0, down = (lane & size) == 0 || size == 64;
            v = low == down ? fmaxf(v, o) : fminf(v, o);
        }
    }
    return v;
}

// Order of (value, index): larger first, NaN above all, then the lower index.  No
// key is ~0, which stands above all of them where the largest is looked for.
constexpr uint32_t NAN_KEY = 0xfffffffeu;
__device__ __forceinline__ uint64_t order_key(float x, int index) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    const uint32_t k = x != x ? NAN_KEY : (b >> 31) ? ~b : b | 0x80000000u;
    return ((uint64_t)k << 32) | (uint32_t)~index;
}

__device__ __forceinline__ int key_index(uint64_t key) { return (int)~(uint32_t)key; }
__device__ __forceinline__ float key_value(uint64_t key) {
    const uint32_t k = (uint32_t)(key >> 32);
    return k == NAN_KEY ? __builtin_nanf("") : __uint_as_float((k >> 31) ? k ^ 0x80000000u : ~k);
}

struct TopShared {
    float bound[2][WAVES];
    uint64_t key[CAND];  // gathered values, as order keys
    uint64_t best[WAVES];
    int count;
    int fresh[4];        // values gathered from a group of chunks, in turn: one barrier a group
};
constexpr int ODD = 1 << 20;          // added to them where a value is no number

// A bound that at least k of the workgroup's values reach: the best wave's
// k-th largest lane maximum, or where it is larger the smallest of the waves'
// k/4-th.  mine: this thread's largest.  All threads call it (and the functions
// below; their tid is opaque in the loop over chunks, see there).
__device__ __forceinline__ float top_bound(TopShared& sh, int tid, int k, float mine) {
    const float v = wave_sorted(mine, tid & 63);
    const float whole = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), k - 1));
    const float part = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), (k - 1) / WAVES));
    if ((tid & 63) == 0) {
        sh.bound[0][tid >> 6] = whole;
        sh.bound[1][tid >> 6] = part;
    }
    __syncthreads();
    float best = sh.bound[0][0], least = sh.bound[1][0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) {
        best = fmaxf(best, sh.bound[0][w]);
        least = fminf(least, sh.bound[1][w]);
    }
    return fmaxf(best, least);
}

__device__ __forceinline__ void top_gather(TopShared& sh, int kept, int* counter, float x, int index) {
    const int at = kept + (atomicAdd(counter, 1) & (ODD - 1));
    if (at < CAND) sh.key[at] = order_key(x, index);
}

// The k best of the `count` gathered values to the front of the list, in
// order.  (Gathered in any order: the result is the same.)  All threads call it.
__device__ __forceinline__ void top_sort(TopShared& sh, int tid, int k, int count) {
    constexpr int EACH = CAND / NT;
    uint64_t key[EACH];
    int rank[EACH];
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
        const int c = tid + e * NT;
        rank[e] = k;
        if (c >= count) continue;
        key[e] = sh.key[c];
        int r = 0;
#pragma unroll 8
        for (int j = 0; j < count; ++j) r += sh.key[j] > key[e];
        rank[e] = r;
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < EACH; ++e)
        if (rank[e] < k) sh.key[rank[e]] = key[e];
    if (tid == 0) sh.count = min(count, k);
    __syncthreads();
}

// One of k passes: the largest of the workgroup's keys below `last`, n a
// thread; 0 where there is none.  All threads call it.
template <class K>
__device__ __forceinline__ uint64_t top_next(TopShared& sh, int tid, int n, uint64_t last, K key) {
    uint64_t all = 0;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        const uint64_t x = key(i);
        if (x < last && x > all) all = x;
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int from = ((tid & 63) ^ d) << 2;
        const uint64_t o = ((uint64_t)(uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)(all >> 32)) << 32) |
                           (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)(uint32_t)all);
        all = o > all ? o : all;
    }
    if ((tid & 63) == 0) sh.best[tid >> 6] = all;
    __syncthreads();
    all = sh.best[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) all = sh.best[w] > all ? sh.best[w] : all;
    __syncthreads();
    return all;
}

// Per segment in the workspace: maximum, sum, weighted sum, then the keys of its
// `top` largest values (0: fewer).
struct SegWs {
    float* stat;    // [rows][segments][4]
    uint64_t* key;  // [rows][segments][top]
};
__host__ __device__ inline SegWs seg_ws(char* ws, int64_t rows, int64_t segments) {
    SegWs w;
    w.stat = (float*)ws;
    w.key = (uint64_t*)(ws + rows * segments * 16);
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
        const uint64_t key = sh.key[threadIdx.x];
        a.top_logprob[at] = r.nan ? __builtin_nanf("") : r.none ? NEG_INF : key_value(key) - r.lse;
        a.top_index[at] = key_index(key);
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
    // (always from the row's own pieces, without a condition: loads under one
    // would wait for each other)
    const int last_piece = (a.vocab + skip - 1) / P;
    auto fetch = [&](int chunk, u32x4 (&v)[C]) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int piece = min(chunk * (NT * C) + c * NT + tid, last_piece);
            v[c] = *reinterpret_cast<const u32x4*>(aligned + (int64_t)piece * 16);
        }
    };
    float m = NEG_INF, s = 0.0f, t = 0.0f, bound = NEG_INF;
    int kept = 0, before = 0, group = chunk0;    // gathered values, those of the groups before; this group's chunk
    if constexpr (TOP) {
        if (tid < 4) sh.fresh[tid] = 0;
        if (tid == 0) sh.count = 0;
    }
    u32x4 v[C];
    fetch(chunk0, v);
    for (int chunk = chunk0; chunk < chunk1; ++chunk) {
        const int first = first_of(chunk);
        float x[N];
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < P; ++j) x[c * P + j] = E::get(v[c], j);
        fetch(min(chunk + 1, chunk1 - 1), v);
        if (first < 0 || first + NT * N > a.vocab) {
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const int i = first + (c * NT + tid) * P + j;
                    if (i < 0 || i >= a.vocab) x[c * P + j] = NEG_INF;
                }
        }
        float mine = max3(x[0], x[1], x[2]);
#pragma unroll
        for (int i = 3; i < N; i += 2) mine = max3(mine, x[i], x[i + 1 < N ? i + 1 : i]);
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
            t1 = fmaf(e, max2(y, -1e30f), t1);                        // e = 0 times a finite y where x = -inf
            // eight at a time, and here: all exponentials at once, next to the
            // first use of their sums, would hold twice the registers
            if (i % 8 == 7) asm volatile("" : "+v"(s1), "+v"(t1));
        }
        s += s1;
        t += t1;
        if constexpr (TOP) {
            // (opaque: what follows from it is worked out anew each time, where
            // kept across the loop it would cost registers and with them waves)
            int tid = threadIdx.x;
            asm volatile("" : "+v"(tid));
            // The first chunk is a group, then four at a time; groups count in turn.
            const int since = chunk - chunk0, turn = ((since + 3) >> 2) & 3;
            if (since == 0) bound = top_bound(sh, tid, k, mine);
            if (s1 != s1) atomicAdd(&sh.fresh[turn], ODD);
            if (mine >= bound) {
                // (few threads after the first chunk; read again, as the values'
                // registers are worth more to the loop above)
                u32x4 w[C];
#pragma unroll
                for (int c = 0; c < C; ++c)
                    w[c] = *reinterpret_cast<const u32x4*>(
                        aligned + (int64_t)min(chunk * (NT * C) + c * NT + tid, last_piece) * 16);
#pragma unroll 1
                for (int c = 0; c < C; ++c) {
                    const int i = first + (c * NT + tid) * P;
#pragma unroll
                    for (int j = 0; j < P; ++j) {
                        const float y = E::get(w[0], j);
                        if (y >= bound && i + j >= 0 && i + j < a.vocab) top_gather(sh, kept, &sh.fresh[turn], y, i + j);
                    }
#pragma unroll
                    for (int d = 0; d + 1 < C; ++d) w[d] = w[d + 1];
                }
            }
            if ((since & 3) && chunk + 1 < chunk1) continue;
            __syncthreads();
            kept += sh.fresh[turn];
            if (tid == 0) sh.fresh[(turn + 2) & 3] = 0;
            if (kept > CAND) {
                // one by one over the group, in the place of what it has gathered
                kept = before;
                const int c0 = max(first_of(group), 0) + tid, c1 = min(first + NT * N, a.vocab);
                uint64_t last = ~0ull;
#pragma unroll 1
                for (int r = 0; r < k; ++r) {
                    last = top_next(sh, tid, (c1 - c0 + NT - 1) / NT, last,
                                    [&](int i) { return order_key(E::at(base, c0 + i * NT), c0 + i * NT); });
                    if (last == 0) break;
                    if (tid == 0) sh.key[kept] = last;
                    ++kept;
                }
                __syncthreads();
            }
            if (kept > (since == 0 ? k : PRUNE)) {
                top_sort(sh, tid, k, kept);
                kept = k;
                const float kth = key_value(sh.key[k - 1]);
                bound = kth == kth ? kth : bound;
            }
            before = kept;
            group = chunk + 1;
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
    if constexpr (TOP) top_sort(sh, tid, k, kept);
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
    const SegWs ws = seg_ws(a.ws, a.rows, a.segments);
    const int64_t at = (int64_t)row * a.segments + seg;
    if (tid == 0) *reinterpret_cast<f32x4*>(ws.stat + at * 4) = f32x4{all, s, t, 0.0f};
    if constexpr (TOP) {
        const int have = sh.count;
        if (tid < k) {
            ws.key[at * k + tid] = tid < have ? sh.key[tid] : 0;
        }
    }
}

// A row's segments joined, in order.
template <int TYPE>
__global__ __launch_bounds__(NT) void logprob_join_kernel(LogprobArgs a) {
    using E = Elem<TYPE>;
    __shared__ TopShared sh;
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 63, k = a.top;
    const SegWs ws = seg_ws(a.ws, a.rows, a.segments);
    const f32x4* stat = reinterpret_cast<const f32x4*>(ws.stat) + (int64_t)row * a.segments;
    const int n = a.segments * k;
    const uint64_t* keys = ws.key + (int64_t)row * n;
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
    uint64_t first = 0;
    for (int g = tid; g < a.segments; g += NT) {
        const uint64_t x = keys[(int64_t)g * k];
        first = x > first ? x : first;
    }
    const float bound = top_bound(sh, tid, k, first ? key_value(first) : NEG_INF);
    if (!r.nan) {
        for (int i = tid; i < n; i += NT) {
            const uint64_t x = keys[i];
            if (x && key_value(x) >= bound) {
                const int at = atomicAdd(&sh.count, 1);
                if (at < CAND) sh.key[at] = x;
            }
        }
    }
    __syncthreads();
    const int count = sh.count;
    __syncthreads();
    if (!r.nan && count <= CAND) {
        top_sort(sh, tid, k, count);
    } else {
        uint64_t last = ~0ull;
        for (int i = 0; i < k; ++i) {
            last = top_next(sh, tid, (n - tid + NT - 1) / NT, last, [&](int e) { return keys[tid + e * NT]; });
            if (tid == 0) sh.key[i] = last;
        }
        __syncthreads();
    }
    write_top(a, row, r, sh);
}

template <bool FAR>
__device__ __forceinline__ u32x4 load_piece(const char* p) {
    if constexpr (FAR) return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
    return *reinterpret_cast<const u32x4*>(p);
}

// The gradient, piece by piece, written past the caches (2048 x 131072 BF16:
// forward and backward 346 -> 329 us, 777 x 50021 FP32: 103 -> 84: what the
// forward pass read stays).  FAR: more logits than the 256 MB Infinity Cache
// holds, so they are read past it too (304 us; the smaller ones 87 us that way).
template <int TYPE, int C, bool FAR>
__global__ __launch_bounds__(NT) void logprob_grad_kernel(LogprobArgs a) {
    using E = Elem<TYPE>;
    constexpr int P = E::PER16, N = C * P;
    const int tid = threadIdx.x;
    const int row = (int)(blockIdx.x / a.segments), seg = blockIdx.x % a.segments;
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
            v[c] = load_piece<FAR>(aligned + ((int64_t)seg * (NT * C) + c * NT + tid) * 16);
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
            // log p, finite where p = 0 (at -1e4 it is, and a factor of up to 1e34 leaves
            // the product finite)
            const float z = fmaxf(E::get(v[c], j) - shift, -1e4f);
            const float p = __builtin_amdgcn_exp2f(z * LOG2E);
            float g = p * fmaf(-ge, z, c0);
            if (i + j == target) g += gl;
            d[j] = none ? 0.0f : g;
        }
        if (same && i >= 0 && i + P <= a.vocab) {
            __builtin_nontemporal_store(E::pack(d), reinterpret_cast<u32x4*>(grad + (int64_t)i * E::BYTES));
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
    const dim3 grid((unsigned)((int64_t)a.rows * a.segments));
    if (a.rows * (int64_t)a.vocab * Elem<TYPE>::BYTES > ((int64_t)256 << 20)) {
        hipLaunchKernelGGL((logprob_grad_kernel<TYPE, C, true>), grid, dim3(NT), 0, stream, a);
    } else {
        hipLaunchKernelGGL((logprob_grad_kernel<TYPE, C, false>), grid, dim3(NT), 0, stream, a);
    }
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
    return rows * cut_of(type, rows, vocab).chunks <= MAX_GROUPS;
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
