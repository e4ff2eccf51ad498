// rms_norm.hip -- root-mean-square norm of rows, with the residual's addition and
// an output in the rows' type, in INT8 or in E4M3 with scales; and its gradient.
//
//   h = x + residual,  rstd = 1 / sqrt(mean h^2 + eps),  y = (h * rstd) * w
//
// Bound by the bytes that it moves: each row is read once, kept in registers (a
// thread holds PIECES pieces of 8 neighbouring elements), reduced once for rstd
// and once for a scale a row, and written once.  The squares are added in FP64:
// a square of a 24-bit number is exact there and the sum's order does not show in
// rstd, so that a code next to a border between two codes does not depend on how
// many threads share a row.  Two FP64 operations an element cost a tenth of the time
// in which the bytes move.
//
// 8192 x 7168 BF16 with a residual into E4M3 blocks: 80 us, 5.1 TB/s, what a large copy
// reaches; without the residual 60 us, bound by the codes' arithmetic (39.5 us without
// codes; both with rows that the last cache holds), into E4M3 rows 54, into INT8 rows 58.  Rows
// of 128 columns fill a quarter of their waves: 262144 of them 91 us, 1.5 TB/s.  Gradient of 3001 x
// 5120 FP16: 27 us and 4 for the columns' sums.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"
#include "layer_sizes.hpp"
#include "layers.hpp"
#include "quotient.hpp"

namespace mpdt {
namespace {

// Loads and stores of 8 elements from any element-aligned address.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));

// 8 elements of a row as they are stored: 4 or 8 registers.
template <int T> struct Piece {
    static constexpr int ES = T == DT_F32 ? 4 : 2;
    static constexpr int W = 2 * ES;
    uint32_t w[W];

    // n elements of 8, the rest 0; PAST the caches, where nobody reads them again
    template <bool PAST = false>
    __device__ __forceinline__ void load(const char* p, int n) {
        if (n >= 8) {
#pragma unroll
            for (int i = 0; i < W / 4; ++i) {
                const u32x4_any* const from = reinterpret_cast<const u32x4_any*>(p + 16 * i);
                u32x4_any v;
                if constexpr (PAST) v = __builtin_nontemporal_load(from);
                else v = *from;
#pragma unroll
                for (int j = 0; j < 4; ++j) w[4 * i + j] = v[j];
            }
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) w[i] = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) {
                    if constexpr (ES == 4) w[e] = reinterpret_cast<const uint32_t*>(p)[e];
                    else w[e >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[e] << (16 * (e & 1));
                }
        }
    }
    __device__ __forceinline__ void store(char* p, int n) const {
        if (n >= 8) {
#pragma unroll
            for (int i = 0; i < W / 4; ++i)
                *reinterpret_cast<u32x4_any*>(p + 16 * i) = u32x4_any{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) {
                    if constexpr (ES == 4) reinterpret_cast<uint32_t*>(p)[e] = w[e];
                    else reinterpret_cast<uint16_t*>(p)[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
                }
        }
    }
    __device__ __forceinline__ float get(int e) const {
        if constexpr (T == DT_F32) return __uint_as_float(w[e]);
        else if constexpr (T == DT_BF16) return __uint_as_float(e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
        else return (float)__builtin_bit_cast(_Float16, (uint16_t)(w[e >> 1] >> (16 * (e & 1))));
    }
    __device__ __forceinline__ void put(int e, float x) {   // rounded once to the type
        if constexpr (T == DT_F32) {
            w[e] = __float_as_uint(x);
        } else {
            // (the FP32 value first: a product that is fused with the conversion to
            // FP16 is rounded only once)
            if constexpr (T == DT_F16) asm("" : "+v"(x));
            const uint32_t b = T == DT_BF16 ? f32_to_bf16_bits(x) : f32_to_f16_bits(x);
            w[e >> 1] = e & 1 ? (w[e >> 1] & 0xffffu) | b << 16 : (w[e >> 1] & 0xffff0000u) | b;
        }
    }
};

// The larger of two magnitudes; NaN where either is.
__device__ __forceinline__ float larger(float a, float b) { return a >= b ? a : (b == b ? (a == a ? b : a) : b); }

template <class V, class F>
__device__ __forceinline__ V over_lanes(V v, int from, F f) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1)
        if (m <= from) v = f(v, __shfl_xor(v, m, 64));
    return v;
}

// v of every thread, joined in one order whatever the threads' timing.
template <int NT, class V, class F>
__device__ __forceinline__ V over_row(V v, V* red, F f) {
    v = over_lanes(v, 32, f);
    if constexpr (NT > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int i = 1; i < NT / 64; ++i) v = f(v, red[i]);
    }
    return v;
}

// The scale of values up to amax; NaN stays.
__device__ __forceinline__ float scale_of(float amax, float qmax) {
    const float s = amax / qmax;
    return s == 0.0f ? 1.0f : s;
}
__device__ __forceinline__ float cut(float x, float most) { return x > most ? most : x < -most ? -most : x; }

// 8 values of y at a scale, as codes.
template <int QUANT>
__device__ __forceinline__ u32x2 codes_of(const float (&y)[8], float scale, float inverse) {
    constexpr float QMAX = QUANT == NORM_I8_ROWS ? 127.0f : 448.0f;
    float q[8];
    // (|y| is at most qmax scales where the scale is a usual one)
    if (divides(scale)) {
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = quotient(y[e], scale, inverse);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = y[e] / scale;
    }
    u32x2 code;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if constexpr (QUANT == NORM_I8_ROWS) {
            code[i] = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float x = cut(q[4 * i + j], QMAX);
                const int c = x == x ? (int)__builtin_rintf(x) : 0;
                code[i] |= (uint32_t)(c & 0xff) << (8 * j);
            }
        } else {
            const float* const x = q + 4 * i;
            const int p = __builtin_amdgcn_cvt_pk_fp8_f32(cut(x[0], QMAX), cut(x[1], QMAX), 0, false);
            code[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(cut(x[2], QMAX), cut(x[3], QMAX), p, true);
        }
    }
    return code;
}

// NT threads to a row (64: four rows to a workgroup of 256).  WT: the weight's type.
template <int T, int WT, int QUANT, int NT, int PIECES>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void rms_norm_kernel(NormArgs a) {
    __shared__ double red_d[NT / 64];
    __shared__ float red_f[NT / 64];
    constexpr int ROWS = NT < 256 ? 256 / NT : 1, ES = Piece<T>::ES;
    const int tid = threadIdx.x % NT;
    const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / NT;
    if (row >= a.rows) return;   // (whole waves; rows that share a workgroup share no barrier)
    const char* x = a.x + row * a.x_b;
    Piece<T> h[PIECES];
    Piece<WT> w[PIECES];
#pragma unroll
    for (int u = 0; u < PIECES; ++u) {
        const int e0 = 8 * (tid + NT * u);
        h[u].template load<true>(x + (int64_t)e0 * ES, a.dim - e0);
    }
    if (a.residual) {
        const char* r = a.residual + row * a.res_b;
        Piece<T> p[PIECES];
#pragma unroll
        for (int u = 0; u < PIECES; ++u) {
            const int e0 = 8 * (tid + NT * u);
            p[u].template load<true>(r + (int64_t)e0 * ES, a.dim - e0);
        }
#pragma unroll
        for (int u = 0; u < PIECES; ++u) {
            const int e0 = 8 * (tid + NT * u);
            w[u].load(a.weight + (int64_t)e0 * Piece<WT>::ES, a.dim - e0);
        }
#pragma unroll
        for (int u = 0; u < PIECES; ++u) {
            const int e0 = 8 * (tid + NT * u);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[u].put(e, h[u].get(e) + p[u].get(e));
            if (a.h) h[u].store(a.h + row * a.h_b + (int64_t)e0 * ES, a.dim - e0);
        }
    } else {
#pragma unroll
        for (int u = 0; u < PIECES; ++u) {
            const int e0 = 8 * (tid + NT * u);
            w[u].load(a.weight + (int64_t)e0 * Piece<WT>::ES, a.dim - e0);
        }
    }
    double sum = 0;
#pragma unroll
    for (int u = 0; u < PIECES; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const double v = h[u].get(e);
            sum = __builtin_fma(v, v, sum);
        }
    sum = over_row<NT>(sum, red_d, [](double p, double q) { return p + q; });
    const float rstd = (float)(1.0 / sqrt(sum / a.dim + a.eps));
    if (a.rstd && tid == 0) a.rstd[row] = rstd;

    // (y is worked out where it is used: kept, it would cost a third of the waves)
    auto y_of = [&](int u, float (&y)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = mul_rn(mul_rn(h[u].get(e), rstd), w[u].get(e));
    };
    // (past the row's end a piece holds 0 * rstd: an amax of 0, or NaN where rstd is, as it is in
    // the whole row then, or where rstd is infinite, and with it every y that is not NaN.  That
    // NaN is left in the scale: to keep it out took registers, and with them up to 30 % of other
    // rows' speed, 4096 x 16384 BF16 into INT8 148 us against 115.)
    auto amax_of = [](const float (&y)[8]) {
        float m = fabsf(y[0]);
#pragma unroll
        for (int e = 1; e < 8; ++e) m = larger(m, fabsf(y[e]));
        return m;
    };
    char* out = a.out + row * a.out_b;
    float scale = 1.0f, inverse = 1.0f, y[8];
    constexpr float QMAX = QUANT == NORM_I8_ROWS ? 127.0f : 448.0f;
    if constexpr (QUANT == NORM_I8_ROWS || QUANT == NORM_E4M3_ROWS) {
        y_of(0, y);
        float m = amax_of(y);
#pragma unroll
        for (int u = 1; u < PIECES; ++u) {
            y_of(u, y);
            m = larger(m, amax_of(y));
        }
        scale = scale_of(over_row<NT>(m, red_f, [](float p, float q) { return larger(p, q); }), QMAX);
        inverse = 1.0f / scale;
        if (tid == 0) a.scales[row * a.ld_scales] = scale;
    }
#pragma unroll
    for (int u = 0; u < PIECES; ++u) {
        const int e0 = 8 * (tid + NT * u), n = a.dim - e0;
        y_of(u, y);
        if constexpr (QUANT == NORM_PLAIN) {
            Piece<T> o;
#pragma unroll
            for (int e = 0; e < 8; ++e) o.put(e, y[e]);
            o.store(out + (int64_t)e0 * ES, n);
        } else {
            if constexpr (QUANT == NORM_E4M3_BLOCKS) {
                // 16 lanes hold a block of 128
                scale = scale_of(over_lanes(amax_of(y), 8, [](float p, float q) { return larger(p, q); }), QMAX);
                inverse = 1.0f / scale;
                if ((tid & 15) == 0 && n > 0) a.scales[row * a.ld_scales + e0 / 128] = scale;
            }
            const u32x2 code = codes_of<QUANT>(y, scale, inverse);
            if (n >= 8) {
                *reinterpret_cast<u32x2_any*>(out + e0) = u32x2_any{code[0], code[1]};
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < n) out[e0 + e] = (char)(code[e >> 2] >> (8 * (e & 3)));
            }
        }
    }
}

template <int T, int WT, int QUANT, int NT, int PIECES>
hipError_t launch_width(const NormArgs& a, hipStream_t stream) {
    constexpr int rows = NT < 256 ? 256 / NT : 1;
    const dim3 grid((unsigned)((a.rows + rows - 1) / rows)), block(NT < 256 ? 256 : NT);
    rms_norm_kernel<T, WT, QUANT, NT, PIECES><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

// Threads to a row and pieces of each.  Few threads with more pieces each spend less on a
// row's reductions (us: 8192 x 6144 FP16 to E4M3 blocks 45.5 by 256 threads of three, 56 of
// four, 60 by 512 of two; 8192 x 7168 60 by 256, 64 by 512).  With a row or less to a CU
// more threads have it done sooner (64 x 7168 7.3 by 256, 4.9 by 1024; with scales a row, which
// take one more reduction over all of its threads, 6.5 and 6.6: not there).
template <int T, int WT, int QUANT>
hipError_t launch_quant(const NormArgs& a, hipStream_t stream) {
    if constexpr (QUANT == NORM_PLAIN || QUANT == NORM_E4M3_BLOCKS)
        if (a.rows <= CUS && a.dim > 2048 && a.dim <= 8192)
            return a.dim <= 4096 ? launch_width<T, WT, QUANT, 512, 1>(a, stream)
                                 : launch_width<T, WT, QUANT, 1024, 1>(a, stream);
    if (a.dim <= 512) return launch_width<T, WT, QUANT, 64, 1>(a, stream);
    if (a.dim <= 1024) return launch_width<T, WT, QUANT, 64, 2>(a, stream);
    if (a.dim <= 2048) return launch_width<T, WT, QUANT, 256, 1>(a, stream);
    if (a.dim <= 4096) return launch_width<T, WT, QUANT, 256, 2>(a, stream);
    if (a.dim <= 6144) return launch_width<T, WT, QUANT, 256, 3>(a, stream);
    if (a.dim <= 8192) return launch_width<T, WT, QUANT, 256, 4>(a, stream);
    if (a.dim <= 16384) return launch_width<T, WT, QUANT, 1024, 2>(a, stream);
    return launch_width<T, WT, QUANT, 1024, 4>(a, stream);
}

template <int T, int WT>
hipError_t launch_norm(const NormArgs& a, hipStream_t stream) {
    switch (a.quant) {
        case NORM_PLAIN: return launch_quant<T, WT, NORM_PLAIN>(a, stream);
        case NORM_I8_ROWS: return launch_quant<T, WT, NORM_I8_ROWS>(a, stream);
        case NORM_E4M3_ROWS: return launch_quant<T, WT, NORM_E4M3_ROWS>(a, stream);
        default: return launch_quant<T, WT, NORM_E4M3_BLOCKS>(a, stream);
    }
}

// ---- gradient ------------------------------------------------------------------

// Each of grad_groups workgroups walks rows of its own; a second launch adds their sums.
template <int T, int WT, int NT, int PIECES>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void rms_norm_grad_kernel(NormGradArgs a) {
    __shared__ float red[2][NT / 64];
    constexpr int ES = Piece<T>::ES, ROWS = NT < 256 ? 256 / NT : 1;
    // (the next row's loads are under way while one is reduced, where registers hold both)
    constexpr bool AHEAD = NT < 1024 || (PIECES == 2 && T != DT_F32);
    // What a row's gradient takes from the row is n * mean(d * n), n = h * rstd.  BF16 and FP32
    // rows keep n: they can be so large or so small that rstd^2 leaves FP32.  The rstd of an
    // FP16 row that is not 0 lies between 2^-16 and 2^32 (or eps is so large that the row's part
    // vanishes): those rows keep h, two elements to a register, and take h * (rstd * (rstd *
    // mean(d * h))), 0 for a row of zeros (8192 x 7168 with a residual: 99 us, 115 with n kept,
    // by half the waves).
    constexpr bool RAW = T == DT_F16;
    const int tid = threadIdx.x % NT, part = threadIdx.x / NT;
    const int64_t step = (int64_t)gridDim.x * ROWS;
    float dw[PIECES][8];
#pragma unroll
    for (int u = 0; u < PIECES; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[u][e] = 0;
    Piece<T> g[PIECES], h[PIECES], r[PIECES];
    auto load_res = [&](int64_t row) {
        if (!a.grad_res) return;
#pragma unroll
        for (int u = 0; u < PIECES; ++u) {
            const int e0 = 8 * (tid + NT * u);
            r[u].load(a.grad_res + row * a.gres_b + (int64_t)e0 * ES, a.dim - e0);
        }
    };
    auto load = [&](int64_t row) {
#pragma unroll
        for (int u = 0; u < PIECES; ++u) {
            const int e0 = 8 * (tid + NT * u);
            g[u].load(a.grad + row * a.grad_b + (int64_t)e0 * ES, a.dim - e0);
            h[u].load(a.h + row * a.h_b + (int64_t)e0 * ES, a.dim - e0);
        }
        if constexpr (AHEAD) load_res(row);
    };
    int turn = 0;
    int64_t row = (int64_t)blockIdx.x * ROWS + part;
    if (AHEAD && row < a.rows) load(row);
    // (rows that share a workgroup are a wave's each and share no barrier)
    for (; row < a.rows; row += step, turn ^= 1) {
        const float rstd = a.rstd[row];
        if constexpr (!AHEAD) load(row);
        float c = 0, d[PIECES][8], x[PIECES][8];
#pragma unroll
        for (int u = 0; u < PIECES; ++u) {
            const int e0 = 8 * (tid + NT * u);
            Piece<WT> w;
            w.load(a.weight + (int64_t)e0 * Piece<WT>::ES, a.dim - e0);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = g[u].get(e);
                x[u][e] = h[u].get(e) * (RAW ? 1.0f : rstd);
                d[u][e] = v * w.get(e);
                c += d[u][e] * x[u][e];
                dw[u][e] += v * (x[u][e] * (RAW ? rstd : 1.0f));
            }
        }
        Piece<T> res[PIECES];
        if constexpr (AHEAD) {
#pragma unroll
            for (int u = 0; u < PIECES; ++u) res[u] = r[u];
            if (row + step < a.rows) load(row + step);
        }
        // (two sets of partial sums in turn: one barrier a row)
        c = over_row<NT>(c, red[turn], [](float p, float q) { return p + q; });
        c = RAW ? rstd * (rstd * (c / a.dim)) : c / a.dim;
        if constexpr (!AHEAD) load_res(row);
#pragma unroll
        for (int u = 0; u < PIECES; ++u) {
            const int e0 = 8 * (tid + NT * u);
            Piece<T> o;
            Piece<WT> w;
            if constexpr (!AHEAD) w.load(a.weight + (int64_t)e0 * Piece<WT>::ES, a.dim - e0);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // (not ahead: g and h are still held, and d and x made of them again)
                if constexpr (!AHEAD) d[u][e] = g[u].get(e) * w.get(e), x[u][e] = h[u].get(e) * (RAW ? 1.0f : rstd);
                float y = rstd * (d[u][e] - x[u][e] * c);
                if (a.grad_res) y += (AHEAD ? res[u] : r[u]).get(e);
                o.put(e, y);
            }
            o.store(a.grad_h + row * a.gh_b + (int64_t)e0 * ES, a.dim - e0);
        }
    }
    if constexpr (ROWS > 1) {
        // the waves' sums, in their order
        __shared__ float sums[ROWS - 1][NT * 8 * PIECES];
        if (part > 0)
#pragma unroll
            for (int u = 0; u < PIECES; ++u)
#pragma unroll
                for (int e = 0; e < 8; ++e) sums[part - 1][(u * 8 + e) * NT + tid] = dw[u][e];
        __syncthreads();
        if (part > 0) return;
#pragma unroll
        for (int k = 0; k < ROWS - 1; ++k)
#pragma unroll
            for (int u = 0; u < PIECES; ++u)
#pragma unroll
                for (int e = 0; e < 8; ++e) dw[u][e] += sums[k][(u * 8 + e) * NT + tid];
    }
    float* to = gridDim.x == 1 ? a.grad_weight : a.ws + (int64_t)blockIdx.x * a.dim;
#pragma unroll
    for (int u = 0; u < PIECES; ++u) {
        const int e0 = 8 * (tid + NT * u);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e0 + e < a.dim) to[e0 + e] = dw[u][e];
    }
}

// Columns' sums of the workgroups: 64 columns to a workgroup, 16 threads of four columns
// beside each other and a 64th of the rows to each such line, joined in order.
__global__ __launch_bounds__(1024) void rms_norm_grad_sum_kernel(const float* ws, int groups, int dim, float* out) {
    constexpr int LINES = 64;
    __shared__ f32x4 part[LINES][16];
    const int x = threadIdx.x & 15, y = threadIdx.x >> 4, col = blockIdx.x * 64 + 4 * x;
    const int lo = groups * y / LINES, hi = groups * (y + 1) / LINES;
    f32x4 s{0, 0, 0, 0};
    if (col + 4 <= dim) {
        typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
#pragma unroll 8
        for (int i = lo; i < hi; ++i) s += *reinterpret_cast<const f32x4_any*>(ws + (int64_t)i * dim + col);
    } else {
        for (int i = lo; i < hi; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col + e < dim) s[e] += ws[(int64_t)i * dim + col + e];
    }
    part[y][x] = s;
    __syncthreads();
    // (halves of the lines onto each other)
#pragma unroll
    for (int n = LINES / 2; n >= 1; n /= 2) {
        if (y < n) part[y][x] += part[y + n][x];
        __syncthreads();
    }
    if (threadIdx.x < 64 && blockIdx.x * 64 + threadIdx.x < (unsigned)dim)
        out[blockIdx.x * 64 + threadIdx.x] = part[0][threadIdx.x >> 2][threadIdx.x & 3];
}

template <int T, int WT>
hipError_t launch_grad(const NormGradArgs& a, int groups, hipStream_t stream) {
    const auto go = [&](auto NT, auto P) {
        constexpr int nt = decltype(NT)::value, p = decltype(P)::value;
        rms_norm_grad_kernel<T, WT, nt, p><<<dim3(groups), dim3(nt < 256 ? 256 : nt), 0, stream>>>(a);
        return hipGetLastError();
    };
    using std::integral_constant;
    if (a.dim <= 512) return go(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    if (a.dim <= 1024) return go(integral_constant<int, 64>{}, integral_constant<int, 2>{});
    if (a.dim <= 2048) return go(integral_constant<int, 256>{}, integral_constant<int, 1>{});
    if (a.dim <= 4096) return go(integral_constant<int, 512>{}, integral_constant<int, 1>{});
    // (8192 x 6144 FP16 68 us, 72 by 512 threads of two, 65 by 256 of three, which take 16.3 where 500
    // x 5120 take 13.2 so; 8192 x 7168 80 by 512 of two, 97 by 1024 of one)
    if (a.dim <= 6144) return go(integral_constant<int, 768>{}, integral_constant<int, 1>{});
    if (a.dim <= 8192) return go(integral_constant<int, 512>{}, integral_constant<int, 2>{});
    if (a.dim <= 16384) return go(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
    return go(integral_constant<int, 1024>{}, integral_constant<int, 4>{});
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t stream) {
    if (a.type == DT_F32) return launch_norm<DT_F32, DT_F32>(a, stream);
    if (a.type == DT_BF16)
        return a.w_f32 ? launch_norm<DT_BF16, DT_F32>(a, stream) : launch_norm<DT_BF16, DT_BF16>(a, stream);
    return a.w_f32 ? launch_norm<DT_F16, DT_F32>(a, stream) : launch_norm<DT_F16, DT_F16>(a, stream);
}

int64_t rms_norm_backward_ws(int64_t rows, int64_t dim) { return grad_sums_bytes(rows, dim); }

hipError_t launch_rms_norm_backward(const NormGradArgs& a, hipStream_t stream) {
    const int groups = grad_groups(a.rows, a.dim);
    if (groups > 0) {
        const hipError_t e = a.type == DT_F32 ? launch_grad<DT_F32, DT_F32>(a, groups, stream)
                             : a.type == DT_BF16 ? (a.w_f32 ? launch_grad<DT_BF16, DT_F32>(a, groups, stream)
                                                            : launch_grad<DT_BF16, DT_BF16>(a, groups, stream))
                                                 : (a.w_f32 ? launch_grad<DT_F16, DT_F32>(a, groups, stream)
                                                            : launch_grad<DT_F16, DT_F16>(a, groups, stream));
        if (e != hipSuccess || groups == 1) return e;
    }
    // (no rows: sums of nothing)
    rms_norm_grad_sum_kernel<<<dim3((a.dim + 63) / 64), dim3(1024), 0, stream>>>(a.ws, groups, a.dim, a.grad_weight);
    return hipGetLastError();
}

}  // namespace mpdt
