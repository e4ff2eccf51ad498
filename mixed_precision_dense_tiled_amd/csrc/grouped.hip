// grouped.hip -- matrix products grouped by expert, for gfx950: rows of A sorted by
// group, each group with a matrix of its own.
//
//   NN, NT   D[i] = A[i] . B[e] (or B[e]^T), rows i of group e
//   TN       D[e] = sum over rows i of group e of A[i]^T G[i]
//
// Where a group begins and ends only the device knows.  Every workgroup finds the
// group of its tile by itself, from a prefix sum over the groups' row tiles; the grid
// is the most tiles that the rows could need.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_common.hpp"
#include "layers.hpp"

namespace mpdt {
namespace {

// ---- groups -----------------------------------------------------------------------

// Inclusive sums and running maxima over a wave's lanes.
__device__ __forceinline__ int lanes_sum(int v, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(v, d);
        if (lane >= d) v += o;
    }
    return v;
}
__device__ __forceinline__ int lanes_max(int v, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(v, d);
        if (lane >= d) v = max(v, o);
    }
    return v;
}

// Rows [lo, hi) of group e where every offset counts as the largest up to it, cut to
// [0, rows]: groups never share a row, whatever the offsets hold.
struct Rows {
    int lo, hi;
};
__device__ __forceinline__ Rows rows_of(const GroupedArgs& g, int e, int lane) {
    int lo = 0;
    for (int i = lane; i <= e; i += 64) lo = max(lo, g.offsets[i]);
    lo = __shfl(lanes_max(lo, lane), 63);
    lo = min(lo, g.rows);
    return {lo, min(max(lo, g.offsets[e + 1]), g.rows)};
}

// Row tile t of all groups' row tiles of BM rows, counted in the order of the groups.
struct RowTile {
    int group;      // -1: there is no such tile
    int lo, hi;     // the group's rows
    int tile, tiles;    // which of the group's tiles, of how many
};
template <int BM>
__device__ __forceinline__ RowTile row_tile(const GroupedArgs& g, int t, int lane) {
    int most = 0, base = 0;
    for (int e0 = 0; e0 < g.groups; e0 += 64) {
        const int e = e0 + lane;
        int end = e < g.groups ? g.offsets[e + 1] : 0;
        int lo = e < g.groups ? g.offsets[e] : 0;
        // (offsets[e] is offsets[e - 1 + 1], so one running maximum gives both ends)
        end = max(max(most, __shfl(lo, 0)), lanes_max(end, lane));
        lo = __shfl_up(end, 1);
        if (lane == 0) lo = max(most, g.offsets[e0]);
        most = __shfl(end, 63);
        lo = min(max(lo, 0), g.rows);
        end = min(max(end, lo), g.rows);
        const int tiles = (end - lo + BM - 1) / BM;
        const int upto = base + lanes_sum(tiles, lane);
        const uint64_t here = __ballot(t < upto);
        if (here) {
            const int l = __ffsll((unsigned long long)here) - 1;
            const int n = __shfl(tiles, l);
            return {e0 + l, __shfl(lo, l), __shfl(end, l), t - (__shfl(upto, l) - n), n};
        }
        base = __shfl(upto, 63);
    }
    return {-1, 0, 0, 0, 0};
}

// ---- any problem --------------------------------------------------------------------

template <GroupedType T> struct KindOf;
template <> struct KindOf<GroupedType::BF16> { static constexpr Kind kind = Kind::BF16; };
template <> struct KindOf<GroupedType::F16> { static constexpr Kind kind = Kind::F16; };
template <> struct KindOf<GroupedType::I8> { static constexpr Kind kind = Kind::I8; };

// One value of D.
template <GroupedType T>
__device__ __forceinline__ void put16(char* D, int64_t at, float v) {
    reinterpret_cast<uint16_t*>(D)[at] = T == GroupedType::F16 ? f32_to_f16_bits(v) : f32_to_bf16_bits(v);
}

// The kernel for rows of any length and alignment: 128 x 128 tiles, four waves of
// 64 x 64, operands through registers (bounded, re-aligned) into one of two LDS stages
// of 64 bytes along the summed axis.  An operand whose rows run along that axis (KC) is
// read back along them; one whose rows lie across it (KS) with the transposing reads.
template <GroupedType T, int MODE>
__global__ __launch_bounds__(256) void grouped_any_kernel(GroupedArgs g) {
    constexpr Kind KD = KindOf<T>::kind;
    using F = Fmt<KD>;
    using Acc = typename F::Acc;
    constexpr int ES = F::ES, BM = 128, BN = 128, KT = 64, KROWS = KT / ES;
    constexpr bool A_KS = MODE == GROUPED_TN, B_KS = MODE != GROUPED_NT;
    constexpr int TILE = 128 * KT;      // bytes of an operand's tile, either way
    constexpr int U = TILE / 16 / 256;  // 16-byte pieces of a thread
    static_assert(ES == 2 || (!A_KS && !B_KS), "8-bit operands along the summed axis");
    __shared__ __attribute__((aligned(1024))) char lds[2][2][TILE];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave >> 1, wn = wave & 1;
    const int tiles_n = (g.N + BN - 1) / BN;

    // the tile: rows [m0, m_end) of A (TN: columns), columns from n0; k from k0 to k1
    int group, m0, m_end, k0, k1;
    const int n0 = (int)(blockIdx.x % tiles_n) * BN;
    if constexpr (MODE == GROUPED_TN) {
        const int tiles_m = (g.M + BM - 1) / BM;
        const int mt = blockIdx.x / tiles_n;
        group = mt / tiles_m;
        m0 = (mt - group * tiles_m) * BM;
        m_end = g.M;
        const Rows r = rows_of(g, group, lane);
        k0 = r.lo;
        k1 = r.hi;
    } else {
        const RowTile r = row_tile<BM>(g, blockIdx.x / tiles_n, lane);
        if (r.group < 0) return;    // (the whole workgroup)
        group = r.group;
        m0 = r.lo + r.tile * BM;
        m_end = r.hi;
        k0 = 0;
        k1 = g.K;
    }
    const char* const B = MODE == GROUPED_TN ? g.B : g.B + group * g.group_b;

    u32x4 ra[U], rb[U];
    // 16-byte pieces of an operand at (row r0 + .., k): KC rows r0 .. r0 + 127 of at most
    // `end` rows, KS rows k of columns r0 ..
    auto load = [&](u32x4 (&v)[U], bool ks, const char* base, int64_t ld, int r0, int end, int k) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = tid + 256 * u;
            const char *p, *stop;
            if (ks) {
                const int row = k + s / 16;     // 256 bytes of a row
                p = base + (int64_t)row * ld + (int64_t)r0 * ES + s % 16 * 16;
                stop = row < k1 ? base + (int64_t)row * ld + (int64_t)end * ES : p;
            } else {
                const int row = r0 + s / 4;     // 64 bytes of a row
                p = base + (int64_t)row * ld + (int64_t)k * ES + s % 4 * 16;
                stop = row < end ? base + (int64_t)row * ld + (int64_t)k1 * ES : p;
            }
            v[u] = load16_row<false>(p, stop);
        }
    };
    auto store = [&](const u32x4 (&v)[U], bool ks, MPDT_LDS char* to) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t s = tid + 256 * u;
            const uint32_t off = ks ? s / 16 * 256 + ((s % 16 ^ swz_b<2>(s / 16)) << 4)
                                    : s / 4 * KT + ((s % 4 ^ swz_a<4>(s / 4)) << 4);
            lds_store16(to, off, v[u]);
        }
    };
    // the operand of an MFMA step: row (column) r0 + lane % 32, 16 bytes along k
    const uint32_t lrow = lane & 31, lhalf = lane >> 5, grp = lane >> 4, gp = lane & 15;
    auto operand = [&](bool ks, const MPDT_LDS char* from, int r0, int step) -> u32x4 {
        if (!ks) {
            const uint32_t r = r0 + lrow, c = step * 2 + lhalf;
            return lds_load16(from, r * KT + ((c ^ swz_a<4>(r)) << 4));
        }
        const uint32_t col = r0 + 16 * (grp & 1), c = (col >> 3) + ((gp & 3) >> 1);
        u32x4 v;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t k = step * 16 + 8 * (grp >> 1) + 4 * h + (gp >> 2);
            const u32x2 w = lds_read_tr16(from, k * 256 + ((c ^ swz_b<2>(k)) << 4) + 8 * (gp & 1));
            v[2 * h] = w[0];
            v[2 * h + 1] = w[1];
        }
        return v;
    };

    Acc acc[2][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i >> 1][i & 1][r] = 0;
    const int steps = k1 > k0 ? (k1 - k0 + KROWS - 1) / KROWS : 0;
    if (steps > 0) {
        load(ra, A_KS, g.A, g.lda_b, m0, m_end, k0);
        load(rb, B_KS, B, g.ldb_b, n0, g.N, k0);
    }
    for (int t = 0; t < steps; ++t) {
        MPDT_LDS char* const sa = lds_cast(lds[t & 1][0]);
        MPDT_LDS char* const sb = lds_cast(lds[t & 1][1]);
        store(ra, A_KS, sa);
        store(rb, B_KS, sb);
        if (t + 1 < steps) {
            load(ra, A_KS, g.A, g.lda_b, m0, m_end, k0 + (t + 1) * KROWS);
            load(rb, B_KS, B, g.ldb_b, n0, g.N, k0 + (t + 1) * KROWS);
        }
        // (two stages: what is stored next was last read before this barrier)
        __syncthreads();
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            u32x4 a[2], b[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                a[i] = operand(A_KS, sa, wm * 64 + i * 32, s);
                b[i] = operand(B_KS, sb, wn * 64 + i * 32, s);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[i][j] = F::mma(a[i], b[j], acc[i][j]);
        }
    }
    // lane element r of a 32 x 32 block: row 8 (r / 4) + 4 lhalf + r % 4, column lrow
    char* const D = MODE == GROUPED_TN ? g.D + group * g.group_d * (g.out16 ? 2 : 4) : g.D;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int col = n0 + wn * 64 + j * 32 + (int)lrow;
        if (col >= g.N) continue;
        float ws = 0, bias = 0;
        if constexpr (T == GroupedType::I8) {
            ws = g.w_scale[group * g.ld_ws + col];
            if (g.bias) bias = g.bias[group * g.ld_bias + col];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int row = m0 + wm * 64 + i * 32 + 8 * (r >> 2) + 4 * (int)lhalf + (r & 3);
                if (row >= m_end) continue;
                const int64_t at = (int64_t)row * g.ldd + col;
                if constexpr (T == GroupedType::I8) {
                    float v = mul_rn(mul_rn((float)acc[i][j][r], g.x_scale[row]), ws);
                    if (g.bias) v = add_rn(v, bias);
                    put16<T>(D, at, v);
                } else {
                    if (g.out16) put16<T>(D, at, acc[i][j][r]);
                    else reinterpret_cast<float*>(D)[at] = acc[i][j][r];
                }
            }
    }
}

// The most row tiles of BM rows that the groups can have.
int64_t most_row_tiles(const GroupedArgs& a, int64_t bm) {
    return a.rows / bm + (a.rows < a.groups ? a.rows : a.groups);
}

int64_t grouped_tiles(int mode, const GroupedArgs& a, int64_t bm, int64_t bn) {
    const int64_t tn = (a.N + bn - 1) / bn;
    return tn * (mode == GROUPED_TN ? (a.M + bm - 1) / bm * a.groups : most_row_tiles(a, bm));
}

template <GroupedType T, int MODE>
hipError_t launch_any(const GroupedArgs& a, hipStream_t stream) {
    grouped_any_kernel<T, MODE><<<dim3((unsigned)grouped_tiles(MODE, a, 128, 128)), dim3(256), 0, stream>>>(a);
    return hipGetLastError();
}

template <GroupedType T>
hipError_t launch_type(int mode, const GroupedArgs& a, hipStream_t stream) {
    if constexpr (T == GroupedType::I8) return launch_any<T, GROUPED_NT>(a, stream);
    else
        return mode == GROUPED_NN ? launch_any<T, GROUPED_NN>(a, stream)
               : mode == GROUPED_NT ? launch_any<T, GROUPED_NT>(a, stream) : launch_any<T, GROUPED_TN>(a, stream);
}

}  // namespace

bool grouped_fits(int mode, const GroupedArgs& a) { return grouped_tiles(mode, a, 128, 128) <= MAX_GROUPS; }

hipError_t launch_grouped(GroupedType type, int mode, const GroupedArgs& a, hipStream_t stream) {
    switch (type) {
        case GroupedType::BF16: return launch_type<GroupedType::BF16>(mode, a, stream);
        case GroupedType::F16: return launch_type<GroupedType::F16>(mode, a, stream);
        default: return launch_type<GroupedType::I8>(mode, a, stream);
    }
}

}  // namespace mpdt
