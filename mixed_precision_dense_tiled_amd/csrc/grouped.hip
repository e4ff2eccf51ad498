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
#include <limits.h>
#include <stdint.h>

#include "gemm_common.hpp"
#include "layer_sizes.hpp"
#include "layers.hpp"

namespace mpdt {
namespace {

// ---- groups -----------------------------------------------------------------------

// Inclusive sums and running maxima over a wave's lanes: within rows of 16 lanes by
// shifts, then the last lane of a row to the row after it, and of two to the other two.
// (Lanes that a step does not reach take `none`, which changes nothing.)
template <class F>
__device__ __forceinline__ int lanes_scan(int v, int none, F f) {
    v = f(v, __builtin_amdgcn_update_dpp(none, v, 0x111 /* row_shr:1 */, 0xf, 0xf, false));
    v = f(v, __builtin_amdgcn_update_dpp(none, v, 0x112, 0xf, 0xf, false));
    v = f(v, __builtin_amdgcn_update_dpp(none, v, 0x114, 0xf, 0xf, false));
    v = f(v, __builtin_amdgcn_update_dpp(none, v, 0x118, 0xf, 0xf, false));
    v = f(v, __builtin_amdgcn_update_dpp(none, v, 0x142 /* row_bcast:15 */, 0xa, 0xf, false));
    v = f(v, __builtin_amdgcn_update_dpp(none, v, 0x143 /* row_bcast:31 */, 0xc, 0xf, false));
    return v;
}
__device__ __forceinline__ int lanes_sum(int v) {
    return lanes_scan(v, 0, [](int a, int b) { return a + b; });
}
__device__ __forceinline__ int lanes_max(int v) {
    return lanes_scan(v, INT_MIN, [](int a, int b) { return max(a, b); });
}

// Rows [lo, hi) of group e where every offset counts as the largest up to it, cut to
// [0, rows]: groups never share a row, whatever the offsets hold.
struct Rows {
    int lo, hi;
};
__device__ __forceinline__ Rows rows_of(const GroupedArgs& g, int e, int lane) {
    int lo = 0;
    for (int i = lane; i <= e; i += 64) lo = max(lo, g.offsets[i]);
    lo = __builtin_amdgcn_readlane(lanes_max(lo), 63);
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
        // (a group begins where the one before it ends: one running maximum gives both)
        end = max(max(most, g.offsets[e0]), lanes_max(end));
        int lo = __shfl_up(end, 1);
        if (lane == 0) lo = max(most, g.offsets[e0]);
        most = __builtin_amdgcn_readlane(end, 63);
        lo = min(max(lo, 0), g.rows);
        end = min(max(end, lo), g.rows);
        const int tiles = (end - lo + BM - 1) / BM;
        const int upto = base + lanes_sum(tiles);
        const uint64_t here = __ballot(t < upto);
        if (here) {
            const int l = __ffsll((unsigned long long)here) - 1;
            const int n = __builtin_amdgcn_readlane(tiles, l);
            return {e0 + l, __builtin_amdgcn_readlane(lo, l), __builtin_amdgcn_readlane(end, l),
                    t - (__builtin_amdgcn_readlane(upto, l) - n), n};
        }
        base = __builtin_amdgcn_readlane(upto, 63);
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
// Bound by the way through registers and a barrier every 64 bytes of k (3001 rows over 11
// groups of 1003 x 1501 FP16: 79 us, 24 by the tiles below).
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

// ---- large problems -------------------------------------------------------------------

constexpr int BN = 256;     // columns of a tile

// A workgroup's piece of D.
struct Tile {
    int group;          // -1: none
    int m0, m_end;      // rows of D (TN: of D[group])
    int n0;
    int k0, k1;         // along the summed axis
    int tm;             // 64 * tm rows
    int turn;           // NT: column tile n begins with K tile n * turn
};

// Lane's group, as its tiles are counted: of 256 rows as far as they go, and for the rows
// that are left a whole, a half or a quarter of one.
struct Counts {
    int lo, end;        // rows of the group
    int whole;          // row tiles of 256 (129 to 255 left over count as one)
    int rest;           // 2: a half tile is left over; 1: a quarter; 0: nothing
};
// The group of this lane among the 64 from e0 on; `most` is the largest offset before
// them, and after the call the largest up to their end.
__device__ __forceinline__ Counts lane_group(const GroupedArgs& g, int e0, int lane, int& most) {
    const int e = e0 + lane;
    int end = e < g.groups ? g.offsets[e + 1] : 0;
    const int begin = max(most, g.offsets[e0]);
    end = max(begin, lanes_max(end));
    const int before = __builtin_amdgcn_update_dpp(begin, end, 0x138 /* wave_shr:1 */, 0xf, 0xf, false);
    most = __builtin_amdgcn_readlane(end, 63);
    const int lo = min(max(before, 0), g.rows);
    end = min(max(end, lo), g.rows);
    const int rows = end - lo, over = rows & 255;
    return {lo, end, (rows >> 8) + (over > 128), over > 128 || over == 0 ? 0 : over > 64 ? 2 : 1};
}

// B^T's rows lie K apart: workgroups that walk along k in step read from the same few
// memory channels wherever K is a multiple of their round.  Column tile n therefore begins
// n times this many bytes further on, an odd number of 128-byte lines, and goes round
// (16 matrices of 4096 x 4096 BF16 over 128 rows: 128 us in step, 98 so; INT8 over 1536
// rows 77 and 62).  Where many tiles share rows of A, they walk in step, for their L2's sake
// (8192 rows, 4096 x 14336: 904 us, 938 with turns).
constexpr int TURN_BYTES = 1920, TURN = TURN_BYTES / 64;

// The share of XCD x in n things: [n x / 8, n (x + 1) / 8).
__device__ __forceinline__ int share(int n, int x) { return (int)((int64_t)n * x / NUM_XCD); }

// Workgroup b's piece.  Workgroups go to the eight XCDs in turn and start in their order.
//   NN, NT  An XCD takes a run of neighbouring tiles, which share rows of A and columns of
//           B in its L2.  Where they make few rounds of one to a CU, it is a run of tiles
//           of each size, the largest first, and whole tiles past the last round are split
//           in halves or quarters where all CUs together then end sooner (12288 rows over
//           32 groups of 2048 x 1408: 282 whole tiles, of which 26 would be a round of
//           their own; 119 us in the groups' order, 100 in this one).  Over many rounds
//           parts of tiles stay beside their neighbours, whose columns of B they share
//           (16384 rows over 8 groups of 4096 x 14336: 1787 us with them last, 1747).
//   TN      The matrices' tiles one group after the other: their work goes by their
//           groups' rows, so every XCD has its part of every group (a run of groups to an
//           XCD left one working for 179 us and another for 103).
template <int MODE, int BM>
__device__ __forceinline__ Tile tile_at(const GroupedArgs& g, int lane) {
    const int tiles_n = (g.N + BN - 1) / BN;
    Tile t{-1, 0, 0, 0, 0, g.K, BM / 64, 0};
    if constexpr (MODE == GROUPED_TN) {
        const int tiles_m = (g.M + BM - 1) / BM, n = blockIdx.x;
        t.group = n / (tiles_m * tiles_n);
        const int in = n - t.group * (tiles_m * tiles_n);
        t.m0 = in % tiles_m * BM;
        t.m_end = g.M;
        t.n0 = in / tiles_m * BN;
        const Rows r = rows_of(g, t.group, lane);
        t.k0 = r.lo;
        t.k1 = r.hi;
        return t;
    }
    Counts first{};
    int most = 0, after_first = 0, whole = 0, half = 0, quarter = 0;
    for (int e0 = 0; e0 < g.groups; e0 += 64) {
        const Counts c = lane_group(g, e0, lane, most);
        if (e0 == 0) {
            first = c;
            after_first = most;
        }
        whole += __builtin_amdgcn_readlane(lanes_sum(c.whole), 63);
        half += __popcll(__ballot(c.rest == 2));
        quarter += __popcll(__ballot(c.rest == 1));
    }
    whole *= tiles_n;
    half *= tiles_n;
    quarter *= tiles_n;
    // many rounds: a run of all tiles to an XCD, parts of tiles in their place
    const bool many = whole >= 4 * CUS;
    t.turn = many ? 0 : TURN;
    const int x = blockIdx.x % NUM_XCD;
    int n = blockIdx.x / NUM_XCD, part = 0, split = 1, rest = 0;    // rest: 2 the half tiles, 1 the quarters, 0 whole ones
    if (many) {
        const int all = whole + half + quarter;
        n += share(all, x);
        if (n >= share(all, x + 1)) return t;
    } else {
        const int full = whole / CUS * CUS, left = whole - full;
        split = left * 4 + half + quarter <= CUS ? 4 : left * 2 + half + quarter <= CUS ? 2 : 1;
        const int a = full / NUM_XCD, b = share(left * split, x + 1) - share(left * split, x);
        const int c = share(half, x + 1) - share(half, x);
        if (n < a) {
            n += x * a;
        } else if ((n -= a) < b) {
            n += share(left * split, x);
            part = n % split;
            n = full + n / split;
            t.tm = 4 / split;
        } else if ((n -= b) < c) {
            n += share(half, x);
            rest = t.tm = 2;
        } else {
            n += share(quarter, x) - c;
            rest = t.tm = 1;
            if (n >= share(quarter, x + 1)) return t;
        }
    }
    // its group
    int row_tile = n / tiles_n, base = 0;
    most = after_first;
    for (int e0 = 0; e0 < g.groups; e0 += 64) {
        const Counts q = e0 == 0 ? first : lane_group(g, e0, lane, most);
        const int count = many ? q.whole + (q.rest > 0) : rest == 0 ? q.whole : q.rest == rest;
        const int upto = base + lanes_sum(count);
        const uint64_t here = __ballot(row_tile < upto);
        if (here) {
            const int l = __ffsll((unsigned long long)here) - 1, of = __builtin_amdgcn_readlane(count, l);
            const int wholes = __builtin_amdgcn_readlane(q.whole, l);
            row_tile -= __builtin_amdgcn_readlane(upto, l) - of;
            t.group = e0 + l;
            t.m_end = __builtin_amdgcn_readlane(q.end, l);
            t.m0 = __builtin_amdgcn_readlane(q.lo, l);
            if (rest) {
                t.m0 += wholes * 256;
                t.n0 = n % tiles_n * BN;
            } else {
                // up to GROUP_M row tiles beside each other, then the next column tile
                const int local = row_tile * tiles_n + n % tiles_n, s = local / (GROUP_M * tiles_n);
                const int high = min(of - s * GROUP_M, GROUP_M), in = local - s * GROUP_M * tiles_n;
                const int m = s * GROUP_M + in % high;
                if (m == wholes) t.tm = __builtin_amdgcn_readlane(q.rest, l);
                t.m0 += m * 256 + part * 64 * t.tm;
                t.n0 = in / high * BN;
                if (t.m0 >= t.m_end) t.group = -1;      // (a part of a tile that is not full)
            }
            return t;
        }
        base = __builtin_amdgcn_readlane(upto, 63);
    }
    return t;
}
// The most workgroups that this takes: row tiles of the groups, the parts past the last
// round, and what the XCDs' shares round up.
int64_t tile_workgroups(const GroupedArgs& a) {
    const int64_t tn = (a.N + BN - 1) / BN;
    return tn * (a.rows / 256 + (a.rows < a.groups ? a.rows : a.groups)) + CUS + 4 * NUM_XCD;
}

// (out of vector divisions: back to scalar registers)
__device__ __forceinline__ Tile scalar(const Tile& t) {
    return {__builtin_amdgcn_readfirstlane(t.group), __builtin_amdgcn_readfirstlane(t.m0),
            __builtin_amdgcn_readfirstlane(t.m_end), __builtin_amdgcn_readfirstlane(t.n0),
            __builtin_amdgcn_readfirstlane(t.k0), __builtin_amdgcn_readfirstlane(t.k1),
            __builtin_amdgcn_readfirstlane(t.tm), __builtin_amdgcn_readfirstlane(t.turn)};
}

constexpr uint32_t NOWHERE = 0x80000000u;   // a lane offset past every buffer range: the load gives zeros

// One operand of a tile: 64 * TT rows (KC), or columns of KS rows (TT 4 or 2), by 64 bytes
// of the summed axis to a stage.  Direct loads move 1 KiB an instruction: 16 rows of 64
// bytes (KC), or 2 rows of 512 (KS; 4 of 256 with TT 2).  The swizzle is on the global side:
// the lane that fills a chunk of LDS reads the chunk that belongs there.
template <bool KS, int TT, int ES>
struct Operand {
    static constexpr int PIECES = TT;       // a wave's
    static constexpr int BYTES = PIECES * 4096;
    static constexpr int ROW = KS ? 128 * TT : 64, LANES = ROW / 16;    // bytes of a row, lanes that load it
    static_assert(!KS || (ES == 2 && TT >= 2), "16-bit rows of at least 128 columns across the summed axis");
    static constexpr int KROWS = 64 / ES;
    uint32_t voff[PIECES];  // from the K tile's first byte; NOWHERE for rows or columns past the end
    int idx[PIECES];        // KC: the chunk's byte along the summed axis; KS: its row
    uint64_t base;          // of K tile 0
    int64_t step;           // bytes to the next K tile
    int64_t back_b;         // bytes by which the last K tile begins earlier
    int have;               // what all K tiles hold along the summed axis, in the units of idx
    uint32_t read0;         // LDS offset of this lane's operand of step 0, 32-row tile 0

    // rows (columns) [r0, end) of the operand at p, summed over `keys` from k0 on, the last
    // tile `back` elements earlier
    __device__ __forceinline__ void init(const char* p, int64_t ld, int r0, int end, int k0, int keys, int back,
                                         int wave, int lane, int w_half) {
        back_b = back * (KS ? ld : ES);
        have = (keys + back) * (KS ? 1 : ES);
        if constexpr (KS) {
            base = (uint64_t)(uintptr_t)p + (uint64_t)((int64_t)k0 * ld + (int64_t)r0 * ES);
            step = (int64_t)KROWS * ld;
        } else {
            base = (uint64_t)(uintptr_t)p + (uint64_t)((int64_t)r0 * ld + (int64_t)k0 * ES);
            step = 64;
        }
#pragma unroll
        for (int u = 0; u < PIECES; ++u) {
            if constexpr (KS) {
                const int row = (wave * PIECES + u) * (64 / LANES) + lane / LANES;
                const uint32_t c = (uint32_t)(lane % LANES) ^ swz_b<2>(row);
                idx[u] = row;
                voff[u] = r0 + (int)c * 8 < end ? (uint32_t)row * (uint32_t)ld + c * 16u : NOWHERE;
            } else {
                const int row = (wave * PIECES + u) * 16 + (lane >> 2);
                const uint32_t c = (uint32_t)(lane & 3) ^ swz_a<4>(row);
                idx[u] = (int)c * 16;
                voff[u] = r0 + row < end ? (uint32_t)row * (uint32_t)ld + c * 16u : NOWHERE;
            }
        }
        const uint32_t lrow = lane & 31, lhalf = lane >> 5, grp = lane >> 4, gp = lane & 15;
        const int first = w_half * 32 * TT;     // this wave's first row (column)
        if constexpr (KS) {
            const uint32_t col = first + 16 * (grp & 1), k = 8 * (grp >> 1) + (gp >> 2);
            read0 = k * ROW + ((((col >> 3) + ((gp & 3) >> 1)) ^ swz_b<2>(k)) << 4) + 8 * (gp & 1);
        } else {
            const uint32_t r = first + lrow;
            read0 = r * 64 + ((lhalf ^ swz_a<4>(r)) << 4);
        }
    }
    // piece u of K tile t; `left`: what the tile holds along the summed axis (KC: bytes)
    __device__ __forceinline__ void load(int u, i32x4 rsrc, MPDT_LDS char* stage, int wave, int left) const {
        const uint32_t v = idx[u] < left ? voff[u] : NOWHERE;
        lds_dma16<0, true>(rsrc, stage + (wave * PIECES + u) * 1024, v, 0u);
    }
    // the buffer of K tile t, which begins at `at` (one that is not there is empty)
    __device__ __forceinline__ i32x4 rsrc(uint64_t at, bool last, bool there) const {
        return rsrc_words(last ? at - (uint64_t)back_b : at, there ? 0x7fffffffu : 0u);
    }
    // what it holds along the summed axis (and more)
    __device__ __forceinline__ int left(int t) const { return have - t * (KS ? KROWS : 64); }
    // the MFMA operand of step s (0, 1) and 32-row tile i
    __device__ __forceinline__ u32x4 read(const MPDT_LDS char* stage, int s, int i) const {
        if constexpr (KS) {
            // (4 rows on, the swizzle repeats; 32 columns on are bits 2 and 3 of the
            // chunk, which the swizzle may have turned over)
            const uint32_t o = (read0 ^ (uint32_t)(i * 64)) + s * 16 * ROW;
            const u32x2 x = lds_read_tr16(stage, o), y = lds_read_tr16(stage, o + 4 * ROW);
            return u32x4{x[0], x[1], y[0], y[1]};
        } else {
            return lds_load16(stage, (read0 ^ (uint32_t)(s * 32)) + i * 32 * 64);
        }
    }
};

// A tile's product by four waves, one to a SIMD: 64 * TM x 256 of D, 32 * TM x 128 a wave
// (TM 4, 2 or 1), accumulated in registers for the whole of k.  A stage holds 64 bytes of k
// of both operands; NS stages are loaded ahead.  For K tile t:
//   phase X: MFMAs of its first step, among them the reads of the second step's operands
//            and the direct loads of B of tile t - 1 + NS;
//   wait for tile t + 1's loads and this wave's reads, barrier;
//   phase Y: MFMAs of the second step, among them the reads of tile t + 1's first step and
//            the direct loads of A of tile t + NS (into the stage of tile t).
// Tiles past the last load nothing (an empty buffer range), so that the count of loads in
// flight is the same everywhere.  Where rows along k end inside a 16-byte piece, the last
// tile is the 64 bytes that end with them: what it repeats of the tile before is cleared
// in both operands.
template <GroupedType T, int MODE, int TM, int LDS>
struct Product {
    using F = Fmt<KindOf<T>::kind>;
    using Acc = typename F::Acc;
    static constexpr int ES = F::ES;
    using OpA = Operand<MODE == GROUPED_TN, TM, ES>;
    using OpB = Operand<MODE != GROUPED_NT, 4, ES>;
    static constexpr int STAGE = OpA::BYTES + OpB::BYTES;
    static constexpr int NS = LDS / STAGE < 6 ? LDS / STAGE : 6;
    static constexpr int LOADS = OpA::PIECES + OpB::PIECES;
    static constexpr int NM = TM * 4, GROUPS = TM + 3;  // MFMAs of a step; operand reads: A0 and B0, B1, B2, B3, A1 ..
    OpA A;
    OpB B;
    int keys, nt, back, from;

    __device__ __forceinline__ void init(const GroupedArgs& g, const Tile& t, int wave, int lane) {
        keys = t.k1 - t.k0;
        nt = (keys + OpA::KROWS - 1) / OpA::KROWS;
        back = MODE != GROUPED_TN && keys * ES % 16 ? nt * OpA::KROWS - keys : 0;
        from = MODE == GROUPED_NT && !back ? t.n0 / BN * t.turn % nt : 0;
        A.init(g.A, g.lda_b, t.m0, t.m_end, t.k0, keys, back, wave, lane, wave >> 1);
        B.init(MODE == GROUPED_TN ? g.B : g.B + t.group * g.group_b, g.ldb_b, t.n0, g.N, t.k0, keys, back, wave, lane,
               wave & 1);
    }

    // The product into acc; LDS is free when every wave has returned.
    __device__ __forceinline__ void run(MPDT_LDS char* lds, int wave, int lane, Acc (&acc)[TM][4]) const {
        // the tile that is loaded next, from `from` on and round
        int pos = from;
        uint64_t at_a = A.base + (uint64_t)(from * A.step), at_b = B.base + (uint64_t)(from * B.step);
        auto step = [&] {
            at_a += (uint64_t)A.step;
            at_b += (uint64_t)B.step;
            if (++pos == nt && MODE == GROUPED_NT) {
                pos = 0;
                at_a = A.base;
                at_b = B.base;
            }
        };
        i32x4 rb{};     // B's buffer of the tile whose loads are due next
        int left_b = 0;
#pragma unroll
        for (int p = 0; p < NS; ++p) {
            const i32x4 ra = A.rsrc(at_a, pos == nt - 1, p < nt);
            const int left_a = A.left(pos);
            rb = B.rsrc(at_b, pos == nt - 1, p < nt);
            left_b = B.left(pos);
            step();
            static_for<0, OpA::PIECES>([&](auto U) { A.load(decltype(U)::value, ra, lds + p * STAGE, wave, left_a); });
            if (p < NS - 1)
                static_for<0, 4>([&](auto U) { B.load(decltype(U)::value, rb, lds + p * STAGE + OpA::BYTES, wave, left_b); });
        }
        u32x4 fa[2][TM], fb[2][4];
        auto read_group = [&](int s, int r, const MPDT_LDS char* stage) {
            if (r == 0) fa[s][0] = A.read(stage, s, 0);
            if (r <= 3) fb[s][r] = B.read(stage + OpA::BYTES, s, r);
            else fa[s][r - 3] = A.read(stage, s, r - 3);
        };
        // (the operands change places: a lane then holds four neighbouring columns of a row)
        auto mma = [&](int s, int i) { acc[i / 4][i % 4] = F::mma(fb[s][i % 4], fa[s][i / 4], acc[i / 4][i % 4]); };

        wait_vmem<(NS - 2) * LOADS + OpA::PIECES>();
        wg_barrier();
#pragma unroll
        for (int r = 0; r < GROUPS; ++r) read_group(0, r, lds);
        int cur = 0;
        for (int k = 0; k < nt - 1; ++k) {
            const int next = cur + 1 == NS ? 0 : cur + 1, prev = cur == 0 ? NS - 1 : cur - 1;
            MPDT_LDS char* const sc = lds + cur * STAGE;
            MPDT_LDS char* const sn = lds + next * STAGE;
            MPDT_LDS char* const sp = lds + prev * STAGE + OpA::BYTES;
            i32x4 ra, rb2;
            int left_a, left_b2;
            static_for<0, NM>([&](auto I) {
                constexpr int i = decltype(I)::value;
                mma(0, i);
                if constexpr (i < GROUPS) read_group(1, i, sc);
                if constexpr (i == NM / 2) {
                    ra = A.rsrc(at_a, pos == nt - 1, k + NS < nt);
                    left_a = A.left(pos);
                }
                if constexpr (i == NM / 2 + 1) {
                    rb2 = B.rsrc(at_b, pos == nt - 1, k + NS < nt);
                    left_b2 = B.left(pos);
                    step();
                }
                // B's four loads on the last slots, every second one where there are 16
                constexpr int STEP = TM == 4 ? 2 : 1, FIRST = NM - 1 - 3 * STEP;
                if constexpr (i >= FIRST && (i - FIRST) % STEP == 0) B.load((i - FIRST) / STEP, rb, sp, wave, left_b);
                __builtin_amdgcn_sched_barrier(0);
            });
            wait_vmem<(NS - 2) * LOADS>();
            wait_lds();
            wg_barrier();
            static_for<0, NM>([&](auto I) {
                constexpr int i = decltype(I)::value;
                mma(1, i);
                if constexpr (i % 4 == 0) A.load(i / 4, ra, sc, wave, left_a);
                // the reads in between: slots 1, 3, 5 .. of 16; every other free one of fewer
                if constexpr (TM == 4) {
                    if constexpr (i % 2 == 1 && i / 2 < GROUPS) read_group(0, i / 2, sn);
                } else if constexpr (TM == 2) {
                    if constexpr (i % 4 != 0 && i - 1 - i / 4 < GROUPS) read_group(0, i - 1 - i / 4, sn);
                } else {
                    read_group(0, i, sn);
                }
                __builtin_amdgcn_sched_barrier(0);
            });
            rb = rb2;
            left_b = left_b2;
            cur = next;
        }
        MPDT_LDS char* const sc = lds + cur * STAGE;
        auto clear = [&](int s) {
            const int n = min(max(back * ES - s * 32 - (lane >> 5) * 16, 0), 16);
#pragma unroll
            for (int i = 0; i < TM; ++i) fa[s][i] = mask_head(fa[s][i], n);
#pragma unroll
            for (int i = 0; i < 4; ++i) fb[s][i] = mask_head(fb[s][i], n);
        };
        if (back) clear(0);
        static_for<0, NM>([&](auto I) {
            constexpr int i = decltype(I)::value;
            mma(0, i);
            if constexpr (i < GROUPS) read_group(1, i, sc);
            __builtin_amdgcn_sched_barrier(0);
        });
        wait_lds();
        if (back) clear(1);
#pragma unroll
        for (int i = 0; i < NM; ++i) mma(1, i);
        // (the empty loads write zeros: they land before LDS is used again)
        wait_vmem<0>();
    }
};

// Four neighbouring values of a vector of n, from c on; 0 past its end.
__device__ __forceinline__ f32x4 four_of(const float* p, int c, int n) {
    typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
    if (c + 4 <= n) {
        const f32x4_any v = *reinterpret_cast<const f32x4_any*>(p + c);
        return f32x4{v[0], v[1], v[2], v[3]};
    }
    f32x4 v{0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 3; ++e)
        if (c + e < n) v[e] = p[c + e];
    return v;
}

// D from the accumulators, through LDS so that it leaves in 16-byte pieces of rows: a wave
// has a quarter of LDS for as many of its blocks of 32 rows by 128 columns as fit.  Lane
// element r of a 32 x 32 block: row lane % 32, column 8 (r / 4) + 4 (lane / 32) + r % 4.
// (m_own, n_own: a tile that was moved back to end with the operand stores from there on)
template <GroupedType T, int MODE, int TM, int LDS, class Out, class Acc>
__device__ __forceinline__ void tile_store(const GroupedArgs& g, const Tile& t, int m_own, int n_own, MPDT_LDS char* lds,
                                           int wave, int lane, const Acc (&acc)[TM][4]) {
    constexpr int ES = (int)sizeof(Out), ROW = 128 * ES, CHUNKS = ROW / 16, PER = 16 / ES;
    constexpr int FIT = LDS / 4 / (32 * ROW), STEP = FIT >= TM ? TM : FIT >= 2 ? 2 : 1;
    static_assert(FIT >= 1, "a block of a wave's rows fits its quarter of LDS");
    typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
    const int wm = wave >> 1, wn = wave & 1, lrow = lane & 31, lhalf = lane >> 5;
    const int row0 = t.m0 + wm * 32 * TM, col0 = t.n0 + wn * 128;
    wg_barrier();       // every wave is done with the stages
    if (row0 >= t.m_end || col0 >= g.N) return;     // (the whole wave)
    MPDT_LDS char* const own = lds + wave * (LDS / 4);
    Out* const D = reinterpret_cast<Out*>(g.D) + (MODE == GROUPED_TN ? t.group * g.group_d : 0);
    f32x4 ws[T == GroupedType::I8 ? 16 : 1], bias[T == GroupedType::I8 ? 16 : 1];
    if constexpr (T == GroupedType::I8) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int col = col0 + (i >> 2) * 32 + 8 * (i & 3) + 4 * lhalf;
            ws[i] = four_of(g.w_scale + t.group * g.ld_ws, col, g.N);
            bias[i] = g.bias ? four_of(g.bias + t.group * g.ld_bias, col, g.N) : f32x4{-0.0f, -0.0f, -0.0f, -0.0f};
        }
    }
#pragma unroll
    for (int i0 = 0; i0 < TM; i0 += STEP) {
#pragma unroll
        for (int i = i0; i < i0 + STEP; ++i) {
            float xs = 0;
            if constexpr (T == GroupedType::I8) {
                const int row = row0 + i * 32 + lrow;
                xs = row < t.m_end ? g.x_scale[row] : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if constexpr (T == GroupedType::I8)     // (x + -0 is x)
                            v[e] = add_rn(mul_rn(mul_rn((float)acc[i][j][4 * q + e], xs), ws[4 * j + q][e]), bias[4 * j + q][e]);
                        else v[e] = acc[i][j][4 * q + e];
                    }
                    // chunk c of row r lies at c ^ r: rows beside each other in other banks
                    const uint32_t r = (i - i0) * 32 + lrow, c = (uint32_t)((j * 32 + 8 * q + 4 * lhalf) * ES) / 16;
                    MPDT_LDS char* const p = own + r * ROW + ((c ^ (r % CHUNKS)) << 4);
                    if constexpr (ES == 4) {
                        *(MPDT_LDS f32x4*)p = f32x4{v[0], v[1], v[2], v[3]};
                    } else {
                        uint32_t h[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) h[e] = T == GroupedType::F16 ? f32_to_f16_bits(v[e]) : f32_to_bf16_bits(v[e]);
                        *(MPDT_LDS u32x2*)(p + 8 * lhalf) = u32x2{h[0] | h[1] << 16, h[2] | h[3] << 16};
                    }
                }
        }
        wait_lds();     // (a wave reads only what it wrote)
        asm volatile("" ::: "memory");
#pragma unroll 4
        for (int q = 0; q < STEP * 32 * CHUNKS / 64; ++q) {
            const int n = q * 64 + lane, r = n / CHUNKS, c = n % CHUNKS;
            const u32x4 v = lds_load16(own, r * ROW + ((c ^ (r % CHUNKS)) << 4));
            const int row = row0 + i0 * 32 + r, col = col0 + c * PER;
            if (row >= t.m_end || row < m_own) continue;
            Out* const to = D + (int64_t)row * g.ldd + col;
            if (col >= n_own && col + PER <= g.N) {
                *reinterpret_cast<u32x4_any*>(to) = v;
            } else {
#pragma unroll
                for (int e = 0; e < PER; ++e) {
                    const uint32_t w = v[e * ES / 4];
                    if (col + e >= n_own && col + e < g.N) {
                        if constexpr (ES == 4) to[e] = __uint_as_float(w);
                        else to[e] = (uint16_t)(w >> (16 * (e & 1)));
                    }
                }
            }
        }
        wait_lds();
        asm volatile("" ::: "memory");
    }
}

template <GroupedType T, int MODE, int TM, int LDS>
__device__ __forceinline__ void tile_run(const GroupedArgs& g, Tile t, MPDT_LDS char* lds, int wave, int lane) {
    typename Fmt<KindOf<T>::kind>::Acc acc[TM][4];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
    // rows across k that end inside a 16-byte piece: the last tile ends with them
    const int m_own = t.m0, n_own = t.n0;
    if (MODE == GROUPED_TN && g.M % 8) t.m0 = min(t.m0, g.M - 64 * TM);
    if (MODE != GROUPED_NT && g.N % 8) t.n0 = min(t.n0, g.N - BN);
    if (t.k1 > t.k0) {
        Product<T, MODE, TM, LDS> p;
        p.init(g, t, wave, lane);
        p.run(lds, wave, lane, acc);
    }
    if constexpr (T == GroupedType::I8) {
        tile_store<T, MODE, TM, LDS, uint16_t>(g, t, m_own, n_own, lds, wave, lane, acc);
    } else {
        if (g.out16) tile_store<T, MODE, TM, LDS, uint16_t>(g, t, m_own, n_own, lds, wave, lane, acc);
        else tile_store<T, MODE, TM, LDS, float>(g, t, m_own, n_own, lds, wave, lane, acc);
    }
}

// 256 x 256 tiles, one workgroup to a CU: bound by the matrix cores at the card's power
// limit (16384 rows over 8 groups of 4096 x 14336 BF16: 1.70 to 1.80 ms by the card, 1070 to 1130
// TFLOP/s; the library's 8192^3 product reaches 1210) where groups are large, by HBM where
// their matrices are read for few rows (INT8, 1536 rows over 16 groups of 4096 x 4096: 70
// us, 4.1 TB/s).
template <GroupedType T, int MODE>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1))) void grouped_tile_kernel(GroupedArgs g) {
    constexpr int LDS = 131072;
    __shared__ __attribute__((aligned(1024))) char lds_[LDS];
    MPDT_LDS char* const lds = lds_cast(lds_);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Tile t = scalar(tile_at<MODE, 256>(g, lane));
    if (t.group < 0) return;    // (the whole workgroup)
    if (t.tm == 4) tile_run<T, MODE, 4, LDS>(g, t, lds, wave, lane);
    else if (t.tm == 2) tile_run<T, MODE, 2, LDS>(g, t, lds, wave, lane);
    else tile_run<T, MODE, 1, LDS>(g, t, lds, wave, lane);
}

// 64 x 256 tiles of A . B, two workgroups to a CU: groups of few rows, whose matrices have
// to be read.  Neighbouring tiles go to different XCDs, so that the card reads whole rows of
// a matrix at a time (8 groups of 4096 x 14336 over 128 rows: 163 us, 5.8 TB/s; 198 with a
// run of tiles to an XCD).
template <GroupedType T>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void grouped_low_kernel(GroupedArgs g) {
    constexpr int LDS = 81920;
    __shared__ __attribute__((aligned(1024))) char lds_[LDS];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tiles_n = (g.N + BN - 1) / BN;
    const RowTile r = row_tile<64>(g, blockIdx.x / tiles_n, lane);
    if (r.group < 0) return;    // (the whole workgroup)
    const int local = r.tile * tiles_n + blockIdx.x % tiles_n;
    const Tile t{r.group, r.lo + local % r.tiles * 64, r.hi, local / r.tiles * BN, 0, g.K, 1, 0};
    tile_run<T, GROUPED_NN, 1, LDS>(g, scalar(t), lds_cast(lds_), wave, lane);
}

// 128 x 256 tiles, two workgroups to a CU: for short sums, whose tiles take as long to
// begin and to store as for their product (384 rows of a weights' gradient: 2 + 3 us and
// 10); another workgroup's product goes on meanwhile.  Weights' gradient of 12288 rows over
// 29 groups of 2048 x 1408 FP16: 116 to 125 us, 565 TFLOP/s, 185 MB of D written; its tiles go
// to the XCDs in turn.  Of the products an XCD takes a run of neighbouring tiles.  (INT8 spills
// 64 registers in tile_store, 16 scales and 16 biases of four columns, outside the loop.)
template <GroupedType T, int MODE>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void grouped_half_kernel(GroupedArgs g) {
    constexpr int LDS = 73728;
    __shared__ __attribute__((aligned(1024))) char lds_[LDS];
    MPDT_LDS char* const lds = lds_cast(lds_);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if constexpr (MODE == GROUPED_TN) {
        tile_run<T, MODE, 2, LDS>(g, scalar(tile_at<MODE, 128>(g, lane)), lds, wave, lane);
    } else {
        const int tiles_n = (g.N + BN - 1) / BN;
        int tiles = 0, most = 0;
        for (int e0 = 0; e0 < g.groups; e0 += 64) {
            const Counts c = lane_group(g, e0, lane, most);
            tiles += __builtin_amdgcn_readlane(lanes_sum((c.end - c.lo + 127) / 128), 63);
        }
        tiles *= tiles_n;
        const int x = blockIdx.x % NUM_XCD, n = share(tiles, x) + blockIdx.x / NUM_XCD;
        if (n >= share(tiles, x + 1)) return;   // (the whole workgroup)
        const RowTile r = row_tile<128>(g, n / tiles_n, lane);
        // up to GROUP_M row tiles beside each other, then the next column tile
        const int local = r.tile * tiles_n + n % tiles_n, s = local / (GROUP_M * tiles_n);
        const int high = min(r.tiles - s * GROUP_M, GROUP_M), in = local - s * GROUP_M * tiles_n;
        const Tile t = scalar(Tile{r.group, r.lo + (s * GROUP_M + in % high) * 128, r.hi, in / high * BN, 0, g.K, 2, 0});
        if (t.m_end - t.m0 > 64) tile_run<T, MODE, 2, LDS>(g, t, lds, wave, lane);
        else tile_run<T, MODE, 1, LDS>(g, t, lds, wave, lane);
    }
}

// ---- few rows --------------------------------------------------------------------------

// One operand of a strip: R rows (KC) of KT bytes along the summed axis, or R columns of
// KROWS rows (KS), all loaded by one wave, 1 KiB an instruction.  The swizzles as above;
// KS rows of 64 columns have 8 pieces, which take turns by pairs over four rows.
template <bool KS, int R, int KT, int ES>
struct Strip {
    static constexpr int KROWS = KT / ES;
    static constexpr int ROW = KS ? R * ES : KT, LANES = ROW / 16;
    static constexpr int BYTES = R * KT, PIECES = BYTES / 1024;
    static_assert(!KS || ES == 2, "16-bit rows across the summed axis");
    uint32_t voff[PIECES];
    int idx[PIECES];
    uint64_t base;
    int64_t step, back_b;
    int have;
    uint32_t read0;

    __device__ __forceinline__ static uint32_t swizzle(uint32_t row) {
        if constexpr (!KS) return swz_a<LANES>(row);
        else if constexpr (LANES == 16) return swz_b<2>(row);
        else return (row & 3u) << 1;
    }
    __device__ __forceinline__ void init(const char* p, int64_t ld, int r0, int end, int keys, int back, int lane) {
        base = (uint64_t)(uintptr_t)p + (uint64_t)(KS ? (int64_t)r0 * ES : (int64_t)r0 * ld);
        step = KS ? (int64_t)KROWS * ld : KT;
        back_b = back * (KS ? ld : ES);
        have = (keys + back) * (KS ? 1 : ES);
#pragma unroll
        for (int u = 0; u < PIECES; ++u) {
            const int row = u * (64 / LANES) + lane / LANES;
            const uint32_t c = (uint32_t)(lane % LANES) ^ swizzle(row);
            idx[u] = KS ? row : (int)c * 16;
            voff[u] = r0 + (KS ? (int)c * 8 : row) < end ? (uint32_t)row * (uint32_t)ld + c * 16u : NOWHERE;
        }
        const uint32_t lrow = lane & 31, lhalf = lane >> 5, grp = lane >> 4, gp = lane & 15;
        if constexpr (KS) {
            const uint32_t k = 8 * (grp >> 1) + (gp >> 2), c = 2 * (grp & 1) + ((gp & 3) >> 1);
            read0 = k * ROW + ((c ^ swizzle(k)) << 4) + 8 * (gp & 1);
        } else {
            read0 = lrow * ROW + ((lhalf ^ swizzle(lrow)) << 4);
        }
    }
    // all of K tile t of nt
    __device__ __forceinline__ void load(int t, int nt, MPDT_LDS char* to) const {
        const uint64_t at = base + (uint64_t)((int64_t)t * step - (t == nt - 1 ? back_b : 0));
        const i32x4 r = rsrc_words(at, t < nt ? 0x7fffffffu : 0u);
        const int left = have - t * (KS ? KROWS : KT);
#pragma unroll
        for (int u = 0; u < PIECES; ++u) lds_dma16<0, true>(r, to + u * 1024, idx[u] < left ? voff[u] : NOWHERE, 0u);
    }
    // the MFMA operand of step s and 32-row (column) tile i
    __device__ __forceinline__ u32x4 read(const MPDT_LDS char* from, int s, int i) const {
        if constexpr (KS) {
            const uint32_t o = (read0 ^ (uint32_t)(i * 64)) + s * 16 * ROW;
            const u32x2 x = lds_read_tr16(from, o), y = lds_read_tr16(from, o + 4 * ROW);
            return u32x4{x[0], x[1], y[0], y[1]};
        } else {
            return lds_load16(from, (read0 ^ (uint32_t)(s * 32)) + i * 32 * ROW);
        }
    }
};

// Few tiles: bound by the reading of the matrices and by how long a workgroup takes for
// its own.  A workgroup takes 32 * MT rows and a strip of 64 columns; its four waves take
// every fourth K tile each, through rings of direct loads of their own that no barrier
// holds up, and their sums are joined in LDS at the end.  8 rows of 8 groups of 2048 x 1408:
// 10.4 us, 24.7 by the tiles above (strips of 128 columns 12.9, rings of twice the depth in
// one workgroup to a CU 12.0).  Those are A . B's; with B^T, whose stages are 128 bytes of k, one
// workgroup has a CU: 12.4 us, INT8 8.0; 8 rows of 8 of 16 groups of 4096 x 4096 46 and 27.
template <GroupedType T, int MODE, int MT>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 2))) void grouped_few_kernel(GroupedArgs g) {
    constexpr int SN = 64;
    using F = Fmt<KindOf<T>::kind>;
    using Acc = typename F::Acc;
    using Sum = typename std::conditional<T == GroupedType::I8, i32x4, f32x4>::type;
    constexpr int ES = F::ES, KT = MODE == GROUPED_NT ? 128 : 64, NJ = SN / 32;
    using OpA = Strip<MODE == GROUPED_TN, 32 * MT, KT, ES>;
    using OpB = Strip<MODE != GROUPED_NT, SN, KT, ES>;
    constexpr int STAGE = OpA::BYTES + OpB::BYTES, LOADS = OpA::PIECES + OpB::PIECES;
    constexpr int PART = 32 * MT * SN * 4;      // a wave's sums
    // (two workgroups to a CU, where rings of two stages and the sums fit its half)
    constexpr int HALF = 163840 / 2 / 4, MOST = 2 * STAGE <= HALF && PART <= HALF ? HALF : 2 * HALF;
    constexpr int NS = MOST / STAGE < 6 ? MOST / STAGE : 6;
    static_assert(NS >= 2 && PART <= NS * STAGE && (NS - 1) * LOADS < 64, "rings and sums fit");
    __shared__ __attribute__((aligned(1024))) char lds_[4 * NS * STAGE];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int strips = (g.N + SN - 1) / SN;
    int group, m_own, m_end, n_own, k0, keys;
    if constexpr (MODE == GROUPED_TN) {
        const int tiles_m = (g.M + 32 * MT - 1) / (32 * MT), tile = blockIdx.x / strips;
        group = tile / tiles_m;
        m_own = (tile - group * tiles_m) * (32 * MT);
        m_end = g.M;
        n_own = blockIdx.x % strips * SN;
        const Rows r = rows_of(g, group, lane);
        k0 = r.lo;
        keys = r.hi - r.lo;
    } else {
        const RowTile rt = row_tile<32 * MT>(g, blockIdx.x / strips, lane);
        if (rt.group < 0) return;   // (the whole workgroup)
        // a group's row tiles of one strip beside each other: they read the same columns
        const int local = rt.tile * strips + blockIdx.x % strips;
        group = rt.group;
        m_own = rt.lo + local % rt.tiles * (32 * MT);
        m_end = rt.hi;
        n_own = local / rt.tiles * SN;
        k0 = 0;
        keys = g.K;
    }
    // (out of vector divisions: back to scalar registers)
    group = __builtin_amdgcn_readfirstlane(group);
    m_own = __builtin_amdgcn_readfirstlane(m_own);
    m_end = __builtin_amdgcn_readfirstlane(m_end);
    n_own = __builtin_amdgcn_readfirstlane(n_own);
    k0 = __builtin_amdgcn_readfirstlane(k0);
    keys = __builtin_amdgcn_readfirstlane(keys);
    const int m0 = MODE == GROUPED_TN && g.M % 8 ? min(m_own, g.M - 32 * MT) : m_own;
    const int n0 = MODE != GROUPED_NT && g.N % 8 ? min(n_own, g.N - SN) : n_own;

    const int nt = (keys + OpA::KROWS - 1) / OpA::KROWS;
    const int back = MODE != GROUPED_TN && (int64_t)keys * ES % 16 ? nt * OpA::KROWS - keys : 0;
    OpA A;
    OpB B;
    A.init(g.A + (int64_t)k0 * g.lda_b, g.lda_b, m0, m_end, keys, back, lane);
    B.init(MODE == GROUPED_TN ? g.B + (int64_t)k0 * g.ldb_b : g.B + group * g.group_b, g.ldb_b, n0, g.N, keys, back, lane);
    Acc acc[MT][NJ];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
    MPDT_LDS char* const ring = lds_cast(lds_) + wave * NS * STAGE;
    // (in turns along k, as above)
    const int from = MODE == GROUPED_NT && !back ? n0 / SN * (TURN_BYTES / KT) % nt : 0;
    auto load = [&](int t, int slot) {
        const int at = t >= nt ? t : t + from >= nt ? t + from - nt : t + from;
        A.load(at, nt, ring + slot * STAGE);
        B.load(at, nt, ring + slot * STAGE + OpA::BYTES);
    };
#pragma unroll
    for (int p = 0; p < NS - 1; ++p) load(wave + 4 * p, p);
    int slot = 0;
    for (int t = wave; t < nt; t += 4) {
        // (the slot that is filled now was read in the last round)
        load(t + 4 * (NS - 1), slot == 0 ? NS - 1 : slot - 1);
        wait_vmem<(NS - 1) * LOADS>();
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" ::: "memory");
        const MPDT_LDS char* const at = ring + slot * STAGE;
        u32x4 a[KT / 32][MT], b[KT / 32][NJ];
#pragma unroll
        for (int s = 0; s < KT / 32; ++s) {
#pragma unroll
            for (int i = 0; i < MT; ++i) a[s][i] = A.read(at, s, i);
#pragma unroll
            for (int j = 0; j < NJ; ++j) b[s][j] = B.read(at + OpA::BYTES, s, j);
        }
        if (back && t == nt - 1) {
            // what the last tile repeats
#pragma unroll
            for (int s = 0; s < KT / 32; ++s) {
                const int n = min(max(back * ES - s * 32 - (lane >> 5) * 16, 0), 16);
#pragma unroll
                for (int i = 0; i < MT; ++i) a[s][i] = mask_head(a[s][i], n);
#pragma unroll
                for (int j = 0; j < NJ; ++j) b[s][j] = mask_head(b[s][j], n);
            }
        }
#pragma unroll
        for (int s = 0; s < KT / 32; ++s)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NJ; ++j) acc[i][j] = F::mma(b[s][j], a[s][i], acc[i][j]);
        wait_lds();
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" ::: "memory");
        slot = slot + 1 == NS ? 0 : slot + 1;
    }
    // join the waves' sums: value (row, column) of wave w at w * PART + (row * SN + column)
    // * 4, pieces of a row turned by the row
    wait_vmem<0>();
    wg_barrier();
    const int lrow = lane & 31, lhalf = lane >> 5;
    constexpr int CHUNKS = SN / 4;
    MPDT_LDS char* const sums = lds_cast(lds_);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int row = i * 32 + lrow, c = j * 8 + 2 * q + lhalf;
                *(MPDT_LDS Sum*)(sums + wave * PART + row * SN * 4 + ((c ^ (row & 15)) << 4)) =
                    Sum{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
            }
    wait_lds();
    wg_barrier();
    typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
    typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
    for (int n = threadIdx.x; n < 32 * MT * CHUNKS; n += 256) {
        const int r = n / CHUNKS, c = n % CHUNKS, row = m0 + r, col = n0 + 4 * c;
        if (row >= m_end || row < m_own || col >= g.N || col + 4 <= n_own) continue;
        Sum v = *(MPDT_LDS Sum*)(sums + r * SN * 4 + ((c ^ (r & 15)) << 4));
#pragma unroll
        for (int w = 1; w < 4; ++w) v += *(MPDT_LDS Sum*)(sums + w * PART + r * SN * 4 + ((c ^ (r & 15)) << 4));
        float f[4];
        if constexpr (T == GroupedType::I8) {
            const float xs = g.x_scale[row];
            const f32x4 ws = four_of(g.w_scale + group * g.ld_ws, col, g.N);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = mul_rn(mul_rn((float)v[e], xs), ws[e]);
            if (g.bias) {
                const f32x4 bias = four_of(g.bias + group * g.ld_bias, col, g.N);
#pragma unroll
                for (int e = 0; e < 4; ++e) f[e] = add_rn(f[e], bias[e]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = v[e];
        }
        const int64_t at = (MODE == GROUPED_TN ? group * g.group_d : 0) + (int64_t)row * g.ldd + col;
        const bool all = col >= n_own && col + 4 <= g.N;
        if (T == GroupedType::I8 || g.out16) {
            uint16_t* const to = reinterpret_cast<uint16_t*>(g.D) + at;
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = T == GroupedType::F16 ? f32_to_f16_bits(f[e]) : f32_to_bf16_bits(f[e]);
            if (all) {
                *reinterpret_cast<u32x2_any*>(to) = u32x2_any{h[0] | h[1] << 16, h[2] | h[3] << 16};
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (col + e >= n_own && col + e < g.N) to[e] = (uint16_t)h[e];
            }
        } else {
            float* const to = reinterpret_cast<float*>(g.D) + at;
            if (all) {
                *reinterpret_cast<u32x4_any*>(to) =
                    u32x4_any{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (col + e >= n_own && col + e < g.N) to[e] = f[e];
            }
        }
    }
}

template <GroupedType T, int MODE>
hipError_t launch_any(const GroupedArgs& a, hipStream_t stream) {
    grouped_any_kernel<T, MODE><<<dim3((unsigned)grouped_tiles(MODE, a, 128, 128)), dim3(256), 0, stream>>>(a);
    return hipGetLastError();
}

// Whether the direct loads can take a problem: a tile's offsets fit in 32 bits, and where
// rows end inside a 16-byte piece there is a whole tile to end with them.
template <GroupedType T, int MODE>
bool by_tiles(const GroupedArgs& a) {
    constexpr int ES = T == GroupedType::I8 ? 1 : 2;
    if (a.lda_b >= (1 << 23) || a.ldb_b >= (1 << 23)) return false;
    if (MODE != GROUPED_TN && a.K * (int64_t)ES % 16 && a.K < 64 / ES) return false;
    if (MODE != GROUPED_NT && a.N % 8 && a.N < BN) return false;
    return MODE != GROUPED_TN || a.M % 8 == 0 || a.M >= 128;
}

// Whether the strips can: as above, with their own widths.
template <GroupedType T, int MODE>
bool by_strips(const GroupedArgs& a) {
    constexpr int ES = T == GroupedType::I8 ? 1 : 2, KT = MODE == GROUPED_NT ? 128 : 64;
    if (a.lda_b >= (1 << 23) || a.ldb_b >= (1 << 23)) return false;
    if (MODE != GROUPED_TN && (a.K == 0 || (a.K * (int64_t)ES % 16 && a.K < KT / ES))) return false;
    if (MODE != GROUPED_NT && a.N % 8 && a.N < 64) return false;
    return MODE != GROUPED_TN || a.M % 8 == 0 || a.M >= 64;
}

template <GroupedType T, int MODE, int MT>
hipError_t launch_few(const GroupedArgs& a, hipStream_t stream) {
    const int64_t groups = grouped_tiles(MODE, a, 32 * MT, 64);
    grouped_few_kernel<T, MODE, MT><<<dim3((unsigned)groups), dim3(256), 0, stream>>>(a);
    return hipGetLastError();
}

template <GroupedType T, int MODE>
hipError_t launch_mode(const GroupedArgs& a, hipStream_t stream) {
    constexpr int64_t ES = T == GroupedType::I8 ? 1 : 2;
    if constexpr (MODE == GROUPED_TN) {
        // Tiles for less than half of the CUs: 64 x 64, each summed by four waves (12357 rows
        // of 2 groups into 768 x 320, 18 tiles: 28 us, 78 by tiles; 16000 rows of 2 into 1001 x
        // 1001, 64 tiles: 90 and 116; 8192 rows of 4 into 1024 x 1024, 128 tiles: 36 and 34)
        if (grouped_tiles(MODE, a, 128, BN) < CUS / 2 && by_strips<T, MODE>(a)) return launch_few<T, MODE, 2>(a, stream);
        if (!by_tiles<T, MODE>(a)) return launch_any<T, MODE>(a, stream);
        grouped_half_kernel<T, MODE><<<dim3((unsigned)grouped_tiles(MODE, a, 128, BN)), dim3(256), 0, stream>>>(a);
    } else {
        // Too few tiles of 64 rows for half of the CUs: strips (512 rows of 4 groups of 2048 x
        // 2048, 96 tiles: 16 us, 31 by tiles; 1024 rows, 160 tiles: 26 either way), two blocks
        // of 32 rows where one would often not do.
        const int64_t low = most_row_tiles(a, 64) * ((a.N + BN - 1) / BN);
        if (low <= CUS / 2 && by_strips<T, MODE>(a))
            return a.rows > 20 * (int64_t)a.groups ? launch_few<T, MODE, 2>(a, stream) : launch_few<T, MODE, 1>(a, stream);
        if (!by_tiles<T, MODE>(a)) return launch_any<T, MODE>(a, stream);
        if constexpr (MODE == GROUPED_NN) {
            // Few rows to a group (128 rows of 16 groups of 4096 x 4096: 86 us, 91 by the larger
            // tiles; 1536 rows: 161 and 101)
            if (a.rows <= 48 * (int64_t)a.groups) {
                grouped_low_kernel<T><<<dim3((unsigned)low), dim3(256), 0, stream>>>(a);
                return hipGetLastError();
            }
        }
        // (Averages are all that is known here.  One group with all rows among 63 empty ones of 2048
        // x 1408: 1200 rows 26 us, 24 where it is the only group; 3000 rows 37 and 35; 8000 57 and 56)
        //
        // Short sums, and somewhat longer ones where all tiles run at once (16384 rows of 16
        // groups of 768 x 2048: 60 us, 67 by the larger tiles; of 4 groups of 128 x 4096 39 and 59;
        // of 8 groups of 512 x 14336 310 and 352; INT8, 9651 rows of 3 groups of 1280 x 5888 116
        // and 132; 3001 rows of 11 groups of 1003 x 1501 24 and 26.  But 16384 rows of 8 groups of
        // 1000 x 14336, with B^T: 804 and 640)
        const int64_t halves = grouped_tiles(MODE, a, 128, BN);
        if (a.K > 0 && a.K * ES <= (halves <= 2 * CUS ? 2048 : 1536)) {
            const int64_t groups = halves + NUM_XCD;
            grouped_half_kernel<T, MODE><<<dim3((unsigned)groups), dim3(256), 0, stream>>>(a);
            return hipGetLastError();
        }
        grouped_tile_kernel<T, MODE><<<dim3((unsigned)tile_workgroups(a)), dim3(256), 0, stream>>>(a);
    }
    return hipGetLastError();
}

template <GroupedType T>
hipError_t launch_type(int mode, const GroupedArgs& a, hipStream_t stream) {
    if constexpr (T == GroupedType::I8) return launch_mode<T, GROUPED_NT>(a, stream);
    else
        return mode == GROUPED_NN ? launch_mode<T, GROUPED_NN>(a, stream)
               : mode == GROUPED_NT ? launch_mode<T, GROUPED_NT>(a, stream) : launch_mode<T, GROUPED_TN>(a, stream);
}

}  // namespace

static_assert(NUM_XCD == 8, "as layer_sizes.hpp counts");
bool grouped_fits(int mode, const GroupedArgs& a) { return tiles_fit(mode, a); }

hipError_t launch_grouped(GroupedType type, int mode, const GroupedArgs& a, hipStream_t stream) {
    switch (type) {
        case GroupedType::BF16: return launch_type<GroupedType::BF16>(mode, a, stream);
        case GroupedType::F16: return launch_type<GroupedType::F16>(mode, a, stream);
        default: return launch_type<GroupedType::I8>(mode, a, stream);
    }
}

}  // namespace mpdt
