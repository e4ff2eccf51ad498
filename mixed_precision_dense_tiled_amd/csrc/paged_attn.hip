// paged_attn.hip -- attention of new tokens over a paged key/value cache.
//
// For sequence b with n keys and nq new tokens (the last nq of the n), token
// t stands at position p = n - nq + t and sees the keys j <= p, with a window
// w only those with j > p - w.  With s_j = scale * (q . k_j), capped to
// cap * tanh(s_j / cap) on request,
//     out = sum_j exp(s_j) v_j / sum_j exp(s_j),   lse = log sum_j exp(s_j);
// a token that sees no key gets out = 0 and lse = -inf.
//
// The work is cut into units (a tile of rows of one KV head; a row is one
// token and one of the query heads that share the KV head) and each unit's
// keys into tiles.  All tiles of all units stand in one line, which the
// workgroups share evenly: each works out the line for itself, or in large
// batches a plan kernel writes it down (lengths are known on the device only),
// each workgroup walks its stretch with a running
// maximum and sum per row, and units that several workgroups share are joined
// by a last kernel.  Batches whose cache rows are short run in one launch,
// one workgroup to a unit.
//
// Two kernels walk the tiles.  Few rows per sequence (single tokens): 16 rows
// by 32 keys on 16x16x32 MFMAs, each wave with key tiles and an LDS ring of its
// own, bound by the cache's bytes.  Many rows (chunks of a prompt): 256 rows by
// 64 keys on 32x32x16 MFMAs, K and V shared by the workgroup, bound by the
// matrix cores and the exponentials.  Both form S^T = K Q^T, so that a lane
// holds scores of a single row: the running maximum and sum are one register
// per row, and the MFMA's output layout is already the operand layout of
// O^T = V^T P^T once V's keys are read in the same order (the transposing LDS
// reads take any order of rows).
//
// Scores, maxima, sums and outputs are FP32.  P is rounded to the type that
// the second MFMA takes (FP16 for FP16 and FP8 caches, BF16 for BF16): single tokens
// in two parts, 16 bits of it and more, which costs no time there; chunks once, as the
// second part would be half again as many MFMAs where these are the bound: one
// rounding per weight, independent from key to key, where the sum of the weights
// keeps them unrounded.  FP8 keys and values are widened exactly;
// their scales are per head and join the score's scale and the output.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "device_common.hpp"
#include "gemm_common.hpp"
#include "serving.hpp"

namespace mpdt {
namespace {

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr float NO_MAX = -3e38f;      // reference of a row that has seen no key: no score lies below
constexpr float FAR = 1048576.0f;     // 2^20: a rounding of 2^-5
constexpr float RESCALE = 8.0f;       // a row's reference moves when its maximum has outgrown it by 2^8
constexpr int PAGES_LDS = 1024;       // page numbers of a stretch held in LDS

typedef __attribute__((ext_vector_type(2))) float f32x2;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(2))) _Float16 f16x2;

// ---- element types ----------------------------------------------------------

struct Bf16 {
    using vec8 = bf16x8;
    static constexpr float P_SHIFT = 0.0f;
    static __device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
    static __device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        bf16x2 r;
        r[0] = (__bf16)a;
        r[1] = (__bf16)b;
        return __builtin_bit_cast(uint32_t, r);
    }
    static __device__ __forceinline__ uint32_t from_fp8_lo(uint32_t w) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
    }
    static __device__ __forceinline__ uint32_t from_fp8_hi(uint32_t w) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true));
    }
    static __device__ __forceinline__ f32x4 mma16(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x16 mma32(u32x4 a, u32x4 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
};

struct F16 {
    // FP16 weights sit 2^7 higher (at most 2^15 with the lazy reference), so
    // that small ones stay clear of the subnormals; the sum carries the same
    // factor and it cancels.
    static constexpr float P_SHIFT = 7.0f;
    static __device__ __forceinline__ float low(uint32_t w) { return (float)__builtin_bit_cast(f16x2, w)[0]; }
    static __device__ __forceinline__ float high(uint32_t w) { return (float)__builtin_bit_cast(f16x2, w)[1]; }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        f16x2 r;
        r[0] = (_Float16)a;
        r[1] = (_Float16)b;
        return __builtin_bit_cast(uint32_t, r);
    }
    static __device__ __forceinline__ uint32_t from_fp8_lo(uint32_t w) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false));
    }
    static __device__ __forceinline__ uint32_t from_fp8_hi(uint32_t w) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true));
    }
    static __device__ __forceinline__ f32x4 mma16(u32x4 a, u32x4 b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x16 mma32(u32x4 a, u32x4 b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    }
};

// 8 FP8 values widened to 8 16-bit ones.
template <class E>
__device__ __forceinline__ u32x4 widen8(u32x2 w) {
    return u32x4{E::from_fp8_lo(w[0]), E::from_fp8_hi(w[0]), E::from_fp8_lo(w[1]), E::from_fp8_hi(w[1])};
}

// ---- the staged rows of K and V in LDS ---------------------------------------
//
// A row is CH chunks of 16 bytes (DP elements, padded to 8 chunks for 96 FP8
// values); chunk c of row r lies at place c ^ swz(r).  LDS has 64 banks of 4
// bytes: 16 places.  A cycle serves 16 lanes of a 16-byte read of K (16 rows,
// one chunk) and 32 lanes of an 8-byte transposing read of V (4 or 8 rows, 64
// or 32 bytes side by side; 16 rows of 16 bytes of FP8 at MF = 16), and the
// swizzles below spread each of these sets over all 16 places.  MF: rows of an
// MFMA tile (16 or 32), which decides the rows that a read of V names.
template <int DP, bool KV8, int MF>
struct Rows {
    static constexpr int CH = KV8 ? (DP <= 64 ? 4 : 8) : DP / 8;
    static constexpr int BYTES = CH * 16;
    static __device__ __forceinline__ int swz_k(int r) {
        if constexpr (CH == 16) return r & 15;
        if constexpr (CH == 8) return (r >> 1) & 7;
        return (r >> 2) & 3;                              // 12 (rows start at 4 places in turn), 4
    }
    static __device__ __forceinline__ int swz_v(int r) {
        if constexpr (KV8 && MF == 32) {                  // rows 0..3 and 8..11
            if constexpr (CH == 8) return ((r >> 1) & 1) << 1 | ((r >> 3) & 1) << 2;
            return ((r >> 3) & 1) << 1;
        }
        if constexpr (KV8) {                              // rows 0..7 and 16..23
            if constexpr (CH == 8) return ((r >> 1) & 3) | ((r >> 4) & 1) << 2;
            return ((r >> 2) & 1) | ((r >> 4) & 1) << 1;
        }
        if constexpr (MF == 32) {                         // rows 0..3, 64 bytes
            if constexpr (CH == 16) return (r & 3) << 2;
            if constexpr (CH == 8) return ((r >> 1) & 1) << 2;
            return 0;
        }
        if constexpr (CH == 16) return (r & 7) << 1;      // rows 0..7, 32 bytes
        if constexpr (CH == 8) return ((r >> 1) & 3) << 1;
        return ((r >> 2) & 1) << 1;
    }
};

// 16 bytes per lane straight into LDS: lane l's land at dst + 16 * l.  As the
// buffer form in device_common.hpp, from 64-bit addresses.
__device__ __forceinline__ void global_to_lds16(const char* src, MPDT_LDS char* dst) {
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 :
                 : "{m0}"((uint32_t)(uintptr_t)dst), "v"((uint64_t)(uintptr_t)src));
}

// The same from a scalar base and a 32-bit offset per lane.  ONCE: the bytes
// are read once (non-temporal), by all but sequences of more than 16 rows.
template <bool ONCE = false>
__device__ __forceinline__ void global_to_lds16(const char* base, uint32_t off, MPDT_LDS char* dst) {
    if constexpr (ONCE)
        asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2 nt"
                     :
                     : "{m0}"((uint32_t)(uintptr_t)dst), "v"(off), "s"((uint64_t)(uintptr_t)base));
    else
        asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                     :
                     : "{m0}"((uint32_t)(uintptr_t)dst), "v"(off), "s"((uint64_t)(uintptr_t)base));
}

__device__ __forceinline__ u32x2 lds_load8(const MPDT_LDS char* base, uint32_t off) {
    return *reinterpret_cast<const MPDT_LDS u32x2*>(base + off);
}

// A value that every lane of the wave has, told to the compiler: numbers read
// from memory would otherwise live in vector registers, and all that depends
// on them.
__device__ __forceinline__ int uni(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ float uni(float x) {
    return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(x)));
}

// ---- sequences, units and the plan --------------------------------------------

// A sequence that the whole wave works on.
__device__ __forceinline__ Seq uniform_seq(const SeqView& v, int64_t page_size, int b) {
    const Seq s = seq_of(v, page_size, b);
    return Seq{uni(s.start), uni(s.nq), uni(s.n)};
}

// Keys [lo, hi) that any of the rows [r0, r1) of a sequence sees.
struct Span32 {
    int lo, hi;
};
__device__ __forceinline__ Span32 keys_of(const Seq& s, int group, int window, int r0, int r1) {
    const int t0 = r0 / group, t1 = (r1 - 1) / group, past = s.n - s.nq;
    Span32 k;
    k.hi = min(max(past + t1 + 1, 0), s.n);
    k.lo = window > 0 ? max(past + t0 + 1 - window, 0) : 0;
    if (k.lo >= k.hi) k.lo = k.hi = 0;
    return k;
}

// The unit that a worker begins and leaves to others (b < 0: none): what the
// joining launch has to know.
struct Cut {
    int32_t b, h, r0, tiles;
    int64_t u0, share;      // the unit's first tile in the line; tiles to a worker
};

// The plan in the workspace: head[0] entries (row tiles), head[1] key tiles
// of all entries, then per entry {sequence, first row, first key tile, key
// tiles} and the key tiles before it.  A KV head repeats the line once more.
struct Plan {
    int32_t* head;
    i32x4* entry;
    int32_t* before;
    int32_t* first;     // row tiles before a sequence
    char* zeros;        // 16 bytes
    Cut* cut;           // per worker
    float* part_o;      // partial outputs, two slots to a worker
    f32x2* part_ml;     // their reference and sum
};

__host__ __device__ inline int64_t up256(int64_t x) { return (x + 255) / 256 * 256; }

__host__ __device__ inline int64_t plan_layout(char* ws, int entries, int seqs, int workers, int tile_rows,
                                               int dp, Plan* p) {
    int64_t at = 0;
    p->head = (int32_t*)(ws + at);
    p->zeros = ws + 128;
    at += 256;
    p->entry = (i32x4*)(ws + at);
    at += up256((int64_t)entries * 16);
    p->before = (int32_t*)(ws + at);
    at += up256(((int64_t)entries + 1) * 4);
    p->first = (int32_t*)(ws + at);
    at += up256(((int64_t)seqs + 1) * 4);
    p->cut = (Cut*)(ws + at);
    at += up256((int64_t)workers * (int64_t)sizeof(Cut));
    p->part_ml = (f32x2*)(ws + at);
    at += up256((int64_t)workers * 2 * tile_rows * 8);
    p->part_o = (float*)(ws + at);
    at += up256((int64_t)workers * 2 * tile_rows * dp * 4);
    return at;
}

// Exclusive sum over the workgroup's threads; total to all.  red: one int a wave.
template <int WAVES>
__device__ __forceinline__ int block_scan(int x, int* red, int& total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int s = x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int y = __shfl_up(s, d);
        if (lane >= d) s += y;
    }
    if (lane == 63) red[wave] = s;
    __syncthreads();
    int base = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        const int r = red[w];
        if (w < wave) base += r;
        total += r;
    }
    __syncthreads();
    return base + s - x;
}

// Entry e of sequence b, its first key tile and key tiles.
__device__ __forceinline__ i32x4 entry_of(const AttnArgs& a, const Seq& s, int b, int r0, int key_tile) {
    const Span32 k = keys_of(s, a.group, a.window, r0, min(r0 + a.tile_rows, s.nq * a.group));
    const int t0 = k.lo / key_tile;
    return i32x4{b, r0, t0, max((k.hi + key_tile - 1) / key_tile - t0, 1)};
}

__global__ __launch_bounds__(1024) void attn_plan_kernel(AttnArgs a, int key_tile) {
    __shared__ int red[16];
    Plan p;
    plan_layout(a.ws, a.entries, a.sv.seqs, a.workers, a.tile_rows, 0, &p);
    int run = 0;
    for (int b0 = 0; b0 < a.sv.seqs; b0 += 1024) {
        const int b = b0 + threadIdx.x;
        int c = 0;
        if (b < a.sv.seqs) {
            const Seq s = seq_of(a.sv, a.kv.page_size, b);
            c = (int)(((int64_t)s.nq * a.group + a.tile_rows - 1) / a.tile_rows);
        }
        int total;
        const int at = run + block_scan<16>(c, red, total);
        if (b < a.sv.seqs) p.first[b] = at;
        run += total;
    }
    const int entries = min(run, a.entries);
    __syncthreads();
    int tiles = 0;
    for (int e0 = 0; e0 < entries; e0 += 1024) {
        const int e = e0 + threadIdx.x;
        i32x4 ent{0, 0, 0, 0};
        if (e < entries) {
            int lo = 0, hi = a.sv.seqs;      // the last sequence whose first row tile is at most e
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (p.first[mid] <= e) lo = mid;
                else hi = mid;
            }
            const Seq s = seq_of(a.sv, a.kv.page_size, lo);
            ent = entry_of(a, s, lo, (e - p.first[lo]) * a.tile_rows, key_tile);
        }
        int total;
        const int at = tiles + block_scan<16>(ent[3], red, total);
        if (e < entries) {
            p.entry[e] = ent;
            p.before[e] = at;
        }
        tiles += total;
    }
    if (threadIdx.x == 0) {
        p.before[entries] = tiles;
        p.head[0] = entries;
        p.head[1] = tiles;
    }
}

// The plan of a small batch, which every workgroup works out for itself in LDS
// (at most NEAR sequences and entries): a launch of its own and the way of its
// numbers through memory cost about 9 us before the first key is read.
constexpr int NEAR = 256;
struct NearPlan {
    i32x4 entry[NEAR];
    Seq seq[NEAR];
    int before[NEAR + 1], first[NEAR];
};

// Plan as the workers see it.
struct Line {
    const NearPlan& near;
    const Plan& far;
    bool is_near;
    int entries, tiles;
    __device__ __forceinline__ i32x4 entry(int e) const {
        const i32x4 x = is_near ? near.entry[e] : far.entry[e];
        return i32x4{uni(x[0]), uni(x[1]), uni(x[2]), uni(x[3])};
    }
    __device__ __forceinline__ int before(int e) const { return uni(is_near ? near.before[e] : far.before[e]); }
    // The entry that holds a tile.
    __device__ __forceinline__ int find(int tile) const {
        int lo = 0, hi = entries;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (before(mid) <= tile) lo = mid;
            else hi = mid;
        }
        return lo;
    }
};

template <int WAVES>
__device__ __forceinline__ void make_line(const AttnArgs& a, int key_tile, NearPlan& n, int* red, Line& line) {
    if (!line.is_near) {
        line.entries = uni(line.far.head[0]);
        line.tiles = uni(line.far.head[1]);
        return;
    }
    const int t = threadIdx.x;
    int c = 0, run, tiles;
    if (t < a.sv.seqs) {
        n.seq[t] = seq_of(a.sv, a.kv.page_size, t);
        c = (int)(((int64_t)n.seq[t].nq * a.group + a.tile_rows - 1) / a.tile_rows);
    }
    const int at = block_scan<WAVES>(c, red, run);
    if (t < a.sv.seqs) n.first[t] = at;
    const int entries = min(run, a.entries);
    __syncthreads();
    i32x4 ent{0, 0, 0, 0};
    if (t < entries) {
        int lo = 0, hi = a.sv.seqs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (n.first[mid] <= t) lo = mid;
            else hi = mid;
        }
        ent = entry_of(a, n.seq[lo], lo, (t - n.first[lo]) * a.tile_rows, key_tile);
        n.entry[t] = ent;
    }
    const int before = block_scan<WAVES>(ent[3], red, tiles);
    if (t < entries) n.before[t] = before;
    __syncthreads();
    line.entries = uni(entries);
    line.tiles = uni(tiles);
}

// Key tiles to a worker.
__device__ __forceinline__ int64_t share_of(const AttnArgs& a, int64_t total) {
    return max((total + a.workers - 1) / a.workers, (int64_t)a.min_tiles);
}

// Numbers of this workgroup's stretch: consecutive stretches run on one XCD
// (workgroups go to the 8 XCDs in turn), so units of one KV head share an L2.
__device__ __forceinline__ int worker_id() {
    const int w = gridDim.x;
    return w % 8 ? (int)blockIdx.x : (int)(blockIdx.x % 8) * (w / 8) + (int)(blockIdx.x / 8);
}

// Row tile `e` of a batch without a plan: all threads of the workgroup look
// for the sequence that holds it (-1: none) and the tile's first row.
template <int WAVES>
__device__ __forceinline__ void find_entry(const AttnArgs& a, int e, int* red, int* box, int& b, int& r0,
                                           Seq& s) {
    if (a.sv.seqs <= 64) {
        // every wave for itself: one sequence a lane
        const int lane = threadIdx.x & 63;
        int c = 0;
        Seq mine{0, 0, 0};
        if (lane < a.sv.seqs) {
            mine = seq_of(a.sv, a.kv.page_size, lane);
            c = (int)(((int64_t)mine.nq * a.group + a.tile_rows - 1) / a.tile_rows);
        }
        int upto = c;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int y = __shfl_up(upto, d);
            if (lane >= d) upto += y;
        }
        const uint64_t in = __ballot(e >= upto - c && e < upto);
        b = in ? __builtin_ctzll(in) : -1;
        if (!in) return;
        r0 = (e - __builtin_amdgcn_readlane(upto - c, b)) * a.tile_rows;
        s = Seq{__builtin_amdgcn_readlane(mine.start, b), __builtin_amdgcn_readlane(mine.nq, b),
                __builtin_amdgcn_readlane(mine.n, b)};
        return;
    }
    if (threadIdx.x == 0) box[0] = -1;
    __syncthreads();
    int run = 0;
    for (int b0 = 0; b0 < a.sv.seqs; b0 += WAVES * 64) {
        const int i = b0 + threadIdx.x;
        int c = 0;
        if (i < a.sv.seqs) {
            const Seq s = seq_of(a.sv, a.kv.page_size, i);
            c = (int)(((int64_t)s.nq * a.group + a.tile_rows - 1) / a.tile_rows);
        }
        int total;
        const int at = run + block_scan<WAVES>(c, red, total);
        if (e >= at && e < at + c) {
            box[0] = i;
            box[1] = (e - at) * a.tile_rows;
        }
        run += total;
        if (run > e) break;
    }
    __syncthreads();
    b = uni(box[0]);
    r0 = uni(box[1]);
    if (b >= 0) s = uniform_seq(a.sv, a.kv.page_size, b);
}

// The byte offsets of the pages that hold the keys from key tile `tile` on,
// into LDS (-1: no such page); returns the tile up to which they reach (at most
// `end`).  clean: all of them exist.  Called by all threads.
template <int NT, int KT>
__device__ __forceinline__ int fetch_pages(const AttnArgs& a, int b, int tile, int end, int64_t* pages, int& first,
                                           bool* clean = nullptr) {
    const int64_t k0 = (int64_t)tile * KT, ps = a.kv.page_size;
    first = (int)(k0 / ps);
    const int64_t reach = ((int64_t)first + PAGES_LDS) * ps / KT;
    const int stop = (int)min((int64_t)end, reach);
    const int last = (int)min(((int64_t)stop * KT - 1) / ps, (int64_t)a.sv.width - 1);
    const int32_t* row = a.sv.table + (int64_t)b * a.sv.ld_table;
    int bad = 0;
    for (int i = threadIdx.x; i <= last - first; i += NT) {
        const int pg = row[first + i];
        const bool ok = pg >= 0 && pg < a.kv.pages;
        pages[i] = ok ? pg * a.kv.page_b : -1;
        bad |= !ok;
    }
    bad = __syncthreads_or(bad);
    if (clean) *clean = !uni(bad);
    return stop;
}

// Place of a key: its page's entry and its slot.
struct Place {
    int entry, slot;
};
__device__ __forceinline__ Place place_of(const PagedKV& kv, int first, int key) {
    const int pi = kv.page_of(key);
    return Place{pi - first, key - pi * kv.page_size};
}

// Byte offset of a key's row in the cache, and whether there is such a key.
__device__ __forceinline__ bool key_offset(const PagedKV& kv, const int64_t* pages, int first, int key, int lo,
                                           int hi, int64_t& off) {
    const Place p = place_of(kv, first, key);
    const int64_t pg = key >= lo && key < hi ? pages[p.entry] : -1;
    off = pg >= 0 ? pg + p.slot * kv.slot_b : 0;
    return pg >= 0;
}

__device__ __forceinline__ int64_t shfl64(int64_t v, int lane) {
    const int lo = __shfl((int)(uint32_t)v, lane), hi = __shfl((int)(v >> 32), lane);
    return (int64_t)(((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo);
}

// a - b of a rounded product a: as one operation with it the difference of two large
// equal scores would be the product's rounding, not zero.
__device__ __forceinline__ float minus(float a, float b) {
#pragma clang fp contract(off)
    return a - b;
}

// The larger of this lane's value and that of the lane 32 (16) on: a swap of
// register halves instead of a way through LDS.
__device__ __forceinline__ float across32(float m) {
    const u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(__float_as_uint(m), __float_as_uint(m), false, false));
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float across16(float m) {
    const u32x2 r = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(__float_as_uint(m), __float_as_uint(m), false, false));
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// Bits first to last (both may lie outside 0 to 63) of a 64-bit word.
__device__ __forceinline__ uint64_t from_to(int first, int last) {
    const uint64_t upto = last >= 63 ? ~0ull : last < 0 ? 0 : (2ull << last) - 1;
    const uint64_t below = first >= 64 ? ~0ull : first <= 0 ? 0 : (1ull << first) - 1;
    return upto & ~below;
}

// Score in base-2 logarithms: s * mul, or capped: cap tanh(y), y = s * scale / cap.
struct Score {
    float mul, cap2, inner;   // inner: 2 * log2(e) * scale / cap
};
__device__ __forceinline__ Score score_of(const AttnArgs& a, float k_scale) {
    Score s;
    s.mul = a.scale * k_scale * LOG2E;
    s.cap2 = fminf(a.softcap * LOG2E, 3e38f);
    s.inner = a.softcap > 0.0f ? 2.0f * LOG2E * a.scale * k_scale / a.softcap : 0.0f;
    // (held finite, so that a product of zero stays a score of zero; NaN stays)
    s.inner = s.inner > 3e38f ? 3e38f : s.inner < -3e38f ? -3e38f : s.inner;
    return s;
}
// How scores are capped.  CAP_ANY, right for every cap: from |y| = 1/2 on tanh(y) = 1 -
// 2 / (exp(2 y) + 1), both ends of which saturate; below, where that difference
// would leave an error of the cap's size in a score near zero, y T(y^2), T of degree 4
// in z^2 with z = 2 log2(e) y, fitted at Chebyshev nodes over |y| <= 1/2 (off by
// 2^-25), times the score itself, so that a cap however large only lets the score
// through.  CAP_NEAR: the first form alone, whose error of up to 2^-22 of the cap is, up
// to CAP_NEAR_MOST, 2^-16 of a weight, 1/16 of its rounding to FP16.  The kernel of
// few rows waits for memory and takes CAP_ANY throughout (64 sequences: 198 us with
// either); the kernel of many rows waits for its softmax (17 sequences in FP16,
// dim 64: CAP_NEAR 126 us, CAP_ANY 148 under a cap of 100, 179 where every
// score passes 1/2).
enum : int { CAP_NONE = 0, CAP_NEAR = 1, CAP_ANY = 2 };
constexpr float CAP_NEAR_MOST = 64.0f;
constexpr float CAP_SMALL = LOG2E;     // |z| at |y| = 1/2
__device__ __forceinline__ float score_exp(const Score& c, float z) {
    return fmaf(-2.0f * c.cap2, __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(z) + 1.0f), c.cap2);
}
__device__ __forceinline__ float score_small(const Score& c, float s, float z) {
    const float x = z * z;
    float t = fmaf(x, 3.565785164028057e-06f, -9.181624045595527e-05f);
    t = fmaf(x, t, 0.001922387513332069f);
    t = fmaf(x, t, -0.040037430822849274f);
    t = fmaf(x, t, 1.0f);
    return s * c.mul * t;
}
// N scores of a lane, capped in place; CAP_ANY four at a time (all side by side would
// hold several registers a score), the exponentials only where one of the wave's
// four reaches 1/2.
template <int CAP, int N>
__device__ __forceinline__ void cap_scores(const Score& c, float (&s)[N]) {
    if constexpr (CAP == CAP_NEAR) {
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = score_exp(c, s[i] * c.inner);
        return;
    }
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        float z[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            z[j] = s[i + j] * c.inner;
            s[i + j] = score_small(c, s[i + j], z[j]);
        }
        const float most = fmaxf(fmaxf(fabsf(z[0]), fabsf(z[1])), fmaxf(fabsf(z[2]), fabsf(z[3])));
        if (__ballot(most >= CAP_SMALL)) {
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i + j] = fabsf(z[j]) >= CAP_SMALL ? score_exp(c, z[j]) : s[i + j];
        }
    }
}

// Four outputs of a row from d on, rounded once to the type of q.
__device__ __forceinline__ void store_out4(const AttnArgs& a, char* row, int d, f32x4 v) {
    u32x2 w;
    if (a.q_type == DT_BF16) {
        w = u32x2{Bf16::pack(v[0], v[1]), Bf16::pack(v[2], v[3])};
    } else {
        w = u32x2{F16::pack(v[0], v[1]), F16::pack(v[2], v[3])};
    }
    *reinterpret_cast<u32x2*>(row + 2 * d) = w;
}

__device__ __forceinline__ float lse_of(float ref, float sum) {
    return sum > 0.0f || sum != sum ? (ref + __builtin_amdgcn_logf(sum)) * LN2 : -__builtin_inff();
}

// ---- few rows: 16 rows by 32 keys a wave ----------------------------------------
//
// Bound by the cache's bytes: 64 sequences of 700 to 8000 keys, 8 KV heads of 128
// in BF16 (1.14 GB): 203 us a pass, 5.6 TB/s; 8 of 9000 to 65000 keys in FP8
// (0.61 GB): 116 us, 5.2 TB/s; a plain stream of 1 GiB reads at 6.7.  Each wave
// keeps a ring of its own, so nothing but its own loads holds it up: 64 to 128 KB
// a CU are in flight.  Non-temporal loads took the kernels from 220 to 200 and from
// 116 to 103 us.
// One sequence of 517 keys and 8 KV heads is eight workgroups on one memory round
// trip after another (numbers, page table, keys): 9 us.

constexpr int DEC_ROWS = 16, DEC_KEYS = 32;
constexpr int DEC_LDS = 128 * 1024;       // rings of a workgroup

// Waves of a workgroup: eight with one or two stages each over 16-bit caches (64
// sequences of dim 128: 203 us against 215 of four waves with twice the stages;
// dim 64: 122 against 133) and where a workgroup has a unit to itself; four over
// FP8 (two stages more a wave: 116 us against 122).
constexpr int dec_waves(bool kv8, bool direct) { return direct || !kv8 ? 8 : 4; }

template <bool KV8, int DP, int WAVES>
struct Dec {
    using R = Rows<DP, KV8, 16>;
    static constexpr int HALF = DEC_KEYS * R::BYTES;         // K rows, then V rows
    static constexpr int STAGE = 2 * HALF;
    static constexpr int FIT = DEC_LDS / (WAVES * STAGE), NST = FIT > 4 ? 4 : FIT;
    static constexpr int LOADS = 2 * DEC_KEYS * R::CH / 64;  // direct loads of a stage
    static constexpr int RING = NST * STAGE;
    static constexpr int OROW = DP * 4 + 16;                 // bytes of a row of outputs in LDS
    static_assert(DEC_ROWS * OROW <= RING, "a wave's outputs fit its ring");
    static_assert((NST - 1) * LOADS < 64, "vmcnt range");
};

// A wave's loads of its key tiles.
template <bool KV8, int DP, int WAVES>
struct DecLoads {
    using D = Dec<KV8, DP, WAVES>;
    using R = typename D::R;
    static constexpr int PER16 = R::CH / 4;      // loads of 16 keys, K or V
    const AttnArgs& a;
    const char *kb, *vb;         // K and V of the head
    const int64_t* pages;
    int first, lo, hi;
    bool fast;                   // pages hold a multiple of 16 tokens, and all of them exist
    uint32_t own_k[PER16], own_v[2][PER16];      // fast: a lane's offset in a load of 16 keys

    __device__ __forceinline__ DecLoads(const AttnArgs& a_, const char* k, const char* v, const int64_t* p)
        : a(a_), kb(k), vb(v), pages(p) {
        static_for<0, PER16>([&](auto i) {
            constexpr int I = decltype(i)::value;
            const int c = I * 64 + (threadIdx.x & 63), r = c / R::CH, pos = c % R::CH;
            const uint32_t row = (uint32_t)(r * a.kv.slot_b);
            own_k[I] = row + in_row((pos ^ R::swz_k(r)) * 16);
            own_v[0][I] = row + in_row((pos ^ R::swz_v(r)) * 16);
            own_v[1][I] = row + in_row((pos ^ R::swz_v(r + 16)) * 16);
        });
    }
    __device__ __forceinline__ int in_row(int from) const {      // (dim below DP: any bytes of the row)
        return from >= a.kv.dim * (KV8 ? 1 : 2) ? 0 : from;
    }

    // Issues the loads of key tile `tile`; returns which of its 32 keys exist.
    // Keys that do not exist are staged as copies of one that does (their weight
    // is zero), so that the count of loads is fixed.
    __device__ __forceinline__ uint32_t issue(int tile, MPDT_LDS char* dst) const {
        const int key0 = tile * DEC_KEYS;
        if (fast && key0 >= lo && key0 + DEC_KEYS <= hi) {
            // 16 keys lie in one page: scalar addresses
            static_for<0, 2>([&](auto gc) {
                constexpr int G = decltype(gc)::value;
                const int key = key0 + 16 * G, pi = a.kv.page_of(key);
                const int64_t e = pages[pi - first];
                const int64_t pg = (int64_t)((uint64_t)(uint32_t)uni((int)(e >> 32)) << 32 | (uint32_t)uni((int)e)) +
                                   (key - pi * a.kv.page_size) * a.kv.slot_b;
                static_for<0, PER16>([&](auto i) {
                    constexpr int I = decltype(i)::value;
                    MPDT_LDS char* to = dst + (G * PER16 + I) * 1024;
                    global_to_lds16<true>(kb + pg, own_k[I], to);
                    global_to_lds16<true>(vb + pg, own_v[G][I], to + D::HALF);
                });
            });
            return 0xffffffffu;
        }
        const int lane = threadIdx.x & 63;
        int64_t off;
        const bool ok = key_offset(a.kv, pages, first, key0 + (lane & 31), lo, hi, off);
        const uint32_t mask = (uint32_t)__ballot(ok);
        if (mask != 0xffffffffu) {
            const int64_t other = shfl64(off, mask ? __builtin_ctz(mask) : 0);
            if (!ok) off = other;
        }
#pragma unroll 1
        for (int i = 0; i < 2 * PER16; ++i) {
            const int c = i * 64 + lane, r = c / R::CH, pos = c % R::CH;
            const int64_t o = shfl64(off, r);
            global_to_lds16(kb + o + in_row((pos ^ R::swz_k(r)) * 16), dst + i * 1024);
            global_to_lds16(vb + o + in_row((pos ^ R::swz_v(r)) * 16), dst + D::HALF + i * 1024);
        }
        return mask;
    }
};

template <class E, class EP, bool KV8, int DP, int CAP, int WAVES>
__device__ __forceinline__ void dec_tile(const MPDT_LDS char* st, const u32x4 (&qf)[DP / 32], const Score& sc,
                                         int dim, uint32_t mask, bool edge, int key0, int qpos, int qlow,
                                         float& ref, float& sum, f32x4 (&o)[DP / 16]) {
    using D = Dec<KV8, DP, WAVES>;
    using R = typename D::R;
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    // All of K's operands are asked for before the first MFMA, and all of V's
    // before the softmax (left to itself the compiler asks for one, waits out
    // the LDS latency, and uses it).
    f32x4 s[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
    u32x4 kf[2][DP / 32];
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            const int r = 16 * ks + n;
            if constexpr (KV8) {
                const u32x2 w = lds_load8(st, r * R::BYTES + ((2 * d + (g >> 1)) ^ R::swz_k(r)) * 16 + (g & 1) * 8);
                kf[ks][d][0] = w[0];
                kf[ks][d][1] = w[1];
            } else {
                kf[ks][d] = lds_load16(st, r * R::BYTES + ((4 * d + g) ^ R::swz_k(r)) * 16);
            }
        }
    const MPDT_LDS char* sv = st + D::HALF;
    u32x4 vf[DP / 16];
#pragma unroll
    for (int t = 0; t < DP / 16; ++t) {
        if constexpr (KV8) {
            const int h = n >> 1, r = (h < 4 ? 4 * g + h : 16 + 4 * g + h - 4);
            const u32x2 w = lds_read_tr8(sv, r * R::BYTES + (t ^ R::swz_v(r)) * 16 + (n & 1) * 8);
            vf[t][0] = w[0];
            vf[t][1] = w[1];
        } else {
            const int r = 4 * g + (n >> 2), c = 2 * t + ((n & 3) >> 1), b = (n & 1) * 8;
            const u32x2 v0 = lds_read_tr16(sv, r * R::BYTES + (c ^ R::swz_v(r)) * 16 + b);
            const u32x2 v1 = lds_read_tr16(sv, (r + 16) * R::BYTES + (c ^ R::swz_v(r + 16)) * 16 + b);
            vf[t] = u32x4{v0[0], v0[1], v1[0], v1[1]};
        }
    }
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (!KV8) {
        // past dim stand other bytes of the row: q is zero there, but zero times an
        // infinite one would be no number (an E4M3 code that is not finite is NaN, there and in its place)
        if (dim < DP) {
#pragma unroll
            for (int d = 0; d < DP / 32; ++d)
                if (32 * d + 8 * g >= dim) kf[0][d] = kf[1][d] = u32x4{0, 0, 0, 0};
        }
    }
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            if constexpr (KV8) s[ks] = E::mma16(widen8<E>(u32x2{kf[ks][d][0], kf[ks][d][1]}), qf[d], s[ks]);
            else s[ks] = E::mma16(kf[ks][d], qf[d], s[ks]);
        }
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = CAP != CAP_NONE ? s[i >> 2][i & 3] : s[i >> 2][i & 3] * sc.mul;
    if constexpr (CAP != CAP_NONE) cap_scores<CAP>(sc, x);
    if (edge) {
        const uint32_t seen = (mask & (uint32_t)from_to(qlow + 1 - key0, qpos - key0)) >> (4 * g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = seen & (1u << (16 * (i >> 2) + (i & 3))) ? x[i] : -__builtin_inff();
        }
    }
    float m = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) m = fmaxf(m, x[i]);
    m = across32(across16(m)) - EP::P_SHIFT;
    if (__ballot(m > ref + RESCALE)) {
        const float to = fmaxf(m, ref), f = __builtin_amdgcn_exp2f(ref - to);
        ref = to;
        sum *= f;
#pragma unroll
        for (int t = 0; t < DP / 16; ++t) o[t] *= f;
    }
    u32x4 p, rest;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = __builtin_amdgcn_exp2f(minus(x[i], ref));
        sum += x[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        p[i] = EP::pack(x[2 * i], x[2 * i + 1]);
        // what its 8 (FP16: 11) bits leave over goes through the MFMA as well (this
        // kernel waits for memory either way)
        rest[i] = EP::pack(x[2 * i] - EP::low(p[i]), x[2 * i + 1] - EP::high(p[i]));
    }
    if constexpr (KV8) {
#pragma unroll
        for (int t = 0; t < DP / 16; ++t) vf[t] = widen8<EP>(u32x2{vf[t][0], vf[t][1]});
    }
#pragma unroll
    for (int t = 0; t < DP / 16; ++t) o[t] = EP::mma16(vf[t], p, o[t]);
#pragma unroll
    for (int t = 0; t < DP / 16; ++t) o[t] = EP::mma16(vf[t], rest, o[t]);
}

// DIRECT: one workgroup to a unit, no plan and no joining.
template <class E, class EP, bool KV8, int DP, int CAP, bool DIRECT>
__global__ __launch_bounds__(64 * dec_waves(KV8, DIRECT)) void attn_decode_kernel(AttnArgs a) {
    constexpr int WAVES = dec_waves(KV8, DIRECT);
    using D = Dec<KV8, DP, WAVES>;
    __shared__ __attribute__((aligned(1024))) char smem[WAVES * D::RING];
    __shared__ int64_t pages[PAGES_LDS];
    __shared__ float ml[2][WAVES][DEC_ROWS];
    __shared__ int red[WAVES], box[2];
    __shared__ NearPlan near;      // (not touched where DIRECT: no LDS then)
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 15, g = lane >> 4;
    MPDT_LDS char* ring = lds_cast(smem) + wave * D::RING;

    Plan p;
    int64_t at = 0, stop = 0, share = 1;
    int worker = 0, e = 0, h = 0;
    int b, r0, t0, tiles;
    Seq s;
    Line line{near, p, a.near != 0, 0, 0};
    if constexpr (DIRECT) {
        find_entry<WAVES>(a, blockIdx.x, red, box, b, r0, s);
        h = blockIdx.y;
        if (b < 0) return;
        at = 0;
        stop = 1;
    } else {
        plan_layout(a.ws, a.entries, a.sv.seqs, a.workers, a.tile_rows, DP, &p);
        make_line<WAVES>(a, DEC_KEYS, near, red, line);
        const int64_t total = (int64_t)line.tiles * a.kv.kv_heads;
        share = share_of(a, total);
        worker = worker_id();
        at = worker * share;
        stop = min(at + share, total);
        if (at >= stop) {
            if (tid == 0) p.cut[worker].b = -1;
            return;
        }
        h = (int)(at / line.tiles);
        e = line.find((int)(at - (int64_t)h * line.tiles));
    }
    bool lead = true;    // the first stretch of this workgroup
    while (at < stop) {
        int seg_a, seg_e;      // key tiles of this stretch within the unit
        int64_t u0 = 0;
        bool whole = true;
        if constexpr (!DIRECT) {
            const i32x4 ent = line.entry(e);
            b = ent[0];
            r0 = ent[1];
            t0 = ent[2];
            tiles = ent[3];
            u0 = (int64_t)h * line.tiles + line.before(e);
            seg_a = (int)(at - u0);
            seg_e = (int)min((int64_t)tiles, stop - u0);
            whole = seg_a == 0 && seg_e == tiles;
        }
        if constexpr (!DIRECT) s = uniform_seq(a.sv, a.kv.page_size, b);
        const int rows = s.nq * a.group, r1 = min(r0 + DEC_ROWS, rows);
        const Span32 kr = keys_of(s, a.group, a.window, r0, r1);
        if constexpr (DIRECT) {
            t0 = kr.lo / DEC_KEYS;
            tiles = max((kr.hi + DEC_KEYS - 1) / DEC_KEYS - t0, 1);
            seg_a = 0;
            seg_e = tiles;
        }
        // this lane's row
        const int row = r0 + n, tok = row / a.group, qh = h * a.group + row % a.group;
        const bool live = row < r1;
        const int qpos = s.n - s.nq + tok, qlow = a.window > 0 ? qpos - a.window : -1;
        u32x4 qf[DP / 32];
#pragma unroll
        for (int d = 0; d < DP / 32; ++d) {
            const int c = 32 * d + 8 * g;
            qf[d] = u32x4{0, 0, 0, 0};
            if (live && c < a.kv.dim)
                qf[d] = *reinterpret_cast<const u32x4*>(a.q + (int64_t)(s.start + tok) * a.q_tok_b +
                                                        qh * a.q_head_b + 2 * c);
        }
        const Score sc = score_of(a, KV8 ? uni(a.kv.k_scale[h]) : 1.0f);
        const char* kb = a.kv.k + h * a.kv.head_b;
        const char* vb = a.kv.v + h * a.kv.head_b;
        // rows of this tile see every key below `all_hi` and from `all_lo` on
        const int all_hi = s.n - s.nq + r0 / a.group + 1;
        const int all_lo = a.window > 0 ? s.n - s.nq + (r1 - 1) / a.group - a.window + 1 : 0;
        DecLoads<KV8, DP, WAVES> loads(a, kb, vb, pages);
        loads.lo = kr.lo;
        loads.hi = kr.hi;
        float ref = NO_MAX, sum = 0.0f;
        f32x4 o[DP / 16];
#pragma unroll
        for (int t = 0; t < DP / 16; ++t) o[t] = f32x4{0, 0, 0, 0};

        for (int pos = seg_a; pos < seg_e;) {
            bool clean;
            const int upto = fetch_pages<64 * WAVES, DEC_KEYS>(a, b, t0 + pos, t0 + seg_e, pages, loads.first,
                                                                   &clean) - t0;
            loads.fast = clean && a.kv.page_size % 16 == 0;
            uint32_t mask[D::NST];
#pragma unroll
            for (int i = 0; i < D::NST - 1; ++i) {
                const int j = pos + wave + i * WAVES;
                mask[i] = 0;
                if (j < upto) mask[i] = loads.issue(t0 + j, ring + i * D::STAGE);
            }
            int slot = 0;
            for (int j = pos + wave; j < upto; j += WAVES) {
                // the stage freed by the last tile takes the loads of the one NST - 1 on
                const int ahead = j + (D::NST - 1) * WAVES;
                const int fill = slot == 0 ? D::NST - 1 : slot - 1;
                mask[D::NST - 1] = 0;
                wait_lds();      // the last tile's reads of that stage have come back
                if (ahead < upto) {
                    mask[D::NST - 1] = loads.issue(t0 + ahead, ring + fill * D::STAGE);
                    wait_vmem<(D::NST - 1) * D::LOADS>();
                } else {
                    wait_vmem<0>();
                }
                __atomic_signal_fence(__ATOMIC_SEQ_CST);
                __builtin_amdgcn_sched_barrier(0);
                const int key0 = (t0 + j) * DEC_KEYS;
                if (mask[0]) {
                    const bool edge = mask[0] != 0xffffffffu || key0 + DEC_KEYS > all_hi || key0 < all_lo;
                    dec_tile<E, EP, KV8, DP, CAP, WAVES>(ring + slot * D::STAGE, qf, sc, a.kv.dim, mask[0], edge, key0,
                                                                  qpos, qlow, ref, sum, o);
                }
                __atomic_signal_fence(__ATOMIC_SEQ_CST);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i + 1 < D::NST; ++i) mask[i] = mask[i + 1];
                slot = slot + 1 == D::NST ? 0 : slot + 1;
            }
            pos = upto;
            __syncthreads();
        }

        // join the waves: each writes its rows over its own ring
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        wait_lds();
#pragma unroll
        for (int t = 0; t < DP / 16; ++t)
            lds_store16(ring, n * D::OROW + (16 * t + 4 * g) * 4, __builtin_bit_cast(u32x4, o[t]));
        if (g == 0) {
            ml[0][wave][n] = ref;
            ml[1][wave][n] = sum;
        }
        __syncthreads();
        if (tid < 16 * DEC_ROWS) {
            const int rr = tid >> 4, dc = tid & 15;
            float top = NO_MAX, den = 0.0f, w[WAVES];
#pragma unroll
            for (int i = 0; i < WAVES; ++i) top = fmaxf(top, ml[0][i][rr]);
#pragma unroll
            for (int i = 0; i < WAVES; ++i) {
                w[i] = __builtin_amdgcn_exp2f(ml[0][i][rr] - top);
                den += w[i] * ml[1][i][rr];
            }
            const int orow = r0 + rr, ot = orow / a.group, oh = h * a.group + orow % a.group;
            const float inv = (den > 0.0f || den != den ? 1.0f / den : 0.0f) * (KV8 ? a.kv.v_scale[h] : 1.0f);
            const int64_t slot_row = ((int64_t)worker * 2 + (lead ? 0 : 1)) * DEC_ROWS + rr;
#pragma unroll
            for (int k = 0; k < (DP + 63) / 64; ++k) {
                const int d = 4 * dc + 64 * k;
                if (d >= DP) break;
                f32x4 v{0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < WAVES; ++i)
                    v += w[i] * __builtin_bit_cast(f32x4, lds_load16(lds_cast(smem) + i * D::RING,
                                                                     rr * D::OROW + d * 4));
                if (whole) {
                    if (orow < r1 && d < a.kv.dim)
                        store_out4(a, a.out + (int64_t)(s.start + ot) * a.o_tok_b + oh * a.o_head_b, d, v * inv);
                } else {
                    *reinterpret_cast<f32x4*>(p.part_o + slot_row * DP + d) = v;
                }
            }
            if (dc == 0) {
                if (whole) {
                    if (orow < r1 && a.lse) a.lse[(int64_t)(s.start + ot) * a.lse_tok + oh] = lse_of(top, den);
                } else {
                    p.part_ml[slot_row] = f32x2{top, den};
                }
            }
        }
        __syncthreads();
        if constexpr (DIRECT) return;
        at += seg_e - seg_a;
        lead = false;
        if (at >= stop && tid == 0) p.cut[worker] = Cut{seg_a == 0 && seg_e < tiles ? b : -1, h, r0, tiles, u0, share};
        if (++e == line.entries) {
            e = 0;
            ++h;
        }
    }
}

// Units that several workers share: their partial sums joined in the order of
// the keys.  One workgroup to 16 rows of the unit that a worker leaves to others.
template <int DP>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
    Plan p;
    plan_layout(a.ws, a.entries, a.sv.seqs, a.workers, a.tile_rows, DP, &p);
    const Cut c = p.cut[blockIdx.x];
    const int rr = blockIdx.y * 16 + (threadIdx.x >> 4), dc = threadIdx.x & 15;
    if (c.b < 0) return;
    const int h = c.h, w0 = blockIdx.x, w1 = (int)((c.u0 + c.tiles - 1) / c.share);
    const int64_t u0 = c.u0, share = c.share;
    const Seq s = seq_of(a.sv, a.kv.page_size, c.b);
    const int row = c.r0 + rr;
    if (row >= s.nq * a.group) return;
    float top = NO_MAX;
    for (int w = w0; w <= w1; ++w) {
        const int64_t sr = ((int64_t)w * 2 + (w * share >= u0 ? 0 : 1)) * a.tile_rows + rr;
        top = fmaxf(top, p.part_ml[sr][0]);
    }
    float den = 0.0f;
    f32x4 v[(DP + 63) / 64];
#pragma unroll
    for (int k = 0; k < (DP + 63) / 64; ++k) v[k] = f32x4{0, 0, 0, 0};
    for (int w = w0; w <= w1; ++w) {
        const int64_t sr = ((int64_t)w * 2 + (w * share >= u0 ? 0 : 1)) * a.tile_rows + rr;
        const f32x2 ml = p.part_ml[sr];
        const float f = __builtin_amdgcn_exp2f(ml[0] - top);
        den += f * ml[1];
#pragma unroll
        for (int k = 0; k < (DP + 63) / 64; ++k)
            if (4 * dc + 64 * k < DP)
                v[k] += f * *reinterpret_cast<const f32x4*>(p.part_o + sr * DP + 4 * dc + 64 * k);
    }
    const int tok = row / a.group, qh = h * a.group + row % a.group;
    const float inv = (den > 0.0f || den != den ? 1.0f / den : 0.0f) *
                      (a.kv.type == DT_E4M3 ? a.kv.v_scale[h] : 1.0f);
    char* orow = a.out + (int64_t)(s.start + tok) * a.o_tok_b + qh * a.o_head_b;
#pragma unroll
    for (int k = 0; k < (DP + 63) / 64; ++k)
        if (4 * dc + 64 * k < a.kv.dim) store_out4(a, orow, 4 * dc + 64 * k, v[k] * inv);
    if (dc == 0 && a.lse) a.lse[(int64_t)(s.start + tok) * a.lse_tok + qh] = lse_of(top, den);
}

// The same for units of few rows over many workers: one workgroup to a row,
// eight groups of 32 threads take every eighth worker, and the eight sums are
// joined in order.
template <int DP>
__global__ __launch_bounds__(256) void attn_join_few_kernel(AttnArgs a) {
    __shared__ f32x4 part[8][DP / 4];
    __shared__ float sums[8], tops[8];
    Plan p;
    plan_layout(a.ws, a.entries, a.sv.seqs, a.workers, a.tile_rows, DP, &p);
    const Cut c = p.cut[blockIdx.x];
    const int rr = blockIdx.y, grp = threadIdx.x >> 5, dc = threadIdx.x & 31;
    if (c.b < 0) return;
    const int h = c.h, w0 = blockIdx.x, w1 = (int)((c.u0 + c.tiles - 1) / c.share);
    const int64_t u0 = c.u0, share = c.share;
    const Seq s = seq_of(a.sv, a.kv.page_size, c.b);
    const int row = c.r0 + rr;
    if (row >= s.nq * a.group) return;
    float top = NO_MAX, den = 0.0f;
    f32x4 v{0, 0, 0, 0};
#pragma unroll 4
    for (int w = w0 + grp; w <= w1; w += 8) {
        const int64_t sr = ((int64_t)w * 2 + (w * share >= u0 ? 0 : 1)) * a.tile_rows + rr;
        const f32x2 ml = p.part_ml[sr];
        f32x4 x{0, 0, 0, 0};
        if (4 * dc < DP) x = *reinterpret_cast<const f32x4*>(p.part_o + sr * DP + 4 * dc);
        const float to = fmaxf(top, ml[0]), f0 = __builtin_amdgcn_exp2f(top - to), f1 = __builtin_amdgcn_exp2f(ml[0] - to);
        v = v * f0 + x * f1;
        den = den * f0 + ml[1] * f1;
        top = to;
    }
    if (4 * dc < DP) part[grp][dc] = v;
    if (dc == 0) {
        tops[grp] = top;
        sums[grp] = den;
    }
    __syncthreads();
    if (grp != 0) return;
    float all = tops[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) all = fmaxf(all, tops[i]);
    den = 0.0f;
    v = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float f = __builtin_amdgcn_exp2f(tops[i] - all);
        den += f * sums[i];
        if (4 * dc < DP) v += part[i][dc] * f;
    }
    const int tok = row / a.group, qh = h * a.group + row % a.group;
    const float inv = (den > 0.0f || den != den ? 1.0f / den : 0.0f) *
                      (a.kv.type == DT_E4M3 ? a.kv.v_scale[h] : 1.0f);
    if (4 * dc < a.kv.dim)
        store_out4(a, a.out + (int64_t)(s.start + tok) * a.o_tok_b + qh * a.o_head_b, 4 * dc, v * inv);
    if (dc == 0 && a.lse) a.lse[(int64_t)(s.start + tok) * a.lse_tok + qh] = lse_of(all, den);
}

// ---- many rows: 256 rows by 64 keys a workgroup ------------------------------------
//
// Eight waves of 32 rows, two to a SIMD.  The two take turns: while one runs
// the MFMAs of O += V P of a tile and S of the next, the other runs its
// softmax, so that matrix and vector units both work all the time; barriers
// between the two phases keep them apart.  K and V tiles are shared by the
// eight waves in a ring of four stages.
//
// Two chunks of 4096 tokens after 12288, 32 heads of 128 over 8 KV heads: 1.80 ms
// of kernel, 1070 TFLOP/s (the library's 8192^3 BF16 product: 1230).  By the clock
// counter a tile's two phases take about 1310 cycles (softmax) and 1470 (32 MFMAs of
// 32 cycles, their LDS reads, the direct loads) besides their barriers; without the
// LDS reads and direct loads the MFMAs alone took 1000.

constexpr int CHK_WAVES = 8, CHK_ROWS = CHK_WAVES * 32, CHK_KEYS = 64;

template <bool KV8, int DP>
struct Chk {
    using R = Rows<DP, KV8, 32>;
    static constexpr int HALF = CHK_KEYS * R::BYTES;
    static constexpr int STAGE = 2 * HALF;
    static constexpr int NST = 4;
    static constexpr int LOADS = 2 * R::CH / CHK_WAVES;   // direct loads of a tile by a wave
    static_assert(2 * R::CH % CHK_WAVES == 0, "whole loads");
};

// One wave's part of the loads of a tile, 16 keys of K or of V: look() asks
// for their pages, found() takes the answer, and step<i>() issues the i-th load, so that the work can stand
// between MFMAs.  PAGE16: pages hold a multiple of 16 tokens, so that a wave's
// keys lie in one page and its address is scalar; a lane's own offset then is
// the same for every tile.  Keys that do not exist are staged as zeros (from
// the workspace): a weight of zero times their value is zero.  So is what lies
// past dim in rows of 16-bit values: q is zero there, but zero times another
// value's infinity would be no number.  (FP8: other bytes of the row; a code
// that is not finite is NaN, there and in its place.)
template <bool KV8, int DP, bool PAGE16>
struct ChkRefill {
    using D = Chk<KV8, DP>;
    using R = typename D::R;
    static constexpr int ROWS = 64 / R::CH;      // keys of a load (rows of 12 chunks: 16 keys of three loads)
    const AttnArgs& a;
    const char *base, *zeros;    // K or V of the head
    const int64_t* pages;
    int first, lo, hi, key16;    // key16: this wave's first key in a tile
    static constexpr uint32_t PAD = ~0u;         // a lane's offset past dim
    bool is_v, clean, padded;
    int lane, key0;
    uint64_t mask;
    int64_t page[PAGE16 ? 1 : D::LOADS];
    uint32_t own[D::LOADS];      // PAGE16: a lane's offset in its load
    const char* from;            // PAGE16: the wave's first key

    __device__ __forceinline__ ChkRefill(const AttnArgs& a_, const char* kb, const char* vb, const char* z, int wave)
        : a(a_), zeros(z) {
        is_v = wave >= CHK_WAVES / 2;
        base = is_v ? vb : kb;
        key16 = wave % (CHK_WAVES / 2) * 16;
        padded = !KV8 && a.kv.dim < DP;
        lane = threadIdx.x & 63;
        if constexpr (PAGE16)
            static_for<0, D::LOADS>([&](auto i) {
                constexpr int I = decltype(i)::value;
                const uint32_t c = chunk_of<I>();
                own[I] = c == PAD ? PAD : (uint32_t)(row_of<I>() * a.kv.slot_b) + c;
            });
    }
    template <int I>
    __device__ __forceinline__ int row_of() const {      // among the wave's 16
        return (I * 64 + lane) / R::CH;
    }
    template <int I>
    __device__ __forceinline__ uint32_t chunk_of() const {
        const int r = key16 + row_of<I>(), pos = (I * 64 + lane) % R::CH;
        const int from = (pos ^ (is_v ? R::swz_v(r) : R::swz_k(r))) * 16;
        return from < a.kv.dim * (KV8 ? 1 : 2) ? from : KV8 ? 0 : PAD;
    }

    // Returns which of the tile's 64 keys exist.
    __device__ __forceinline__ uint64_t look(int tile) {
        key0 = tile * CHK_KEYS;
        // (opaque, so that what follows from it is worked out anew for each tile:
        // kept in registers across the loop it would push others into scratch,
        // whose loads wait for all loads in flight)
        lane = threadIdx.x & 63;
        asm volatile("" : "+v"(lane));
        if constexpr (PAGE16) {
            page[0] = pages[a.kv.page_of(key0 + key16) - first];
        } else {
            static_for<0, D::LOADS>([&](auto i) {
                constexpr int I = decltype(i)::value;
                page[I] = pages[place_of(a.kv, first, key0 + key16 + row_of<I>()).entry];
            });
        }
        mask = from_to(lo - key0, hi - 1 - key0);
        if (!clean) mask &= __ballot(pages[place_of(a.kv, first, key0 + lane).entry] >= 0);
        return mask;
    }
    // The page numbers have come back.
    __device__ __forceinline__ void found() {
        if constexpr (PAGE16) {
            const int key = key0 + key16, pi = a.kv.page_of(key);
            const int64_t pg =
                (int64_t)((uint64_t)(uint32_t)uni((int)(page[0] >> 32)) << 32 | (uint32_t)uni((int)page[0]));
            from = base + pg + (key - pi * a.kv.page_size) * a.kv.slot_b;
        }
    }
    template <int I>
    __device__ __forceinline__ void step(MPDT_LDS char* dst) {
        MPDT_LDS char* d = dst + (is_v ? D::HALF : 0) + (key16 * R::CH / 64 + I) * 1024;
        if constexpr (PAGE16) {
            if (~mask || padded) {
                const char* src = from + own[I];
                global_to_lds16((mask >> (key16 + row_of<I>())) & 1 && own[I] != PAD ? src : zeros, d);
            } else {
                global_to_lds16(from, own[I], d);
            }
        } else {
            const int slot = place_of(a.kv, first, key0 + key16 + row_of<I>()).slot;
            const uint32_t c = chunk_of<I>();
            const char* src = base + (page[I] + slot * a.kv.slot_b + c);
            global_to_lds16((mask >> (key16 + row_of<I>())) & 1 && c != PAD ? src : zeros, d);
        }
    }
    __device__ __forceinline__ void steps(MPDT_LDS char* dst) {
        static_for<0, D::LOADS>([&](auto i) { step<decltype(i)::value>(dst); });
    }
};

// Weights of a tile from its scores, with the running maximum and sum.  A weight's
// exponent is one operation, s * mul - ref: the rounding of ref = max * mul stays
// in it, for all keys alike, until it grows to several units.  From FAR on the
// difference to the maximum's own product (raw) comes first (always: 1850 -> 1926
// us for two 4096-token chunks).
template <class EP, int DP, int CAP>
__device__ __forceinline__ void chk_weights(f32x16 (&s)[2], const Score& sc, uint64_t mask, bool edge, int key0,
                                            int qpos, int qlow, float& ref, float& raw, float& sum,
                                            f32x16 (&o)[(DP + 31) / 32], u32x4 (&p)[4]) {
    const int h = (threadIdx.x & 63) >> 5;
    if constexpr (CAP != CAP_NONE) {
        float c[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) c[i] = s[i >> 4][i & 15];
        cap_scores<CAP>(sc, c);
#pragma unroll
        for (int i = 0; i < 32; ++i) s[i >> 4][i & 15] = c[i];
    }
    if (edge) {
        // the keys of this half of the wave that the row sees, in the order of
        // its registers
        const uint64_t seen = (mask & from_to(qlow + 1 - key0, qpos - key0)) >> (4 * h);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const uint32_t w = (uint32_t)(seen >> (32 * ks));
                s[ks][i] = w & (1u << (8 * (i >> 2) + (i & 3))) ? s[ks][i] : -__builtin_inff();
            }
    }
    const float mul = CAP != CAP_NONE ? 1.0f : sc.mul;       // positive
    float m = s[0][0], m1 = s[1][0];            // (two chains)
#pragma unroll
    for (int i = 1; i < 16; ++i) {
        m = fmaxf(m, s[0][i]);
        m1 = fmaxf(m1, s[1][i]);
    }
    const float top = across32(fmaxf(m, m1));
    m = top * mul - EP::P_SHIFT;
    if (__ballot(m > ref + RESCALE)) {
        const float to = fmaxf(m, ref), f = __builtin_amdgcn_exp2f(ref - to);
        if constexpr (CAP == CAP_NONE) raw = m > ref ? top : raw;
        ref = to;
        sum *= f;
#pragma unroll
        for (int t = 0; t < (DP + 31) / 32; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[t][i] *= f;
    }
    float from = ref;
    if constexpr (CAP == CAP_NONE) {
        if (__ballot(fabsf(ref) > FAR && ref != NO_MAX)) {
            from = -EP::P_SHIFT;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                for (int i = 0; i < 16; ++i) s[ks][i] -= raw;
        }
    }
    float add = 0.0f;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            s[ks][i] = __builtin_amdgcn_exp2f(fmaf(s[ks][i], mul, -from));
            add += s[ks][i];
        }
    sum += add;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            p[kk][i] = EP::pack(s[kk >> 1][8 * (kk & 1) + 2 * i], s[kk >> 1][8 * (kk & 1) + 2 * i + 1]);
    // all of it here: the compiler would move the exponentials past the barrier,
    // next to the MFMAs that take them
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) asm volatile("" : "+v"(p[kk]));
    asm volatile("" : "+v"(sum));
}

// The MFMAs of a phase: O^T += V^T P^T of one tile (DO_V) and S^T = K Q^T of
// the next (DO_K), in groups of four or so whose operands are read from LDS
// two groups ahead.  (Left to itself the compiler reads each operand right
// before its MFMA and waits out the LDS latency 32 times a tile.)
template <class E, class EP, bool KV8, int DP>
struct ChkMma {
    using D = Chk<KV8, DP>;
    using R = typename D::R;
    static constexpr int DT = (DP + 31) / 32, NV = 4, NK = DP / 32, AHEAD = 2, NBUF = AHEAD + 1;
    struct Frag {
        u32x4 x[4];
    };
    Frag buf[NBUF];

    // Where this lane reads: its byte in the first operand of K and of V.  The
    // others follow by flipping bits of the chunk (rows of 12 chunks: by adding
    // four chunks at a time, which their swizzle leaves alone).
    uint32_t k_at, v_at;
    __device__ __forceinline__ ChkMma() {
        const int lane = threadIdx.x & 63, n = lane & 31, h = lane >> 5, l16 = lane & 15, sub = (lane >> 4) & 1;
        k_at = n * R::BYTES + (h ^ R::swz_k(n)) * 16;
        if constexpr (KV8) {
            const int k = l16 >> 1, r = 4 * h + (k < 4 ? k : k + 4);
            v_at = D::HALF + r * R::BYTES + (sub ^ R::swz_v(r)) * 16 + (l16 & 1) * 8;
        } else {
            const int r = 4 * h + (l16 >> 2);
            v_at = D::HALF + r * R::BYTES + ((2 * sub + ((l16 & 3) >> 1)) ^ R::swz_v(r)) * 16 + (l16 & 1) * 8;
        }
    }
    // four: groups of four chunks; two: a pair of chunks
    static __device__ __forceinline__ uint32_t chunk(uint32_t at, int four, int two) {
        if constexpr (R::CH == 12) return (at ^ (two * 32)) + four * 64;
        return at ^ (four * 64 + two * 32);
    }

    // operands of V: keys 16 kk to 16 kk + 15, all of dim
    __device__ __forceinline__ void load_v(Frag& f, const MPDT_LDS char* st, int kk) {
#pragma unroll
        for (int t = 0; t < DT; ++t) {
            if constexpr (KV8) {
                const u32x2 w = lds_read_tr8(st, chunk(v_at, t / 2, t % 2) + 16 * kk * R::BYTES);
                f.x[t][0] = w[0];
                f.x[t][1] = w[1];
            } else {
                const uint32_t at = chunk(v_at, t, 0) + 16 * kk * R::BYTES;
                const u32x2 v0 = lds_read_tr16(st, at), v1 = lds_read_tr16(st, at + 8 * R::BYTES);
                f.x[t] = u32x4{v0[0], v0[1], v1[0], v1[1]};
            }
        }
    }
    static __device__ __forceinline__ void mma_v(const Frag& f, const u32x4& p, f32x16 (&o)[DT]) {
#pragma unroll
        for (int t = 0; t < DT; ++t) {
            if constexpr (KV8) o[t] = EP::mma32(widen8<EP>(u32x2{f.x[t][0], f.x[t][1]}), p, o[t]);
            else o[t] = EP::mma32(f.x[t], p, o[t]);
        }
    }
    // operands of K: all 64 keys, 32 values of dim
    __device__ __forceinline__ void load_k(Frag& f, const MPDT_LDS char* st, int d) {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            if constexpr (KV8) {
                f.x[ks] = lds_load16(st, chunk(k_at, d / 2, d % 2) + 32 * ks * R::BYTES);
            } else {
                f.x[ks] = lds_load16(st, chunk(k_at, d, 0) + 32 * ks * R::BYTES);
                f.x[2 + ks] = lds_load16(st, chunk(k_at, d, 1) + 32 * ks * R::BYTES);
            }
        }
    }
    static __device__ __forceinline__ void mma_k(const Frag& f, const u32x4& q0, const u32x4& q1, f32x16 (&s)[2]) {
        if constexpr (KV8) {
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) s[ks] = E::mma32(widen8<E>(u32x2{f.x[ks][0], f.x[ks][1]}), q0, s[ks]);
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) s[ks] = E::mma32(widen8<E>(u32x2{f.x[ks][2], f.x[ks][3]}), q1, s[ks]);
        } else {
            s[0] = E::mma32(f.x[0], q0, s[0]);
            s[1] = E::mma32(f.x[1], q0, s[1]);
            s[0] = E::mma32(f.x[2], q1, s[0]);
            s[1] = E::mma32(f.x[3], q1, s[1]);
        }
    }

    template <bool DO_V, int G>
    __device__ __forceinline__ void load(const MPDT_LDS char* sv, const MPDT_LDS char* sk) {
        if constexpr (DO_V && G < NV) load_v(buf[G % NBUF], sv, G);
        else load_k(buf[G % NBUF], sk, DO_V ? G - NV : G);
    }
    // the first groups, from the phase before
    template <bool DO_V, bool DO_K>
    __device__ __forceinline__ void begin(const MPDT_LDS char* sv, const MPDT_LDS char* sk) {
        constexpr int NG = (DO_V ? NV : 0) + (DO_K ? NK : 0);
        static_for<0, AHEAD < NG ? AHEAD : NG>([&](auto g) { load<DO_V, decltype(g)::value>(sv, sk); });
    }
    // between(g): work of the caller's after group g
    template <bool DO_V, bool DO_K, class Fn>
    __device__ __forceinline__ void finish(const MPDT_LDS char* sv, const MPDT_LDS char* sk, const u32x4 (&p)[4],
                                           const u32x4 (&qf)[DP / 16], f32x16 (&o)[DT], f32x16 (&s)[2], Fn&& between) {
        constexpr int NG = (DO_V ? NV : 0) + (DO_K ? NK : 0);
        if constexpr (DO_K) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[0][i] = s[1][i] = 0.0f;
        }
        static_for<0, NG>([&](auto gc) {
            constexpr int g = decltype(gc)::value;
            if constexpr (g + AHEAD < NG) load<DO_V, g + AHEAD>(sv, sk);
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (DO_V && g < NV) {
                mma_v(buf[g % NBUF], p[g], o);
            } else {
                constexpr int d = DO_V ? g - NV : g;
                mma_k(buf[g % NBUF], qf[2 * d], qf[2 * d + 1], s);
            }
            __builtin_amdgcn_sched_barrier(0);
            between(gc);
        });
    }
};

template <class E, class EP, bool KV8, int DP, int CAP, bool PAGE16>
__global__ __launch_bounds__(64 * CHK_WAVES) __attribute__((amdgpu_waves_per_eu(2, 2))) void attn_chunk_kernel(
    AttnArgs a) {
    using D = Chk<KV8, DP>;
    using MMA = ChkMma<E, EP, KV8, DP>;
    constexpr int DT = (DP + 31) / 32, NST = D::NST;
    __shared__ __attribute__((aligned(1024))) char smem[NST * D::STAGE];
    __shared__ int64_t pages[PAGES_LDS];
    __shared__ int red[CHK_WAVES];
    __shared__ NearPlan near;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = lane & 31, half = lane >> 5;
    const bool second = wave >= CHK_WAVES / 2;     // waves w and w + 4 share a SIMD
    MPDT_LDS char* lds = lds_cast(smem);
    Plan p;
    plan_layout(a.ws, a.entries, a.sv.seqs, a.workers, a.tile_rows, DP, &p);
    Line line{near, p, a.near != 0, 0, 0};
    make_line<CHK_WAVES>(a, CHK_KEYS, near, red, line);
    const int64_t total = (int64_t)line.tiles * a.kv.kv_heads, share = share_of(a, total);
    const int worker = worker_id();
    int64_t at = worker * share;
    const int64_t stop = min(at + share, total);
    if (at >= stop) {
        if (tid == 0) p.cut[worker].b = -1;
        return;
    }
    // 16 bytes of zeros for keys that do not exist (every worker writes the same)
    if (tid < 4) reinterpret_cast<int32_t*>(p.zeros)[tid] = 0;
    __syncthreads();
    int h = (int)(at / line.tiles), e = line.find((int)(at - (int64_t)h * line.tiles));
    bool lead = true;
    while (at < stop) {
        const i32x4 ent = line.entry(e);
        const int b = ent[0], r0 = ent[1], t0 = ent[2], tiles = ent[3];
        const int64_t u0 = (int64_t)h * line.tiles + line.before(e);
        const int seg_a = (int)(at - u0), seg_e = (int)min((int64_t)tiles, stop - u0);
        const bool whole = seg_a == 0 && seg_e == tiles;
        const Seq s = uniform_seq(a.sv, a.kv.page_size, b);
        const int rows = s.nq * a.group, r1 = min(r0 + CHK_ROWS, rows);
        const Span32 kr = keys_of(s, a.group, a.window, r0, r1);
        const int past = s.n - s.nq;
        // this wave's rows: [w0, w1)
        const int w0 = r0 + wave * 32, w1 = min(w0 + 32, r1);
        const bool busy = w0 < w1;
        const int w_hi = busy ? past + (w1 - 1) / a.group : -1;          // last key that any of them sees
        const int all_hi = busy ? past + w0 / a.group + 1 : 0;           // every one sees keys below
        const int all_lo = a.window > 0 && busy ? past + (w1 - 1) / a.group - a.window + 1 : 0;
        const int w_lo = a.window > 0 && busy ? past + w0 / a.group - a.window + 1 : 0;
        const int row = w0 + n, tok = row / a.group, qh = h * a.group + row % a.group;
        const int qpos = past + tok, qlow = a.window > 0 ? qpos - a.window : -1;
        Score sc = score_of(a, KV8 ? uni(a.kv.k_scale[h]) : 1.0f);
        // the largest score is the factor times the largest product where the
        // factor is positive: a negative one goes to q's signs, a zero to q, and one
        // that is no number too (hidden keys keep their -inf)
        uint32_t keep = 0xffffffffu, flip = 0;
        if constexpr (CAP == CAP_NONE) {
            if (sc.mul < 0.0f) flip = 0x80008000u;
            if (!(fabsf(sc.mul) > 0.0f)) keep = 0;
            if (sc.mul != sc.mul) flip = 0x7fff7fffu;
            sc.mul = fabsf(sc.mul) > 0.0f ? fabsf(sc.mul) : 1.0f;
        }
        u32x4 qf[DP / 16];
#pragma unroll
        for (int d = 0; d < DP / 16; ++d) {
            // (an FP8 key's 16 bytes are two steps of its half of the wave)
            const int c = KV8 ? 32 * (d / 2) + 16 * half + 8 * (d % 2) : 16 * d + 8 * half;
            qf[d] = u32x4{0, 0, 0, 0};
            if (row < r1 && c < a.kv.dim)
                qf[d] = *reinterpret_cast<const u32x4*>(a.q + (int64_t)(s.start + tok) * a.q_tok_b +
                                                        qh * a.q_head_b + 2 * c);
            qf[d] = (qf[d] & keep) ^ flip;
        }
        float ref = NO_MAX, raw = 0.0f, sum = 0.0f;
        f32x16 o[DT], sc_tile[2];
        u32x4 pw[4];
        MMA mma;
#pragma unroll
        for (int t = 0; t < DT; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[t][i] = 0.0f;
        const char* kb = a.kv.k + h * a.kv.head_b;
        const char* vb = a.kv.v + h * a.kv.head_b;

        for (int pos = seg_a; pos < seg_e;) {
            int first;
            bool clean;
            const int upto =
                fetch_pages<64 * CHK_WAVES, CHK_KEYS>(a, b, t0 + pos, t0 + seg_e, pages, first, &clean) - t0;
            // tiles [ja, jb) hold keys that this wave's rows see
            int ja = upto, jb = upto;
            if (busy && w_hi >= w_lo) {
                ja = min(max(max(w_lo, 0) / CHK_KEYS - t0, pos), upto);
                jb = min(max(w_hi < 0 ? pos : w_hi / CHK_KEYS + 1 - t0, ja), upto);
            }
            uint64_t mask[NST];      // which keys of the tiles j, j + 1, ... exist
            ChkRefill<KV8, DP, PAGE16> refill(a, kb, vb, p.zeros, wave);
            refill.pages = pages;
            refill.first = first;
            refill.clean = clean;
            refill.lo = kr.lo;
            refill.hi = kr.hi;
            // (past the end the last tile comes again, into a stage that nobody
            // reads: the count of loads in flight is always the same)
#pragma unroll
            for (int i = 0; i < NST - 1; ++i) {
                mask[i] = refill.look(t0 + min(pos + i, upto - 1));
                refill.found();
                refill.steps(lds + i * D::STAGE);
            }
            wait_vmem<(NST - 2) * D::LOADS>();
            wg_barrier();
            int j = pos, slot = 0;
            // From here on the first four waves run one phase ahead.  A tile j
            // has landed for all before a first wave's MFMAs of tile j - 1, and
            // its stage is free after a second wave's MFMAs of tile j: it takes
            // the loads of tile j + NST in the MFMA phase of tile j + 1.
            auto landed = [&] { wait_vmem<(NST - 3) * D::LOADS>(); };
            auto look = [&] { mask[NST - 1] = refill.look(t0 + min(j + NST - 1, upto - 1)); };
            auto free_stage = [&] { return lds + (slot == 0 ? NST - 1 : slot - 1) * D::STAGE; };
            // The MFMA phase goes first where both waves of the SIMD could issue.
            auto enter_mma = [&] {
                refill.found();
                if (!second) landed();
                wg_barrier();
                __builtin_amdgcn_s_setprio(1);
            };
            auto leave_mma = [&] {
                __builtin_amdgcn_s_setprio(0);
                if (second) landed();
                wait_lds();
                wg_barrier();
#pragma unroll
                for (int i = 0; i + 1 < NST; ++i) mask[i] = mask[i + 1];
                slot = slot + 1 == NST ? 0 : slot + 1;
                ++j;
            };
            auto here = [&] { return lds + slot * D::STAGE; };
            auto there = [&] { return lds + (slot + 1 == NST ? 0 : slot + 1) * D::STAGE; };
            auto weights = [&] {
                const int key0 = (t0 + j) * CHK_KEYS;
                const bool edge = ~mask[0] || key0 + CHK_KEYS > all_hi || key0 < all_lo;
                chk_weights<EP, DP, CAP>(sc_tile, sc, mask[0], edge, key0, qpos, qlow, ref, raw, sum, o, pw);
                mma.template begin<true, false>(here(), here());
            };
            auto nothing = [](auto) {};
            if (ja == pos && ja < jb) {
                mma.template begin<false, true>(lds, lds);
                mma.template finish<false, true>(lds, lds, pw, qf, o, sc_tile, nothing);
            }
            if (second) {
                landed();
                wg_barrier();
            }
            while (j < ja) {
                look();
                enter_mma();
                refill.steps(free_stage());
                if (j + 1 == ja && ja < jb) {
                    mma.template begin<false, true>(there(), there());
                    mma.template finish<false, true>(there(), there(), pw, qf, o, sc_tile, nothing);
                }
                leave_mma();
            }
            while (j + 1 < jb) {
                look();
                weights();
                enter_mma();
                MPDT_LDS char* to = free_stage();
                mma.template finish<true, true>(here(), there(), pw, qf, o, sc_tile, [&](auto g) {
                    // (after V's groups, whose operands are the most LDS reads)
                    constexpr int i = decltype(g)::value - (MMA::NV + MMA::NK - D::LOADS);
                    if constexpr (i >= 0 && i < D::LOADS) refill.template step<i>(to);
                });
                leave_mma();
            }
            if (j < jb) {
                look();
                weights();
                enter_mma();
                refill.steps(free_stage());
                mma.template finish<true, false>(here(), here(), pw, qf, o, sc_tile, nothing);
                leave_mma();
            }
            while (j < upto) {
                look();
                enter_mma();
                refill.steps(free_stage());
                leave_mma();
            }
            wait_vmem<0>();
            if (!second) wg_barrier();
            pos = upto;
            __syncthreads();     // page numbers and stages are free again
        }

        const float den = sum + __shfl_xor(sum, 32);
        int n_out = threadIdx.x & 31;       // (opaque: nothing of this is kept across the loop)
        asm volatile("" : "+v"(n_out));
        const int out_row = w0 + n_out;
        if (out_row < r1) {
            const int tok = out_row / a.group, qh = h * a.group + out_row % a.group;
            if (whole) {
                const float inv = (den > 0.0f || den != den ? 1.0f / den : 0.0f) * (KV8 ? a.kv.v_scale[h] : 1.0f);
                char* orow = a.out + (int64_t)(s.start + tok) * a.o_tok_b + qh * a.o_head_b;
#pragma unroll
                for (int t = 0; t < DT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int d = 32 * t + 8 * i + 4 * half;
                        if (d < a.kv.dim)
                            store_out4(a, orow, d, f32x4{o[t][4 * i], o[t][4 * i + 1], o[t][4 * i + 2],
                                                         o[t][4 * i + 3]} * inv);
                    }
                if (half == 0 && a.lse) a.lse[(int64_t)(s.start + tok) * a.lse_tok + qh] = lse_of(ref, den);
            } else {
                const int64_t sr = ((int64_t)worker * 2 + (lead ? 0 : 1)) * CHK_ROWS + wave * 32 + n;
#pragma unroll
                for (int t = 0; t < DT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<f32x4*>(p.part_o + sr * DP + 32 * t + 8 * i + 4 * half) =
                            f32x4{o[t][4 * i], o[t][4 * i + 1], o[t][4 * i + 2], o[t][4 * i + 3]};
                if (half == 0) p.part_ml[sr] = f32x2{ref, den};
            }
        }
        at += seg_e - seg_a;
        lead = false;
        if (at >= stop && tid == 0) p.cut[worker] = Cut{seg_a == 0 && seg_e < tiles ? b : -1, h, r0, tiles, u0, share};
        if (++e == line.entries) {
            e = 0;
            ++h;
        }
    }
}

// ---- choice and launch -----------------------------------------------------------

constexpr int DP_OF(int dim) { return dim <= 64 ? 64 : dim <= 96 ? 96 : 128; }
constexpr int CUS = 256;
// Caches at most this long: one launch, a workgroup to a unit (replayed from a
// graph, 8 KV heads: one sequence of 1000 keys 10.6 us, 64 of them 48; shared out
// and joined 12.5 and 54).
constexpr int DIRECT_KEYS = 1024;

struct Shape {
    bool few, direct;
    int tile_rows, key_tile, workers, min_tiles, entries;
};

// Few rows to a sequence on average: the 16-row kernel.  Above, a 256-row tile
// reads the cache once where 16-row tiles would read it rows / 16 times.
Shape shape_of(const AttnArgs& a) {
    Shape s;
    const int64_t rows = (int64_t)a.sv.tokens * a.group;
    s.few = rows <= (int64_t)32 * a.sv.seqs;
    s.tile_rows = s.few ? DEC_ROWS : CHK_ROWS;
    s.key_tile = s.few ? DEC_KEYS : CHK_KEYS;
    s.workers = CUS;
    s.min_tiles = 4;
    s.entries = (int)(rows / s.tile_rows + std::min<int64_t>(a.sv.seqs, a.sv.tokens));
    s.direct = s.few && (int64_t)a.sv.width * a.kv.page_size <= DIRECT_KEYS &&
               s.entries <= LAUNCH_THREADS / (64 * dec_waves(true, true));
    return s;
}

template <class E, class EP, bool KV8, int DP, int CAP>
hipError_t launch_as(const AttnArgs& a, const Shape& s, hipStream_t stream) {
    hipError_t err;
    constexpr int FEW_CAP = CAP == CAP_NONE ? CAP_NONE : CAP_ANY;
    if (s.direct) {
        hipLaunchKernelGGL((attn_decode_kernel<E, EP, KV8, DP, FEW_CAP, true>),
                           dim3((unsigned)s.entries, (unsigned)a.kv.kv_heads),
                           dim3(64 * dec_waves(KV8, true)), 0, stream, a);
        return hipGetLastError();
    }
    if (!a.near) hipLaunchKernelGGL(attn_plan_kernel, dim3(1), dim3(1024), 0, stream, a, s.key_tile);
    if ((err = hipGetLastError()) != hipSuccess) return err;
    if (s.few) {
        hipLaunchKernelGGL((attn_decode_kernel<E, EP, KV8, DP, FEW_CAP, false>), dim3((unsigned)s.workers),
                           dim3(64 * dec_waves(KV8, false)), 0, stream, a);
    } else if (a.kv.page_size % 16 == 0) {
        hipLaunchKernelGGL((attn_chunk_kernel<E, EP, KV8, DP, CAP, true>), dim3((unsigned)s.workers),
                           dim3(64 * CHK_WAVES), 0, stream, a);
    } else {
        hipLaunchKernelGGL((attn_chunk_kernel<E, EP, KV8, DP, CAP, false>), dim3((unsigned)s.workers),
                           dim3(64 * CHK_WAVES), 0, stream, a);
    }
    if ((err = hipGetLastError()) != hipSuccess) return err;
    // a workgroup to a row only where units are cut into several pieces: 8 long
    // sequences of 8 heads (4 pieces a unit) 4.3 us, 16 rows to a workgroup 8.7;
    // 64 sequences (0.5 pieces a unit) 9.7 us against 5.5
    if (s.few && s.workers >= 2 * (int64_t)s.entries * a.kv.kv_heads) {
        hipLaunchKernelGGL((attn_join_few_kernel<DP>), dim3((unsigned)s.workers, DEC_ROWS), dim3(256), 0, stream, a);
    } else {
        hipLaunchKernelGGL((attn_join_kernel<DP>), dim3((unsigned)s.workers, s.tile_rows / 16), dim3(256), 0, stream, a);
    }
    return hipGetLastError();
}

template <class E, class EP, bool KV8, int DP>
hipError_t launch_cap(const AttnArgs& a, const Shape& s, hipStream_t stream) {
    if (a.softcap == 0.0f) return launch_as<E, EP, KV8, DP, CAP_NONE>(a, s, stream);
    return a.softcap <= CAP_NEAR_MOST ? launch_as<E, EP, KV8, DP, CAP_NEAR>(a, s, stream)
                                      : launch_as<E, EP, KV8, DP, CAP_ANY>(a, s, stream);
}

template <class E, class EP, bool KV8>
hipError_t launch_dim(const AttnArgs& a, const Shape& s, hipStream_t stream) {
    switch (DP_OF(a.kv.dim)) {
        case 64: return launch_cap<E, EP, KV8, 64>(a, s, stream);
        case 96: return launch_cap<E, EP, KV8, 96>(a, s, stream);
        default: return launch_cap<E, EP, KV8, 128>(a, s, stream);
    }
}

}  // namespace

int64_t attn_workspace(const AttnArgs& a) {
    const Shape s = shape_of(a);
    if (s.direct) return 0;
    Plan p;
    return plan_layout(nullptr, s.entries, a.sv.seqs, s.workers, s.tile_rows, DP_OF(a.kv.dim), &p);
}

hipError_t launch_paged_attention(const AttnArgs& in, hipStream_t stream) {
    AttnArgs a = in;
    const Shape s = shape_of(a);
    a.tile_rows = s.tile_rows;
    a.entries = s.entries;
    a.workers = s.workers;
    a.min_tiles = s.min_tiles;
    a.near = a.sv.seqs <= NEAR && s.entries <= NEAR;
    const bool kv8 = a.kv.type == DT_E4M3;
    if (a.q_type == DT_BF16) {
        return kv8 ? launch_dim<Bf16, F16, true>(a, s, stream) : launch_dim<Bf16, Bf16, false>(a, s, stream);
    }
    return kv8 ? launch_dim<F16, F16, true>(a, s, stream) : launch_dim<F16, F16, false>(a, s, stream);
}

}  // namespace mpdt
