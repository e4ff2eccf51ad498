// kv_cache.hip -- writing keys and values into a paged cache, and the
// bookkeeping of its pages: forking sequences, extending, freeing and
// bringing a fragmented cache together.
//
// Nothing here computes; every operator is bound by the bytes that it moves
// or, at the sizes of single tokens, by its launches.  Page decisions depend
// on counters in device memory, so one workgroup makes them (prefix sums over
// counters and rows) and a second launch does the moving; no host read is
// needed in between.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "device_common.hpp"
#include "serving.hpp"

namespace mpdt {
namespace {

// ---- new keys and values into their pages ----------------------------------------

__device__ __forceinline__ float widen(uint16_t x, bool bf16) {
    return bf16 ? __uint_as_float((uint32_t)x << 16) : (float)__builtin_bit_cast(_Float16, x);
}

// x / scale, cut to the format's range (NaN stays), rounded to nearest even.
__device__ __forceinline__ float cut448(float x) { return x > 448.0f ? 448.0f : x < -448.0f ? -448.0f : x; }

// APPEND_TOKENS tokens to a workgroup: one lane each finds where its token belongs,
// then all threads move the rows, 8 elements at a time.  8800 tokens of 8 heads of
// 128 in BF16 (72 MB): 13.0 us, 5.5 TB/s (14.3 with a load and a store in turn); 4801
// tokens into FP8 (30 MB): 14.5 us, of which the bytes are 6.
template <bool TO8>
__global__ __launch_bounds__(256) void append_kernel(AppendArgs a) {
    __shared__ int64_t dst[APPEND_TOKENS];
    const int t0 = blockIdx.x * APPEND_TOKENS;
    if (threadIdx.x < 64) {
        // one wave finds each token's sequence, the last that starts at or before
        // it: among up to 64 in one look (a lane each), else by halves
        const int lane = threadIdx.x, t = t0 + lane;
        int seq = 0;
        if (a.sv.seqs <= 64) {
            const int start = lane < a.sv.seqs ? a.sv.cu_q[lane] : 0x7fffffff;
#pragma unroll
            for (int k = 0; k < APPEND_TOKENS; ++k) {
                const int upto = __popcll(__ballot(start <= t0 + k));
                if (lane == k) seq = upto > 0 ? upto - 1 : 0;
            }
        } else if (lane < APPEND_TOKENS) {
            int hi = a.sv.seqs;
            while (hi - seq > 1) {
                const int mid = (seq + hi) / 2;
                if (a.sv.cu_q[mid] <= t) seq = mid;
                else hi = mid;
            }
        }
        if (lane < APPEND_TOKENS) {
            int64_t off = -1;
            const Seq s = seq_of(a.sv, a.kv.page_size, seq);
            const int pos = s.n - (s.start + s.nq - t);
            if (t >= s.start && t < s.start + s.nq && pos >= 0) {
                const int pi = a.kv.page_of(pos);
                const int pg = a.sv.table[(int64_t)seq * a.sv.ld_table + pi];
                if (pg >= 0 && pg < a.kv.pages) off = pg * a.kv.page_b + (pos - pi * a.kv.page_size) * a.kv.slot_b;
            }
            dst[lane] = off;
        }
    }
    __syncthreads();
    const int per_row = a.kv.dim / 8, per_tok = a.kv.kv_heads * per_row;
    const bool bf16 = a.type == DT_BF16;
    const int n = 2 * APPEND_TOKENS * per_tok;
    // eight loads of a thread at a time, then their stores: all of a workgroup's where
    // a token is 8 heads of 128 (smaller rows leave slots empty, which read the last
    // piece again)
    constexpr int U = 8;
    for (int i0 = threadIdx.x; i0 < n; i0 += 256 * U) {
        u32x4 x[U];
        char* to[U];
        float scale[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = min(i0 + u * 256, n - 1);
            const int k = i / per_tok, c = i - k * per_tok, h = c / per_row, e = c - h * per_row;
            const bool is_v = k & 1;
            // (a token past the last reads the last one's row, which is there)
            const int t = min(t0 + (k >> 1), a.sv.tokens - 1);
            const char* src = is_v ? a.v_new + t * a.v_tok_b + h * a.v_head_b : a.k_new + t * a.k_tok_b + h * a.k_head_b;
            x[u] = *reinterpret_cast<const u32x4*>(src + 16 * e);
            const int64_t off = dst[k >> 1];
            to[u] = off < 0 || i0 + u * 256 >= n
                        ? nullptr
                        : (is_v ? a.kv.v : a.kv.k) + off + h * a.kv.head_b + (TO8 ? 8 : 16) * e;
            if constexpr (TO8) scale[u] = (is_v ? a.kv.v_scale : a.kv.k_scale)[h];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!to[u]) continue;
            if constexpr (TO8) {
                float f[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    f[j] = cut448(widen((uint16_t)(x[u][j >> 1] >> (16 * (j & 1))), bf16) / scale[u]);
                u32x2 w;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    int q = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * j], f[4 * j + 1], 0, false);
                    q = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * j + 2], f[4 * j + 3], q, true);
                    w[j] = (uint32_t)q;
                }
                *reinterpret_cast<u32x2*>(to[u]) = w;
            } else {
                *reinterpret_cast<u32x4*>(to[u]) = x[u];
            }
        }
    }
}

// ---- pages -------------------------------------------------------------------------

constexpr int PLAN_THREADS = 1024;

__device__ __forceinline__ int held_pages(int len, int page) {
    return len <= 0 ? 0 : (int)(((int64_t)len + page - 1) / page);
}

// Exclusive sum over the workgroup; total to all.
__device__ __forceinline__ int plan_scan(int x, int* red, int& total) {
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
    for (int w = 0; w < PLAN_THREADS / 64; ++w) {
        const int r = red[w];
        if (w < wave) base += r;
        total += r;
    }
    __syncthreads();
    return base + s - x;
}

// The first `need` pages without a holder, in ascending order, into list;
// returns how many there were (at most need).
__device__ __forceinline__ int free_pages(const int32_t* refs, int pages, int need, int32_t* list, int* red) {
    int found = 0;
    for (int p0 = 0; p0 < pages && found < need; p0 += 4 * PLAN_THREADS) {
        const int p = p0 + 4 * threadIdx.x;
        int r[4], c = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = p + i < pages ? refs[p + i] : 1;
#pragma unroll
        for (int i = 0; i < 4; ++i) c += r[i] == 0;
        int total;
        int at = found + plan_scan(c, red, total);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (r[i] == 0) {
                if (at < need) list[at] = p + i;
                ++at;
            }
        found += total;
    }
    __syncthreads();
    return min(found, need);
}

// Workspace: [0] moves, [1] whether the call goes through; list and map.
struct PagesWs {
    int32_t *head, *list, *row_at;
};
__host__ __device__ inline PagesWs pages_ws(int32_t* ws, int pages) {
    return PagesWs{ws, ws + 16, ws + 16 + 2 * (int64_t)pages};
}

// Whether a row names another one, so that this call may write it.
__device__ __forceinline__ bool names_another(const PagesArgs& a, int row) {
    const int p = a.which[row];
    return p >= 0 && p < a.rows && p != row;
}
// Parent of a row, or -1.  A parent that may be written by this call has no settled
// contents; rows that name one are left as they are.
__device__ __forceinline__ int parent_of(const PagesArgs& a, int row) {
    return names_another(a, row) && !names_another(a, a.which[row]) ? a.which[row] : -1;
}

// Fork, first launch: part-filled pages wanted, free ones found for them in
// the order of the rows.  ws list: the new page of each copy; row_at: a row's copy or -1.
__global__ __launch_bounds__(PLAN_THREADS) void fork_plan_kernel(PagesArgs a) {
    __shared__ int red[PLAN_THREADS / 64];
    const PagesWs w = pages_ws(a.ws, a.pages);
    int need = 0;
    for (int r0 = 0; r0 < a.rows; r0 += PLAN_THREADS) {
        const int r = r0 + threadIdx.x;
        const int p = r < a.rows ? parent_of(a, r) : -1;
        const int part = p >= 0 && a.lens[p] > 0 && a.lens[p] % a.page_size != 0 && a.lens[p] / a.page_size < a.width;
        int total;
        const int at = need + plan_scan(part, red, total);
        if (r < a.rows) w.row_at[r] = part ? at : -1;
        need += total;
    }
    const int got = free_pages(a.refs, a.pages, need, w.list, red);
    const bool go = got == need;
    if (go)
        for (int i = threadIdx.x; i < need; i += PLAN_THREADS) a.refs[w.list[i]] = 1;
    if (threadIdx.x == 0) {
        w.head[1] = go;
        if (a.shortfall) a.shortfall[0] = need - got;
    }
}

// Bytes from one block to another by all threads of the workgroup.
template <bool WIDE>
__device__ __forceinline__ void copy_bytes(const char* src, char* dst, int64_t n) {
    if constexpr (WIDE) {
        const u32x4* s = reinterpret_cast<const u32x4*>(src);
        u32x4* d = reinterpret_cast<u32x4*>(dst);
        const int64_t c = n / 16;
        int64_t i = threadIdx.x;
        for (; i + 7 * 256 < c; i += 8 * 256) {
            u32x4 v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = __builtin_nontemporal_load(s + i + k * 256);
#pragma unroll
            for (int k = 0; k < 8; ++k) __builtin_nontemporal_store(v[k], d + i + k * 256);
        }
        for (; i < c; i += 256) d[i] = s[i];
    } else {
        for (int64_t i = threadIdx.x; i < n; i += 256) dst[i] = src[i];
    }
}

// Fork, second launch (32 rows of 8 planes, pages of 32 KB: 5.6 us, after a plan
// of 4.4): one workgroup to a row and a plane of the cache (the
// last y: the row's table, length and counters).
template <bool WIDE>
__global__ __launch_bounds__(256) void fork_move_kernel(PagesArgs a) {
    const PagesWs w = pages_ws(a.ws, a.pages);
    const int r = blockIdx.x, p = parent_of(a, r);
    if (p < 0 || !w.head[1]) return;
    const int at = w.row_at[r], len = a.lens[p], full = len > 0 ? min(len / a.page_size, a.width) : 0;
    const int32_t* from = a.table + (int64_t)p * a.ld_table;
    if (blockIdx.y == (unsigned)a.planes) {
        int32_t* to = a.table + (int64_t)r * a.ld_table;
        for (int c = threadIdx.x; c < a.width; c += 256) {
            const int pg = from[c];
            to[c] = at >= 0 && c == full ? w.list[at] : pg;
            if (c < full && pg >= 0 && pg < a.pages) atomicAdd(a.refs + pg, 1);
        }
        if (threadIdx.x == 0) a.lens[r] = len;
        return;
    }
    if (at < 0) return;
    const int src = from[full], dst = w.list[at];
    if (src < 0 || src >= a.pages) return;
    char* plane = a.kv + blockIdx.y * a.plane_b;
    copy_bytes<WIDE>(plane + src * a.page_stride_b, plane + dst * a.page_stride_b, a.page_bytes);
}

// Extend every row by which[row] tokens: one workgroup, one launch.
__global__ __launch_bounds__(PLAN_THREADS) void extend_kernel(PagesArgs a) {
    __shared__ int red[PLAN_THREADS / 64];
    __shared__ int64_t past;        // pages past the table's width
    const PagesWs w = pages_ws(a.ws, a.pages);
    if (threadIdx.x == 0) past = 0;
    __syncthreads();
    int need = 0;                   // (at most rows * width)
    for (int r0 = 0; r0 < a.rows; r0 += PLAN_THREADS) {
        const int r = r0 + threadIdx.x;
        int more = 0, over = 0;
        if (r < a.rows) {
            const int len = max(a.lens[r], 0), add = max(a.which[r], 0), have = held_pages(len, a.page_size);
            const int64_t want = ((int64_t)len + add + a.page_size - 1) / a.page_size;
            more = (int)(min(want, (int64_t)a.width) - min(have, a.width));
            over = (int)max((int64_t)0, min(want - a.width, (int64_t)1 << 30));
        }
        if (over) atomicAdd((unsigned long long*)&past, (unsigned long long)over);
        int total;
        const int at = need + plan_scan(more, red, total);
        if (r < a.rows) w.row_at[r] = at;
        need += total;
    }
    __syncthreads();
    // (where a row is full no page is taken for any)
    const int got = past == 0 ? free_pages(a.refs, a.pages, need, w.list, red) : 0;
    const bool go = past == 0 && got == need;
    if (threadIdx.x == 0 && a.shortfall) a.shortfall[0] = (int)min(need + past - got, (int64_t)0x7fffffff);
    if (!go) return;
    for (int r = threadIdx.x; r < a.rows; r += PLAN_THREADS) {
        const int len = max(a.lens[r], 0), add = max(a.which[r], 0), have = held_pages(len, a.page_size);
        const int64_t want = held_pages(len + add, a.page_size);
        int32_t* row = a.table + (int64_t)r * a.ld_table;
        const int at = w.row_at[r];
        for (int i = have; i < want; ++i) {
            const int pg = w.list[at + i - have];
            row[i] = pg;
            a.refs[pg] = 1;
        }
        if (add) a.lens[r] = len + add;
    }
}

// Rows with a mark give their pages back: one workgroup to a row.
__global__ __launch_bounds__(256) void free_kernel(PagesArgs a) {
    const int r = blockIdx.x;
    if (a.which[r] == 0) return;
    const int held = min(held_pages(a.lens[r], a.page_size), a.width);
    int32_t* row = a.table + (int64_t)r * a.ld_table;
    for (int c = threadIdx.x; c < a.width; c += 256) {
        const int pg = row[c];
        if (c < held && pg >= 0 && pg < a.pages) atomicSub(a.refs + pg, 1);
        row[c] = -1;
    }
    __syncthreads();
    if (threadIdx.x == 0) a.lens[r] = 0;
}

// Compact, first launch: with n pages in use, the holes below n and the used
// pages from n on, paired in ascending order.  list: holes, then (from pages
// on) movers.
__global__ __launch_bounds__(PLAN_THREADS) void compact_plan_kernel(PagesArgs a) {
    __shared__ int red[PLAN_THREADS / 64];
    const PagesWs w = pages_ws(a.ws, a.pages);
    int live = 0;
    for (int p0 = 0; p0 < a.pages; p0 += 4 * PLAN_THREADS) {
        int c = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = p0 + 4 * threadIdx.x + i;
            c += p < a.pages && a.refs[p] > 0;
        }
        int total;
        plan_scan(c, red, total);
        live += total;
    }
    int holes = 0, movers = 0;
    for (int p0 = 0; p0 < a.pages; p0 += 4 * PLAN_THREADS) {
        const int p = p0 + 4 * threadIdx.x;
        int kind[4], ch = 0, cm = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool in = p + i < a.pages, used = in && a.refs[p + i] > 0;
            kind[i] = !in ? 0 : p + i < live ? (used ? 0 : 1) : (used ? 2 : 0);
            ch += kind[i] == 1;
            cm += kind[i] == 2;
        }
        int th, tm;
        int ah = holes + plan_scan(ch, red, th), am = movers + plan_scan(cm, red, tm);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (kind[i] == 1) w.list[ah++] = p + i;
            if (kind[i] == 2) w.list[a.pages + am++] = p + i;
        }
        holes += th;
        movers += tm;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < movers; i += PLAN_THREADS) {
        const int hole = w.list[i], from = w.list[a.pages + i];
        a.refs[hole] = a.refs[from];
        a.refs[from] = 0;
    }
    if (threadIdx.x == 0) {
        w.head[0] = movers;
        w.head[1] = live;
    }
}

// Compact, second launch: pages move (sources lie at or past `live`, targets
// below it), and the tables follow them.  2036 pages of 32 KB in 32 planes (4.3 GB
// read and written): 798 us, 5.35 TB/s, where a 2 GiB copy runs at 4.98.
template <bool WIDE>
__global__ __launch_bounds__(256) void compact_move_kernel(PagesArgs a, int table_wgs) {
    const PagesWs w = pages_ws(a.ws, a.pages);
    const int movers = w.head[0], live = w.head[1];
    const int32_t* from = w.list + a.pages;
    if ((int)blockIdx.x < table_wgs) {
        const int64_t cells = (int64_t)a.rows * a.width;
        for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < cells; i += (int64_t)table_wgs * 256) {
            int32_t* cell = a.table + (i / a.width) * a.ld_table + i % a.width;
            const int pg = *cell;
            if (pg < live || pg >= a.pages) continue;
            int lo = 0, hi = movers;
            while (lo < hi) {
                const int mid = (lo + hi) / 2;
                if (from[mid] < pg) lo = mid + 1;
                else hi = mid;
            }
            if (lo < movers && from[lo] == pg) *cell = w.list[lo];
        }
        return;
    }
    const int64_t jobs = (int64_t)movers * a.planes, step = gridDim.x - table_wgs;
    for (int64_t j = blockIdx.x - table_wgs; j < jobs; j += step) {
        const int plane = (int)(j / movers), m = (int)(j - (int64_t)plane * movers);
        char* base = a.kv + plane * a.plane_b;
        copy_bytes<WIDE>(base + from[m] * a.page_stride_b, base + w.list[m] * a.page_stride_b, a.page_bytes);
    }
}

bool wide_pages(const PagesArgs& a) {
    return ((uintptr_t)a.kv | (uintptr_t)a.plane_b | (uintptr_t)a.page_stride_b | (uintptr_t)a.page_bytes) % 16 == 0;
}

}  // namespace

hipError_t launch_paged_append(const AppendArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)((a.sv.tokens + APPEND_TOKENS - 1) / APPEND_TOKENS));
    if (a.kv.type == DT_E4M3) {
        hipLaunchKernelGGL(append_kernel<true>, grid, dim3(256), 0, stream, a);
    } else {
        hipLaunchKernelGGL(append_kernel<false>, grid, dim3(256), 0, stream, a);
    }
    return hipGetLastError();
}

int64_t pages_workspace(int64_t pages, int64_t rows) { return (16 + 2 * pages + rows) * 4; }

hipError_t launch_cache_fork(const PagesArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL(fork_plan_kernel, dim3(1), dim3(PLAN_THREADS), 0, stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)a.rows, (unsigned)a.planes + 1);
    if (wide_pages(a)) {
        hipLaunchKernelGGL(fork_move_kernel<true>, grid, dim3(256), 0, stream, a);
    } else {
        hipLaunchKernelGGL(fork_move_kernel<false>, grid, dim3(256), 0, stream, a);
    }
    return hipGetLastError();
}

hipError_t launch_cache_extend(const PagesArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL(extend_kernel, dim3(1), dim3(PLAN_THREADS), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_cache_free(const PagesArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL(free_kernel, dim3((unsigned)a.rows), dim3(256), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_cache_compact(const PagesArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL(compact_plan_kernel, dim3(1), dim3(PLAN_THREADS), 0, stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t cells = (int64_t)a.rows * a.width;
    const int table_wgs = (int)std::min<int64_t>((cells + 255) / 256, 64);
    const int64_t jobs = (int64_t)a.pages * a.planes;      // at most
    const unsigned wgs = (unsigned)(table_wgs + std::min<int64_t>(jobs, 2048));
    if (wide_pages(a)) {
        hipLaunchKernelGGL(compact_move_kernel<true>, dim3(wgs), dim3(256), 0, stream, a, table_wgs);
    } else {
        hipLaunchKernelGGL(compact_move_kernel<false>, dim3(wgs), dim3(256), 0, stream, a, table_wgs);
    }
    return hipGetLastError();
}

}  // namespace mpdt
