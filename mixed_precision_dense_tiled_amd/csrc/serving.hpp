// serving.hpp -- internal (C++) interface between the C ABI and the serving
// kernels: paged key/value cache, attention over it, page bookkeeping and
// token log probabilities.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mpdt {

// Element types (the values of the C ABI's mpdt_dtype).
enum : int { DT_BF16 = 0, DT_F16 = 1, DT_F32 = 2, DT_E4M3 = 3 };

// A launch holds fewer than 2^32 threads along x.
constexpr int64_t LAUNCH_THREADS = 0xffffffffll;
constexpr int64_t MAX_GROUPS = LAUNCH_THREADS / 256;     // workgroups of 256 threads

// One layer's paged cache.  Strides in BYTES, the same for K and V; a row is
// dim elements side by side.
struct PagedKV {
    char* k;
    char* v;
    int64_t page_b, slot_b, head_b;
    const float* k_scale;   // [kv_heads], E4M3 only
    const float* v_scale;
    int64_t pages;
    int page_size;
    uint32_t page_mul;      // key / page_size = (mulhi(key, page_mul) + key) >> page_shift, key < 2^31
    int page_shift;
    int kv_heads, dim, type;

    __host__ __device__ int page_of(int key) const {
        const uint32_t k = (uint32_t)key;
        return (int)(((uint32_t)((uint64_t)k * page_mul >> 32) + k) >> page_shift);
    }
};

// Which sequence holds which pages, and how long it is.
struct SeqView {
    const int32_t* table;   // [seqs, width], rows ld_table apart
    int64_t ld_table;
    const int32_t* cu_q;    // [seqs + 1]
    const int32_t* lens;    // [seqs]
    int seqs, width;
    int tokens;             // rows of q / of the new keys
};

// A sequence as every operator sees it: numbers that point outside the batch are
// cut to it.  Its last nq of n tokens are the rows from `start` on.
struct Seq {
    int start, nq, n;
};
__device__ __forceinline__ Seq seq_of(const SeqView& v, int64_t page_size, int b) {
    Seq s;
    const int c0 = v.cu_q[b], c1 = v.cu_q[b + 1];
    s.start = min(max(c0, 0), v.tokens);
    s.nq = min(max(c1, s.start), v.tokens) - s.start;
    const int64_t most = page_size * v.width;
    s.n = (int)min((int64_t)max(v.lens[b], 0), most);
    return s;
}

struct AttnArgs {
    PagedKV kv;
    SeqView sv;
    const char* q;          // strides in bytes
    int64_t q_tok_b, q_head_b;
    char* out;
    int64_t o_tok_b, o_head_b;
    float* lse;             // [tokens, heads] or null
    int64_t lse_tok;        // elements between tokens
    float scale, softcap;
    int window;             // 0: none
    int heads, group;       // group = heads / kv_heads
    int q_type;             // DT_BF16 or DT_F16
    // set by the launcher
    char* ws;
    int tile_rows;          // rows (token, head of the group) of a unit
    int entries;            // upper bound of the row tiles over all sequences
    int workers;            // workgroups that share the key tiles
    int min_tiles;          // fewest key tiles for a workgroup
    int near;               // every workgroup plans for itself
};
int64_t attn_workspace(const AttnArgs& a);
hipError_t launch_paged_attention(const AttnArgs& a, hipStream_t stream);

constexpr int APPEND_TOKENS = 8;    // new tokens to a workgroup
struct AppendArgs {
    PagedKV kv;
    SeqView sv;
    const char* k_new;      // strides in bytes
    const char* v_new;
    int64_t k_tok_b, k_head_b, v_tok_b, v_head_b;
    int type;               // of the new rows
};
hipError_t launch_paged_append(const AppendArgs& a, hipStream_t stream);

// Page bookkeeping.  kv: planes x pages blocks of page_bytes.
struct PagesArgs {
    char* kv;
    int64_t plane_b, page_stride_b, page_bytes;
    int planes;
    int pages;
    int32_t* refs;          // [pages]
    int32_t* table;         // [rows, width]
    int64_t ld_table;
    int32_t* lens;          // [rows]
    const int32_t* which;   // [rows]: parents, new tokens or drop marks
    int rows, width, page_size;
    int32_t* ws;
    int32_t* shortfall;     // pages wanted and not free (may be null)
};
int64_t pages_workspace(int64_t pages, int64_t rows);
hipError_t launch_cache_fork(const PagesArgs& a, hipStream_t stream);
hipError_t launch_cache_extend(const PagesArgs& a, hipStream_t stream);
hipError_t launch_cache_free(const PagesArgs& a, hipStream_t stream);
hipError_t launch_cache_compact(const PagesArgs& a, hipStream_t stream);

struct LogprobArgs {
    const char* logits;
    int64_t ld_b;           // bytes between rows
    int type;
    const int64_t* targets; // [rows]
    int rows;
    int vocab;
    int top;
    float* logprob;
    float* lse;
    float* entropy;
    float* top_logprob;     // [rows, top]
    int64_t* top_index;
    char* ws;
    int segments;           // pieces of a row, one workgroup each (set by the launcher)
    int chunks;             // chunks of a segment
    // backward
    const float* g_logprob; // [rows] or null
    const float* g_entropy;
    char* grad;
    int64_t ld_grad_b;
};
constexpr int LOGPROB_MAX_TOP = 64;
bool logprob_fits(int type, int64_t rows, int64_t vocab);   // the gradient's launch
int64_t logprob_workspace(int type, int64_t rows, int64_t vocab, int top);
hipError_t launch_token_logprobs(const LogprobArgs& a, hipStream_t stream);
hipError_t launch_token_logprobs_backward(const LogprobArgs& a, hipStream_t stream);

}  // namespace mpdt
