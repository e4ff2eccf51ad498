// serving_abi.hip -- the C ABI of the serving operators (mpdt_serving.h):
// host-side argument validation and launch.  No device code lives here.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "abi_common.hpp"
#include "mpdt_serving.h"
#include "serving.hpp"

static_assert(MPDT_BF16 == mpdt::DT_BF16 && MPDT_F16 == mpdt::DT_F16 && MPDT_F32 == mpdt::DT_F32 &&
                  MPDT_E4M3 == mpdt::DT_E4M3,
              "element types of the C ABI and the kernels agree");

namespace {

using mpdt::abi_check_device;
using mpdt::abi_fail;
using mpdt::abi_launched;

constexpr int64_t kMaxDim = int64_t(1) << 30;
constexpr int64_t kMaxSpan = int64_t(1) << 46;   // bytes

mpdt_status invalid(const char* fn, const char* what) { return abi_fail(MPDT_ERROR_INVALID_VALUE, fn, what); }
mpdt_status misaligned(const char* fn, const char* what) { return abi_fail(MPDT_ERROR_MISALIGNED, fn, what); }

bool off(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }
bool in_dims(int64_t v, int64_t lo) { return v >= lo && v <= kMaxDim; }

// A strided operand: bytes from its first to past its last.
struct Bytes {
    uintptr_t lo = 0, hi = 0;
    bool meets(const Bytes& o) const { return lo < o.hi && o.lo < hi; }
};
struct Axis {
    int64_t n, stride;   // stride in bytes
};
// False where a stride is negative or the operand spans 2^46 bytes or more.
bool span(const void* p, std::initializer_list<Axis> axes, int64_t inner, Bytes* out) {
    *out = Bytes{};
    int64_t reach = inner;
    for (const Axis& a : axes) {
        if (a.n <= 0) return true;
        if (a.stride < 0 || (a.n > 1 && a.stride > kMaxSpan / (a.n - 1))) return false;
        reach += (a.n - 1) * a.stride;
        if (reach >= kMaxSpan) return false;
    }
    out->lo = reinterpret_cast<uintptr_t>(p);
    out->hi = out->lo + (uintptr_t)reach;
    return true;
}

// Whether no two elements share a byte, for rows of `inner` bytes laid out by
// strides that nest (in any order of the axes).
bool apart(std::initializer_list<Axis> axes, int64_t inner) {
    Axis by[3];
    int n = 0;
    for (const Axis& a : axes)
        if (a.n > 1) by[n++] = a;
    std::sort(by, by + n, [](const Axis& x, const Axis& y) { return x.stride < y.stride; });
    int64_t reach = inner;
    for (int i = 0; i < n; ++i) {
        if (by[i].stride < reach) return false;
        reach += (by[i].n - 1) * by[i].stride;
    }
    return true;
}

int size_of(int dtype) { return dtype == MPDT_F32 ? 4 : dtype == MPDT_E4M3 ? 1 : 2; }

// The cache and the batch, checked and in the kernels' form; k and v: their bytes.
mpdt_status check_cache(const char* fn, const mpdt_paged_kv* kv, const mpdt_sequences* sq, mpdt::PagedKV* o,
                        mpdt::SeqView* v, Bytes* bk, Bytes* bv) {
    if (!kv || !sq) return invalid(fn, "cache or sequences NULL");
    if (kv->dtype != MPDT_BF16 && kv->dtype != MPDT_F16 && kv->dtype != MPDT_E4M3)
        return invalid(fn, "unknown cache type");
    if (!in_dims(kv->pages, 1) || !in_dims(kv->page_size, 1) || kv->kv_heads < 1 || kv->kv_heads > 65535)
        return invalid(fn, "pages, page_size or kv_heads out of range");
    if (kv->dim < 16 || kv->dim > 128 || kv->dim % 16) return invalid(fn, "dim must be a multiple of 16 up to 128");
    if (!in_dims(sq->seqs, 0) || !in_dims(sq->tokens, 0) || !in_dims(sq->width, 1))
        return invalid(fn, "seqs, tokens or width out of range");
    if (sq->width > kMaxDim / kv->page_size) return invalid(fn, "width * page_size must be at most 2^30");
    if (sq->ld_table < sq->width) return invalid(fn, "ld_table < width");
    if (!kv->k || !kv->v || !sq->table || !sq->cu_q || !sq->lens) return invalid(fn, "NULL pointer");
    const int es = size_of(kv->dtype);
    if (off(kv->k, 16) || off(kv->v, 16) || kv->page_stride * es % 16 || kv->slot_stride * es % 16 ||
        kv->head_stride * es % 16)
        return misaligned(fn, "rows of the cache must start on 16-byte boundaries");
    if (off(sq->table, 4) || off(sq->cu_q, 4) || off(sq->lens, 4))
        return misaligned(fn, "pointer not aligned to its element size");
    if (kv->dtype == MPDT_E4M3 && (!kv->k_scale || !kv->v_scale)) return invalid(fn, "an E4M3 cache needs scales");
    if (kv->dtype == MPDT_E4M3 && (off(kv->k_scale, 4) || off(kv->v_scale, 4)))
        return misaligned(fn, "pointer not aligned to its element size");
    if (kv->slot_stride >= (int64_t(1) << 26)) return invalid(fn, "slot_stride must be below 2^26");
    const std::initializer_list<Axis> axes = {{kv->pages, kv->page_stride * es},
                                              {kv->page_size, kv->slot_stride * es},
                                              {kv->kv_heads, kv->head_stride * es}};
    if (!span(kv->k, axes, kv->dim * es, bk) || !span(kv->v, axes, kv->dim * es, bv))
        return invalid(fn, "cache too large, or a negative stride");
    Bytes t;
    if (!span(sq->table, {{sq->seqs, sq->ld_table * 4}}, sq->width * 4, &t)) return invalid(fn, "table too large");
    o->k = (char*)kv->k;
    o->v = (char*)kv->v;
    o->page_b = kv->page_stride * es;
    o->slot_b = kv->slot_stride * es;
    o->head_b = kv->head_stride * es;
    o->k_scale = kv->k_scale;
    o->v_scale = kv->v_scale;
    o->pages = kv->pages;
    o->page_size = (int)kv->page_size;
    // division by a constant, rounded-up reciprocal: with s = ceil(log2 d) and
    // m = floor(2^32 (2^s - d) / d) + 1, n / d = (mulhi(n, m) + n) >> s
    o->page_shift = 0;
    while ((int64_t(1) << o->page_shift) < kv->page_size) ++o->page_shift;
    o->page_mul = (uint32_t)((((uint64_t(1) << o->page_shift) - kv->page_size) << 32) / kv->page_size + 1);
    o->kv_heads = (int)kv->kv_heads;
    o->dim = (int)kv->dim;
    o->type = kv->dtype;
    v->table = sq->table;
    v->ld_table = sq->ld_table;
    v->cu_q = sq->cu_q;
    v->lens = sq->lens;
    v->seqs = (int)sq->seqs;
    v->width = (int)sq->width;
    v->tokens = (int)sq->tokens;
    return MPDT_SUCCESS;
}

mpdt_status check_attention_sizes(const char* fn, const mpdt_paged_kv* kv, const mpdt_sequences* sq, int64_t heads) {
    if (heads < 1 || heads > 65535 || heads % kv->kv_heads) return invalid(fn, "heads must be a multiple of kv_heads");
    const int64_t group = heads / kv->kv_heads;
    // (units and key tiles of one head are counted in 32 bits)
    if (sq->tokens > kMaxDim / group) return invalid(fn, "tokens * heads / kv_heads must be at most 2^30");
    const int64_t units = sq->tokens * group / 16 + std::min(sq->seqs, sq->tokens);
    if (units > 0 && (sq->width * kv->page_size + 31) / 32 + 1 > int64_t(0x7fffffff) / units)
        return invalid(fn, "the batch has too many tiles of rows and keys");
    return MPDT_SUCCESS;
}

}  // namespace

MPDT_EXPORT mpdt_status paged_kv_append(const mpdt_paged_kv* kv, const mpdt_sequences* sq, int dtype,
                                        const void* k_new, int64_t k_token, int64_t k_head, const void* v_new,
                                        int64_t v_token, int64_t v_head, void* stream) {
    const char* fn = "paged_kv_append";
    mpdt::AppendArgs a{};
    Bytes bk, bv, nk, nv;
    mpdt_status s = check_cache(fn, kv, sq, &a.kv, &a.sv, &bk, &bv);
    if (s != MPDT_SUCCESS) return s;
    if ((dtype != MPDT_BF16 && dtype != MPDT_F16) || (kv->dtype != MPDT_E4M3 && dtype != kv->dtype))
        return invalid(fn, "new keys must have the cache's type, or a 16-bit one for an E4M3 cache");
    if (sq->tokens == 0 || sq->seqs == 0) return MPDT_SUCCESS;
    if (sq->tokens > mpdt::MAX_GROUPS * mpdt::APPEND_TOKENS) return invalid(fn, "too many tokens");
    if (!k_new || !v_new) return invalid(fn, "NULL pointer");
    if (off(k_new, 16) || off(v_new, 16) || k_token % 8 || k_head % 8 || v_token % 8 || v_head % 8)
        return misaligned(fn, "new rows must start on 16-byte boundaries");
    if (!span(k_new, {{sq->tokens, k_token * 2}, {kv->kv_heads, k_head * 2}}, kv->dim * 2, &nk) ||
        !span(v_new, {{sq->tokens, v_token * 2}, {kv->kv_heads, v_head * 2}}, kv->dim * 2, &nv))
        return invalid(fn, "operand too large, or a negative stride");
    if (nk.meets(bk) || nk.meets(bv) || nv.meets(bk) || nv.meets(bv))
        return abi_fail(MPDT_ERROR_ALIASING, fn, "new rows overlap the cache");
    if (!apart({{kv->pages, a.kv.page_b}, {kv->page_size, a.kv.slot_b}, {kv->kv_heads, a.kv.head_b}},
               kv->dim * size_of(kv->dtype)))
        return abi_fail(MPDT_ERROR_ALIASING, fn, "rows of the cache overlap each other");
    if ((s = abi_check_device(fn)) != MPDT_SUCCESS) return s;
    a.k_new = (const char*)k_new;
    a.v_new = (const char*)v_new;
    a.k_tok_b = k_token * 2;
    a.k_head_b = k_head * 2;
    a.v_tok_b = v_token * 2;
    a.v_head_b = v_head * 2;
    a.type = dtype;
    return abi_launched(mpdt::launch_paged_append(a, (hipStream_t)stream), fn);
}

MPDT_EXPORT int64_t paged_attention_workspace(const mpdt_paged_kv* kv, const mpdt_sequences* sq, int64_t heads) {
    const char* fn = "paged_attention_workspace";
    mpdt::AttnArgs a{};
    Bytes bk, bv;
    if (check_cache(fn, kv, sq, &a.kv, &a.sv, &bk, &bv) != MPDT_SUCCESS ||
        check_attention_sizes(fn, kv, sq, heads) != MPDT_SUCCESS)
        return -1;
    if (sq->tokens == 0 || sq->seqs == 0) return 0;
    a.heads = (int)heads;
    a.group = (int)(heads / kv->kv_heads);
    return mpdt::attn_workspace(a);
}

MPDT_EXPORT mpdt_status paged_attention(const mpdt_paged_kv* kv, const mpdt_sequences* sq, int64_t heads, int q_dtype,
                                        const void* q, int64_t q_token, int64_t q_head, void* out, int64_t out_token,
                                        int64_t out_head, float* lse, int64_t lse_token, float scale, float softcap,
                                        int64_t window, void* workspace, int64_t workspace_bytes, void* stream) {
    const char* fn = "paged_attention";
    mpdt::AttnArgs a{};
    Bytes bk, bv, bq, bo, bl, bw;
    mpdt_status s = check_cache(fn, kv, sq, &a.kv, &a.sv, &bk, &bv);
    if (s != MPDT_SUCCESS) return s;
    if ((s = check_attention_sizes(fn, kv, sq, heads)) != MPDT_SUCCESS) return s;
    if ((q_dtype != MPDT_BF16 && q_dtype != MPDT_F16) || (kv->dtype != MPDT_E4M3 && q_dtype != kv->dtype))
        return invalid(fn, "q must have the cache's type, or a 16-bit one for an E4M3 cache");
    if (!std::isfinite(scale) || !std::isfinite(softcap) || softcap < 0.0f)
        return invalid(fn, "scale must be finite, softcap finite and not negative");
    if (window < 0) return invalid(fn, "window must not be negative");
    if (sq->tokens == 0 || sq->seqs == 0) return MPDT_SUCCESS;
    if (!q || !out) return invalid(fn, "q or out is NULL");
    if (lse && lse_token < heads) return invalid(fn, "lse_token < heads");
    if (off(q, 16) || off(out, 16) || q_token % 8 || q_head % 8 || out_token % 8 || out_head % 8)
        return misaligned(fn, "rows of q and out must start on 16-byte boundaries");
    if (lse && off(lse, 4)) return misaligned(fn, "pointer not aligned to its element size");
    if (!span(q, {{sq->tokens, q_token * 2}, {heads, q_head * 2}}, kv->dim * 2, &bq) ||
        !span(out, {{sq->tokens, out_token * 2}, {heads, out_head * 2}}, kv->dim * 2, &bo) ||
        !span(lse, {{lse ? sq->tokens : 0, lse_token * 4}}, heads * 4, &bl))
        return invalid(fn, "operand too large, or a negative stride");
    a.heads = (int)heads;
    a.group = (int)(heads / kv->kv_heads);
    const int64_t need = mpdt::attn_workspace(a);
    if (workspace_bytes < need || (need > 0 && !workspace)) return invalid(fn, "workspace too small");
    if (need > 0 && off(workspace, 256)) return misaligned(fn, "workspace must start on a 256-byte boundary");
    (void)span(workspace, {{need > 0, 0}}, need, &bw);
    if (!apart({{sq->tokens, out_token * 2}, {heads, out_head * 2}}, kv->dim * 2))
        return abi_fail(MPDT_ERROR_ALIASING, fn, "rows of out overlap each other");
    if (bo.meets(bq) || bo.meets(bk) || bo.meets(bv) || bl.meets(bq) || bl.meets(bk) || bl.meets(bv) || bl.meets(bo) ||
        bw.meets(bq) || bw.meets(bk) || bw.meets(bv) || bw.meets(bo) || bw.meets(bl))
        return abi_fail(MPDT_ERROR_ALIASING, fn, "an output or the workspace overlaps another operand");
    if ((s = abi_check_device(fn)) != MPDT_SUCCESS) return s;
    a.q = (const char*)q;
    a.q_tok_b = q_token * 2;
    a.q_head_b = q_head * 2;
    a.out = (char*)out;
    a.o_tok_b = out_token * 2;
    a.o_head_b = out_head * 2;
    a.lse = lse;
    a.lse_tok = lse_token;
    a.scale = scale;
    a.softcap = softcap;
    a.window = (int)std::min(window, kMaxDim);
    a.q_type = q_dtype;
    a.ws = (char*)workspace;
    return abi_launched(mpdt::launch_paged_attention(a, (hipStream_t)stream), fn);
}

namespace {

mpdt_status check_pages(const char* fn, const mpdt_pages* c, bool moves, const int32_t* which, bool needs_which,
                        int32_t* shortfall, void* ws, int64_t ws_bytes, bool needs_ws, mpdt::PagesArgs* a) {
    if (!c) return invalid(fn, "cache NULL");
    if (!in_dims(c->pages, 0) || !in_dims(c->page_size, 1) || !in_dims(c->rows, 0) || !in_dims(c->width, 1) ||
        !in_dims(c->planes, 0) || c->planes > 65534 || c->rows > mpdt::MAX_GROUPS)
        return invalid(fn, "planes, pages, page_size, rows or width out of range");
    if (c->width > kMaxDim / c->page_size || c->width > kMaxDim / std::max<int64_t>(c->rows, 1))
        return invalid(fn, "width * page_size and rows * width must be at most 2^30");
    if (c->ld_table < c->width) return invalid(fn, "ld_table < width");
    a->pages = (int)c->pages;
    a->rows = (int)c->rows;
    if (c->rows == 0) return MPDT_SUCCESS;
    if ((c->pages > 0 && !c->refs) || !c->table || !c->lens || (needs_which && !which)) return invalid(fn, "NULL pointer");
    if (off(c->refs, 4) || off(c->table, 4) || off(c->lens, 4) || off(which, 4) || off(shortfall, 4) || off(ws, 4))
        return misaligned(fn, "pointer not aligned to its element size");
    Bytes bkv, bt;
    if (moves && c->planes > 0 && c->pages > 0) {
        if (!c->kv) return invalid(fn, "kv is NULL");
        if (c->page_bytes < 0 || c->page_stride < c->page_bytes) return invalid(fn, "page_stride < page_bytes");
        if (!span(c->kv, {{c->planes, c->plane_stride}, {c->pages, c->page_stride}}, c->page_bytes, &bkv))
            return invalid(fn, "cache too large, or a negative stride");
        if (c->planes > 1 && c->plane_stride < (c->pages - 1) * c->page_stride + c->page_bytes &&
            c->page_stride < (c->planes - 1) * c->plane_stride + c->page_bytes)
            return invalid(fn, "planes overlap");
    }
    if (!span(c->table, {{c->rows, c->ld_table * 4}}, c->width * 4, &bt)) return invalid(fn, "table too large");
    if (needs_ws && (ws_bytes < mpdt::pages_workspace(c->pages, c->rows) || !ws))
        return invalid(fn, "workspace too small");
    // everything that is written lies apart from everything else
    Bytes parts[7];
    int n = 0;
    parts[n++] = bkv;
    parts[n++] = bt;
    (void)span(c->refs, {{1, 0}}, c->pages * 4, &parts[n++]);
    (void)span(c->lens, {{1, 0}}, c->rows * 4, &parts[n++]);
    if (needs_which) (void)span(which, {{1, 0}}, c->rows * 4, &parts[n++]);
    if (shortfall) (void)span(shortfall, {{1, 0}}, 4, &parts[n++]);
    if (needs_ws) (void)span(ws, {{1, 0}}, mpdt::pages_workspace(c->pages, c->rows), &parts[n++]);
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < i; ++j)
            if (parts[i].meets(parts[j])) return abi_fail(MPDT_ERROR_ALIASING, fn, "operands overlap");
    a->kv = (char*)c->kv;
    a->plane_b = c->plane_stride;
    a->page_stride_b = c->page_stride;
    a->page_bytes = c->page_bytes;
    a->planes = moves ? (int)c->planes : 0;
    a->refs = c->refs;
    a->table = c->table;
    a->ld_table = c->ld_table;
    a->lens = c->lens;
    a->which = which;
    a->width = (int)c->width;
    a->page_size = (int)c->page_size;
    a->ws = (int32_t*)ws;
    a->shortfall = shortfall;
    return MPDT_SUCCESS;
}

}  // namespace

MPDT_EXPORT int64_t cache_pages_workspace(int64_t pages, int64_t rows) {
    return in_dims(pages, 0) && in_dims(rows, 0) ? mpdt::pages_workspace(pages, rows) : -1;
}

MPDT_EXPORT mpdt_status cache_fork(const mpdt_pages* c, const int32_t* parent, int32_t* shortfall, void* workspace,
                                   int64_t workspace_bytes, void* stream) {
    const char* fn = "cache_fork";
    mpdt::PagesArgs a{};
    mpdt_status s = check_pages(fn, c, true, parent, true, shortfall, workspace, workspace_bytes, true, &a);
    if (s != MPDT_SUCCESS || c->rows == 0) return s;
    if ((s = abi_check_device(fn)) != MPDT_SUCCESS) return s;
    return abi_launched(mpdt::launch_cache_fork(a, (hipStream_t)stream), fn);
}

MPDT_EXPORT mpdt_status cache_extend(const mpdt_pages* c, const int32_t* add, int32_t* shortfall, void* workspace,
                                     int64_t workspace_bytes, void* stream) {
    const char* fn = "cache_extend";
    mpdt::PagesArgs a{};
    mpdt_status s = check_pages(fn, c, false, add, true, shortfall, workspace, workspace_bytes, true, &a);
    if (s != MPDT_SUCCESS || c->rows == 0) return s;
    if ((s = abi_check_device(fn)) != MPDT_SUCCESS) return s;
    return abi_launched(mpdt::launch_cache_extend(a, (hipStream_t)stream), fn);
}

MPDT_EXPORT mpdt_status cache_free(const mpdt_pages* c, const int32_t* drop, void* stream) {
    const char* fn = "cache_free";
    mpdt::PagesArgs a{};
    mpdt_status s = check_pages(fn, c, false, drop, true, nullptr, nullptr, 0, false, &a);
    if (s != MPDT_SUCCESS || c->rows == 0) return s;
    if ((s = abi_check_device(fn)) != MPDT_SUCCESS) return s;
    return abi_launched(mpdt::launch_cache_free(a, (hipStream_t)stream), fn);
}

MPDT_EXPORT mpdt_status cache_compact(const mpdt_pages* c, void* workspace, int64_t workspace_bytes, void* stream) {
    const char* fn = "cache_compact";
    mpdt::PagesArgs a{};
    mpdt_status s = check_pages(fn, c, true, nullptr, false, nullptr, workspace, workspace_bytes, true, &a);
    if (s != MPDT_SUCCESS || c->rows == 0 || c->pages == 0) return s;
    if ((s = abi_check_device(fn)) != MPDT_SUCCESS) return s;
    return abi_launched(mpdt::launch_cache_compact(a, (hipStream_t)stream), fn);
}

namespace {

mpdt_status check_logits(const char* fn, int dtype, int64_t rows, int64_t vocab, const void* logits, int64_t ld,
                         const int64_t* targets, Bytes* b) {
    if (dtype != MPDT_BF16 && dtype != MPDT_F16 && dtype != MPDT_F32) return invalid(fn, "unknown type of logits");
    if (!in_dims(rows, 0) || !in_dims(vocab, 1)) return invalid(fn, "rows or vocab out of range");
    if (rows == 0) return MPDT_SUCCESS;
    if (!logits || !targets) return invalid(fn, "logits or targets is NULL");
    if (ld < vocab) return invalid(fn, "ld < vocab");
    if (off(logits, size_of(dtype)) || off(targets, 8))
        return misaligned(fn, "pointer not aligned to its element size");
    if (!span(logits, {{rows, ld * size_of(dtype)}}, vocab * size_of(dtype), b))
        return invalid(fn, "operand too large");
    if (rows > mpdt::MAX_GROUPS) return invalid(fn, "too many rows");
    return MPDT_SUCCESS;
}

}  // namespace

MPDT_EXPORT int64_t token_logprobs_workspace(int dtype, int64_t rows, int64_t vocab, int64_t top) {
    if ((dtype != MPDT_BF16 && dtype != MPDT_F16 && dtype != MPDT_F32) || !in_dims(rows, 0) || !in_dims(vocab, 1) ||
        top < 0 || top > mpdt::LOGPROB_MAX_TOP)
        return -1;
    return mpdt::logprob_workspace(dtype, rows, vocab, (int)top);
}

MPDT_EXPORT mpdt_status token_logprobs(int dtype, int64_t rows, int64_t vocab, const void* logits, int64_t ld,
                                       const int64_t* targets, int64_t top, float* logprob, float* lse,
                                       float* entropy, float* top_logprobs, int64_t* top_indices, void* workspace,
                                       int64_t workspace_bytes, void* stream) {
    const char* fn = "token_logprobs";
    Bytes bx, outs[6];
    mpdt_status s = check_logits(fn, dtype, rows, vocab, logits, ld, targets, &bx);
    if (s != MPDT_SUCCESS) return s;
    if (top < 0 || top > mpdt::LOGPROB_MAX_TOP || top > vocab)
        return invalid(fn, "top must be at most 64 and at most vocab");
    if (rows == 0) return MPDT_SUCCESS;
    if (!logprob || !lse || !entropy || (top > 0 && (!top_logprobs || !top_indices)))
        return invalid(fn, "output is NULL");
    const int64_t need = mpdt::logprob_workspace(dtype, rows, vocab, (int)top);
    if (workspace_bytes < need || (need > 0 && !workspace)) return invalid(fn, "workspace too small");
    if (off(logprob, 4) || off(lse, 4) || off(entropy, 4) || (top > 0 && (off(top_logprobs, 4) || off(top_indices, 8))) ||
        off(workspace, 16))
        return misaligned(fn, "pointer not aligned to its element size (workspace: 16 bytes)");
    Bytes bt;
    (void)span(targets, {{1, 0}}, rows * 8, &bt);
    (void)span(logprob, {{1, 0}}, rows * 4, &outs[0]);
    (void)span(lse, {{1, 0}}, rows * 4, &outs[1]);
    (void)span(entropy, {{1, 0}}, rows * 4, &outs[2]);
    (void)span(top_logprobs, {{top > 0, 0}}, rows * top * 4, &outs[3]);
    (void)span(top_indices, {{top > 0, 0}}, rows * top * 8, &outs[4]);
    (void)span(workspace, {{need > 0, 0}}, need, &outs[5]);
    for (int i = 0; i < 6; ++i) {
        bool meets = outs[i].meets(bx) || outs[i].meets(bt);
        for (int j = 0; j < i; ++j) meets = meets || outs[i].meets(outs[j]);
        if (meets) return abi_fail(MPDT_ERROR_ALIASING, fn, "an output or the workspace overlaps another operand");
    }
    if ((s = abi_check_device(fn)) != MPDT_SUCCESS) return s;
    mpdt::LogprobArgs a{};
    a.logits = (const char*)logits;
    a.ld_b = ld * size_of(dtype);
    a.type = dtype;
    a.targets = targets;
    a.rows = (int)rows;
    a.vocab = (int)vocab;
    a.top = (int)top;
    a.logprob = logprob;
    a.lse = lse;
    a.entropy = entropy;
    a.top_logprob = top_logprobs;
    a.top_index = top_indices;
    a.ws = (char*)workspace;
    return abi_launched(mpdt::launch_token_logprobs(a, (hipStream_t)stream), fn);
}

MPDT_EXPORT mpdt_status token_logprobs_backward(int dtype, int64_t rows, int64_t vocab, const void* logits, int64_t ld,
                                                const int64_t* targets, const float* lse, const float* entropy,
                                                const float* g_logprob, const float* g_entropy, void* grad,
                                                int64_t ld_grad, void* stream) {
    const char* fn = "token_logprobs_backward";
    Bytes bx, bg, ins[5];
    mpdt_status s = check_logits(fn, dtype, rows, vocab, logits, ld, targets, &bx);
    if (s != MPDT_SUCCESS) return s;
    if (rows == 0) return MPDT_SUCCESS;
    if (!mpdt::logprob_fits(dtype, rows, vocab)) return invalid(fn, "too many rows");
    if (!lse || !entropy || !grad) return invalid(fn, "lse, entropy or grad is NULL");
    if (ld_grad < vocab) return invalid(fn, "ld_grad < vocab");
    if (off(lse, 4) || off(entropy, 4) || off(g_logprob, 4) || off(g_entropy, 4) || off(grad, size_of(dtype)))
        return misaligned(fn, "pointer not aligned to its element size");
    if (!span(grad, {{rows, ld_grad * size_of(dtype)}}, vocab * size_of(dtype), &bg))
        return invalid(fn, "operand too large");
    (void)span(targets, {{1, 0}}, rows * 8, &ins[0]);
    (void)span(lse, {{1, 0}}, rows * 4, &ins[1]);
    (void)span(entropy, {{1, 0}}, rows * 4, &ins[2]);
    (void)span(g_logprob, {{g_logprob != nullptr, 0}}, rows * 4, &ins[3]);
    (void)span(g_entropy, {{g_entropy != nullptr, 0}}, rows * 4, &ins[4]);
    bool meets = bg.meets(bx);
    for (const Bytes& b : ins) meets = meets || bg.meets(b);
    if (meets) return abi_fail(MPDT_ERROR_ALIASING, fn, "grad overlaps an input");
    if ((s = abi_check_device(fn)) != MPDT_SUCCESS) return s;
    mpdt::LogprobArgs a{};
    a.logits = (const char*)logits;
    a.ld_b = ld * size_of(dtype);
    a.type = dtype;
    a.targets = targets;
    a.rows = (int)rows;
    a.vocab = (int)vocab;
    a.lse = const_cast<float*>(lse);
    a.entropy = const_cast<float*>(entropy);
    a.g_logprob = g_logprob;
    a.g_entropy = g_entropy;
    a.grad = (char*)grad;
    a.ld_grad_b = ld_grad * size_of(dtype);
    return abi_launched(mpdt::launch_token_logprobs_backward(a, (hipStream_t)stream), fn);
}
