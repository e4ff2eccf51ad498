// serving_checks.hpp -- host-side checks that the C ABI of the serving operators
// (serving_abi.hip) and of the layers (layers_abi.hip) share: spans of strided
// operands, overlaps, and a paged cache with its batch.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include <algorithm>
#include <initializer_list>

#include "abi_common.hpp"
#include "mpdt_serving.h"
#include "serving.hpp"

namespace {

using mpdt::abi_check_device;
using mpdt::abi_fail;
using mpdt::abi_launched;

constexpr int64_t kMaxDim = int64_t(1) << 30;
constexpr int64_t kMaxSpan = int64_t(1) << 46;   // bytes

inline mpdt_status invalid(const char* fn, const char* what) { return abi_fail(MPDT_ERROR_INVALID_VALUE, fn, what); }
inline mpdt_status misaligned(const char* fn, const char* what) { return abi_fail(MPDT_ERROR_MISALIGNED, fn, what); }

inline bool off(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }
inline bool in_dims(int64_t v, int64_t lo) { return v >= lo && v <= kMaxDim; }

// A strided operand: bytes from its first to past its last.
struct Bytes {
    uintptr_t lo = 0, hi = 0;
    bool meets(const Bytes& o) const { return lo < o.hi && o.lo < hi; }
};
struct Axis {
    int64_t n, stride;   // stride in bytes
};
// False where a stride is negative or the operand spans 2^46 bytes or more.
inline bool span(const void* p, std::initializer_list<Axis> axes, int64_t inner, Bytes* out) {
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
inline bool apart(std::initializer_list<Axis> axes, int64_t inner) {
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

inline int size_of(int dtype) { return dtype == MPDT_F32 ? 4 : dtype == MPDT_E4M3 ? 1 : 2; }

// The cache and the batch, checked and in the kernels' form; k and v: their bytes.
inline mpdt_status check_cache(const char* fn, const mpdt_paged_kv* kv, const mpdt_sequences* sq, mpdt::PagedKV* o,
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

}  // namespace
