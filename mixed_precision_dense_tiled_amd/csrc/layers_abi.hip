// layers_abi.hip -- the C ABI of a decoder layer's operators (mpdt_layers.h):
// host-side argument validation and launch.  No device code lives here.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <cmath>

#include "abi_common.hpp"
#include "layers.hpp"
#include "mpdt_layers.h"
#include "serving_checks.hpp"

static_assert(MPDT_NORM_PLAIN == mpdt::NORM_PLAIN && MPDT_NORM_I8_ROWS == mpdt::NORM_I8_ROWS &&
                  MPDT_NORM_E4M3_ROWS == mpdt::NORM_E4M3_ROWS && MPDT_NORM_E4M3_BLOCKS == mpdt::NORM_E4M3_BLOCKS,
              "outputs of a norm in the C ABI and the kernels agree");

namespace {

mpdt_status aliased(const char* fn, const char* what) { return abi_fail(MPDT_ERROR_ALIASING, fn, what); }

// A matrix of a call, for its checks.
struct Mat {
    const void* p;
    int64_t rows, cols, ld;
    int es;                 // bytes of an element
    const char* name;
    Bytes bytes{};
    bool is(const Mat& o) const { return p == o.p && ld == o.ld && es == o.es; }
};
mpdt_status check_mat(const char* fn, Mat& m) {
    if (!m.p) return invalid(fn, "NULL pointer");
    if (m.ld < m.cols) return invalid(fn, "a leading dimension is smaller than its row");
    if (off(m.p, m.es)) return misaligned(fn, "pointer not aligned to its element size");
    if (m.ld > kMaxSpan || !span(m.p, {{m.rows, m.ld * m.es}}, m.cols * m.es, &m.bytes))
        return invalid(fn, "operand too large");
    return MPDT_SUCCESS;
}
mpdt_status check_vec(const char* fn, const void* p, int64_t n, int es, Bytes* out) {
    if (!p) return invalid(fn, "NULL pointer");
    if (off(p, es)) return misaligned(fn, "pointer not aligned to its element size");
    out->lo = reinterpret_cast<uintptr_t>(p);
    out->hi = out->lo + (uintptr_t)(n * es);
    return MPDT_SUCCESS;
}

// Rows of two operands with one stride between tokens that lie side by side within
// it, as the slices of one wide row do.
bool side_by_side(const void* p, int64_t span_p, const void* q, int64_t span_q, int64_t stride) {
    if (stride <= 0) return false;
    const int64_t d = reinterpret_cast<intptr_t>(q) - reinterpret_cast<intptr_t>(p);
    const int64_t at = (d % stride + stride) % stride;
    return at >= span_p && at + span_q <= stride;
}

bool float_type(int t) { return t == MPDT_BF16 || t == MPDT_F16 || t == MPDT_F32; }
bool half_type(int t) { return t == MPDT_BF16 || t == MPDT_F16; }

mpdt_status check_norm(const char* fn, int dtype, int64_t rows, int64_t dim, int w_dtype) {
    if (!float_type(dtype)) return invalid(fn, "rows must be BF16, FP16 or FP32");
    if (w_dtype != dtype && w_dtype != MPDT_F32) return invalid(fn, "the weight must have the rows' type or FP32");
    if (!in_dims(rows, 0) || dim < 1 || dim > mpdt::NORM_MAX_DIM)
        return invalid(fn, "rows out of range, or dim outside 1 .. 32768");
    return MPDT_SUCCESS;
}

}  // namespace

#define TRY(call)                                  \
    do {                                           \
        const mpdt_status s_ = (call);             \
        if (s_ != MPDT_SUCCESS) return s_;         \
    } while (0)

MPDT_EXPORT mpdt_status rms_norm(int dtype, int64_t rows, int64_t dim, const void* x, int64_t ldx,
                                 const void* residual, int64_t ld_res, int w_dtype, const void* weight, double eps,
                                 int norm_out, void* out, int64_t ld_out, float* scales, int64_t ld_scales,
                                 void* h_out, int64_t ld_h, float* rstd, void* stream) {
    const char* fn = "rms_norm";
    TRY(check_norm(fn, dtype, rows, dim, w_dtype));
    if (rows > mpdt::NORM_MAX_ROWS) return invalid(fn, "too many rows: at most 4194303 to a call");
    if (!(eps >= 0) || !std::isfinite(eps)) return invalid(fn, "eps must be finite and not negative");
    if (norm_out < MPDT_NORM_PLAIN || norm_out > MPDT_NORM_E4M3_BLOCKS) return invalid(fn, "unknown output");
    if (h_out && !residual) return invalid(fn, "h_out needs a residual");
    if (rows == 0) return MPDT_SUCCESS;
    const int es = size_of(dtype), os = norm_out == MPDT_NORM_PLAIN ? es : 1;
    Mat mx{x, rows, dim, ldx, es, "x"}, mr{residual, rows, dim, ld_res, es, "residual"},
        mo{out, rows, dim, ld_out, os, "out"}, mh{h_out, rows, dim, ld_h, es, "h_out"};
    Bytes bw, brstd;
    TRY(check_mat(fn, mx));
    if (residual) TRY(check_mat(fn, mr));
    TRY(check_mat(fn, mo));
    if (h_out) TRY(check_mat(fn, mh));
    TRY(check_vec(fn, weight, dim, size_of(w_dtype), &bw));
    if (rstd) TRY(check_vec(fn, rstd, rows, 4, &brstd));
    const int64_t cols = norm_out == MPDT_NORM_E4M3_BLOCKS ? (dim + 127) / 128 : 1;
    Mat ms{scales, rows, cols, ld_scales, 4, "scales"};
    if (norm_out != MPDT_NORM_PLAIN) TRY(check_mat(fn, ms));
    // (an absent operand spans nothing)
    const bool out_in_place = norm_out == MPDT_NORM_PLAIN && (mo.is(mx) || (residual && mo.is(mr)));
    if (!out_in_place && (mo.bytes.meets(mx.bytes) || mo.bytes.meets(mr.bytes)))
        return aliased(fn, "out overlaps x or the residual");
    const bool h_in_place = h_out && (mh.is(mx) || mh.is(mr));
    if (h_out && !h_in_place && (mh.bytes.meets(mx.bytes) || mh.bytes.meets(mr.bytes)))
        return aliased(fn, "h_out overlaps x or the residual");
    // in place of one operand, the other must lie apart
    if ((out_in_place || h_in_place) && residual && mx.bytes.meets(mr.bytes) && !mx.is(mr))
        return aliased(fn, "x and the residual overlap, and one is written");
    if (mo.bytes.meets(mh.bytes)) return aliased(fn, "out overlaps h_out");
    for (const Bytes& b : {bw, ms.bytes, brstd})
        if (b.meets(mo.bytes) || b.meets(mh.bytes)) return aliased(fn, "out or h_out overlaps a vector");
    for (const Bytes& b : {mx.bytes, mr.bytes, bw})
        if (b.meets(ms.bytes) || b.meets(brstd)) return aliased(fn, "scales or rstd overlap an input");
    if (ms.bytes.meets(brstd)) return aliased(fn, "scales overlap rstd");
    TRY(abi_check_device(fn));
    mpdt::NormArgs a{};
    a.x = (const char*)x;
    a.x_b = ldx * es;
    a.residual = (const char*)residual;
    a.res_b = ld_res * es;
    a.h = (char*)h_out;
    a.h_b = ld_h * es;
    a.weight = (const char*)weight;
    a.eps = eps;
    a.out = (char*)out;
    a.out_b = ld_out * os;
    a.scales = scales;
    a.ld_scales = ld_scales;
    a.rstd = rstd;
    a.rows = (int)rows;
    a.dim = (int)dim;
    a.type = dtype;
    a.w_f32 = w_dtype == MPDT_F32;
    a.quant = norm_out;
    return abi_launched(mpdt::launch_rms_norm(a, (hipStream_t)stream), fn);
}

MPDT_EXPORT int64_t rms_norm_backward_workspace(int64_t rows, int64_t dim) {
    const char* fn = "rms_norm_backward_workspace";
    if (check_norm(fn, MPDT_F32, rows, dim, MPDT_F32) != MPDT_SUCCESS) return -1;
    return mpdt::rms_norm_backward_ws(rows, dim);
}

MPDT_EXPORT mpdt_status rms_norm_backward(int dtype, int64_t rows, int64_t dim, const void* grad, int64_t ld_grad,
                                          const void* h, int64_t ld_h, int w_dtype, const void* weight,
                                          const float* rstd, const void* grad_residual, int64_t ld_gres,
                                          void* grad_h, int64_t ld_gh, float* grad_weight, void* workspace,
                                          int64_t workspace_bytes, void* stream) {
    const char* fn = "rms_norm_backward";
    TRY(check_norm(fn, dtype, rows, dim, w_dtype));
    const int es = size_of(dtype);
    Mat mg{grad, rows, dim, ld_grad, es, "grad"}, mh{h, rows, dim, ld_h, es, "h"},
        mr{grad_residual, rows, dim, ld_gres, es, "grad_residual"}, mo{grad_h, rows, dim, ld_gh, es, "grad_h"};
    Bytes bw, brstd, bgw, bws;
    TRY(check_vec(fn, grad_weight, dim, 4, &bgw));
    if (rows > 0) {
        TRY(check_mat(fn, mg));
        TRY(check_mat(fn, mh));
        if (grad_residual) TRY(check_mat(fn, mr));
        TRY(check_mat(fn, mo));
        TRY(check_vec(fn, weight, dim, size_of(w_dtype), &bw));
        TRY(check_vec(fn, rstd, rows, 4, &brstd));
    }
    const int64_t need = mpdt::rms_norm_backward_ws(rows, dim);
    if (workspace_bytes < need || (need && !workspace)) return invalid(fn, "workspace too small");
    if (need) {
        if (off(workspace, 4)) return misaligned(fn, "workspace not aligned to 4 bytes");
        TRY(check_vec(fn, workspace, need / 4, 4, &bws));
    }
    const bool in_place = rows > 0 && (mo.is(mg) || (grad_residual && mo.is(mr)));
    if (mo.bytes.meets(mh.bytes)) return aliased(fn, "grad_h overlaps h");
    if (!in_place && (mo.bytes.meets(mg.bytes) || mo.bytes.meets(mr.bytes)))
        return aliased(fn, "grad_h overlaps a gradient");
    if (in_place && grad_residual && mg.bytes.meets(mr.bytes) && !mg.is(mr))
        return aliased(fn, "the gradients overlap, and one is written");
    for (const Bytes& b : {mg.bytes, mh.bytes, mr.bytes, mo.bytes, bw, brstd})
        if (b.meets(bgw) || b.meets(bws)) return aliased(fn, "grad_weight or the workspace overlap an operand");
    if (mo.bytes.meets(bw) || mo.bytes.meets(brstd)) return aliased(fn, "grad_h overlaps a vector");
    if (bgw.meets(bws)) return aliased(fn, "grad_weight overlaps the workspace");
    TRY(abi_check_device(fn));
    mpdt::NormGradArgs a{};
    a.grad = (const char*)grad;
    a.grad_b = ld_grad * es;
    a.h = (const char*)h;
    a.h_b = ld_h * es;
    a.weight = (const char*)weight;
    a.rstd = rstd;
    a.grad_res = (const char*)grad_residual;
    a.gres_b = ld_gres * es;
    a.grad_h = (char*)grad_h;
    a.gh_b = ld_gh * es;
    a.grad_weight = grad_weight;
    a.ws = (float*)workspace;
    a.rows = (int)rows;
    a.dim = (int)dim;
    a.type = dtype;
    a.w_f32 = w_dtype == MPDT_F32;
    return abi_launched(mpdt::launch_rms_norm_backward(a, (hipStream_t)stream), fn);
}

MPDT_EXPORT mpdt_status paged_kv_append_rope(const mpdt_paged_kv* kv, const mpdt_sequences* sq, int dtype,
                                             const void* k_new, int64_t k_token, int64_t k_head, const void* v_new,
                                             int64_t v_token, int64_t v_head, const float* inv_freq, int64_t pairs,
                                             int interleaved, int64_t heads, const void* q, int64_t q_token,
                                             int64_t q_head, void* q_out, int64_t qo_token, int64_t qo_head,
                                             void* stream) {
    const char* fn = "paged_kv_append_rope";
    mpdt::RopeArgs r{};
    mpdt::AppendArgs& a = r.ap;
    Bytes bk, bv, nk, nv, bf, bq, bo, bt;
    TRY(check_cache(fn, kv, sq, &a.kv, &a.sv, &bk, &bv));
    if (!half_type(dtype) || (kv->dtype != MPDT_E4M3 && dtype != kv->dtype))
        return invalid(fn, "new keys must have the cache's type, or a 16-bit one for an E4M3 cache");
    if (pairs < 1 || 2 * pairs > kv->dim) return invalid(fn, "pairs must be between 1 and dim / 2");
    if (interleaved != 0 && interleaved != 1) return invalid(fn, "interleaved must be 0 or 1");
    if (heads < 0 || heads > 65535) return invalid(fn, "heads out of range");
    TRY(check_vec(fn, inv_freq, pairs, 4, &bf));
    if (sq->tokens == 0 || sq->seqs == 0) return MPDT_SUCCESS;
    if (sq->tokens > mpdt::MAX_GROUPS) return invalid(fn, "too many tokens");
    if (!k_new || !v_new) return invalid(fn, "NULL pointer");
    if ((heads > 0) != (q != nullptr) || (heads > 0) != (q_out != nullptr))
        return invalid(fn, "q and q_out go with heads, neither without");
    if (off(k_new, 16) || off(v_new, 16) || k_token % 8 || k_head % 8 || v_token % 8 || v_head % 8)
        return misaligned(fn, "new rows must start on 16-byte boundaries");
    if (heads > 0 && (off(q, 16) || off(q_out, 16) || q_token % 8 || q_head % 8 || qo_token % 8 || qo_head % 8))
        return misaligned(fn, "rows of q must start on 16-byte boundaries");
    const int64_t row = kv->dim * 2;
    if (!span(k_new, {{sq->tokens, k_token * 2}, {kv->kv_heads, k_head * 2}}, row, &nk) ||
        !span(v_new, {{sq->tokens, v_token * 2}, {kv->kv_heads, v_head * 2}}, row, &nv) ||
        !span(q, {{sq->tokens, q_token * 2}, {heads, q_head * 2}}, row, &bq) ||
        !span(q_out, {{sq->tokens, qo_token * 2}, {heads, qo_head * 2}}, row, &bo))
        return invalid(fn, "operand too large, or a negative stride");
    // what the call reads besides: where its tokens belong
    Bytes small[4];
    TRY(check_vec(fn, sq->cu_q, sq->seqs + 1, 4, &small[0]));
    TRY(check_vec(fn, sq->lens, sq->seqs, 4, &small[1]));
    if (!span(sq->table, {{sq->seqs, sq->ld_table * 4}}, sq->width * 4, &bt)) return invalid(fn, "table too large");
    for (const Bytes* b : {&nk, &nv, &bq, &bf, &small[0], &small[1], &bt}) {
        if (b->meets(bk) || b->meets(bv)) return aliased(fn, "an operand overlaps the cache");
        if (b == &bq || !b->meets(bo)) continue;
        // (q_out may be the q of a tensor that holds q, k and v of a token side by side)
        const int64_t own = (heads - 1) * qo_head * 2 + row;
        if (b == &nk && k_token == qo_token &&
            side_by_side(q_out, own, k_new, (kv->kv_heads - 1) * k_head * 2 + row, k_token * 2)) continue;
        if (b == &nv && v_token == qo_token &&
            side_by_side(q_out, own, v_new, (kv->kv_heads - 1) * v_head * 2 + row, v_token * 2)) continue;
        return aliased(fn, "q_out overlaps an operand");
    }
    if (bk.meets(bo) || bv.meets(bo)) return aliased(fn, "q_out overlaps the cache");
    if (bo.meets(bq) && !(q == q_out && q_token == qo_token && q_head == qo_head))
        return aliased(fn, "q_out overlaps q other than exactly");
    if (!apart({{kv->pages, a.kv.page_b}, {kv->page_size, a.kv.slot_b}, {kv->kv_heads, a.kv.head_b}},
               kv->dim * size_of(kv->dtype)))
        return aliased(fn, "rows of the cache overlap each other");
    if (heads > 0 && !apart({{sq->tokens, qo_token * 2}, {heads, qo_head * 2}}, row))
        return aliased(fn, "rows of q_out overlap each other");
    TRY(abi_check_device(fn));
    a.k_new = (const char*)k_new;
    a.v_new = (const char*)v_new;
    a.k_tok_b = k_token * 2;
    a.k_head_b = k_head * 2;
    a.v_tok_b = v_token * 2;
    a.v_head_b = v_head * 2;
    a.type = dtype;
    r.inv_freq = inv_freq;
    r.pairs = (int)pairs;
    r.interleaved = interleaved;
    r.heads = (int)heads;
    r.q = (const char*)q;
    r.q_tok_b = q_token * 2;
    r.q_head_b = q_head * 2;
    r.q_out = (char*)q_out;
    r.qo_tok_b = qo_token * 2;
    r.qo_head_b = qo_head * 2;
    return abi_launched(mpdt::launch_paged_append_rope(r, (hipStream_t)stream), fn);
}

namespace {

// The groups and one stack of matrices (groups of rows x cols at stride elements).
struct Stack {
    const void* p;
    int64_t rows, cols, ld, stride;
    int es;
    bool written;
    Bytes bytes{};
};
mpdt_status check_stack(const char* fn, int64_t groups, Stack& m) {
    if (!m.p) return invalid(fn, "NULL pointer");
    if (m.ld < m.cols) return invalid(fn, "a leading dimension is smaller than its row");
    if (off(m.p, m.es)) return misaligned(fn, "pointer not aligned to its element size");
    if (m.ld > kMaxSpan || m.stride > kMaxSpan ||
        !span(m.p, {{groups, m.stride * m.es}, {m.rows, m.ld * m.es}}, m.cols * m.es, &m.bytes))
        return invalid(fn, "operand too large, or a negative stride");
    if (m.written && !apart({{groups, m.stride}, {m.rows, m.ld}}, m.cols))
        return aliased(fn, "rows of the output overlap each other");
    return MPDT_SUCCESS;
}
mpdt_status check_groups(const char* fn, int64_t groups, int64_t rows, int64_t N, int64_t K, const int32_t* offsets,
                         Bytes* bo) {
    if (groups < 0 || groups > 65535) return invalid(fn, "groups must be at most 65535");
    if (!in_dims(rows, 0) || !in_dims(N, 0) || !in_dims(K, 0)) return invalid(fn, "rows, N or K out of range");
    return check_vec(fn, offsets, groups + 1, 4, bo);
}

}  // namespace

MPDT_EXPORT mpdt_status gemm_grouped(int dtype, int64_t groups, int64_t rows, int64_t N, int64_t K, const void* A,
                                     int64_t lda, const void* B, int64_t ldb, int64_t stride_b, int trans_b,
                                     const int32_t* offsets, void* D, int64_t ldd, int d16, void* stream) {
    const char* fn = "gemm_grouped";
    if (!half_type(dtype)) return invalid(fn, "operands must be BF16 or FP16");
    if ((trans_b != 0 && trans_b != 1) || (d16 != 0 && d16 != 1)) return invalid(fn, "trans_b and d16 must be 0 or 1");
    Bytes boff;
    TRY(check_groups(fn, groups, rows, N, K, offsets, &boff));
    if (groups == 0 || rows == 0 || N == 0) return MPDT_SUCCESS;
    Mat ma{A, rows, K, lda, 2, "A"}, md{D, rows, N, ldd, d16 ? 2 : 4, "D"};
    Stack mb{B, trans_b ? N : K, trans_b ? K : N, ldb, stride_b, 2, false};
    if (K > 0) {
        TRY(check_mat(fn, ma));
        TRY(check_stack(fn, groups, mb));
    }
    TRY(check_mat(fn, md));
    if (md.bytes.meets(ma.bytes) || md.bytes.meets(mb.bytes) || md.bytes.meets(boff))
        return aliased(fn, "D overlaps an operand");
    mpdt::GroupedArgs a{};
    a.A = (const char*)A;
    a.B = (const char*)B;
    a.D = (char*)D;
    a.lda_b = lda * 2;
    a.ldb_b = ldb * 2;
    a.group_b = stride_b * 2;
    a.ldd = ldd;
    a.offsets = offsets;
    a.groups = (int)groups;
    a.rows = (int)rows;
    a.N = (int)N;
    a.K = (int)K;
    a.out16 = d16;
    const int mode = trans_b ? mpdt::GROUPED_NT : mpdt::GROUPED_NN;
    if (!mpdt::grouped_fits(mode, a)) return invalid(fn, "too many tiles");
    TRY(abi_check_device(fn));
    return abi_launched(mpdt::launch_grouped(dtype == MPDT_BF16 ? mpdt::GroupedType::BF16 : mpdt::GroupedType::F16,
                                             mode, a, (hipStream_t)stream), fn);
}

MPDT_EXPORT mpdt_status gemm_grouped_wgrad(int dtype, int64_t groups, int64_t rows, int64_t N, int64_t K,
                                           const void* A, int64_t lda, const void* G, int64_t ldg,
                                           const int32_t* offsets, void* D, int64_t ldd, int64_t stride_d, int d16,
                                           void* stream) {
    const char* fn = "gemm_grouped_wgrad";
    if (!half_type(dtype)) return invalid(fn, "operands must be BF16 or FP16");
    if (d16 != 0 && d16 != 1) return invalid(fn, "d16 must be 0 or 1");
    Bytes boff;
    TRY(check_groups(fn, groups, rows, N, K, offsets, &boff));
    if (groups == 0 || N == 0 || K == 0) return MPDT_SUCCESS;
    Mat ma{A, rows, K, lda, 2, "A"}, mg{G, rows, N, ldg, 2, "G"};
    Stack md{D, K, N, ldd, stride_d, d16 ? 2 : 4, true};
    if (rows > 0) {
        TRY(check_mat(fn, ma));
        TRY(check_mat(fn, mg));
    }
    TRY(check_stack(fn, groups, md));
    if (md.bytes.meets(ma.bytes) || md.bytes.meets(mg.bytes) || md.bytes.meets(boff))
        return aliased(fn, "D overlaps an operand");
    mpdt::GroupedArgs a{};
    a.A = (const char*)A;
    a.B = (const char*)G;
    a.D = (char*)D;
    a.lda_b = lda * 2;
    a.ldb_b = ldg * 2;
    a.ldd = ldd;
    a.group_d = stride_d;
    a.offsets = offsets;
    a.groups = (int)groups;
    a.rows = (int)rows;
    a.M = (int)K;
    a.N = (int)N;
    a.out16 = d16;
    if (!mpdt::grouped_fits(mpdt::GROUPED_TN, a)) return invalid(fn, "too many tiles");
    TRY(abi_check_device(fn));
    return abi_launched(mpdt::launch_grouped(dtype == MPDT_BF16 ? mpdt::GroupedType::BF16 : mpdt::GroupedType::F16,
                                             mpdt::GROUPED_TN, a, (hipStream_t)stream), fn);
}

MPDT_EXPORT mpdt_status gemm_grouped_w8a8(int64_t groups, int64_t rows, int64_t N, int64_t K, const int8_t* X,
                                          int64_t ldx, const float* x_scale, const int8_t* W, int64_t ldw,
                                          int64_t stride_w, const float* w_scale, int64_t ld_ws, const float* bias,
                                          int64_t ld_bias, const int32_t* offsets, uint16_t* Y, int64_t ldy,
                                          void* stream) {
    const char* fn = "gemm_grouped_w8a8";
    Bytes boff, bxs;
    TRY(check_groups(fn, groups, rows, N, K, offsets, &boff));
    if (groups == 0 || rows == 0 || N == 0) return MPDT_SUCCESS;
    Mat mx{X, rows, K, ldx, 1, "X"}, my{Y, rows, N, ldy, 2, "Y"}, ms{w_scale, groups, N, ld_ws, 4, "w_scale"},
        mb{bias, groups, N, ld_bias, 4, "bias"};
    Stack mw{W, N, K, ldw, stride_w, 1, false};
    if (K > 0) {
        TRY(check_mat(fn, mx));
        TRY(check_stack(fn, groups, mw));
    }
    TRY(check_vec(fn, x_scale, rows, 4, &bxs));
    TRY(check_mat(fn, ms));
    if (bias) TRY(check_mat(fn, mb));
    TRY(check_mat(fn, my));
    for (const Bytes& b : {mx.bytes, mw.bytes, bxs, ms.bytes, mb.bytes, boff})
        if (my.bytes.meets(b)) return aliased(fn, "Y overlaps an operand");
    mpdt::GroupedArgs a{};
    a.A = (const char*)X;
    a.B = (const char*)W;
    a.D = (char*)Y;
    a.lda_b = ldx;
    a.ldb_b = ldw;
    a.group_b = stride_w;
    a.ldd = ldy;
    a.offsets = offsets;
    a.groups = (int)groups;
    a.rows = (int)rows;
    a.N = (int)N;
    a.K = (int)K;
    a.out16 = 1;
    a.x_scale = x_scale;
    a.w_scale = w_scale;
    a.bias = bias;
    a.ld_ws = ld_ws;
    a.ld_bias = ld_bias;
    if (!mpdt::grouped_fits(mpdt::GROUPED_NT, a)) return invalid(fn, "too many tiles");
    TRY(abi_check_device(fn));
    return abi_launched(mpdt::launch_grouped(mpdt::GroupedType::I8, mpdt::GROUPED_NT, a, (hipStream_t)stream), fn);
}
