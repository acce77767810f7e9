// ops_api.cpp -- the C ABI of the routing and 4-bit operators: argument checks,
// then one launcher each (route.cu, moe.cu, fp4_quant.cu, fp4_gemm.cu).
#include "../../include/c3_api.h"
#include "c3_internal.h"

#include <cmath>

namespace c3 {

constexpr int64_t kMaxRows = 0x7FFFFFFF;  // row numbers are 32-bit
constexpr int kMaxTopk = 32;              // a warp's lanes
constexpr int kMaxExperts = 1024;

static_assert(C3_TILE_ROWS == kTileRows, "tile rows");

static bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
static bool is_type(int t) { return t == C3_F32 || t == C3_BF16; }
static size_t type_bytes(int t) { return t == C3_BF16 ? 2 : 4; }

static int check_router(const c3_router* r, RouteArgs* a) {
    if (!r) return set_error(C3_EINVAL, "router is NULL");
    if (r->experts < 1 || r->experts > kMaxExperts) return set_error(C3_EINVAL, "experts must be 1..1024");
    if (r->groups < 1 || r->experts % r->groups) return set_error(C3_EINVAL, "groups must divide experts");
    if (r->topk_groups < 1 || r->topk_groups > r->groups) return set_error(C3_EINVAL, "topk_groups must be 1..groups");
    if (r->topk < 1 || r->topk > kMaxTopk || r->topk > r->experts / r->groups * r->topk_groups)
        return set_error(C3_EINVAL, "topk must be 1..32 and at most the experts of topk_groups groups");
    if (r->group_best != 1 && r->group_best != 2) return set_error(C3_EINVAL, "group_best must be 1 or 2");
    if (r->group_best == 2 && r->experts / r->groups < 2)
        return set_error(C3_EINVAL, "group_best 2 needs two experts a group");
    if (r->score != C3_SCORE_SOFTMAX && r->score != C3_SCORE_SIGMOID) return set_error(C3_EINVAL, "unknown score");
    if (r->renorm != 0 && r->renorm != 1) return set_error(C3_EINVAL, "renorm must be 0 or 1");
    if (!is_type(r->logits_type)) return set_error(C3_EINVAL, "unknown logits_type");
    if (!std::isfinite(r->scale)) return set_error(C3_EINVAL, "scale must be finite");
    if (!aligned(r->bias, 4)) return set_error(C3_EALIGN, "bias must be 4-byte aligned");
    a->bias = r->bias;
    a->experts = r->experts;
    a->topk = r->topk;
    a->groups = r->groups;
    a->topk_groups = r->topk_groups;
    a->group_best = r->group_best;
    a->score = r->score;
    a->renorm = r->renorm;
    a->by_score = r->bias != nullptr;
    a->pairs = r->groups > 1 && r->group_best == 2;
    a->scale = r->scale;
    return C3_OK;
}

static int check_tokens(int64_t tokens, int topk) {
    if (tokens < 0) return set_error(C3_EINVAL, "negative tokens");
    if (topk < 1 || topk > kMaxTopk) return set_error(C3_EINVAL, "topk must be 1..32");
    if (tokens > kMaxRows / topk) return set_error(C3_EUNSUP, "more than 2^31 choices");
    return C3_OK;
}

static int check_fp4(const c3_fp4* m, Fp4* q) {
    if (!m) return set_error(C3_EINVAL, "4-bit matrix is NULL");
    if (m->format != C3_FP4_MX && m->format != C3_FP4_NV) return set_error(C3_EINVAL, "unknown 4-bit format");
    if (m->rows < 0 || m->cols < 1 || m->count < 1)
        return set_error(C3_EINVAL, "a 4-bit matrix needs rows >= 0, cols >= 1 and count >= 1");
    if (m->format == C3_FP4_MX && m->tensor_scale) return set_error(C3_EINVAL, "C3_FP4_MX has no tensor_scale");
    // (a tile's rows past the last one must still have 32-bit numbers)
    if (m->cols > kMaxRows || m->count > 65535 || (m->rows && m->count > (kMaxRows - 1023) / m->rows))
        return set_error(C3_EUNSUP, "4-bit matrix near or above 2^31 rows or columns");
    if (m->rows) {
        if (!m->codes || !m->scales) return set_error(C3_EINVAL, "codes or scales is NULL");
        if (!aligned(m->codes, 16) || !aligned(m->scales, 16))
            return set_error(C3_EALIGN, "codes and scales must be 16-byte aligned");
    }
    if (!aligned(m->tensor_scale, 4)) return set_error(C3_EALIGN, "tensor_scale must be 4-byte aligned");
    q->codes = static_cast<uint8_t*>(m->codes);
    q->scales = static_cast<uint8_t*>(m->scales);
    q->tensor_scale = m->tensor_scale;
    q->rows = m->rows;
    q->cols = m->cols;
    q->count = m->count;
    q->nv = m->format == C3_FP4_NV;
    return C3_OK;
}

static int check_product(const Fp4& a, const Fp4& b, const void* C, int c_type, int sm_budget) {
    if (a.cols != b.cols) return set_error(C3_EINVAL, "the operands' columns differ");
    if (a.nv != b.nv) return set_error(C3_EINVAL, "the operands' formats differ");
    if (!is_type(c_type)) return set_error(C3_EINVAL, "unknown c_type");
    if (sm_budget < 0) return set_error(C3_EINVAL, "negative sm_budget");
    if (a.rows && b.rows) {
        if (!C) return set_error(C3_EINVAL, "C is NULL");
        if (!aligned(C, 16)) return set_error(C3_EALIGN, "C must be 16-byte aligned");
    }
    return C3_OK;
}

}  // namespace c3

using namespace c3;

extern "C" {

int c3_route(const c3_router* r, const void* logits, int64_t ld, int64_t tokens, int32_t* idx, float* weights,
             c3_stream s) {
    RouteArgs a;
    int rc = check_router(r, &a);
    if (rc) return rc;
    if ((rc = check_tokens(tokens, a.topk))) return rc;
    if (ld < a.experts) return set_error(C3_EINVAL, "ld is below experts");
    if (tokens == 0) return C3_OK;
    if (!logits || !idx || !weights) return set_error(C3_EINVAL, "logits, idx or weights is NULL");
    if (!aligned(logits, type_bytes(r->logits_type)) || !aligned(idx, 4) || !aligned(weights, 4))
        return set_error(C3_EALIGN, "a pointer is not aligned to its element");
    return route_launch(logits, r->logits_type == C3_BF16, ld, tokens, a, idx, weights, static_cast<cudaStream_t>(s));
}

int c3_route_backward(const c3_router* r, const void* logits, int64_t ld, int64_t tokens, const int32_t* idx,
                      const float* dweights, void* dlogits, int64_t dld, c3_stream s) {
    RouteArgs a;
    int rc = check_router(r, &a);
    if (rc) return rc;
    if ((rc = check_tokens(tokens, a.topk))) return rc;
    if (ld < a.experts || dld < a.experts) return set_error(C3_EINVAL, "a row distance is below experts");
    if (tokens == 0) return C3_OK;
    if (!logits || !idx || !dweights || !dlogits)
        return set_error(C3_EINVAL, "logits, idx, dweights or dlogits is NULL");
    const size_t sz = type_bytes(r->logits_type);
    if (!aligned(logits, sz) || !aligned(dlogits, sz) || !aligned(idx, 4) || !aligned(dweights, 4))
        return set_error(C3_EALIGN, "a pointer is not aligned to its element");
    return route_backward_launch(logits, r->logits_type == C3_BF16, ld, tokens, a, idx, dweights, dlogits, dld,
                                 static_cast<cudaStream_t>(s));
}

int64_t c3_moe_rows(int64_t tokens, int topk, int experts) {
    int rc = check_tokens(tokens, topk);
    if (rc) return rc;
    if (experts < 1 || experts > kMaxExperts) return set_error(C3_EINVAL, "experts must be 1..1024");
    const int64_t rows = order_rows(tokens, topk, experts);
    return rows > kMaxRows ? set_error(C3_EUNSUP, "more than 2^31 rows") : rows;
}

size_t c3_moe_order_bytes(int64_t tokens, int topk, int experts) {
    if (c3_moe_rows(tokens, topk, experts) < 0) return 0;
    return order_bytes(tokens, topk, experts);
}

int c3_moe_order(const int32_t* idx, int64_t tokens, int topk, int experts, int32_t* slot, int32_t* row_of,
                 int64_t rows, int32_t* offsets, int32_t* counts, void* work, size_t work_bytes, c3_stream s) {
    const int64_t need = c3_moe_rows(tokens, topk, experts);
    if (need < 0) return (int)need;
    if (rows < need || rows > kMaxRows) return set_error(C3_EINVAL, "rows is below c3_moe_rows, or above 2^31-1");
    if (!offsets || !counts || (rows && !row_of)) return set_error(C3_EINVAL, "offsets, counts or row_of is NULL");
    if (tokens) {
        if (!idx || !slot || !work) return set_error(C3_EINVAL, "idx, slot or work is NULL");
        if (work_bytes < order_bytes(tokens, topk, experts))
            return set_error(C3_EINVAL, "work is smaller than c3_moe_order_bytes");
    }
    if (!aligned(idx, 4) || !aligned(slot, 4) || !aligned(row_of, 4) || !aligned(offsets, 4) || !aligned(counts, 4) ||
        !aligned(work, 4))
        return set_error(C3_EALIGN, "a pointer is not 4-byte aligned");
    return order_launch(idx, tokens, topk, experts, slot, row_of, rows, offsets, counts, work,
                        static_cast<cudaStream_t>(s));
}

size_t c3_fp4_code_bytes(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 1 || rows > kMaxRows || cols > kMaxRows) return 0;
    return (size_t)rows * (size_t)((cols + 31) / 32 * 16);
}

size_t c3_fp4_scale_bytes(int64_t rows, int64_t cols, int format) {
    if (rows < 0 || cols < 1 || rows > kMaxRows || cols > kMaxRows) return 0;
    if (format != C3_FP4_MX && format != C3_FP4_NV) return 0;
    Fp4 q{};
    q.rows = rows;
    q.cols = cols;
    q.nv = format == C3_FP4_NV;
    return (size_t)q.scale_bytes();
}

int c3_fp4_quantize(const void* x, int x_type, int64_t x_rows, int64_t x_cols, int64_t ld, int transpose,
                    const int32_t* row_of, const c3_fp4* m, c3_stream s) {
    Fp4 q;
    int rc = check_fp4(m, &q);
    if (rc) return rc;
    if (!is_type(x_type)) return set_error(C3_EINVAL, "unknown x_type");
    if (transpose != 0 && transpose != 1) return set_error(C3_EINVAL, "transpose must be 0 or 1");
    if (x_rows < 0 || x_cols < 0 || x_rows > kMaxRows || x_cols > kMaxRows || ld < x_cols)
        return set_error(C3_EINVAL, "bad x_rows, x_cols or ld");
    if (row_of) {
        if (transpose || q.count != 1) return set_error(C3_EINVAL, "row_of goes with one matrix and no transpose");
        if (x_cols != q.cols) return set_error(C3_EINVAL, "x and the 4-bit matrix differ in columns");
        if (!aligned(row_of, 4)) return set_error(C3_EALIGN, "row_of must be 4-byte aligned");
    } else if (transpose ? (x_rows != q.cols || x_cols != q.rows) : (x_rows != q.rows || x_cols != q.cols)) {
        return set_error(C3_EINVAL, "x and the 4-bit matrix differ in size");
    }
    if (q.rows == 0) return C3_OK;
    if (!x && x_rows) return set_error(C3_EINVAL, "x is NULL");
    if (!aligned(x, type_bytes(x_type))) return set_error(C3_EALIGN, "x is not aligned to its element");
    return fp4_quantize_launch(x, x_type == C3_BF16, x_rows, ld, transpose, row_of, q, static_cast<cudaStream_t>(s));
}

int c3_fp4_dequantize(const c3_fp4* m, void* x, int x_type, int64_t ld, c3_stream s) {
    Fp4 q;
    int rc = check_fp4(m, &q);
    if (rc) return rc;
    if (!is_type(x_type)) return set_error(C3_EINVAL, "unknown x_type");
    if (ld < q.cols) return set_error(C3_EINVAL, "ld is below cols");
    if (q.rows == 0) return C3_OK;
    if (!x) return set_error(C3_EINVAL, "x is NULL");
    if (!aligned(x, type_bytes(x_type))) return set_error(C3_EALIGN, "x is not aligned to its element");
    return fp4_dequantize_launch(q, x, x_type == C3_BF16, ld, static_cast<cudaStream_t>(s));
}

int c3_fp4_gemm(const c3_fp4* a, const c3_fp4* b, void* C, int c_type, int sm_budget, c3_stream s) {
    Fp4 qa, qb;
    int rc = check_fp4(a, &qa);
    if (rc) return rc;
    if ((rc = check_fp4(b, &qb))) return rc;
    if (qa.count != 1 || qb.count != 1) return set_error(C3_EINVAL, "a product takes one matrix each (count 1)");
    if ((rc = check_product(qa, qb, C, c_type, sm_budget))) return rc;
    if (qa.rows == 0 || qb.rows == 0) return C3_OK;
    DeviceState* ds = device_state();
    if (!ds) return C3_ECUDA;
    return fp4_gemm_launch(qa, qb, nullptr, nullptr, C, c_type == C3_BF16, sm_budget, static_cast<cudaStream_t>(s),
                           ds->status);
}

int c3_fp4_gemm_experts(const c3_fp4* x, const c3_fp4* w, const int32_t* offsets, const int32_t* counts, void* C,
                        int c_type, int sm_budget, c3_stream s) {
    Fp4 qx, qw;
    int rc = check_fp4(x, &qx);
    if (rc) return rc;
    if ((rc = check_fp4(w, &qw))) return rc;
    if (qx.count != 1) return set_error(C3_EINVAL, "the tokens are one matrix (count 1)");
    if (qw.count > kMaxExperts) return set_error(C3_EINVAL, "experts must be 1..1024");
    if ((rc = check_product(qx, qw, C, c_type, sm_budget))) return rc;
    if (!offsets || !counts) return set_error(C3_EINVAL, "offsets or counts is NULL");
    if (!aligned(offsets, 4) || !aligned(counts, 4)) return set_error(C3_EALIGN, "offsets or counts is misaligned");
    if (qx.rows == 0 || qw.rows == 0) return C3_OK;
    DeviceState* ds = device_state();
    if (!ds) return C3_ECUDA;
    return fp4_gemm_launch(qx, qw, offsets, counts, C, c_type == C3_BF16, sm_budget, static_cast<cudaStream_t>(s),
                           ds->status);
}

static int check_combine(int64_t rows, int64_t cols, int64_t tokens, int topk) {
    int rc = check_tokens(tokens, topk);
    if (rc) return rc;
    if (rows < 0 || cols < 0) return set_error(C3_EINVAL, "negative rows or cols");
    if (rows > kMaxRows || cols > kMaxRows) return set_error(C3_EUNSUP, "above 2^31-1 rows or columns");
    return C3_OK;
}

int c3_moe_combine(const void* y, int y_type, int64_t rows, int64_t cols, const int32_t* slot, const float* weights,
                   int64_t tokens, int topk, void* out, int out_type, c3_stream s) {
    int rc = check_combine(rows, cols, tokens, topk);
    if (rc) return rc;
    if (!is_type(y_type) || !is_type(out_type)) return set_error(C3_EINVAL, "unknown type");
    if (tokens == 0 || cols == 0) return C3_OK;
    if ((!y && rows) || !slot || !out) return set_error(C3_EINVAL, "y, slot or out is NULL");
    if (!aligned(y, type_bytes(y_type)) || !aligned(out, type_bytes(out_type)) || !aligned(slot, 4) ||
        !aligned(weights, 4))
        return set_error(C3_EALIGN, "a pointer is not aligned to its element");
    return combine_launch(y, y_type == C3_BF16, rows, cols, slot, weights, tokens, topk, out, out_type == C3_BF16,
                          static_cast<cudaStream_t>(s));
}

int c3_moe_combine_backward(const void* dout, int dout_type, const void* y, int y_type, int64_t rows, int64_t cols,
                            const int32_t* slot, const float* weights, int64_t tokens, int topk, void* dy,
                            float* dweights, c3_stream s) {
    int rc = check_combine(rows, cols, tokens, topk);
    if (rc) return rc;
    if (!is_type(dout_type) || !is_type(y_type)) return set_error(C3_EINVAL, "unknown type");
    if (tokens == 0) return C3_OK;
    if (!slot || (cols && (!dout || (rows && !dy) || (dweights && rows && !y))))
        return set_error(C3_EINVAL, "dout, y, slot or dy is NULL");
    if (!aligned(dout, type_bytes(dout_type)) || !aligned(y, type_bytes(y_type)) || !aligned(dy, type_bytes(y_type)) ||
        !aligned(slot, 4) || !aligned(weights, 4) || !aligned(dweights, 4))
        return set_error(C3_EALIGN, "a pointer is not aligned to its element");
    return combine_backward_launch(dout, dout_type == C3_BF16, y, y_type == C3_BF16, rows, cols, slot, weights, tokens,
                                   topk, dy, dweights, static_cast<cudaStream_t>(s));
}

}  // extern "C"
