// api_train.cu -- the C ABI of the training operators beside the stack's backward:
// the router's balance loss with its gradient, orthogonalised updates.  Argument checks and launches only;
// see include/fs.h for the contracts.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "../../include/fs.h"
#include "kernels.h"

using namespace fs;

#define FS_TRY(expr)                                                                 \
    do {                                                                             \
        cudaError_t e_ = (expr);                                                     \
        if (e_ != cudaSuccess) return static_cast<fs_status>(cuda_error_status(e_)); \
    } while (0)
#define FS_CHECK(expr)              \
    do {                            \
        fs_status s_ = (expr);      \
        if (s_ != FS_OK) return s_; \
    } while (0)

namespace {

fs_status need(const void* p, unsigned align) {
    if (!p) return FS_ERR_INVALID_ARG;
    return (reinterpret_cast<uintptr_t>(p) & (align - 1)) ? FS_ERR_UNSUPPORTED : FS_OK;
}
fs_status maybe(const void* p, unsigned align) { return p ? need(p, align) : FS_OK; }

constexpr int64_t kMaxStride = int64_t(1) << 36;

fs_status check_balance(const fs_balance_desc* d) {
    if (!d || d->T < 1 || d->E < 1 || d->k < 1 || d->k > d->E || d->n_seqs < 1) return FS_ERR_INVALID_ARG;
    if (d->gate < FS_GATE_SOFTMAX || d->gate > FS_GATE_SIGMOID_NORM || !std::isfinite(d->coef)) return FS_ERR_INVALID_ARG;
    if (d->E > kMaxExperts || d->k > kMaxTopK || d->T > 0x7fffffff - 8192 || d->n_seqs > 65535) return FS_ERR_UNSUPPORTED;
    return FS_OK;
}

fs_status row_stride(const fs_balance_desc* d, int64_t row) {
    if (row < d->E) return FS_ERR_INVALID_ARG;
    return row <= kMaxStride ? FS_OK : FS_ERR_UNSUPPORTED;
}

// The operands of both directions.
fs_status balance_args(const fs_balance_desc* d, const float* logits, int64_t row, const float* bias, const int32_t* cu,
                       const uint8_t* mask, BalanceArgs* a) {
    FS_CHECK(check_balance(d));
    FS_CHECK(need(logits, 4));
    FS_CHECK(row_stride(d, row));
    FS_CHECK(maybe(bias, 4));
    FS_CHECK(maybe(cu, 4));
    if (!cu && d->n_seqs != 1) return FS_ERR_INVALID_ARG;
    *a = BalanceArgs{};
    a->z = logits; a->z_row = row; a->bias = bias; a->mask = mask; a->cu = cu;
    a->T = d->T; a->E = d->E; a->k = d->k; a->S = d->n_seqs; a->coef = d->coef;
    a->sigmoid = d->gate == FS_GATE_SIGMOID || d->gate == FS_GATE_SIGMOID_NORM;
    return FS_OK;
}

// ---- orthogonalised updates
constexpr int kMaxDim = 16384;

// Powers of two for X, A and B, from the largest singular value that the steps can
// reach: s <= 1 at first (the Frobenius norm is 1), then max |a s + b s^3 + c s^5|.
// X, A = X X^T and B have entries no larger than their own largest singular values; each
// is stored below 2^14, a factor of four under fp16's end for what rounding adds.
fs_status ortho_scales(const fs_orthogonalize_desc* d, OrthoScales* sc) {
    double s = 1.0, top = 1.0, btop = 0.0;
    for (int k = 0; k < d->steps; ++k) {
        const double a = d->coefs[3 * k], b = d->coefs[3 * k + 1], c = d->coefs[3 * k + 2];
        if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return FS_ERR_INVALID_ARG;
        // |a x + b x^3 + c x^5| on [0, s]: its ends and where a + 3 b u + 5 c u^2 = 0, u = x^2;
        // |b u + c u^2|: its ends and u = -b / 2c
        double next = 0.0;
        const auto point = [&](double u) {
            if (!(u > 0.0) || u > s * s) return;
            next = std::max(next, std::sqrt(u) * std::fabs(a + u * (b + u * c)));
            btop = std::max(btop, u * std::fabs(b + u * c));
        };
        point(s * s);
        if (c != 0.0) {
            const double disc = 9.0 * b * b - 20.0 * a * c;
            if (disc >= 0.0) {
                point((-3.0 * b + std::sqrt(disc)) / (10.0 * c));
                point((-3.0 * b - std::sqrt(disc)) / (10.0 * c));
            }
            point(-b / (2.0 * c));
        } else if (b != 0.0) {
            point(-a / (3.0 * b));
        }
        s = next;
        top = std::max(top, s);
        if (!(s <= 8.0) || !(btop <= 1024.0)) return FS_ERR_UNSUPPORTED;      // the steps would not stay bounded
    }
    const auto below = [](double limit, double v) { return static_cast<float>(std::exp2(std::floor(std::log2(limit / v)))); };
    sc->x = below(16384.0, top);
    sc->a = below(16384.0, top * top);
    sc->b = below(16384.0, std::max(btop, 1.0));
    return FS_OK;
}

fs_status check_ortho(const fs_orthogonalize_desc* d, OrthoScales* sc) {
    if (!d || d->batch < 1 || d->m < 1 || d->n < 1 || d->steps < 1) return FS_ERR_INVALID_ARG;
    if (d->dtype < FS_BF16 || d->dtype > FS_MXFP4) return FS_ERR_INVALID_ARG;
    if (!std::isfinite(d->scale) || !(d->eps >= 0.f) || !std::isfinite(d->eps)) return FS_ERR_INVALID_ARG;
    if (d->dtype != FS_BF16 && d->dtype != FS_F32) return FS_ERR_UNSUPPORTED;
    if (d->m > kMaxDim || d->n > kMaxDim || d->steps > kMaxOrthoSteps) return FS_ERR_UNSUPPORTED;
    return ortho_scales(d, sc);
}

// Strides of a [batch, m, n] operand: rows inside matrices.
fs_status ortho_strides(const fs_orthogonalize_desc* d, int64_t row, int64_t mat) {
    if (row < d->n || (d->batch > 1 && mat < (d->m - 1) * row + d->n)) return FS_ERR_INVALID_ARG;
    return row <= (int64_t(1) << 31) && mat <= kMaxStride ? FS_OK : FS_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" {

size_t fs_orthogonalize_ws_bytes(const fs_orthogonalize_desc* desc) {
    OrthoScales sc;
    if (check_ortho(desc, &sc) != FS_OK) return 0;
    return ortho_ws_bytes(desc->batch, desc->m, desc->n);
}

fs_status fs_orthogonalize(const fs_orthogonalize_desc* desc, const void* g, int64_t g_row, int64_t g_mat, void* out,
                           int64_t out_row, int64_t out_mat, void* ws, size_t ws_bytes, void* stream) {
    OrthoArgs o;
    FS_CHECK(check_ortho(desc, &o.scales));
    o.f32 = desc->dtype == FS_F32;
    FS_CHECK(need(g, o.f32 ? 4 : 2));
    FS_CHECK(need(out, 2));
    FS_CHECK(ortho_strides(desc, g_row, g_mat));
    FS_CHECK(ortho_strides(desc, out_row, out_mat));
    if (!ws) return FS_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < ortho_ws_bytes(desc->batch, desc->m, desc->n))
        return FS_ERR_WORKSPACE;
    o.g = g; o.g_row = g_row; o.g_mat = desc->batch > 1 ? g_mat : 0;
    o.out = static_cast<__nv_bfloat16*>(out); o.out_row = out_row;
    o.out_mat = desc->batch > 1 ? out_mat : (desc->m * out_row + 7) / 8 * 8;      // one matrix: any legal stride
    o.batch = desc->batch; o.m = desc->m; o.n = desc->n; o.steps = desc->steps;
    o.coefs = desc->coefs; o.eps = desc->eps; o.scale = desc->scale;
    FS_TRY(launch_orthogonalize(o, ws, static_cast<cudaStream_t>(stream)));
    return FS_OK;
}

size_t fs_balance_ws_bytes(const fs_balance_desc* desc) {
    if (check_balance(desc) != FS_OK) return 0;
    return balance_ws_bytes(desc->T, desc->E, desc->n_seqs);
}

fs_status fs_balance_loss(const fs_balance_desc* desc, const float* logits, int64_t logits_row, const float* bias,
                          const int32_t* topk_idx, const int32_t* cu, const uint8_t* mask, int32_t* counts,
                          int32_t* tokens, float* probs, float* loss, void* ws, size_t ws_bytes, void* stream) {
    BalanceArgs a;
    FS_CHECK(balance_args(desc, logits, logits_row, bias, cu, mask, &a));
    FS_CHECK(need(topk_idx, 4));
    FS_CHECK(need(counts, 4));
    FS_CHECK(need(tokens, 4));
    FS_CHECK(need(probs, 4));
    FS_CHECK(need(loss, 4));
    if (!ws) return FS_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < fs_balance_ws_bytes(desc)) return FS_ERR_WORKSPACE;
    a.idx = topk_idx; a.counts = counts; a.tokens = tokens; a.probs = probs; a.loss = loss;
    FS_TRY(launch_balance(a, ws, static_cast<cudaStream_t>(stream)));
    return FS_OK;
}

fs_status fs_balance_loss_backward(const fs_balance_desc* desc, const float* logits, int64_t logits_row,
                                   const float* bias, const int32_t* cu, const uint8_t* mask, const int32_t* counts,
                                   const int32_t* tokens, const float* d_loss, float* d_logits, int64_t d_row,
                                   void* stream) {
    BalanceArgs a;
    FS_CHECK(balance_args(desc, logits, logits_row, bias, cu, mask, &a));
    FS_CHECK(need(counts, 4));
    FS_CHECK(need(tokens, 4));
    FS_CHECK(maybe(d_loss, 4));
    FS_CHECK(need(d_logits, 4));
    FS_CHECK(row_stride(desc, d_row));
    a.counts = const_cast<int32_t*>(counts);
    a.tokens = const_cast<int32_t*>(tokens);
    FS_TRY(launch_balance_backward(a, d_loss, d_logits, d_row, static_cast<cudaStream_t>(stream)));
    return FS_OK;
}

}  // extern "C"
