// api_train.cu -- the C ABI of the training operators beside the stack's backward:
// the router's balance loss with its gradient.  Argument checks and launches only;
// see include/fs.h for the contracts.
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

}  // namespace

extern "C" {

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
