// api_latent.cu -- the C ABI of the attention operators: rotary positions, the
// paged latent cache, absorbed and expanded latent attention.  Argument checks
// and launches only; see include/fs.h for the contracts.
#include <cfloat>
#include <cmath>

#include "../../include/fs.h"
#include "kernels.h"
#include "latent.cuh"

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

fs_status need(const void* p, unsigned align = 16) {
    if (!p) return FS_ERR_INVALID_ARG;
    return (reinterpret_cast<uintptr_t>(p) & (align - 1)) ? FS_ERR_UNSUPPORTED : FS_OK;
}

// Strides (elements of es bytes) of a [rows, heads, width] operand: 16-byte
// multiples, positive where the extent is above one.  An output's elements must
// be distinct: heads inside rows or rows inside heads.
fs_status strides(int64_t rows, int64_t heads, int64_t width, int64_t row, int64_t head, int es, bool output) {
    const int64_t q = 16 / es, lim = int64_t(1) << 36;
    if (row < 0 || head < 0) return FS_ERR_INVALID_ARG;
    if (rows > 1 && (row % q || row > lim)) return FS_ERR_UNSUPPORTED;
    if (heads > 1 && (head % q || head > lim)) return FS_ERR_UNSUPPORTED;
    if ((rows > 1 && row == 0) || (heads > 1 && head == 0)) return FS_ERR_UNSUPPORTED;
    if (!output) return FS_OK;
    const bool heads_in = (heads == 1 || head >= width) && (rows == 1 || row >= (heads - 1) * head + width);
    const bool rows_in = (rows == 1 || row >= width) && (heads == 1 || head >= (rows - 1) * row + width);
    return heads_in || rows_in ? FS_OK : FS_ERR_INVALID_ARG;
}

// Frequencies of `rope` as 64-bit fractions of a turn per position.
fs_status rope_table(const fs_rope_desc* r, bool inverse, RopeTab* tab) {
    if (!r) return FS_ERR_INVALID_ARG;
    if (r->d_rot < 2 || (r->layout != FS_ROPE_INTERLEAVED && r->layout != FS_ROPE_HALF)) return FS_ERR_INVALID_ARG;
    if (!(r->base > 1.0) || !std::isfinite(r->base) || !(r->factor >= 1.0) || !std::isfinite(r->factor) ||
        !(r->mscale >= FLT_MIN) || !(r->mscale <= FLT_MAX))
        return FS_ERR_INVALID_ARG;
    if (r->d_rot % 16 || r->d_rot > kMaxRot) return FS_ERR_UNSUPPORTED;
    const double two_pi = 6.283185307179586476925286766559;
    const int d = r->d_rot;
    double lo = 0, hi = 0;
    if (r->factor > 1.0) {
        if (!(r->orig_len > 0.0) || !std::isfinite(r->orig_len) || !(r->beta_slow > 0.0) ||
            !(r->beta_fast > r->beta_slow) || !std::isfinite(r->beta_fast))
            return FS_ERR_INVALID_ARG;
        lo = std::floor(d * std::log(r->orig_len / (r->beta_fast * two_pi)) / (2.0 * std::log(r->base)));
        hi = std::ceil(d * std::log(r->orig_len / (r->beta_slow * two_pi)) / (2.0 * std::log(r->base)));
        lo = lo > 0 ? lo : 0;
        hi = hi < d - 1 ? hi : d - 1;
    }
    const double span = hi - lo > 1e-3 ? hi - lo : 1e-3;
    for (int i = 0; i < d / 2; ++i) {
        double f = std::pow(r->base, -2.0 * i / d);
        if (r->factor > 1.0) {
            double ramp = (i - lo) / span;
            ramp = ramp < 0 ? 0 : (ramp > 1 ? 1 : ramp);
            f = f / r->factor * ramp + f * (1.0 - ramp);
        }
        tab->frac[i] = static_cast<uint64_t>(std::ldexp(f / two_pi, 64));   // f <= 1: below one turn
    }
    tab->mscale = static_cast<float>(r->mscale);
    tab->d_rot = d;
    tab->half = r->layout == FS_ROPE_HALF;
    tab->inverse = inverse;
    return FS_OK;
}

fs_status check_cache(const fs_latent_cache* c) {
    if (!c || c->n_pages < 1 || c->page_size < 1) return FS_ERR_INVALID_ARG;
    if (c->dtype < FS_BF16 || c->dtype > FS_MXFP8) return FS_ERR_INVALID_ARG;
    if (c->dtype != FS_BF16 && c->dtype != FS_FP8) return FS_ERR_UNSUPPORTED;
    if (c->n_pages > 0x7fffffffLL) return FS_ERR_UNSUPPORTED;      // block tables are int32
    const int64_t rec = c->dtype == FS_FP8 ? kRecFp8 : kRecBf16;   // a record's byte offset is an int64
    return c->n_pages * c->page_size <= INT64_MAX / rec ? FS_OK : FS_ERR_UNSUPPORTED;
}
bool is_fp8(const fs_latent_cache* c) { return c->dtype == FS_FP8; }
int64_t n_slots(const fs_latent_cache* c) { return c->n_pages * c->page_size; }

constexpr int kMaxHeads = 128, kMaxNq = 16;
constexpr int kMaxRows = 1 << 29;      // packed rows: the kernels' sums and differences of two row indexes fit an int32

fs_status check_decode(int32_t H, int32_t B, int32_t n_q) {
    if (H < 1 || B < 1 || n_q < 1) return FS_ERR_INVALID_ARG;
    if (H > kMaxHeads || n_q > kMaxNq || static_cast<int64_t>(B) * n_q * H > 0x7fffffffLL - 1024)
        return FS_ERR_UNSUPPORTED;
    return FS_OK;
}

fs_status check_prefill(const fs_latent_prefill_desc* d) {
    if (!d || d->heads < 1 || d->n_seqs < 1 || d->Tq < 1 || d->Tk < 1) return FS_ERR_INVALID_ARG;
    if (d->heads > kMaxHeads || d->Tq > kMaxRows || d->Tk > kMaxRows) return FS_ERR_UNSUPPORTED;
    // row tiles of 128 times heads index a grid
    if ((static_cast<int64_t>(d->Tq) / 128 + d->n_seqs + 1) * d->heads > 0x7fffffffLL ||
        (static_cast<int64_t>(d->Tk) / 128 + d->n_seqs + 1) * d->heads > 0x7fffffffLL)
        return FS_ERR_UNSUPPORTED;
    return std::isfinite(d->scale) && d->scale > 0.f ? FS_OK : FS_ERR_INVALID_ARG;
}

// The operands that the forward and the backward share.
fs_status prefill_args(const fs_latent_prefill_desc* d, const fs_rows* q, const fs_rows* kn, const fs_rows* kr,
                       const fs_rows* v, const int32_t* cu_q, const int32_t* cu_k, LatentPrefillArgs* a) {
    FS_CHECK(check_prefill(d));
    const int64_t H = d->heads;
    if (!q || !kn || !kr || !v) return FS_ERR_INVALID_ARG;
    FS_CHECK(need(q->p));
    FS_CHECK(need(kn->p));
    FS_CHECK(need(kr->p));
    FS_CHECK(need(v->p));
    FS_CHECK(need(cu_q, 4));
    FS_CHECK(need(cu_k, 4));
    FS_CHECK(strides(d->Tq, H, kDqk, q->row, q->head, 2, false));
    FS_CHECK(strides(d->Tk, H, kNope, kn->row, kn->head, 2, false));
    FS_CHECK(strides(d->Tk, 1, kRope, kr->row, 0, 2, false));
    FS_CHECK(strides(d->Tk, H, kDv, v->row, v->head, 2, false));
    *a = LatentPrefillArgs{};
    a->H = d->heads; a->B = d->n_seqs; a->Tq = d->Tq; a->Tk = d->Tk;
    a->causal = d->causal != 0;
    a->scale = d->scale;
    a->q = static_cast<const __nv_bfloat16*>(q->p); a->q_row = q->row; a->q_head = q->head;
    a->kn = static_cast<const __nv_bfloat16*>(kn->p); a->kn_row = kn->row; a->kn_head = kn->head;
    a->kr = static_cast<const __nv_bfloat16*>(kr->p); a->kr_row = kr->row;
    a->v = static_cast<const __nv_bfloat16*>(v->p); a->v_row = v->row; a->v_head = v->head;
    a->cu_q = cu_q;
    a->cu_k = cu_k;
    a->err = dev_error_ptr();
    return FS_OK;
}

}  // namespace

extern "C" {

fs_status fs_rope(const fs_rope_desc* rope, int64_t T, int32_t H, int32_t dtype, const int32_t* pos, const void* x,
                  int64_t x_row, int64_t x_head, void* y, int64_t y_row, int64_t y_head, int32_t inverse,
                  void* stream) {
    if (T < 1 || H < 1 || dtype < FS_BF16 || dtype > FS_MXFP8) return FS_ERR_INVALID_ARG;
    if (dtype != FS_BF16 && dtype != FS_F32) return FS_ERR_UNSUPPORTED;
    if (T > 0x7fffffffLL || H > 65536) return FS_ERR_UNSUPPORTED;
    RopeTab tab;
    FS_CHECK(rope_table(rope, inverse != 0, &tab));
    FS_CHECK(need(pos, 4));
    FS_CHECK(need(x));
    FS_CHECK(need(y));
    const int es = dtype == FS_F32 ? 4 : 2;
    FS_CHECK(strides(T, H, tab.d_rot, x_row, x_head, es, false));
    FS_CHECK(strides(T, H, tab.d_rot, y_row, y_head, es, true));
    FS_TRY(launch_rope(tab, dtype == FS_F32, T, H, pos, x, x_row, x_head, y, y_row, y_head,
                       static_cast<cudaStream_t>(stream)));
    return FS_OK;
}

size_t fs_latent_cache_bytes(const fs_latent_cache* desc) {
    if (check_cache(desc) != FS_OK) return 0;
    return static_cast<size_t>(n_slots(desc)) * (is_fp8(desc) ? kRecFp8 : kRecBf16);
}

fs_status fs_latent_cache_write(const fs_latent_cache* desc, int64_t T, const void* c, int64_t c_row,
                                const void* k_rope, int64_t k_row, const fs_rope_desc* rope, const int32_t* pos,
                                const int64_t* slots, void* cache, void* stream) {
    FS_CHECK(check_cache(desc));
    if (T < 1) return FS_ERR_INVALID_ARG;
    if (T > 0x7fffffffLL) return FS_ERR_UNSUPPORTED;
    FS_CHECK(need(c));
    FS_CHECK(need(k_rope));
    FS_CHECK(need(slots, 8));
    FS_CHECK(need(cache));
    FS_CHECK(strides(T, 1, kLatent, c_row, 0, 2, false));
    FS_CHECK(strides(T, 1, kRope, k_row, 0, 2, false));
    RopeTab tab;
    if (rope) {
        FS_CHECK(rope_table(rope, false, &tab));
        if (tab.d_rot != kRope) return FS_ERR_UNSUPPORTED;
        FS_CHECK(need(pos, 4));
    }
    FS_TRY(launch_cache_write(rope ? &tab : nullptr, is_fp8(desc), T, c, c_row, k_rope, k_row, pos, slots, cache,
                              n_slots(desc), static_cast<cudaStream_t>(stream)));
    return FS_OK;
}

fs_status fs_latent_cache_read(const fs_latent_cache* desc, const void* cache, int64_t T, const int64_t* slots,
                               void* c, int64_t c_row, void* k_rope, int64_t k_row, void* stream) {
    FS_CHECK(check_cache(desc));
    if (T < 1) return FS_ERR_INVALID_ARG;
    if (T > 0x7fffffffLL) return FS_ERR_UNSUPPORTED;
    FS_CHECK(need(cache));
    FS_CHECK(need(slots, 8));
    FS_CHECK(need(c));
    FS_CHECK(need(k_rope));
    FS_CHECK(strides(T, 1, kLatent, c_row, 0, 2, true));
    FS_CHECK(strides(T, 1, kRope, k_row, 0, 2, true));
    FS_TRY(launch_cache_read(is_fp8(desc), T, slots, cache, n_slots(desc), c, c_row, k_rope, k_row,
                             static_cast<cudaStream_t>(stream)));
    return FS_OK;
}

size_t fs_latent_decode_ws_bytes(int32_t heads, int32_t B, int32_t n_q) {
    if (check_decode(heads, B, n_q) != FS_OK) return 0;
    return latent_decode_ws_bytes(heads, B, n_q);
}

fs_status fs_latent_decode(const fs_latent_cache* desc, int32_t heads, int32_t B, int32_t n_q,
                           const fs_rows* q_latent, const fs_rows* q_rope, const void* cache,
                           const int32_t* block_table, int32_t max_pages, int64_t table_row, const int32_t* seq_lens,
                           float scale, const fs_rows_out* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
    FS_CHECK(check_cache(desc));
    FS_CHECK(check_decode(heads, B, n_q));
    if (!q_latent || !q_rope || !out || max_pages < 1 || table_row < 0 || (B > 1 && table_row < max_pages) ||
        !std::isfinite(scale) || !(scale > 0.f))
        return FS_ERR_INVALID_ARG;
    FS_CHECK(need(q_latent->p));
    FS_CHECK(need(q_rope->p));
    FS_CHECK(need(cache));
    FS_CHECK(need(block_table, 4));
    FS_CHECK(need(seq_lens, 4));
    FS_CHECK(need(out->p));
    if (lse) FS_CHECK(need(lse, 4));
    if (n_slots(desc) > 0x7fffffffLL) return FS_ERR_UNSUPPORTED;       // records are addressed by int32
    const int64_t rows = static_cast<int64_t>(B) * n_q;
    FS_CHECK(strides(rows, heads, kLatent, q_latent->row, q_latent->head, 2, false));
    FS_CHECK(strides(rows, heads, kRope, q_rope->row, q_rope->head, 2, false));
    FS_CHECK(strides(rows, heads, kLatent, out->row, out->head, 2, true));
    if (!ws) return FS_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < latent_decode_ws_bytes(heads, B, n_q))
        return FS_ERR_WORKSPACE;
    LatentDecodeArgs a{};
    a.H = heads; a.B = B; a.n_q = n_q;
    a.page_size = desc->page_size; a.max_pages = max_pages;
    a.n_pages = desc->n_pages; a.table_row = table_row;
    a.ql = static_cast<const __nv_bfloat16*>(q_latent->p); a.ql_row = q_latent->row; a.ql_head = q_latent->head;
    a.qr = static_cast<const __nv_bfloat16*>(q_rope->p); a.qr_row = q_rope->row; a.qr_head = q_rope->head;
    a.cache = static_cast<const uint8_t*>(cache);
    a.table = block_table;
    a.seq_lens = seq_lens;
    a.scale = scale;
    a.out = static_cast<__nv_bfloat16*>(out->p); a.o_row = out->row; a.o_head = out->head;
    a.lse = lse;
    a.err = dev_error_ptr();
    FS_TRY(launch_latent_decode(a, is_fp8(desc), ws, static_cast<cudaStream_t>(stream)));
    return FS_OK;
}

fs_status fs_latent_prefill(const fs_latent_prefill_desc* desc, const fs_rows* q, const fs_rows* k_nope,
                            const fs_rows* k_rope, const fs_rows* v, const int32_t* cu_q, const int32_t* cu_k,
                            const fs_rows_out* out, float* lse, void* stream) {
    LatentPrefillArgs a;
    FS_CHECK(prefill_args(desc, q, k_nope, k_rope, v, cu_q, cu_k, &a));
    if (!out) return FS_ERR_INVALID_ARG;
    FS_CHECK(need(out->p));
    FS_CHECK(need(lse, 4));
    FS_CHECK(strides(desc->Tq, desc->heads, kDv, out->row, out->head, 2, true));
    a.out_w = static_cast<__nv_bfloat16*>(out->p);
    a.o_row = out->row;
    a.o_head = out->head;
    a.lse_w = lse;
    FS_TRY(launch_latent_prefill(a, static_cast<cudaStream_t>(stream)));
    return FS_OK;
}

size_t fs_latent_prefill_backward_ws_bytes(int32_t heads, int32_t Tq, int32_t Tk) {
    if (heads < 1 || heads > kMaxHeads || Tq < 1 || Tk < 1 || Tq > kMaxRows || Tk > kMaxRows) return 0;
    return latent_backward_ws_bytes(heads, Tq, Tk);
}

fs_status fs_latent_prefill_backward(const fs_latent_prefill_desc* desc, const fs_rows* q, const fs_rows* k_nope,
                                     const fs_rows* k_rope, const fs_rows* v, const int32_t* cu_q,
                                     const int32_t* cu_k, const fs_rows* out, const float* lse, const fs_rows* d_out,
                                     const fs_rows_out* dq, const fs_rows_out* dk_nope, const fs_rows_out* dk_rope,
                                     const fs_rows_out* dv, void* ws, size_t ws_bytes, void* stream) {
    LatentPrefillArgs a;
    FS_CHECK(prefill_args(desc, q, k_nope, k_rope, v, cu_q, cu_k, &a));
    if (!out || !d_out || !dq || !dk_nope || !dk_rope || !dv) return FS_ERR_INVALID_ARG;
    const int64_t H = desc->heads, Tq = desc->Tq, Tk = desc->Tk;
    FS_CHECK(need(out->p));
    FS_CHECK(need(lse, 4));
    FS_CHECK(need(d_out->p));
    FS_CHECK(need(dq->p));
    FS_CHECK(need(dk_nope->p));
    FS_CHECK(need(dk_rope->p));
    FS_CHECK(need(dv->p));
    FS_CHECK(strides(Tq, H, kDv, out->row, out->head, 2, false));
    FS_CHECK(strides(Tq, H, kDv, d_out->row, d_out->head, 2, false));
    FS_CHECK(strides(Tq, H, kDqk, dq->row, dq->head, 2, true));
    FS_CHECK(strides(Tk, H, kNope, dk_nope->row, dk_nope->head, 2, true));
    FS_CHECK(strides(Tk, 1, kRope, dk_rope->row, 0, 2, true));
    FS_CHECK(strides(Tk, H, kDv, dv->row, dv->head, 2, true));
    if (!ws) return FS_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < latent_backward_ws_bytes(desc->heads, desc->Tq, desc->Tk))
        return FS_ERR_WORKSPACE;
    a.out = static_cast<const __nv_bfloat16*>(out->p); a.o_row = out->row; a.o_head = out->head;
    a.lse = lse;
    a.d_out = static_cast<const __nv_bfloat16*>(d_out->p); a.do_row = d_out->row; a.do_head = d_out->head;
    a.dq = static_cast<__nv_bfloat16*>(dq->p); a.dq_row = dq->row; a.dq_head = dq->head;
    a.dkn = static_cast<__nv_bfloat16*>(dk_nope->p); a.dkn_row = dk_nope->row; a.dkn_head = dk_nope->head;
    a.dkr = static_cast<__nv_bfloat16*>(dk_rope->p); a.dkr_row = dk_rope->row;
    a.dv = static_cast<__nv_bfloat16*>(dv->p); a.dv_row = dv->row; a.dv_head = dv->head;
    FS_TRY(launch_latent_backward(a, ws, static_cast<cudaStream_t>(stream)));
    return FS_OK;
}

}  // extern "C"
