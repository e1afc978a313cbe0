// lq_layers.hip — C ABI of the norm with an 8-bit checkpoint, of the 4-bit integer layer
// and of the layer of many experts (declared in include/lq.h): argument checks and workspace sizes. Every check runs before the
// first launch, so a call that fails writes nothing.
#include <stddef.h>
#include <stdint.h>

#include "lq_linear.h"

using namespace lql;

namespace {

bool aligned(const void* p) { return ((uintptr_t)p & 15u) == 0u; }
template <class... P>
bool all_aligned(P... p) {
  return (aligned(p) && ...);
}
bool is_dtype(int d) { return d == LQ_F32 || d == LQ_BF16 || d == LQ_F16; }
bool is_ckpt_format(int f) { return f == LQ_INT8 || f == LQ_E4M3; }
bool is_side(int64_t v) { return v >= 0 && v <= 0x7FFFFFFF; }
bool is_width(int64_t v) { return v >= 0 && v <= 1 << 21; }
bool is_stride(int64_t ld, int64_t cols) { return ld >= cols && ld <= (int64_t)1 << 31; }
int status_of(hipError_t e) { return e == hipSuccess ? LQ_OK : LQ_ERR_HIP; }

// ------------------------------------------------------------ the norm
int check_norm(const lq_norm_desc* d) {
  if (!d) return LQ_ERR_NULL;
  if (!is_dtype(d->dtype) || !is_dtype(d->weight_dtype) || d->ckpt_format < LQ_INT8 || d->ckpt_format > LQ_E3M2)
    return LQ_ERR_BAD_DESC;
  if (!(d->eps >= 0.0f) || d->eps > 3.4e38f) return LQ_ERR_BAD_DESC;
  if (!is_ckpt_format(d->ckpt_format) || (d->weight_dtype != d->dtype && d->weight_dtype != LQ_F32))
    return LQ_ERR_UNSUPPORTED;
  if (!is_side(d->rows) || !is_side(d->cols)) return LQ_ERR_SHAPE;
  if (!is_stride(d->ld_x, d->cols) || !is_stride(d->ld_residual, d->cols) || !is_stride(d->ld_h, d->cols) ||
      !is_stride(d->ld_y, d->cols))
    return LQ_ERR_SHAPE;
  if (d->cols > kNormColumns) return LQ_ERR_UNSUPPORTED;
  return LQ_OK;
}
NormArgs norm_args(const lq_norm_desc* d) {
  NormArgs a = {};
  a.rows = d->rows;
  a.cols = d->cols;
  a.ldx = d->ld_x;
  a.ldr = d->ld_residual;
  a.ldh = d->ld_h;
  a.ldy = d->ld_y;
  a.eps = d->eps;
  a.wide = d->weight_dtype == LQ_F32;
  return a;
}


// ------------------------------------------------------------ the 4-bit integer layer
int check_int4(const lq_int4_desc* d) {
  if (!d) return LQ_ERR_NULL;
  if (!is_dtype(d->in_dtype) || !is_dtype(d->out_dtype) || d->zero_points < 0 || d->zero_points > 1 ||
      d->reserved != 0) return LQ_ERR_BAD_DESC;
  if (d->x_format < -1 || d->x_format > LQ_E3M2) return LQ_ERR_BAD_DESC;
  if (d->x_format != -1 && !is_ckpt_format(d->x_format)) return LQ_ERR_UNSUPPORTED;
  if (d->group != 32 && d->group != 64 && d->group != 128) return LQ_ERR_UNSUPPORTED;
  if (!is_side(d->m) || !is_width(d->n) || !is_width(d->k) || d->k % d->group != 0) return LQ_ERR_SHAPE;
  if (d->m > 65535 * (int64_t)16) return LQ_ERR_UNSUPPORTED;
  return LQ_OK;
}

// ------------------------------------------------------------ the layer of many experts
int check_experts(const lq_experts_desc* d) {
  if (!d) return LQ_ERR_NULL;
  if (!is_dtype(d->in_dtype) || !is_dtype(d->out_dtype)) return LQ_ERR_BAD_DESC;
  if (d->ckpt_format < LQ_INT8 || d->ckpt_format > LQ_E3M2) return LQ_ERR_BAD_DESC;
  if (!is_ckpt_format(d->ckpt_format)) return LQ_ERR_UNSUPPORTED;
  if (d->experts < 1 || !is_side(d->m) || d->n < 1 || !is_width(d->n) || d->k < 1 || !is_width(d->k) ||
      !is_side(d->experts * d->n))
    return LQ_ERR_SHAPE;
  if (d->experts > kMostExperts) return LQ_ERR_UNSUPPORTED;
  return LQ_OK;
}
size_t round256(size_t b) { return (b + 255) / 256 * 256; }
// x as an MX4 operand: codes, then scales, each from a multiple of 256 bytes.
size_t experts_codes(const lq_experts_desc* d) { return round256((size_t)(d->m * mx4_groups(d->k) * 64)); }
size_t experts_operand(const lq_experts_desc* d) {
  return experts_codes(d) + round256((size_t)(mx4_scale_rows(d->m) * mx4_groups(d->k) * 4));
}

}  // namespace

extern "C" {

int lq_rmsnorm(const lq_norm_desc* d, const void* x, const void* residual, const void* weight, void* h, void* y,
               void* ckpt_codes, void* ckpt_scales, void* rs, void* stream) {
  const int rc = check_norm(d);
  if (rc) return rc;
  if (!ckpt_codes != !ckpt_scales) return LQ_ERR_NULL;
  if (d->rows == 0 || d->cols == 0) return LQ_OK;
  if (!x || !weight || (!h && !y && !ckpt_codes && !rs)) return LQ_ERR_NULL;
  if (!all_aligned(x, residual, weight, (const void*)h, (const void*)y, (const void*)ckpt_codes,
                   (const void*)ckpt_scales, (const void*)rs))
    return LQ_ERR_ALIGN;
  NormArgs a = norm_args(d);
  a.x = x;
  a.r = residual;
  a.w = weight;
  a.h = h;
  a.y = y;
  a.codes = (uint8_t*)ckpt_codes;
  a.scales = (uint8_t*)ckpt_scales;
  a.rs = (float*)rs;
  return status_of(launch_rmsnorm(d->dtype, d->ckpt_format, a, (hipStream_t)stream));
}

size_t lq_rmsnorm_workspace_bytes(const lq_norm_desc* d) {
  if (check_norm(d)) return 0;
  const size_t b = d->rows > 0 ? (size_t)(norm_planes(d->rows, d->cols) * plane_stride(d->cols)) * 4 : 0;
  return b ? b : 256;
}

int lq_rmsnorm_backward(const lq_norm_desc* d, const void* dy, const void* dh, const void* h, const void* weight,
                        const void* rs, void* dx, const void* dw_in, void* dw, void* ws, size_t ws_bytes, void* stream) {
  const int rc = check_norm(d);
  if (rc) return rc;
  if (d->cols == 0 || (d->rows == 0 && !dw)) return LQ_OK;
  if (d->rows > 0 && (!dy || !h || !weight || !rs || !dx)) return LQ_ERR_NULL;
  if (!all_aligned(dy, dh, h, weight, rs, (const void*)dx, dw_in, (const void*)dw, (const void*)ws)) return LQ_ERR_ALIGN;
  if (dw && (!ws || ws_bytes < lq_rmsnorm_workspace_bytes(d))) return LQ_ERR_WORKSPACE;
  NormArgs a = norm_args(d);
  a.x = dy;
  a.r = dh;
  a.h = const_cast<void*>(h);
  a.w = weight;
  a.rs = (float*)const_cast<void*>(rs);
  a.y = dx;
  a.planes = dw ? (float*)ws : nullptr;
  return status_of(launch_rmsnorm_backward(d->dtype, a, (const float*)dw_in, (float*)dw, (hipStream_t)stream));
}

size_t lq_int4_packed_bytes(const lq_int4_desc* d) {
  if (check_int4(d)) return 0;
  return int4_codes_bytes(d->n, d->k) + int4_scales_bytes(d->n, d->k, d->group) * (d->zero_points ? 2 : 1);
}

int lq_int4_pack(const lq_int4_desc* d, const void* codes, const void* scales, const void* zeros, void* packed,
                 void* stream) {
  const int rc = check_int4(d);
  if (rc) return rc;
  if (d->n == 0 || d->k == 0) return LQ_OK;
  if (!codes || !scales || !packed || !zeros != !d->zero_points) return LQ_ERR_NULL;
  if (!all_aligned(codes, scales, zeros, (const void*)packed)) return LQ_ERR_ALIGN;
  return status_of(launch_int4_pack(d, codes, scales, zeros, packed, (hipStream_t)stream));
}

size_t lq_int4_workspace_bytes(const lq_int4_desc* d) {
  if (check_int4(d)) return 0;
  const size_t b = int4_rows_bytes(d);
  return b ? b : 16;
}

int lq_int4_linear(const lq_int4_desc* d, const void* x, const void* x_scales, const void* packed, void* y, void* ws,
                   size_t ws_bytes, void* stream) {
  const int rc = check_int4(d);
  if (rc) return rc;
  if ((d->x_format == -1 && !is_stride(d->ld_in, d->k)) || !is_stride(d->ld_out, d->n)) return LQ_ERR_SHAPE;
  if (d->m == 0 || d->n == 0) return LQ_OK;
  if (!y || (d->k > 0 && (!x || !packed || !x_scales != (d->x_format == -1)))) return LQ_ERR_NULL;
  if (!all_aligned(x, x_scales, packed, (const void*)y, (const void*)ws)) return LQ_ERR_ALIGN;
  if (!ws || ws_bytes < lq_int4_workspace_bytes(d)) return LQ_ERR_WORKSPACE;
  return status_of(launch_int4_linear(d, x, x_scales, packed, y, ws, (hipStream_t)stream));
}

size_t lq_experts_workspace_bytes(const lq_experts_desc* d) {
  if (check_experts(d)) return 0;
  // the most of: the forward call's operand; a gradient's padded dy, and dx's parts' sums
  const size_t dy = reads_in_place(d->m, d->n, d->ld_in) ? 0 : round256((size_t)(d->m * padded_columns(d->n)) * 2);
  const size_t back = d->m ? dy + planes_bytes(split_experts_dgrad(d->m, d->n, d->k, d->experts), d->m, d->k) : 0;
  const size_t b = experts_operand(d) > back ? experts_operand(d) : back;
  return b ? b : 256;
}

int lq_mx4_experts(const lq_experts_desc* d, const void* x, const void* offsets, const void* w_codes, const void* w_scales,
                   void* y, void* ckpt_codes, void* ckpt_scales, void* ws, size_t ws_bytes, void* stream) {
  const int rc = check_experts(d);
  if (rc) return rc;
  if (!is_stride(d->ld_in, d->k) || !is_stride(d->ld_out, d->n)) return LQ_ERR_SHAPE;
  if (!ckpt_codes != !ckpt_scales) return LQ_ERR_NULL;
  if (d->m == 0) return LQ_OK;
  if (!x || !offsets || !w_codes || !w_scales || !y) return LQ_ERR_NULL;
  if (!all_aligned(x, offsets, w_codes, w_scales, (const void*)y, (const void*)ckpt_codes, (const void*)ckpt_scales,
                   (const void*)ws))
    return LQ_ERR_ALIGN;
  if (!ws || ws_bytes < lq_experts_workspace_bytes(d)) return LQ_ERR_WORKSPACE;
  const Experts e = {(const int32_t*)offsets, d->experts};
  const hipStream_t s = (hipStream_t)stream;
  if (experts_in_place(d->m, d->k, d->experts) && !ckpt_codes)
    return status_of(launch_mx4_experts_few(d->in_dtype, x, d->ld_in, e, w_codes, w_scales, d->m, d->n, d->k, d->out_dtype,
                                            y, d->ld_out, s));
  uint8_t *codes = (uint8_t*)ws, *scales = (uint8_t*)ws + experts_codes(d);
  if (launch_mx4_quantize(d->in_dtype, d->ckpt_format, x, d->m, d->k, d->ld_in, codes, scales, ckpt_codes, ckpt_scales, s) !=
      hipSuccess)
    return LQ_ERR_HIP;
  return status_of(launch_mx4_experts(codes, scales, e, w_codes, w_scales, d->m, d->n, d->k, d->out_dtype, y, d->ld_out, s));
}

int lq_mx4_experts_dgrad(const lq_experts_desc* d, const void* dy, const void* offsets, const void* w_codes,
                         const void* w_scales, void* dx, void* ws, size_t ws_bytes, void* stream) {
  const int rc = check_experts(d);
  if (rc) return rc;
  if (d->in_dtype != LQ_BF16) return LQ_ERR_UNSUPPORTED;
  if (!is_stride(d->ld_in, d->n) || !is_stride(d->ld_out, d->k)) return LQ_ERR_SHAPE;
  if (d->m == 0) return LQ_OK;
  if (!dy || !offsets || !w_codes || !w_scales || !dx) return LQ_ERR_NULL;
  if (!all_aligned(dy, offsets, w_codes, w_scales, (const void*)dx, (const void*)ws)) return LQ_ERR_ALIGN;
  if (!ws || ws_bytes < lq_experts_workspace_bytes(d)) return LQ_ERR_WORKSPACE;
  const Experts e = {(const int32_t*)offsets, d->experts};
  return status_of(launch_mx4_experts_dgrad(dy, e, d->m, d->n, d->ld_in, w_codes, w_scales, d->k, d->out_dtype, dx,
                                            d->ld_out, ws, (hipStream_t)stream));
}

int lq_ckpt8_experts_wgrad(const lq_experts_desc* d, const void* dy, const void* offsets, const void* ckpt_codes,
                           const void* ckpt_scales, const void* dw_in, void* dw, void* ws, size_t ws_bytes, void* stream) {
  const int rc = check_experts(d);
  if (rc) return rc;
  if (d->in_dtype != LQ_BF16 || d->out_dtype != LQ_F32) return LQ_ERR_UNSUPPORTED;
  if (!is_stride(d->ld_in, d->n) || !is_stride(d->ld_out, d->k)) return LQ_ERR_SHAPE;
  if (!dw || (d->m > 0 && (!dy || !offsets || !ckpt_codes || !ckpt_scales))) return LQ_ERR_NULL;
  if (!all_aligned(dy, offsets, ckpt_codes, ckpt_scales, dw_in, (const void*)dw, (const void*)ws)) return LQ_ERR_ALIGN;
  if (!ws || ws_bytes < lq_experts_workspace_bytes(d)) return LQ_ERR_WORKSPACE;
  if (d->m == 0)
    return status_of(launch_constant(d->experts * d->n, d->k, LQ_F32, dw_in, dw, d->ld_out, (hipStream_t)stream));
  const Experts e = {(const int32_t*)offsets, d->experts};
  return status_of(launch_ckpt8_experts_wgrad(d->ckpt_format, dy, e, d->m, d->n, d->ld_in, ckpt_codes, ckpt_scales, d->k,
                                              (const float*)dw_in, (float*)dw, d->ld_out, ws, (hipStream_t)stream));
}

}  // extern "C"
