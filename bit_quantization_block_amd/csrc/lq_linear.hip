// lq_linear.hip — C ABI of the low-bit linear layer (declared in include/lq.h):
// argument checks and workspace sizes. Every check runs before the first
// launch, so a call that fails writes nothing.
#include <stddef.h>
#include <stdint.h>

#include <algorithm>

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
// One side of a matrix; products of two sides and a stride stay within 64 bits.
bool is_side(int64_t v) { return v >= 0 && v <= 0x7FFFFFFF; }
// A row of W: its bytes times the 256 rows of a tile stay within 32 bits.
bool is_width(int64_t v) { return v >= 0 && v <= 1 << 21; }
bool is_stride(int64_t ld, int64_t cols) { return ld >= cols && ld <= (int64_t)1 << 31; }

int status_of(hipError_t e) { return e == hipSuccess ? LQ_OK : LQ_ERR_HIP; }

int check_linear(const lq_linear_desc* d) {
  if (!d) return LQ_ERR_NULL;
  if (!is_dtype(d->in_dtype) || !is_dtype(d->out_dtype) || d->reserved != 0) return LQ_ERR_BAD_DESC;
  if (d->ckpt_format < LQ_INT8 || d->ckpt_format > LQ_E3M2) return LQ_ERR_BAD_DESC;
  if (!is_ckpt_format(d->ckpt_format)) return LQ_ERR_UNSUPPORTED;
  if (!is_side(d->m) || !is_width(d->n) || !is_width(d->k)) return LQ_ERR_SHAPE;
  return LQ_OK;
}

// The forward call's copy of x as an MX4 operand: codes, then scales, each
// from a multiple of 256 bytes.
size_t round256(size_t b) { return (b + 255) / 256 * 256; }
size_t operand_codes(const lq_linear_desc* d) { return round256((size_t)(d->m * mx4_groups(d->k) * 64)); }
size_t operand_bytes(const lq_linear_desc* d) {
  return operand_codes(d) + round256((size_t)(mx4_scale_rows(d->m) * mx4_groups(d->k) * 4));
}

}  // namespace

namespace lql {

namespace {

// What a tile of a product costs, in microseconds: a fixed part, and a step of
// its contraction with almost no other workgroup running, with one on each of
// 256 compute units, and with more of them on each. Results of 16 bits of a
// product and of 32 bits of a gradient are in the fixed part; the further bytes of
// a 32-bit product, or of what dw is added to, pass at `rate` TB/s.
struct TileCost { int tile, most; double fixed, alone, full[4], rate; };
// (64: 11008 x 4096 times 64 rows 9.5 us in one part, 14.6 in two; 128: 2048 x
// 4096 x 4096 23.2 us, with 256 30.0; 256: 8192 x 8192 x 8192 262 us)
constexpr TileCost kProductTiles[] = {{1, 3, 3.0, 0.18, {0, 0.20, 0.34, 0.50}, 2.5},
                                      {2, 2, 3.5, 0.22, {0, 0.38, 0.62}, 2.5},
                                      {4, 1, 6.0, 0.55, {0, 0.95}, 5.0}};
// (dx, 128: 64 x 4096 x 4096 32 us in one part, 16.5 in eight, 2048 x 4096 x
// 4096 68 us; 256: 83 us for the latter, 8192 x 11008 x 4096 549 us. dw, whose
// tile has four bytes an element to write: 128: 4096 x 512 x 512 41 us in one
// part, 17 in eight, 2000 x 3000 x 1500 38 us; 256: 58 us for the latter, 8192 x
// 11008 x 4096 700 us)
constexpr TileCost kDgradTiles[] = {{2, 2, 5.0, 0.43, {0, 0.59, 0.99}, 0}, {4, 1, 9.0, 1.06, {0, 1.54}, 0}};
constexpr TileCost kWgradTiles[] = {{2, 2, 6.0, 0.56, {0, 0.70, 1.17}, 8.0}, {4, 1, 14.5, 1.27, {0, 1.71}, 4.3}};

// The tile and the number of parts that the figures above say is fastest. Few
// tiles over a long contraction gain from parts (512 x 1024 outputs over 16384:
// 130 us in one part, 32 in eight); adding the parts up costs a launch and their
// sums' way through memory and back.
// Rows that lie by expert end in a tile of their own each, half of one on the
// average.
template <size_t N>
Split cheapest(const TileCost (&tiles)[N], int64_t rows, int64_t cols, int64_t steps, double further, int experts = 0, int most = 32) {
  const double cus = compute_units();
  Split best = {tiles[0].tile, 1, (int)steps};
  double least = 1e300;
  const int64_t ends = rows < experts ? rows : experts;
  for (const TileCost& c : tiles) {
    const int64_t side = 64 * c.tile, count = ((rows + side - 1) / side + ends / 2) * ((cols + side - 1) / side);
    for (int64_t wanted : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
      if (wanted > most) break;
      const int64_t part = (steps + wanted - 1) / wanted, parts = part ? (steps + part - 1) / part : 1;
      if (wanted > 1 && (part < 4 || parts != wanted)) continue;
      const double wgs = (double)count * parts, planes = (double)parts * rows * cols * 4;
      if (parts > 1 && planes > 256e6) continue;
      double us = c.fixed;
      if (wgs <= cus) {
        us += part * (c.alone + (c.full[1] - c.alone) * wgs / cus);
      } else {
        double left = wgs;   // full rounds, then what is left over
        us = 0.0;
        while (left > 0) {
          const int each = left >= cus * c.most ? c.most : (int)((left + cus - 1) / cus);
          const double rounds = left >= cus * c.most ? (double)(int64_t)(left / (cus * c.most)) : 1.0;
          us += rounds * (c.fixed + part * c.full[each]);
          left -= rounds * cus * each;
        }
      }
      if (parts > 1) us += 2.5 + (planes * 2 + further) / 4.5e6;
      else if (further > 0) us += further / (c.rate * 1e6);
      if (us < least) {
        least = us;
        best = {c.tile, (int)parts, (int)part};
      }
    }
  }
  return best;
}

}  // namespace

Split split_product(int64_t m, int64_t n, int64_t k, int out_dtype) {
  return cheapest(kProductTiles, m, n, mx4_groups(k), out_dtype == LQ_F32 ? (double)m * n * 2 : 0.0);
}
Split split_dgrad(int64_t m, int64_t n, int64_t k) { return cheapest(kDgradTiles, m, k, (n + 63) / 64, 0.0); }
Split split_wgrad(int64_t m, int64_t n, int64_t k, bool adds) {
  return cheapest(kWgradTiles, n, k, (m + 63) / 64, adds ? (double)n * k * 4 : 0.0);
}
int expert_tile(int64_t m, int64_t n, int64_t k, int experts) {
  return cheapest(kProductTiles, m, n, mx4_groups(k), 0.0, experts, 1).tile;
}
Split split_experts_dgrad(int64_t m, int64_t n, int64_t k, int experts) {
  return cheapest(kDgradTiles, m, k, (n + 63) / 64, 0.0, experts);
}

}  // namespace lql

extern "C" {

size_t lq_mx4_codes_bytes(int64_t rows, int64_t cols) {
  return is_side(rows) && is_side(cols) ? (size_t)(rows * mx4_groups(cols) * 64) : 0;
}
size_t lq_mx4_scales_bytes(int64_t rows, int64_t cols) {
  return is_side(rows) && is_side(cols) ? (size_t)(mx4_scale_rows(rows) * mx4_groups(cols) * 4) : 0;
}
size_t lq_ckpt8_codes_bytes(int64_t rows, int64_t cols) {
  return is_side(rows) && is_side(cols) ? (size_t)(rows * ckpt_pitch(cols)) : 0;
}
size_t lq_ckpt8_scales_bytes(int64_t rows, int64_t cols) {
  return is_side(rows) && is_side(cols) ? (size_t)(rows * ckpt_scale_pitch(cols)) : 0;
}

size_t lq_linear_workspace_bytes(const lq_linear_desc* d) {
  if (check_linear(d)) return 0;
  // the most of: the forward call's operand and its parts' sums; a gradient
  // call's padded dy and its parts' sums
  const size_t forward = operand_bytes(d) + planes_bytes(split_product(d->m, d->n, d->k, d->out_dtype), d->m, d->n);
  const size_t dy = !reads_in_place(d->m, d->n, d->ld_in) ? round256((size_t)(d->m * padded_columns(d->n)) * 2) : 0;
  const size_t dx = planes_bytes(split_dgrad(d->m, d->n, d->k), d->m, d->k);
  const size_t dw0 = planes_bytes(split_wgrad(d->m, d->n, d->k, false), d->n, d->k);
  const size_t dw1 = planes_bytes(split_wgrad(d->m, d->n, d->k, true), d->n, d->k);
  const size_t backward = dy + std::max(dx, std::max(dw0, dw1)), b = std::max(forward, backward);
  return b ? b : 256;
}

int lq_mx4_quantize(const lq_linear_desc* d, const void* x, void* codes, void* scales, void* ckpt_codes,
                    void* ckpt_scales, void* stream) {
  const int rc = check_linear(d);
  if (rc) return rc;
  if (!is_stride(d->ld_in, d->k)) return LQ_ERR_SHAPE;
  if (!codes != !scales || !ckpt_codes != !ckpt_scales) return LQ_ERR_NULL;
  if (d->m == 0 || d->k == 0) return LQ_OK;
  if (!x || (!codes && !ckpt_codes)) return LQ_ERR_NULL;
  if (!all_aligned(x, codes, scales, ckpt_codes, ckpt_scales)) return LQ_ERR_ALIGN;
  return status_of(launch_mx4_quantize(d->in_dtype, d->ckpt_format, x, d->m, d->k, d->ld_in, codes, scales, ckpt_codes,
                                       ckpt_scales, (hipStream_t)stream));
}

int lq_mx4_product(const lq_linear_desc* d, const void* x_codes, const void* x_scales, const void* w_codes,
                   const void* w_scales, void* y, void* ws, size_t ws_bytes, void* stream) {
  const int rc = check_linear(d);
  if (rc) return rc;
  if (!is_stride(d->ld_out, d->n)) return LQ_ERR_SHAPE;
  if (d->m == 0 || d->n == 0) return LQ_OK;
  if (!y || (d->k > 0 && (!x_codes || !x_scales || !w_codes || !w_scales))) return LQ_ERR_NULL;
  if (!all_aligned(x_codes, x_scales, w_codes, w_scales, (const void*)y, (const void*)ws)) return LQ_ERR_ALIGN;
  if (!ws || ws_bytes < lq_linear_workspace_bytes(d)) return LQ_ERR_WORKSPACE;
  return status_of(launch_mx4_product(x_codes, x_scales, w_codes, w_scales, d->m, d->n, d->k, d->out_dtype, y,
                                      d->ld_out, ws, (hipStream_t)stream));
}

int lq_mx4_linear(const lq_linear_desc* d, const void* x, const void* w_codes, const void* w_scales, void* y,
                  void* ckpt_codes, void* ckpt_scales, void* ws, size_t ws_bytes, void* stream) {
  const int rc = check_linear(d);
  if (rc) return rc;
  if (!is_stride(d->ld_in, d->k) || !is_stride(d->ld_out, d->n)) return LQ_ERR_SHAPE;
  if (!ckpt_codes != !ckpt_scales) return LQ_ERR_NULL;
  if (d->m == 0) return LQ_OK;
  if ((d->n > 0 && !y) || (d->k > 0 && (!x || (d->n > 0 && (!w_codes || !w_scales))))) return LQ_ERR_NULL;
  if (!all_aligned(x, w_codes, w_scales, (const void*)y, (const void*)ckpt_codes, (const void*)ckpt_scales,
                   (const void*)ws))
    return LQ_ERR_ALIGN;
  if (!ws || ws_bytes < lq_linear_workspace_bytes(d)) return LQ_ERR_WORKSPACE;
  if (few_rows(d->m, d->n, d->k) && d->n > 0 && d->k > 0 && !ckpt_codes)
    return status_of(launch_mx4_few(d->in_dtype, x, d->ld_in, w_codes, w_scales, d->m, d->n, d->k, d->out_dtype, y,
                                    d->ld_out, (hipStream_t)stream));
  uint8_t *codes = (uint8_t*)ws, *scales = (uint8_t*)ws + operand_codes(d);
  if (d->k > 0) {
    const hipError_t e = launch_mx4_quantize(d->in_dtype, d->ckpt_format, x, d->m, d->k, d->ld_in, codes, scales,
                                             ckpt_codes, ckpt_scales, (hipStream_t)stream);
    if (e != hipSuccess) return LQ_ERR_HIP;
  }
  if (d->n == 0) return LQ_OK;
  return status_of(launch_mx4_product(codes, scales, w_codes, w_scales, d->m, d->n, d->k, d->out_dtype, y, d->ld_out,
                                      (uint8_t*)ws + operand_bytes(d), (hipStream_t)stream));
}

int lq_mx4_dgrad(const lq_linear_desc* d, const void* dy, const void* w_codes, const void* w_scales, void* dx,
                 void* ws, size_t ws_bytes, void* stream) {
  const int rc = check_linear(d);
  if (rc) return rc;
  if (d->in_dtype != LQ_BF16) return LQ_ERR_UNSUPPORTED;
  if (!is_stride(d->ld_in, d->n) || !is_stride(d->ld_out, d->k)) return LQ_ERR_SHAPE;
  if (d->m == 0 || d->k == 0) return LQ_OK;
  if (!dx || (d->n > 0 && (!dy || !w_codes || !w_scales))) return LQ_ERR_NULL;
  if (!all_aligned(dy, w_codes, w_scales, (const void*)dx, (const void*)ws)) return LQ_ERR_ALIGN;
  if (!ws || ws_bytes < lq_linear_workspace_bytes(d)) return LQ_ERR_WORKSPACE;
  return status_of(launch_mx4_dgrad(dy, d->m, d->n, d->ld_in, w_codes, w_scales, d->k, d->out_dtype, dx, d->ld_out,
                                    ws, (hipStream_t)stream));
}

int lq_ckpt8_wgrad(const lq_linear_desc* d, const void* dy, const void* ckpt_codes, const void* ckpt_scales,
                   const void* dw_in, void* dw, void* ws, size_t ws_bytes, void* stream) {
  const int rc = check_linear(d);
  if (rc) return rc;
  if (d->in_dtype != LQ_BF16 || d->out_dtype != LQ_F32) return LQ_ERR_UNSUPPORTED;
  if (!is_stride(d->ld_in, d->n) || !is_stride(d->ld_out, d->k)) return LQ_ERR_SHAPE;
  if (d->n == 0 || d->k == 0) return LQ_OK;
  if (!dw || (d->m > 0 && (!dy || !ckpt_codes || !ckpt_scales))) return LQ_ERR_NULL;
  if (!all_aligned(dy, ckpt_codes, ckpt_scales, dw_in, (const void*)dw, (const void*)ws)) return LQ_ERR_ALIGN;
  if (!ws || ws_bytes < lq_linear_workspace_bytes(d)) return LQ_ERR_WORKSPACE;
  return status_of(launch_ckpt8_wgrad(d->ckpt_format, dy, d->m, d->n, d->ld_in, ckpt_codes, ckpt_scales, d->k,
                                      (const float*)dw_in, (float*)dw, d->ld_out, ws, (hipStream_t)stream));
}

int lq_linear_kernels(const lq_linear_desc* d, int call, int also, char* names, size_t bytes) {
  // (no buffer is touched: any aligned address stands for one)
  void *const b = (void*)(uintptr_t)256, *const opt = also ? b : nullptr;
  const size_t ws = ~(size_t)0;
  lqd::PlanScope scope(names, bytes);
  int rc = LQ_ERR_BAD_DESC;
  switch (call) {
    case LQ_CALL_QUANTIZE: rc = lq_mx4_quantize(d, b, b, b, opt, opt, nullptr); break;
    case LQ_CALL_PRODUCT: rc = lq_mx4_product(d, b, b, b, b, b, b, ws, nullptr); break;
    case LQ_CALL_LINEAR: rc = lq_mx4_linear(d, b, b, b, b, opt, opt, b, ws, nullptr); break;
    case LQ_CALL_DGRAD: rc = lq_mx4_dgrad(d, b, b, b, b, b, ws, nullptr); break;
    case LQ_CALL_WGRAD: rc = lq_ckpt8_wgrad(d, b, b, b, opt, b, b, ws, nullptr); break;
  }
  return rc < 0 ? rc : scope.rec.count;
}

static int check_swiglu(const lq_swiglu_desc* d) {
  if (!d) return LQ_ERR_NULL;
  if (!is_dtype(d->dtype) || d->ckpt_format < LQ_INT8 || d->ckpt_format > LQ_E3M2) return LQ_ERR_BAD_DESC;
  if (!is_ckpt_format(d->ckpt_format)) return LQ_ERR_UNSUPPORTED;
  if (!is_side(d->rows) || !is_side(d->cols) || !is_stride(d->ld, d->cols) || !is_stride(d->ld_h, d->cols))
    return LQ_ERR_SHAPE;
  return LQ_OK;
}

int lq_swiglu_ckpt8(const lq_swiglu_desc* d, const void* gate, const void* up, void* h, void* gate_codes,
                    void* gate_scales, void* up_codes, void* up_scales, void* stream) {
  const int rc = check_swiglu(d);
  if (rc) return rc;
  const bool keep = gate_codes != nullptr;
  if (!gate_scales == keep || !up_codes == keep || !up_scales == keep) return LQ_ERR_NULL;
  if (d->rows == 0 || d->cols == 0) return LQ_OK;
  if (!gate || !up || (!h && !keep)) return LQ_ERR_NULL;
  if (!all_aligned(gate, up, (const void*)h, (const void*)gate_codes, (const void*)gate_scales, (const void*)up_codes,
                   (const void*)up_scales))
    return LQ_ERR_ALIGN;
  return status_of(launch_swiglu(d->dtype, d->ckpt_format, gate, up, d->rows, d->cols, d->ld, h, d->ld_h, gate_codes,
                                 gate_scales, up_codes, up_scales, (hipStream_t)stream));
}

int lq_swiglu_ckpt8_backward(const lq_swiglu_desc* d, const void* dh, const void* gate_codes, const void* gate_scales,
                             const void* up_codes, const void* up_scales, void* dgate, void* dup, void* stream) {
  const int rc = check_swiglu(d);
  if (rc) return rc;
  if (d->rows == 0 || d->cols == 0) return LQ_OK;
  if (!dh || !gate_codes || !gate_scales || !up_codes || !up_scales || !dgate || !dup) return LQ_ERR_NULL;
  if (!all_aligned(dh, gate_codes, gate_scales, up_codes, up_scales, (const void*)dgate, (const void*)dup))
    return LQ_ERR_ALIGN;
  return status_of(launch_swiglu_backward(d->dtype, d->ckpt_format, dh, d->rows, d->cols, d->ld_h, gate_codes,
                                          gate_scales, up_codes, up_scales, dgate, dup, d->ld, (hipStream_t)stream));
}

}  // extern "C"
