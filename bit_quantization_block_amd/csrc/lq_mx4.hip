// lq_mx4.hip — 4-bit microscaled quantisation and product.
#include "lq_linear.h"

namespace lql {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));

// ---------------------------------------------------------------- quantise
// One wave per 512 columns of a row; a lane holds 8 consecutive elements, so
// every load and store instruction of a wave covers one stretch of whole
// lines, and a block of 32 is the four lanes of a quad. One read of x gives
// the 4-bit operand and the 8-bit checkpoint.
template <int DT, int F>
__global__ __launch_bounds__(256) void k_mx4_quantize(const void* x, int64_t m, int64_t k, int64_t ldx,
                                                      uint8_t* codes, uint8_t* scales, uint8_t* ck, uint8_t* cks) {
  const int64_t segs = (k + 511) / 512;
  for (int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); unit < m * segs; unit += (int64_t)gridDim.x * 4) {
  const int64_t row = unit / segs;
  const int lane = threadIdx.x & 63;
  const int64_t col = (unit % segs) * 512 + lane * 8;
  const int valid = col >= k ? 0 : (k - col >= 8 ? 8 : (int)(k - col));
  float v[8];
  load8<DT>((const typename El<DT>::T*)x + row * ldx, col, valid, v);
  const uint32_t amax = quad_max(amax8_bits(v));
  if (codes) {
    const uint32_t sb = scale_byte<LQ_E2M1>(amax);
    const uint32_t w = encode_e2m1(v, scale_recip(sb));
    if (col < (k + 255) / 256 * 256) *(uint32_t*)(codes + row * mx4_pitch(k) + col / 2) = w;
    if ((lane & 3) == 0) scales[row * mx4_scale_pitch(k) + col / 32] = (uint8_t)sb;
  }
  if (ck && col < ckpt_pitch(k)) {
    const uint32_t sb = scale_byte<F>(amax);
    const uint2 w = encode8<F>(v, scale_recip(sb));
    *(uint2*)(ck + row * ckpt_pitch(k) + col) = w;
    if ((lane & 3) == 0) cks[row * ckpt_scale_pitch(k) + col / 32] = (uint8_t)sb;
  }
  }
}

// ---------------------------------------------------------------- product
// One wave per 32 x 32 tile of y, operands straight from memory.
template <int OUT>
__global__ __launch_bounds__(256) void k_mx4_product(const uint8_t* a, const uint8_t* as, const uint8_t* w,
                                                     const uint8_t* ws, int64_t m, int64_t n, int64_t k, void* y,
                                                     int64_t ldy) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t across = (n + 63) / 64;
  const int64_t row0 = blockIdx.x / across * 64 + (wave >> 1) * 32, col0 = blockIdx.x % across * 64 + (wave & 1) * 32;
  const int r = lane & 31, h = lane >> 5;
  const int64_t ar = row0 + r < m ? row0 + r : m - 1, wr = col0 + r < n ? col0 + r : n - 1;
  const int64_t p = mx4_pitch(k), sp = mx4_scale_pitch(k);
  v16f acc;
#pragma unroll
  for (int i = 0; i < 16; i++) acc[i] = 0.0f;
  for (int64_t b = h; b < p / 16; b += 2) {
    const v4i av = *(const v4i*)(a + ar * p + b * 16), wv = *(const v4i*)(w + wr * p + b * 16);
    const v8i A = {av[0], av[1], av[2], av[3], 0, 0, 0, 0}, W = {wv[0], wv[1], wv[2], wv[3], 0, 0, 0, 0};
    acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(A, W, acc, 4, 4, 0, as[ar * sp + b], 0, ws[wr * sp + b]);
  }
#pragma unroll
  for (int i = 0; i < 16; i++) {
    const int64_t row = row0 + 8 * (i / 4) + 4 * h + i % 4, col = col0 + r;
    if (row < m && col < n) ((typename El<OUT>::T*)y)[row * ldy + col] = narrow<OUT>(acc[i]);
  }
}

template <int DT>
hipError_t quantize_dt(int format, const void* x, int64_t m, int64_t k, int64_t ldx, void* codes, void* scales,
                       void* ck, void* cks, hipStream_t s) {
  const dim3 g(stream_grid(m * ((k + 511) / 512)));
  if (format == LQ_INT8)
    hipLaunchKernelGGL((k_mx4_quantize<DT, LQ_INT8>), g, dim3(256), 0, s, x, m, k, ldx, (uint8_t*)codes,
                       (uint8_t*)scales, (uint8_t*)ck, (uint8_t*)cks);
  else
    hipLaunchKernelGGL((k_mx4_quantize<DT, LQ_E4M3>), g, dim3(256), 0, s, x, m, k, ldx, (uint8_t*)codes,
                       (uint8_t*)scales, (uint8_t*)ck, (uint8_t*)cks);
  return hipGetLastError();
}

template <int OUT>
hipError_t product_dt(const void* a, const void* as, const void* w, const void* ws, int64_t m, int64_t n, int64_t k,
                      void* y, int64_t ldy, hipStream_t s) {
  hipLaunchKernelGGL((k_mx4_product<OUT>), dim3((unsigned)((n + 63) / 64 * ((m + 63) / 64))), dim3(256), 0, s,
                     (const uint8_t*)a, (const uint8_t*)as, (const uint8_t*)w, (const uint8_t*)ws, m, n, k, y, ldy);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx4_quantize(int in_dtype, int ckpt_format, const void* x, int64_t m, int64_t k, int64_t ldx,
                               void* codes, void* scales, void* ck, void* cks, hipStream_t s) {
  switch (in_dtype) {
    case LQ_F32: return quantize_dt<LQ_F32>(ckpt_format, x, m, k, ldx, codes, scales, ck, cks, s);
    case LQ_BF16: return quantize_dt<LQ_BF16>(ckpt_format, x, m, k, ldx, codes, scales, ck, cks, s);
    default: return quantize_dt<LQ_F16>(ckpt_format, x, m, k, ldx, codes, scales, ck, cks, s);
  }
}

hipError_t launch_mx4_product(const void* a_codes, const void* a_scales, const void* w_codes, const void* w_scales,
                              int64_t m, int64_t n, int64_t k, int out_dtype, void* y, int64_t ldy, hipStream_t s) {
  switch (out_dtype) {
    case LQ_F32: return product_dt<LQ_F32>(a_codes, a_scales, w_codes, w_scales, m, n, k, y, ldy, s);
    case LQ_BF16: return product_dt<LQ_BF16>(a_codes, a_scales, w_codes, w_scales, m, n, k, y, ldy, s);
    default: return product_dt<LQ_F16>(a_codes, a_scales, w_codes, w_scales, m, n, k, y, ldy, s);
  }
}

}  // namespace lql
