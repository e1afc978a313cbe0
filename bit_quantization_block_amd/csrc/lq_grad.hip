// lq_grad.hip — the linear layer's gradients: dx = dy W from the 4-bit weights,
// dw = dw0 + dy^T x8 from the 8-bit checkpoint of x.
#include "lq_linear.h"

namespace lql {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));

// A 64 x 64 tile of the result per workgroup, 32 of the contraction at a time
// through LDS, both operands laid out with the contraction along the row.
struct Tiles {
  __attribute__((aligned(16))) uint16_t a[64][40];
  __attribute__((aligned(16))) uint16_t b[64][40];
};

__device__ __forceinline__ void multiply(const Tiles& t, int lane, int wave, v16f& acc) {
  const int r = lane & 31, h = lane >> 5;
#pragma unroll
  for (int kk = 0; kk < 32; kk += 16) {
    const v8bf A = *(const v8bf*)&t.a[(wave >> 1) * 32 + r][kk + 8 * h], B = *(const v8bf*)&t.b[(wave & 1) * 32 + r][kk + 8 * h];
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(A, B, acc, 0, 0, 0);
  }
}

template <int OUT>
__global__ __launch_bounds__(256) void k_mx4_dgrad(const uint16_t* dy, int64_t m, int64_t n, int64_t lddy,
                                                   const uint8_t* w, const uint8_t* ws, int64_t k, void* dx,
                                                   int64_t lddx) {
  __shared__ Tiles t;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t across = (k + 63) / 64;
  const int64_t row0 = blockIdx.x / across * 64, col0 = blockIdx.x % across * 64;
  v16f acc;
#pragma unroll
  for (int i = 0; i < 16; i++) acc[i] = 0.0f;
  for (int64_t j0 = 0; j0 < n; j0 += 32) {
    for (int e = threadIdx.x; e < 64 * 32; e += 256) {
      const int64_t row = row0 + e / 32, j = j0 + e % 32;
      t.a[e / 32][e % 32] = row < m && j < n ? dy[row * lddy + j] : (uint16_t)0;
      const int64_t col = col0 + e % 64, jw = j0 + e / 64;
      uint16_t b = 0;
      if (col < k && jw < n) {
        const uint32_t c = w[mx4_code_at(n, jw, col)] >> (4 * (col & 1)) & 15u;
        float v[8];
        lqd::fp4_unpack8(c, v);
        b = narrow<LQ_BF16>(v[0] * scale_value(ws[mx4_scale_at(n, jw, col)]));
      }
      t.b[e % 64][e / 64] = b;
    }
    __syncthreads();
    multiply(t, lane, wave, acc);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 16; i++) {
    const int64_t row = row0 + (wave >> 1) * 32 + 8 * (i / 4) + 4 * (lane >> 5) + i % 4, col = col0 + (wave & 1) * 32 + (lane & 31);
    if (row < m && col < k) ((typename El<OUT>::T*)dx)[row * lddx + col] = narrow<OUT>(acc[i]);
  }
}

template <int F>
__global__ __launch_bounds__(256) void k_ckpt8_wgrad(const uint16_t* dy, int64_t m, int64_t n, int64_t lddy,
                                                     const uint8_t* x, const uint8_t* xs, int64_t k, const float* dw_in,
                                                     float* dw, int64_t lddw) {
  __shared__ Tiles t;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t across = (k + 63) / 64;
  const int64_t row0 = blockIdx.x / across * 64, col0 = blockIdx.x % across * 64;
  const int64_t p = ckpt_pitch(k), sp = ckpt_scale_pitch(k);
  v16f acc;
#pragma unroll
  for (int i = 0; i < 16; i++) acc[i] = 0.0f;
  for (int64_t i0 = 0; i0 < m; i0 += 32) {
    for (int e = threadIdx.x; e < 64 * 32; e += 256) {
      const int64_t i = i0 + e / 64, row = row0 + e % 64, col = col0 + e % 64;
      t.a[e % 64][e / 64] = i < m && row < n ? dy[i * lddy + row] : (uint16_t)0;
      uint16_t b = 0;
      if (i < m && col < k) {
        float v[4];
        decode4<F>(x[i * p + col], scale_value(xs[i * sp + col / 32]), v);
        b = narrow<LQ_BF16>(v[0]);
      }
      t.b[e % 64][e / 64] = b;
    }
    __syncthreads();
    multiply(t, lane, wave, acc);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 16; i++) {
    const int64_t row = row0 + (wave >> 1) * 32 + 8 * (i / 4) + 4 * (lane >> 5) + i % 4, col = col0 + (wave & 1) * 32 + (lane & 31);
    if (row < n && col < k) dw[row * lddw + col] = acc[i] + (dw_in ? dw_in[row * lddw + col] : 0.0f);
  }
}

template <int OUT>
hipError_t dgrad_dt(const void* dy, int64_t m, int64_t n, int64_t lddy, const void* w, const void* ws, int64_t k,
                    void* dx, int64_t lddx, hipStream_t s) {
  hipLaunchKernelGGL((k_mx4_dgrad<OUT>), dim3((unsigned)((k + 63) / 64 * ((m + 63) / 64))), dim3(256), 0, s,
                     (const uint16_t*)dy, m, n, lddy, (const uint8_t*)w, (const uint8_t*)ws, k, dx, lddx);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx4_dgrad(const void* dy, int64_t m, int64_t n, int64_t lddy, const void* w_codes,
                            const void* w_scales, int64_t k, int out_dtype, void* dx, int64_t lddx, hipStream_t s) {
  switch (out_dtype) {
    case LQ_F32: return dgrad_dt<LQ_F32>(dy, m, n, lddy, w_codes, w_scales, k, dx, lddx, s);
    case LQ_BF16: return dgrad_dt<LQ_BF16>(dy, m, n, lddy, w_codes, w_scales, k, dx, lddx, s);
    default: return dgrad_dt<LQ_F16>(dy, m, n, lddy, w_codes, w_scales, k, dx, lddx, s);
  }
}

hipError_t launch_ckpt8_wgrad(int format, const void* dy, int64_t m, int64_t n, int64_t lddy, const void* x_codes,
                              const void* x_scales, int64_t k, const float* dw_in, float* dw, int64_t lddw,
                              hipStream_t s) {
  const dim3 g((unsigned)((k + 63) / 64 * ((n + 63) / 64)));
  if (format == LQ_INT8)
    hipLaunchKernelGGL((k_ckpt8_wgrad<LQ_INT8>), g, dim3(256), 0, s, (const uint16_t*)dy, m, n, lddy,
                       (const uint8_t*)x_codes, (const uint8_t*)x_scales, k, dw_in, dw, lddw);
  else
    hipLaunchKernelGGL((k_ckpt8_wgrad<LQ_E4M3>), g, dim3(256), 0, s, (const uint16_t*)dy, m, n, lddy,
                       (const uint8_t*)x_codes, (const uint8_t*)x_scales, k, dw_in, dw, lddw);
  return hipGetLastError();
}

}  // namespace lql
