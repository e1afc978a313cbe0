// lq_swiglu.hip — the gated activation h = silu(g) u with 8-bit checkpoints of g
// and u, and its backward pass from them:
//
//   s = 1 / (1 + exp(-g))   du = dh g s   dg = dh u s (1 + g (1 - s))
//
// with g and u in the backward pass as the checkpoints hold them. Both passes
// read and write each matrix once and keep nothing; they are bound by memory. At
// 8192 x 11008 of bf16: 123 us forward and 121 us backward, 5.9 and 6.0 TB/s
// (8.06 bytes an element), above the 5.2 TB/s of a large copy, since most of what
// is written goes past the caches. Vector work was the bound before it was cut:
// codes decoded by sub-word converts, rounded by one fused multiply-add, 16-bit
// maxima two at a time, and no division to find a place (184 us backward with
// 64-bit places, the library's exp and a divided sigmoid). At 8192 x 11008 of
// binary32: 237 us forward and 262 us backward, 5.3 and 4.8 TB/s (14.06 bytes an
// element).
#include "lq_linear.h"

namespace lql {
namespace {

// 1 / (1 + exp(-g)), in binary32; an exp that overflows gives 0.
// For 32-bit matrices the library's exp and an IEEE division: off by a unit in
// exp's last place and the roundings of the sum and the quotient; the memory's time
// hides them (237 and 262 us, and with the short form below too).
// For 16-bit matrices, whose results keep 11 bits at most, a third of the
// instructions, without which vector work would be the bound: exp(-g) = 2^t
// (1 + ln2 rest), with t = -g log2(e) rounded and its remainder exact by fused
// multiply-adds over log2(e) in two parts. v_exp_f32 and v_rcp_f32 are good to a
// unit in the last place, which with the sum's and the products' roundings makes
// at most 7 * 2^-24 relative.
template <int DT>
__device__ __forceinline__ float sigmoid(float g) {
  if constexpr (DT == LQ_F32) return 1.0f / (1.0f + expf(-g));
  constexpr float hi = -1.4426950216293335f, lo = -1.925963e-08f, ln2 = 0.6931471805599453f;
  const float t = g * hi, rest = __builtin_fmaf(g, lo, __builtin_fmaf(g, hi, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  // (an infinite g has no remainder, and neither have an exp of 0 or infinity)
  const float fine = __builtin_fabsf(t) < 128.0f ? __builtin_fmaf(e * ln2, rest, e) : e;
  // (1 + exp)/4 keeps the reciprocal, which has no subnormal numbers, a normal one
  return 0.25f * __builtin_amdgcn_rcpf(__builtin_fmaf(fine, 0.25f, 0.25f));
}

template <int DT, int F>
__device__ __forceinline__ void keep(const Raw8<DT>& raw, const float v[8], uint8_t* codes, uint8_t* scales, int64_t row,
                                     int64_t col, int64_t cols, int lane) {
  const uint32_t sb = scale_byte<F>(quad_max(amax8_bits<DT>(raw)));
  const uint2 w = encode8<F>(v, scale_recip(sb));
  if (col < ckpt_pitch(cols)) {
    __builtin_nontemporal_store(__builtin_bit_cast(uint64_t, w), (uint64_t*)(codes + row * ckpt_pitch(cols) + col));
    if ((lane & 3) == 0) scales[row * ckpt_scale_pitch(cols) + col / 32] = (uint8_t)sb;
  }
}

// One wave per 512 columns of a row, 8 consecutive elements per lane, four rows
// a workgroup.
template <int DT, int F>
__global__ __launch_bounds__(256) void k_swiglu(const void* gate, const void* up, int64_t rows, int64_t cols,
                                                int64_t ld, void* h, int64_t ldh, uint8_t* gc, uint8_t* gs,
                                                uint8_t* uc, uint8_t* us) {
  typedef typename El<DT>::T T;
  const int lane = threadIdx.x & 63;
  const int64_t col = (int64_t)blockIdx.x * 512 + lane * 8;
  const int valid = col >= cols ? 0 : (cols - col >= 8 ? 8 : (int)(cols - col));
  for (int64_t row = (int64_t)blockIdx.y * 4 + (threadIdx.x >> 6); row < rows; row += (int64_t)gridDim.y * 4) {
    const Raw8<DT> rg = load_raw8<DT>((const T*)gate + row * ld, col, valid), ru = load_raw8<DT>((const T*)up + row * ld, col, valid);
    float g[8], u[8];
    widen8<DT>(rg, g);
    widen8<DT>(ru, u);
    if (gc) {
      keep<DT, F>(rg, g, gc, gs, row, col, cols, lane);
      keep<DT, F>(ru, u, uc, us, row, col, cols, lane);
    }
    if (h) {
#pragma unroll
      for (int i = 0; i < 8; i++) g[i] = g[i] * sigmoid<DT>(g[i]) * u[i];
      store8<DT>((T*)h + row * ldh, col, valid, g);
    }
  }
}

template <int DT, int F>
__global__ __launch_bounds__(256) void k_swiglu_backward(const void* dh, int64_t rows, int64_t cols, int64_t lddh,
                                                         const uint8_t* gc, const uint8_t* gs, const uint8_t* uc,
                                                         const uint8_t* us, void* dgate, void* dup, int64_t ld) {
  typedef typename El<DT>::T T;
  const int64_t col = (int64_t)blockIdx.x * 512 + (threadIdx.x & 63) * 8;
  if (col >= cols) return;
  const int valid = cols - col >= 8 ? 8 : (int)(cols - col);
  for (int64_t row = (int64_t)blockIdx.y * 4 + (threadIdx.x >> 6); row < rows; row += (int64_t)gridDim.y * 4) {
    const int64_t code = row * ckpt_pitch(cols) + col, scale = row * ckpt_scale_pitch(cols) + col / 32;
    const uint2 wg = *(const uint2*)(gc + code), wu = *(const uint2*)(uc + code);
    const float sg = scale_value(gs[scale]), su = scale_value(us[scale]);
    float d[8], g[8], u[8];
    load8<DT>((const T*)dh + row * lddh, col, valid, d);
    decode4<F>(wg.x, sg, g);
    decode4<F>(wg.y, sg, g + 4);
    decode4<F>(wu.x, su, u);
    decode4<F>(wu.y, su, u + 4);
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const float s = sigmoid<DT>(g[i]);
      u[i] = d[i] * u[i] * s * (1.0f + g[i] * (1.0f - s));
      g[i] = d[i] * (g[i] * s);
    }
    store8<DT>((T*)dgate + row * ld, col, valid, u);
    store8<DT>((T*)dup + row * ld, col, valid, g);
  }
}

template <int DT, int F>
hipError_t forward_dt(const void* gate, const void* up, int64_t rows, int64_t cols, int64_t ld, void* h, int64_t ldh,
                      void* gc, void* gs, void* uc, void* us, hipStream_t s) {
  const dim3 grid = matrix_grid((cols + 511) / 512, rows);
  hipLaunchKernelGGL((k_swiglu<DT, F>), grid, dim3(256), 0, s, gate, up, rows, cols, ld, h, ldh, (uint8_t*)gc,
                     (uint8_t*)gs, (uint8_t*)uc, (uint8_t*)us);
  return hipGetLastError();
}
template <int DT, int F>
hipError_t backward_dt(const void* dh, int64_t rows, int64_t cols, int64_t lddh, const void* gc, const void* gs,
                       const void* uc, const void* us, void* dgate, void* dup, int64_t ld, hipStream_t s) {
  const dim3 grid = matrix_grid((cols + 511) / 512, rows);
  hipLaunchKernelGGL((k_swiglu_backward<DT, F>), grid, dim3(256), 0, s, dh, rows, cols, lddh, (const uint8_t*)gc,
                     (const uint8_t*)gs, (const uint8_t*)uc, (const uint8_t*)us, dgate, dup, ld);
  return hipGetLastError();
}

}  // namespace

#define LQ_PICK(fn, ...)                                                                  \
  if (format == LQ_INT8) {                                                                \
    if (dtype == LQ_F32) return fn<LQ_F32, LQ_INT8>(__VA_ARGS__);                         \
    if (dtype == LQ_BF16) return fn<LQ_BF16, LQ_INT8>(__VA_ARGS__);                       \
    return fn<LQ_F16, LQ_INT8>(__VA_ARGS__);                                              \
  }                                                                                       \
  if (dtype == LQ_F32) return fn<LQ_F32, LQ_E4M3>(__VA_ARGS__);                           \
  if (dtype == LQ_BF16) return fn<LQ_BF16, LQ_E4M3>(__VA_ARGS__);                         \
  return fn<LQ_F16, LQ_E4M3>(__VA_ARGS__);

hipError_t launch_swiglu(int dtype, int format, const void* gate, const void* up, int64_t rows, int64_t cols,
                         int64_t ld, void* h, int64_t ldh, void* gc, void* gs, void* uc, void* us, hipStream_t s) {
  LQ_PICK(forward_dt, gate, up, rows, cols, ld, h, ldh, gc, gs, uc, us, s)
}

hipError_t launch_swiglu_backward(int dtype, int format, const void* dh, int64_t rows, int64_t cols, int64_t lddh,
                                  const void* gc, const void* gs, const void* uc, const void* us, void* dgate,
                                  void* dup, int64_t ld, hipStream_t s) {
  LQ_PICK(backward_dt, dh, rows, cols, lddh, gc, gs, uc, us, dgate, dup, ld, s)
}

}  // namespace lql
