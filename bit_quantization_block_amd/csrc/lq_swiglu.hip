// lq_swiglu.hip — the gated activation h = silu(g) u with 8-bit checkpoints of g
// and u, and its backward pass from them.
#include "lq_linear.h"

namespace lql {
namespace {

// 1 / (1 + exp(-g)) in binary32: exp's library function and an IEEE division,
// so that binary32 outputs are good to a few units in the last place; an
// exp that overflows gives 0.
__device__ __forceinline__ float sigmoid(float g) { return 1.0f / (1.0f + expf(-g)); }

template <int F>
__device__ __forceinline__ void keep(const float v[8], uint8_t* codes, uint8_t* scales, int64_t row, int64_t col,
                                     int64_t cols, int lane) {
  const uint32_t sb = scale_byte<F>(quad_max(amax8_bits(v)));
  const uint2 w = encode8<F>(v, scale_recip(sb));
  if (col < ckpt_pitch(cols)) {
    *(uint2*)(codes + row * ckpt_pitch(cols) + col) = w;
    if ((lane & 3) == 0) scales[row * ckpt_scale_pitch(cols) + col / 32] = (uint8_t)sb;
  }
}
template <int F>
__device__ __forceinline__ void recall(float v[8], const uint8_t* codes, const uint8_t* scales, int64_t row,
                                       int64_t col, int64_t cols) {
  const uint2 w = *(const uint2*)(codes + row * ckpt_pitch(cols) + col);
  const float s = scale_value(scales[row * ckpt_scale_pitch(cols) + col / 32]);
  decode4<F>(w.x, s, v);
  decode4<F>(w.y, s, v + 4);
}

// One wave per 512 columns of a row, 8 consecutive elements per lane.
template <int DT, int F>
__global__ __launch_bounds__(256) void k_swiglu(const void* gate, const void* up, int64_t rows, int64_t cols,
                                                int64_t ld, void* h, int64_t ldh, uint8_t* gc, uint8_t* gs,
                                                uint8_t* uc, uint8_t* us) {
  typedef typename El<DT>::T T;
  const int64_t segs = (cols + 511) / 512;
  for (int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); unit < rows * segs; unit += (int64_t)gridDim.x * 4) {
  const int64_t row = unit / segs;
  const int lane = threadIdx.x & 63;
  const int64_t col = (unit % segs) * 512 + lane * 8;
  const int valid = col >= cols ? 0 : (cols - col >= 8 ? 8 : (int)(cols - col));
  float g[8], u[8];
  load8<DT>((const T*)gate + row * ld, col, valid, g);
  load8<DT>((const T*)up + row * ld, col, valid, u);
  if (gc) keep<F>(g, gc, gs, row, col, cols, lane);
  if (uc) keep<F>(u, uc, us, row, col, cols, lane);
  if (h) {
#pragma unroll
    for (int i = 0; i < 8; i++) g[i] = g[i] * sigmoid(g[i]) * u[i];
    store8<DT>((T*)h + row * ldh, col, valid, g);
  }
  }
}

template <int DT, int F>
__global__ __launch_bounds__(256) void k_swiglu_backward(const void* dh, int64_t rows, int64_t cols, int64_t lddh,
                                                         const uint8_t* gc, const uint8_t* gs, const uint8_t* uc,
                                                         const uint8_t* us, void* dgate, void* dup, int64_t ld) {
  typedef typename El<DT>::T T;
  const int64_t segs = (cols + 511) / 512;
  for (int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); unit < rows * segs; unit += (int64_t)gridDim.x * 4) {
  const int64_t row = unit / segs;
  const int64_t col = (unit % segs) * 512 + (threadIdx.x & 63) * 8;
  if (col >= cols) continue;
  const int valid = cols - col >= 8 ? 8 : (int)(cols - col);
  float d[8], g[8], u[8];
  load8<DT>((const T*)dh + row * lddh, col, valid, d);
  recall<F>(g, gc, gs, row, col, cols);
  recall<F>(u, uc, us, row, col, cols);
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const float s = sigmoid(g[i]);
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
  const dim3 grid(stream_grid(rows * ((cols + 511) / 512)));
  hipLaunchKernelGGL((k_swiglu<DT, F>), grid, dim3(256), 0, s, gate, up, rows, cols, ld, h, ldh, (uint8_t*)gc,
                     (uint8_t*)gs, (uint8_t*)uc, (uint8_t*)us);
  return hipGetLastError();
}
template <int DT, int F>
hipError_t backward_dt(const void* dh, int64_t rows, int64_t cols, int64_t lddh, const void* gc, const void* gs,
                       const void* uc, const void* us, void* dgate, void* dup, int64_t ld, hipStream_t s) {
  const dim3 grid(stream_grid(rows * ((cols + 511) / 512)));
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
