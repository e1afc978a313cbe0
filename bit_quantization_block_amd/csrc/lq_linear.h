// lq_linear.h — device-side pieces shared by the low-bit linear layer's kernels
// (lq_mx4.hip, lq_grad.hip, lq_swiglu.hip) and the launchers that lq_linear.hip
// calls.
//
// Two stored forms of a rows x cols matrix, both in blocks of 32 along a row
// with one UE8M0 scale each, the smallest 2^e with Qmax * 2^e >= max|block|:
//   MX4 operand    E2M1 codes in groups of 128 columns, group by group, a
//                  group's 64 bytes of every row one after the other; scales
//                  likewise, 4 bytes a row (rows padded to a multiple of 4).
//                  Elements past cols are zeros. The rows of a tile then have
//                  each step's codes and scales in one stretch of whole cache
//                  lines (with each row in one stretch instead, a step's 64
//                  bytes a row cost the memory pipe as much as 128, and its
//                  scales more than its codes).
//   8-bit checkpoint  INT8 or E4M3 codes, rows padded with zeros to 32
//                  elements; one scale byte per block
// For cols a multiple of 32 the checkpoint is byte for byte what lq_quantize
// writes for INT8 / E4M3, PER_BLOCK 32, UE8M0; the MX4 operand holds the codes
// and scales that it writes for E2M1, in another order.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include <atomic>

#include "lq.h"
#include "lq_device.h"
#include "lq_plan.h"

namespace lql {

constexpr int kBlock = 32;

__host__ __device__ inline int64_t mx4_groups(int64_t cols) { return (cols + 127) / 128; }
__host__ __device__ inline int64_t mx4_scale_rows(int64_t rows) { return (rows + 3) / 4 * 4; }
// Places of the byte that holds a row's element col, and of the scale of its block.
__host__ __device__ inline int64_t mx4_code_at(int64_t rows, int64_t row, int64_t col) {
  return ((col >> 7) * rows + row) * 64 + (col >> 1 & 63);
}
__host__ __device__ inline int64_t mx4_scale_at(int64_t rows, int64_t row, int64_t col) {
  return ((col >> 7) * mx4_scale_rows(rows) + row) * 4 + (col >> 5 & 3);
}
__host__ __device__ inline int64_t ckpt_pitch(int64_t cols) { return (cols + 31) / 32 * 32; }
__host__ __device__ inline int64_t ckpt_scale_pitch(int64_t cols) { return (cols + 31) / 32; }

// ------------------------------------------------------------ floats in memory
template <int DT> struct El;
template <> struct El<LQ_F32> { typedef float T; static constexpr int bytes = 4; };
template <> struct El<LQ_BF16> { typedef uint16_t T; static constexpr int bytes = 2; };
template <> struct El<LQ_F16> { typedef uint16_t T; static constexpr int bytes = 2; };

template <int DT>
__device__ __forceinline__ float widen(typename El<DT>::T b) {
  if constexpr (DT == LQ_F32) return b;
  else if constexpr (DT == LQ_BF16) return __uint_as_float((uint32_t)b << 16);
  else return (float)__builtin_bit_cast(_Float16, b);
}
// Round to the stored type, to nearest even (bf16 through the compiler's own
// conversion, one instruction on gfx950).
template <int DT>
__device__ __forceinline__ typename El<DT>::T narrow(float f) {
  if constexpr (DT == LQ_F32) return f;
  else if constexpr (DT == LQ_BF16) return __builtin_bit_cast(uint16_t, (__bf16)f);
  else return __builtin_bit_cast(uint16_t, (_Float16)f);
}

// Eight consecutive elements of a row as they are stored, the first `valid` of
// which exist; the rest are zero. Rows need not start at a multiple of 16 bytes
// (the caller's row stride is any number of elements): the vector loads carry
// the element's alignment, which gfx950's global memory instructions take as
// they are.
template <int DT>
struct Raw8 { typename El<DT>::T t[8]; };
template <int DT>
__device__ __forceinline__ Raw8<DT> load_raw8(const void* row, int64_t col, int valid) {
  typedef typename El<DT>::T T;
  const T* p = (const T*)row + col;
  Raw8<DT> r;
  if (valid >= 8) {
    __builtin_memcpy(r.t, p, sizeof(r.t));
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) r.t[i] = i < valid ? p[i] : (T)0;
  }
  return r;
}
template <int DT>
__device__ __forceinline__ void widen8(const Raw8<DT>& r, float v[8]) {
#pragma unroll
  for (int i = 0; i < 8; i++) v[i] = widen<DT>(r.t[i]);
}
template <int DT>
__device__ __forceinline__ void load8(const void* row, int64_t col, int valid, float v[8]) {
  widen8<DT>(load_raw8<DT>(row, col, valid), v);
}
// 16 bytes of a result, past the caches: what these kernels write is larger than
// an L2, and lines that it would have to make room for and give back cost more
// than they are worth to the next reader. 8192 x 11008 x 4096 forward 203 instead
// of 224 us, 2548 x 16384 x 256 30 instead of 46; 154 x 11008 x 4096 added to dw
// 72 instead of 92; the gated unit 123 instead of 141 forward, 121 instead of 150
// backward. A gated MLP's forward of these kernels, each of which reads what the
// last one wrote, takes 765 instead of 816 us at 8192 x 11008 x 4096, 134 instead
// of 145 at 1024 rows, and 2 us of 31 more at 256 rows of 2048 x 1024.
__device__ __forceinline__ void store16(void* p, const void* v) {
  typedef uint32_t v4 __attribute__((ext_vector_type(4), aligned(2)));
  v4 w;
  __builtin_memcpy(&w, v, 16);
  __builtin_nontemporal_store(w, (v4*)p);
}
// Eight results of a streaming kernel. (32-bit ones take two stores a lane that
// each cover half of every line, and are 8% slower past the caches.)
template <int DT>
__device__ __forceinline__ void store8(void* row, int64_t col, int valid, const float v[8]) {
  typedef typename El<DT>::T T;
  T* p = (T*)row + col;
  T t[8];
#pragma unroll
  for (int i = 0; i < 8; i++) t[i] = narrow<DT>(v[i]);
  if (valid >= 8) {
    if constexpr (sizeof(T) == 2) store16(p, t);
    else __builtin_memcpy(p, t, sizeof(t));
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++)
      if (i < valid) p[i] = t[i];
  }
}

// ------------------------------------------------------------ block scales
// A scale byte from the bits of max|block|. Qmax = 2^(qexp-1) * (1 + f): the
// exponent field of amax, one more if amax's significand is above Qmax's,
// less Qmax's own exponent; clamped at 2^-127. A block that holds an infinity
// or a NaN (whose bits, without the sign, are the largest) gets the NaN scale
// 0xFF, and what is computed from it is NaN: a spoiled activation shows.
template <int F> struct Sig;   // significand field of Qmax
template <> struct Sig<LQ_E2M1> { static constexpr uint32_t bits = 0x400000u; };   // 1.5
template <> struct Sig<LQ_INT8> { static constexpr uint32_t bits = 0x7E0000u; };   // 127 / 64
template <> struct Sig<LQ_E4M3> { static constexpr uint32_t bits = 0x600000u; };   // 1.75
constexpr uint32_t kInfBits = 0x7F800000u;
template <int F>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  const int e = (int)((amax_bits + (0x7FFFFFu - Sig<F>::bits)) >> 23) + 1 - lqd::Fmt<F>::qexp;
  return amax_bits >= kInfBits ? 255u : (uint32_t)(e < 0 ? 0 : e);
}
// 2^-e of a finite scale byte (e = byte - 127), exact; 0 for the NaN scale,
// whose block's codes are all zero.
__device__ __forceinline__ float scale_recip(uint32_t byte) {
  return byte == 255u ? 0.0f : __uint_as_float((254u - byte) << 23);
}
// The scale's value: 2^(byte-127), subnormal for byte 0, NaN for 0xFF (both
// are the exponent field with the top fraction bit set).
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __uint_as_float((byte << 23) | ((byte == 0u || byte == 255u) ? 0x00400000u : 0u));
}

// max over the four lanes of a quad, in all four
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);
  v = v > o ? v : o;
  o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true);
  return v > o ? v : o;
}
// The bits of max|v| as binary32, of eight elements: magnitudes order like their
// bits, also where a comparison of the values would lose a NaN; 16-bit ones two
// at a time.
typedef uint16_t v2u16 __attribute__((ext_vector_type(2)));
template <int DT>
__device__ __forceinline__ uint32_t amax8_bits(const Raw8<DT>& r) {
  if constexpr (DT == LQ_F32) {
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const uint32_t b = __float_as_uint(r.t[i]) & 0x7FFFFFFFu;
      a = a > b ? a : b;
    }
    return a;
  } else {
    uint32_t w[4];
    __builtin_memcpy(w, r.t, 16);
    v2u16 top = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; i++) top = __builtin_elementwise_max(top, __builtin_bit_cast(v2u16, w[i] & 0x7FFF7FFFu));
    return __float_as_uint(widen<DT>(top[0] > top[1] ? top[0] : top[1]));
  }
}

// Eight elements of one block as codes; r the scale's reciprocal, 0 for the
// NaN scale (an infinite or NaN element times 0 is NaN, so the codes are
// cleared explicitly).
__device__ __forceinline__ uint32_t encode_e2m1(const float v[8], float r) {
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; i++) q[i] = v[i] * r;
  return r == 0.0f ? 0u : lqd::fp4_pack8(q);
}
template <int F>
__device__ __forceinline__ uint2 encode8(const float v[8], float r) {
  uint2 w;
  if constexpr (F == LQ_INT8) {
    // v r is exact and at most 127 in magnitude; adding 1.5 * 2^23 rounds it to
    // an integer, half to even, whose low byte is the code
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; i++) c[i] = __float_as_uint(__builtin_fmaf(v[i], r, 12582912.0f));
    const uint32_t ab = __builtin_amdgcn_perm(c[1], c[0], 0x0C0C0400u), cd = __builtin_amdgcn_perm(c[3], c[2], 0x04000C0Cu);
    const uint32_t ef = __builtin_amdgcn_perm(c[5], c[4], 0x0C0C0400u), gh = __builtin_amdgcn_perm(c[7], c[6], 0x04000C0Cu);
    w.x = ab | cd;
    w.y = ef | gh;
  } else {
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; i++) q[i] = lqd::clampf(v[i] * r, -448.0f, 448.0f);
    w.x = lqd::fp8_pack4<LQ_E4M3>(q[0], q[1], q[2], q[3]);
    w.y = lqd::fp8_pack4<LQ_E4M3>(q[4], q[5], q[6], q[7]);
  }
  if (r == 0.0f) w = make_uint2(0u, 0u);
  return w;
}
// The values of four 8-bit codes times the scale.
template <int F>
__device__ __forceinline__ void decode4(uint32_t w, float s, float o[4]) {
  if constexpr (F == LQ_INT8) {
#pragma unroll
    for (int i = 0; i < 4; i++) o[i] = (float)(int8_t)(w >> (8 * i)) * s;
  } else {
    lqd::fp8_unpack4<LQ_E4M3>(w, o);
#pragma unroll
    for (int i = 0; i < 4; i++) o[i] *= s;
  }
}

// A launch over a matrix: `across` workgroups in x, and in y one for each four
// rows, each taking several beyond the grid's limit.
inline dim3 matrix_grid(int64_t across, int64_t rows) {
  const int64_t bands = (rows + 3) / 4;
  return dim3((unsigned)across, (unsigned)(bands < 65535 ? bands : 65535));
}

// Whether a gradient reads dy where it lies, or a copy in the workspace with rows
// of a multiple of 64 elements, padded by zeros. Rows that are no multiples of 16
// bytes are read in place too (dx 77 x 1001 x 520 11 us, 13.5 with a copy; 8192 x
// 11004 x 4096 563 us, 601 with one), but not
//  - with strides whose 256 rows pass 32-bit offsets, or
//  - where the last element alone makes up the first half of a 4-byte word
//    that ends the last row's loads (n odd) and the second half of one of memory:
//    the load's word would reach past the matrix, perhaps into a page that is not
//    there.
inline bool reads_in_place(int64_t m, int64_t n, int64_t lddy) {
  if (lddy > 1 << 21) return false;
  if (n % 8 == 0 && lddy % 8 == 0) return true;
  if (n % 2 != 0 && ((m - 1) * lddy + n) % 2 == 0) return false;
  return true;
}
inline int64_t padded_columns(int64_t n) { return (n + 63) / 64 * 64; }

// ------------------------------------------------------------ rows by expert
// Rows of x, y and dy lie expert by expert: offsets[e] .. offsets[e + 1] - 1 are
// expert e's, on the device. Whatever they hold, the ranges taken from them ascend and
// stay within the m rows.
constexpr int kMostExperts = 512;
struct Experts {
  const int32_t* offsets;
  int count;
};
// Inclusive scan over a wave (0 changes nothing in `op`): within rows of 16, then the rows' last lanes on to the next rows.
template <class OP>
__device__ __forceinline__ uint32_t wave_scan(uint32_t v, OP op) {
  v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, false));   // row_shr 1
  v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, false));
  v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, false));
  v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, false));
  v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false));   // row_bcast 15, to rows 1 and 3
  v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false));   // row_bcast 31, to rows 2 and 3
  return v;
}
// A wave's table of the experts' ranges, one expert in each lane of each register: the
// tiles' LDS leaves no room for one (512 experts' 4 KB keep a second workgroup of 128 x
// 128 off a compute unit).
struct ExpertTable {
  uint32_t end[kMostExperts / 64];     // of each expert's rows
  uint32_t tiles[kMostExperts / 64];   // of `side` rows up to each expert's last
  uint32_t first;                      // row of the first expert's

  __device__ __forceinline__ void scan(const Experts& x, int64_t m, uint32_t side) {
    const int lane = threadIdx.x & 63;
    auto offset = [&](int i) {
      const int32_t raw = x.offsets[i < x.count ? i : x.count];
      return raw < 0 ? 0u : raw > m ? (uint32_t)m : (uint32_t)raw;
    };
    uint32_t top = first = __builtin_amdgcn_readfirstlane(offset(0)), sum = 0;
#pragma unroll
    for (int c = 0; c < kMostExperts / 64; c++) end[c] = tiles[c] = 0;
#pragma unroll
    for (int c = 0; c < kMostExperts / 64; c++) {
      if (c * 64 >= x.count) break;   // (one branch for up to 64 experts, here and below)
      uint32_t e = offset(c * 64 + lane + 1);   // (of lanes past the last expert, the last end again)
      e = e > top ? e : top;
      e = wave_scan(e, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
      const uint32_t before = (uint32_t)__builtin_amdgcn_update_dpp((int)top, (int)e, 0x138, 0xF, 0xF, false);   // wave_shr 1
      const uint32_t t = wave_scan((e - before + side - 1) / side, [](uint32_t a, uint32_t b) { return a + b; });
      end[c] = e;
      tiles[c] = sum + t;
      top = __builtin_amdgcn_readlane(e, 63);
      sum = __builtin_amdgcn_readlane(tiles[c], 63);
    }
  }
  // Of expert i (uniform).
  static __device__ __forceinline__ uint32_t pick(const uint32_t (&v)[kMostExperts / 64], uint32_t i) {
    uint32_t r = __builtin_amdgcn_readlane(v[0], i % 64);
    if (i >= 64) {
#pragma unroll
      for (int c = 1; c < kMostExperts / 64; c++)
        if (i / 64 == c) r = __builtin_amdgcn_readlane(v[c], i % 64);
    }
    return r;
  }
  __device__ __forceinline__ uint32_t row_end(uint32_t i) const { return pick(end, i); }
  __device__ __forceinline__ uint32_t row_begin(uint32_t i) const { return i ? pick(end, i - 1) : first; }
  __device__ __forceinline__ uint32_t tiles_to(uint32_t i) const { return pick(tiles, i); }
  __device__ __forceinline__ uint32_t tiles_before(uint32_t i) const { return i ? pick(tiles, i - 1) : 0; }
  // The expert of the t-th tile of rows (t below all of them).
  __device__ __forceinline__ uint32_t at(uint32_t t, int count) const {
    uint32_t n = 0;
#pragma unroll
    for (int c = 0; c < kMostExperts / 64; c++) {
      if (c * 64 >= count) break;
      n += (uint32_t)__builtin_popcountll(__ballot(tiles[c] <= t && c * 64 + (int)(threadIdx.x & 63) < count));
    }
    return n;
  }
};
// One expert's rows straight from memory. (By scalar loads: a vector load's wait is one for all that is on its way.)
__device__ __forceinline__ void expert_rows(const Experts& x, int64_t m, int e, int64_t& begin, int64_t& end) {
  const auto offsets = (const __attribute__((address_space(4))) int32_t*)(uintptr_t)x.offsets;
  const int32_t b = offsets[e], n = offsets[e + 1];
  begin = b < 0 ? 0 : b > m ? m : b;
  end = n < begin ? begin : n > m ? m : n;
}

// ------------------------------------------------------------ shapes of the products
// Compute units of the current device (256 on MI355X, or with no device).
inline int compute_units() {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  int cus = cached[dev].load(std::memory_order_relaxed);
  if (cus == 0) {
    if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0) cus = 256;
    cached[dev].store(cus, std::memory_order_relaxed);
  }
  return cus;
}
// How a product of rows x cols over `steps` steps of its contraction is shared
// out: tiles of 64 tile x 64 tile, each of whose contraction is cut into
// `parts` runs of `part` steps, whose sums are added up afterwards.
struct Split { int tile, parts, part; };
Split split_product(int64_t m, int64_t n, int64_t k, int out_dtype);                                     // steps of 128
Split split_dgrad(int64_t m, int64_t n, int64_t k), split_wgrad(int64_t m, int64_t n, int64_t k, bool adds);   // steps of 64
// Workspace of the parts' sums: planes with rows of a multiple of 4 values.
__host__ __device__ inline int64_t plane_stride(int64_t cols) { return (cols + 3) / 4 * 4; }
inline size_t planes_bytes(const Split& c, int64_t rows, int64_t cols) {
  return c.parts > 1 ? (size_t)c.parts * (size_t)(rows * plane_stride(cols)) * 4 : 0;
}

// The tile of a product over rows that lie by expert: rows / experts of them on the average (steps of 128, of 64, of 64).
int expert_tile(int64_t m, int64_t n, int64_t k, int experts);
Split split_experts_dgrad(int64_t m, int64_t n, int64_t k, int experts);

// ------------------------------------------------------------ launchers
// Instead of launching, the kernel's name and its template arguments for a plan being recorded (lq_plan.h).
#define LQ_PLAN(grid, threads, ...) lqd::plan_add((int64_t)(grid).x * (grid).y, threads, __VA_ARGS__)
// (lq_mx4.hip, lq_grad.hip, lq_swiglu.hip; arguments checked by lq_linear.hip)
hipError_t launch_mx4_quantize(int in_dtype, int ckpt_format, const void* x, int64_t m, int64_t k, int64_t ldx,
                               void* codes, void* scales, void* ckpt_codes, void* ckpt_scales, hipStream_t s);
hipError_t launch_constant(int64_t rows, int64_t cols, int dtype, const void* in, void* y, int64_t ldy, hipStream_t s);
// (of the experts' rows only)
hipError_t launch_join_experts(const Experts& e, int64_t rows, int64_t cols, int dtype, int parts, const float* planes, void* y,
                               int64_t ldy, hipStream_t s);
hipError_t launch_join(int64_t rows, int64_t cols, int dtype, int parts, const float* planes, const float* in, void* y,
                       int64_t ldy, hipStream_t s);
hipError_t launch_mx4_product(const void* a_codes, const void* a_scales, const void* w_codes, const void* w_scales,
                              int64_t m, int64_t n, int64_t k, int out_dtype, void* y, int64_t ldy, void* planes,
                              hipStream_t s);
// The forward product of a few rows straight from x: at most kFewBlocks blocks
// of it (padded to whole groups), which each workgroup, of 16 columns or more,
// quantises into its LDS. With more than one workgroup on a compute unit that work
// counts more than once, and a launch of its own for it is sooner worth it (in
// place, or apart; 11008 x 4096: 8 rows 8.2 or 9.0 us, 12 rows 9.9 or 9.3; 4096 x
// 4096: 12 rows 6.0 or 8.0, 16 rows 7.0 or 7.6).
constexpr int64_t kFewRows = 16, kFewBlocks = 2048, kFewBlocksWide = 1024;
inline bool few_rows(int64_t m, int64_t n, int64_t k) {
  return m <= kFewRows && m * mx4_groups(k) * 4 <= (n <= 16 * compute_units() ? kFewBlocks : kFewBlocksWide);
}
hipError_t launch_mx4_few(int in_dtype, const void* x, int64_t ldx, const void* w_codes, const void* w_scales, int64_t m,
                          int64_t n, int64_t k, int out_dtype, void* y, int64_t ldy, hipStream_t s);
hipError_t launch_mx4_dgrad(const void* dy, int64_t m, int64_t n, int64_t lddy, const void* w_codes,
                            const void* w_scales, int64_t k, int out_dtype, void* dx, int64_t lddx, void* ws,
                            hipStream_t s);
hipError_t launch_ckpt8_wgrad(int format, const void* dy, int64_t m, int64_t n, int64_t lddy, const void* x_codes,
                              const void* x_scales, int64_t k, const float* dw_in, float* dw, int64_t lddw, void* ws,
                              hipStream_t s);
hipError_t launch_swiglu(int dtype, int format, const void* gate, const void* up, int64_t rows, int64_t cols,
                         int64_t ld, void* h, int64_t ldh, void* gc, void* gs, void* uc, void* us, hipStream_t s);
hipError_t launch_swiglu_backward(int dtype, int format, const void* dh, int64_t rows, int64_t cols, int64_t lddh,
                                  const void* gc, const void* gs, const void* uc, const void* us, void* dgate,
                                  void* dup, int64_t ld, hipStream_t s);

// The norm (lq_rmsnorm.hip; arguments checked by lq_layers.hip). Backward, x is dy, r is dh and y is dx, and without
// dw there are no planes.
struct NormArgs {
  const void *x, *r, *w;
  void *h, *y;
  uint8_t *codes, *scales;
  float *rs, *planes;
  int64_t rows, cols, ldx, ldr, ldh, ldy;
  float eps;
  bool wide;   // w is binary32
};
constexpr int64_t kNormColumns = 16384;
int64_t norm_planes(int64_t rows, int64_t cols);
hipError_t launch_rmsnorm(int dtype, int format, const NormArgs& a, hipStream_t s);
hipError_t launch_rmsnorm_backward(int dtype, const NormArgs& a, const float* dw_in, float* dw, hipStream_t s);

// The 4-bit integer layer (lq_int4.hip): a packed layer is codes, then scales, then zero points.
size_t int4_codes_bytes(int64_t n, int64_t k);
size_t int4_scales_bytes(int64_t n, int64_t k, int group);
size_t int4_rows_bytes(const lq_int4_desc* d);
hipError_t launch_int4_pack(const lq_int4_desc* d, const void* codes, const void* scales, const void* zeros, void* packed,
                            hipStream_t s);
hipError_t launch_int4_linear(const lq_int4_desc* d, const void* x, const void* x_scales, const void* packed, void* y,
                              void* ws, hipStream_t s);

// The layer of many experts (lq_mx4.hip, lq_grad.hip): W is an MX4 operand of experts * n rows.
bool experts_in_place(int64_t m, int64_t k, int experts);
hipError_t launch_mx4_experts_few(int in_dtype, const void* x, int64_t ldx, const Experts& e, const void* w_codes,
                                  const void* w_scales, int64_t m, int64_t n, int64_t k, int out_dtype, void* y, int64_t ldy,
                                  hipStream_t s);
hipError_t launch_mx4_experts(const void* a_codes, const void* a_scales, const Experts& e, const void* w_codes,
                              const void* w_scales, int64_t m, int64_t n, int64_t k, int out_dtype, void* y, int64_t ldy,
                              hipStream_t s);
hipError_t launch_mx4_experts_dgrad(const void* dy, const Experts& e, int64_t m, int64_t n, int64_t lddy,
                                    const void* w_codes, const void* w_scales, int64_t k, int out_dtype, void* dx,
                                    int64_t lddx, void* ws, hipStream_t s);
hipError_t launch_ckpt8_experts_wgrad(int format, const void* dy, const Experts& e, int64_t m, int64_t n, int64_t lddy,
                                      const void* x_codes, const void* x_scales, int64_t k, const float* dw_in, float* dw,
                                      int64_t lddw, void* ws, hipStream_t s);

}  // namespace lql
