// lq_int4.hip — few rows of x times 4-bit integer weights with a scale, and a zero
// point or none, for each group of 32, 64 or 128 along k:
//
//   y[m, n] = sum over groups g of s[n, g] * sum over k in g of (q[n, k] - z[n, g]) x[m, k]
//
// The call is bound by reading W once. A code becomes the 16-bit float 16 + u, u = q +
// 8, by a shift and a mask (its mantissa's upper bits are u); the matrix cores add up
// (16 + u) x in binary32, exact products all, and with a row of ones next to W the sum
// of x; a group's end takes 24 + z times that sum off and multiplies by the scale:
//
//   sum (q - z) x = sum (16 + u) x - (24 + z) sum x
//
// What is taken off is a few times what is left (codes of normal weights: 24 against a
// root mean square of about 4), so the sums' rounding counts that much more: 2^-22 of
// the row's |x| |w| instead of 2^-24.
#include "lq_linear.h"

namespace lql {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

constexpr int kStep = 128;   // of the contraction: 64 bytes of a row of W
constexpr int kWaves = 8;
// The sources of x besides the float types: 8-bit checkpoints.
constexpr int kInt8 = 3, kE4m3 = 4;

// ---------------------------------------------------------------- packing
// Codes [step][row][64 bytes], rows padded to a multiple of 32: the 16 rows of a tile
// are a kilobyte in one stretch. Word 4 p + i of a row's 64 bytes holds the columns 32 i
// + 8 p .. + 7, so that the 16 bytes of the lane (row, p) are what it multiplies in four
// products of 32 columns each; element e of a word is nibble e / 2 (+ 4 if e is odd), so
// that a shift and a mask leave two neighbours in the two halves of a register. Scales
// and zero points [step][group of the step][row].
__host__ __device__ inline int64_t padded_rows(int64_t n) { return (n + 31) / 32 * 32; }
__host__ __device__ inline int64_t steps_of(int64_t k) { return (k + kStep - 1) / kStep; }

__global__ __launch_bounds__(256) void k_int4_pack(const uint8_t* codes, const uint16_t* scales, const uint16_t* zeros,
                                                   int64_t n, int64_t k, int group, uint8_t* out, uint16_t* s, uint16_t* z) {
  const int64_t np = padded_rows(n), row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= np) return;
  const int word = threadIdx.x & 15, at = threadIdx.x >> 4 & 3;   // 4 steps a wave, a word a lane
  const int each = kStep / group;
  for (int64_t step = (int64_t)blockIdx.y * 4 + at; step < steps_of(k); step += (int64_t)gridDim.y * 4) {
    const int64_t col = step * kStep + (word & 3) * 32 + (word >> 2) * 8;
    uint32_t v = 0;
    if (row < n && col < k) {
      const uint32_t w = *(const uint32_t*)(codes + row * (k / 2) + col / 2) ^ 0x88888888u;
#pragma unroll
      for (int e = 0; e < 8; e++) v |= (w >> (4 * e) & 15u) << (4 * (e / 2 + (e & 1) * 4));
    }
    *(uint32_t*)(out + (step * np + row) * 64 + word * 4) = v;
    if (word < each) {
      const int64_t g = step * each + word, to = (step * each + word) * np + row;
      const bool there = row < n && g * group < k;
      s[to] = there ? scales[row * (k / group) + g] : (uint16_t)0;
      if (zeros) z[to] = there ? zeros[row * (k / group) + g] : (uint16_t)0;
    }
  }
}

// ---------------------------------------------------------------- x
// Eight elements of a row of x as they are stored.
template <int SRC> struct X8 { v4i v; };
template <> struct X8<LQ_F32> { v4f v[2]; };
template <> struct X8<kInt8> { uint2 v; uint32_t s; };
template <> struct X8<kE4m3> { uint2 v; uint32_t s; };
// What the matrix cores take of them: one operand, of binary32 three, whose sum they are
// (8 + 8 + 8 significant bits, each the rounding of what the last left).
template <int SRC> struct Parts { static constexpr int n = SRC == LQ_F32 ? 3 : 1; v4i v[n]; };

__device__ __forceinline__ uint32_t pair_bf16(float lo, float hi) {
  return (uint32_t)narrow<LQ_BF16>(lo) | (uint32_t)narrow<LQ_BF16>(hi) << 16;
}
// (an infinity's or a NaN's remainder is NaN, and so are the sums it goes into)
__device__ __forceinline__ void split3(float v, uint16_t out[3]) {
#pragma unroll
  for (int p = 0; p < 3; p++) {
    out[p] = narrow<LQ_BF16>(v);
    v -= widen<LQ_BF16>(out[p]);
  }
}
template <int SRC>
__device__ __forceinline__ Parts<SRC> operands(const X8<SRC>& x) {
  Parts<SRC> o;
  if constexpr (SRC == LQ_F32) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      uint16_t a[3], b[3];
      split3(x.v[i / 2][i % 2 * 2], a);
      split3(x.v[i / 2][i % 2 * 2 + 1], b);
#pragma unroll
      for (int p = 0; p < 3; p++) o.v[p][i] = (int)((uint32_t)a[p] | (uint32_t)b[p] << 16);
    }
  } else if constexpr (SRC == kInt8 || SRC == kE4m3) {
    constexpr int F = SRC == kInt8 ? LQ_INT8 : LQ_E4M3;
    const float s = scale_value(x.s);
    float v[8];
    decode4<F>(x.v.x, s, v);
    decode4<F>(x.v.y, s, v + 4);
#pragma unroll
    for (int i = 0; i < 4; i++) o.v[0][i] = (int)pair_bf16(v[2 * i], v[2 * i + 1]);
  } else {
    o.v[0] = x.v;
  }
  return o;
}

struct Int4Args {
  const void* x;
  const uint8_t* xs;       // a checkpoint's scales
  const uint8_t* w;
  const uint16_t *s, *z;
  void* y;
  int64_t m, n, k, ldx, ldy;
  int out, turns;          // y's type; times that the contraction runs through W (the parts of binary32 x, one after another)
};

// Eight codes of W as 16 + u in the operand's type: j = 0..3 picks nibbles j and j + 4.
template <int SRC>
__device__ __forceinline__ v4i widen_codes(uint32_t w) {
  v4i o;
  if constexpr (SRC == LQ_F16) {   // binary16: exponent of 16, a step of 2^-6
    o[0] = (int)((w << 6 & 0x03C003C0u) | 0x4C004C00u);
    o[1] = (int)((w << 2 & 0x03C003C0u) | 0x4C004C00u);
    o[2] = (int)((w >> 2 & 0x03C003C0u) | 0x4C004C00u);
    o[3] = (int)((w >> 6 & 0x03C003C0u) | 0x4C004C00u);
  } else {   // bfloat16: a step of 2^-3
    o[0] = (int)((w << 3 & 0x00780078u) | 0x41804180u);
    o[1] = (int)((w >> 1 & 0x00780078u) | 0x41804180u);
    o[2] = (int)((w >> 5 & 0x00780078u) | 0x41804180u);
    o[3] = (int)((w >> 9 & 0x00780078u) | 0x41804180u);
  }
  return o;
}
template <int SRC>
__device__ __forceinline__ v4f multiply(v4i a, v4i b, v4f c) {
  if constexpr (SRC == LQ_F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// ---------------------------------------------------------------- product
// Up to 16 CT rows of x, from 16 CT blockIdx.y on. Eight waves of a workgroup share 16 R
// rows of W, each taking a run of the contraction's steps; their sums meet in LDS. A
// wave's scales go to LDS first, kBank bytes of them at a time (in registers they would
// take as many as the codes, twice that with groups of 32).
constexpr int kBank = 8192;

template <int SRC, int R, int CT, int G>
__global__ __launch_bounds__(64 * kWaves) void k_int4(const Int4Args a) {
  constexpr int each = kStep / G, per = G / 32;   // groups of a step, products of a group
  constexpr int U = CT == 4 ? 1 : R * CT >= 2 ? 2 : 4;   // steps of W asked for at a time
  constexpr bool kept = SRC == kInt8 || SRC == kE4m3;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kWaves * kBank];
  static_assert(R * CT * 1024 <= kBank, "");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int64_t row0 = (int64_t)blockIdx.x * 16 * R, first = (int64_t)blockIdx.y * 16 * CT, np = padded_rows(a.n);
  const int steps = (int)steps_of(a.k), all = steps * a.turns, run = (all + kWaves - 1) / kWaves;
  const int begin = wave * run, end = begin + run < all ? begin + run : all;
  const int64_t spitch = ckpt_scale_pitch(a.k);
  uint8_t* const bank = lds + wave * kBank;

  // The scales, then the zero points, of steps t .. t + count - 1: of each group 16 R rows.
  constexpr int kGroup = 32 * R, kScales = each * kGroup;   // bytes of a group, of a step
  const int fits = kBank / (kScales * (a.z ? 2 : 1));
  auto step_of = [&](int t) { return a.turns > 1 ? t % steps : t; };
  auto bank_scales = [&](int t, int count) {
    const int units = count * kScales / 16, both = a.z ? 2 * units : units;
    for (int i = lane; i < both; i += 64) {
      const int u = i < units ? i : i - units, group = u * 16 / kGroup, at = u * 16 % kGroup / 2;
      const uint16_t* p = (i < units ? a.s : a.z) + ((int64_t)step_of(t + group / each) * each + group % each) * np + row0 + at;
      *(v4i*)(bank + i * 16) = *(const v4i*)p;
    }
    __builtin_amdgcn_wave_barrier();   // (LDS serves a wave's instructions in order)
  };

  struct Weights { v4i c[U][R]; };
  auto load_w = [&](Weights& b, int t) {
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int64_t g = step_of(t + u < all ? t + u : all - 1);
#pragma unroll
      for (int i = 0; i < R; i++) b.c[u][i] = *(const v4i*)(a.w + (g * np + row0 + i * 16 + r) * 64 + q * 16);
    }
  };
  struct Rows { X8<SRC> x[4][CT]; };
  auto load_x = [&](Rows& b, int t, int begin_i, int end_i) {
    const int turn = a.turns > 1 ? t / steps : 0, g = t - turn * steps;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int64_t col = (int64_t)g * kStep + i * 32 + q * 8;
#pragma unroll
      for (int c = 0; c < CT; c++) {
        if (i < begin_i || i >= end_i) continue;
        const int64_t row = first + c * 16 + r;
        X8<SRC> v = {};
        if (row < a.m && col < a.k) {
          if constexpr (kept) {
            v.v = *(const uint2*)((const uint8_t*)a.x + row * a.ldx + col);
            v.s = a.xs[row * spitch + col / 32];
          } else {
            __builtin_memcpy(&v, (const typename El<SRC>::T*)a.x + row * a.ldx + turn * a.k + col, sizeof(v));
          }
        }
        b.x[i][c] = v;
      }
    }
  };

  const v4f none = {0.0f, 0.0f, 0.0f, 0.0f};
  v4f y[R][CT];
#pragma unroll
  for (int i = 0; i < R; i++)
#pragma unroll
    for (int c = 0; c < CT; c++) y[i][c] = none;
  constexpr int one2 = SRC == LQ_F16 ? 0x3C003C00 : 0x3F803F80;
  const v4i ones = {one2, one2, one2, one2};

  Weights now, next;
  Rows here, ahead;
  if (begin < end) {
    bank_scales(begin, end - begin < fits ? end - begin : fits);
    load_x(here, begin, 0, CT < 4 ? 4 : 1);
    load_w(now, begin);
  }
  int banked = begin;   // the first step of the bank's
  for (int t = begin; t < end; t += U) {
    if (t + U < end) load_w(next, t + U);
#pragma unroll
    for (int u = 0; u < U; u++) {
      if (t + u >= end) break;
      if (t + u - banked == fits) {
        __builtin_amdgcn_wave_barrier();
        banked = t + u;
        bank_scales(banked, end - banked < fits ? end - banked : fits);
      }
      if (CT < 4 && t + u + 1 < end) load_x(ahead, t + u + 1, 0, 4);
      const uint8_t* const scales = bank + (t + u - banked) * kScales + q * 8;
      const int zeros = (end - banked < fits ? end - banked : fits) * kScales;
      v4f acc[R][CT], sum[CT];
#pragma unroll
      for (int i = 0; i < 4; i++) {
        // (a whole step of 64 rows does not fit in the registers)
        if (CT == 4 && (i < 3 || t + u + 1 < end)) load_x(here, t + u + (i + 1) / 4, (i + 1) % 4, (i + 1) % 4 + 1);
        Parts<SRC> x[CT];
#pragma unroll
        for (int c = 0; c < CT; c++) {
          x[c] = operands<SRC>(here.x[i][c]);
          if (i % per == 0) sum[c] = none;
#pragma unroll
          for (int p = 0; p < Parts<SRC>::n; p++) sum[c] = multiply<SRC>(ones, x[c].v[p], sum[c]);
        }
#pragma unroll
        for (int j = 0; j < R; j++) {
          const v4i w = widen_codes<SRC>((uint32_t)now.c[u][j][i]);
#pragma unroll
          for (int c = 0; c < CT; c++) {
            if (i % per == 0) acc[j][c] = none;
#pragma unroll
            for (int p = 0; p < Parts<SRC>::n; p++) acc[j][c] = multiply<SRC>(w, x[c].v[p], acc[j][c]);
          }
        }
        if (i % per == per - 1) {
          const int at = i / per * kGroup;
#pragma unroll
          for (int j = 0; j < R; j++) {
            uint16_t s[4], z[4];
            __builtin_memcpy(s, __builtin_assume_aligned(scales + at + j * 32, 8), 8);
            if (a.z) __builtin_memcpy(z, __builtin_assume_aligned(scales + zeros + at + j * 32, 8), 8);
#pragma unroll
            for (int e = 0; e < 4; e++) {
              const float scale = widen<LQ_F16>(s[e]), off = a.z ? 24.0f + widen<LQ_F16>(z[e]) : 24.0f;
#pragma unroll
              for (int c = 0; c < CT; c++)
                y[j][c][e] = __builtin_fmaf(scale, __builtin_fmaf(-off, sum[c][e], acc[j][c][e]), y[j][c][e]);
            }
          }
        }
      }
      if (CT < 4) here = ahead;
    }
    now = next;
  }
  // (a wave's bank is its own until here)
  v4f(*const sums)[R * CT][64] = (v4f(*)[R * CT][64])lds;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < R; i++)
#pragma unroll
    for (int c = 0; c < CT; c++) sums[wave][i * CT + c][lane] = y[i][c];
  __syncthreads();
  // A lane's four sums are columns 4q .. 4q + 3 of one row of y.
  for (int t = wave; t < R * CT; t += kWaves) {
    v4f s = sums[0][t][lane];
#pragma unroll
    for (int v = 1; v < kWaves; v++) s += sums[v][t][lane];
    const int64_t row = first + t % CT * 16 + r, col = row0 + t / CT * 16 + 4 * q;
    if (row >= a.m) continue;
#pragma unroll
    for (int e = 0; e < 4; e++)
      if (col + e < a.n) {
        const int64_t at = row * a.ldy + col + e;
        if (a.out == LQ_F32) ((float*)a.y)[at] = s[e];
        else ((uint16_t*)a.y)[at] = a.out == LQ_BF16 ? narrow<LQ_BF16>(s[e]) : narrow<LQ_F16>(s[e]);
      }
  }
}

// x as bfloat16 operands in rows of k elements, of binary32 three times k: what many
// workgroups would otherwise convert again, for more than 16 rows.
template <int SRC>
__global__ __launch_bounds__(256) void k_int4_rows(const void* x, const uint8_t* xs, int64_t m, int64_t k, int64_t ldx,
                                                   uint16_t* out) {
  constexpr bool kept = SRC == kInt8 || SRC == kE4m3;
  const int64_t col = ((int64_t)blockIdx.x * 64 + (threadIdx.x & 63)) * 8;
  if (col >= k) return;
  for (int64_t row = (int64_t)blockIdx.y * 4 + (threadIdx.x >> 6); row < m; row += (int64_t)gridDim.y * 4) {
    X8<SRC> v;
    if constexpr (kept) {
      v.v = *(const uint2*)((const uint8_t*)x + row * ldx + col);
      v.s = xs[row * ckpt_scale_pitch(k) + col / 32];
    } else {
      __builtin_memcpy(&v, (const float*)x + row * ldx + col, sizeof(v));
    }
    const Parts<SRC> o = operands<SRC>(v);
#pragma unroll
    for (int p = 0; p < Parts<SRC>::n; p++)
      *(v4i*)(out + (row * Parts<SRC>::n + p) * k + col) = o.v[p];
  }
}

template <int SRC, int R, int CT>
hipError_t product_of(const Int4Args& a, int group, hipStream_t s) {
  const dim3 grid((unsigned)((a.n + 16 * R - 1) / (16 * R)), (unsigned)((a.m + 16 * CT - 1) / (16 * CT)));
  if (group == 32) hipLaunchKernelGGL((k_int4<SRC, R, CT, 32>), grid, dim3(64 * kWaves), 0, s, a);
  else if (group == 64) hipLaunchKernelGGL((k_int4<SRC, R, CT, 64>), grid, dim3(64 * kWaves), 0, s, a);
  else hipLaunchKernelGGL((k_int4<SRC, R, CT, 128>), grid, dim3(64 * kWaves), 0, s, a);
  return hipGetLastError();
}
template <int SRC>
hipError_t few(const Int4Args& a, int group, hipStream_t s) {
  if (a.n >= 32 * (int64_t)compute_units()) return product_of<SRC, 2, 1>(a, group, s);
  return product_of<SRC, 1, 1>(a, group, s);
}
template <int SRC>
hipError_t many(const Int4Args& a, int group, hipStream_t s) {
  if (a.m <= 16) return few<SRC>(a, group, s);
  if (a.m > 32) return product_of<SRC, 1, 4>(a, group, s);
  if (a.n >= 32 * (int64_t)compute_units()) return product_of<SRC, 2, 2>(a, group, s);
  return product_of<SRC, 1, 2>(a, group, s);
}

}  // namespace

size_t int4_codes_bytes(int64_t n, int64_t k) { return (size_t)(steps_of(k) * padded_rows(n) * 64); }
size_t int4_scales_bytes(int64_t n, int64_t k, int group) { return (size_t)(steps_of(k) * (kStep / group) * padded_rows(n) * 2); }

// The rows that a call converts into its workspace.
size_t int4_rows_bytes(const lq_int4_desc* d) {
  const bool kept = d->x_format == LQ_INT8 || d->x_format == LQ_E4M3;
  if (d->m <= 16 || (!kept && d->in_dtype != LQ_F32)) return 0;
  return (size_t)(d->m * d->k * (kept ? 1 : 3) * 2);
}

hipError_t launch_int4_pack(const lq_int4_desc* d, const void* codes, const void* scales, const void* zeros, void* packed,
                            hipStream_t s) {
  uint8_t* const out = (uint8_t*)packed;
  uint16_t* const to = (uint16_t*)(out + int4_codes_bytes(d->n, d->k));
  uint16_t* const z = (uint16_t*)((uint8_t*)to + int4_scales_bytes(d->n, d->k, d->group));
  const int64_t bands = (steps_of(d->k) + 3) / 4;
  const dim3 grid((unsigned)((padded_rows(d->n) + 3) / 4), (unsigned)(bands < 65535 ? bands : 65535));
  hipLaunchKernelGGL(k_int4_pack, grid, dim3(256), 0, s, (const uint8_t*)codes, (const uint16_t*)scales,
                     (const uint16_t*)zeros, d->n, d->k, d->group, out, to, z);
  return hipGetLastError();
}

hipError_t launch_int4_linear(const lq_int4_desc* d, const void* x, const void* x_scales, const void* packed, void* y,
                              void* ws, hipStream_t s) {
  if (d->k == 0) return launch_constant(d->m, d->n, d->out_dtype, nullptr, y, d->ld_out, s);
  Int4Args a = {};
  a.x = x;
  a.xs = (const uint8_t*)x_scales;
  a.w = (const uint8_t*)packed;
  a.s = (const uint16_t*)(a.w + int4_codes_bytes(d->n, d->k));
  a.z = d->zero_points ? (const uint16_t*)((const uint8_t*)a.s + int4_scales_bytes(d->n, d->k, d->group)) : nullptr;
  a.y = y;
  a.m = d->m;
  a.n = d->n;
  a.k = d->k;
  a.ldx = d->ld_in;
  a.ldy = d->ld_out;
  a.out = d->out_dtype;
  a.turns = 1;
  const int src = d->x_format == LQ_INT8 ? kInt8 : d->x_format == LQ_E4M3 ? kE4m3 : d->in_dtype;
  if (src >= kInt8) a.ldx = ckpt_pitch(d->k);
  if (int4_rows_bytes(d) > 0) {
    const dim3 g = matrix_grid((d->k + 511) / 512, d->m);
    if (src == LQ_F32) hipLaunchKernelGGL((k_int4_rows<LQ_F32>), g, dim3(256), 0, s, x, a.xs, d->m, d->k, a.ldx, (uint16_t*)ws);
    else if (src == kInt8) hipLaunchKernelGGL((k_int4_rows<kInt8>), g, dim3(256), 0, s, x, a.xs, d->m, d->k, a.ldx, (uint16_t*)ws);
    else hipLaunchKernelGGL((k_int4_rows<kE4m3>), g, dim3(256), 0, s, x, a.xs, d->m, d->k, a.ldx, (uint16_t*)ws);
    if (hipGetLastError() != hipSuccess) return hipErrorLaunchFailure;
    a.turns = src == LQ_F32 ? 3 : 1;
    a.x = ws;
    a.ldx = d->k * a.turns;
    return many<LQ_BF16>(a, d->group, s);
  }
  switch (src) {
    case LQ_F32: return few<LQ_F32>(a, d->group, s);
    case LQ_BF16: return many<LQ_BF16>(a, d->group, s);
    case LQ_F16: return many<LQ_F16>(a, d->group, s);
    case kInt8: return few<kInt8>(a, d->group, s);
    default: return few<kE4m3>(a, d->group, s);
  }
}

}  // namespace lql
