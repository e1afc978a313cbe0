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
// What is added up and taken off is up to 31 |x| of every element, whatever is left of it, so
// the sums' rounding goes with the row's sum of s |x|, and not with |x| |w|: at most 11
// 2^-24 of that sum, 1e-7 to 1.5e-6 of y's root mean square, on normal activations with
// some channels 20 times as loud (300 rows of W, k of 1024 to 40960, groups of 32 to 128);
// 10 to 160 2^-24 of it, up to 1e-4 of y's, where channels are 1000 times as loud and their
// codes are the zero point, so that nothing at all is left of them.
#include "lq_linear.h"

namespace lql {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

constexpr int kStep = 128;   // of the contraction: 64 bytes of a row of W
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
  } else if constexpr (SRC == kInt8) {   // (exact: the upper half of the binary32 product)
    const float s = scale_value(x.s);
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const uint32_t w = i < 2 ? x.v.x : x.v.y;
      const float a = (float)(int8_t)(w >> (i % 2 * 16)) * s, b = (float)(int8_t)(w >> (i % 2 * 16 + 8)) * s;
      o.v[0][i] = (int)__builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
    }
  } else if constexpr (SRC == kE4m3) {
    const float s = scale_value(x.s);
    o.v[0][0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)x.v.x, s, false));
    o.v[0][1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)x.v.x, s, true));
    o.v[0][2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)x.v.y, s, false));
    o.v[0][3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)x.v.y, s, true));
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
  int place_bits;          // of a staged row: log2 of its units of eight elements, rounded up
  int out, turns;          // y's type; times that the contraction runs through W (the parts of binary32 x, one after another)
};

// What the matrix cores multiply by, 16 + u and one, is held times a power of two where x
// has binary32's range: a group's (16 + u) x, and (24 + z) times its sum of x, are up to
// 2^12 times an element (2^14.3 for zero points of 128), and 2^120 of that would be an
// infinity. The scale, times 2^8, makes up for it; every step is exact.
template <int SRC> struct Held { static constexpr float up = 256.0f, down = 1.0f / up; };
template <> struct Held<LQ_F16> { static constexpr float up = 1.0f, down = 1.0f; };   // (x up to 65504)

// Eight codes of W as 16 + u in the operand's type, times Held's 2^-8: j = 0..3 picks nibbles j and j + 4.
// binary16: exponent of 16, a step of 2^-6; bfloat16: of 2^-4, a step of 2^-3 times 2^-8. (The two constants
// are in registers of either kind: an instruction takes one from a scalar one, and no
// literal besides.)
template <int SRC>
struct Widen {
  uint32_t mask, magic;
  __device__ __forceinline__ Widen() : mask(SRC == LQ_F16 ? 0x03C003C0u : 0x00780078u), magic(SRC == LQ_F16 ? 0x4C004C00u : 0x3D803D80u) {
    asm volatile("" : "+s"(mask));
    asm volatile("" : "+v"(magic));
  }
  __device__ __forceinline__ v4i operator()(uint32_t w) const {
    constexpr bool f16 = SRC == LQ_F16;
    v4i o;
    o[0] = (int)(((f16 ? w << 6 : w << 3) & mask) | magic);
    o[1] = (int)(((f16 ? w << 2 : w >> 1) & mask) | magic);
    o[2] = (int)(((f16 ? w >> 2 : w >> 5) & mask) | magic);
    o[3] = (int)(((f16 ? w >> 6 : w >> 9) & mask) | magic);
    return o;
  }
};
template <int SRC>
__device__ __forceinline__ v4f multiply(v4i a, v4i b, v4f c) {
  if constexpr (SRC == LQ_F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// ---------------------------------------------------------------- product
// Up to 16 CT rows of x, from 16 CT blockIdx.y on. The waves of a workgroup share 16
// rows of W, each taking a run of the contraction's steps; their sums meet in LDS.
// STAGED: x fits in LDS as operands, which the workgroup makes of it while its first
// reads of W are on their way. Otherwise a launch before has laid x out as operands, and
// every wave reads its run of them beside its run of W, as many steps ahead, each part
// into the registers that a product has just emptied. (Loads return in the order in
// which they were asked for: a wait for x asked for late would be one for all of W asked
// for before.)
// A wave's scales and offsets 24 + z go through LDS as binary32, a page of as many steps'
// as fit in its bank, and the next page is on its way meanwhile: converted there, each
// is converted once instead of by the sixteen lanes that multiply by it.
// Measured, W in memory, within a graph: one row of 11008 x 4096 9.5 us, 16 rows of 4096 x
// 11008 from an 8-bit checkpoint 15.4 us (11.9 with W in the last-level cache), 64 rows of
// 4096 x 4096 15 us, 8 rows of 16384 x 16384 55 us. One row reads W at 2.5 TB/s, which its
// start and end bound (the large W streams no faster for eight rows: there the sums of a
// step's groups and the widening of its codes do); many rows are bound by x's operands,
// which every workgroup reads from the caches: 64 rows of 11008 x 4096 33.8 us.
constexpr int kBank = 4096;          // bytes of a wave's scales
constexpr int kStaged = 131072;      // of x, beside eight waves' banks all of a compute unit's LDS
constexpr int kStagedTwice = 65536;  // beside four waves', half of it

// Bytes from row to row of the staged x: four rows' 64 bytes lie in different banks.
__host__ __device__ inline int64_t staged_pitch(int64_t k) { return (k * 2 + 255) / 256 * 256 + 64; }

template <int SRC, int CT, int G, bool STAGED, int kWaves>
__global__ __launch_bounds__(64 * kWaves, STAGED ? 4 : 2) void k_int4(const Int4Args a) {
  constexpr int each = kStep / G, per = G / 32;         // groups of a step, products of a group
  constexpr int D = STAGED || CT == 1 ? 4 : 2;          // steps asked for ahead, or twice that where x is staged
  constexpr bool kept = SRC == kInt8 || SRC == kE4m3;
  constexpr int parts = Parts<SRC>::n;
  extern __shared__ __attribute__((aligned(128))) uint8_t lds[];   // product_of()'s bytes
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int64_t row0 = (int64_t)blockIdx.x * 16, first = (int64_t)blockIdx.y * 16 * CT, np = padded_rows(a.n);
  const int steps = (int)steps_of(a.k), all = steps * a.turns, run = (all + kWaves - 1) / kWaves;
  const int begin = wave * run, end = begin + run < all ? begin + run : all;
  const int rows = a.m - first < 16 * CT ? (int)(a.m - first) : 16 * CT;
  uint8_t *const bank = lds + wave * kBank, *const xlds = lds + kWaves * kBank;
  auto step_of = [&](int t) {   // of W (selects: a branch or a division costs more), for steps up to the wave's last
    t = t < all ? t : all - 1;
    t = t >= steps ? t - steps : t;
    return t >= steps ? t - steps : t;
  };

  // The scales, then the offsets, of steps t .. t + count - 1: of each group 16 rows. The loop below takes D
  // steps without a branch between them; those past the wave's last multiply its last by scales of zero.
  constexpr int kGroup = 64, kScales = each * kGroup, kUnits = kBank / 2 / 16 / 64;   // bytes of a group, of a step
  constexpr int fits = kBank / (kScales * 2);
  static_assert(fits % (2 * D) == 0 && kUnits * 64 == fits * kScales / 16, "");
  struct Bank { v4i v[kUnits]; };
  auto load_bank = [&](Bank& b, int t, int count) {
    const int units = count * kScales / 32, both = 2 * units;   // of eight in memory
#pragma unroll
    for (int k = 0; k < kUnits; k++) {
      const int i = k * 64 + lane, u = i < units ? i : i - units, group = u * 32 / kGroup, at = u * 32 % kGroup / 4;
      b.v[k] = v4i{0, 0, 0, 0};
      if (i < (a.z ? both : units) && t + group / each < end)
        b.v[k] = *(const v4i*)((i < units ? a.s : a.z) + ((int64_t)step_of(t + group / each) * each + group % each) * np + row0 + at);
    }
  };
  auto keep_bank = [&](const Bank& b, int count) {
    const int units = count * kScales / 32, both = 2 * units;
    __builtin_amdgcn_wave_barrier();   // (LDS serves a wave's instructions in order)
#pragma unroll
    for (int k = 0; k < kUnits; k++) {
      const int i = k * 64 + lane;
      if (i < both) {
        const float more = i < units ? 0.0f : 24.0f, times = i < units ? Held<SRC>::up : 1.0f;
        uint16_t h[8];
        __builtin_memcpy(h, &b.v[k], 16);
#pragma unroll
        for (int f = 0; f < 2; f++) {
          v4f v;
#pragma unroll
          for (int e = 0; e < 4; e++) v[e] = __builtin_fmaf(widen<LQ_F16>(h[4 * f + e]), times, more);
          *(v4f*)(bank + i * 32 + f * 16) = v;
        }
      }
    }
    __builtin_amdgcn_wave_barrier();
  };

  struct Weights { v4i w[D]; };
  // The step of x that comes next, likewise (see below): 4 CT operands of a kilobyte, in the order of k_int4_rows().
  struct Rows { v4i x[4][CT]; };
  int xt = begin;
  const uint8_t* const x0 = (const uint8_t*)a.x + (int64_t)blockIdx.y * all * (CT * 4096);
  __amdgpu_buffer_rsrc_t rows_of_step;
  auto load_x = [&](Rows& b, int i) {
    if (i == 0) {
      rows_of_step = __builtin_amdgcn_make_buffer_rsrc((void*)(x0 + (int64_t)(xt < all ? xt : all - 1) * (CT * 4096)), 0, xt < end ? CT * 4096 : 0, 0x00020000);
      xt++;
    }
#pragma unroll
    for (int c = 0; c < CT; c++)
      b.x[i][c] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rows_of_step, lane * 16, (i * CT + c) * 1024, 0));
  };
  // The step of W that comes next; past the wave's last, zeros that are not read. (By its stretch, and asked for without a
  // branch: with an address in vector registers, or loads that some paths lack, the compiler waits for all that is on its
  // way where it need not.)
  const uint32_t wo = (uint32_t)r * 64 + q * 16;
  const int64_t wstep = np * 64;
  int wt = begin;
  const uint8_t* const w0 = a.w + row0 * 64;
  auto load_w = [&](v4i& w) {
    const auto stretch = __builtin_amdgcn_make_buffer_rsrc((void*)(w0 + step_of(wt) * wstep), 0, wt < end ? 1024 : 0, 0x00020000);
    w = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(stretch, (int)wo, 0, 0));
    wt++;
  };
  auto load = [&](Weights& b) {
#pragma unroll
    for (int u = 0; u < D; u++) load_w(b.w[u]);
  };

  const v4f none = {0.0f, 0.0f, 0.0f, 0.0f};
  v4f y[CT];
#pragma unroll
  for (int c = 0; c < CT; c++) y[c] = none;
  constexpr int one2 = SRC == LQ_F16 ? 0x3C003C00 : 0x3B803B80;   // (bfloat16: 2^-8, as the codes)
  static_assert(Held<SRC>::down == (SRC == LQ_F16 ? 1.0f : 0x1p-8f), "the constants here and in Widen");
  const v4i ones = {one2, one2, one2, one2};
  const uint8_t* const xrow = xlds + (r < rows ? r : 0) * staged_pitch(a.k) + q * 16;
  const int64_t plane = rows * staged_pitch(a.k);
  const Widen<SRC> widen;
  int banked = begin;   // the first step of the bank's
  constexpr int kSet = STAGED ? 2 * D : D;   // steps of the loop's body
  auto count_from = [&](int t) { return end - t < fits ? (end - t + kSet - 1) / kSet * kSet : fits; };
  // Step t; x of step t + D takes the place of each part of this one's.
  auto multiply_step = [&](const v4i& codes, Rows& rows_, int t) {
    const uint8_t* const scales = bank + (t - banked) * kScales + q * 16;
    const int offsets = count_from(banked) * kScales;   // (after the page's scales)
    asm volatile("" ::: "memory");   // (left alone, the compiler reads what several steps take from LDS before the first, and spills)
    __builtin_amdgcn_sched_barrier(0);
    v4f scale[each], off[each];
    auto read_scales = [&](int g) {
      scale[g] = *(const v4f*)(scales + g * kGroup);
      off[g] = *(const v4f*)(scales + offsets + g * kGroup);
    };
    constexpr bool early = CT < 3 && each < 4;   // (of four groups a step, they would take too many registers)
    if (early) {
#pragma unroll
      for (int g = 0; g < each; g++) read_scales(g);
    }
    v4f acc[CT], sum[CT];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      if (!early && i % per == 0) read_scales(i / per);
      Parts<SRC> x[CT];
#pragma unroll
      for (int c = 0; c < CT; c++) {
        if constexpr (STAGED) {
#pragma unroll
          for (int p = 0; p < parts; p++) x[c].v[p] = *(const v4i*)(xrow + p * plane + (t < end ? t : end - 1) * (kStep * 2) + i * 64);
        } else {
          x[c].v[0] = rows_.x[i][c];
        }
        if (i % per == 0) sum[c] = none;
#pragma unroll
        for (int p = 0; p < parts; p++) sum[c] = multiply<SRC>(ones, x[c].v[p], sum[c]);
      }
      const v4i w = widen((uint32_t)codes[i]);
#pragma unroll
      for (int c = 0; c < CT; c++) {
        if (i % per == 0) acc[c] = none;
#pragma unroll
        for (int p = 0; p < parts; p++) acc[c] = multiply<SRC>(w, x[c].v[p], acc[c]);
      }
      if (!STAGED) load_x(rows_, i);
      if (i % per == per - 1) {
#pragma unroll
        for (int e = 0; e < 4; e++)
#pragma unroll
          for (int c = 0; c < CT; c++)
            y[c][e] = __builtin_fmaf(scale[i / per][e], __builtin_fmaf(-off[i / per][e], sum[c][e], acc[c][e]), y[c][e]);
        // (left alone, the compiler has the sums of all of the step's groups in registers at a time)
        if (!early) __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  Bank coming;
  // Loads return in the order in which they are asked for: first what is waited for first.
  Weights even, odd;
  Rows x[STAGED ? 1 : D];
  if constexpr (STAGED) {
    // units of eight elements, two of a thread's ahead of W; a row's take a power of two of places
    const int units = steps * (kStep / 8), total = rows << a.place_bits;
    auto unit = [&](int i) {
      const int row = i >> a.place_bits, col = (i & ((1 << a.place_bits) - 1)) * 8;
      X8<SRC> v = {};
      if (col < a.k) {
        if constexpr (kept) {
          v.v = *(const uint2*)((const uint8_t*)a.x + row * a.ldx + col);
          v.s = a.xs[row * ckpt_scale_pitch(a.k) + col / 32];
        } else {
          constexpr int size = El<kept ? LQ_F32 : SRC>::bytes;
          __builtin_memcpy(&v, (const uint8_t*)a.x + (row * a.ldx + col) * size, sizeof(v));
        }
      }
      return v;
    };
    auto stage = [&](int i, const X8<SRC>& v) {
      const int row = i >> a.place_bits, col = i & ((1 << a.place_bits) - 1);
      if (col >= units) return;
      const Parts<SRC> o = operands<SRC>(v);
#pragma unroll
      for (int p = 0; p < parts; p++) *(v4i*)(xlds + row * staged_pitch(a.k) + p * plane + col * 16) = o.v[p];
    };
    constexpr int kThreads = 64 * kWaves;
    int i = threadIdx.x;
    X8<SRC> mine = {}, second = {};
    if (i < total) mine = unit(i);
    if (i + kThreads < total) second = unit(i + kThreads);
    asm volatile("" ::: "memory");
    if (begin < end) {
      load_bank(coming, begin, count_from(begin));
      load(even);
    }
    asm volatile("" ::: "memory");
    if (i < total) stage(i, mine);
    if (i + kThreads < total) stage(i + kThreads, second);
    for (i += 2 * kThreads; i < total; i += 2 * kThreads) {
      mine = unit(i);
      if (i + kThreads < total) second = unit(i + kThreads);
      stage(i, mine);
      if (i + kThreads < total) stage(i + kThreads, second);
    }
    __syncthreads();
  } else if (begin < end) {
    load_bank(coming, begin, count_from(begin));
#pragma unroll
    for (int u = 0; u < D; u++) {
#pragma unroll
      for (int i = 0; i < 4; i++) load_x(x[u], i);
      load_w(even.w[u]);
    }
  }
  if (begin < end) keep_bank(coming, count_from(begin));
  while (banked < end) {   // pages of scales
    if (banked + fits < end) load_bank(coming, banked + fits, count_from(banked + fits));
    const int stop = banked + fits < end ? banked + fits : end;
    if constexpr (STAGED) {
      for (int t = banked; t < stop; t += 2 * D) {
        load(odd);
#pragma unroll
        for (int u = 0; u < D; u++) multiply_step(even.w[u], x[0], t + u);
        load(even);
        if (t + D < stop) {
#pragma unroll
          for (int u = 0; u < D; u++) multiply_step(odd.w[u], x[0], t + D + u);
        }
      }
    } else {
      for (int t = banked; t < stop; t += D) {
#pragma unroll
        for (int u = 0; u < D; u++) {
          multiply_step(even.w[u], x[u], t + u);
          load_w(even.w[u]);
        }
      }
    }
    banked += fits;
    if (banked < end) keep_bank(coming, count_from(banked));
  }
  // (a wave's bank is its own until here)
  v4f(*const sums)[CT][64] = (v4f(*)[CT][64])lds;
  __syncthreads();
#pragma unroll
  for (int c = 0; c < CT; c++) sums[wave][c][lane] = y[c];
  __syncthreads();
  // A lane's four sums are columns 4q .. 4q + 3 of one row of y.
  if (wave >= CT) return;
  v4f s = sums[0][wave][lane];
#pragma unroll
  for (int v = 1; v < kWaves; v++) s += sums[v][wave][lane];
  const int64_t row = first + wave * 16 + r, col = row0 + 4 * q;
  if (row >= a.m) return;
#pragma unroll
  for (int e = 0; e < 4; e++)
    if (col + e < a.n) {
      const int64_t at = row * a.ldy + col + e;
      if (a.out == LQ_F32) ((float*)a.y)[at] = s[e];
      else ((uint16_t*)a.y)[at] = a.out == LQ_BF16 ? narrow<LQ_BF16>(s[e]) : narrow<LQ_F16>(s[e]);
    }
}

// x as operands: bands of 16 CT rows, of each band its steps (of binary32 first all of
// the first parts', then the second's and the third's), of a step four products, of a
// product CT times 16 rows x 4 units of eight elements; zeros past the last row and
// column. One unit a thread.
template <int SRC>
__global__ __launch_bounds__(256) void k_int4_rows(const void* x, const uint8_t* xs, int64_t m, int64_t k, int64_t ldx,
                                                   int ct, uint8_t* out) {
  constexpr bool kept = SRC == kInt8 || SRC == kE4m3;
  constexpr int parts = Parts<SRC>::n;
  const int64_t steps = steps_of(k), unit = (int64_t)blockIdx.x * 256 + threadIdx.x;   // of a row, padded
  if (unit >= steps * 16) return;
  const int64_t step = unit >> 4, col = unit * 8;
  const int i = (int)(unit >> 2 & 3), q = (int)(unit & 3);
  const int64_t bands = (m + 16 * ct - 1) / (16 * ct);
  for (int64_t row = blockIdx.y; row < bands * 16 * ct; row += gridDim.y) {
    X8<SRC> v = {};
    if (row < m && col < k) {
      if constexpr (kept) {
        v.v = *(const uint2*)((const uint8_t*)x + row * ldx + col);
        v.s = xs[row * ckpt_scale_pitch(k) + col / 32];
      } else {
        constexpr int size = El<kept ? LQ_F32 : SRC>::bytes;
        __builtin_memcpy(&v, (const uint8_t*)x + (row * ldx + col) * size, sizeof(v));
      }
    }
    const Parts<SRC> o = operands<SRC>(v);
    const int64_t band = row / (16 * ct);
    const int in = (int)(row - band * 16 * ct);
#pragma unroll
    for (int p = 0; p < parts; p++)
      *(v4i*)(out + (((band * parts + p) * steps + step) * 4 + i) * (ct * 1024) + (in >> 4) * 1024 + (q * 16 + (in & 15)) * 16) = o.v[p];
  }
}

template <int SRC, int CT, bool STAGED, int kWaves>
hipError_t product_of(Int4Args a, int group, hipStream_t s) {
  const dim3 grid((unsigned)((a.n + 15) / 16), (unsigned)((a.m + 16 * CT - 1) / (16 * CT)));
  const int64_t x = STAGED ? a.m * staged_pitch(a.k) * Parts<SRC>::n : 0;
  const unsigned lds = (unsigned)(kWaves * kBank + x);
  static_assert(kWaves * kBank >= CT * 1024 * kWaves, "the waves' sums lie there in the end");
  while ((1 << a.place_bits) < steps_of(a.k) * (kStep / 8) && a.place_bits < 20) a.place_bits++;
  constexpr int least = CT == 4 ? 64 : 32;   // (many()'s rule)
  if (group == least) hipLaunchKernelGGL((k_int4<SRC, CT, least, STAGED, kWaves>), grid, dim3(64 * kWaves), lds, s, a);
  else if (group == 64) hipLaunchKernelGGL((k_int4<SRC, CT, 64, STAGED, kWaves>), grid, dim3(64 * kWaves), lds, s, a);
  else hipLaunchKernelGGL((k_int4<SRC, CT, 128, STAGED, kWaves>), grid, dim3(64 * kWaves), lds, s, a);
  return hipGetLastError();
}
// Whether x is staged: what it takes beside the eight waves' banks.
inline bool staged(int64_t m, int64_t k, int parts) { return m <= 16 && m * staged_pitch(k) * parts <= kStaged; }
template <int SRC>
hipError_t few(const Int4Args& a, int group, hipStream_t s) {
  // Four waves where that leaves two workgroups or more for a compute unit, else eight: one row of 11008 x 4096 9.5 us by
  // four and 12.7 by eight, of 4096 x 11008 12.2 by four and 10.6 by eight, of 4096 x 4096 6.3 and 6.4.
  if (a.n >= 32 * (int64_t)compute_units() && a.m * staged_pitch(a.k) * Parts<SRC>::n <= kStagedTwice)
    return product_of<SRC, 1, true, 4>(a, group, s);
  return product_of<SRC, 1, true, 8>(a, group, s);
}
// Tiles of 16 rows that a workgroup takes of operands in memory. (64 rows' sums for four groups a step, of 32, do not fit
// in the registers.)
inline int row_tiles(int64_t m, int group) { return m <= 16 ? 1 : m <= 32 || (m > 48 && group == 32) ? 2 : m <= 48 ? 3 : 4; }
template <int SRC>
hipError_t many(const Int4Args& a, int group, hipStream_t s) {
  switch (row_tiles(a.m, group)) {
    case 1: return product_of<SRC, 1, false, 8>(a, group, s);
    case 2: return product_of<SRC, 2, false, 8>(a, group, s);
    case 3: return product_of<SRC, 3, false, 8>(a, group, s);
    default: return product_of<SRC, 4, false, 8>(a, group, s);
  }
}
template <int SRC>
hipError_t rows_as_operands(const lq_int4_desc* d, const void* x, const void* xs, int64_t ldx, void* ws, hipStream_t s) {
  const int ct = row_tiles(d->m, d->group);
  const int64_t rows = (d->m + 16 * ct - 1) / (16 * ct) * (16 * ct);
  const dim3 g((unsigned)((steps_of(d->k) * 16 + 255) / 256), (unsigned)(rows < 65535 ? rows : 65535));
  hipLaunchKernelGGL((k_int4_rows<SRC>), g, dim3(256), 0, s, x, (const uint8_t*)xs, d->m, d->k, ldx, ct, (uint8_t*)ws);
  return hipGetLastError();
}

}  // namespace

size_t int4_codes_bytes(int64_t n, int64_t k) { return (size_t)(steps_of(k) * padded_rows(n) * 64); }
size_t int4_scales_bytes(int64_t n, int64_t k, int group) { return (size_t)(steps_of(k) * (kStep / group) * padded_rows(n) * 2); }

// The operands that a call lays out in its workspace.
size_t int4_rows_bytes(const lq_int4_desc* d) {
  const int parts = d->x_format == -1 && d->in_dtype == LQ_F32 ? 3 : 1;
  if (staged(d->m, d->k, parts)) return 0;
  const int64_t band = 16 * row_tiles(d->m, d->group);
  return (size_t)((d->m + band - 1) / band * band * steps_of(d->k) * kStep * 2 * parts);
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
  if (int4_rows_bytes(d) == 0) switch (src) {
    case LQ_F32: return few<LQ_F32>(a, d->group, s);
    case LQ_BF16: return few<LQ_BF16>(a, d->group, s);
    case LQ_F16: return few<LQ_F16>(a, d->group, s);
    case kInt8: return few<kInt8>(a, d->group, s);
    default: return few<kE4m3>(a, d->group, s);
  }
  hipError_t e;
  switch (src) {
    case LQ_F32: e = rows_as_operands<LQ_F32>(d, x, x_scales, a.ldx, ws, s); break;
    case LQ_BF16: e = rows_as_operands<LQ_BF16>(d, x, x_scales, a.ldx, ws, s); break;
    case LQ_F16: e = rows_as_operands<LQ_F16>(d, x, x_scales, a.ldx, ws, s); break;
    case kInt8: e = rows_as_operands<kInt8>(d, x, x_scales, a.ldx, ws, s); break;
    default: e = rows_as_operands<kE4m3>(d, x, x_scales, a.ldx, ws, s); break;
  }
  if (e != hipSuccess) return e;
  a.turns = src == LQ_F32 ? 3 : 1;
  a.x = ws;
  return src == LQ_F16 ? many<LQ_F16>(a, d->group, s) : many<LQ_BF16>(a, d->group, s);
}

}  // namespace lql
