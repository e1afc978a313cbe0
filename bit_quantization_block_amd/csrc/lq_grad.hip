// lq_grad.hip — the linear layer's gradients: dx = dy W from the 4-bit weights,
// dw = dw0 + dy^T x8 from the 8-bit checkpoint of x.
#include "lq_linear.h"

namespace lql {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));

// Both gradients are matrix products A B over bfloat16 operands: E2M1 and INT8
// values times a power of two have at most 7 significant bits, E4M3 values 4,
// so the stored operand is exact in bfloat16 (8 bits; its exponents are
// binary32's) and is converted once, on its way into LDS.
//   dgrad: A = dy [m, n], B = W [n, k]; the contraction runs along dy's rows
//          and down W's columns
//   wgrad: A = dy^T, B = x8 [m, k]; it runs down the columns of both
// An operand whose contraction runs down the columns lies in LDS as it lies in
// memory and is read with ds_read_b64_tr_b16, which hands each lane of a group
// of 16 four rows of one column: two of them are the eight consecutive
// contraction values that a lane of v_mfma_f32_32x32x16_bf16 takes.
//
// A workgroup of 2 x 2 waves makes a (64 FM) x (64 FN) tile, 64 of the
// contraction a step. LDS holds two steps; the step after the next is on its way
// in registers. Each step's loads, conversions, LDS writes and reads go between
// its products, a few instructions at a time, so that the matrix cores are
// never without work; one barrier a step.
enum Kind { kDgrad, kWgrad };
constexpr int kStep = 64;

template <int KIND, int FM, int FN>
struct GradLds {
  // dgrad's dy: 128 bytes a row, its 16-byte units in the order u ^ (row / 2 & 7) (16 lanes at a time read 16
  // different units of 256 bytes)
  static constexpr int kRowA = KIND == kDgrad ? 2 * kStep : 128 * FM + 64, kRowsA = KIND == kDgrad ? 64 * FM : kStep;
  // columns: four rows that a transposing read takes at a time start 64 bytes apart in the banks
  static constexpr int kRowB = 128 * FN + 64;
  __attribute__((aligned(128))) uint8_t a[2][kRowsA * kRowA];
  __attribute__((aligned(128))) uint8_t b[2][kStep * kRowB];
};

// A stretch of memory for buffer loads: what lies past its end reads as zero.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t stretch(const void* p, int64_t bytes) {
  const uint64_t b = (uint64_t)(uintptr_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)b), hi = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32));
  void* q = (void*)(uintptr_t)((uint64_t)hi << 32 | lo);
  return __builtin_amdgcn_make_buffer_rsrc(q, 0, __builtin_amdgcn_readfirstlane((uint32_t)(bytes > 0 ? bytes : 0)), 0x00020000);
}
__device__ __forceinline__ v4i load16(__amdgpu_buffer_rsrc_t s, uint32_t offset) {
  return __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(s, (int)offset, 0, 0));
}
__device__ __forceinline__ uint32_t load1(__amdgpu_buffer_rsrc_t s, uint32_t offset) {
  return (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(s, (int)offset, 0, 0);
}
__device__ __forceinline__ v4s read_columns(const uint8_t* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)p);
}

// Eight E2M1 codes times their scale as bfloat16.
__device__ __forceinline__ v4i widen_e2m1(uint32_t w, float s) {
  v4i o;
  o[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
  o[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
  o[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
  o[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
  return o;
}
// Four 8-bit codes times their scale. INT8: code + 128 is an unsigned byte, so
// one conversion and one fused multiply-add give the exact binary32 value,
// whose upper half is the bfloat16.
template <int F>
__device__ __forceinline__ uint2 widen_8(uint32_t w, float s) {
  uint2 o;
  if constexpr (F == LQ_INT8) {
    const uint32_t u = w ^ 0x80808080u;
    const float off = -128.0f * s;
    const uint32_t a = __float_as_uint(__builtin_fmaf((float)(u & 0xFFu), s, off));
    const uint32_t b = __float_as_uint(__builtin_fmaf((float)(u >> 8 & 0xFFu), s, off));
    const uint32_t c = __float_as_uint(__builtin_fmaf((float)(u >> 16 & 0xFFu), s, off));
    const uint32_t d = __float_as_uint(__builtin_fmaf((float)(u >> 24), s, off));
    o.x = __builtin_amdgcn_perm(b, a, 0x07060302u);
    o.y = __builtin_amdgcn_perm(d, c, 0x07060302u);
  } else {
    o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, s, false));
    o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, s, true));
  }
  return o;
}

struct GradArgs {
  const uint16_t* dy;
  int64_t m, n, k, lddy;
  int64_t row;             // elements of a row of dy that may be read: n, or n padded; a multiple of 8
  const uint8_t *b, *bs;   // W's codes and scales, or the checkpoint's
  const float* in;         // dw_in
  void* out;
  int64_t ldo;
  uint32_t tm, tn;
};

// F: the checkpoint's format (wgrad); OUT: the result's type.
template <int KIND, int F, int OUT, int FM, int FN>
__global__ __launch_bounds__(256, FM * FN >= 16 ? 1 : 2) void k_grad(const GradArgs g) {
  typedef typename El<OUT>::T T;
  typedef GradLds<KIND, FM, FN> Lds;
  constexpr int BM = 64 * FM, BN = 64 * FN;
  __shared__ Lds lds;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 31, h = lane >> 5, wm = wave >> 1, wn = wave & 1;

  // The XCD's share of the tiles is a contiguous run in bands of 4 rows of tiles (as in the 4-bit product).
  const uint32_t total = g.tm * g.tn, xcd = blockIdx.x % 8, per8 = total / 8, more = total % 8;
  const uint32_t t0 = xcd * per8 + (xcd < more ? xcd : more) + blockIdx.x / 8;
  const uint32_t band = t0 / (4 * g.tn), first = band * 4, high = g.tm - first < 4 ? g.tm - first : 4, in = t0 - band * 4 * g.tn;
  const int64_t row0 = (int64_t)__builtin_amdgcn_readfirstlane(first + in % high) * BM;
  const int64_t col0 = (int64_t)__builtin_amdgcn_readfirstlane(in / high) * BN;

  const int64_t rows = KIND == kDgrad ? g.m : g.n, depth = KIND == kDgrad ? g.n : g.m;   // of A
  const int steps = (int)((depth + kStep - 1) / kStep);

  // ---- A: 16 bytes a load, 2 FM loads a step
  constexpr int kLoadsA = 2 * FM;
  uint32_t ao[kLoadsA], aw[kLoadsA];   // place in memory from the step's corner on, place in LDS
#pragma unroll
  for (int i = 0; i < kLoadsA; i++) {
    if (KIND == kDgrad) {
      const uint32_t row = (wave * kLoadsA + i) * 8 + (lane >> 3), u = lane & 7;
      ao[i] = (uint32_t)(row * g.lddy * 2) + u * 16;
      aw[i] = row * Lds::kRowA + (u ^ (row >> 1 & 7)) * 16;
    } else {
      constexpr int across = 8 * FM;   // lanes of a row
      const uint32_t row = (wave * kLoadsA + i) * (64 / across) + lane / across, u = lane % across;
      ao[i] = (uint32_t)(row * g.lddy * 2) + u * 16;
      aw[i] = row * Lds::kRowA + u * 16;
    }
  }
  v4i ra[kLoadsA];
  const int64_t left = rows - row0 < BM ? rows - row0 : BM;   // of A's rows (dgrad) or columns (wgrad)
  // dgrad: units past the row's end are sent past the stretch's end, as rows past m are.
  auto corner_a = [&](int t) {
    const int64_t at = (int64_t)t * kStep;
    if (KIND == kDgrad) return stretch(g.dy + row0 * g.lddy + at, at < depth ? ((left - 1) * g.lddy + g.row - at) * 2 : 0);
    const int64_t deep = depth - at < kStep ? depth - at : kStep;
    return stretch(g.dy + at * g.lddy + row0, deep > 0 ? ((deep - 1) * g.lddy + g.row - row0) * 2 : 0);
  };
  auto load_a = [&](__amdgpu_buffer_rsrc_t s, int t, int i) {
    uint32_t o = ao[i];
    if (KIND == kDgrad) o = (int64_t)t * kStep + (lane & 7) * 8 < g.row ? o : 0xFFFFFFF0u;
    ra[i] = load16(s, o);
  };

  // ---- B: dgrad: 32 codes of a row of W (one block); wgrad: 16 codes of a row of x8 (half a block)
  constexpr int kLoadsB = KIND == kDgrad ? FN / 2 : FN;
  v4i rb[kLoadsB];
  uint32_t rs[kLoadsB];
  struct CornerB { __amdgpu_buffer_rsrc_t c[KIND == kDgrad ? FN / 2 : 1], s[KIND == kDgrad ? FN / 2 : 1]; };
  auto corner_b = [&](int t) {
    CornerB c;
    const int64_t at = (int64_t)t * kStep;
    if (KIND == kDgrad) {
#pragma unroll
      for (int i = 0; i < FN / 2; i++) {
        const int64_t group = col0 / 128 + i;
        const bool real = group < mx4_groups(g.k) && at < depth;
        c.c[i] = stretch(g.b + (group * g.n + at) * 64, real ? (depth - at < kStep ? depth - at : kStep) * 64 : 0);
        c.s[i] = stretch(g.bs + (group * mx4_scale_rows(g.n) + at) * 4, real ? (depth - at < kStep ? depth - at : kStep) * 4 : 0);
      }
    } else {
      const int64_t deep = depth - at < kStep ? depth - at : kStep, p = ckpt_pitch(g.k), sp = ckpt_scale_pitch(g.k);
      c.c[0] = stretch(g.b + at * p + col0, deep > 0 ? (deep - 1) * p + p - col0 : 0);
      c.s[0] = stretch(g.bs + at * sp + col0 / 32, deep > 0 ? (deep - 1) * sp + sp - col0 / 32 : 0);
    }
    return c;
  };
  uint32_t bo[kLoadsB], bso[kLoadsB], bw[kLoadsB];
#pragma unroll
  for (int i = 0; i < kLoadsB; i++) {
    if (KIND == kDgrad) {
      const uint32_t row = tid >> 2, q = tid & 3;
      bo[i] = row * 64 + q * 16;
      bso[i] = row * 4 + q;
      bw[i] = row * Lds::kRowB + i * 256 + q * 64;
    } else {
      const uint32_t row = (i * 256 + tid) / (4 * FN), c = (i * 256 + tid) % (4 * FN);
      bo[i] = (uint32_t)(row * ckpt_pitch(g.k)) + c * 16;
      bso[i] = (uint32_t)(row * ckpt_scale_pitch(g.k)) + c / 2;
      bw[i] = row * Lds::kRowB + c * 32;
    }
  }
  auto load_b = [&](const CornerB& c, int i) {
    const int j = KIND == kDgrad ? i : 0;
    rb[i] = load16(c.c[j], bo[i]);
    rs[i] = load1(c.s[j], bso[i]);
  };
  // One quarter of load i: 8 codes of W (16 bytes) or 4 of x8 (8 bytes).
  auto put_b = [&](int st, int i, int part) {
    const float s = scale_value(rs[i]);
    if (KIND == kDgrad) {
      // lanes of one 16-lane turn write different 16 bytes of their 64, so that they meet different banks
      const int turn = (part + (tid >> 2)) & 3;
      const uint32_t lo = turn & 1 ? rb[i][1] : rb[i][0], hi = turn & 1 ? rb[i][3] : rb[i][2];
      *(v4i*)&lds.b[st][bw[i] + turn * 16] = widen_e2m1(turn & 2 ? hi : lo, s);
    } else {
      *(uint2*)&lds.b[st][bw[i] + part * 8] = widen_8<F>(rb[i][part], s);
    }
  };

  // ---- operands of 16 of the contraction
  struct Operands { v4i a[FM], b[FN]; };
  Operands P, Q;
  const uint32_t ra0 = KIND == kDgrad ? 0 : (8 * h + ((lane & 15) >> 2)) * Lds::kRowA + (wm * 32 * FM + (lane >> 4 & 1) * 16 + (lane & 3) * 4) * 2;
  const uint32_t rb0 = (8 * h + ((lane & 15) >> 2)) * Lds::kRowB + (wn * 32 * FN + (lane >> 4 & 1) * 16 + (lane & 3) * 4) * 2;
  auto columns = [&](const uint8_t* p, int row) {
    const v4s x = read_columns(p), y = read_columns(p + 4 * row);
    typedef short v8s __attribute__((ext_vector_type(8)));
    const v8s v = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
    return __builtin_bit_cast(v4i, v);
  };
  auto read = [&](int st, int q, Operands& o, int f) {
    if (f < FM) {
      if (KIND == kDgrad) {
        const int row = wm * 32 * FM + f * 32 + r;
        o.a[f] = *(const v4i*)&lds.a[st][row * Lds::kRowA + ((2 * q + h) ^ (r >> 1 & 7)) * 16];
      } else {
        o.a[f] = columns(&lds.a[st][ra0 + q * 16 * Lds::kRowA + f * 64], Lds::kRowA);
      }
    } else {
      o.b[f - FM] = columns(&lds.b[st][rb0 + q * 16 * Lds::kRowB + (f - FM) * 64], Lds::kRowB);
    }
  };

  v16f acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; i++)
#pragma unroll
    for (int j = 0; j < FN; j++)
#pragma unroll
      for (int e = 0; e < 16; e++) acc[i][j][e] = 0.0f;
  constexpr int per = FM * FN;
  auto multiply = [&](const Operands& o, auto between) {
#pragma unroll
    for (int i = 0; i < FM; i++)
#pragma unroll
      for (int j = 0; j < FN; j++) {
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, o.b[j]), __builtin_bit_cast(v8bf, o.a[i]), acc[i][j], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
        between(i * FN + j);
        __builtin_amdgcn_sched_barrier(0);
      }
  };
  // The `reads` of the next operands go under the first half of a quarter's products.
  auto spread = [&](int done, int from, int to, int count, auto what) {
#pragma unroll
    for (int f = 0; f < count; f++)
      if (from + f * (to - from) / count == done) what(f);
  };

  {
    const auto ca = corner_a(0);
    const auto cb = corner_b(0);
#pragma unroll
    for (int i = 0; i < kLoadsA; i++) load_a(ca, 0, i);
#pragma unroll
    for (int i = 0; i < kLoadsB; i++) load_b(cb, i);
  }
#pragma unroll
  for (int i = 0; i < kLoadsA; i++) *(v4i*)&lds.a[0][aw[i]] = ra[i];
#pragma unroll
  for (int i = 0; i < kLoadsB; i++)
#pragma unroll
    for (int q = 0; q < 4; q++) put_b(0, i, q);
  {
    const auto ca = corner_a(1);
    const auto cb = corner_b(1);
#pragma unroll
    for (int i = 0; i < kLoadsA; i++) load_a(ca, 1, i);
#pragma unroll
    for (int i = 0; i < kLoadsB; i++) load_b(cb, i);
  }
  __syncthreads();
#pragma unroll
  for (int f = 0; f < FM + FN; f++) read(0, 0, P, f);

  for (int t = 0; t < steps; t++) {
    const int st = t & 1, other = st ^ 1;
    const auto ca = corner_a(t + 2);
    const auto cb = corner_b(t + 2);
    // first quarter: the next step's dy goes into LDS, the one after it is asked for
    multiply(P, [&](int done) {
      spread(done, 0, per / 2, FM + FN, [&](int f) { read(st, 1, Q, f); });
      spread(done, per / 2, per, kLoadsA, [&](int i) {
        *(v4i*)&lds.a[other][aw[i]] = ra[i];
        load_a(ca, t + 2, i);
      });
    });
    // second and third quarter: likewise W or x8, converted
    multiply(Q, [&](int done) {
      spread(done, 0, per / 2, FM + FN, [&](int f) { read(st, 2, P, f); });
      spread(done, per / 2, per, 2 * kLoadsB, [&](int f) { put_b(other, f / 4, f % 4); });
    });
    multiply(P, [&](int done) {
      spread(done, 0, per / 2, FM + FN, [&](int f) { read(st, 3, Q, f); });
      spread(done, per / 2, per, 2 * kLoadsB, [&](int f) { put_b(other, (2 * kLoadsB + f) / 4, (2 * kLoadsB + f) % 4); });
      if (done == per - 1) {
#pragma unroll
        for (int i = 0; i < kLoadsB; i++) load_b(cb, i);
      }
    });
    // the next step is in LDS, and nobody reads this one any more
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    multiply(Q, [&](int done) {
      spread(done, 0, per / 2, FM + FN, [&](int f) { read(other, 0, P, f); });
    });
  }

  // A lane holds row r of a 32 x 32 block of the result, columns 8q + 4h .. + 3:
  // each wave turns 32 rows at a time through LDS into row stretches. (The sums
  // are pinned to accumulation registers up to here.)
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
  for (int i = 0; i < FM; i++)
#pragma unroll
    for (int j = 0; j < FN; j++) asm volatile("" : "+a"(acc[i][j]));
  constexpr int kRow = 32 * FN * (int)sizeof(T) + 16, V = 16 / (int)sizeof(T), units = 32 * FN / V;
  static_assert(4 * 32 * kRow <= (int)sizeof(Lds), "");
  uint8_t* mine = (uint8_t*)&lds + wave * 32 * kRow;
  const int64_t r0 = row0 + wm * 32 * FM, c0 = col0 + wn * 32 * FN;
#pragma unroll
  for (int i = 0; i < FM; i++) {
#pragma unroll
    for (int j = 0; j < FN; j++)
#pragma unroll
      for (int q = 0; q < 4; q++) {
        T v[4];
#pragma unroll
        for (int e = 0; e < 4; e++) v[e] = narrow<OUT>(acc[i][j][4 * q + e]);
        __builtin_memcpy(__builtin_assume_aligned(mine + r * kRow + (j * 32 + 8 * q + 4 * h) * (int)sizeof(T), 4 * sizeof(T)), v, sizeof(v));
      }
    asm volatile("" ::: "memory");
#pragma unroll
    for (int u0 = 0; u0 < units / 2; u0++) {
      const int u = u0 * 64 + lane, rr = u / units, cc = u % units * V;
      const int64_t row = r0 + i * 32 + rr, col = c0 + cc;
      T v[V];
      __builtin_memcpy(v, __builtin_assume_aligned(mine + rr * kRow + cc * (int)sizeof(T), 16), 16);
      if (row < rows && col < g.k) {
        T* o = (T*)g.out + row * g.ldo + col;
        if (g.k - col >= V) {
          if constexpr (KIND == kWgrad) {
            if (g.in) {
              float w[V];
              __builtin_memcpy(w, g.in + row * g.ldo + col, 16);
#pragma unroll
              for (int e = 0; e < V; e++) v[e] += w[e];
            }
          }
          __builtin_memcpy(o, v, 16);
        } else {
#pragma unroll
          for (int e = 0; e < V; e++)
            if (col + e < g.k) {
              if constexpr (KIND == kWgrad) o[e] = v[e] + (g.in ? g.in[row * g.ldo + col + e] : 0.0f);
              else o[e] = v[e];
            }
        }
      }
    }
    asm volatile("" ::: "memory");
  }
}

// dy with rows of a multiple of 64 elements, zeros past n.
__global__ __launch_bounds__(256) void k_pad_rows(const uint16_t* dy, int64_t m, int64_t n, int64_t ld, uint16_t* out,
                                                  int64_t ldo) {
  const int64_t across = (ldo + 511) / 512;
  for (int64_t u = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); u < m * across; u += (int64_t)gridDim.x * 4) {
    const int64_t row = u / across, col = u % across * 512 + (threadIdx.x & 63) * 8;
    if (col >= ldo) continue;
    uint16_t v[8];
    const uint16_t* p = dy + row * ld + col;
    if (n - col >= 8) {
      __builtin_memcpy(v, p, 16);
    } else {
#pragma unroll
      for (int e = 0; e < 8; e++) v[e] = col + e < n ? p[e] : (uint16_t)0;
    }
    __builtin_memcpy(__builtin_assume_aligned(out + row * ldo + col, 16), v, 16);
  }
}

template <int KIND, int F, int OUT, int FM, int FN>
hipError_t grad_tiled(GradArgs& g, hipStream_t s) {
  const int64_t rows = KIND == kDgrad ? g.m : g.n;
  g.tm = (uint32_t)((rows + 64 * FM - 1) / (64 * FM));
  g.tn = (uint32_t)((g.k + 64 * FN - 1) / (64 * FN));
  hipLaunchKernelGGL((k_grad<KIND, F, OUT, FM, FN>), dim3(g.tm * g.tn), dim3(256), 0, s, g);
  return hipGetLastError();
}
template <int KIND, int F, int OUT>
hipError_t grad(GradArgs g, void* ws, hipStream_t s) {
  if (needs_padding(g.n, g.lddy)) {
    const int64_t ld = padded_columns(g.n);
    hipLaunchKernelGGL(k_pad_rows, dim3(stream_grid(g.m * ((ld + 511) / 512))), dim3(256), 0, s, g.dy, g.m, g.n, g.lddy, (uint16_t*)ws, ld);
    if (hipGetLastError() != hipSuccess) return hipErrorLaunchFailure;
    g.dy = (const uint16_t*)ws;
    g.lddy = g.row = ld;
  }
  const int64_t rows = KIND == kDgrad ? g.m : g.n;
  if ((rows + 255) / 256 * ((g.k + 255) / 256) >= 200) return grad_tiled<KIND, F, OUT, 4, 4>(g, s);
  return grad_tiled<KIND, F, OUT, 2, 2>(g, s);
}

}  // namespace

hipError_t launch_mx4_dgrad(const void* dy, int64_t m, int64_t n, int64_t lddy, const void* w_codes,
                            const void* w_scales, int64_t k, int out_dtype, void* dx, int64_t lddx, void* ws,
                            hipStream_t s) {
  if (n == 0) return launch_constant(m, k, out_dtype, nullptr, dx, lddx, s);
  const GradArgs g = {(const uint16_t*)dy, m, n, k, lddy, n, (const uint8_t*)w_codes, (const uint8_t*)w_scales, nullptr, dx, lddx, 0, 0};
  switch (out_dtype) {
    case LQ_F32: return grad<kDgrad, LQ_E2M1, LQ_F32>(g, ws, s);
    case LQ_BF16: return grad<kDgrad, LQ_E2M1, LQ_BF16>(g, ws, s);
    default: return grad<kDgrad, LQ_E2M1, LQ_F16>(g, ws, s);
  }
}

hipError_t launch_ckpt8_wgrad(int format, const void* dy, int64_t m, int64_t n, int64_t lddy, const void* x_codes,
                              const void* x_scales, int64_t k, const float* dw_in, float* dw, int64_t lddw, void* ws,
                              hipStream_t s) {
  if (m == 0) return launch_constant(n, k, LQ_F32, dw_in, dw, lddw, s);
  const GradArgs g = {(const uint16_t*)dy, m, n, k, lddy, n, (const uint8_t*)x_codes, (const uint8_t*)x_scales, dw_in, dw, lddw, 0, 0};
  if (format == LQ_INT8) return grad<kWgrad, LQ_INT8, LQ_F32>(g, ws, s);
  return grad<kWgrad, LQ_E4M3, LQ_F32>(g, ws, s);
}

}  // namespace lql
