// lq_grad.hip — the linear layer's gradients: dx = dy W from the 4-bit weights,
// dw = dw0 + dy^T x8 from the 8-bit checkpoint of x.
#include <stddef.h>

#include <type_traits>

#include "lq_linear.h"

namespace lql {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));

// Both gradients are matrix products A B over bfloat16 operands: E2M1 and INT8
// values times a power of two have at most 7 significant bits, E4M3 values 4,
// so the stored operand is exact in bfloat16 (8 bits; its exponents are
// binary32's) and is converted once, on its way into LDS. (But below 2^-126
// bfloat16 holds multiples of 2^-133 only. The scales end at 2^-127: E2M1's unit of
// 2^-1 and INT8's of 1 stay above, E4M3's of 2^-9 does not for scales below
// 2^-124, whose values the conversion rounds, half to even.)
//   dgrad: A = dy [m, n], B = W [n, k]; the contraction runs along dy's rows
//          and down W's columns
//   wgrad: A = dy^T, B = x8 [m, k]; it runs down the columns of both
// An operand whose contraction runs down the columns lies in LDS as it lies in
// memory and is read with ds_read_b64_tr_b16, which hands each lane of a group
// of 16 four rows of one column: two of them are the eight consecutive
// contraction values that a lane of v_mfma_f32_32x32x16_bf16 takes.
//
// A workgroup of 2 x 2 waves makes a (64 FM) x (64 FN) tile, 64 of the
// contraction a step. LDS holds two steps; the next two are on their way in
// registers (with one, a step of 256 x 256 waited for its loads: 1.5 us against
// the 0.85 us of its products on an idle chip). Each step's loads, conversions, LDS writes and reads go between
// its products, a few instructions at a time, so that the matrix cores are
// never without work; one barrier a step.
//
// dx 8192 x 11008 x 4096 506 to 620 us (1.2 to 1.5 PFLOP/s), dw from E4M3 582 us
// (1.27), from INT8 650 us (1.14; twice the vector instructions to convert it). The
// library's bf16 product, all operands in memory at 2 bytes, takes 574 us for the
// first and 836 us for dw's order of operands, and 8192^3 at 1.2 to 1.3 PFLOP/s.
// The large dx keeps the matrix cores busy 72% of the cycles, at 1.8 of 2.4 GHz. The
// 128 x 128 tile with one workgroup a compute unit keeps them busy 31%, LDS 40% and
// vector issue 8%: one wave on a SIMD has no other's work for its waits. 1024 x 4096
// x 4096 35 us, where the library takes 42; dw of those sizes, in 256 x 256 tiles,
// 41 us (23% busy: 16 steps, and then 256 KB of results a compute unit).
enum Kind { kDgrad, kWgrad };
constexpr int kStep = 64;

// Place of a row's 16-byte unit in a column operand. A transposing read takes
// four rows, 64 bytes of each: they lie in the four 64-byte quarters of the
// banks. A store has one unit of each of 16 rows: all 16 lie apart.
__device__ __forceinline__ int column_unit(int row, int unit) { return unit ^ ((row & 3) << 2 | (row >> 2 & 3)); }

template <int KIND, int FM, int FN>
struct GradLds {
  // dgrad's dy: 128 bytes a row, its 16-byte units in the order u ^ (row / 2 & 7) (16 lanes at a time read 16
  // different units of 256 bytes)
  static constexpr int kRowA = KIND == kDgrad ? 2 * kStep : 128 * FM, kRowsA = KIND == kDgrad ? 64 * FM : kStep;
  // columns: 16-byte units in the order of column_unit()
  static constexpr int kRowB = 128 * FN;
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
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ v4i load16(__amdgpu_buffer_rsrc_t s, uint32_t offset, uint32_t further = 0) {
  return __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(s, (int)offset, (int)further, 0));
}
__device__ __forceinline__ uint8_t load1(__amdgpu_buffer_rsrc_t s, uint32_t offset, uint32_t further = 0) {
  return __builtin_amdgcn_raw_buffer_load_b8(s, (int)offset, (int)further, 0);
}
// LDS by address. The few registers that a thread's places come from are made
// opaque, and all else is an instruction's constant offset (at most 65535):
// left alone, the compiler keeps every place in a register of its own, 60 of
// them, and spills.
typedef uint32_t place_t;
__device__ __forceinline__ place_t place(place_t p) {
  asm volatile("" : "+v"(p));
  return p;
}
__device__ __forceinline__ v4i get16(place_t p) { return *(const __attribute__((address_space(3))) v4i*)p; }
__device__ __forceinline__ void put16(place_t p, v4i v) { *(__attribute__((address_space(3))) v4i*)p = v; }
__device__ __forceinline__ v4s read_columns(place_t p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)p);
}

// Two INT8 codes times their scale as bfloat16: bytes `first` and first + 1 of w.
// The binary32 product is exact, and its upper half is the bfloat16.
__device__ __forceinline__ int widen_int8(uint32_t w, int first, float s) {
  const uint32_t a = __float_as_uint((float)(int8_t)(w >> 8 * first) * s);
  const uint32_t b = __float_as_uint((float)(int8_t)(w >> 8 * (first + 1)) * s);
  return (int)__builtin_amdgcn_perm(b, a, 0x07060302u);
}

struct GradArgs {
  const uint16_t* dy;
  int64_t m, n, k, lddy;
  int64_t row;             // elements of a row of dy that may be read: n, or n padded
  const uint8_t *b, *bs;   // W's codes and scales, or the checkpoint's
  const float* in;         // dw_in
  void* out;
  int64_t ldo;
  uint32_t tm, tn;
  int parts, part;         // of the contraction: steps of each; with parts > 1, out is `parts` planes
};

// F: the checkpoint's format (wgrad); OUT: the result's type; RAGGED (dgrad): dy's
// rows end inside a unit of 8 elements, of whose last the rest is cut off.
template <int KIND, int F, int OUT, int FM, int FN, bool RAGGED>
__global__ __launch_bounds__(256, FM * FN >= 16 ? 1 : 2) void k_grad(const GradArgs g) {
  typedef typename El<OUT>::T T;
  typedef GradLds<KIND, FM, FN> Lds;
  constexpr int BM = 64 * FM, BN = 64 * FN;
  __shared__ Lds lds;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 31, h = lane >> 5, wm = wave >> 1, wn = wave & 1;

  // The XCD's share of the tiles is a contiguous run in bands of 4 rows of tiles (as in the 4-bit product).
  const uint32_t tiles = g.tm * g.tn, total = tiles * g.parts, xcd = blockIdx.x % 8, per8 = total / 8, more = total % 8;
  const uint32_t mine8 = xcd * per8 + (xcd < more ? xcd : more) + blockIdx.x / 8;
  const uint32_t part = __builtin_amdgcn_readfirstlane(mine8 / tiles), t0 = mine8 - part * tiles;
  const uint32_t band = t0 / (4 * g.tn), first = band * 4, high = g.tm - first < 4 ? g.tm - first : 4, in = t0 - band * 4 * g.tn;
  const int64_t row0 = (int64_t)__builtin_amdgcn_readfirstlane(first + in % high) * BM;
  const int64_t col0 = (int64_t)__builtin_amdgcn_readfirstlane(in / high) * BN;

  const int64_t rows = KIND == kDgrad ? g.m : g.n, depth = KIND == kDgrad ? g.n : g.m;   // of A
  const int all = (int)((depth + kStep - 1) / kStep), begin = (int)part * g.part;
  const int steps = begin + g.part < all ? begin + g.part : all;

  // ---- A: 16 bytes a load, 2 FM loads a step
  constexpr int kLoadsA = 2 * FM;
  const place_t lds0 = (place_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)&lds;
  const place_t ldsb = lds0 + (place_t)offsetof(Lds, b);
  uint32_t ao;               // place in memory of the first load, from the step's corner on; load i is `astep` i further
  constexpr int kPlacesA = KIND == kDgrad ? 2 : kLoadsA;   // (the order of the units repeats every other load, or not at all)
  place_t aw[kPlacesA];      // in LDS, of the first loads
  constexpr int awide = KIND == kDgrad ? 8 * Lds::kRowA : 8 / FM * Lds::kRowA;   // LDS bytes of a load's rows
  const uint32_t astep = (uint32_t)((KIND == kDgrad ? 8 : 8 / FM) * g.lddy * 2);
  {
    constexpr int across = KIND == kDgrad ? 8 : 8 * FM;   // lanes of a row
    const int row = wave * kLoadsA * (64 / across) + lane / across, u = lane % across;
    ao = (uint32_t)(row * g.lddy * 2) + u * 16;
#pragma unroll
    for (int i = 0; i < kPlacesA; i++) {
      const int rr = row + i * (64 / across);
      aw[i] = place(lds0 + row * Lds::kRowA + i * awide + (KIND == kDgrad ? u ^ (rr >> 1 & 7) : column_unit(rr, u)) * 16);
    }
  }
  v4i ra[2][kLoadsA];   // of the even and the odd steps
  const int64_t left = rows - row0 < BM ? rows - row0 : BM;   // of A's rows (dgrad) or columns (wgrad)

  // ---- where the next loads begin, moved on by a few scalar instructions a step (one wave on a SIMD has no other's
  // slots to hide them in: with each stretch worked out anew, 40 more of them, a step of the 128 x 128 tile took
  // 0.50 us instead of 0.43 on an idle chip, the weight gradient's 0.63 instead of 0.53). What a stretch's end cuts off reads as zero: rows past the tile's last, the
  // contraction past the part's end.
  constexpr int kPieces = KIND == kDgrad ? FN / 2 : 1;   // groups of W, or the checkpoint
  const int64_t pitch = ckpt_pitch(g.k), spitch = ckpt_scale_pitch(g.k);
  const int64_t start = (int64_t)begin * kStep, end = (int64_t)steps * kStep < depth ? (int64_t)steps * kStep : depth;
  // dgrad: dy's stretch moves along the rows, and its end stays where it is; units past the rows' end are sent out of
  // it one by one. W's groups lie still, and the step's place in them moves.
  const int columns_end = steps == all ? (int)g.row : steps * kStep;
  uint32_t wstep = (uint32_t)start * 64, wsstep = (uint32_t)start * 4;
  // wgrad: all three move down the rows, 64 at a time, the part's last step with what is left
  int to_come = steps - begin;
  const uint8_t *pa8 = (const uint8_t*)(KIND == kDgrad ? g.dy + row0 * g.lddy + start : g.dy + start * g.lddy + row0);
  const uint8_t *pc8 = g.b + start * pitch + col0, *ps8 = g.bs + start * spitch + col0 / 32;
  const int64_t tail = end - start - (to_come - 1) * (int64_t)kStep;   // rows of the last step
  // (a load's every 4 bytes have to end before the stretch does: of rows of odd length, 2 more are let in, which the
  // rules of reads_in_place() keep inside the matrix or its last 4 bytes)
  const int64_t row_bytes = (g.row + (g.row & 1)) * 2;
  auto size_a = [&](int64_t rows_left) { return (uint32_t)((rows_left - 1) * g.lddy * 2 + row_bytes - row0 * 2); };   // (below 2^31)
  auto size_c = [&](int64_t rows_left) { return (uint32_t)(rows_left * pitch - col0); };
  auto size_s = [&](int64_t rows_left) { return (uint32_t)(rows_left * spitch - col0 / 32); };
  const uint32_t last_a = uniform(size_a(tail)), last_c = uniform(size_c(tail)), last_s = uniform(size_s(tail));
  uint32_t bytes_a = uniform(KIND == kDgrad ? (uint32_t)((left - 1) * g.lddy * 2 + row_bytes - start * 2) : size_a(kStep));
  uint32_t bytes_c = uniform(size_c(kStep)), bytes_s = uniform(size_s(kStep));
  const uint32_t move_a = uniform((uint32_t)(KIND == kDgrad ? kStep * 2 : kStep * 2 * g.lddy)), move_c = uniform((uint32_t)(kStep * pitch)), move_s = uniform((uint32_t)(kStep * spitch));
  __amdgpu_buffer_rsrc_t sa, sc[kPieces], ss[kPieces];
  if (KIND == kDgrad) {
#pragma unroll
    for (int i = 0; i < kPieces; i++) {
      const int64_t panel = col0 / 128 + i;
      const bool real = panel < mx4_groups(g.k);
      sc[i] = stretch(g.b + panel * g.n * 64, real ? end * 64 : 0);
      ss[i] = stretch(g.bs + panel * mx4_scale_rows(g.n) * 4, real ? end * 4 : 0);
    }
  }
  auto point = [&] {
    if (KIND == kWgrad) {
      if (to_come == 1) bytes_a = last_a, bytes_c = last_c, bytes_s = last_s;
      if (to_come <= 0) bytes_a = bytes_c = bytes_s = 0;
      sc[0] = stretch(pc8, bytes_c);
      ss[0] = stretch(ps8, bytes_s);
      pc8 += move_c;
      ps8 += move_s;
    }
    to_come--;
    sa = stretch(pa8, (int)bytes_a);
    pa8 += move_a;
    if (KIND == kDgrad) bytes_a -= move_a;
  };
  auto load_a = [&](int t, int set, int i) {
    uint32_t o = ao;
    if (KIND == kDgrad) o = t * kStep + (lane & 7) * 8 < columns_end ? o : 0xFFFFFFF0u;
    ra[set][i] = load16(sa, o, i * astep);
  };
  v4i keep, cut;   // RAGGED: of the lane's unit in the contraction's last step, and in the step that is put into LDS
  if (RAGGED) {
#pragma unroll
    for (int d = 0; d < 4; d++) {
      const int there = (int)g.n - (all - 1) * kStep - (lane & 7) * 8 - 2 * d;
      keep[d] = there >= 2 ? -1 : there == 1 ? 0xFFFF : 0;
    }
  }
  auto cut_for = [&](int t) {
    if (RAGGED) {
#pragma unroll
      for (int d = 0; d < 4; d++) cut[d] = t == all - 1 ? keep[d] : -1;
    }
  };
  auto put_a = [&](int st, int set, int i) {
    put16(aw[i % kPlacesA] + st * (place_t)sizeof(lds.a[0]) + i / kPlacesA * kPlacesA * awide, RAGGED ? ra[set][i] & cut : ra[set][i]);
  };

  // ---- B: dgrad: 32 codes of a row of W (one block); wgrad: 16 codes of a row of x8 (half a block)
  constexpr int kLoadsB = KIND == kDgrad ? FN / 2 : FN;
  v4i rb[2][kLoadsB];
  uint8_t rs[2][kLoadsB];
  // (dgrad: a wave takes one block of each of the 64 rows, load i in group i; wgrad: half a block of rows 4 or 8 a wave)
  constexpr int kUnitsB = KIND == kDgrad ? 4 * kLoadsB : 2 * kLoadsB, kEach = kUnitsB / kLoadsB;   // 8 codes each
  const int brow = KIND == kDgrad ? lane : tid / (4 * FN), bcol = KIND == kDgrad ? wave : tid % (4 * FN);
  constexpr int bwide = KIND == kDgrad ? 256 : 256 / (4 * FN) * Lds::kRowB;                       // LDS bytes from load to load
  const uint32_t bo = (uint32_t)(brow * (KIND == kDgrad ? 64 : pitch)) + bcol * 16, bstep = KIND == kDgrad ? 0 : (uint32_t)(256 / (4 * FN) * pitch);
  const uint32_t bso = (uint32_t)(brow * (KIND == kDgrad ? 4 : spitch)) + (KIND == kDgrad ? bcol : bcol / 2);
  const uint32_t bsstep = KIND == kDgrad ? 0 : (uint32_t)(256 / (4 * FN) * spitch);
  place_t bw[kEach];
#pragma unroll
  for (int u = 0; u < kEach; u++) bw[u] = place(ldsb + brow * Lds::kRowB + column_unit(brow, bcol * kEach + u) * 16);
  auto load_b = [&](int set, int i) {
    const int j = KIND == kDgrad ? i : 0;
    rb[set][i] = load16(sc[j], bo, KIND == kDgrad ? wstep : i * bstep);
    rs[set][i] = load1(ss[j], bso, KIND == kDgrad ? wsstep : i * bsstep);
    if (KIND == kDgrad && i == kLoadsB - 1) {
      wstep += kStep * 64;
      wsstep += kStep * 4;
    }
  };
  // Unit i of the step's W or x8: 8 codes, converted in kBits bits and stored with the last.
  constexpr int kBits = KIND == kWgrad && F == LQ_INT8 ? 4 : 2;
  static_assert(kUnitsB == kLoadsA, "a thread has as many units of either operand");
  float scale[kLoadsB];
  v4i made;
  auto put_b = [&](int st, int set, int i, int bit) {
    const int l = i / kEach, u = i % kEach;
    const float s = scale[l];
    if (KIND == kDgrad) {
      const uint32_t w = rb[set][l][u];
      if (bit == 0) {
        made[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
        made[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
      } else {
        made[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
        made[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
      }
    } else if (F == LQ_INT8) {
      made[bit] = widen_int8((uint32_t)rb[set][l][2 * u + bit / 2], bit % 2 * 2, s);
    } else {
      const int w = rb[set][l][2 * u + bit];
      made[2 * bit] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, false));
      made[2 * bit + 1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, true));
    }
    if (bit == kBits - 1) put16(bw[u] + st * (place_t)sizeof(lds.b[0]) + l * bwide, made);
  };

  // ---- operands of 16 of the contraction
  struct Operands { v4i a[FM], b[FN]; };
  Operands P, Q;
  // Place of the lane's piece of four rows of 32 columns from `col` on, rows 8h .. + 3 or, four further, 8h + 4 .. + 7.
  const int crow = 8 * h + ((lane & 15) >> 2);
  auto piece = [&](int row_bytes, int col, int further) {
    const int row = crow + further, c = col + (lane >> 4 & 1) * 16 + (lane & 3) * 4;
    return row * row_bytes + column_unit(row, c >> 3) * 16 + (c & 7) * 2;
  };
  place_t pa[KIND == kDgrad ? 4 : 2 * FM], pb[2 * FN];
#pragma unroll
  for (int x = 0; x < 2; x++) {
    if (KIND == kWgrad) {
#pragma unroll
      for (int f = 0; f < FM; f++) pa[2 * f + x] = place(lds0 + piece(Lds::kRowA, wm * 32 * FM + f * 32, 4 * x));
    }
#pragma unroll
    for (int f = 0; f < FN; f++) pb[2 * f + x] = place(ldsb + piece(Lds::kRowB, wn * 32 * FN + f * 32, 4 * x));
  }
  if (KIND == kDgrad) {
#pragma unroll
    for (int q = 0; q < 4; q++) pa[q] = place(lds0 + (wm * 32 * FM + r) * Lds::kRowA + ((2 * q + h) ^ (r >> 1 & 7)) * 16);
  }
  auto columns = [&](place_t p, place_t q) {
    const v4s x = read_columns(p), y = read_columns(q);
    typedef short v8s __attribute__((ext_vector_type(8)));
    const v8s v = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
    return __builtin_bit_cast(v4i, v);
  };
  auto read = [&](int st, int q, Operands& o, int f) {
    const place_t a = st * (place_t)sizeof(lds.a[0]), b = st * (place_t)sizeof(lds.b[0]) + q * 16 * Lds::kRowB;
    if (f < FM) {
      if (KIND == kDgrad) o.a[f] = get16(pa[q] + a + f * 32 * Lds::kRowA);
      else o.a[f] = columns(pa[2 * f % (2 * FM)] + a + q * 16 * Lds::kRowA, pa[(2 * f + 1) % (2 * FM)] + a + q * 16 * Lds::kRowA);
    } else {
      o.b[f - FM] = columns(pb[2 * (f - FM)] + b, pb[2 * (f - FM) + 1] + b);
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
  // One quarter's products; `between` runs after each. 28 of a product's 32 cycles are free for other
  // instructions: what goes between two products is kept to about six of them (in bursts of 16 the conversions
  // alone cost a third of the step), and scheduling barriers keep it there.
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
  // `count` pieces of work over `over` places between products
  auto spread = [&](int done, int over, int count, auto what) {
#pragma unroll
    for (int f = 0; f < count; f++)
      if (f * over / count == done) what(f);
  };

  auto load = [&](int t, int set) {
    point();
#pragma unroll
    for (int i = 0; i < kLoadsA; i++) load_a(t, set, i);
#pragma unroll
    for (int i = 0; i < kLoadsB; i++) load_b(set, i);
  };
  auto take_scales = [&](int set, int i) {
    scale[i] = scale_value(rs[set][i]);
  };
  load(begin, 0);
  load(begin + 1, 1);
  cut_for(begin);
#pragma unroll
  for (int i = 0; i < kLoadsA; i++) put_a(0, 0, i);
#pragma unroll
  for (int i = 0; i < kLoadsB; i++) take_scales(0, i);
#pragma unroll
  for (int i = 0; i < kUnitsB * kBits; i++) put_b(0, 0, i / kBits, i % kBits);
  load(begin + 2, 0);
  point();
#pragma unroll
  for (int i = 0; i < kLoadsB; i++) take_scales(1, i);
  __syncthreads();
#pragma unroll
  for (int f = 0; f < FM + FN; f++) read(0, 0, P, f);

  // Step t, in LDS stage ST: the next step's data, which came into registers two
  // steps ago, goes into the other stage, and the step three on is asked for.
  auto step = [&](auto stage, int t) {
    constexpr int ST = decltype(stage)::value, OTHER = ST ^ 1;
    // The units of either operand go over three quarters. Each quarter also reads the next one's operands, early
    // enough for the last to arrive.
    constexpr int window = (per * 3 + 3) / 4, bits = kUnitsB * kBits, bit_third = (bits + 2) / 3, third = (kLoadsA + 2) / 3;
    auto work = [&](int quarter, int done) {
      const int a0 = quarter * third, an = kLoadsA - a0 < third ? kLoadsA - a0 : third;
      spread(done, per, an, [&](int f) {
        put_a(OTHER, OTHER, a0 + f);
        load_a(t + 3, OTHER, a0 + f);
      });
      const int b0 = quarter * bit_third, bn = bits - b0 < bit_third ? bits - b0 : bit_third;
      spread(done, per, bn, [&](int f) { put_b(OTHER, OTHER, (b0 + f) / kBits, (b0 + f) % kBits); });
    };
    cut_for(t + 1);
    multiply(P, [&](int done) {
      spread(done, window, FM + FN, [&](int f) { read(ST, 1, Q, f); });
      work(0, done);
    });
    multiply(Q, [&](int done) {
      spread(done, window, FM + FN, [&](int f) { read(ST, 2, P, f); });
      work(1, done);
    });
    multiply(P, [&](int done) {
      spread(done, window, FM + FN, [&](int f) { read(ST, 3, Q, f); });
      work(2, done);
    });
    // the next step is in LDS, and nobody reads this one any more
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    multiply(Q, [&](int done) {
      spread(done, window, FM + FN, [&](int f) { read(OTHER, 0, P, f); });
      spread(done, per / 2, kLoadsB, [&](int i) { load_b(OTHER, i); });
      spread(done, per / 2, kLoadsB, [&](int i) { take_scales(ST, i); });
      if (done == per / 2) point();
    });
  };
  // (of an odd number of steps, the last is followed by one of zeros)
  for (int t = begin; t < steps; t += 2) {
    step(std::integral_constant<int, 0>(), t);
    step(std::integral_constant<int, 1>(), t + 1);
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
  // What dw is added to, of 32 rows: asked for a block of rows ahead (a load may not pass a store that might be to the
  // same place: one by one, 154 x 11008 x 4096 took 123 us, and with 8 at a time 20 us more in 256 x 256 tiles).
  constexpr int kStores = units / 2;
  v4f base[2][kStores];
  auto load_base = [&](int i) {
    if (KIND == kWgrad && g.in) {
#pragma unroll
      for (int b = 0; b < kStores; b++) {
        const int u = b * 64 + lane;
        const int64_t row = r0 + i * 32 + u / units, col = c0 + u % units * V;
        if (row < rows && g.k - col >= V) __builtin_memcpy(&base[i % 2][b], g.in + row * g.ldo + col, 16);
      }
    }
  };
  load_base(0);
#pragma unroll
  for (int i = 0; i < FM; i++) {
    if (i + 1 < FM) load_base(i + 1);
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
    for (int b = 0; b < kStores; b++) {
      const int u = b * 64 + lane, rr = u / units, cc = u % units * V;
      const int64_t row = r0 + i * 32 + rr, col = c0 + cc;
      T v[V];
      __builtin_memcpy(v, __builtin_assume_aligned(mine + rr * kRow + cc * (int)sizeof(T), 16), 16);
      if (row < rows && col < g.k) {
        T* o = (T*)g.out + (part * rows + row) * g.ldo + col;
        if (g.k - col >= V) {
          if constexpr (KIND == kWgrad) {
            if (g.in) {
#pragma unroll
              for (int e = 0; e < V; e++) v[e] += base[i % 2][b][e];
            }
          }
          store16(o, v);
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
  const int64_t col = (int64_t)blockIdx.x * 512 + (threadIdx.x & 63) * 8;
  if (col >= ldo) return;
  for (int64_t row = (int64_t)blockIdx.y * 4 + (threadIdx.x >> 6); row < m; row += (int64_t)gridDim.y * 4) {
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
  constexpr bool kMayBe = KIND == kDgrad;
  const int64_t rows = KIND == kDgrad ? g.m : g.n;
  g.tm = (uint32_t)((rows + 64 * FM - 1) / (64 * FM));
  g.tn = (uint32_t)((g.k + 64 * FN - 1) / (64 * FN));
  const dim3 grid(g.tm * g.tn * g.parts);
  if (lqd::g_plan) return LQ_PLAN(grid, 256, "k_grad<%d, %d, %d, %d, %d, %s>", KIND, F, OUT, FM, FN, lqd::tf(kMayBe && g.row % 8 != 0));
  if (kMayBe && g.row % 8 != 0) hipLaunchKernelGGL((k_grad<KIND, F, OUT, FM, FN, kMayBe>), grid, dim3(256), 0, s, g);
  else hipLaunchKernelGGL((k_grad<KIND, F, OUT, FM, FN, false>), grid, dim3(256), 0, s, g);
  return hipGetLastError();
}
template <int KIND, int F, int OUT>
hipError_t grad_tile(int tile, GradArgs& g, hipStream_t s) {
  return tile == 4 ? grad_tiled<KIND, F, OUT, 4, 4>(g, s) : grad_tiled<KIND, F, OUT, 2, 2>(g, s);
}
template <int KIND, int F, int OUT>
hipError_t grad(GradArgs g, void* ws, hipStream_t s) {
  uint8_t* planes = (uint8_t*)ws;
  if (!reads_in_place(g.m, g.n, g.lddy)) {
    const int64_t ld = padded_columns(g.n);
    const dim3 grid = matrix_grid((ld + 511) / 512, g.m);
    if (lqd::g_plan) {
      (void)LQ_PLAN(grid, 256, "k_pad_rows");
    } else {
      hipLaunchKernelGGL(k_pad_rows, grid, dim3(256), 0, s, g.dy, g.m, g.n, g.lddy, (uint16_t*)ws, ld);
      if (hipGetLastError() != hipSuccess) return hipErrorLaunchFailure;
    }
    g.dy = (const uint16_t*)ws;
    g.lddy = g.row = ld;
    planes += (g.m * ld * 2 + 255) / 256 * 256;
  }
  const int64_t rows = KIND == kDgrad ? g.m : g.n;
  const Split c = KIND == kDgrad ? split_dgrad(g.m, g.n, g.k) : split_wgrad(g.m, g.n, g.k, g.in != nullptr);
  g.parts = c.parts;
  g.part = c.part;
  if (c.parts == 1) return grad_tile<KIND, F, OUT>(c.tile, g, s);
  void* const out = g.out;
  const float* const in = g.in;
  const int64_t ldo = g.ldo;
  g.out = planes;
  g.in = nullptr;
  g.ldo = plane_stride(g.k);
  const hipError_t e = grad_tile<KIND, F, LQ_F32>(c.tile, g, s);
  return e != hipSuccess ? e : launch_join(rows, g.k, OUT, c.parts, (const float*)planes, in, out, ldo, s);
}

}  // namespace

hipError_t launch_mx4_dgrad(const void* dy, int64_t m, int64_t n, int64_t lddy, const void* w_codes,
                            const void* w_scales, int64_t k, int out_dtype, void* dx, int64_t lddx, void* ws,
                            hipStream_t s) {
  if (n == 0) return launch_constant(m, k, out_dtype, nullptr, dx, lddx, s);
  const GradArgs g = {(const uint16_t*)dy, m, n, k, lddy, n, (const uint8_t*)w_codes, (const uint8_t*)w_scales, nullptr, dx, lddx, 0, 0, 1, 0};
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
  const GradArgs g = {(const uint16_t*)dy, m, n, k, lddy, n, (const uint8_t*)x_codes, (const uint8_t*)x_scales, dw_in, dw, lddw, 0, 0, 1, 0};
  if (format == LQ_INT8) return grad<kWgrad, LQ_INT8, LQ_F32>(g, ws, s);
  return grad<kWgrad, LQ_E4M3, LQ_F32>(g, ws, s);
}

}  // namespace lql
