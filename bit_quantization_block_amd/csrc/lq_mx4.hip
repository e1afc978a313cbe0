// lq_mx4.hip — 4-bit microscaled quantisation and product.
#include <type_traits>

#include "lq_linear.h"

namespace lql {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));

// ---------------------------------------------------------------- quantise
// One wave per 4 rows x 128 columns, four side by side in a workgroup; a lane
// holds 8 consecutive elements, so a block of 32 is the four lanes of a quad,
// and the wave's codes are 256 bytes in one stretch. One read of x gives the
// 4-bit operand and the 8-bit checkpoint: bound by memory, 8192 x 4096 of bf16
// 17 us (4.9 TB/s, a large copy's 5.1), with the checkpoint 20 us (5.9 TB/s).
template <int DT, int F>
__global__ __launch_bounds__(256) void k_mx4_quantize(const void* x, int64_t m, int64_t k, int64_t ldx,
                                                      uint8_t* codes, uint8_t* scales, uint8_t* ck, uint8_t* cks) {
  const int lane = threadIdx.x & 63;
  const int64_t col = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * 128 + (lane & 15) * 8;
  if (col / 128 >= mx4_groups(k)) return;
  for (int64_t row = (int64_t)blockIdx.y * 4 + (lane >> 4); row < m; row += (int64_t)gridDim.y * 4) {
    const int valid = col >= k ? 0 : (k - col >= 8 ? 8 : (int)(k - col));
    const Raw8<DT> raw = load_raw8<DT>((const typename El<DT>::T*)x + row * ldx, col, valid);
    const uint32_t amax = quad_max(amax8_bits<DT>(raw));
    float v[8];
    widen8<DT>(raw, v);
    if (codes) {
      const uint32_t sb = scale_byte<LQ_E2M1>(amax);
      *(uint32_t*)(codes + mx4_code_at(m, row, col)) = encode_e2m1(v, scale_recip(sb));
      if ((lane & 3) == 0) scales[mx4_scale_at(m, row, col)] = (uint8_t)sb;
    }
    if (ck && col < ckpt_pitch(k)) {
      const uint32_t sb = scale_byte<F>(amax);
      *(uint2*)(ck + row * ckpt_pitch(k) + col) = encode8<F>(v, scale_recip(sb));
      if ((lane & 3) == 0) cks[row * ckpt_scale_pitch(k) + col / 32] = (uint8_t)sb;
    }
  }
}

// ---------------------------------------------------------------- product
// y = x W^T on the matrix cores: v_mfma_scale_f32_32x32x64_f8f6f4 takes 32
// E2M1 codes and a scale byte per lane, so a lane's operand is exactly one
// stored block and nothing is converted. The contraction's order is free as
// long as both operands agree: within a step of 128, half h of a wave takes
// blocks 2h and 2h+1, whose scales are two neighbouring bytes.
//
// A workgroup of 2 x 2 waves makes (64 FM) x (64 FN) tiles, 32 FM x 32 FN per
// wave, one after the other. Codes and scales go from memory to LDS without
// passing through registers, a step of 128 of the contraction (64 bytes a row)
// at a time into a ring of four stages, three of them in flight; the transfers
// run on across the end of a tile, so the next tile starts with its first steps
// in LDS, and a tile's results leave through a part of LDS of their own.
//
// 8192 x 4096 x 11008 163 us (4.5 PFLOP/s), 8192 x 8192 x 8192 271 us (4.1), 8192
// x 11008 x 4096 177 to 200 us (3.7 to 4.2; 5.4 tiles a compute unit take 6 turns,
// and each turn writes 32 MB). A loop of nothing but these products on random
// operands reaches 5.8 PFLOP/s at 1.4 to 1.7 GHz, where power holds it; here the
// matrix cores are busy 46% of the cycles at 1.9 GHz: what is missing is the last
// turn, and work beside a tile's end (6 of its 33 us).
// 256 x 256 tiles read each operand half as often as 128 x 128 ones; those, and 64
// x 64, are for products of few tiles (2048 x 4096 x 4096: 23 us against 30).
constexpr int kStages = 4;
// A row's four 16-byte units are stored in the order u ^ (row / 4 & 3): the 16
// lanes that the LDS serves at a time (0-3, 12-15, 20-27 and so on) then read
// 16 different units of 256 bytes.
__device__ __forceinline__ int swizzled(int row, int unit) { return (unit ^ (row >> 2 & 3)) * 16; }

// A stretch of memory for buffer loads: what lies past its end reads as zero.
__device__ __forceinline__ v4i stretch(const uint8_t* p, uint32_t bytes) {
  const uint64_t b = (uint64_t)(uintptr_t)p;
  const v4i d = {(int)__builtin_amdgcn_readfirstlane((uint32_t)b), (int)__builtin_amdgcn_readfirstlane((uint32_t)(b >> 32)),
                 (int)__builtin_amdgcn_readfirstlane(bytes), 0x00020000};
  return d;
}
// 16 bytes per lane from the stretch's byte `offset` on to LDS address lds + 16 * lane.
__device__ __forceinline__ void to_lds(v4i from, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(__builtin_amdgcn_readfirstlane(lds)),
               "v"(offset), "s"(from)
               : "memory");
}
// Waits until all but the wave's N newest transfers (and stores) are done and
// its LDS reads have returned, then for the workgroup.
template <int N>
__device__ __forceinline__ void drain_and_meet() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

template <int FM, int FN>
struct ProductLds {
  static constexpr int kOut = FM * FN >= 16 ? 4096 : 2048;   // bytes a wave turns results through
  __attribute__((aligned(128))) uint8_t x[kStages][64 * FM][64];
  __attribute__((aligned(128))) uint8_t w[kStages][64 * FN][64];
  __attribute__((aligned(128))) uint8_t s[kStages][2][256][4];   // scales of x, of W
  __attribute__((aligned(128))) uint8_t out[4][kOut];
};

// Tile i of an XCD's share. Consecutive workgroups go round-robin to the 8
// XCDs, each with an L2 of its own: an XCD takes a contiguous run of the tiles,
// ordered in bands of 4 rows of tiles, so that the 32 tiles it works on at a
// time share 4 row blocks of x and 8 of W.
__device__ __forceinline__ void tile_at(uint32_t t, uint32_t tm, uint32_t tn, uint32_t& row, uint32_t& col) {
  const uint32_t band = t / (4 * tn), first = band * 4, high = tm - first < 4 ? tm - first : 4, in = t - band * 4 * tn;
  row = __builtin_amdgcn_readfirstlane(first + in % high);
  col = __builtin_amdgcn_readfirstlane(in / high);
}

template <int OUT, int FM, int FN>
__global__ __launch_bounds__(256, FM * FN >= 16 ? 1 : 2) void k_mx4_product(const uint8_t* x, const uint8_t* xs, const uint8_t* w, const uint8_t* ws,
                                                        int64_t m, int64_t n, int64_t k, void* y, int64_t ldy,
                                                        uint32_t tm, uint32_t tn, uint32_t parts, int part_groups) {
  typedef typename El<OUT>::T T;
  constexpr int BM = 64 * FM, BN = 64 * FN;
  __shared__ ProductLds<FM, FN> lds;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 31, h = lane >> 5, wm = wave >> 1, wn = wave & 1;

  // This workgroup's tiles: its XCD's share, every `slots`-th from its own on.
  // With the contraction in parts, part p of a tile is a tile of its own, whose
  // sums go to plane p of y.
  const uint32_t total = tm * tn * parts, xcd = blockIdx.x % 8, slots = (gridDim.x - xcd + 7) / 8;
  const uint32_t per = total / 8, more = total % 8, begin = xcd * per + (xcd < more ? xcd : more);
  const uint32_t end = begin + per + (xcd < more ? 1 : 0);
  uint32_t tile = begin + blockIdx.x / 8;
  if (tile >= end) return;

  // A tile takes at least four steps, so that the transfers reach into the next
  // tile only; steps past the contraction's end read zeros.
  const int groups = (int)mx4_groups(k), steps = part_groups < 4 ? 4 : part_groups;
  struct Tile {
    const uint8_t *x, *w, *xs, *ws;   // codes and scales of its first rows, in group 0
    uint32_t rows, cols;              // that exist, at most BM and BN; 0: no tile
    int deep;                         // groups of the contraction
  };
  auto place = [&](uint32_t row, uint32_t col, uint32_t part, bool real) {
    const int64_t r0 = (int64_t)row * BM, c0 = (int64_t)col * BN, g0 = (int64_t)part * part_groups;
    Tile t;
    t.x = x + (g0 * m + r0) * 64;
    t.w = w + (g0 * n + c0) * 64;
    t.xs = xs + (g0 * mx4_scale_rows(m) + r0) * 4;
    t.ws = ws + (g0 * mx4_scale_rows(n) + c0) * 4;
    t.deep = groups - g0 < part_groups ? groups - (int)g0 : part_groups;
    t.rows = real ? (uint32_t)(m - r0 < BM ? m - r0 : BM) : 0;
    t.cols = real ? (uint32_t)(n - c0 < BN ? n - c0 : BN) : 0;
    return t;
  };
  uint32_t trow, tcol, tpart, nrow, ncol, npart;
  auto tile_of = [&](uint32_t t, uint32_t& row, uint32_t& col, uint32_t& part) {
    part = parts == 1 ? 0 : __builtin_amdgcn_readfirstlane(t / (tm * tn));
    tile_at(t - part * (tm * tn), tm, tn, row, col);
  };
  tile_of(tile, trow, tcol, tpart);
  Tile now = place(trow, tcol, tpart, true), next;
  uint32_t following;
  auto look_ahead = [&] {
    following = tile + slots;
    tile_of(following < end ? following : tile, nrow, ncol, npart);
    next = place(nrow, ncol, npart, following < end);
  };
  look_ahead();

  // One transfer is 16 rows of codes, or the scales of up to 256 rows (even
  // waves fetch those of x, odd ones those of W).
  constexpr int kFetches = FM + FN + 1;
  uint32_t xo[FM], wo[FN];
#pragma unroll
  for (int i = 0; i < FM; i++) {
    const uint32_t t = (wave * FM + i) * 16 + (lane >> 2);
    xo[i] = t * 64 + swizzled(t, lane & 3);
  }
#pragma unroll
  for (int i = 0; i < FN; i++) {
    const uint32_t t = (wave * FN + i) * 16 + (lane >> 2);
    wo[i] = t * 64 + swizzled(t, lane & 3);
  }
  auto lds_at = [](const void* p) { return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)p; };
  const uint32_t lx = lds_at(&lds.x[0][wave * FM * 16][0]), lw = lds_at(&lds.w[0][wave * FN * 16][0]), ls = lds_at(&lds.s[0][wave & 1][0][0]);
  const int64_t xgroup = m * 64, wgroup = n * 64, sgroup = mx4_scale_rows(wave & 1 ? n : m) * 4;
  // The step whose transfers come next: what is left of its rows in memory.
  struct Cursor {
    const uint8_t *x, *w, *s;
    int t, deep;
  } at = {now.x, now.w, wave & 1 ? now.ws : now.xs, 0, now.deep};
  uint32_t xbytes = now.rows * 64, wbytes = now.cols * 64, sbytes = ((wave & 1 ? now.cols : now.rows) + 3) / 4 * 16;
  v4i fx, fw, fs;
  auto point_x = [&] { fx = stretch(at.x, at.t < at.deep ? xbytes : 0); };
  auto point_w = [&] { fw = stretch(at.w, at.t < at.deep ? wbytes : 0); };
  auto point_s = [&] { fs = stretch(at.s, at.t < at.deep ? sbytes : 0); };
  // (the transfers run four steps ahead: past the end of this tile, they are the next one's)
  auto advance = [&] {
    const bool wrap = ++at.t == steps;
    at.x = wrap ? next.x : at.x + xgroup;
    at.w = wrap ? next.w : at.w + wgroup;
    at.s = wrap ? (wave & 1 ? next.ws : next.xs) : at.s + sgroup;
    xbytes = wrap ? next.rows * 64 : xbytes;
    wbytes = wrap ? next.cols * 64 : wbytes;
    sbytes = wrap ? ((wave & 1 ? next.cols : next.rows) + 3) / 4 * 16 : sbytes;
    at.t = wrap ? 0 : at.t;
    at.deep = wrap ? next.deep : at.deep;
  };
  // Transfer f into stage `st`.
  auto fetch = [&](int st, int f) {
    if (f < FM) to_lds(fx, xo[f], lx + st * BM * 64 + f * 1024);
    else if (f < FM + FN) to_lds(fw, wo[f - FM], lw + st * BN * 64 + (f - FM) * 1024);
    else to_lds(fs, lane * 16, ls + st * 2048);
  };

  // Operands of half a step: 32-row fragments of x and W; the scales of a step.
  struct Operands { v4i x[FM], w[FN]; };
  struct Scales { int x[FM], w[FN]; };
  Operands A, B;
  Scales E, F;
  auto read = [&](int st, int s, Operands& o, int f) {
    const int u = swizzled(r, 2 * h + s);
    if (f < FM) o.x[f] = *(const v4i*)&lds.x[st][wm * 32 * FM + f * 32 + r][u];
    else o.w[f - FM] = *(const v4i*)&lds.w[st][wn * 32 * FN + (f - FM) * 32 + r][u];
  };
  auto read_scale = [&](int st, Scales& e, int f) {
    if (f < FM) e.x[f] = *(const uint16_t*)&lds.s[st][0][wm * 32 * FM + f * 32 + r][2 * h];
    else e.w[f - FM] = *(const uint16_t*)&lds.s[st][1][wn * 32 * FN + (f - FM) * 32 + r][2 * h];
  };
  v16f acc[FM][FN];
  // One half's products; `between` runs after each.
  auto multiply = [&](auto which, const Operands& o, auto between) {
    constexpr int s = decltype(which)::value;
#pragma unroll
    for (int i = 0; i < FM; i++)
#pragma unroll
      for (int j = 0; j < FN; j++) {
        const v8i P = {o.w[j][0], o.w[j][1], o.w[j][2], o.w[j][3], 0, 0, 0, 0};
        const v8i Q = {o.x[i][0], o.x[i][1], o.x[i][2], o.x[i][3], 0, 0, 0, 0};
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(P, Q, acc[i][j], 4, 4, s, E.w[j], s, E.x[i]);
        __builtin_amdgcn_sched_barrier(0);
        between(i * FN + j);
        __builtin_amdgcn_sched_barrier(0);
      }
  };
  typedef std::integral_constant<int, 0> First;
  typedef std::integral_constant<int, 1> Second;

  // Three steps, and the first transfers of a fourth (the rest run under the
  // first products).
  constexpr int early = (kFetches + 1) / 2, late = kFetches - early;
#pragma unroll
  for (int t = 0; t < 4; t++) {
    if (t > 0) advance();
    point_x();
    point_w();
    point_s();
#pragma unroll
    for (int f = 0; f < (t < 3 ? kFetches : early); f++) fetch(t, f);
  }
  drain_and_meet<2 * kFetches + early>();
#pragma unroll
  for (int f = 0; f < FM + FN; f++) {
    read(0, 0, A, f);
    read_scale(0, E, f);
  }
  int st = 0;
  for (;;) {
#pragma unroll
    for (int i = 0; i < FM; i++)
#pragma unroll
      for (int j = 0; j < FN; j++)
#pragma unroll
        for (int e = 0; e < 16; e++) acc[i][j][e] = 0.0f;
    // A step. Under the first half's products the second half's operands are
    // read, and the last of the transfers into the previous stage run. Then the
    // next step has landed (two more are on their way) and nobody reads this
    // stage any more: under the second half's products the next step's first
    // operands are read and the transfers into this stage begin. Reads and
    // transfers go one between two products: issued together they stall the
    // wave, and the matrix core with it, until the memory pipes have taken them
    // all. The scheduling barriers keep them there: left alone, the compiler
    // moves all products below the last wait.
    for (int t = 0; t < steps; t++) {
      constexpr int per = FM * FN, reads = FM + FN;
      const int before = (st + 3) & 3, after = (st + 1) & 3;
      multiply(First(), A, [&](int done) {
#pragma unroll
        for (int f = 0; f < reads; f++)
          if (f * per / (2 * reads) == done) read(st, 1, B, f);
#pragma unroll
        for (int f = 0; f < late; f++)
          if (per / 2 + f * (per - per / 2) / (late + 1) == done) fetch(before, early + f);
        if (done == per - 1) {
          advance();
          point_x();
          point_w();
          point_s();
        }
      });
      drain_and_meet<2 * kFetches>();
      multiply(Second(), B, [&](int done) {
#pragma unroll
        for (int f = 0; f < reads; f++)
          if (f * per / (2 * reads) == done) {
            read(after, 0, A, f);
            read_scale(after, F, f);
          }
#pragma unroll
        for (int f = 0; f < early; f++)
          if (per / 2 + f * (per - per / 2) / early == done) fetch(st, f);
      });
      E = F;
      st = after;
    }

    // A lane holds row r of a 32 x 32 block of y, columns 8q + 4h .. + 3: each
    // wave turns 32 rows x CW columns at a time through LDS into row stretches.
    // (The sums are pinned to accumulation registers up to here: the conversions
    // below want ordinary ones, and the allocator would move the sums there and
    // spill the rest. The lane's number is made opaque: every address of this part would
    // otherwise be kept in registers through the whole loop over the tiles.)
    constexpr int kRow = ProductLds<FM, FN>::kOut / 32, CW = kRow / (int)sizeof(T), V = 16 / (int)sizeof(T), units = CW / V;
#pragma unroll
    for (int i = 0; i < FM; i++)
#pragma unroll
      for (int j = 0; j < FN; j++) asm volatile("" : "+a"(acc[i][j]));
    int l = lane;
    asm volatile("" : "+v"(l));
    uint8_t* mine = lds.out[wave];
    uint8_t* const put = mine + (l & 31) * kRow;
    const int turn = (l & 31) >> 1, part = (l >> 5) * 4 * (int)sizeof(T);
    const int64_t row0 = (int64_t)trow * BM + wm * 32 * FM, col0 = (int64_t)tcol * BN + wn * 32 * FN;
    const int rr = l / units, cc = l % units;
    T* const out = (T*)y + (tpart * m + row0 + rr) * ldy + col0 + cc * V;
    const int rows_left = (int)(m - row0 < 32 * FM ? m - row0 : 32 * FM) - rr, cols_left = (int)(n - col0 < 32 * FN ? n - col0 : 32 * FN) - cc * V;
#pragma unroll
    for (int i = 0; i < FM; i++)
#pragma unroll
      for (int c = 0; c < 32 * FN / CW; c++) {
#pragma unroll
        for (int g = 0; g < CW / 8; g++) {
          const int j = (c * CW + g * 8) / 32, q = (c * CW + g * 8) % 32 / 8;
          T v[4];
#pragma unroll
          for (int e = 0; e < 4; e++) v[e] = narrow<OUT>(acc[i][j][4 * q + e]);
          const int at = g * 8 * (int)sizeof(T) + part;
          __builtin_memcpy(__builtin_assume_aligned(put + (((at >> 4) ^ turn) & (units - 1)) * 16 + (at & 15), 4 * sizeof(T)), v, sizeof(v));
        }
        asm volatile("" ::: "memory");
#pragma unroll
        for (int g = 0; g < units / 2; g++) {
          constexpr int rows = 64 / units;   // a store instruction's
          T v[V];
          __builtin_memcpy(v, __builtin_assume_aligned(mine + (g * rows + rr) * kRow + ((cc ^ ((g * rows + rr) >> 1)) & (units - 1)) * 16, 16), 16);
          if (i * 32 + g * rows < rows_left && c * CW < cols_left) {
            T* o = out + (int64_t)(i * 32 + g * rows) * ldy + c * CW;
            if (cols_left - c * CW >= V) {
              store16(o, v);
            } else {
#pragma unroll
              for (int e = 0; e < V; e++)
                if (c * CW + e < cols_left) o[e] = v[e];
            }
          }
        }
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
      }
    if (following >= end) break;
    tile = following;
    trow = nrow;
    tcol = ncol;
    tpart = npart;
    now = next;
    look_ahead();
  }
  // (the transfers after the last step wrote zeros into LDS: they end before it is given away)
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// ---------------------------------------------------------------- a few rows
// Up to 16 CT rows of x, 64 at most: the call is bound by reading W once. Eight waves of a
// workgroup share 16 R rows of W, each taking a run of the contraction's groups
// with v_mfma_scale_f32_16x16x128_f8f6f4, whose operand of 16 rows and 128
// columns is one kilobyte of W as it is stored; their sums meet in LDS. With SRC
// a float type (up to kFewRows rows) every workgroup quantises x itself, a block
// a thread, into LDS while its first reads of W are on their way: a launch of
// its own for x would cost a quarter of the call. Otherwise x is an MX4 operand.
//
// With W in memory, call after call in a graph: 1 x 4096 x 4096 4.3 us, 1 x 11008 x
// 4096 7.4, 1 x 8192 x 8192 9.9, 8 x 11008 x 4096 9.0: 2.6 us, which the smallest
// call takes, and W's bytes at 5.1 TB/s, the rate of a large copy. Asked for after
// W, x came behind all of it: 4.9, 7.7, 10.2 and 10.5 us. Loads of twice as many
// groups in flight cost the registers of a third of the waves: 8.6 for the 7.7.
typedef float v4f __attribute__((ext_vector_type(4)));
constexpr int kOperand = -1;
constexpr int kFewWaves = 8;

// One block of x as it is stored, `valid` of whose 32 elements exist; its codes
// and scale byte.
template <int SRC>
struct Block { typename El<SRC>::T t[32]; };
template <int SRC>
__device__ __forceinline__ Block<SRC> load_block(const typename El<SRC>::T* p, int valid) {
  Block<SRC> b;
  if (valid >= 32) {
    __builtin_memcpy(b.t, p, sizeof(b.t));
  } else {
#pragma unroll
    for (int i = 0; i < 32; i++) b.t[i] = i < valid ? p[i] : (typename El<SRC>::T)0;
  }
  return b;
}
template <int SRC>
__device__ __forceinline__ v4i quantise_block(const Block<SRC>& block, uint32_t& scale) {
  float v[32];
#pragma unroll
  for (int i = 0; i < 32; i++) v[i] = widen<SRC>(block.t[i]);
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 32; i++) {
    const uint32_t b = __float_as_uint(v[i]) & 0x7FFFFFFFu;
    amax = amax > b ? amax : b;
  }
  scale = scale_byte<LQ_E2M1>(amax);
  const float r = scale_recip(scale);
  v4i out;
#pragma unroll
  for (int i = 0; i < 4; i++) out[i] = (int)encode_e2m1(v + 8 * i, r);
  return out;
}

template <int SRC, int OUT, int R, int CT>
__global__ __launch_bounds__(64 * kFewWaves) void k_mx4_few(const void* x, int64_t ldx, const uint8_t* xs, const uint8_t* w,
                                                            const uint8_t* ws, int64_t m, int64_t n, int64_t k, void* y,
                                                            int64_t ldy) {
  typedef typename El<OUT>::T T;
  constexpr bool own = SRC != kOperand;
  __shared__ v4f sums[kFewWaves][R * CT][64];
  __shared__ v4i xcodes[own ? kFewBlocks : 1];
  __shared__ uint8_t xscales[own ? kFewBlocks : 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int64_t row0 = (int64_t)blockIdx.x * 16 * R;
  const int groups = (int)mx4_groups(k), per = (groups + kFewWaves - 1) / kFewWaves;
  const int begin = wave * per, end = begin + per < groups ? begin + per : groups;
  const int64_t wstep = mx4_scale_rows(n) * 4, xstep = mx4_scale_rows(m) * 4;
  int64_t wrow[R];   // rows past the last are the last again
#pragma unroll
  for (int i = 0; i < R; i++) wrow[i] = row0 + i * 16 + r < n ? row0 + i * 16 + r : n - 1;

  constexpr int U = CT == 4 ? 2 : 4;   // groups whose reads are in flight together (4 of 64 rows' would leave one wave on a SIMD)
  struct Reads {
    v4i wc[U][R], xc[own ? 1 : U][CT];
    uint32_t we[U][R], xe[own ? 1 : U][CT];
  };
  auto load = [&](Reads& a, int g0) {
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int g = g0 + u < groups ? g0 + u : groups - 1;
#pragma unroll
      for (int i = 0; i < R; i++) {
        a.wc[u][i] = *(const v4i*)(w + (g * n + wrow[i]) * 64 + q * 16);
        a.we[u][i] = ws[g * wstep + wrow[i] * 4 + q];
      }
      if constexpr (!own) {
#pragma unroll
        for (int c = 0; c < CT; c++) {
          const int64_t at = c * 16 + r < m ? c * 16 + r : m - 1;
          a.xc[u][c] = *(const v4i*)((const uint8_t*)x + (g * m + at) * 64 + q * 16);
          a.xe[u][c] = xs[g * xstep + at * 4 + q];
        }
      }
    }
  };
  Reads a, b;
  if constexpr (own) {
    // loads return in the order they were asked for: a thread's first two blocks of x, then W, whose way here hides the rest
    const int blocks = groups * 4, all = (int)m * blocks;
    auto block = [&](int i) {
      const int row = i / blocks, col = (i - row * blocks) * 32;
      return load_block<SRC>((const typename El<SRC>::T*)x + row * ldx + col, k - col < 32 ? (int)(k - col) : 32);
    };
    auto keep = [&](int i, const Block<SRC>& v) {
      uint32_t e;
      xcodes[i] = quantise_block<SRC>(v, e);
      xscales[i] = (uint8_t)e;
    };
    constexpr int kThreads = 64 * kFewWaves;
    int i = threadIdx.x;
    Block<SRC> mine, second;
    if (i < all) mine = block(i);
    if (i + kThreads < all) second = block(i + kThreads);
    asm volatile("" ::: "memory");
    if (begin < end) load(a, begin);
    if (i < all) keep(i, mine);
    if (i + kThreads < all) keep(i + kThreads, second);
    for (i += 2 * kThreads; i < all; i += kThreads) keep(i, block(i));
    __syncthreads();
  } else {
    if (begin < end) load(a, begin);
  }
  v4f acc[R][CT];
#pragma unroll
  for (int i = 0; i < R; i++)
#pragma unroll
    for (int c = 0; c < CT; c++) acc[i][c] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  for (int g0 = begin; g0 < end; g0 += U) {
    if (g0 + U < end) load(b, g0 + U);
#pragma unroll
    for (int u = 0; u < U; u++)
      if (g0 + u < end) {
#pragma unroll
        for (int c = 0; c < CT; c++) {
          v4i xc = {0, 0, 0, 0};
          uint32_t xe = 0;
          if constexpr (own) {
            if (r < m) {
              const int at = (r * groups + g0 + u) * 4 + q;
              xc = xcodes[at];
              xe = xscales[at];
            }
          } else {
            xc = a.xc[u][c];
            xe = a.xe[u][c];
          }
#pragma unroll
          for (int i = 0; i < R; i++) {
            const v8i A = {a.wc[u][i][0], a.wc[u][i][1], a.wc[u][i][2], a.wc[u][i][3], 0, 0, 0, 0};
            const v8i B = {xc[0], xc[1], xc[2], xc[3], 0, 0, 0, 0};
            acc[i][c] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, acc[i][c], 4, 4, 0, (int)a.we[u][i], 0, (int)xe);
          }
        }
      }
    a = b;
  }
#pragma unroll
  for (int i = 0; i < R; i++)
#pragma unroll
    for (int c = 0; c < CT; c++) sums[wave][i * CT + c][lane] = acc[i][c];
  __syncthreads();
  // A lane's four sums are columns 4q .. 4q + 3 of one row of y.
  for (int t = wave; t < R * CT; t += kFewWaves) {
    v4f s = sums[0][t][lane];
#pragma unroll
    for (int v = 1; v < kFewWaves; v++) s += sums[v][t][lane];
    const int64_t row = t % CT * 16 + r, col = row0 + t / CT * 16 + 4 * q;
    if (row < m) {
      T* o = (T*)y + row * ldy + col;
#pragma unroll
      for (int e = 0; e < 4; e++)
        if (col + e < n) o[e] = narrow<OUT>(s[e]);
    }
  }
}

template <int DT>
hipError_t quantize_dt(int format, const void* x, int64_t m, int64_t k, int64_t ldx, void* codes, void* scales,
                       void* ck, void* cks, hipStream_t s) {
  const dim3 g = matrix_grid((mx4_groups(k) + 3) / 4, m);
  if (lqd::g_plan) return LQ_PLAN(g, 256, "k_mx4_quantize<%d, %d>", DT, format);
  if (format == LQ_INT8)
    hipLaunchKernelGGL((k_mx4_quantize<DT, LQ_INT8>), g, dim3(256), 0, s, x, m, k, ldx, (uint8_t*)codes,
                       (uint8_t*)scales, (uint8_t*)ck, (uint8_t*)cks);
  else
    hipLaunchKernelGGL((k_mx4_quantize<DT, LQ_E4M3>), g, dim3(256), 0, s, x, m, k, ldx, (uint8_t*)codes,
                       (uint8_t*)scales, (uint8_t*)ck, (uint8_t*)cks);
  return hipGetLastError();
}

// One workgroup a compute unit for the 256 x 256 tile (its LDS), more for the
// smaller ones. With parts > 1, y is `parts` planes of m x n.
template <int OUT, int FM, int FN>
hipError_t product_tiled(const void* a, const void* as, const void* w, const void* ws, int64_t m, int64_t n, int64_t k,
                         int parts, int part_groups, void* y, int64_t ldy, hipStream_t s) {
  const int64_t tm = (m + 64 * FM - 1) / (64 * FM), tn = (n + 64 * FN - 1) / (64 * FN), tiles = tm * tn * parts;
  const int64_t most = (int64_t)compute_units() * (int)(163840 / sizeof(ProductLds<FM, FN>));
  const dim3 grid((unsigned)(tiles < most ? tiles : most));
  if (lqd::g_plan) return LQ_PLAN(grid, 256, "k_mx4_product<%d, %d, %d>", OUT, FM, FN);
  hipLaunchKernelGGL((k_mx4_product<OUT, FM, FN>), grid, dim3(256), 0, s,
                     (const uint8_t*)a, (const uint8_t*)as, (const uint8_t*)w, (const uint8_t*)ws, m, n, k, y, ldy,
                     (uint32_t)tm, (uint32_t)tn, (uint32_t)parts, part_groups);
  return hipGetLastError();
}
template <int SRC, int OUT, int CT>
hipError_t few(const void* x, int64_t ldx, const void* xs, const void* w, const void* ws, int64_t m, int64_t n, int64_t k,
               void* y, int64_t ldy, hipStream_t s) {
  // 32 rows of W a workgroup where that leaves one for each compute unit, else 16 (W read from memory, one call after
  // another in a graph: 1 x 8192 x 4096 5.6 us, with 16 rows 6.2; 1 x 11008 x 4096 7.7 or 8.5; 8 x 11008 x 4096 9.2 or
  // 11.5; 24 x 8192 x 4096 9.4 or 11.7; but 1 x 4096 x 4096 4.6 or 4.3, 1 x 4096 x 11008 9.3 or 7.6, 24 x 4096 x 4096
  // 8.7 or 7.8)
  const int r = CT < 4 && n >= 32 * (int64_t)compute_units() ? 2 : 1;
  const dim3 grid((unsigned)((n + 16 * r - 1) / (16 * r)));
  if (lqd::g_plan) return LQ_PLAN(grid, 64 * kFewWaves, "k_mx4_few<%d, %d, %d, %d>", SRC, OUT, r, CT);
  if (r == 2) {
    hipLaunchKernelGGL((k_mx4_few<SRC, OUT, CT < 4 ? 2 : 1, CT>), grid, dim3(64 * kFewWaves), 0, s, x, ldx,
                       (const uint8_t*)xs, (const uint8_t*)w, (const uint8_t*)ws, m, n, k, y, ldy);
  } else {
    hipLaunchKernelGGL((k_mx4_few<SRC, OUT, 1, CT>), grid, dim3(64 * kFewWaves), 0, s, x, ldx,
                       (const uint8_t*)xs, (const uint8_t*)w, (const uint8_t*)ws, m, n, k, y, ldy);
  }
  return hipGetLastError();
}
template <int OUT>
hipError_t few_src(int in_dtype, const void* x, int64_t ldx, const void* w, const void* ws, int64_t m, int64_t n, int64_t k,
                   void* y, int64_t ldy, hipStream_t s) {
  switch (in_dtype) {
    case LQ_F32: return few<LQ_F32, OUT, 1>(x, ldx, nullptr, w, ws, m, n, k, y, ldy, s);
    case LQ_BF16: return few<LQ_BF16, OUT, 1>(x, ldx, nullptr, w, ws, m, n, k, y, ldy, s);
    default: return few<LQ_F16, OUT, 1>(x, ldx, nullptr, w, ws, m, n, k, y, ldy, s);
  }
}

template <int OUT>
hipError_t product_tile(int tile, const void* a, const void* as, const void* w, const void* ws, int64_t m, int64_t n,
                        int64_t k, int parts, int part_groups, void* y, int64_t ldy, hipStream_t s) {
  if (tile == 4) return product_tiled<OUT, 4, 4>(a, as, w, ws, m, n, k, parts, part_groups, y, ldy, s);
  if (tile == 2) return product_tiled<OUT, 2, 2>(a, as, w, ws, m, n, k, parts, part_groups, y, ldy, s);
  return product_tiled<OUT, 1, 1>(a, as, w, ws, m, n, k, parts, part_groups, y, ldy, s);
}
template <int OUT>
hipError_t product_dt(const void* a, const void* as, const void* w, const void* ws, int64_t m, int64_t n, int64_t k,
                      void* y, int64_t ldy, void* planes, hipStream_t s) {
  if (k == 0) return launch_constant(m, n, OUT, nullptr, y, ldy, s);
  if (m <= 16) return few<kOperand, OUT, 1>(a, 0, as, w, ws, m, n, k, y, ldy, s);
  if (m <= 32) return few<kOperand, OUT, 2>(a, 0, as, w, ws, m, n, k, y, ldy, s);
  // Every workgroup reads all of x, 4 times its share of W at 64 rows: worth it with one on a compute unit and not too
  // much of x (W in memory; 64 x 4096 x 4096 9.8 us, in tiles 12.9; 64 x 1024 x 4096 9.4 or 11.4; but 64 x 4096 x 11008
  // 18.2 or 17.2, 64 x 8192 x 8192 24.6 or 19.5)
  if (m <= 64 && n <= 16 * (int64_t)compute_units() && k <= 8192) return few<kOperand, OUT, 4>(a, 0, as, w, ws, m, n, k, y, ldy, s);
  const Split c = split_product(m, n, k, OUT);
  if (c.parts == 1) return product_tile<OUT>(c.tile, a, as, w, ws, m, n, k, 1, c.part, y, ldy, s);
  const hipError_t e = product_tile<LQ_F32>(c.tile, a, as, w, ws, m, n, k, c.parts, c.part, planes, plane_stride(n), s);
  return e != hipSuccess ? e : launch_join(m, n, OUT, c.parts, (const float*)planes, nullptr, y, ldy, s);
}

// y = in, or zeros: what is left of a product over an empty contraction.
template <typename T>
__global__ __launch_bounds__(256) void k_constant(int64_t rows, int64_t cols, const T* in, T* y, int64_t ldy) {
  const int64_t col = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
  if (col >= cols) return;
  for (int64_t row = (int64_t)blockIdx.y * 4 + (threadIdx.x >> 6); row < rows; row += (int64_t)gridDim.y * 4)
    y[row * ldy + col] = in ? in[row * ldy + col] : (T)0;
}

// y = in + the planes' sum, in the planes' order: four columns a lane, a wave's
// on one row.
template <int OUT>
__global__ __launch_bounds__(256) void k_join(int64_t rows, int64_t cols, int parts, const float* planes,
                                              const float* in, void* y, int64_t ldy) {
  const int64_t stride = plane_stride(cols), plane = rows * stride;
  const int64_t col = (int64_t)blockIdx.x * 256 + (threadIdx.x & 63) * 4;
  if (col >= cols) return;
  for (int64_t row = (int64_t)blockIdx.y * 4 + (threadIdx.x >> 6); row < rows; row += (int64_t)gridDim.y * 4) {
    const float* p = planes + row * stride + col;
    float4 s = *(const float4*)p;
#pragma unroll 4
    for (int i = 1; i < parts; i++) {
      const float4 t = *(const float4*)(p + i * plane);
      s.x += t.x;
      s.y += t.y;
      s.z += t.z;
      s.w += t.w;
    }
    const float v[4] = {s.x, s.y, s.z, s.w};
    typename El<OUT>::T* o = (typename El<OUT>::T*)y + row * ldy + col;
    typename El<OUT>::T t[4];
#pragma unroll
    for (int e = 0; e < 4; e++) t[e] = narrow<OUT>(in && col + e < cols ? v[e] + in[row * ldy + col + e] : v[e]);
    if (cols - col >= 4) {
      __builtin_memcpy(o, t, sizeof(t));
    } else {
#pragma unroll
      for (int e = 0; e < 4; e++)
        if (col + e < cols) o[e] = t[e];
    }
  }
}

}  // namespace

hipError_t launch_join(int64_t rows, int64_t cols, int dtype, int parts, const float* planes, const float* in, void* y,
                       int64_t ldy, hipStream_t s) {
  const dim3 g = matrix_grid((cols + 255) / 256, rows);
  if (lqd::g_plan) return LQ_PLAN(g, 256, "k_join<%d>", dtype);
  if (dtype == LQ_F32) hipLaunchKernelGGL((k_join<LQ_F32>), g, dim3(256), 0, s, rows, cols, parts, planes, in, y, ldy);
  else if (dtype == LQ_BF16) hipLaunchKernelGGL((k_join<LQ_BF16>), g, dim3(256), 0, s, rows, cols, parts, planes, in, y, ldy);
  else hipLaunchKernelGGL((k_join<LQ_F16>), g, dim3(256), 0, s, rows, cols, parts, planes, in, y, ldy);
  return hipGetLastError();
}

hipError_t launch_constant(int64_t rows, int64_t cols, int dtype, const void* in, void* y, int64_t ldy, hipStream_t s) {
  const dim3 g = matrix_grid((cols + 63) / 64, rows);
  if (lqd::g_plan) return LQ_PLAN(g, 256, "k_constant<%s>", dtype == LQ_F32 ? "float" : "unsigned short");
  if (dtype == LQ_F32)
    hipLaunchKernelGGL((k_constant<float>), g, dim3(256), 0, s, rows, cols, (const float*)in, (float*)y, ldy);
  else
    hipLaunchKernelGGL((k_constant<uint16_t>), g, dim3(256), 0, s, rows, cols, (const uint16_t*)in, (uint16_t*)y, ldy);
  return hipGetLastError();
}

hipError_t launch_mx4_quantize(int in_dtype, int ckpt_format, const void* x, int64_t m, int64_t k, int64_t ldx,
                               void* codes, void* scales, void* ck, void* cks, hipStream_t s) {
  switch (in_dtype) {
    case LQ_F32: return quantize_dt<LQ_F32>(ckpt_format, x, m, k, ldx, codes, scales, ck, cks, s);
    case LQ_BF16: return quantize_dt<LQ_BF16>(ckpt_format, x, m, k, ldx, codes, scales, ck, cks, s);
    default: return quantize_dt<LQ_F16>(ckpt_format, x, m, k, ldx, codes, scales, ck, cks, s);
  }
}

hipError_t launch_mx4_few(int in_dtype, const void* x, int64_t ldx, const void* w_codes, const void* w_scales, int64_t m,
                          int64_t n, int64_t k, int out_dtype, void* y, int64_t ldy, hipStream_t s) {
  switch (out_dtype) {
    case LQ_F32: return few_src<LQ_F32>(in_dtype, x, ldx, w_codes, w_scales, m, n, k, y, ldy, s);
    case LQ_BF16: return few_src<LQ_BF16>(in_dtype, x, ldx, w_codes, w_scales, m, n, k, y, ldy, s);
    default: return few_src<LQ_F16>(in_dtype, x, ldx, w_codes, w_scales, m, n, k, y, ldy, s);
  }
}

hipError_t launch_mx4_product(const void* a_codes, const void* a_scales, const void* w_codes, const void* w_scales,
                              int64_t m, int64_t n, int64_t k, int out_dtype, void* y, int64_t ldy, void* planes,
                              hipStream_t s) {
  switch (out_dtype) {
    case LQ_F32: return product_dt<LQ_F32>(a_codes, a_scales, w_codes, w_scales, m, n, k, y, ldy, planes, s);
    case LQ_BF16: return product_dt<LQ_BF16>(a_codes, a_scales, w_codes, w_scales, m, n, k, y, ldy, planes, s);
    default: return product_dt<LQ_F16>(a_codes, a_scales, w_codes, w_scales, m, n, k, y, ldy, planes, s);
  }
}

}  // namespace lql
