// lq_rmsnorm.hip — root-mean-square norm with the residual's addition before it and
// an 8-bit checkpoint of its result, and its backward pass:
//
//   h = x + r    rs = 1 / sqrt(mean(h^2) + eps)    n = h rs    y = n w
//   g = dy w     dx = dh + rs (g - n mean(g n))    dw = dw_in + sum over rows of dy n
//
// (forward, n is the quotient to the nearest; backward, the product with the rounded rs
// that the forward pass keeps)
//
// h is the rounded sum, as the residual stream keeps it, in both passes; the
// checkpoint is of the rounded y, whether y is written or not: it holds what the
// checkpoint of a layer called on y would. Sums are in binary32, of a row whose squares
// leave its range times a power of two.
//
// Both passes read and write each matrix once and are bound by memory: a row stays
// in the registers of T threads, V times eight elements each, from its load to its
// last store, and the next row's loads are on their way meanwhile. 8192 x 4096 bf16:
// forward with the residual, h, y and the checkpoint 58 us (5.2 TB/s of what it reads and
// writes), backward 55.5 us (4.8 TB/s; dw's planes are the rest); a copy of 1 GiB reaches
// 5.2 TB/s.
#include "lq_linear.h"

namespace lql {
namespace {

// Sum over a wave, the same in every lane: within rows of 16 by DPP, then the four rows.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_add<0xB1>(v);    // quad_perm [1,0,3,2]
  v = dpp_add<0x4E>(v);    // quad_perm [2,3,0,1]
  v = dpp_add<0x141>(v);   // row_half_mirror
  v = dpp_add<0x140>(v);   // row_mirror
  const int b = __float_as_int(v);
  return (__int_as_float(__builtin_amdgcn_readlane(b, 0)) + __int_as_float(__builtin_amdgcn_readlane(b, 16))) +
         (__int_as_float(__builtin_amdgcn_readlane(b, 32)) + __int_as_float(__builtin_amdgcn_readlane(b, 48)));
}

// T threads share a row; a workgroup has one row at a time, or four of 64 threads.
template <int T>
struct Shape {
  static constexpr int threads = T < 256 ? 256 : T, rows = threads / T, waves = T / 64;
};

// A thread's row of the workgroup's, the same over a wave.
template <int T>
__device__ __forceinline__ int own_row() {
  return T == 64 ? __builtin_amdgcn_readfirstlane(threadIdx.x / 64) : 0;
}

// The sum over a row's threads. `turn` alternates from call to call: a wave that is a
// call ahead writes the other slots, and with the barrier of that call everyone has
// read these.
template <int T>
__device__ __forceinline__ float row_sum(float v, float (*slots)[16], int turn) {
  v = wave_sum(v);
  if constexpr (T == 64) return v;
  constexpr int waves = Shape<T>::waves;
  if ((threadIdx.x & 63) == 0) slots[turn][threadIdx.x >> 6] = v;
  __syncthreads();
  float s = slots[turn][0];
#pragma unroll
  for (int i = 1; i < waves; i++) s += slots[turn][i];
  return s;
}

// Eight elements as they lie in memory, in words, from column col on; zeros past the
// row's end. There the row's last eight are loaded and moved down: loads one by one
// take a register and an address each, for all of a thread's units at a time.
template <int DT>
struct Words { uint32_t w[2 * El<DT>::bytes]; };
template <int DT>
__device__ __forceinline__ Words<DT> load_words(const void* row, int col, int cols) {
  typedef typename El<DT>::T E;
  const E* p = (const E*)row;
  constexpr int N = 2 * El<DT>::bytes;
  Words<DT> r = {};
  if (col >= cols) return r;
  const int past = col + 8 - cols;   // of the eight
  if (cols >= 8) {
    __builtin_memcpy(r.w, p + (past > 0 ? cols - 8 : col), sizeof(r.w));
    if (past > 0) {
#pragma unroll
      for (int by = 4; by >= 1; by /= 2) {
        Words<DT> m;
#pragma unroll
        for (int k = 0; k < N; k++) {
          constexpr int size = (int)sizeof(E);
          const int words = by * size / 4;
          if (by * size >= 4) m.w[k] = k + words < N ? r.w[(k + words) % N] : 0;
          else m.w[k] = __builtin_amdgcn_alignbit(k + 1 < N ? r.w[(k + 1) % N] : 0, r.w[k], 16);
        }
        if (past & by) r = m;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 7; i++)
      if (i < cols) {   // (col is 0)
        uint32_t b = 0;
        __builtin_memcpy(&b, p + i, sizeof(E));
        r.w[i * (int)sizeof(E) / 4] |= b << (8 * (i * (int)sizeof(E) % 4));
      }
  }
  return r;
}
template <int DT>
__device__ __forceinline__ Raw8<DT> raw(const Words<DT>& r) {
  Raw8<DT> t;
  __builtin_memcpy(t.t, r.w, sizeof(t.t));
  return t;
}
// The weights of eight elements: in the matrices' type or binary32; zero past the row.
template <int DT>
__device__ __forceinline__ void load_unit(const void* w, bool wide, int col, int cols, float out[8]) {
  if (wide) widen8<LQ_F32>(raw<LQ_F32>(load_words<LQ_F32>(w, col, cols)), out);
  else widen8<DT>(raw<DT>(load_words<DT>(w, col, cols)), out);
}
template <int DT>
__device__ __forceinline__ void hide(Words<DT>& r) {
#pragma unroll
  for (int i = 0; i < (int)(sizeof(r.w) / 4); i++) asm volatile("" : "+v"(r.w[i]));
}

// The root of a row's mean square (with eps), and its reciprocal, from the sum of the squares.
// Where binary32 cannot hold that sum as it is, infinite, as of finite values from about
// 2^57 on, or so small (without an eps beside it) that squares get lost below the subnormal
// numbers, it is taken anew of the row times a power of two: 2^-72 leaves the largest
// values' squares below 2^112, 2^96 the smallest ones' above 2^-106. A row that holds an
// infinity or a NaN gets a NaN, and is NaN throughout.
// (The sum is the same in all of a row's threads, and so is the way that they take. `slots`
// is this call's alone: the next row's first sum, whose barrier everyone has to pass, is
// between its reads and the next call's writes.)
struct Root { float root, rs; };
template <int DT, int T, int V>
__device__ __forceinline__ Root root_of(const Raw8<DT> (&h)[V], float sum, float cols, float eps, float (*slots)[16]) {
  const bool low = sum < 0x1p-100f && eps < 0x1p-90f, high = !(sum + eps < __builtin_inff());
  if (__builtin_expect(!low && !high, 1)) {
    const float root = sqrtf(sum / cols + eps);
    return {root, 1.0f / root};
  }
  const float power = low ? 0x1p96f : 0x1p-72f;
  float again = 0.0f;
#pragma unroll
  for (int c = 0; c < V; c++) {
    float v[8];
    widen8<DT>(h[c], v);
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const float s = v[i] * power;
      again = __builtin_fmaf(s, s, again);
    }
  }
  again = row_sum<T>(again, slots, 0);
  if (!(again < __builtin_inff())) again = __builtin_nanf("");
  const float root = sqrtf(again / cols + eps * power * power);
  return {root * (low ? 0x1p-96f : 0x1p72f), power / root};
}

template <int DT, int F, int T, int V>
__global__ __launch_bounds__(Shape<T>::threads) void k_rmsnorm(const NormArgs a) {
  typedef typename El<DT>::T E;
  __shared__ float slots[2][16], more_slots[1][16];
  const int lane = T == 64 ? threadIdx.x & 63 : threadIdx.x;
  const int cols = (int)a.cols;
  int valid[V];
#pragma unroll
  for (int c = 0; c < V; c++) {
    const int left = cols - (c * T + lane) * 8;
    valid[c] = left <= 0 ? 0 : (left >= 8 ? 8 : left);
  }
  const int64_t step = (int64_t)gridDim.x * Shape<T>::rows, pitch = ckpt_pitch(a.cols);
  int64_t row = (int64_t)blockIdx.x * Shape<T>::rows + own_row<T>();
  Words<DT> x[V], r[V];
  auto load = [&](int64_t at) {
#pragma unroll
    for (int c = 0; c < V; c++) x[c] = load_words<DT>((const E*)a.x + at * a.ldx, (c * T + lane) * 8, cols);
    if (a.r) {
#pragma unroll
      for (int c = 0; c < V; c++) r[c] = load_words<DT>((const E*)a.r + at * a.ldr, (c * T + lane) * 8, cols);
    }
  };
  if (row < a.rows) load(row);
  float w[V][8];
#pragma unroll
  for (int c = 0; c < V; c++) load_unit<DT>(a.w, a.wide, (c * T + lane) * 8, cols, w[c]);
  // (rows of 256 threads and more: the whole workgroup leaves the loop together)
  for (int turn = 0; row < a.rows; row += step, turn ^= 1) {
    Raw8<DT> h[V];
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < V; c++) {
      h[c] = raw<DT>(x[c]);
      if (a.r) {
        const Raw8<DT> more = raw<DT>(r[c]);
#pragma unroll
        for (int i = 0; i < 8; i++) h[c].t[i] = narrow<DT>(widen<DT>(h[c].t[i]) + widen<DT>(more.t[i]));
      }
      float v[8];
      widen8<DT>(h[c], v);
#pragma unroll
      for (int i = 0; i < 8; i++) sum = __builtin_fmaf(v[i], v[i], sum);
    }
    if (row + step < a.rows) load(row + step);
    if (a.h) {
#pragma unroll
      for (int c = 0; c < V; c++) {
        float v[8];
        widen8<DT>(h[c], v);
        store8<DT>((E*)a.h + row * a.ldh, (int64_t)(c * T + lane) * 8, valid[c], v);
      }
    }
    const auto [root, rs] = root_of<DT, T, V>(h, row_sum<T>(sum, slots, turn), (float)a.cols, a.eps, more_slots);
    if (a.rs && lane == 0) a.rs[row] = rs;
#pragma unroll
    for (int c = 0; c < V; c++) {
      const int64_t col = (int64_t)(c * T + lane) * 8;
      float v[8];
      widen8<DT>(h[c], v);
      Raw8<DT> y;
#pragma unroll
      for (int i = 0; i < 8; i++) {
        // h / root to the nearest: the product with rs, whose own rounding it has, and what that leaves of h times rs
        float n = v[i] * rs;
        n = __builtin_fmaf(__builtin_fmaf(-n, root, v[i]), rs, n);
        y.t[i] = narrow<DT>(n * w[c][i]);
        if (i >= valid[c]) y.t[i] = (E)0;   // (0 times an infinite rs is no zero)
      }
      widen8<DT>(y, v);
      if (a.y) store8<DT>((E*)a.y + row * a.ldy, col, valid[c], v);
      if (a.codes) {
        const uint32_t sb = scale_byte<F>(quad_max(amax8_bits<DT>(y)));
        const uint2 code = encode8<F>(v, scale_recip(sb));
        if (col < pitch) {
          *(uint2*)(a.codes + row * pitch + col) = code;
          if ((lane & 3) == 0) a.scales[row * ckpt_scale_pitch(a.cols) + col / 32] = (uint8_t)sb;
        }
      }
    }
  }
}

// dw: a workgroup adds up its rows' share in registers, in the rows' order, and
// leaves it as a plane of its own; k_norm_join adds the planes. The order depends on
// the sizes alone.
template <int DT, int T, int V>
__global__ __launch_bounds__(Shape<T>::threads) void k_rmsnorm_backward(const NormArgs a) {
  typedef typename El<DT>::T E;
  typedef Shape<T> S;
  constexpr bool ahead = V <= 2;   // (with four units, neither the next row's loads nor the weights fit in the registers)
  __shared__ float slots[2][16];
  __shared__ float shares[T == 64 ? S::rows : 1][T == 64 ? 64 * V * 8 : 1];
  const int lane = T == 64 ? threadIdx.x & 63 : threadIdx.x;
  const int cols = (int)a.cols;
  int valid[V];
#pragma unroll
  for (int c = 0; c < V; c++) {
    const int left = cols - (c * T + lane) * 8;
    valid[c] = left <= 0 ? 0 : (left >= 8 ? 8 : left);
  }
  const int64_t step = (int64_t)gridDim.x * S::rows;
  int64_t row = (int64_t)blockIdx.x * S::rows + own_row<T>();
  Words<DT> dy[V], h[V], dh[V];
  float rs = 0.0f;
  auto load = [&](int64_t at) {
#pragma unroll
    for (int c = 0; c < V; c++) {
      dy[c] = load_words<DT>((const E*)a.x + at * a.ldx, (c * T + lane) * 8, cols);
      h[c] = load_words<DT>((const E*)a.h + at * a.ldh, (c * T + lane) * 8, cols);
    }
    if (a.r) {
#pragma unroll
      for (int c = 0; c < V; c++) dh[c] = load_words<DT>((const E*)a.r + at * a.ldr, (c * T + lane) * 8, cols);
    }
    rs = a.rs[at];
  };
  if (row < a.rows) load(row);
  float w[ahead ? V : 1][8], share[V][8];
  if constexpr (ahead) {
#pragma unroll
    for (int c = 0; c < V; c++) load_unit<DT>(a.w, a.wide, (c * T + lane) * 8, cols, w[c]);
  }
#pragma unroll
  for (int c = 0; c < V; c++)
#pragma unroll
    for (int i = 0; i < 8; i++) share[c][i] = 0.0f;
  for (int turn = 0; row < a.rows; row += step, turn ^= 1) {
    const float scale = rs;
    // of unit c: n and dy
    auto values = [&](int c, float n[8], float g[8]) {
      widen8<DT>(raw<DT>(dy[c]), g);
      widen8<DT>(raw<DT>(h[c]), n);
#pragma unroll
      for (int i = 0; i < 8; i++) n[i] *= scale;
    };
    auto add_up = [&](int c, const float n[8], float g[8], const float w[8], float& sum) {
#pragma unroll
      for (int i = 0; i < 8; i++) {
        share[c][i] = __builtin_fmaf(g[i], n[i], share[c][i]);
        g[i] *= w[i];
        sum = __builtin_fmaf(g[i], n[i], sum);
      }
    };
    auto finish = [&](int c, const float n[8], float g[8], float mean, const float base[8]) {
#pragma unroll
      for (int i = 0; i < 8; i++) {
        g[i] = scale * __builtin_fmaf(-n[i], mean, g[i]);
        if (a.r) g[i] += base[i];
      }
      store8<DT>((E*)a.y + row * a.ldy, (int64_t)(c * T + lane) * 8, valid[c], g);
    };
    float sum = 0.0f;
    if constexpr (ahead) {
      float g[V][8], n[V][8], base[V][8];
#pragma unroll
      for (int c = 0; c < V; c++) {
        values(c, n[c], g[c]);
        if (a.r) widen8<DT>(raw<DT>(dh[c]), base[c]);
        add_up(c, n[c], g[c], w[c], sum);
      }
      if (row + step < a.rows) load(row + step);
      const float mean = row_sum<T>(sum, slots, turn) / (float)a.cols;
#pragma unroll
      for (int c = 0; c < V; c++) finish(c, n[c], g[c], mean, base[c]);
    } else {
      float g[8], n[8], base[8];
#pragma unroll
      for (int c = 0; c < V; c++) {
        __builtin_amdgcn_sched_barrier(0);
        load_unit<DT>(a.w, a.wide, (c * T + lane) * 8, cols, w[0]);
        values(c, n, g);
        add_up(c, n, g, w[0], sum);
      }
      const float mean = row_sum<T>(sum, slots, turn) / (float)a.cols;
      // (made opaque: left alone, the compiler keeps every unit's values in registers besides the elements, and spills)
#pragma unroll
      for (int c = 0; c < V; c++) hide(h[c]), hide(dy[c]);
#pragma unroll
      for (int c = 0; c < V; c++) {
        __builtin_amdgcn_sched_barrier(0);
        load_unit<DT>(a.w, a.wide, (c * T + lane) * 8, cols, w[0]);
        values(c, n, g);
#pragma unroll
        for (int i = 0; i < 8; i++) g[i] *= w[0][i];
        if (a.r) widen8<DT>(raw<DT>(dh[c]), base);
        finish(c, n, g, mean, base);
      }
      if (row + step < a.rows) load(row + step);
    }
  }
  if (!a.planes) return;
  float* const plane = a.planes + (int64_t)blockIdx.x * plane_stride(a.cols);
  if constexpr (T == 64) {
    const int mine = own_row<T>();
#pragma unroll
    for (int c = 0; c < V; c++)
#pragma unroll
      for (int i = 0; i < 8; i++) shares[mine][(c * 8 + i) * 64 + lane] = share[c][i];
    __syncthreads();
    if (mine != 0) return;
#pragma unroll
    for (int c = 0; c < V; c++)
#pragma unroll
      for (int i = 0; i < 8; i++)
#pragma unroll
        for (int k = 1; k < S::rows; k++) share[c][i] += shares[k][(c * 8 + i) * 64 + lane];
  }
#pragma unroll
  for (int c = 0; c < V; c++)
#pragma unroll
    for (int i = 0; i < 8; i++)
      if (i < valid[c]) plane[(int64_t)(c * T + lane) * 8 + i] = share[c][i];
}

// dw = dw_in + the planes' sum: 32 columns a workgroup, 32 groups of planes side by
// side. What a thread reads does not depend on what it has read, so eight planes' loads
// are on their way at a time.
__global__ __launch_bounds__(1024) void k_norm_join(int64_t cols, int planes, const float* from, const float* in, float* dw) {
  __shared__ float part[32][33];
  const int c = threadIdx.x & 31, group = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + c, stride = plane_stride(cols);
  float s = 0.0f;
  if (col < cols)
    for (int p = group; p < planes; p += 256) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const int at = p + 32 * j;
        v[j] = from[(at < planes ? at : p) * stride + col];
      }
#pragma unroll
      for (int j = 0; j < 8; j++) s += p + 32 * j < planes ? v[j] : 0.0f;
    }
  part[group][c] = s;
  __syncthreads();
  if (group != 0 || col >= cols) return;
#pragma unroll
  for (int k = 1; k < 32; k++) s += part[k][c];
  dw[col] = in ? in[col] + s : s;
}

// Workgroups of a pass over the rows. Forward: six for a compute unit where a thread has
// one unit of eight elements of a 16-bit type, else four (16384 x 2048 bf16: 57 us by six,
// 66 by four, 72 by seven; 8192 x 4096 bf16: 67 and 57; 8192 x 2048 f32: 69 and 66).
inline int rows_at_once(int64_t cols) { return cols <= 1024 ? Shape<64>::rows : 1; }
inline int64_t forward_groups(int64_t rows, int64_t cols, bool wide) {
  const int each = rows_at_once(cols);
  const int64_t wanted = (rows + each - 1) / each, most = (int64_t)compute_units() * (cols <= 2048 && !wide ? 6 : 4);
  return wanted < most ? wanted : most;
}
// Backward: as many as run at once, since each leaves a plane of dw (8192 x 4096 bf16, of 256
// threads: 67 us by three for a compute unit, which fit, 83 by two, 88 by four; 16384 x 2048:
// 56 by four, 61 by three); of few rows two rows for each where that leaves one for each
// compute unit (1000 x 2048: 10.9 us, a row for each 14.5).
inline int64_t backward_groups(int64_t rows, int64_t cols) {
  const int each = rows_at_once(cols), fit = cols <= 512 ? 4 : cols <= 1024 ? 3 : cols <= 2048 ? 4 : cols <= 4096 ? 2 : 1;
  const int64_t units = compute_units(), most = units * fit;
  int64_t wanted = (rows + each - 1) / each;
  if (wanted > units) wanted = wanted / 2 > units ? wanted / 2 : units;
  return wanted < most ? wanted : most;
}
// Threads of a row, and its units of eight elements for each. A wave alone up to 1024 columns:
// it waits for no other (16384 x 1024 bf16: forward 27 us, by 256 threads 31; backward 36 and
// 43). Then as few units as the threads of a workgroup allow in the backward pass, whose
// units take most registers (8192 x 4096 bf16: 56 us by 512 threads, 67 by 256; 8192 x 8192:
// 110 by 1024, 149 by 512); forward, more workgroups are worth more (8192 x 8192: 111 us by
// 512 threads, 130 by 1024) up to 8192 columns (4096 x 16384: 119 us by 1024 threads, 160 by
// 512; of binary32, and in the backward pass, two units' registers are too many for 1024).
template <int DT, int F>
hipError_t forward(const NormArgs& a, hipStream_t s) {
#define LQ_NORM(T, V)                                                                                                  \
  {                                                                                                                    \
    hipLaunchKernelGGL((k_rmsnorm<DT, F, T, V>), dim3((unsigned)forward_groups(a.rows, a.cols, DT == LQ_F32)),         \
                       dim3(Shape<T>::threads), 0, s, a);                                                              \
    return hipGetLastError();                                                                                          \
  }
  if (a.cols <= 512) LQ_NORM(64, 1)
  if (a.cols <= 1024) LQ_NORM(64, 2)
  if (a.cols <= 2048) LQ_NORM(256, 1)
  if (a.cols <= 4096) LQ_NORM(256, 2)
  if (a.cols <= 8192) LQ_NORM(512, 2)
  if constexpr (DT == LQ_F32) LQ_NORM(512, 4)
  else LQ_NORM(1024, 2)
#undef LQ_NORM
}
template <int DT>
hipError_t backward(const NormArgs& a, hipStream_t s) {
#define LQ_NORM(T, V)                                                                                                  \
  {                                                                                                                    \
    hipLaunchKernelGGL((k_rmsnorm_backward<DT, T, V>), dim3((unsigned)backward_groups(a.rows, a.cols)),                \
                       dim3(Shape<T>::threads), 0, s, a);                                                              \
    return hipGetLastError();                                                                                          \
  }
  if (a.cols <= 512) LQ_NORM(64, 1)
  if (a.cols <= 1024) LQ_NORM(64, 2)
  if (a.cols <= 2048) LQ_NORM(256, 1)
  if (a.cols <= 4096) LQ_NORM(512, 1)
  if (a.cols <= 8192) LQ_NORM(1024, 1)
  LQ_NORM(512, 4)
#undef LQ_NORM
}

}  // namespace

int64_t norm_planes(int64_t rows, int64_t cols) { return backward_groups(rows, cols); }

hipError_t launch_rmsnorm(int dtype, int format, const NormArgs& a, hipStream_t s) {
  if (format == LQ_INT8) {
    if (dtype == LQ_F32) return forward<LQ_F32, LQ_INT8>(a, s);
    if (dtype == LQ_BF16) return forward<LQ_BF16, LQ_INT8>(a, s);
    return forward<LQ_F16, LQ_INT8>(a, s);
  }
  if (dtype == LQ_F32) return forward<LQ_F32, LQ_E4M3>(a, s);
  if (dtype == LQ_BF16) return forward<LQ_BF16, LQ_E4M3>(a, s);
  return forward<LQ_F16, LQ_E4M3>(a, s);
}

hipError_t launch_rmsnorm_backward(int dtype, const NormArgs& a, const float* dw_in, float* dw, hipStream_t s) {
  if (a.rows > 0) {
    const hipError_t e = dtype == LQ_F32    ? backward<LQ_F32>(a, s)
                         : dtype == LQ_BF16 ? backward<LQ_BF16>(a, s)
                                            : backward<LQ_F16>(a, s);
    if (e != hipSuccess) return e;
  }
  if (!dw) return hipSuccess;
  hipLaunchKernelGGL(k_norm_join, dim3((unsigned)((a.cols + 31) / 32)), dim3(1024), 0, s, a.cols,
                     (int)(a.rows > 0 ? norm_planes(a.rows, a.cols) : 0), a.planes, dw_in, dw);
  return hipGetLastError();
}

}  // namespace lql
