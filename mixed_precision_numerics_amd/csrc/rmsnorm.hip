// RMS norm with the residual's addition and 16-bit or FP8 outputs, and its
// backward pass from the stored input or from an FP8 checkpoint (gfx950).
//
//   h = round(x + res),  r = 1 / sqrt(mean(h^2) + eps),  y = (h r) gamma
//   n = h r,  g = dy gamma,  dx = r (g - n mean(g n)) + dres,  dgamma = sum_rows dy n
//
// Sums, statistics and products are FP32; h is rounded once to the stream's
// type (what the next layer and the backward pass see is what is normalised),
// y and dx once to theirs.
#include "tiles.hpp"

namespace amp {
namespace {

struct NormArgs {
  const void* x; int64_t ldx;
  const void* res; int64_t ldr;
  const void* gamma; int gt;
  float eps;
  void* h; int64_t ldh;
  void* y; int yt; int64_t ldy;
  const float* scale; float* amax;
  amp_fp8_tiles yq, ck;
  float* rstd;
  int64_t rows, cols;
};

// Sum over the 16 lanes of a DPP row, in every lane (each adds the same pairs).
__device__ __forceinline__ float sum16(float v) {
#define AMP_ADD(ctl) v += bitsf(static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(fbits(v)), ctl, 0xf, 0xf, false)));
  AMP_ADD(0x128) AMP_ADD(0x124) AMP_ADD(0x122) AMP_ADD(0x121)
#undef AMP_ADD
  return v;
}
// Sum over a wave, in every lane, without the LDS: rotations within rows of
// 16, then the rows and the halves exchanged.
__device__ __forceinline__ float wave_sum(float v) {
  v = sum16(v);
  const auto a = __builtin_amdgcn_permlane16_swap(fbits(v), fbits(v), false, false);
  v = bitsf(a[0]) + bitsf(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(fbits(v), fbits(v), false, false);
  return bitsf(b[0]) + bitsf(b[1]);
}

// Sum over the T threads of a row, T a multiple of 64; with T == 64 a row is
// one wave's, else every thread of the block calls.  `red` holds two sets of
// 16 words; a caller that loops uses them in `turn`, so that one barrier a row
// is enough: a wave that runs ahead writes the other set.
__device__ __forceinline__ float row_sum(float v, int T, float* red, int turn) {
  v = wave_sum(v);
  if (T > kWave) {
    const int w = threadIdx.x / kWave, W = T / kWave, first = w / W * W, k = threadIdx.x % 16;
    float* set = red + turn * 16;
    if (threadIdx.x % kWave == 0) set[w] = v;
    __syncthreads();
    v = sum16(k < W ? set[first + k] : 0.0f);
  }
  return v;
}

// x + res rounded to the stream's type, one vector.
template <int XT>
__device__ __forceinline__ u32x4 join(u32x4 a, u32x4 b) {
  constexpr int E = kVec<XT>;
  float p[E], q[E];
  widen<XT>(a, p);
  widen<XT>(b, q);
#pragma unroll
  for (int k = 0; k < E; ++k) p[k] += q[k];
  return narrow<XT>(p);
}

template <int XT>
__device__ __forceinline__ float sum_squares(u32x4 w, float ss) {
  constexpr int E = kVec<XT>;
  float h[E];
  widen<XT>(w, h);
#pragma unroll
  for (int k = 0; k < E; ++k) ss = __builtin_fmaf(h[k], h[k], ss);
  return ss;
}

// N <= 4 vectors of a row, `step` columns apart from column c on, in 1x128
// tiles.  Lane k of a tile's lane group stores the scale of vector k's tile.
template <int E, int N, bool FULL>
__device__ __forceinline__ void store_tiles(const amp_fp8_tiles& o, int64_t row, int64_t c0, int c, int step, int n,
                                            bool live, const float (&v)[N][E]) {
  constexpr int G = kTileK / E;
  uint32_t m[N], top = 0, w[N][E / 4];
  float sc[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    m[k] = group_max<G>(mag(abs_max<E>(0.0f, v[k])));
    top = top > m[k] ? top : m[k];
  }
  const float inv = tile_scales<N>(m, fp8_max(o.type), sc);
  const int mine = c / kTileK * kTileK + (threadIdx.x & 3) * step;   // where that tile begins
  if (threadIdx.x % G < N && (FULL || mine < n) && live) o.s[(c0 + mine) / kTileK * o.lds + row] = inv;
  encode<N, E, false>(o.type, top >= kInfBits, w, [&](int k, int e) __attribute__((always_inline)) { return v[k][e] * sc[k]; });
  uint8_t* q = o.q + row * o.ldq + c0;
#pragma unroll
  for (int k = 0; k < N; ++k)
    if (live) store_codes<E, FULL>(q, c + k * step, n, w[k]);
}

// Every output of N vectors of h with their factors gm; returns their |y|
// maximum.  c0: the first column of this chunk of the row, of which n are left.
template <int XT, int N, bool FULL>
__device__ __forceinline__ float norm_outputs(const NormArgs& a, const u32x4 (&w)[N], const float (&gm)[N][kVec<XT>], int64_t row,
                                              int64_t c0, int c, int step, int n, bool live, float r, float scale) {
  constexpr int E = kVec<XT>;
  float y[N][E], am = 0.0f;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    widen<XT>(w[k], y[k]);
#pragma unroll
    for (int e = 0; e < E; ++e) y[k][e] = y[k][e] * r * gm[k][e];
    am = abs_max<E>(am, y[k]);
  }
  if (a.y) {
    const int yb = a.yt == AMP_F16 || a.yt == AMP_BF16 ? 2 : 1;
    store_plain<N, E, FULL>(static_cast<uint8_t*>(a.y) + (row * a.ldy + c0) * yb, a.yt, c, step, n, live, scale, am, y);
  }
  if (a.yq.q) store_tiles<E, N, FULL>(a.yq, row, c0, c, step, n, live, y);
  if (a.ck.q) {
#pragma unroll
    for (int k = 0; k < N; ++k) widen<XT>(w[k], y[k]);
    store_tiles<E, N, FULL>(a.ck, row, c0, c, step, n, live, y);
  }
  return am;
}

// T threads hold a row in registers, V vectors each.  WAVE: T is 64 and a
// block of 256 works on four rows; else the block's T threads on one.  FULL:
// the row is V T whole vectors.
//
// HBM-bound.  One row per wave or block and no loop over rows: in a loop the
// next row's loads wait for this row's stores (one counter holds both) and
// every stream's pointer stays in vector registers; 16381 x 5120 BF16 took
// 124-166 us with the loop and 99 without.  T is a power of two: a block of 3
// or 5 waves fills the four SIMDs unevenly (the same rows in 5 waves: 166 us).
template <int XT, int V, bool WAVE, bool FULL>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void rmsnorm_rows(const NormArgs a) {
  constexpr int E = kVec<XT>, N = V % 2 == 0 ? 2 : V == 3 ? 3 : 1;
  __shared__ float red[32];
  __shared__ uint32_t redm[16];
  const int T = WAVE ? kWave : blockDim.x;
  const int64_t row = WAVE ? static_cast<int64_t>(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave)
                           : static_cast<int64_t>(blockIdx.x);
  const int c = (WAVE ? threadIdx.x % kWave : threadIdx.x) * E, step = T * E, n = left(a.cols);
  const bool live = !WAVE || row < a.rows;
  const float scale = a.scale ? *a.scale : 1.0f;
  const uint32_t seen = amax_seen(a.amax);
  u32x4 h[V / N][N];
#pragma unroll
  for (int v = 0; v < V; ++v)
    h[v / N][v % N] = live ? load_vec<XT, FULL>(elem<XT>(a.x, row * a.ldx), c + v * step, n) : u32x4{0u, 0u, 0u, 0u};
  if (a.res) {
    u32x4 q[V];
#pragma unroll
    for (int v = 0; v < V; ++v) q[v] = live ? load_vec<XT, FULL>(elem<XT>(a.res, row * a.ldr), c + v * step, n) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int v = 0; v < V; ++v) h[v / N][v % N] = join<XT>(h[v / N][v % N], q[v]);
  }
  // (sums of two vectors are trimmed like one)
#pragma unroll
  for (int v = 0; v < V; ++v) h[v / N][v % N] = trim_vec<XT, FULL>(h[v / N][v % N], c + v * step, n);
  float ss = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) ss = sum_squares<XT>(h[v / N][v % N], ss);
  if (a.h && live) {
#pragma unroll
    for (int v = 0; v < V; ++v) store_vec<XT, FULL>(elem<XT>(a.h, row * a.ldh), c + v * step, n, h[v / N][v % N]);
  }
  ss = row_sum(ss, T, red, 0);
  const float r = 1.0f / sqrtf(ss / static_cast<float>(a.cols) + a.eps);
  if (a.rstd && live && c == 0) a.rstd[row] = r;
  float am = 0.0f;
#pragma unroll
  for (int p = 0; p < V / N; ++p) {
    float gm[N][E];
#pragma unroll
    for (int k = 0; k < N; ++k) load_cols<E, FULL>(a.gamma, a.gt, c + (p * N + k) * step, n, gm[k]);
    am = __builtin_elementwise_maximum(am, norm_outputs<XT, N, FULL>(a, h[p], gm, row, 0, c + p * N * step, step, n, live, r, scale));
  }
  // a wave past the last row holds zeros, whose y is NaN where eps is 0
  if (a.amax) block_amax(live ? am : 0.0f, seen, redm, a.amax);
}

// Rows too long for the registers: a block walks its row twice (the second
// reads come from the caches; 1024 x 73728 with residual and tiles BF16 133 us =
// 4.0 TB/s, 1024 x 65536 FP32 with a checkpoint and a 16-bit y 149 = 3.2; 1024 x
// 65536 BF16, the longest that the registers hold, 89 = 5.3).  In place, h is
// what the second walk reads.
template <int XT>
__global__ __launch_bounds__(1024) void rmsnorm_long(const NormArgs a) {
  constexpr int E = kVec<XT>, T = 1024;
  __shared__ float red[32];
  __shared__ uint32_t redm[16];
  const int c = threadIdx.x * E;
  const float scale = a.scale ? *a.scale : 1.0f;
  const uint32_t seen = amax_seen(a.amax);
  float am = 0.0f;
  const int64_t row = blockIdx.x;
  float ss = 0.0f;
  for (int64_t c0 = 0; c0 < a.cols; c0 += T * E) {
    const int n = left(a.cols - c0);
    u32x4 w = load_vec<XT>(elem<XT>(a.x, row * a.ldx + c0), c, n);
    if (a.res) w = join<XT>(w, load_vec<XT>(elem<XT>(a.res, row * a.ldr + c0), c, n));
    w = trim_vec<XT>(w, c, n);
    if (a.h) store_vec<XT>(elem<XT>(a.h, row * a.ldh + c0), c, n, w);
    ss = sum_squares<XT>(w, ss);
  }
  ss = row_sum(ss, T, red, 0);
  const float r = 1.0f / sqrtf(ss / static_cast<float>(a.cols) + a.eps);
  if (a.rstd && threadIdx.x == 0) a.rstd[row] = r;
  for (int64_t c0 = 0; c0 < a.cols; c0 += T * E) {
    const int n = left(a.cols - c0);
    u32x4 w[1];
    if (a.h) {
      w[0] = load_vec<XT>(elem<XT>(a.h, row * a.ldh + c0), c, n);
    } else {
      w[0] = load_vec<XT>(elem<XT>(a.x, row * a.ldx + c0), c, n);
      if (a.res) w[0] = join<XT>(w[0], load_vec<XT>(elem<XT>(a.res, row * a.ldr + c0), c, n));
    }
    w[0] = trim_vec<XT>(w[0], c, n);
    float gm[1][E];
    load_cols<E>(a.gamma ? elem_of(a.gt, a.gamma, c0) : nullptr, a.gt, c, n, gm[0]);
    am = __builtin_elementwise_maximum(am, norm_outputs<XT, 1, false>(a, w, gm, row, c0, c, 0, n, true, r, scale));
  }
  if (a.amax) block_amax(am, seen, redm, a.amax);
}

// Threads per row and vectors per thread.  Many rows: the pair that covers
// the row with the fewest idle slots, of those the one with the most threads
// (4096 columns BF16, 8192 rows: 512 x 1, 256 x 2 and 128 x 4 within 2 %; 5120:
// 128 x 5 99 us, 256 x 3 with a sixth of the slots idle 123).  Below 1024 rows
// the machine is not full and a row's own latency counts, so as few vectors
// per thread as 1024 threads allow (64 rows of 4096: 512 x 1 4.0 us, 128 x 4
// 5.5).
struct RowShape { int T, V; };
RowShape row_shape(int64_t rows, int64_t nv) {
  RowShape best{0, 0};
  for (int T = 64; T <= 1024; T *= 2) {
    const int64_t V = (nv + T - 1) / T;
    if (V > (T == 64 ? 4 : 8)) continue;
    if (best.T == 0 || (rows < 1024 ? V < best.V : V * T <= static_cast<int64_t>(best.V) * best.T)) best = {T, static_cast<int>(V)};
  }
  return best;
}

// Rows a launch: the threads of a grid are counted in 32 bits.
constexpr int64_t kRowsPerLaunch = 1 << 21;

template <int XT, int V>
void launch_rows(const NormArgs& a, int T, bool full, hipStream_t s) {
  const unsigned rows = static_cast<unsigned>(a.rows);
  if (T == 64) {
    if constexpr (V <= 4) {
      if (full) rmsnorm_rows<XT, V, true, true><<<(rows + 3) / 4, 256, 0, s>>>(a);
      else rmsnorm_rows<XT, V, true, false><<<(rows + 3) / 4, 256, 0, s>>>(a);
    }
  } else {
    if (full) rmsnorm_rows<XT, V, false, true><<<rows, T, 0, s>>>(a);
    else rmsnorm_rows<XT, V, false, false><<<rows, T, 0, s>>>(a);
  }
}

template <int XT>
hipError_t dispatch_rmsnorm(const NormArgs& whole, hipStream_t s) {
  constexpr int E = kVec<XT>;
  const RowShape p = row_shape(whole.rows, (whole.cols + E - 1) / E);
  for (int64_t r0 = 0; r0 < whole.rows; r0 += kRowsPerLaunch) {
    NormArgs a = whole;
    a.rows = whole.rows - r0 < kRowsPerLaunch ? whole.rows - r0 : kRowsPerLaunch;
    a.x = elem<XT>(a.x, r0 * a.ldx);
    if (a.res) a.res = elem<XT>(a.res, r0 * a.ldr);
    if (a.h) a.h = elem<XT>(a.h, r0 * a.ldh);
    if (a.y) a.y = static_cast<uint8_t*>(a.y) + r0 * a.ldy * dtype_bytes(a.yt);
    if (a.yq.q) { a.yq.q += r0 * a.yq.ldq; a.yq.s += r0; }
    if (a.ck.q) { a.ck.q += r0 * a.ck.ldq; a.ck.s += r0; }
    if (a.rstd) a.rstd += r0;
    const bool full = a.cols == static_cast<int64_t>(p.T) * p.V * E;
    switch (p.V) {
      case 0: rmsnorm_long<XT><<<static_cast<unsigned>(a.rows), 1024, 0, s>>>(a); break;
      case 1: launch_rows<XT, 1>(a, p.T, full, s); break;
      case 2: launch_rows<XT, 2>(a, p.T, full, s); break;
      case 3: launch_rows<XT, 3>(a, p.T, full, s); break;
      case 4: launch_rows<XT, 4>(a, p.T, full, s); break;
      case 5: launch_rows<XT, 5>(a, p.T, full, s); break;
      case 6: launch_rows<XT, 6>(a, p.T, full, s); break;
      case 7: launch_rows<XT, 7>(a, p.T, full, s); break;
      default: launch_rows<XT, 8>(a, p.T, full, s); break;
    }
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

// ------------------------------------------------------------ backward ---

struct NormBackArgs {
  const void* dy; int64_t lddy;
  const void* h; int64_t ldh;
  amp_fp8_tiles ck;
  const void* gamma; int gt;
  const float* rstd;
  const void* dres; int64_t lddr;
  void* dx; int64_t lddx;
  float* part;
  int64_t rows, cols;
};

// The compiler no longer knows what was formed from w: those values are formed
// again at its next use instead of staying in registers.
__device__ __forceinline__ void forget(uint32_t& w) { asm("" : "+v"(w)); }
__device__ __forceinline__ void forget(u32x4& w) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t t = w[k];
    forget(t);
    w[k] = t;
  }
}

// One vector of h from the stored tensor (type XT) or the checkpoint.
template <int XT, bool CK>
struct HRaw {
  static constexpr int E = kVec<XT>;
  u32x4 w;
  uint32_t q[E / 4];
  float s;
  // column c of the n that the row has from column c0 on
  template <bool FULL>
  __device__ __forceinline__ void load(const NormBackArgs& a, int64_t row, int64_t c0, int c, int n) {
    if constexpr (CK) {
      load_codes<E, FULL>(a.ck.q + row * a.ck.ldq + c0, c, n, q);
      // a lane past the row holds zero codes; it reads the last tile's scale
      s = a.ck.s[(c0 + (FULL || c < n ? c : n - 1)) / kTileK * a.ck.lds + row];
    } else {
      w = load_vec<XT, FULL>(elem<XT>(a.h, row * a.ldh + c0), c, n);
    }
  }
  template <bool FULL>
  __device__ __forceinline__ void trim(int c, int n) {
    if constexpr (CK) trim_codes<E, FULL>(q, c, n);
    else w = trim_vec<XT, FULL>(w, c, n);
  }
  __device__ __forceinline__ void forget_values() {
    if constexpr (CK) {
#pragma unroll
      for (int k = 0; k < E / 4; ++k) forget(q[k]);
    } else {
      forget(w);
    }
  }
  __device__ __forceinline__ void values(const NormBackArgs& a, float (&v)[E]) const {
    if constexpr (CK) decode<E>(a.ck.type, q, s, v);
    else widen<XT>(w, v);
  }
};

// dx, one vector: m is the row's mean of g n.
template <int E>
__device__ __forceinline__ void dx_of(const float (&dy)[E], const float (&h)[E], const float (&gm)[E], float r, float m, float (&d)[E]) {
#pragma unroll
  for (int k = 0; k < E; ++k) d[k] = r * (dy[k] * gm[k] - h[k] * r * m);
}

// T threads a row, V vectors each, S rows at a time in a block of T S
// threads; a block strides over the rows with its sums of dy n in registers
// and writes one row of partial sums at the end (no atomics: the result does
// not depend on the order in which blocks run).  FULL: the row is V T whole
// vectors.
//
// HBM-bound (8192 x 4096 BF16 from a checkpoint with dres: 44 us = 5.4 TB/s,
// and 4 us for dgamma_sum).  The next row's loads go out before this row's
// stores: loads and stores complete in one count, so loads issued behind the
// stores would wait for them.  They are issued without a branch (dy stands in
// for an absent dres), so that the wait for them can be counted.  One block a CU: 128
// partial rows keep half the machine idle, 512 cost more to write and add up
// (1000 x 4096: 13 us with 256, 16 with 512, 15 with 128).
template <int XT, bool CK, int V, int S, bool FULL>
__global__ __launch_bounds__(S > 1 ? 512 : 1024) void rmsnorm_back_rows(const NormBackArgs a) {
  constexpr int E = kVec<XT>;
  __shared__ float red[32];
  __shared__ float sums[S > 1 ? (512 / S) * V * E : 1];
  const int T = S > 1 ? 512 / S : blockDim.x;
  const int sub = S > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / T) : 0;
  const int tid = S > 1 ? threadIdx.x % T : threadIdx.x, n = left(a.cols);
  const float inv_n = 1.0f / static_cast<float>(a.cols);
  const void* res = a.dres ? a.dres : a.dy;
  const int64_t ldr = a.dres ? a.lddr : a.lddy, step = static_cast<int64_t>(gridDim.x) * S;
  float dg[V][E] = {}, gm[V][E];
  struct Row { u32x4 dy[V], res[V]; HRaw<XT, CK> h[V]; float r; };
  auto fetch = [&](int64_t row) __attribute__((always_inline)) {
    row = row < a.rows ? row : a.rows - 1;   // read again, not used
    Row w;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * T + tid) * E;
      w.dy[v] = load_vec<XT, FULL>(elem<XT>(a.dy, row * a.lddy), c, n);
      w.h[v].template load<FULL>(a, row, 0, c, n);
      w.res[v] = load_vec<XT, FULL>(elem<XT>(res, row * ldr), c, n);
    }
    w.r = a.rstd[row];
    return w;
  };
  int64_t row = static_cast<int64_t>(blockIdx.x) * S + sub;
  Row w = fetch(row);
#pragma unroll
  for (int v = 0; v < V; ++v) load_cols<E, FULL>(a.gamma, a.gt, (v * T + tid) * E, n, gm[v]);
  int turn = 0;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * S; r0 < a.rows; r0 += step, row += step) {
    const bool live = row < a.rows;
    float dot = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float dy[E], h[E];
      const int c = (v * T + tid) * E;
      w.dy[v] = trim_vec<XT, FULL>(w.dy[v], c, n);
      w.h[v].template trim<FULL>(c, n);
      widen<XT>(w.dy[v], dy);
      w.h[v].values(a, h);
#pragma unroll
      for (int k = 0; k < E; ++k) {
        dy[k] *= h[k] * w.r;
        dot = __builtin_fmaf(dy[k], gm[v][k], dot);
        dg[v][k] += live ? dy[k] : 0.0f;
      }
    }
    const Row next = fetch(row + step);
    const float m = row_sum(dot, T, red, turn) * inv_n;
    turn ^= 1;
    if (a.dx && live) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float dy[E], h[E], d[E];
        if constexpr (V > 1) {   // 2000 x 12000 BF16 stored: 41 us, 66 without
          forget(w.dy[v]);
          w.h[v].forget_values();
        }
        widen<XT>(w.dy[v], dy);
        w.h[v].values(a, h);
        dx_of<E>(dy, h, gm[v], w.r, m, d);
        if (a.dres) {
          widen<XT>(trim_vec<XT, FULL>(w.res[v], (v * T + tid) * E, n), dy);
#pragma unroll
          for (int k = 0; k < E; ++k) d[k] += dy[k];
        }
        store_vec<XT, FULL>(elem<XT>(a.dx, row * a.lddx), (v * T + tid) * E, n, narrow<XT>(d));
      }
    }
    w = next;
  }
  if (a.part == nullptr) return;
  if constexpr (S > 1) {
    for (int k = S - 1; k > 0; --k) {
      __syncthreads();
      if (sub == k) {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int e = 0; e < E; ++e) sums[(v * E + e) * T + tid] = dg[v][e];
      }
      __syncthreads();
      if (sub == k - 1) {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int e = 0; e < E; ++e) dg[v][e] += sums[(v * E + e) * T + tid];
      }
    }
    if (sub != 0) return;
  }
  float* p = a.part + static_cast<int64_t>(blockIdx.x) * a.cols;
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int q = 0; q < E / 4; ++q) {
      const u32x4 w4 = {fbits(dg[v][4 * q]), fbits(dg[v][4 * q + 1]), fbits(dg[v][4 * q + 2]), fbits(dg[v][4 * q + 3])};
      store_vec<AMP_F32, FULL>(p, (v * T + tid) * E + 4 * q, n, w4);
    }
  }
}

// Few rows (launch and latency count): one launch, whose first blocks sum 32
// columns of dy n over every row, with no partial sums in memory, while the
// others form dx, S rows of 512 / S threads a block.  dy and h are read twice,
// the second time from the caches.  Against rmsnorm_back_rows and dgamma_sum,
// BF16: 1 x 4096 3.7 us (5.7), 64 x 1000 3.6 (6.7), 512 x 4096 8.7 (9.6), 512 x
// 512 5.0 (6.4); beyond kFewRows the columns' blocks last longest (1000 x 2047
// 13.1 against 11.0, 2000 x 512 17.8 against 7.9).  The bound of 512 vectors is
// where one vector a thread ends; wider rows were not measured in this form (1 x
// 5120 takes 3.4 and 2.7 us in two launches).
template <int XT, bool CK, int S>
__global__ __launch_bounds__(512) void rmsnorm_back_few(const NormBackArgs a, float* dgamma, int sums) {
  constexpr int E = kVec<XT>, kCols = 32, G = kCols / E, P = 512 / G, R = 4;
  __shared__ float part[P][kCols + 1], more[16][kCols + 1], red[32];
  const int n = left(a.cols);
  if (static_cast<int>(blockIdx.x) < sums) {
    const int c0 = blockIdx.x * kCols, c = c0 + threadIdx.x % G * E, strand = threadIdx.x / G;
    float dg[E] = {};
    for (int64_t r0 = strand; r0 < a.rows; r0 += P * R) {
      u32x4 wd[R];
      HRaw<XT, CK> hr[R];
      float r[R];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int64_t row = r0 + i * P < a.rows ? r0 + i * P : a.rows - 1;   // read again, not used
        wd[i] = load_vec<XT>(elem<XT>(a.dy, row * a.lddy), c, n);
        hr[i].template load<false>(a, row, 0, c, n);
        r[i] = a.rstd[row];
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        float dy[E], h[E];
        hr[i].template trim<false>(c, n);
        widen<XT>(trim_vec<XT>(wd[i], c, n), dy);
        hr[i].values(a, h);
#pragma unroll
        for (int k = 0; k < E; ++k) dg[k] += r0 + i * P < a.rows ? dy[k] * (h[k] * r[i]) : 0.0f;
      }
    }
#pragma unroll
    for (int k = 0; k < E; ++k) part[strand][threadIdx.x % G * E + k] = dg[k];
    __syncthreads();
    const int col = threadIdx.x % kCols, group = threadIdx.x / kCols;
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < P / 16; ++k) t += part[group * (P / 16) + k][col];
    more[group][col] = t;
    __syncthreads();
    if (threadIdx.x < kCols && c0 + col < n) {
      t = 0.0f;
#pragma unroll
      for (int k = 0; k < 16; ++k) t += more[k][col];
      dgamma[c0 + col] = t;
    }
    return;
  }
  constexpr int T = 512 / S;
  const int sub = S > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / T) : 0, c = threadIdx.x % T * E;
  const int64_t row = static_cast<int64_t>(blockIdx.x - sums) * S + sub;
  const bool live = row < a.rows;
  const int64_t at = live ? row : a.rows - 1;   // read again, not used
  u32x4 wd = load_vec<XT>(elem<XT>(a.dy, at * a.lddy), c, n), wr = {0u, 0u, 0u, 0u};
  HRaw<XT, CK> hr;
  hr.template load<false>(a, at, 0, c, n);
  if (a.dres) wr = load_vec<XT>(elem<XT>(a.dres, at * a.lddr), c, n);
  const float r = a.rstd[at];
  float dy[E], h[E], gm[E], d[E], dot = 0.0f;
  load_cols<E>(a.gamma, a.gt, c, n, gm);
  widen<XT>(trim_vec<XT>(wd, c, n), dy);
  hr.template trim<false>(c, n);
  hr.values(a, h);
#pragma unroll
  for (int k = 0; k < E; ++k) dot = __builtin_fmaf(dy[k] * (h[k] * r), gm[k], dot);
  const float m = row_sum(dot, T, red, 0) / static_cast<float>(a.cols);
  if (!live) return;
  dx_of<E>(dy, h, gm, r, m, d);
  if (a.dres) {
    widen<XT>(trim_vec<XT>(wr, c, n), dy);
#pragma unroll
    for (int k = 0; k < E; ++k) d[k] += dy[k];
  }
  store_vec<XT>(elem<XT>(a.dx, row * a.lddx), c, n, narrow<XT>(d));
}

// Rows of more than two vectors in each of 1024 threads, whose sums and next
// row have no registers: dx by one block a row, and the sums of dy n in a pass
// of their own, which reads dy and h again.  (Kept together with the sums in
// the LDS, 2000 x 28672 BF16 took 238 us, and in the work area 440, both measured
// before the values were formed again after the row's sum.)  HBM-bound
// with both passes' reads: 2000 x 20480 BF16 stored 97 us = 4.2 TB/s, from a
// checkpoint with dres 107 (143 while the values of dy and h stayed in
// registers over the row's sum, which spilled).
template <int XT, bool CK, int V>
__global__ __launch_bounds__(1024) void rmsnorm_dx_rows(const NormBackArgs a) {
  constexpr int E = kVec<XT>, T = 1024;
  __shared__ float red[32];
  const int64_t row = blockIdx.x;
  const int n = left(a.cols);
  u32x4 wd[V], wr[V];
  HRaw<XT, CK> hr[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * T + threadIdx.x) * E;
    wd[v] = load_vec<XT>(elem<XT>(a.dy, row * a.lddy), c, n);
    hr[v].template load<false>(a, row, 0, c, n);
    if (a.dres) wr[v] = load_vec<XT>(elem<XT>(a.dres, row * a.lddr), c, n);
  }
  const float r = a.rstd[row];
  float dot = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * T + threadIdx.x) * E;
    float dy[E], h[E], gm[E];
    wd[v] = trim_vec<XT>(wd[v], c, n);
    hr[v].template trim<false>(c, n);
    widen<XT>(wd[v], dy);
    hr[v].values(a, h);
    load_cols<E>(a.gamma, a.gt, c, n, gm);
#pragma unroll
    for (int k = 0; k < E; ++k) dot = __builtin_fmaf(dy[k] * (h[k] * r), gm[k], dot);
  }
  const float m = row_sum(dot, T, red, 0) / static_cast<float>(a.cols);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * T + threadIdx.x) * E;
    float dy[E], h[E], gm[E], d[E];
    if constexpr (CK) {
      forget(wd[v]);
      hr[v].forget_values();
    }
    widen<XT>(wd[v], dy);
    hr[v].values(a, h);
    load_cols<E>(a.gamma, a.gt, c, n, gm);
    dx_of<E>(dy, h, gm, r, m, d);
    if (a.dres) {
      widen<XT>(trim_vec<XT>(wr[v], c, n), dy);
#pragma unroll
      for (int k = 0; k < E; ++k) d[k] += dy[k];
    }
    store_vec<XT>(elem<XT>(a.dx, row * a.lddx), c, n, narrow<XT>(d));
  }
}

// Longer rows still: the block walks its row twice, two blocks a CU (2000 x
// 32768 BF16 from a checkpoint with dres 163 us, with one 187; 1024 x 65536 stored
// 173 us = 3.9 TB/s of both passes' reads).
template <int XT, bool CK>
__global__ __launch_bounds__(1024, 8) void rmsnorm_dx_long(const NormBackArgs a) {
  constexpr int E = kVec<XT>, T = 1024;
  __shared__ float red[32];
  const int64_t row = blockIdx.x;
  const int c = threadIdx.x * E;
  const float r = a.rstd[row];
  float dot = 0.0f, m = 0.0f;
  for (int pass = 0; pass < 2; ++pass) {
    for (int64_t c0 = 0; c0 < a.cols; c0 += T * E) {
      const int n = left(a.cols - c0);
      if (c >= n) break;
      float dy[E], h[E], gm[E], d[E];
      HRaw<XT, CK> hr;
      const u32x4 w = load_vec<XT>(elem<XT>(a.dy, row * a.lddy + c0), c, n);
      hr.template load<false>(a, row, c0, c, n);
      hr.template trim<false>(c, n);
      widen<XT>(trim_vec<XT>(w, c, n), dy);
      hr.values(a, h);
      load_cols<E>(a.gamma ? elem_of(a.gt, a.gamma, c0) : nullptr, a.gt, c, n, gm);
      if (pass == 0) {
#pragma unroll
        for (int k = 0; k < E; ++k) dot = __builtin_fmaf(dy[k] * (h[k] * r), gm[k], dot);
      } else {
        dx_of<E>(dy, h, gm, r, m, d);
        if (a.dres) {
          widen<XT>(trim_vec<XT>(load_vec<XT>(elem<XT>(a.dres, row * a.lddr + c0), c, n), c, n), dy);
#pragma unroll
          for (int k = 0; k < E; ++k) d[k] += dy[k];
        }
        store_vec<XT>(elem<XT>(a.dx, row * a.lddx + c0), c, n, narrow<XT>(d));
      }
    }
    if (pass == 0) m = row_sum(dot, T, red, 0) / static_cast<float>(a.cols);
  }
}

// Partial sums of dy n down the columns: 256 threads take 256 vectors of
// every gridDim.y-th row, four rows in flight.
template <int XT, bool CK>
__global__ __launch_bounds__(256) void dgamma_part(const NormBackArgs a) {
  constexpr int E = kVec<XT>, R = 4;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * (256 * E);
  const int c = threadIdx.x * E, n = left(a.cols - c0);
  const int64_t step = gridDim.y;
  float dg[E] = {};
  for (int64_t r0 = blockIdx.y; r0 < a.rows; r0 += step * R) {
    u32x4 wd[R];
    HRaw<XT, CK> hr[R];
    float r[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t row = r0 + i * step < a.rows ? r0 + i * step : a.rows - 1;   // read again, not used
      wd[i] = load_vec<XT>(elem<XT>(a.dy, row * a.lddy + c0), c, n);
      hr[i].template load<false>(a, row, c0, c, n);
      r[i] = a.rstd[row];
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float dy[E], h[E];
      hr[i].template trim<false>(c, n);
      widen<XT>(trim_vec<XT>(wd[i], c, n), dy);
      hr[i].values(a, h);
#pragma unroll
      for (int k = 0; k < E; ++k) dg[k] += r0 + i * step < a.rows ? dy[k] * (h[k] * r[i]) : 0.0f;
    }
  }
  float* p = a.part + static_cast<int64_t>(blockIdx.y) * a.cols + c0;
#pragma unroll
  for (int q = 0; q < E / 4; ++q)
    store_vec<AMP_F32>(p, c + 4 * q, n, u32x4{fbits(dg[4 * q]), fbits(dg[4 * q + 1]), fbits(dg[4 * q + 2]), fbits(dg[4 * q + 3])});
}

// dgamma[c] = sum over the P <= AMP_RMSNORM_PARTIALS rows of partial sums, in
// a fixed order: 32 columns a block, 8 lanes of 4 columns by 128 strands of
// rows, whose loads are all in flight together.
__global__ __launch_bounds__(1024) void dgamma_sum(const float* __restrict__ part, int P, int64_t cols,
                                                   float* __restrict__ dgamma) {
  constexpr int kStrands = 128, kLoads = AMP_RMSNORM_PARTIALS / kStrands;
  __shared__ float sums[kStrands][33], more[32][33];
  const int lane = threadIdx.x % 8, strand = threadIdx.x / 8;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * 32;
  const int n = left(cols - c0);
  u32x4 w[kLoads];
#pragma unroll
  for (int k = 0; k < kLoads; ++k) {
    const int p = strand + k * kStrands;
    w[k] = p < P ? load_vec<AMP_F32>(part + p * cols + c0, 4 * lane, n) : u32x4{0u, 0u, 0u, 0u};
  }
#pragma unroll
  for (int k = 0; k < kLoads; ++k) w[k] = trim_vec<AMP_F32>(w[k], 4 * lane, n);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < kLoads; ++k) t += bitsf(w[k][e]);
    sums[strand][4 * lane + e] = t;
  }
  __syncthreads();
  const int col = threadIdx.x % 32, group = threadIdx.x / 32;
  float t = 0.0f;
#pragma unroll
  for (int k = 0; k < kStrands / 32; ++k) t += sums[group * (kStrands / 32) + k][col];
  more[group][col] = t;
  __syncthreads();
  if (threadIdx.x < 32 && col < n) {
    t = 0.0f;
#pragma unroll
    for (int k = 0; k < 32; ++k) t += more[k][col];
    dgamma[c0 + col] = t;
  }
}

constexpr int64_t kFewRows = 512;   // rmsnorm_back_few

template <int XT, bool CK>
hipError_t dispatch_back(const NormBackArgs& a, float* dgamma, hipStream_t s) {
  const int64_t nv = (a.cols + kVec<XT> - 1) / kVec<XT>;
  int64_t blocks = 0;
#define AMP_BACK(V, S, B)                                                                              \
  do {                                                                                                 \
    blocks = (a.rows + (S) - 1) / (S);                                                                 \
    if (blocks > AMP_RMSNORM_PARTIALS) blocks = AMP_RMSNORM_PARTIALS;                                  \
    if (a.cols == static_cast<int64_t>((B) / (S)) * (V) * kVec<XT>)                                    \
      rmsnorm_back_rows<XT, CK, V, S, true><<<static_cast<unsigned>(blocks), B, 0, s>>>(a);            \
    else                                                                                               \
      rmsnorm_back_rows<XT, CK, V, S, false><<<static_cast<unsigned>(blocks), B, 0, s>>>(a);           \
  } while (0)
  // (not where dx takes the place of dy or h, which the columns' blocks still read)
  const bool over = a.dx && (a.dx == a.dy || a.dx == a.h);
  if (a.rows > 0 && a.rows <= kFewRows && nv <= 512 && !(dgamma && over)) {
    const int sums = dgamma ? static_cast<int>((a.cols + 31) / 32) : 0;
    const int S = nv <= 64 ? 8 : nv <= 128 ? 4 : nv <= 256 ? 2 : 1;
    const unsigned grid = static_cast<unsigned>(sums + (a.dx ? (a.rows + S - 1) / S : 0));
    if (S == 8) rmsnorm_back_few<XT, CK, 8><<<grid, 512, 0, s>>>(a, dgamma, sums);
    else if (S == 4) rmsnorm_back_few<XT, CK, 4><<<grid, 512, 0, s>>>(a, dgamma, sums);
    else if (S == 2) rmsnorm_back_few<XT, CK, 2><<<grid, 512, 0, s>>>(a, dgamma, sums);
    else rmsnorm_back_few<XT, CK, 1><<<grid, 512, 0, s>>>(a, dgamma, sums);
    return hipGetLastError();
  }
  if (a.rows > 0) {
    if (nv <= 64) AMP_BACK(1, 8, 512);
    else if (nv <= 128) AMP_BACK(1, 4, 512);
    else if (nv <= 256) AMP_BACK(1, 2, 512);
    else if (nv <= 512) AMP_BACK(1, 1, 512);
    else if (nv <= 1024) AMP_BACK(1, 1, 1024);
    else if (nv <= 2 * 1024) AMP_BACK(2, 1, 1024);
    else {
      if (dgamma) {   // before dx, which may take the place of dy or h
        // about eight blocks a CU, each with at least four rows
        const int64_t x = (nv + 255) / 256;
        blocks = (a.rows + 3) / 4 < 2048 / x + 1 ? (a.rows + 3) / 4 : 2048 / x + 1;
        if (blocks > AMP_RMSNORM_PARTIALS) blocks = AMP_RMSNORM_PARTIALS;
        dgamma_part<XT, CK><<<dim3(static_cast<unsigned>(x), static_cast<unsigned>(blocks)), 256, 0, s>>>(a);
      }
      // four vectors of 16-bit gradients and of codes with their scales do not
      // fit the registers (2000 x 32768: 198 us, walked twice 163)
      constexpr bool kFour = !CK || XT == AMP_F32;
      constexpr int64_t kMost = 1 << 21;   // rows a launch: a grid's threads are counted in 32 bits
      for (int64_t r0 = 0; a.dx && r0 < a.rows; r0 += kMost) {
        NormBackArgs b = a;
        b.dy = elem<XT>(a.dy, r0 * a.lddy);
        if (CK) { b.ck.q += r0 * a.ck.ldq; b.ck.s += r0; }
        else b.h = elem<XT>(a.h, r0 * a.ldh);
        b.rstd += r0;
        if (a.dres) b.dres = elem<XT>(a.dres, r0 * a.lddr);
        b.dx = elem<XT>(a.dx, r0 * a.lddx);
        const unsigned rows = static_cast<unsigned>(a.rows - r0 < kMost ? a.rows - r0 : kMost);
        if (nv <= 3 * 1024) rmsnorm_dx_rows<XT, CK, 3><<<rows, 1024, 0, s>>>(b);
        else if (kFour && nv <= 4 * 1024) rmsnorm_dx_rows<XT, CK, kFour ? 4 : 3><<<rows, 1024, 0, s>>>(b);
        else rmsnorm_dx_long<XT, CK><<<rows, 1024, 0, s>>>(b);
      }
    }
    if (hipError_t e = hipGetLastError()) return e;
  }
#undef AMP_BACK
  if (dgamma)
    dgamma_sum<<<static_cast<unsigned>((a.cols + 31) / 32), 1024, 0, s>>>(a.part, static_cast<int>(blocks), a.cols, dgamma);
  return hipGetLastError();
}

template <int XT>
hipError_t dispatch_back_h(const NormBackArgs& a, float* dgamma, hipStream_t s) {
  return a.ck.q ? dispatch_back<XT, true>(a, dgamma, s) : dispatch_back<XT, false>(a, dgamma, s);
}

}  // namespace

hipError_t launch_rmsnorm(const void* x, int xt, int64_t rows, int64_t cols, int64_t ldx, const void* res, int64_t ldr,
                          const void* gamma, int gt, float eps, void* h, int64_t ldh, void* y, int yt, int64_t ldy,
                          const float* scale, float* amax, const amp_fp8_tiles& yq, const amp_fp8_tiles& ckpt,
                          float* rstd, hipStream_t s) {
  const NormArgs a{x, ldx, res, ldr, gamma, gt, eps, h, ldh, y, yt, ldy, scale, amax, yq, ckpt, rstd, rows, cols};
  switch (xt) {
    case AMP_F32: return dispatch_rmsnorm<AMP_F32>(a, s);
    case AMP_BF16: return dispatch_rmsnorm<AMP_BF16>(a, s);
    default: return dispatch_rmsnorm<AMP_F16>(a, s);
  }
}

hipError_t launch_rmsnorm_backward(const void* dy, int dt, int64_t rows, int64_t cols, int64_t lddy, const void* h,
                                   int64_t ldh, const amp_fp8_tiles& ckpt, const void* gamma, int gt,
                                   const float* rstd, const void* dres, int64_t lddr, void* dx, int64_t lddx,
                                   float* dgamma, float* work, hipStream_t s) {
  const NormBackArgs a{dy, lddy, h, ldh, ckpt, gamma, gt, rstd, dres, lddr, dx, lddx, dgamma ? work : nullptr, rows, cols};
  switch (dt) {
    case AMP_F32: return dispatch_back_h<AMP_F32>(a, dgamma, s);
    case AMP_BF16: return dispatch_back_h<AMP_BF16>(a, dgamma, s);
    default: return dispatch_back_h<AMP_F16>(a, dgamma, s);
  }
}

}  // namespace amp
