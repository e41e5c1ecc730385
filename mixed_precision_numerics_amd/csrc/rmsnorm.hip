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

template <int XT>
__device__ __forceinline__ const void* row_of(const void* p, int64_t i) {
  return XT == AMP_F32 ? static_cast<const void*>(static_cast<const float*>(p) + i)
                       : static_cast<const void*>(static_cast<const uint16_t*>(p) + i);
}
template <int XT>
__device__ __forceinline__ void* row_of(void* p, int64_t i) {
  return const_cast<void*>(row_of<XT>(const_cast<const void*>(p), i));
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
  return v;
}

// Sum over the T threads of a row (T >= 64; every thread of the block calls).
// `red` holds two sets of T / 64 words used in turn, so one barrier a row is
// enough: a wave that runs ahead writes the other set.
template <int T>
__device__ __forceinline__ float row_sum(float v, float* red, int turn) {
  v = wave_sum(v);
  if constexpr (T > kWave) {
    constexpr int W = T / kWave;
    const int w = threadIdx.x / kWave, first = w / W * W;
    float* set = red + turn * (blockDim.x / kWave);
    if (threadIdx.x % kWave == 0) set[w] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int k = 0; k < W; ++k) v += set[first + k];
  }
  return v;
}

// x + res rounded to the stream's type, one vector.
template <int XT>
__device__ __forceinline__ u32x4 join(u32x4 w, const NormArgs& a, int64_t row, int64_t c) {
  constexpr int E = kVec<XT>;
  float p[E], q[E];
  widen<XT>(w, p);
  widen<XT>(load_vec<XT>(row_of<XT>(a.res, row * a.ldr), c, a.cols), q);
#pragma unroll
  for (int k = 0; k < E; ++k) p[k] += q[k];
  return narrow<XT>(p);
}

// Every output of one vector of h; returns its |y| maximum.
template <int XT>
__device__ __forceinline__ float norm_outputs(const NormArgs& a, u32x4 w, int64_t row, int64_t c, bool live, float r, float scale) {
  constexpr int E = kVec<XT>;
  float h[E], gm[E], y[E];
  widen<XT>(w, h);
  load_cols<E>(a.gamma, a.gt, c, a.cols, gm);
#pragma unroll
  for (int k = 0; k < E; ++k) y[k] = h[k] * r * gm[k];
  const float am = abs_max<E>(0.0f, y);
  if (a.yq.q) store_tile<E>(a.yq, row, c, a.cols, c / kTileK, live, y);
  if (a.ck.q) store_tile<E>(a.ck, row, c, a.cols, c / kTileK, live, h);
  if (a.y && live) store_plain<E>(a.y, a.yt, row * a.ldy, c, a.cols, scale, am, y);
  return am;
}

// T threads hold a row in registers, V vectors each; B threads a block.
template <int XT, int T, int V, int B>
__global__ __launch_bounds__(B) void rmsnorm_rows(const NormArgs a) {
  constexpr int E = kVec<XT>;
  __shared__ float red[2 * (B / kWave)];
  __shared__ uint32_t redm[B / kWave];
  const int tid = threadIdx.x % T, sub = threadIdx.x / T;
  const float scale = a.scale ? *a.scale : 1.0f;
  float am = 0.0f;
  int turn = 0;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * (B / T); r0 < a.rows; r0 += static_cast<int64_t>(gridDim.x) * (B / T)) {
    const int64_t row = r0 + sub;
    const bool live = row < a.rows;
    u32x4 w[V];
    float ss = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int64_t c = static_cast<int64_t>(v * T + tid) * E;
      w[v] = u32x4{0u, 0u, 0u, 0u};
      if (live) w[v] = load_vec<XT>(row_of<XT>(a.x, row * a.ldx), c, a.cols);
    }
    if (a.res) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (live) w[v] = join<XT>(w[v], a, row, static_cast<int64_t>(v * T + tid) * E);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float h[E];
      widen<XT>(w[v], h);
#pragma unroll
      for (int k = 0; k < E; ++k) ss += h[k] * h[k];
    }
    if (a.h && live) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        store_vec<XT>(row_of<XT>(a.h, row * a.ldh), static_cast<int64_t>(v * T + tid) * E, a.cols, w[v]);
    }
    ss = row_sum<T>(ss, red, turn);
    turn ^= 1;
    const float r = 1.0f / sqrtf(ss / static_cast<float>(a.cols) + a.eps);
    if (a.rstd && live && tid == 0) a.rstd[row] = r;
#pragma unroll
    for (int v = 0; v < V; ++v)
      am = __builtin_elementwise_maximum(am, norm_outputs<XT>(a, w[v], row, static_cast<int64_t>(v * T + tid) * E, live, r, scale));
  }
  if (a.amax) {
    const uint32_t m = block_max_u32<B>(mag(am), redm);
    if (threadIdx.x == 0 && m != 0) amax_update(a.amax, m);
  }
}

// Rows too long for the registers: a block walks its row twice (the second
// reads come from the caches).  In place, h is what the second walk reads.
template <int XT>
__global__ __launch_bounds__(1024) void rmsnorm_long(const NormArgs a) {
  constexpr int E = kVec<XT>, T = 1024;
  __shared__ float red[2 * (T / kWave)];
  __shared__ uint32_t redm[T / kWave];
  const float scale = a.scale ? *a.scale : 1.0f;
  float am = 0.0f;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    float ss = 0.0f;
    for (int64_t c = static_cast<int64_t>(threadIdx.x) * E; c < a.cols; c += T * E) {
      u32x4 w = load_vec<XT>(row_of<XT>(a.x, row * a.ldx), c, a.cols);
      if (a.res) w = join<XT>(w, a, row, c);
      if (a.h) store_vec<XT>(row_of<XT>(a.h, row * a.ldh), c, a.cols, w);
      float h[E];
      widen<XT>(w, h);
#pragma unroll
      for (int k = 0; k < E; ++k) ss += h[k] * h[k];
    }
    ss = row_sum<T>(ss, red, turn);
    turn ^= 1;
    const float r = 1.0f / sqrtf(ss / static_cast<float>(a.cols) + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = r;
    // whole waves stay in the loop: a tile's lanes exchange their maxima
    for (int64_t c0 = 0; c0 < a.cols; c0 += T * E) {
      const int64_t c = c0 + static_cast<int64_t>(threadIdx.x) * E;
      u32x4 w;
      if (a.h) {
        w = load_vec<XT>(row_of<XT>(a.h, row * a.ldh), c, a.cols);
      } else {
        w = load_vec<XT>(row_of<XT>(a.x, row * a.ldx), c, a.cols);
        if (a.res) w = join<XT>(w, a, row, c);
      }
      am = __builtin_elementwise_maximum(am, norm_outputs<XT>(a, w, row, c, true, r, scale));
    }
  }
  if (a.amax) {
    const uint32_t m = block_max_u32<T>(mag(am), redm);
    if (threadIdx.x == 0 && m != 0) amax_update(a.amax, m);
  }
}

template <int XT>
hipError_t dispatch_rmsnorm(const NormArgs& a, hipStream_t s) {
  const int64_t nv = (a.cols + kVec<XT> - 1) / kVec<XT>;
#define AMP_NORM(T, V, B)                                                                              \
  do {                                                                                                 \
    int64_t blocks = (a.rows + (B) / (T) - 1) / ((B) / (T));                                           \
    if (blocks > (1 << 20)) blocks = 1 << 20;                                                          \
    rmsnorm_rows<XT, T, V, B><<<static_cast<unsigned>(blocks), B, 0, s>>>(a);                          \
  } while (0)
  if (nv <= 64) AMP_NORM(64, 1, 256);
  else if (nv <= 128) AMP_NORM(64, 2, 256);
  else if (nv <= 256) AMP_NORM(64, 4, 256);
  else if (nv <= 512) AMP_NORM(256, 2, 256);
  else if (nv <= 1024) AMP_NORM(256, 4, 256);
  else if (nv <= 2048) AMP_NORM(1024, 2, 1024);
  else if (nv <= 8192) AMP_NORM(1024, 8, 1024);
  else rmsnorm_long<XT><<<static_cast<unsigned>(a.rows < (1 << 20) ? a.rows : (1 << 20)), 1024, 0, s>>>(a);
#undef AMP_NORM
  return hipGetLastError();
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

// One vector of h from the stored tensor (type XT) or the checkpoint.
template <int XT, bool CK>
struct HRaw {
  static constexpr int E = kVec<XT>;
  u32x4 w;
  uint32_t q[E / 4];
  float s;
  __device__ __forceinline__ void load(const NormBackArgs& a, int64_t row, int64_t c) {
    if constexpr (CK) {
      load_codes<E>(a.ck.q + row * a.ck.ldq, c, a.cols, q);
      s = c < a.cols ? a.ck.s[c / kTileK * a.ck.lds + row] : 0.0f;
    } else {
      w = load_vec<XT>(row_of<XT>(a.h, row * a.ldh), c, a.cols);
    }
  }
  __device__ __forceinline__ void values(const NormBackArgs& a, float (&v)[E]) const {
    if constexpr (CK) decode<E>(a.ck.type, q, s, v);
    else widen<XT>(w, v);
  }
};

// T threads a row, V vectors each, B / T rows in flight a block; a block
// strides over the rows with its sums of dy n in registers and writes one row
// of partial sums at the end (no atomics: the result does not depend on the
// order in which blocks run).
template <int XT, bool CK, int T, int V, int B>
__global__ __launch_bounds__(B) void rmsnorm_back_rows(const NormBackArgs a) {
  constexpr int E = kVec<XT>, S = B / T;
  __shared__ float red[2 * (B / kWave)];
  __shared__ float sums[S > 1 ? T * V * E : 1];
  const int tid = threadIdx.x % T, sub = threadIdx.x / T;
  float dg[V][E] = {};
  const float inv_n = 1.0f / static_cast<float>(a.cols);
  int turn = 0;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * S; r0 < a.rows; r0 += static_cast<int64_t>(gridDim.x) * S) {
    const int64_t row = r0 + sub;
    const bool live = row < a.rows;
    u32x4 wd[V];
    HRaw<XT, CK> hr[V];
    if (live) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int64_t c = static_cast<int64_t>(v * T + tid) * E;
        wd[v] = load_vec<XT>(row_of<XT>(a.dy, row * a.lddy), c, a.cols);
        hr[v].load(a, row, c);
      }
    }
    const float r = live ? a.rstd[row] : 0.0f;
    float dot = 0.0f;
    if (live) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float dy[E], h[E], gm[E];
        widen<XT>(wd[v], dy);
        hr[v].values(a, h);
        load_cols<E>(a.gamma, a.gt, static_cast<int64_t>(v * T + tid) * E, a.cols, gm);
#pragma unroll
        for (int k = 0; k < E; ++k) {
          const float n = h[k] * r;
          dot += dy[k] * gm[k] * n;
          dg[v][k] += dy[k] * n;
        }
      }
    }
    if (a.dx) {
      const float m = row_sum<T>(dot, red, turn) * inv_n;
      turn ^= 1;
      if (live) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int64_t c = static_cast<int64_t>(v * T + tid) * E;
          float dy[E], h[E], gm[E], d[E] = {};
          widen<XT>(wd[v], dy);
          hr[v].values(a, h);
          load_cols<E>(a.gamma, a.gt, c, a.cols, gm);
          if (a.dres) widen<XT>(load_vec<XT>(row_of<XT>(a.dres, row * a.lddr), c, a.cols), d);
#pragma unroll
          for (int k = 0; k < E; ++k) {
            const float t = r * (dy[k] * gm[k] - h[k] * r * m);
            d[k] = a.dres ? t + d[k] : t;
          }
          store_vec<XT>(row_of<XT>(a.dx, row * a.lddx), c, a.cols, narrow<XT>(d));
        }
      }
    }
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
    const int64_t c = static_cast<int64_t>(v * T + tid) * E;
#pragma unroll
    for (int q = 0; q < E / 4; ++q) {
      const float4 f = {dg[v][4 * q], dg[v][4 * q + 1], dg[v][4 * q + 2], dg[v][4 * q + 3]};
      const u32x4 w = {fbits(f.x), fbits(f.y), fbits(f.z), fbits(f.w)};
      store_vec<AMP_F32>(p, c + 4 * q, a.cols, w);
    }
  }
}

// Rows too long for the registers: two walks, the partial sums kept in the
// block's own row of the work area.
template <int XT, bool CK>
__global__ __launch_bounds__(1024) void rmsnorm_back_long(const NormBackArgs a) {
  constexpr int E = kVec<XT>, T = 1024;
  __shared__ float red[2 * (T / kWave)];
  const float inv_n = 1.0f / static_cast<float>(a.cols);
  float* p = a.part ? a.part + static_cast<int64_t>(blockIdx.x) * a.cols : nullptr;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float r = a.rstd[row];
    float dot = 0.0f;
    for (int64_t c = static_cast<int64_t>(threadIdx.x) * E; c < a.cols; c += T * E) {
      float dy[E], h[E], gm[E];
      HRaw<XT, CK> hr;
      widen<XT>(load_vec<XT>(row_of<XT>(a.dy, row * a.lddy), c, a.cols), dy);
      hr.load(a, row, c);
      hr.values(a, h);
      load_cols<E>(a.gamma, a.gt, c, a.cols, gm);
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const float n = h[k] * r;
        dot += dy[k] * gm[k] * n;
        if (p && c + k < a.cols) p[c + k] = (row == blockIdx.x ? 0.0f : p[c + k]) + dy[k] * n;
      }
    }
    if (a.dx) {
      const float m = row_sum<T>(dot, red, turn) * inv_n;
      turn ^= 1;
      for (int64_t c = static_cast<int64_t>(threadIdx.x) * E; c < a.cols; c += T * E) {
        float dy[E], h[E], gm[E], d[E] = {};
        HRaw<XT, CK> hr;
        widen<XT>(load_vec<XT>(row_of<XT>(a.dy, row * a.lddy), c, a.cols), dy);
        hr.load(a, row, c);
        hr.values(a, h);
        load_cols<E>(a.gamma, a.gt, c, a.cols, gm);
        if (a.dres) widen<XT>(load_vec<XT>(row_of<XT>(a.dres, row * a.lddr), c, a.cols), d);
#pragma unroll
        for (int k = 0; k < E; ++k) {
          const float t = r * (dy[k] * gm[k] - h[k] * r * m);
          d[k] = a.dres ? t + d[k] : t;
        }
        store_vec<XT>(row_of<XT>(a.dx, row * a.lddx), c, a.cols, narrow<XT>(d));
      }
    }
  }
}

// dgamma[c] = sum over the P rows of partial sums, in a fixed order: 32
// columns a block, 8 lanes of 4 columns by 32 strands of rows.
__global__ __launch_bounds__(256) void dgamma_sum(const float* __restrict__ part, int64_t P, int64_t cols,
                                                  float* __restrict__ dgamma) {
  __shared__ float sums[32][33];
  const int lane = threadIdx.x % 8, strand = threadIdx.x / 8;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + 4 * lane;
  float t[4] = {};
  for (int64_t p = strand; p < P; p += 32) {
    const u32x4 w = load_vec<AMP_F32>(part + p * cols, c, cols);
#pragma unroll
    for (int k = 0; k < 4; ++k) t[k] += bitsf(w[k]);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) sums[strand][4 * lane + k] = t[k];
  __syncthreads();
  if (threadIdx.x < 32) {
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < 32; ++k) v += sums[k][threadIdx.x];
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
    if (col < cols) dgamma[col] = v;
  }
}

template <int XT, bool CK>
hipError_t dispatch_back(const NormBackArgs& a, float* dgamma, hipStream_t s) {
  const int64_t nv = (a.cols + kVec<XT> - 1) / kVec<XT>;
  int64_t blocks = 0;
#define AMP_BACK(T, V, B)                                                                              \
  do {                                                                                                 \
    blocks = (a.rows + (B) / (T) - 1) / ((B) / (T));                                                   \
    if (blocks > AMP_RMSNORM_PARTIALS) blocks = AMP_RMSNORM_PARTIALS;                                  \
    rmsnorm_back_rows<XT, CK, T, V, B><<<static_cast<unsigned>(blocks), B, 0, s>>>(a);                 \
  } while (0)
  if (a.rows > 0) {
    if (nv <= 64) AMP_BACK(64, 1, 512);
    else if (nv <= 128) AMP_BACK(64, 2, 512);
    else if (nv <= 256) AMP_BACK(128, 2, 512);
    else if (nv <= 512) AMP_BACK(256, 2, 512);
    else if (nv <= 1024) AMP_BACK(512, 2, 512);
    else if (nv <= 2048) AMP_BACK(1024, 2, 1024);
    else if (nv <= 4096) AMP_BACK(1024, 4, 1024);
    else {
      blocks = a.rows < AMP_RMSNORM_PARTIALS ? a.rows : AMP_RMSNORM_PARTIALS;
      rmsnorm_back_long<XT, CK><<<static_cast<unsigned>(blocks), 1024, 0, s>>>(a);
    }
    if (hipError_t e = hipGetLastError()) return e;
  }
#undef AMP_BACK
  if (dgamma)
    dgamma_sum<<<static_cast<unsigned>((a.cols + 31) / 32), 256, 0, s>>>(a.part, blocks, a.cols, dgamma);
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
