// Gated activation with 16-bit or FP8 outputs, and its backward pass from the
// stored input or from an FP8 checkpoint (gfx950).
//
//   x = [g | u],  s = 1 / (1 + exp(-g)),  y = g s u
//   du = dy g s,  dg = dy u s (1 + g (1 - s))
//
// FP32 arithmetic, one rounding per output.  With e = exp(-g) the factor
// 1 - s is e s, which keeps its relative precision where s is near 1.
#include "tiles.hpp"

namespace amp {
namespace {

struct GateArgs {
  const void* x; int64_t ldx;
  const void* dy; int64_t lddy;
  void* y; int yt; int64_t ldy;
  const float* scale; float* amax;
  amp_fp8_tiles yq, ck;          // forward: outputs; backward: ck is the input
  amp_fp8_tiles dxq, dxqt, yqt;  // backward
  int64_t rows, cols;
};

// s = 1 / (1 + e), e = exp(-g), from the hardware's exponential and
// reciprocal (each within an ulp; the scaled argument's roundings grow with
// |g|, so that e is off by up to |g| 2^-22 and s by that times 1 - s).  Below g
// = -87 s leaves the normal range and may be 0, as e overflows at -89.  g = -inf
// gives s = 0 and, as in the formula, 0 * inf = NaN for g s.  Where e overflows
// s is 0 and e s a NaN, of which the minimum makes 1 (a NaN g leaves one in s).
struct Gate { float s, om; };   // s and 1 - s
__device__ __forceinline__ Gate gate(float g) {
  const float e = __builtin_amdgcn_exp2f(g * -1.4426950408889634f);
  const float s = __builtin_amdgcn_rcpf(1.0f + e);
  return {s, __builtin_fminf(e * s, 1.0f)};
}

// Index along K of the tile that holds column c of half `half`: the tiles
// start again at the second half.
__device__ __forceinline__ int64_t tile_of(int64_t c, int half, int64_t cols) {
  return c / kTileK + (half ? (cols + kTileK - 1) / kTileK : 0);
}

// One vector of R rows (S apart, from row0 on) in 1x128 tiles; `blk` is the
// tile's index along K.  Lane i of a tile's lane group stores row i's scale.
template <int E, int R, bool FULL>
__device__ __forceinline__ void store_row_tiles(const amp_fp8_tiles& o, int64_t row0, int S, int64_t rows, int64_t c0, int c,
                                                int n, int64_t blk, const float (&v)[R][E]) {
  constexpr int G = kTileK / E;
  uint32_t m[R], top = 0, w[R][E / 4];
  float sc[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    m[i] = group_max<G>(mag(abs_max<E>(0.0f, v[i])));
    top = top > m[i] ? top : m[i];
  }
  const float inv = tile_scales<R>(m, fp8_max(o.type), sc);
  const int64_t mine = row0 + (threadIdx.x & 3) * S;
  if (threadIdx.x % G < R && mine < rows && (FULL || c / kTileK * kTileK < n)) o.s[blk * o.lds + mine] = inv;
  encode<R, E, false>(o.type, top >= kInfBits, w, [&](int i, int k) __attribute__((always_inline)) { return v[i][k] * sc[i]; });
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (row0 + i * S < rows) store_codes<E, FULL>(o.q + (row0 + i * S) * o.ldq + c0, c, n, w[i]);
}

// W threads cover W vectors of a row, 256 / W rows side by side and R of
// those groups one after the other; blockIdx.x runs along the row.  FULL: the
// row is whole spans of W vectors.  HBM-bound: 8192 x 14336 BF16 with tiles and
// checkpoint 137 us = 6.1 TB/s, 4096 x 14336 FP32 102 = 6.4; one row of 14336 2.5
// us in a captured graph, the launch.
template <int XT, int W, int R, bool FULL>
__global__ __launch_bounds__(256) void swiglu_rows(const GateArgs a) {
  constexpr int E = kVec<XT>, S = 256 / W;
  __shared__ uint32_t redm[256 / kWave];
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * (W * E);   // the block's first column
  const int c = threadIdx.x % W * E, n = left(a.cols - c0);
  const int sub = W >= kWave ? __builtin_amdgcn_readfirstlane(threadIdx.x / W) : threadIdx.x / W;
  const int64_t row0 = static_cast<int64_t>(blockIdx.y) * (S * R) + sub;
  const float scale = a.scale ? *a.scale : 1.0f;
  const uint32_t seen = amax_seen(a.amax);
  u32x4 wg[R], wu[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t row = row0 + i * S;
    wg[i] = wu[i] = u32x4{0u, 0u, 0u, 0u};
    if (row < a.rows) {
      const void* p = elem<XT>(a.x, row * a.ldx + c0);
      wg[i] = load_vec<XT, FULL>(p, c, n);
      wu[i] = load_vec<XT, FULL>(elem<XT>(p, a.cols), c, n);
    }
  }
  float y[R][E], am = 0.0f;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    float g[E], u[E];
    wg[i] = trim_vec<XT, FULL>(wg[i], c, n);
    wu[i] = trim_vec<XT, FULL>(wu[i], c, n);
    widen<XT>(wg[i], g);
    widen<XT>(wu[i], u);
#pragma unroll
    for (int k = 0; k < E; ++k) y[i][k] = g[k] * gate(g[k]).s * u[k];
    am = abs_max<E>(am, y[i]);
  }
  if (a.y) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t row = row0 + i * S, at = (row * a.ldy + c0) * (a.yt == AMP_F16 || a.yt == AMP_BF16 ? 2 : 1);
      store_plain<1, E, FULL>(static_cast<uint8_t*>(a.y) + at, a.yt, c, 0, n, row < a.rows, scale, am,
                              reinterpret_cast<const float(&)[1][E]>(y[i]));
    }
  }
  if (a.yq.q) store_row_tiles<E, R, FULL>(a.yq, row0, S, a.rows, c0, c, n, (c0 + c) / kTileK, y);
  if (a.ck.q) {
#pragma unroll
    for (int i = 0; i < R; ++i) widen<XT>(wg[i], y[i]);
    store_row_tiles<E, R, FULL>(a.ck, row0, S, a.rows, c0, c, n, tile_of(c0 + c, 0, a.cols), y);
#pragma unroll
    for (int i = 0; i < R; ++i) widen<XT>(wu[i], y[i]);
    amp_fp8_tiles up = a.ck;
    up.q += a.cols;
    store_row_tiles<E, R, FULL>(up, row0, S, a.rows, c0, c, n, tile_of(c0 + c, 1, a.cols), y);
  }
  if (a.amax) block_amax(am, seen, redm, a.amax);
}

// Backward with dx in the gradient's own type only: element-wise, laid out
// as above; HBM-bound (8192 x 14336 BF16 stored 182 us = 6.4 TB/s, from a
// checkpoint 151 = 6.3; 777 x 2049 FP16 stored 6.0 in a captured graph, 776 x 2048
// 3.9, 2.8 at the copy rate: rows of odd length begin at any byte, which reads
// 1.26 times the bytes).
template <int XT, bool CK, int W, int R, bool FULL>
__global__ __launch_bounds__(256) void swiglu_back_rows(const GateArgs a) {
  constexpr int E = kVec<XT>, S = 256 / W;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * (W * E);
  const int c = threadIdx.x % W * E, n = left(a.cols - c0);
  const int sub = W >= kWave ? __builtin_amdgcn_readfirstlane(threadIdx.x / W) : threadIdx.x / W;
  const int64_t row0 = static_cast<int64_t>(blockIdx.y) * (S * R) + sub;
  if (!FULL && c >= n) return;
  u32x4 wd[R], wg[R], wu[R];
  uint32_t qg[R][E / 4], qu[R][E / 4];
  float sg[R], su[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t row = row0 + i * S < a.rows ? row0 + i * S : a.rows - 1;   // read again, not used
    wd[i] = load_vec<XT, FULL>(elem<XT>(a.dy, row * a.lddy + c0), c, n);
    if constexpr (CK) {
      const uint8_t* q = a.ck.q + row * a.ck.ldq + c0;
      load_codes<E, FULL>(q, c, n, qg[i]);
      load_codes<E, FULL>(q + a.cols, c, n, qu[i]);
      sg[i] = a.ck.s[tile_of(c0 + c, 0, a.cols) * a.ck.lds + row];
      su[i] = a.ck.s[tile_of(c0 + c, 1, a.cols) * a.ck.lds + row];
    } else {
      const void* p = elem<XT>(a.x, row * a.ldx + c0);
      wg[i] = load_vec<XT, FULL>(p, c, n);
      wu[i] = load_vec<XT, FULL>(elem<XT>(p, a.cols), c, n);
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t row = row0 + i * S;
    if (row >= a.rows) return;
    float g[E], u[E], dy[E], dg[E], du[E];
    widen<XT>(trim_vec<XT, FULL>(wd[i], c, n), dy);
    if constexpr (CK) {
      trim_codes<E, FULL>(qg[i], c, n);
      trim_codes<E, FULL>(qu[i], c, n);
      decode<E>(a.ck.type, qg[i], sg[i], g);
      decode<E>(a.ck.type, qu[i], su[i], u);
    } else {
      widen<XT>(trim_vec<XT, FULL>(wg[i], c, n), g);
      widen<XT>(trim_vec<XT, FULL>(wu[i], c, n), u);
    }
#pragma unroll
    for (int k = 0; k < E; ++k) {
      const Gate p = gate(g[k]);
      const float t = dy[k] * p.s;
      du[k] = t * g[k];
      dg[k] = t * u[k] * __builtin_fmaf(g[k], p.om, 1.0f);
    }
    void* p = elem<XT>(a.y, row * a.ldy + c0);
    store_vec<XT, FULL>(p, c, n, narrow<XT>(dg));
    store_vec<XT, FULL>(elem<XT>(p, a.cols), c, n, narrow<XT>(du));
  }
}

// Backward with FP8 operands: one 128x128 region of dy, g and u per block,
// read once.  DX: some form of dx is asked for, not y^T alone.  dg and du are
// formed in registers and leave from there in every form asked for: dx in dy's
// type, dx in row tiles (dgrad), dx^T in tiles along the rows (wgrad).  Then y
// leaves as y^T.  From a checkpoint dg, du and two blocks a CU take every
// register, so y is formed again from g and u, except for the kKeep rows a
// thread that the LDS has room for; stored inputs take twice the registers and
// one block a CU (held to two they spilled, 4096 x 14336 BF16 330 us), whose
// LDS holds all of y.
//
// Bound by the vector ALUs and the two blocks' turns on them (8192 x 14336
// from a checkpoint: 236 us = 4.6 TB/s, 51 operations per element of y, the
// ALUs 74 % busy; 257 us with no row kept, 237 with two).  Stored, 4096 x 14336 BF16: 178 us with all of y kept,
// 184 with none.
template <int XT, bool CK, bool DX>
__global__ __launch_bounds__(kRegThreads, CK ? 4 : 2) void swiglu_back_region(const GateArgs a) {
  __shared__ RegLds<2> l;
  __shared__ uint32_t rmax[2][kTileK];
  __shared__ float rscale[2][kTileK], gscale[2][kTileK];
  constexpr int kKeep = CK ? 1 : kRegRows, kFirst = kRegRows - kKeep;   // y is kept of rows kFirst on
  __shared__ u32x4 kept[kKeep][kRegCols / 4][kRegThreads];
  constexpr int GB = CK ? 1 : kBytes<XT>;
  const Region g(a.rows, a.cols, true);
  const int t = threadIdx.x;
  RegRaw<kBytes<XT>> xd;
  RegRaw<GB> xg, xu;
#pragma unroll
  for (int i = 0; i < kRegRows; ++i) {
    const int64_t row = g.row(i);
    xd.load(g, i, elem<XT>(a.dy, row * a.lddy + g.c0));
    const uint8_t* p = CK ? a.ck.q + row * a.ck.ldq + g.c0 : static_cast<const uint8_t*>(elem<XT>(a.x, row * a.ldx + g.c0));
    xg.load(g, i, p);
    xu.load(g, i, p + a.cols * GB);
  }
  if constexpr (CK) {
    if (t < 2 * kTileK) {
      const int r = t % kTileK;   // 0 past the last row: the zeros there stay zeros
      gscale[t / kTileK][r] = r < g.nrows ? a.ck.s[tile_of(g.c0, t / kTileK, a.cols) * a.ck.lds + g.r0 + r] : 0.0f;
    }
  }
  xd.trim(g);
  xg.trim(g);
  xu.trim(g);
  if constexpr (CK) __syncthreads();
  auto gu = [&](int i, float (&vg)[kRegCols], float (&vu)[kRegCols]) __attribute__((always_inline)) {
    if constexpr (CK) {
      decode<kRegCols>(a.ck.type, xg.w[i], gscale[0][g.r() + i], vg);
      decode<kRegCols>(a.ck.type, xu.w[i], gscale[1][g.r() + i], vu);
    } else {
      reg_values<XT>(xg.w[i], vg);
      reg_values<XT>(xu.w[i], vu);
    }
  };
  if constexpr (DX) {
    float v[2][kRegRows][kRegCols];   // dg, du
#pragma unroll
    for (int i = 0; i < kRegRows; ++i) {
      float vg[kRegCols], vu[kRegCols], dy[kRegCols];
      gu(i, vg, vu);
      reg_values<XT>(xd.w[i], dy);
#pragma unroll
      for (int k = 0; k < kRegCols; ++k) {
        const Gate p = gate(vg[k]);
        const float d = dy[k] * p.s;
        v[0][i][k] = d * vu[k] * __builtin_fmaf(vg[k], p.om, 1.0f);
        v[1][i][k] = d * vg[k];
        vu[k] = vg[k] * p.s * vu[k];
      }
      if (i >= kFirst) {
#pragma unroll
        for (int q = 0; q < kRegCols / 4; ++q)
          kept[i - kFirst][q][t] = u32x4{fbits(vu[4 * q]), fbits(vu[4 * q + 1]), fbits(vu[4 * q + 2]), fbits(vu[4 * q + 3])};
      }
    }
    if (a.y) {
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < kRegRows; ++i) {
          if (g.r() + i >= g.nrows) continue;
          void* p = elem<XT>(a.y, g.row(i) * a.ldy + (n ? a.cols : 0) + g.c0);
          constexpr int E = kVec<XT>;
#pragma unroll
          for (int q = 0; q < kRegCols / E; ++q)
            store_vec<XT>(p, g.c() + q * E, g.ncols, narrow<XT>(reinterpret_cast<const float(&)[E]>(v[n][i][q * E])));
        }
    }
    const amp_fp8_tiles o[2] = {a.dxqt, a.dxqt};
    const int64_t first[2] = {g.c0, a.cols + g.c0};
    if (a.dxq.q) {
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < kRegRows; ++i) {
          const uint32_t m = group_max<16>(mag(abs_max<kRegCols>(0.0f, v[n][i])));
          if (t % 16 == 0) rmax[n][g.r() + i] = m;
        }
    }
    if (a.dxqt.q) reg_maxima<2>(l, g, v);
    __syncthreads();
    if (a.dxqt.q) reg_scales<2>(l, g, o, first);
    if (a.dxq.q && t >= 2 * kTileK) {
      const int n = (t - 2 * kTileK) / kTileK, r = t % kTileK;
      const uint32_t m = rmax[n][r];
      const float sc = scale_of(m, fp8_max(a.dxq.type));
      rscale[n][r] = m >= kInfBits ? -sc : sc;   // sign: the tile holds a NaN or infinity
      if (r < g.nrows) a.dxq.s[tile_of(g.c0, n, a.cols) * a.dxq.lds + g.r0 + r] = 1.0f / sc;
    }
    __syncthreads();
    if (a.dxq.q) {
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        float sc[kRegRows];
        uint32_t w[kRegRows][2];
        bool special = false;
#pragma unroll
        for (int i = 0; i < kRegRows; ++i) {
          sc[i] = rscale[n][g.r() + i];
          special |= sc[i] < 0.0f;
        }
        encode<kRegRows, kRegCols, false>(a.dxq.type, special, w,
                                          [&](int i, int k) __attribute__((always_inline)) { return v[n][i][k] * fabsf(sc[i]); });
        // cols is a multiple of 128 here
#pragma unroll
        for (int i = 0; i < kRegRows; ++i)
          if (g.r() + i < g.nrows)
            *reinterpret_cast<u32x2_any*>(a.dxq.q + g.row(i) * a.dxq.ldq + (n ? a.cols : 0) + g.c0 + g.c()) = u32x2{w[i][0], w[i][1]};
      }
    }
    if (a.dxqt.q) {
      reg_codes<2>(l, g, o, first, v);
      if (a.yqt.q) __syncthreads();
    }
  }
  if (a.yqt.q) {
    float v[1][kRegRows][kRegCols];
#pragma unroll
    for (int i = 0; i < kRegRows; ++i) {
      if (DX && i >= kFirst) {
#pragma unroll
        for (int k = 0; k < kRegCols; ++k) v[0][i][k] = bitsf(kept[i - kFirst][k / 4][t][k % 4]);
      } else {
        float vg[kRegCols], vu[kRegCols];
        gu(i, vg, vu);
#pragma unroll
        for (int k = 0; k < kRegCols; ++k) v[0][i][k] = vg[k] * gate(vg[k]).s * vu[k];
      }
    }
    const amp_fp8_tiles o[1] = {a.yqt};
    const int64_t first[1] = {g.c0};
    RegLds<1>& l1 = reinterpret_cast<RegLds<1>&>(l);
    reg_maxima<1>(l1, g, v);
    __syncthreads();
    reg_scales<1>(l1, g, o, first);
    __syncthreads();
    reg_codes<1>(l1, g, o, first, v);
  }
}

// The widest W whose whole vectors overshoot the row by at most an eighth
// (a tile's lanes stay together in every case).
int row_width(int64_t cols, int e) {
  for (int w : {256, 64}) {
    const int64_t span = static_cast<int64_t>(w) * e;
    if ((cols + span - 1) / span * span * 8 <= cols * 9) return w;
  }
  return 32;
}

// Calls f(first row, rows) for slices of at most `most` rows.
template <typename F>
hipError_t in_slices(int64_t rows, int64_t most, F f) {
  for (int64_t r0 = 0; r0 < rows; r0 += most) {
    f(r0, rows - r0 < most ? rows - r0 : most);
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

template <int XT, int W, int R>
hipError_t run_swiglu(const GateArgs& whole, hipStream_t s) {
  constexpr int E = kVec<XT>, per = 256 / W * R;
  const bool full = whole.cols % (W * E) == 0;
  return in_slices(whole.rows, grid_rows((whole.cols + W * E - 1) / (W * E)) * per, [&](int64_t r0, int64_t rows) {
    GateArgs a = whole;
    a.rows = rows;
    a.x = elem<XT>(a.x, r0 * a.ldx);
    if (a.y) a.y = static_cast<uint8_t*>(a.y) + r0 * a.ldy * dtype_bytes(a.yt);
    if (a.yq.q) { a.yq.q += r0 * a.yq.ldq; a.yq.s += r0; }
    if (a.ck.q) { a.ck.q += r0 * a.ck.ldq; a.ck.s += r0; }
    const dim3 grid(static_cast<unsigned>((a.cols + W * E - 1) / (W * E)), static_cast<unsigned>((rows + per - 1) / per));
    if (full) swiglu_rows<XT, W, R, true><<<grid, 256, 0, s>>>(a);
    else swiglu_rows<XT, W, R, false><<<grid, 256, 0, s>>>(a);
  });
}

template <int XT>
hipError_t dispatch_swiglu(const GateArgs& a, hipStream_t s) {
  switch (row_width(a.cols, kVec<XT>)) {
    case 256: return run_swiglu<XT, 256, 2>(a, s);
    case 64: return run_swiglu<XT, 64, 2>(a, s);
    default: return run_swiglu<XT, 32, 2>(a, s);
  }
}

template <int XT, bool CK, int W, int R>
hipError_t run_swiglu_back(const GateArgs& whole, hipStream_t s) {
  constexpr int E = kVec<XT>, per = 256 / W * R;
  const bool full = whole.cols % (W * E) == 0;
  return in_slices(whole.rows, grid_rows((whole.cols + W * E - 1) / (W * E)) * per, [&](int64_t r0, int64_t rows) {
    GateArgs a = whole;
    a.rows = rows;
    a.dy = elem<XT>(a.dy, r0 * a.lddy);
    a.y = elem<XT>(a.y, r0 * a.ldy);
    if (CK) { a.ck.q += r0 * a.ck.ldq; a.ck.s += r0; }
    else a.x = elem<XT>(a.x, r0 * a.ldx);
    const dim3 grid(static_cast<unsigned>((a.cols + W * E - 1) / (W * E)), static_cast<unsigned>((rows + per - 1) / per));
    if (full) swiglu_back_rows<XT, CK, W, R, true><<<grid, 256, 0, s>>>(a);
    else swiglu_back_rows<XT, CK, W, R, false><<<grid, 256, 0, s>>>(a);
  });
}

template <int XT, bool CK>
hipError_t dispatch_swiglu_back(const GateArgs& whole, hipStream_t s) {
  if (whole.dxq.q || whole.dxqt.q || whole.yqt.q) {
    return in_slices(whole.rows, grid_rows((whole.cols + kTileK - 1) / kTileK) * kTileK, [&](int64_t r0, int64_t rows) {
      GateArgs a = whole;
      a.rows = rows;
      a.dy = elem<XT>(a.dy, r0 * a.lddy);
      if (a.y) a.y = elem<XT>(a.y, r0 * a.ldy);
      if (CK) { a.ck.q += r0 * a.ck.ldq; a.ck.s += r0; }
      else a.x = elem<XT>(a.x, r0 * a.ldx);
      if (a.dxq.q) { a.dxq.q += r0 * a.dxq.ldq; a.dxq.s += r0; }
      if (a.dxqt.q) { a.dxqt.q += r0; a.dxqt.s += r0 / kTileK * a.dxqt.lds; }
      if (a.yqt.q) { a.yqt.q += r0; a.yqt.s += r0 / kTileK * a.yqt.lds; }
      const dim3 grid(static_cast<unsigned>((a.cols + kTileK - 1) / kTileK), static_cast<unsigned>((rows + kTileK - 1) / kTileK));
      if (a.y || a.dxq.q || a.dxqt.q) swiglu_back_region<XT, CK, true><<<grid, kRegThreads, 0, s>>>(a);
      else swiglu_back_region<XT, CK, false><<<grid, kRegThreads, 0, s>>>(a);
    });
  }
  switch (row_width(whole.cols, kVec<XT>)) {
    case 256: return run_swiglu_back<XT, CK, 256, 2>(whole, s);
    case 64: return run_swiglu_back<XT, CK, 64, 2>(whole, s);
    default: return run_swiglu_back<XT, CK, 32, 2>(whole, s);
  }
}

template <int XT>
hipError_t dispatch_swiglu_back_x(const GateArgs& a, hipStream_t s) {
  return a.ck.q ? dispatch_swiglu_back<XT, true>(a, s) : dispatch_swiglu_back<XT, false>(a, s);
}

}  // namespace

hipError_t launch_swiglu(const void* x, int xt, int64_t rows, int64_t cols, int64_t ldx, void* y, int yt, int64_t ldy,
                         const float* scale, float* amax, const amp_fp8_tiles& yq, const amp_fp8_tiles& ckpt, hipStream_t s) {
  GateArgs a{};
  a.x = x; a.ldx = ldx; a.y = y; a.yt = yt; a.ldy = ldy; a.scale = scale; a.amax = amax;
  a.yq = yq; a.ck = ckpt; a.rows = rows; a.cols = cols;
  switch (xt) {
    case AMP_F32: return dispatch_swiglu<AMP_F32>(a, s);
    case AMP_BF16: return dispatch_swiglu<AMP_BF16>(a, s);
    default: return dispatch_swiglu<AMP_F16>(a, s);
  }
}

hipError_t launch_swiglu_backward(const void* dy, int dt, int64_t rows, int64_t cols, int64_t lddy, const void* x, int64_t ldx,
                                  const amp_fp8_tiles& ckpt, void* dx, int64_t lddx, const amp_fp8_tiles& dxq,
                                  const amp_fp8_tiles& dxqt, const amp_fp8_tiles& yqt, hipStream_t s) {
  GateArgs a{};
  a.x = x; a.ldx = ldx; a.dy = dy; a.lddy = lddy; a.y = dx; a.ldy = lddx;
  a.ck = ckpt; a.dxq = dxq; a.dxqt = dxqt; a.yqt = yqt; a.rows = rows; a.cols = cols;
  switch (dt) {
    case AMP_F32: return dispatch_swiglu_back_x<AMP_F32>(a, s);
    case AMP_BF16: return dispatch_swiglu_back_x<AMP_BF16>(a, s);
    default: return dispatch_swiglu_back_x<AMP_F16>(a, s);
  }
}

}  // namespace amp
