// Device helpers shared by the fused block operators (norm, gated activation,
// requantization): 16-byte element vectors, FP8 encoding and decoding, and the
// 1x128-tile scaling of amp_quantize_blockwise.
//
// Rows need no alignment: gfx950 loads and stores dwords and wider at any
// byte address, so a row of odd length costs extra cache lines, not another
// code path.  Only a row's last, partial vector goes element by element.
#pragma once
#include "common.hpp"
#include "formats.hpp"

namespace amp {

constexpr int kTileK = 128;

typedef u32x4 u32x4_any __attribute__((aligned(1)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));
typedef uint32_t u32_any __attribute__((aligned(1)));

// Elements of a 16-byte vector of an input type; a 1x128 tile is 128 / kVec
// adjacent lanes.
template <int XT> constexpr int kVec = XT == AMP_F32 ? 4 : 8;

// One vector of row `p` from column c on; columns past `cols` read as zero.
template <int XT>
__device__ __forceinline__ u32x4 load_vec(const void* p, int64_t c, int64_t cols) {
  constexpr int E = kVec<XT>;
  u32x4 w = {0u, 0u, 0u, 0u};
  if constexpr (XT == AMP_F32) {
    const float* x = static_cast<const float*>(p) + c;
    if (c + E <= cols) return *reinterpret_cast<const u32x4_any*>(x);
#pragma unroll
    for (int k = 0; k < E; ++k)
      if (c + k < cols) w[k] = fbits(x[k]);
  } else {
    const uint16_t* x = static_cast<const uint16_t*>(p) + c;
    if (c + E <= cols) return *reinterpret_cast<const u32x4_any*>(x);
#pragma unroll
    for (int k = 0; k < E; ++k)
      if (c + k < cols) w[k / 2] |= static_cast<uint32_t>(x[k]) << (16 * (k & 1));
  }
  return w;
}

template <int XT>
__device__ __forceinline__ void widen(u32x4 w, float (&v)[kVec<XT>]) {
  if constexpr (XT == AMP_F32) {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = bitsf(w[k]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = XT == AMP_BF16 ? bitsf(w[k] << 16) : f16_to_f32(w[k] & 0xffffu);
      v[2 * k + 1] = XT == AMP_BF16 ? bitsf(w[k] & 0xffff0000u) : f16_to_f32(w[k] >> 16);
    }
  }
}

// Values rounded to XT and packed as load_vec returns them.
template <int XT>
__device__ __forceinline__ u32x4 narrow(const float (&v)[kVec<XT>]) {
  u32x4 w;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (XT == AMP_F32) w[k] = fbits(v[k]);
    else if constexpr (XT == AMP_BF16) w[k] = f32_to_bf16(v[2 * k]) | (f32_to_bf16(v[2 * k + 1]) << 16);
    else w[k] = f32_to_f16(v[2 * k]) | (f32_to_f16(v[2 * k + 1]) << 16);
  }
  return w;
}

template <int XT>
__device__ __forceinline__ void store_vec(void* p, int64_t c, int64_t cols, u32x4 w) {
  constexpr int E = kVec<XT>;
  if constexpr (XT == AMP_F32) {
    float* x = static_cast<float*>(p) + c;
    if (c + E <= cols) { *reinterpret_cast<u32x4_any*>(x) = w; return; }
#pragma unroll
    for (int k = 0; k < E; ++k)
      if (c + k < cols) x[k] = bitsf(w[k]);
  } else {
    uint16_t* x = static_cast<uint16_t*>(p) + c;
    if (c + E <= cols) { *reinterpret_cast<u32x4_any*>(x) = w; return; }
#pragma unroll
    for (int k = 0; k < E; ++k)
      if (c + k < cols) x[k] = static_cast<uint16_t>(w[k / 2] >> (16 * (k & 1)));
  }
}

// E per-column factors of type ct in {F32, F16, BF16} (p NULL: 1).
template <int E>
__device__ __forceinline__ void load_cols(const void* p, int ct, int64_t c, int64_t cols, float (&v)[E]) {
  if (p == nullptr) {
#pragma unroll
    for (int k = 0; k < E; ++k) v[k] = 1.0f;
  } else if (ct == AMP_F32) {
    const float* x = static_cast<const float*>(p) + c;
    if (c + E <= cols) {
#pragma unroll
      for (int q = 0; q < E / 4; ++q) {
        const u32x4 w = *reinterpret_cast<const u32x4_any*>(x + 4 * q);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[4 * q + k] = bitsf(w[k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < E; ++k) v[k] = c + k < cols ? x[k] : 0.0f;
    }
  } else {
    const uint16_t* x = static_cast<const uint16_t*>(p) + c;
    uint32_t h[E / 2];
    if (c + E <= cols) {
#pragma unroll
      for (int q = 0; q < E / 4; ++q) {
        const u32x2 w = *reinterpret_cast<const u32x2_any*>(x + 4 * q);
        h[2 * q] = w.x;
        h[2 * q + 1] = w.y;
      }
    } else {
#pragma unroll
      for (int q = 0; q < E / 2; ++q) {
        h[q] = c + 2 * q < cols ? x[2 * q] : 0u;
        if (c + 2 * q + 1 < cols) h[q] |= static_cast<uint32_t>(x[2 * q + 1]) << 16;
      }
    }
    if (ct == AMP_BF16) {
#pragma unroll
      for (int q = 0; q < E / 2; ++q) { v[2 * q] = bitsf(h[q] << 16); v[2 * q + 1] = bitsf(h[q] & 0xffff0000u); }
    } else {
#pragma unroll
      for (int q = 0; q < E / 2; ++q) { v[2 * q] = f16_to_f32(h[q] & 0xffffu); v[2 * q + 1] = f16_to_f32(h[q] >> 16); }
    }
  }
}

// ---- FP8 ------------------------------------------------------------------

__device__ __forceinline__ float fp8_max(int yt) { return yt == AMP_E4M3 ? 448.0f : 57344.0f; }

// max(m, |v[0..E)|), NaN above everything (two elements an instruction).
template <int E>
__device__ __forceinline__ float abs_max(float m, const float (&v)[E]) {
#pragma unroll
  for (int k = 0; k < E; k += 2)
    m = __builtin_elementwise_maximum(__builtin_elementwise_maximum(m, fabsf(v[k])), fabsf(v[k + 1]));
  return m;
}

// Bits of an abs_max result without a NaN's sign: their unsigned order is the
// order of the values, NaN above infinity.
__device__ __forceinline__ uint32_t mag(float m) { return fbits(m) & 0x7fffffffu; }

// Codes of E scaled values, four to a word, as f32_to_e4m3 / f32_to_e5m2
// would round each: `special` says that one of them may be NaN.  Without one
// the clamp and half a conversion instruction per element are all there is.
template <int E>
__device__ __forceinline__ void encode(int yt, const float (&t)[E], bool special, uint32_t (&w)[E / 4]) {
  if (special) {
#pragma unroll
    for (int q = 0; q < E / 4; ++q) {
      w[q] = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[q] |= (yt == AMP_E4M3 ? f32_to_e4m3(t[4 * q + k]) : f32_to_e5m2(t[4 * q + k])) << (8 * k);
    }
    return;
  }
  const float m = fp8_max(yt);
#pragma unroll
  for (int q = 0; q < E / 4; ++q) {
    float y[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = __builtin_amdgcn_fmed3f(t[4 * q + k], -m, m);
    if (yt == AMP_E4M3) {
      const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
      w[q] = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], lo, true));
    } else {
      const int lo = __builtin_amdgcn_cvt_pk_bf8_f32(y[0], y[1], 0, false);
      w[q] = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_bf8_f32(y[2], y[3], lo, true));
    }
  }
}

template <int E>
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t c, int64_t cols, const uint32_t (&w)[E / 4]) {
  if (c + E <= cols) {
    if constexpr (E == 8) {
      u32x2 d = {w[0], w[1]};
      *reinterpret_cast<u32x2_any*>(p + c) = d;
    } else {
      *reinterpret_cast<u32_any*>(p + c) = w[0];
    }
  } else {
#pragma unroll
    for (int k = 0; k < E; ++k)
      if (c + k < cols) p[c + k] = static_cast<uint8_t>(w[k / 4] >> (8 * (k & 3)));
  }
}

// Values of E codes from column c on; columns past `cols` read as zero.
template <int E>
__device__ __forceinline__ void load_codes(const uint8_t* p, int64_t c, int64_t cols, uint32_t (&w)[E / 4]) {
  if (c + E <= cols) {
    if constexpr (E == 8) {
      const u32x2 d = *reinterpret_cast<const u32x2_any*>(p + c);
      w[0] = d.x;
      w[1] = d.y;
    } else {
      w[0] = *reinterpret_cast<const u32_any*>(p + c);
    }
  } else {
#pragma unroll
    for (int q = 0; q < E / 4; ++q) w[q] = 0;
#pragma unroll
    for (int k = 0; k < E; ++k)
      if (c + k < cols) w[k / 4] |= static_cast<uint32_t>(p[c + k]) << (8 * (k & 3));
  }
}

template <int E>
__device__ __forceinline__ void decode(int xt, const uint32_t (&w)[E / 4], float mul, float (&v)[E]) {
#pragma unroll
  for (int q = 0; q < E / 4; ++q) {
    const int wq = static_cast<int>(w[q]);
    if (xt == AMP_E4M3) {
      const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(wq, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(wq, true);
      v[4 * q] = lo[0] * mul; v[4 * q + 1] = lo[1] * mul; v[4 * q + 2] = hi[0] * mul; v[4 * q + 3] = hi[1] * mul;
    } else {
      const auto lo = __builtin_amdgcn_cvt_pk_f32_bf8(wq, false), hi = __builtin_amdgcn_cvt_pk_f32_bf8(wq, true);
      v[4 * q] = lo[0] * mul; v[4 * q + 1] = lo[1] * mul; v[4 * q + 2] = hi[0] * mul; v[4 * q + 3] = hi[1] * mul;
    }
  }
}

// Scale of a tile from its amax bits: fp8_max / amax, or 1 where that is not
// a positive finite number (an amax of 0, inf or NaN, or one so small that
// the quotient overflows).
__device__ __forceinline__ float scale_of(uint32_t amax, float fmax) {
  const float sc = fmax / bitsf(amax);
  return fbits(sc) - 1u < 0x7f7fffffu ? sc : 1.0f;
}

// Unsigned maximum over groups of G = 16 or 32 adjacent lanes (all active).
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  uint32_t o;
#define AMP_ROR(ctl)                                                                                           \
  o = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), ctl, 0xf, 0xf, false));        \
  v = v > o ? v : o;
  AMP_ROR(0x128) AMP_ROR(0x124) AMP_ROR(0x122) AMP_ROR(0x121)   // rotations by 8, 4, 2, 1 in a row of 16
#undef AMP_ROR
  if constexpr (G == 32) {
    o = static_cast<uint32_t>(__builtin_amdgcn_ds_swizzle(static_cast<int>(v), 0x401f));   // lane ^ 16
    v = v > o ? v : o;
  }
  return v;
}

// Quantize one vector of a row in 1x128 tiles: the 128 / E lanes of a tile
// call together (lanes past `cols` hold zeros), `blk` is the tile's index
// along K in the scale array.
template <int E>
__device__ __forceinline__ void store_tile(const amp_fp8_tiles& o, int64_t row, int64_t c, int64_t c_end, int64_t blk,
                                           bool live, const float (&v)[E]) {
  const uint32_t am = group_max<kTileK / E>(mag(abs_max<E>(0.0f, v)));
  const float sc = scale_of(am, fp8_max(o.type));
  float t[E];
#pragma unroll
  for (int k = 0; k < E; ++k) t[k] = v[k] * sc;
  uint32_t w[E / 4];
  encode<E>(o.type, t, am >= 0x7f800000u, w);
  if (live) {
    store_codes<E>(o.q + row * o.ldq, c, c_end, w);
    if (threadIdx.x % (kTileK / E) == 0 && c < c_end) o.s[blk * o.lds + row] = 1.0f / sc;
  }
}

// One vector of a plain output: 16 bits, or FP8 of the values times `scale`.
template <int E>
__device__ __forceinline__ void store_plain(void* y, int yt, int64_t at, int64_t c, int64_t cols, float scale, float am,
                                            const float (&v)[E]) {
  if (yt == AMP_E4M3 || yt == AMP_E5M2) {
    float t[E];
#pragma unroll
    for (int k = 0; k < E; ++k) t[k] = v[k] * scale;
    uint32_t w[E / 4];
    // inf * 0-like scales aside, a product is NaN only for a NaN or infinite factor
    encode<E>(yt, t, mag(am) >= 0x7f800000u || mag(scale) >= 0x7f800000u, w);
    store_codes<E>(static_cast<uint8_t*>(y) + at, c, cols, w);
    return;
  }
  uint32_t h[E / 2];
#pragma unroll
  for (int q = 0; q < E / 2; ++q) {
    const float a = v[2 * q] * scale, b = v[2 * q + 1] * scale;
    h[q] = yt == AMP_BF16 ? f32_to_bf16(a) | (f32_to_bf16(b) << 16) : f32_to_f16(a) | (f32_to_f16(b) << 16);
  }
  uint16_t* p = static_cast<uint16_t*>(y) + at + c;
  if (c + E <= cols) {
    if constexpr (E == 8) {
      const u32x4 w = {h[0], h[1], h[2], h[3]};
      *reinterpret_cast<u32x4_any*>(p) = w;
    } else {
      const u32x2 w = {h[0], h[1]};
      *reinterpret_cast<u32x2_any*>(p) = w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < E; ++k)
      if (c + k < cols) p[k] = static_cast<uint16_t>(h[k / 2] >> (16 * (k & 1)));
  }
}

// ---- 128x128 regions written transposed -------------------------------------
// 512 threads hold a region of a [rows, cols] tensor: thread t the 8 rows
// 8 (t / 32) .. + 7 of the 4 columns 4 (t % 32) .. + 3, so that a row's 128
// columns are 32 adjacent lanes and a thread's transposed codes are whole
// 8-byte units.
constexpr int kRegThreads = 512;
constexpr int kRegRows = 8, kRegCols = 4;

// Where the 8-byte unit `u` (rows 8u .. 8u+7) of column c lies among the 128
// transposed rows of 128 bytes: the exclusive-ors spread one column of a
// wave's 32 column groups over all 64 banks, and keep 16-byte pairs and whole
// rows together for the reads.
__device__ __forceinline__ int reg_at(int c, int u) {
  return (c ^ ((c >> 5) & 1)) * kTileK + 8 * (u ^ (2 * ((c >> 2) & 7)));
}

template <int N>
struct RegLds {
  union {
    uint32_t part[N][16][kTileK];                        // column maxima of the 16 thread rows
    __align__(16) uint8_t codes[N][kTileK * kTileK];     // transposed codes
  };
  float scale[N][kTileK];
};

// Write N regions v[n] transposed: o[n] is the [cols, rows] output whose row
// col0[n] + j is the region's column j (o[n].q NULL: none).  `rows` and
// `ncols` bound the region.  Three block barriers.
template <int N>
__device__ __forceinline__ void store_regions_t(RegLds<N>& l, const amp_fp8_tiles (&o)[N], const int64_t (&col0)[N],
                                                int64_t row0, int64_t rows, int ncols,
                                                const float (&v)[N][kRegRows][kRegCols]) {
  const int t = threadIdx.x, cg = t % 32, rg = t / 32;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    u32x4 m;
#pragma unroll
    for (int j = 0; j < kRegCols; ++j) {
      float a = 0.0f;
#pragma unroll
      for (int i = 0; i < kRegRows; i += 2)
        a = __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, fabsf(v[n][i][j])), fabsf(v[n][i + 1][j]));
      m[j] = mag(a);
    }
    *reinterpret_cast<u32x4*>(&l.part[n][rg][4 * cg]) = m;
  }
  __syncthreads();
  if (t < N * kTileK) {
    const int n = t / kTileK, c = t % kTileK;
    uint32_t m = 0;
#pragma unroll
    for (int g = 0; g < 16; ++g) m = m > l.part[n][g][c] ? m : l.part[n][g][c];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if (k != n) continue;
      const float sc = scale_of(m, fp8_max(o[k].type));
      // the sign carries whether the tile holds a NaN or infinity
      l.scale[k][c] = m >= 0x7f800000u ? -sc : sc;
      if (o[k].q && c < ncols) o[k].s[row0 / kTileK * o[k].lds + col0[k] + c] = 1.0f / sc;
    }
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) {
    if (!o[n].q) continue;
    const f32x4 sc = *reinterpret_cast<const f32x4*>(&l.scale[n][4 * cg]);
#pragma unroll
    for (int j = 0; j < kRegCols; ++j) {
      float f[kRegRows];
#pragma unroll
      for (int i = 0; i < kRegRows; ++i) f[i] = v[n][i][j] * fabsf(sc[j]);
      uint32_t w[2];
      encode<kRegRows>(o[n].type, f, sc[j] < 0.0f, w);
      const u32x2 d = {w[0], w[1]};
      *reinterpret_cast<u32x2*>(&l.codes[n][reg_at(4 * cg + j, rg)]) = d;
    }
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) {
    if (!o[n].q) continue;
#pragma unroll
    for (int it = 0; it < 2; ++it) {
      const int c = it * 64 + t / 8, b = t % 8 * 16;
      if (c >= ncols) continue;
      const u32x4 w = *reinterpret_cast<const u32x4*>(&l.codes[n][reg_at(c, b / 8)]);
      uint8_t* p = o[n].q + (col0[n] + c) * o[n].ldq + row0 + b;
      if (row0 + b + 16 <= rows) {
        *reinterpret_cast<u32x4_any*>(p) = w;
      } else {
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (row0 + b + k < rows) p[k] = static_cast<uint8_t>(w[k / 4] >> (8 * (k & 3)));
      }
    }
  }
}

}  // namespace amp
