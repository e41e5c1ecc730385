// Device helpers shared by the fused block operators (norm, gated activation,
// requantization): 16-byte element vectors, FP8 encoding and decoding, and the
// 1x128-tile scaling of amp_quantize_blockwise.
//
// Rows need no alignment: gfx950 loads and stores dwords and wider at any
// byte address, so a row of odd length costs extra cache lines, not another
// code path.  A row's last, partial vector is loaded as the whole vector that
// ends with the row and stored element by element.
//
// The operators are HBM-bound only as long as the vector ALUs keep up (about
// 50 operations per element at one 16-bit stream's rate), so addresses are a
// wave-uniform row pointer plus a 32-bit offset, and a tile's two divisions
// are shared out over the lanes of a quad.
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
template <int XT> constexpr int kBytes = XT == AMP_F32 ? 4 : 2;

// p advanced by i elements of type XT.
template <int XT>
__host__ __device__ __forceinline__ const void* elem(const void* p, int64_t i) { return static_cast<const uint8_t*>(p) + i * kBytes<XT>; }
template <int XT>
__host__ __device__ __forceinline__ void* elem(void* p, int64_t i) { return static_cast<uint8_t*>(p) + i * kBytes<XT>; }
// p advanced by i elements of the run-time type t.
__device__ __forceinline__ const void* elem_of(int t, const void* p, int64_t i) {
  return static_cast<const uint8_t*>(p) + i * (t == AMP_F32 ? 4 : 2);
}

// Row blocks of a grid with x blocks along the columns: within the bound of
// the y dimension and with the grid's threads (512 a block at most) countable
// in 32 bits.
inline int64_t grid_rows(int64_t x) {
  const int64_t y = (1 << 22) / x;
  return y < 1 ? 1 : y > 65535 ? 65535 : y;
}

// The number of columns left, as the 32-bit bound that the helpers take (they
// see at most one chunk of a row).
__device__ __forceinline__ int left(int64_t n) { return n > (1 << 24) ? 1 << 24 : static_cast<int>(n); }

// Loads and stores of 16, 8 and 4 bytes at p + off, of any alignment (the
// under-aligned types are named in the casts: as template arguments they
// would lose the attribute).
__device__ __forceinline__ const uint8_t* at(const void* p, uint32_t off) { return static_cast<const uint8_t*>(p) + off; }
__device__ __forceinline__ uint8_t* at(void* p, uint32_t off) { return static_cast<uint8_t*>(p) + off; }
__device__ __forceinline__ u32x4 ld16(const void* p, uint32_t off) { return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(at(p, off))); }
__device__ __forceinline__ u32x2 ld8(const void* p, uint32_t off) { return __builtin_nontemporal_load(reinterpret_cast<const u32x2_any*>(at(p, off))); }
__device__ __forceinline__ uint32_t ld4(const void* p, uint32_t off) { return __builtin_nontemporal_load(reinterpret_cast<const u32_any*>(at(p, off))); }
__device__ __forceinline__ void st16(void* p, uint32_t off, u32x4 v) { __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any*>(at(p, off))); }
__device__ __forceinline__ void st8(void* p, uint32_t off, u32x2 v) { __builtin_nontemporal_store(v, reinterpret_cast<u32x2_any*>(at(p, off))); }
__device__ __forceinline__ void st4(void* p, uint32_t off, uint32_t v) { __builtin_nontemporal_store(v, reinterpret_cast<u32_any*>(at(p, off))); }

// The 16 bytes of w moved down by `bytes` (1..15), zeros moved in.
__device__ __forceinline__ u32x4 drop_low(u32x4 w, int bytes) {
  if (bytes & 8) w = u32x4{w[2], w[3], 0u, 0u};
  if (bytes & 4) w = u32x4{w[1], w[2], w[3], 0u};
  const int s = 8 * (bytes & 3);
  return u32x4{__builtin_amdgcn_alignbit(w[1], w[0], s), __builtin_amdgcn_alignbit(w[2], w[1], s),
               __builtin_amdgcn_alignbit(w[3], w[2], s), w[3] >> s};
}

// One vector at column c of the n columns at p, to be passed through trim_vec
// before use: near the row's end it is the row's last whole vector, and what
// the lane does not hold is dropped later, so that no load waits for another.
// FULL: the caller knows that the vector lies within the row (each bound that
// is checked is a branch, and a row has dozens of vectors).  Non-temporal:
// these tensors are read once.
template <int XT, bool FULL = false>
__device__ __forceinline__ u32x4 load_vec(const void* p, int c, int n) {
  constexpr int E = kVec<XT>;
  if constexpr (FULL) return ld16(p, static_cast<uint32_t>(c) * kBytes<XT>);
  if (n >= E) return ld16(p, static_cast<uint32_t>(c < n - E ? c : n - E) * kBytes<XT>);
  u32x4 w = {0u, 0u, 0u, 0u};   // a row shorter than one vector
#pragma unroll
  for (int k = 0; k < E; ++k)
    if (c + k < n) {
      if constexpr (XT == AMP_F32) w[k] = static_cast<const uint32_t*>(p)[c + k];
      else w[k / 2] |= static_cast<uint32_t>(static_cast<const uint16_t*>(p)[c + k]) << (16 * (k & 1));
    }
  return w;
}

// What load_vec's vector holds of the row from column c on, zeros past its end.
template <int XT, bool FULL = false>
__device__ __forceinline__ u32x4 trim_vec(u32x4 w, int c, int n) {
  constexpr int E = kVec<XT>;
  if (FULL || n < E || c + E <= n) return w;
  return c < n ? drop_low(w, (c + E - n) * kBytes<XT>) : u32x4{0u, 0u, 0u, 0u};
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

// Two values rounded to 16 bits, nearest even (a NaN stays one; its payload
// is the hardware's).
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack16(bool bf16, float a, float b) {
  const f32x2 v = {a, b};
  return bf16 ? __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2))
              : __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
}

// Values rounded to XT and packed as load_vec returns them.
template <int XT>
__device__ __forceinline__ u32x4 narrow(const float (&v)[kVec<XT>]) {
  u32x4 w;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (XT == AMP_F32) w[k] = fbits(v[k]);
    else w[k] = pack16(XT == AMP_BF16, v[2 * k], v[2 * k + 1]);
  }
  return w;
}

// W 32-bit words holding 2 W 16-bit elements, to column c of the n at p.
template <int W, bool FULL = false>
__device__ __forceinline__ void store16(void* p, int c, int n, const uint32_t (&h)[W]) {
  if (FULL || c + 2 * W <= n) {
    if constexpr (W == 4) st16(p, 2u * c, u32x4{h[0], h[1], h[2], h[3]});
    else st8(p, 2u * c, u32x2{h[0], h[1]});
  } else {
#pragma unroll
    for (int k = 0; k < 2 * W; ++k)
      if (c + k < n) static_cast<uint16_t*>(p)[c + k] = static_cast<uint16_t>(h[k / 2] >> (16 * (k & 1)));
  }
}

template <int XT, bool FULL = false>
__device__ __forceinline__ void store_vec(void* p, int c, int n, u32x4 w) {
  if constexpr (XT == AMP_F32) {
    if (FULL || c + 4 <= n) {
      st16(p, 4u * c, w);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (c + k < n) static_cast<float*>(p)[c + k] = bitsf(w[k]);
    }
  } else {
    const uint32_t h[4] = {w[0], w[1], w[2], w[3]};
    store16<4, FULL>(p, c, n, h);
  }
}

// E per-column factors of type ct in {F32, F16, BF16} (p NULL: 1), read by
// every row and so through the caches.
template <int E, bool FULL = false>
__device__ __forceinline__ void load_cols(const void* p, int ct, int c, int n, float (&v)[E]) {
  if (p == nullptr) {
#pragma unroll
    for (int k = 0; k < E; ++k) v[k] = 1.0f;
  } else if (ct == AMP_F32) {
    const float* x = static_cast<const float*>(p);
    if (FULL || c + E <= n) {
#pragma unroll
      for (int q = 0; q < E / 4; ++q) {
        const u32x4 w = *reinterpret_cast<const u32x4_any*>(x + static_cast<uint32_t>(c + 4 * q));
#pragma unroll
        for (int k = 0; k < 4; ++k) v[4 * q + k] = bitsf(w[k]);
      }
    } else {
      // element loads with the index held inside the row: no branch, no wait between them
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const float t = x[c + k < n ? c + k : n - 1];
        v[k] = c + k < n ? t : 0.0f;
      }
    }
  } else {
    const uint16_t* x = static_cast<const uint16_t*>(p);
    uint32_t h[E / 2];
    if (FULL || c + E <= n) {
      if constexpr (E == 8) {
        const u32x4 w = *reinterpret_cast<const u32x4_any*>(x + static_cast<uint32_t>(c));
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = w[k];
      } else {
        const u32x2 w = *reinterpret_cast<const u32x2_any*>(x + static_cast<uint32_t>(c));
        h[0] = w.x;
        h[1] = w.y;
      }
    } else {
#pragma unroll
      for (int q = 0; q < E / 2; ++q) {
        const uint32_t lo = x[c + 2 * q < n ? c + 2 * q : n - 1], hi = x[c + 2 * q + 1 < n ? c + 2 * q + 1 : n - 1];
        h[q] = (c + 2 * q < n ? lo : 0u) | (c + 2 * q + 1 < n ? hi << 16 : 0u);
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
constexpr uint32_t kInfBits = 0x7f800000u;

// Codes of the N x E values val(n, k), four to a word.
template <int YT, int N, int E, typename F>
__device__ __forceinline__ void convert(uint32_t (&w)[N][E / 4], F val) {
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int q = 0; q < E; q += 4) {
      if constexpr (YT == AMP_E4M3) {
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(val(n, q), val(n, q + 1), 0, false);
        w[n][q / 4] = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(val(n, q + 2), val(n, q + 3), lo, true));
      } else {
        const int lo = __builtin_amdgcn_cvt_pk_bf8_f32(val(n, q), val(n, q + 1), 0, false);
        w[n][q / 4] = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_bf8_f32(val(n, q + 2), val(n, q + 3), lo, true));
      }
    }
}

// Four codes with every NaN, whatever its sign and payload, as 0x7F: the
// magnitudes above the format's largest (and, in E5M2, above infinity's 0x7C)
// carry into the sign's place when the distance to 0x80 is added.
template <int YT>
__device__ __forceinline__ uint32_t canon_nan(uint32_t w) {
  const uint32_t nan = ((w & 0x7f7f7f7fu) + (YT == AMP_E4M3 ? 0x01010101u : 0x03030303u)) & 0x80808080u;
  return (w & ~nan) | (nan - (nan >> 7));
}

// The codes that f32_to_e4m3 / f32_to_e5m2 give.  `special`, for any lane of
// the wave, says that one of the lane's values may be NaN or infinite (codes
// 0x7F and +-max); without one a value costs half a conversion instruction.
// CLAMP: values may lie beyond the format's range; those scaled by their own
// tile's amax do not: they reach at most fp8_max (1 + 2^-22), which the
// conversion rounds to fp8_max (measured).  val is evaluated on the path that
// is taken, so that the values need no registers of their own.
template <int N, int E, bool CLAMP, typename F>
__device__ __forceinline__ void encode(int yt, bool special, uint32_t (&w)[N][E / 4], F val) {
  const float m = fp8_max(yt);
  if (__builtin_amdgcn_ballot_w64(special)) {
    // clamped with NaN kept
    auto y = [&](int n, int k) __attribute__((always_inline)) {
      return __builtin_elementwise_minimum(__builtin_elementwise_maximum(val(n, k), -m), m);
    };
    if (yt == AMP_E4M3) convert<AMP_E4M3, N, E>(w, y);
    else convert<AMP_E5M2, N, E>(w, y);
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int q = 0; q < E / 4; ++q) w[n][q] = yt == AMP_E4M3 ? canon_nan<AMP_E4M3>(w[n][q]) : canon_nan<AMP_E5M2>(w[n][q]);
    return;
  }
  auto y = [&](int n, int k) __attribute__((always_inline)) {
    return CLAMP ? __builtin_amdgcn_fmed3f(val(n, k), -m, m) : val(n, k);
  };
  if (yt == AMP_E4M3) convert<AMP_E4M3, N, E>(w, y);
  else convert<AMP_E5M2, N, E>(w, y);
}

// E codes to column c of the n at p.
template <int E, bool FULL = false>
__device__ __forceinline__ void store_codes(uint8_t* p, int c, int n, const uint32_t (&w)[E / 4]) {
  if (FULL || c + E <= n) {
    if constexpr (E == 8) st8(p, c, u32x2{w[0], w[1]});
    else st4(p, c, w[0]);
  } else {
#pragma unroll
    for (int k = 0; k < E; ++k)
      if (c + k < n) p[c + k] = static_cast<uint8_t>(w[k / 4] >> (8 * (k & 3)));
  }
}

// E codes at column c of the n at p, and what they hold of the row: as
// load_vec and trim_vec.
template <int E, bool FULL = false>
__device__ __forceinline__ void load_codes(const uint8_t* p, int c, int n, uint32_t (&w)[E / 4]) {
  const int e = FULL || c <= n - E ? c : n - E;
  if (FULL || n >= E) {
    if constexpr (E == 8) {
      const u32x2 d = ld8(p, e);
      w[0] = d.x;
      w[1] = d.y;
    } else {
      w[0] = ld4(p, e);
    }
    return;
  }
#pragma unroll
  for (int q = 0; q < E / 4; ++q) w[q] = 0;
#pragma unroll
  for (int k = 0; k < E; ++k)   // a row shorter than E
    if (c + k < n) w[k / 4] |= static_cast<uint32_t>(p[c + k]) << (8 * (k & 3));
}

template <int E, bool FULL = false>
__device__ __forceinline__ void trim_codes(uint32_t (&w)[E / 4], int c, int n) {
  if (FULL || n < E || c + E <= n) return;
  const int s = 8 * (c + E - n);
  if constexpr (E == 8) {
    const uint64_t v = c < n ? ((static_cast<uint64_t>(w[1]) << 32) | w[0]) >> s : 0u;
    w[0] = static_cast<uint32_t>(v);
    w[1] = static_cast<uint32_t>(v >> 32);
  } else {
    w[0] = c < n ? w[0] >> s : 0u;
  }
}

// Values of E codes times `mul`.
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

// Value of lane K of the quad in all its lanes.
template <int K>
__device__ __forceinline__ float quad(float v) {
  return bitsf(static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(fbits(v)), K * 0x55, 0xf, 0xf, true)));
}

// Scales of N <= 4 tiles whose maxima am[] every lane of the tiles' lane group
// holds: lane k of each quad divides for tile k (two divisions for up to four
// tiles, in place of two each).  Returns 1 / scale of tile lane % 4.
template <int N>
__device__ __forceinline__ float tile_scales(const uint32_t (&am)[N], float fmax, float (&sc)[N]) {
  const int k = threadIdx.x & 3;
  uint32_t m = am[0];
  if constexpr (N > 1) m = k == 1 ? am[1] : m;
  if constexpr (N > 2) m = k == 2 ? am[2] : m;
  if constexpr (N > 3) m = k == 3 ? am[3] : m;
  const float s = scale_of(m, fmax);
  sc[0] = N > 1 ? quad<0>(s) : s;
  if constexpr (N > 1) sc[1] = quad<1>(s);
  if constexpr (N > 2) sc[2] = quad<2>(s);
  if constexpr (N > 3) sc[3] = quad<3>(s);
  return 1.0f / s;
}

// N vectors, `step` columns apart, of a plain output at p (its row): 16 bits,
// or FP8, of the values times `scale`; `am` is their abs_max before.  A
// product is NaN or infinite only with such a factor or by overflow, which the
// FP8 clamp and the 16-bit rounding handle without the special path.
template <int N, int E, bool FULL = false>
__device__ __forceinline__ void store_plain(void* p, int yt, int c, int step, int n, bool live, float scale, float am,
                                            const float (&v)[N][E]) {
  const bool special = mag(am) >= kInfBits || mag(scale) >= kInfBits;
  auto t = [&](int k, int e) __attribute__((always_inline)) { return v[k][e] * scale; };
  if (yt == AMP_E4M3 || yt == AMP_E5M2) {
    uint32_t w[N][E / 4];
    encode<N, E, true>(yt, special, w, t);
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (live) store_codes<E, FULL>(static_cast<uint8_t*>(p), c + k * step, n, w[k]);
    return;
  }
  uint32_t h[N][E / 2];
  if (__builtin_amdgcn_ballot_w64(special)) {
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int q = 0; q < E / 2; ++q)
        h[k][q] = yt == AMP_BF16 ? f32_to_bf16(t(k, 2 * q)) | (f32_to_bf16(t(k, 2 * q + 1)) << 16)
                                 : f32_to_f16(t(k, 2 * q)) | (f32_to_f16(t(k, 2 * q + 1)) << 16);
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int q = 0; q < E / 2; ++q) h[k][q] = pack16(yt == AMP_BF16, t(k, 2 * q), t(k, 2 * q + 1));
  }
#pragma unroll
  for (int k = 0; k < N; ++k)
    if (live) store16<E / 2, FULL>(p, c + k * step, n, h[k]);
}

// ---- amax of an output ------------------------------------------------------

// A value that *d_amax holds or exceeds from now on, read ahead of the work
// so that its latency is hidden (0 without d_amax).
__device__ __forceinline__ uint32_t amax_seen(const float* d_amax) {
  return d_amax ? __hip_atomic_load(reinterpret_cast<const uint32_t*>(d_amax), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP) : 0u;
}

// Maximum over a block of at most 16 waves into *d_amax; blocks that do not
// exceed what they saw at their start leave without touching it.
__device__ __forceinline__ void block_amax(float am, uint32_t seen, uint32_t* red, float* d_amax) {
  uint32_t m = mag(am);
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    const uint32_t o = static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), off, kWave));
    m = m > o ? m : o;
  }
  if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int k = 1; k < static_cast<int>(blockDim.x) / kWave; ++k) m = m > red[k] ? m : red[k];
    if (canon_amax(m) > seen) amax_update(d_amax, m);
  }
}

// ---- 128x128 regions written transposed -------------------------------------
// 512 threads hold a region of a [rows, cols] tensor: thread t the 4 rows
// 4 (t / 16) .. + 3 of the 8 columns 8 (t % 16) .. + 7, so that a row's 128
// columns are 16 adjacent lanes and a thread's transposed codes whole words.
// The pieces of 128 bytes that a region writes to each row are stored through
// the caches (non-temporal: 2 % slower).
constexpr int kRegThreads = 512;
constexpr int kRegRows = 4, kRegCols = 8;

// The region's place: its first row and column, and what the tensor has of
// it.  SPANS: each of the 8 XCDs (block b runs on b % 8) takes one contiguous
// span of the regions, row by row.
struct Region {
  int64_t r0, c0;
  int nrows, ncols;
  __device__ __forceinline__ Region(int64_t rows, int64_t cols, bool spans) {
    uint32_t k = blockIdx.y * gridDim.x + blockIdx.x;
    if (spans) {
      const uint32_t n = gridDim.x * gridDim.y, x = k % 8;
      k = x * (n / 8) + (x < n % 8 ? x : n % 8) + k / 8;
    }
    r0 = static_cast<int64_t>(k / gridDim.x) * kTileK;
    c0 = static_cast<int64_t>(k % gridDim.x) * kTileK;
    nrows = left(rows - r0) < kTileK ? left(rows - r0) : kTileK;
    ncols = left(cols - c0) < kTileK ? left(cols - c0) : kTileK;
  }
  __device__ __forceinline__ bool whole() const { return nrows == kTileK && ncols == kTileK; }
  // this thread's first row and column in the region
  __device__ __forceinline__ int r() const { return threadIdx.x / 16 * kRegRows; }
  __device__ __forceinline__ int c() const { return threadIdx.x % 16 * kRegCols; }
  // the tensor's row that stands for this thread's row i (the last one past the end)
  __device__ __forceinline__ int64_t row(int i) const { return r0 + (r() + i < nrows ? r() + i : nrows - 1); }
};

// This thread's elements of a region of 32-, 16- or 8-bit elements, a row at a
// time as D dwords.  The loads carry no branch and no dependence (a lane past
// the edge reads the nearest place inside), so that all are in flight
// together; trim() then drops what the lane does not hold.
template <int BYTES>
struct RegRaw {
  static constexpr int D = kRegCols * BYTES / 4;
  uint32_t w[kRegRows][D];

  // row i, its columns at p (the row's element c0)
  __device__ __forceinline__ void load(const Region& g, int i, const void* p) {
    if (g.ncols < kRegCols) {
#pragma unroll
      for (int d = 0; d < D; ++d) w[i][d] = 0;
#pragma unroll
      for (int k = 0; k < kRegCols; ++k) {
        const int e = k < g.ncols ? k : g.ncols - 1;
        const uint32_t v = BYTES == 4 ? static_cast<const uint32_t*>(p)[e] : BYTES == 2 ? static_cast<const uint16_t*>(p)[e]
                                                                                       : static_cast<const uint8_t*>(p)[e];
        w[i][k * BYTES / 4] |= k < g.ncols ? v << (8 * (k * BYTES % 4)) : 0u;
      }
      return;
    }
    const uint32_t e = static_cast<uint32_t>(g.c() < g.ncols - kRegCols ? g.c() : g.ncols - kRegCols) * BYTES;
    if constexpr (D == 2) {
      const u32x2 v = ld8(p, e);
      w[i][0] = v.x;
      w[i][1] = v.y;
    } else {
#pragma unroll
      for (int q = 0; q < D / 4; ++q) {
        const u32x4 v = ld16(p, e + 16 * q);
#pragma unroll
        for (int k = 0; k < 4; ++k) w[i][4 * q + k] = v[k];
      }
    }
  }

  // zeros past the region's edges
  __device__ __forceinline__ void trim(const Region& g) {
    if (g.whole()) return;
    const int drop = g.ncols < kRegCols ? (g.c() ? kRegCols : 0) : g.c() - (g.ncols - kRegCols);
#pragma unroll
    for (int i = 0; i < kRegRows; ++i) {
      const bool in = g.r() + i < g.nrows && drop < kRegCols;
      uint32_t v[D];
#pragma unroll
      for (int d = 0; d < D; ++d) v[d] = in ? w[i][d] : 0u;
      if (drop > 0) {
        // a shift down by drop * BYTES bytes, one power of two at a time
#pragma unroll
        for (int b = 4; b >= 1; b /= 2) {
          const int by = b * BYTES;
          if ((drop & b) == 0) continue;
#pragma unroll
          for (int d = 0; d < D; ++d) {
            if (by >= 4) v[d] = d + by / 4 < D ? v[d + by / 4] : 0u;
            else v[d] = __builtin_amdgcn_alignbit(d + 1 < D ? v[d + 1] : 0u, v[d], 8 * by);
          }
        }
      }
#pragma unroll
      for (int d = 0; d < D; ++d) w[i][d] = v[d];
    }
  }
};

template <int XT>
__device__ __forceinline__ void reg_values(const uint32_t (&w)[kRegCols * kBytes<XT> / 4], float (&v)[kRegCols]) {
#pragma unroll
  for (int k = 0; k < kRegCols; ++k) {
    if constexpr (XT == AMP_F32) v[k] = bitsf(w[k]);
    else if constexpr (XT == AMP_BF16) v[k] = bitsf(k & 1 ? w[k / 2] & 0xffff0000u : w[k / 2] << 16);
    else v[k] = f16_to_f32(k & 1 ? w[k / 2] >> 16 : w[k / 2] & 0xffffu);
  }
}

// Where the 4 transposed codes of rows 4u .. 4u+3 of column c lie: 128 rows
// of 128 bytes, one per column, the exclusive-ors spread one column of a
// wave's 16 column groups by 4 row groups over all 64 banks and keep 16-byte
// pieces and whole rows together for the reads.
__device__ __forceinline__ int reg_at(int c, int u) {
  return (c ^ ((c >> 6) & 1)) * kTileK + 4 * (u ^ (4 * ((c >> 3) & 7)));
}

template <int N>
struct RegLds {
  union {
    uint32_t part[N][32][kTileK];                        // column maxima of the 32 thread rows
    __align__(16) uint8_t codes[N][kTileK * kTileK];     // transposed codes
  };
  float scale[N][kTileK];
};

// Write N regions v[n] transposed in three steps with block barriers between
// them: column maxima, scales, codes.  o[n] is the [cols, rows] output whose
// row col0[n] + j is the region's column j (o[n].q NULL: none).
template <int N>
__device__ __forceinline__ void reg_maxima(RegLds<N>& l, const Region& g, const float (&v)[N][kRegRows][kRegCols]) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
    u32x4 m[2];
#pragma unroll
    for (int j = 0; j < kRegCols; ++j) {
      float a = 0.0f;
#pragma unroll
      for (int i = 0; i < kRegRows; i += 2)
        a = __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, fabsf(v[n][i][j])), fabsf(v[n][i + 1][j]));
      m[j / 4][j % 4] = mag(a);
    }
    u32x4* p = reinterpret_cast<u32x4*>(&l.part[n][threadIdx.x / 16][g.c()]);
    p[0] = m[0];
    p[1] = m[1];
  }
}

template <int N>
__device__ __forceinline__ void reg_scales(RegLds<N>& l, const Region& g, const amp_fp8_tiles (&o)[N], const int64_t (&col0)[N]) {
  const int t = threadIdx.x;
  if (t >= N * kTileK) return;
  const int n = __builtin_amdgcn_readfirstlane(t / kTileK), c = t % kTileK;
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 32; ++k) m = m > l.part[n][k][c] ? m : l.part[n][k][c];
  amp_fp8_tiles ot = o[0];
  int64_t first = col0[0];
#pragma unroll
  for (int k = 1; k < N; ++k)
    if (k == n) { ot = o[k]; first = col0[k]; }
  const float sc = scale_of(m, fp8_max(ot.type));
  // the sign carries whether the tile holds a NaN or infinity
  l.scale[n][c] = m >= kInfBits ? -sc : sc;
  if (ot.q && c < g.ncols) ot.s[g.r0 / kTileK * ot.lds + first + c] = 1.0f / sc;
}

template <int N>
__device__ __forceinline__ void reg_codes(RegLds<N>& l, const Region& g, const amp_fp8_tiles (&o)[N], const int64_t (&col0)[N],
                                          const float (&v)[N][kRegRows][kRegCols]) {
  const int t = threadIdx.x;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    if (!o[n].q) continue;
    float sc[kRegCols];
    bool special = false;
#pragma unroll
    for (int j = 0; j < kRegCols; ++j) {
      sc[j] = l.scale[n][g.c() + j];
      special |= sc[j] < 0.0f;
    }
    uint32_t w[kRegCols][1];
    encode<kRegCols, kRegRows, false>(o[n].type, special, w, [&](int j, int i) __attribute__((always_inline)) { return v[n][i][j] * fabsf(sc[j]); });
#pragma unroll
    for (int j = 0; j < kRegCols; ++j) *reinterpret_cast<uint32_t*>(&l.codes[n][reg_at(g.c() + j, t / 16)]) = w[j][0];
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) {
    if (!o[n].q) continue;
#pragma unroll
    for (int it = 0; it < 2; ++it) {
      const int c = it * 64 + t / 8, b = t % 8 * 16;
      if (c >= g.ncols) continue;
      const u32x4 w = *reinterpret_cast<const u32x4*>(&l.codes[n][reg_at(c, b / 4)]);
      uint8_t* p = o[n].q + (col0[n] + c) * o[n].ldq + g.r0;
      if (b + 16 <= g.nrows) {
        *reinterpret_cast<u32x4_any*>(p + b) = w;
      } else {
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (b + k < g.nrows) p[b + k] = static_cast<uint8_t>(w[k / 4] >> (8 * (k & 3)));
      }
    }
  }
}

}  // namespace amp
