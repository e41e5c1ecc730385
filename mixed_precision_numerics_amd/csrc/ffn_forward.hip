// Forward pass of a gated feed-forward block: both projections, the activation
// and the product in one kernel (gfx950).
//
//   [g | u] = x [Wg; Wu]^T,  y = g sigmoid(g) u
//
// Many tokens: gate_tiles (ffn.hpp).  Few tokens: the weights stream past
// them once, which is all the time there is.
#include "ffn.hpp"

namespace amp {
namespace {

template <int ET>
__device__ __forceinline__ f32x4 mfma16x16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (ET == AMP_F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// Up to 16 MT tokens.  A block owns 16 FT features; its NW waves share the
// summed dimension, 32 KC elements a wave and turn, straight from memory into
// the 16x16x32 instruction's operands (weights as rows, tokens as columns: lane
// l holds row l % 16 and elements 8 (l / 16) .. + 7), and join their sums in LDS.
template <int ET, int MT, int FT, int NW, int KC>
__global__ __launch_bounds__(NW * 64) void gate_few(ProductArgs g) {
  __shared__ float part[NW][2 * FT][4][64];
  const int lane = threadIdx.x & 63, wave = wave_id(), q = lane >> 4, i16 = lane & 15;
  const int64_t f0 = static_cast<int64_t>(blockIdx.x) * (16 * FT);
  const uint16_t* x = static_cast<const uint16_t*>(g.A);
  const uint16_t* w = static_cast<const uint16_t*>(g.B);
  const uint16_t *pw[2 * FT], *px[MT];
#pragma unroll
  for (int i = 0; i < FT; ++i) {
    const int64_t f = f0 + 16 * i + i16, row = f < g.N ? f : g.N - 1;
    pw[i] = w + row * g.ldb + 8 * q;
    pw[FT + i] = w + (g.N + row) * g.ldb + 8 * q;
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t m = 16 * i + i16;
    px[i] = x + (m < g.M ? m : g.M - 1) * g.lda + 8 * q;
  }
  f32x4 acc[2 * FT][MT];
#pragma unroll
  for (int i = 0; i < 2 * FT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  int64_t k = wave * (32 * KC);
  for (; k + 32 * KC <= g.K; k += NW * (32 * KC)) {
    u32x4 a[2 * FT][KC], b[MT][KC];
#pragma unroll
    for (int c = 0; c < KC; ++c) {
#pragma unroll
      for (int i = 0; i < 2 * FT; ++i) a[i][c] = ld16u(pw[i] + k + 32 * c);
#pragma unroll
      for (int j = 0; j < MT; ++j) b[j][c] = ld16u(px[j] + k + 32 * c);
    }
#pragma unroll
    for (int c = 0; c < KC; ++c)
#pragma unroll
      for (int i = 0; i < 2 * FT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[i][j] = mfma16x16<ET>(a[i][c], b[j][c], acc[i][j]);
  }
  // the one wave whose turn meets the end; zeros behind it on both sides
  for (; k < g.K; k += 32) {
    const int64_t left = g.K - k - 8 * q;
    const int n = left < 0 ? 0 : left < 8 ? static_cast<int>(left) : 8;
    u32x4 b[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) b[j] = ld16_part(px[j] + k, n);
#pragma unroll
    for (int i = 0; i < 2 * FT; ++i) {
      const u32x4 a = ld16_part(pw[i] + k, n);
#pragma unroll
      for (int j = 0; j < MT; ++j) acc[i][j] = mfma16x16<ET>(a, b[j], acc[i][j]);
    }
  }
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    if (j) __syncthreads();
#pragma unroll
    for (int i = 0; i < 2 * FT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) part[wave][i][r][lane] = acc[i][j][r];
    __syncthreads();
    // row 4 (l / 16) + r of a tile, token l % 16; neighbouring threads store neighbouring features
    for (int o = threadIdx.x; o < 256 * FT; o += NW * 64) {
      const int fl = o % (16 * FT), tok = o / (16 * FT), at = (fl % 16 / 4) * 16 + tok;
      const int64_t f = f0 + fl, m = 16 * j + tok;
      if (f >= g.N || m >= g.M) continue;
      float a = 0.0f, u = 0.0f;
#pragma unroll
      for (int v = 0; v < NW; ++v) {
        a += part[v][fl / 16][fl % 4][at];
        u += part[v][FT + fl / 16][fl % 4][at];
      }
      if (g.C) static_cast<uint16_t*>(g.C)[m * g.ldc + f] = static_cast<uint16_t>(to16<ET>(a * gate(a).s * u));
      if (g.gu) {
        uint16_t* p = static_cast<uint16_t*>(g.gu) + m * g.ldgu + f;
        p[0] = static_cast<uint16_t>(to16<ET>(a));
        p[g.N] = static_cast<uint16_t>(to16<ET>(u));
      }
    }
  }
}

template <int ET, int MT, int FT, int NW, int KC>
hipError_t launch_few(const ProductArgs& g, hipStream_t s) {
  gate_few<ET, MT, FT, NW, KC><<<static_cast<unsigned>(ceil_div(g.N, 16 * FT)), NW * 64, 0, s>>>(g);
  return hipGetLastError();
}

template <int ET>
hipError_t launch_forward(const ProductArgs& g, hipStream_t s) {
  if (g.M <= 16) return launch_few<ET, 1, 1, 8, 4>(g, s);
  if (g.M <= 32) return launch_few<ET, 2, 2, 4, 2>(g, s);
  if (g.M <= 48) return launch_few<ET, 3, 2, 4, 2>(g, s);
  if (g.M <= 64) return launch_few<ET, 4, 2, 4, 2>(g, s);
  return launch_gate<ET, kOutGate>(g, s);
}

}  // namespace

hipError_t launch_gemm_swiglu(int64_t M, int64_t F, int64_t K, const void* x, int t, int64_t ldx, const void* w,
                              int64_t ldw, void* y, int64_t ldy, void* gu, int64_t ldgu, hipStream_t s) {
  ProductArgs g{};
  g.A = x; g.lda = ldx; g.B = w; g.ldb = ldw; g.M = M; g.N = F; g.K = K;
  g.C = y; g.ldc = ldy; g.gu = gu; g.ldgu = ldgu; g.splits = 1;
  return t == AMP_BF16 ? launch_forward<AMP_BF16>(g, s) : launch_forward<AMP_F16>(g, s);
}

}  // namespace amp
