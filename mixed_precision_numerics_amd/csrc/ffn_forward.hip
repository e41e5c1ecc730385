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

// Eight elements at any 2-byte address from the dwords that hold them, shifted into
// place (each dword read holds one of the elements: none lies outside the
// operand's pages).  Waves that only stream would wait for 16-byte loads at odd
// addresses: 1 x 4097 x 14336 106 us, so 64.
typedef uint32_t u32x4_dw __attribute__((ext_vector_type(4), aligned(4)));
struct Piece {
  u32x4 w;
  uint32_t last;
  static __device__ __forceinline__ uint32_t odd(const uint16_t* p) { return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 2u; }
  __device__ __forceinline__ void load(const uint16_t* p) {
    const uint32_t* q = reinterpret_cast<const uint32_t*>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t(2));
    w = *reinterpret_cast<const u32x4_dw*>(q);
    last = q[3 + (odd(p) >> 1)];
  }
  __device__ __forceinline__ u32x4 shifted(uint32_t by) const {
    return u32x4{__builtin_amdgcn_alignbit(w[1], w[0], by), __builtin_amdgcn_alignbit(w[2], w[1], by),
                 __builtin_amdgcn_alignbit(w[3], w[2], by), __builtin_amdgcn_alignbit(last, w[3], by)};
  }
};

// Up to 16 tokens.  A block owns 16 features; its waves share the summed
// dimension, 64 elements a wave and turn, straight from memory into the 16x16x32
// instruction's operands (weights as rows, tokens as columns: lane l holds row l %
// 16 and elements 8 (l / 16) .. + 7), and join their sums in LDS.  16 waves a block
// keep 64 KB of weights a CU in flight: 1 x 4096 x 14336 BF16 43 us = 5.5 TB/s (8
// waves with 128 elements a turn: 46), 1 x 5120 x 20480 72 us = 5.8 TB/s (81).
constexpr int kFewTokens = 16, kFewWaves = 16, kFewTurn = 64;

// WHOLE: every row is whole 16-byte pieces.
template <int ET, bool WHOLE>
__global__ __launch_bounds__(kFewWaves * 64) void gate_few(ProductArgs g) {
  constexpr int kC = kFewTurn / 32;
  __shared__ float part[kFewWaves][2][4][64];
  const int lane = threadIdx.x & 63, wave = wave_id(), q = lane >> 4, i16 = lane & 15;
  const int64_t f0 = static_cast<int64_t>(blockIdx.x) * 16;
  const int64_t f = f0 + i16 < g.N ? f0 + i16 : g.N - 1, m = i16 < g.M ? i16 : g.M - 1;
  const uint16_t* w = static_cast<const uint16_t*>(g.B) + 8 * q;
  const uint16_t* const px = static_cast<const uint16_t*>(g.A) + m * g.lda + 8 * q;
  const uint16_t* const pw[2] = {w + f * g.ldb, w + (g.N + f) * g.ldb};
  f32x4 acc[2] = {};
  int64_t k = wave * kFewTurn;
  for (; k + kFewTurn <= g.K; k += kFewWaves * kFewTurn) {
    Piece a[2][kC], b[kC];
    auto load = [&](Piece& v, const uint16_t* p) __attribute__((always_inline)) {
      if constexpr (WHOLE) v.w = ld16(p);
      else v.load(p);
    };
    auto value = [&](const Piece& v, const uint16_t* p) __attribute__((always_inline)) {
      if constexpr (WHOLE) return v.w;
      else return v.shifted(8 * Piece::odd(p));
    };
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      load(a[0][c], pw[0] + k + 32 * c);
      load(a[1][c], pw[1] + k + 32 * c);
      load(b[c], px + k + 32 * c);
    }
    // (k and 32 c are even: a row's pieces are all odd or all even)
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const u32x4 x = value(b[c], px);
      acc[0] = mfma16x16<ET>(value(a[0][c], pw[0]), x, acc[0]);
      acc[1] = mfma16x16<ET>(value(a[1][c], pw[1]), x, acc[1]);
    }
  }
  // the one wave whose turn meets the end; zeros behind it on both sides
  for (; k < g.K; k += 32) {
    const int64_t left = g.K - k - 8 * q;
    const int n = left < 0 ? 0 : left < 8 ? static_cast<int>(left) : 8;
    const u32x4 b = ld16_part(px + k, n);
    acc[0] = mfma16x16<ET>(ld16_part(pw[0] + k, n), b, acc[0]);
    acc[1] = mfma16x16<ET>(ld16_part(pw[1] + k, n), b, acc[1]);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) part[wave][i][r][lane] = acc[i][r];
  __syncthreads();
  // row 4 (l / 16) + r of a tile, token l % 16; neighbouring threads store neighbouring features
  const int fl = threadIdx.x % 16, tok = threadIdx.x / 16, at = fl / 4 * 16 + tok;
  if (threadIdx.x >= 256 || f0 + fl >= g.N || tok >= g.M) return;
  float a = 0.0f, u = 0.0f;
#pragma unroll
  for (int v = 0; v < kFewWaves; ++v) {
    a += part[v][0][fl % 4][at];
    u += part[v][1][fl % 4][at];
  }
  if (g.C) static_cast<uint16_t*>(g.C)[tok * g.ldc + f0 + fl] = static_cast<uint16_t>(to16<ET>(a * gate(a).s * u));
  if (g.gu) {
    uint16_t* p = static_cast<uint16_t*>(g.gu) + tok * g.ldgu + f0 + fl;
    p[0] = static_cast<uint16_t>(to16<ET>(a));
    p[g.N] = static_cast<uint16_t>(to16<ET>(u));
  }
}

template <int ET>
hipError_t launch_forward(const ProductArgs& g, hipStream_t s) {
  if (g.M > kFewTokens) return launch_gate<ET, kOutGate>(g, s);
  const unsigned blocks = static_cast<unsigned>(ceil_div(g.N, 16));
  if (aligned(g.A, 16) && aligned(g.B, 16) && g.lda % 8 == 0 && g.ldb % 8 == 0) gate_few<ET, true><<<blocks, kFewWaves * 64, 0, s>>>(g);
  else gate_few<ET, false><<<blocks, kFewWaves * 64, 0, s>>>(g);
  return hipGetLastError();
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
