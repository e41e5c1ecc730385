// Products of a gated feed-forward block on the matrix cores (gfx950): one
// tile kernel for the fused forward pass, its recomputing backward form and
// the two gradient products.
//
//   forward      [g | u] = x [Wg; Wu]^T,  y = g sigmoid(g) u   (kOutGate)
//   backward     dg, du of dy from g, u formed again           (kOutGrad)
//   gradients    dx = [dg | du] W,  dW = [dg | du]^T x         (kOutC)
//
// A block of four waves (2 x 2) owns an output tile of 64 MB x 64 NB (columns of
// both projections together: a wave's first NB/2 blocks of 32 columns are gate
// columns, the others the up columns of the same features, so that a lane's
// accumulators pair up with no exchange).  The summed dimension advances 64
// elements at a time through a ring of LDS slots that direct loads fill up to D
// steps ahead, one load for each row of 32x32x16 products, with one meeting of the
// block a step.  Operands are contiguous along the summed dimension (KC) or along
// their rows of outputs (then read with transposing LDS reads).
//
// Bound by the matrix cores from a few hundred tokens on.  A 256 x 256 tile needs
// half the LDS reads and half the loads of a 128 x 128 tile a product, which
// is worth more than a second block on the CU (8192 x 4096 x 14336 BF16 with [g | u]
// kept: 1445 us against 2021); 128 x 128 tiles, two to a CU, are for outputs of fewer
// large tiles than CUs and short sums.  At that size the K loop runs at 89 % of the
// matrix cores' rate, the tiles' ends cost 11 us of a CU each (of 106), and the last
// round leaves 6 % of the machine idle; 1.33 PFLOP/s where a library product of the
// same operands, without gate or second output, reaches 1.5.
//
// Edges.  Output rows and columns past the end are read from the last valid
// one (their results are not stored), so no load leaves the operand.  What
// does not fill a step of the summed dimension is put into LDS through
// registers, masked with zeros on both sides (a NaN behind a row's end must
// not meet a zero), as the first step of a tile.  Operands without 16-byte
// rows go that way in every step (FAST == false), where loads that are not
// 16-byte aligned bound them: 1000 x 4097 x 14336 390 us against 190 to 200 for 4096.
#pragma once
#include <type_traits>

#include "common.hpp"
#include "ffn_choice.hpp"
#include "formats.hpp"
#include "gate.hpp"
#include "mfma.hpp"

namespace amp {
namespace {

enum Out : int { kOutC = 0, kOutGate = 1, kOutGrad = 2 };

struct ProductArgs {
  const void* A;           // [M, K], or [K, M] where M is contiguous
  const void* B;           // [N, K] ([2N, K] with a gate), or [K, N]
  int64_t M, N, K;         // N: columns of the output (features with a gate)
  int64_t lda, ldb;
  void* C; int64_t ldc;    // the product; with a gate y (may be NULL)
  void* gu; int64_t ldgu;  // kOutGate: [g | u] (may be NULL); kOutGrad: [dg | du]
  const void* dy; int64_t lddy;
  int out32;               // kOutC: C is FP32
  int splits;              // parts of the summed dimension; > 1: C is FP32 [splits][M][N]
};

// 16 bytes at any 2-byte address in one load or store.
typedef uint32_t u32x4_u __attribute__((ext_vector_type(4), aligned(2)));

template <int ET>
__device__ __forceinline__ float from16(uint32_t c) {
  return ET == AMP_BF16 ? bf16_to_f32(c) : f16_to_f32(c);
}
template <int ET>
__device__ __forceinline__ uint32_t to16(float x) {
  if constexpr (ET == AMP_BF16) return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
  else return __builtin_bit_cast(uint16_t, static_cast<_Float16>(x));
}
template <int ET>
__device__ __forceinline__ uint32_t to16x2(float x, float y) { return to16<ET>(x) | to16<ET>(y) << 16; }

template <int ET>
__device__ __forceinline__ f32x16 mfma16(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (ET == AMP_F16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// Eight elements from p on of which the first n exist, zeros behind them.  The
// loads of an incomplete piece are under way together, past its end from its
// first element.
__device__ __forceinline__ u32x4 ld16_part(const uint16_t* p, int n) {
  if (n >= 8) return *reinterpret_cast<const u32x4_u*>(p);
  u32x4 v = {0u, 0u, 0u, 0u};
  if (n > 0) {
    uint32_t e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = p[j < n ? j : 0];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j >> 1] |= (j < n ? e[j] : 0u) << (16 * (j & 1));
  }
  return v;
}

// v without its first `by` elements (0 .. 8), zeros behind what is left.
__device__ __forceinline__ u32x4 without(u32x4 v, int by) {
  const bool half = by & 1;
  if (by & 2) v = u32x4{v[1], v[2], v[3], 0u};
  if (by & 4) v = u32x4{v[2], v[3], 0u, 0u};
  if (by & 8) v = u32x4{0u, 0u, 0u, 0u};
  return u32x4{half ? __builtin_amdgcn_alignbit(v[1], v[0], 16) : v[0], half ? __builtin_amdgcn_alignbit(v[2], v[1], 16) : v[1],
               half ? __builtin_amdgcn_alignbit(v[3], v[2], 16) : v[2], half ? v[3] >> 16 : v[3]};
}

// How far a piece of which n elements exist is loaded before its place, so as to
// end with them; `without` of as many puts them there.
__device__ __forceinline__ int back_of(int n) { return n >= 8 ? 0 : n <= 0 ? 8 : 8 - n; }

// LDS writes of one wave before its own reads of them (and reads before the
// next writes): a wave's LDS operations complete in order, the compiler has to
// keep that order.
__device__ __forceinline__ void wave_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// Epilogue of one wave.  The products are formed as B A^T, which leaves a lane
// four neighbouring columns of one row in each four accumulator registers: lane l
// holds row l % 32 and columns 8 q + 4 (l / 32) + e in register 4 q + e.  A band of
// 32 rows x 32 NBW columns leaves through this wave's LDS region as whole 16-byte
// pieces of rows; the pitch, a row's bytes + 16, spreads 16 rows over all banks.
// value(nb, r): the element of column block nb in register r.  Several bands are put
// before the first is stored: LDS latency is met once.
template <int CT, int NBW>
struct BandOut {
  static constexpr int kES = CT == AMP_F32 ? 4 : 2, kRow = NBW * 32 * kES, kPitch = kRow + 16, kBytes = 32 * kPitch;
  static constexpr int kLPR = kRow / 16, kRPP = 64 / kLPR, kEPL = 16 / kES;
  template <typename V>
  static __device__ __forceinline__ void put(V&& value, uint8_t* buf) {
    const int lane = threadIdx.x & 63;
    uint8_t* mine = buf + (lane & 31) * kPitch + (lane >> 5) * 4 * kES;
#pragma unroll
    for (int nb = 0; nb < NBW; ++nb)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float x[4] = {value(nb, 4 * q), value(nb, 4 * q + 1), value(nb, 4 * q + 2), value(nb, 4 * q + 3)};
        uint8_t* p = mine + (nb * 32 + 8 * q) * kES;
        if constexpr (CT == AMP_F32) *reinterpret_cast<u32x4*>(p) = u32x4{fbits(x[0]), fbits(x[1]), fbits(x[2]), fbits(x[3])};
        else *reinterpret_cast<u32x2*>(p) = u32x2{to16x2<CT>(x[0], x[1]), to16x2<CT>(x[2], x[3])};
      }
  }
  static __device__ __forceinline__ void store(void* C, int64_t ldc, int64_t row0, int64_t col0, int64_t M, int64_t N, const uint8_t* buf) {
    const int lane = threadIdx.x & 63;
    const int64_t col = col0 + (lane % kLPR) * kEPL;
#pragma unroll
    for (int ps = 0; ps < 32 / kRPP; ++ps) {
      const int rl = ps * kRPP + lane / kLPR;
      const int64_t row = row0 + rl;
      const uint8_t* q = buf + rl * kPitch + (lane % kLPR) * 16;
      if (row >= M || col >= N) continue;
      uint8_t* out = static_cast<uint8_t*>(C) + (row * ldc + col) * kES;
      if (col + kEPL <= N) {
        *reinterpret_cast<u32x4_u*>(out) = *reinterpret_cast<const u32x4*>(q);
      } else {
        for (int j = 0; j < N - col; ++j) {
          if constexpr (CT == AMP_F32) reinterpret_cast<float*>(out)[j] = reinterpret_cast<const float*>(q)[j];
          else reinterpret_cast<uint16_t*>(out)[j] = reinterpret_cast<const uint16_t*>(q)[j];
        }
      }
    }
  }
};

// The reverse way for a band of a 16-bit matrix: its pieces on their way into
// registers (zeros outside), then through LDS into the lanes' elements, four of
// one row in v[nb][q].
template <int NBW>
struct BandIn {
  static constexpr int kRow = NBW * 64, kPitch = kRow + 16, kBytes = 32 * kPitch, kLPR = kRow / 16, kRPP = 64 / kLPR;
  u32x4 w[32 / kRPP];
  __device__ __forceinline__ void load(const void* X, int64_t ldx, int64_t row0, int64_t col0, int64_t M, int64_t N) {
    const int lane = threadIdx.x & 63;
    const int64_t col = col0 + (lane % kLPR) * 8;
    const int left = col < N ? static_cast<int>(N - col < 8 ? N - col : 8) : 0;
#pragma unroll
    for (int ps = 0; ps < 32 / kRPP; ++ps) {
      const int64_t row = row0 + ps * kRPP + lane / kLPR;
      w[ps] = row < M ? ld16_part(static_cast<const uint16_t*>(X) + row * ldx + col, left) : u32x4{0u, 0u, 0u, 0u};
    }
  }
  __device__ __forceinline__ void put(uint8_t* buf) const {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int ps = 0; ps < 32 / kRPP; ++ps)
      *reinterpret_cast<u32x4*>(buf + (ps * kRPP + lane / kLPR) * kPitch + (lane % kLPR) * 16) = w[ps];
  }
  static __device__ __forceinline__ void spread(u32x2 (&v)[NBW][4], const uint8_t* buf) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int nb = 0; nb < NBW; ++nb)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        v[nb][q] = *reinterpret_cast<const u32x2*>(buf + (lane & 31) * kPitch + (nb * 32 + 8 * q + 4 * (lane >> 5)) * 2);
  }
};

// A direct-to-LDS load of 16 bytes a lane (64 lanes fill 1 KB from dst on) that
// the compiler does not track: the kernel waits for it by count.
__device__ __forceinline__ void to_lds(__amdgpu_buffer_rsrc_t rsrc, uint32_t dst, uint32_t voff, uint32_t soff) {
  asm volatile("buffer_load_dwordx4 %0, %1, %2 offen lds" ::"v"(voff), "s"(rsrc), "s"(__builtin_amdgcn_readfirstlane(soff)),
               "{m0}"(__builtin_amdgcn_readfirstlane(dst)));
}

constexpr int kStepBytes = 2 * kStepK;                   // bytes of a row of a step
static_assert(kStepBytes == kRowBytes, "the slots' layout");

// The same in an output-contiguous stage, rows of `pitch` bytes along K.
__device__ __forceinline__ int mn_at(int k, int c, int pitch) { return k * pitch + ((c ^ (4 * (k & 3))) << 4); }

// LDS of a ring that reaches D steps ahead: slots of one operand's step.
constexpr int lds_bytes(int MB, int NB, int D) { return (2 * D + 1) * 64 * (MB > NB ? MB : NB) * kStepBytes; }

// Block `block` of the product's tiles, part z of the summed dimension.
template <int ET, bool A_KC, bool B_KC, int OUT, int MB, int NB, int D, bool FAST>
__device__ __forceinline__ void product(const ProductArgs& g, uint32_t block, uint32_t z, uint8_t* smem) {
  constexpr bool kGate = OUT != kOutC;
  static_assert(!kGate || (A_KC && B_KC), "the projections' operands are K-contiguous");
  constexpr int BM = 64 * MB, BN = 64 * NB, BNO = kGate ? BN / 2 : BN, NBH = NB / 2;
  constexpr int kSlots = 2 * D + 1, kSlot = lds_bytes(MB, NB, D) / kSlots;      // a slot holds one operand of a step
  constexpr int kLA = 2 * MB, kLB = 2 * NB;                    // direct loads of a wave and operand

  // Blocks of one XCD (every eighth) take one contiguous run of tiles, eight
  // tile rows at a time, so that its L2 holds the operands' shared parts.
  const uint32_t nbm = static_cast<uint32_t>((g.M + BM - 1) / BM), nbn = static_cast<uint32_t>((g.N + BNO - 1) / BNO);
  const uint32_t total = nbm * nbn, xcd = block % 8, most = total % 8;
  const uint32_t tile = xcd * (total / 8) + (xcd < most ? xcd : most) + block / 8;
  constexpr uint32_t kGroup = 8;
  const uint32_t first_m = tile / (kGroup * nbn) * kGroup;
  const uint32_t gsz = nbm - first_m < kGroup ? nbm - first_m : kGroup;
  const uint32_t in_group = tile % (kGroup * nbn);
  const int64_t m0 = static_cast<int64_t>(__builtin_amdgcn_readfirstlane(first_m + in_group % gsz)) * BM;
  const int64_t n0 = static_cast<int64_t>(__builtin_amdgcn_readfirstlane(in_group / gsz)) * BNO;

  const int t = threadIdx.x, lane = t & 63, wave = wave_id();
  const int wm = wave >> 1, wn = wave & 1, l32 = lane & 31, h = lane >> 5;
  const int rows_a = static_cast<int>(g.M - m0 < BM ? g.M - m0 : BM);       // what the tile holds of each operand
  const int rows_b = static_cast<int>(g.N - n0 < BNO ? g.N - n0 : BNO);
  const uint16_t* A = static_cast<const uint16_t*>(g.A) + (A_KC ? m0 * g.lda : m0);
  const uint16_t* B = static_cast<const uint16_t*>(g.B) + (B_KC ? n0 * g.ldb : n0);
  const uint32_t lda_b = static_cast<uint32_t>(g.lda * 2), ldb_b = static_cast<uint32_t>(g.ldb * 2);

  // The steps of this block: whole ones, what is left over being the first.
  const int whole = __builtin_amdgcn_readfirstlane(static_cast<int>(g.K / kStepK)), tail = __builtin_amdgcn_readfirstlane(g.K % kStepK != 0), steps = whole + tail;
  const int s0 = __builtin_amdgcn_readfirstlane(static_cast<int>(static_cast<int64_t>(steps) * z / g.splits));
  const int s1 = __builtin_amdgcn_readfirstlane(static_cast<int>(static_cast<int64_t>(steps) * (z + 1) / g.splits));
  auto first_k = [&](int s) __attribute__((always_inline)) { return __builtin_amdgcn_readfirstlane((tail ? (s == 0 ? whole : s - 1) : s) * kStepK); };

  // LDS row r of the B stage: with a gate, the feature and the projection that
  // it holds; rows past the end repeat the last.
  auto row_b = [&](int r) __attribute__((always_inline)) -> int64_t {
    if constexpr (!kGate) return r < rows_b ? r : rows_b - 1;
    const int f = r / (32 * NB) * (16 * NB) + r % (16 * NB);
    return (f < rows_b ? f : rows_b - 1) + (r / (16 * NB) % 2 ? g.N : 0);
  };

  // ---- direct loads of a whole step, 1 KB of LDS each.  KC: eight rows; lane l
  // fetches the chunk that belongs at byte 16 l.  Else: K-rows, likewise.
  uint32_t va[A_KC ? kLA : 2], vb[B_KC ? kLB : 2];
  constexpr int kChA = BM / 8, kChB = BN / 8, kRowsA = 64 / kChA, kRowsB = 64 / kChB;   // chunks of a K-row, K-rows of a load
  const int part = kGate ? wave & 1 : 0;
  const uint16_t* Bw = B + (part ? g.N * g.ldb : 0);      // the wave's projection
  if constexpr (FAST) {
#pragma unroll
    for (int i = 0; i < (A_KC ? kLA : 2); ++i) {
      if constexpr (A_KC) {
        const int r = wave * 8 * kLA + 8 * i + lane / 8;
        va[i] = static_cast<uint32_t>(r < rows_a ? r : rows_a - 1) * lda_b + (((lane & 7) ^ (lane >> 3) ^ ((wave * kLA + i) & 7)) << 4);
      } else {
        const int k = i * kRowsA + lane / kChA, c = (lane % kChA) ^ (4 * (k & 3));
        va[i] = static_cast<uint32_t>(lane / kChA) * lda_b + static_cast<uint32_t>(c < rows_a / 8 ? c : rows_a / 8 - 1) * 16;
      }
    }
#pragma unroll
    for (int i = 0; i < (B_KC ? kLB : 2); ++i) {
      if constexpr (B_KC) {
        const int f = (kGate ? wave >> 1 : wave) * 8 * kLB + 8 * i + lane / 8;
        vb[i] = static_cast<uint32_t>(f < rows_b ? f : rows_b - 1) * ldb_b + (((lane & 7) ^ (lane >> 3) ^ ((wave * kLB + i) & 7)) << 4);
      } else {
        const int k = i * kRowsB + lane / kChB, c = (lane % kChB) ^ (4 * (k & 3));
        vb[i] = static_cast<uint32_t>(lane / kChB) * ldb_b + static_cast<uint32_t>(c < rows_b / 8 ? c : rows_b / 8 - 1) * 16;
      }
    }
  }
  // bytes from the operand's first to its last element in the tile (KC) or the step
  const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint16_t*>(A), 0, static_cast<int>(A_KC ? (rows_a - 1) * lda_b + g.K * 2 : 0), 0x00020000);
  const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint16_t*>(Bw), 0, static_cast<int>(B_KC ? (rows_b - 1) * ldb_b + g.K * 2 : 0), 0x00020000);
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_void*)smem));
  // Load i of a wave's share; past the end the last step is loaded once more,
  // into a slot that nobody reads.
  auto direct_a = [&](int s, int slot, int i) __attribute__((always_inline)) {
    const int k0 = ((s < s1 ? s : s1 - 1) - tail) * kStepK;
    const uint32_t dst = lds0 + slot * kSlot + (wave * kLA + i) * 1024;
    if constexpr (A_KC) {
      to_lds(ra, dst, va[i], static_cast<uint32_t>(k0 * 2));
    } else {
      const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<uint16_t*>(A + k0 * g.lda), 0, static_cast<int>((kStepK - 1) * lda_b + rows_a * 2), 0x00020000);
      to_lds(r, dst, va[kRowsA == 2 ? i & 1 : 0], static_cast<uint32_t>(wave * (kStepK / 4) + kRowsA * i) * lda_b);
    }
  };
  auto direct_b = [&](int s, int slot, int i) __attribute__((always_inline)) {
    const int k0 = ((s < s1 ? s : s1 - 1) - tail) * kStepK;
    const uint32_t dst = lds0 + slot * kSlot + (wave * kLB + i) * 1024;
    if constexpr (B_KC) {
      to_lds(rb, dst, vb[i], static_cast<uint32_t>(k0 * 2));
    } else {
      const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<uint16_t*>(B + k0 * g.ldb), 0, static_cast<int>((kStepK - 1) * ldb_b + rows_b * 2), 0x00020000);
      to_lds(r, dst, vb[kRowsB == 2 ? i & 1 : 0], static_cast<uint32_t>(wave * (kStepK / 4) + kRowsB * i) * ldb_b);
    }
  };

  // ---- the same through registers, masked.  Where every step has incomplete pieces
  // (outputs contiguous), one is loaded as the last whole piece of its row and put
  // right on its way into LDS: branches would have the loads wait for one another
  // (the backward call of 300 x 1001 x 2047 BF16 38 us, so 35).  Rows of fewer than eight
  // elements have no whole piece.
  u32x4 ha[kLA], hb[kLB];
  const bool short_a = !A_KC && g.M < 8, short_b = !B_KC && g.N < 8;
  auto left_of = [&](int s) __attribute__((always_inline)) {
    const int64_t left = g.K - first_k(s);
    return static_cast<int>(left < kStepK ? left : kStepK);
  };
  auto fetch_a = [&](int s) __attribute__((always_inline)) {
    const int k0 = first_k(s), n = left_of(s);
#pragma unroll
    for (int i = 0; i < kLA; ++i) {
      const int e = t + 256 * i;
      if constexpr (A_KC) {
        const int r = e >> 3, c = 8 * (e & 7);
        ha[i] = ld16_part(A + (r < rows_a ? r : rows_a - 1) * g.lda + k0 + c, n - c);
      } else {
        const int k = e / kChA, c = 8 * (e % kChA);
        const uint16_t* p = A + static_cast<int64_t>(k0 + (k < n ? k : n - 1)) * g.lda;
        ha[i] = short_a ? ld16_part(p + c, k < n ? rows_a - c : 0) : *reinterpret_cast<const u32x4_u*>(p + (c + 8 <= rows_a ? c : rows_a - 8));
      }
    }
  };
  auto fetch_b = [&](int s) __attribute__((always_inline)) {
    const int k0 = first_k(s), n = left_of(s);
#pragma unroll
    for (int i = 0; i < kLB; ++i) {
      const int e = t + 256 * i;
      if constexpr (B_KC) {
        const int c = 8 * (e & 7);
        hb[i] = ld16_part(B + row_b(e >> 3) * g.ldb + k0 + c, n - c);
      } else {
        const int k = e / kChB, c = 8 * (e % kChB);
        const uint16_t* p = B + static_cast<int64_t>(k0 + (k < n ? k : n - 1)) * g.ldb;
        hb[i] = short_b ? ld16_part(p + c, k < n ? rows_b - c : 0) : *reinterpret_cast<const u32x4_u*>(p + (c + 8 <= rows_b ? c : rows_b - 8));
      }
    }
  };
  auto put_a = [&](int s, int slot) __attribute__((always_inline)) {
    if constexpr (!A_KC) {
      const int n = left_of(s);
      if (!short_a && (n < kStepK || rows_a < BM)) {
#pragma unroll
        for (int i = 0; i < kLA; ++i) {
          const int e = t + 256 * i;
          ha[i] = without(ha[i], e / kChA < n ? back_of(rows_a - 8 * (e % kChA)) : 8);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kLA; ++i) {
      const int e = t + 256 * i;
      *reinterpret_cast<u32x4*>(smem + slot * kSlot + (A_KC ? swz(e >> 3, e & 7) : mn_at(e / kChA, e % kChA, BM * 2))) = ha[i];
    }
  };
  auto put_b = [&](int s, int slot) __attribute__((always_inline)) {
    if constexpr (!B_KC) {
      const int n = left_of(s);
      if (!short_b && (n < kStepK || rows_b < BN)) {
#pragma unroll
        for (int i = 0; i < kLB; ++i) {
          const int e = t + 256 * i;
          hb[i] = without(hb[i], e / kChB < n ? back_of(rows_b - 8 * (e % kChB)) : 8);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kLB; ++i) {
      const int e = t + 256 * i;
      *reinterpret_cast<u32x4*>(smem + slot * kSlot + (B_KC ? swz(e >> 3, e & 7) : mn_at(e / kChB, e % kChB, BN * 2))) = hb[i];
    }
  };

  // ---- fragments of 16 along K: KC, chunk 2 ks + h of the lane's row; else two
  // transposing reads
  const uint32_t sw = static_cast<uint32_t>((h ^ l32 ^ (l32 >> 3)) & 7) << 4;      // rows 32 apart: ^ 4 chunks
  const uint32_t arow = static_cast<uint32_t>(wm * 32 * MB + l32) * kStepBytes + sw;
  const uint32_t brow = static_cast<uint32_t>(wn * 32 * NB + l32) * kStepBytes + sw;
  const int tq = lane >> 4, ts = lane & 15, tk = 8 * (tq >> 1) + (ts >> 2);
  auto tr_at = [&](int c0, int b, int pitch) __attribute__((always_inline)) {
    return static_cast<uint32_t>(mn_at(tk, (c0 >> 3) + 4 * b + 2 * (tq & 1) + ((ts & 3) >> 1), pitch) + 8 * (ts & 1));
  };
  u32x4 fa[2][MB], fb[2][NB];
  auto frag_a = [&](int slot, int ks, int i, u32x4& v) __attribute__((always_inline)) {
    const uint8_t* st = smem + slot * kSlot;
    if constexpr (A_KC) v = *reinterpret_cast<const u32x4*>(st + (arow ^ static_cast<uint32_t>((2 * ks ^ 4 * (i & 1)) << 4)) + i * 32 * kStepBytes);
    else v = frag_tr<BM * 2>(st, tr_at(wm * 32 * MB, i, BM * 2), ks);
  };
  auto frag_b = [&](int slot, int ks, int i, u32x4& v) __attribute__((always_inline)) {
    const uint8_t* st = smem + slot * kSlot;
    if constexpr (B_KC) v = *reinterpret_cast<const u32x4*>(st + (brow ^ static_cast<uint32_t>((2 * ks ^ 4 * (i & 1)) << 4)) + i * 32 * kStepBytes);
    else v = frag_tr<BN * 2>(st, tr_at(wn * 32 * NB, i, BN * 2), ks);
  };
  // Part p of n of a slice's fragments, the columns' first: the next slice's
  // first products need all of them and one of the rows'.
  auto frag_part = [&](int sa, int sb, int ks, int p, int n) __attribute__((always_inline)) {
    constexpr int kAll = MB + NB;
#pragma unroll
    for (int j = 0; j < kAll; ++j)
      if (j >= kAll * p / n && j < kAll * (p + 1) / n) {
        if (j < NB) frag_b(sb, ks, j, fb[ks & 1][j]);
        else frag_a(sa, ks, j - NB, fa[ks & 1][j - NB]);
      }
  };

  // Operand slots form a ring, A and B of a step side by side: while step s is
  // multiplied the operands up to B of step s + D - 1 and A of step s + D are on
  // their way, one load for each row of products (the first of B as soon as the step
  // before has met).  Loads land in order, so they are waited for by count.
  constexpr int kMeet = 3 * MB, kAhead = MB - 1, kFlying = (D - 1) * kLA + (D - 2) * kLB;
  static_assert(4 * MB == kLA + kLB, "a load for each row of products");
  auto after = [](int slot, int n) __attribute__((always_inline)) { return slot + n >= kSlots ? slot + n - kSlots : slot + n; };
  const bool more = s0 + 1 < s1;
  if (s0 < s1) {
    if (!FAST || (tail && s0 == 0)) {
      fetch_a(s0);
      put_a(s0, 0);
      fetch_b(s0);
      put_b(s0, 1);
    } else {
#pragma unroll
      for (int i = 0; i < kLA; ++i) direct_a(s0, 0, i);
#pragma unroll
      for (int i = 0; i < kLB; ++i) direct_b(s0, 1, i);
    }
    if (FAST && more) {
#pragma unroll
      for (int d = 1; d < D; ++d) {
#pragma unroll
        for (int i = 0; i < kLA; ++i) direct_a(s0 + d, 2 * d, i);
#pragma unroll
        for (int i = 0; i < (d + 1 < D ? kLB : kAhead); ++i) direct_b(s0 + d, 2 * d + 1, i);
      }
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kFlying + kAhead) : "memory");
    } else {
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    }
    if (!FAST && more) {
      fetch_a(s0 + 1);
      fetch_b(s0 + 1);
    }
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    frag_part(0, 1, 0, 0, 1);
  }
  f32x16 acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  // One step, slots sa and sa + 1: four slices of 16, a slice's products row by
  // row, between them the next slice's fragments and the loads.  The block meets
  // once, after the last slice's first row: the next step has landed, and every wave
  // has its last fragments of this one.  The compiler keeps to this order.
  auto step = [&](int s, int sa, auto next) __attribute__((always_inline)) {
    constexpr bool MORE = decltype(next)::value;
    const int sb = after(sa, 1), na = after(sa, 2), nb = after(sa, 3);
    if constexpr (MORE && !FAST) {
      put_a(s + 1, na);
      put_b(s + 1, nb);
      if (s + 2 < s1) {
        fetch_a(s + 2);
        fetch_b(s + 2);
      }
    }
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      const int cur = ks & 1;
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        const int region = ks * MB + i, l = region + kAhead;
        if constexpr (MORE && FAST) {
          if (region > kMeet) direct_b(s + D, sa, region - kMeet - 1);
          else if (l < kLB) direct_b(s + D - 1, after(sa, 2 * D - 1), l);
          else direct_a(s + D, after(sa, 2 * D), l - kLB);
        }
        if (ks < 3) frag_part(sa, sb, ks + 1, i, MB - 1);
        else if (MORE && i > 0) frag_part(na, nb, 0, i - 1, MB - 1);
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = mfma16<ET>(fb[cur][j], fa[cur][i], acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);
        if (MORE && region == kMeet) {
          if constexpr (FAST) {
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kFlying) : "memory");
          } else {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
          }
          __builtin_amdgcn_s_barrier();
          asm volatile("" ::: "memory");
        }
      }
    }
  };
  if (s0 < s1) {
    int s = s0, sa = 0;
    for (; s + 1 < s1; ++s) {
      step(s, sa, std::true_type{});
      sa = after(sa, 2);
    }
    step(s, sa, std::false_type{});
  }

  // ---- epilogue: a quarter of the slots for each wave's bands
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  constexpr int kBandCols = kGate ? 16 * NB : 32 * NB, kRegion = kSlots * kSlot / 4;
  uint8_t* buf = smem + wave * kRegion;
  const int64_t row0 = m0 + wm * 32 * MB, col0 = n0 + wn * kBandCols;
  if constexpr (OUT == kOutC) {
    auto leave = [&](auto band, void* C) __attribute__((always_inline)) {
      using Out = decltype(band);
      constexpr int kAtOnce = MB * Out::kBytes <= kRegion ? MB : MB / 2;
      static_assert(kAtOnce * Out::kBytes <= kRegion, "the bands exceed a wave's part of the slots");
#pragma unroll
      for (int i0 = 0; i0 < MB; i0 += kAtOnce) {
        wave_lds();
#pragma unroll
        for (int i = i0; i < i0 + kAtOnce; ++i)
          Out::put([&](int nb, int r) __attribute__((always_inline)) { return acc[i][nb][r]; }, buf + (i - i0) * Out::kBytes);
        wave_lds();
#pragma unroll
        for (int i = i0; i < i0 + kAtOnce; ++i) Out::store(C, g.ldc, row0 + 32 * i, col0, g.M, g.N, buf + (i - i0) * Out::kBytes);
      }
    };
    if (g.out32) leave(BandOut<AMP_F32, NB>{}, static_cast<float*>(g.C) + z * g.M * g.N);
    else leave(BandOut<ET, NB>{}, g.C);
  } else {
    using Out = BandOut<ET, NBH>;
    void* const gu2 = static_cast<uint16_t*>(g.gu) + g.N;       // the up half of [g | u]
    auto store = [&](void* C, int64_t ldc, int i, int place) __attribute__((always_inline)) {
      Out::store(C, ldc, row0 + 32 * i, col0, g.M, g.N, buf + place * Out::kBytes);
    };
    auto put = [&](int i, int half, int place) __attribute__((always_inline)) {
      Out::put([&](int nb, int r) __attribute__((always_inline)) { return acc[i][half * NBH + nb][r]; }, buf + place * Out::kBytes);
    };
    if constexpr (OUT == kOutGate) {
      static_assert(2 * MB * Out::kBytes <= kRegion, "the bands exceed a wave's part of the slots");
      if (g.gu) {
#pragma unroll
        for (int i = 0; i < MB; ++i) {
          put(i, 0, 2 * i);
          put(i, 1, 2 * i + 1);
        }
        wave_lds();
#pragma unroll
        for (int i = 0; i < MB; ++i) {
          store(g.gu, g.ldgu, i, 2 * i);
          store(gu2, g.ldgu, i, 2 * i + 1);
        }
        wave_lds();
      }
      if (g.C) {
#pragma unroll
        for (int i = 0; i < MB; ++i)
          Out::put([&](int nb, int r) __attribute__((always_inline)) {
            const float x = acc[i][nb][r];
            return x * gate(x).s * acc[i][NBH + nb][r];
          }, buf + i * Out::kBytes);
        wave_lds();
#pragma unroll
        for (int i = 0; i < MB; ++i) store(g.C, g.ldc, i, i);
      }
    } else {
      // dy first, all of it; then y, dg and du of one band after the other
      using In = BandIn<NBH>;
      static_assert(MB * In::kBytes + 3 * Out::kBytes <= kRegion, "the bands exceed a wave's part of the slots");
      uint8_t* const dys = buf + 3 * Out::kBytes;
      In in[MB];
#pragma unroll
      for (int i = 0; i < MB; ++i) in[i].load(g.dy, g.lddy, row0 + 32 * i, col0, g.M, g.N);
#pragma unroll
      for (int i = 0; i < MB; ++i) in[i].put(dys + i * In::kBytes);
      wave_lds();
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        u32x2 dy[NBH][4];
        In::spread(dy, dys + i * In::kBytes);
        if (g.C)
          Out::put([&](int nb, int r) __attribute__((always_inline)) {
            const float x = acc[i][nb][r];
            return x * gate(x).s * acc[i][NBH + nb][r];
          }, buf + 2 * Out::kBytes);
        // dg = dy s u (1 + g (1 - s)) and du = dy s g in place of g and u
#pragma unroll
        for (int nb = 0; nb < NBH; ++nb)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const float x = acc[i][nb][r], u = acc[i][NBH + nb][r];
            const Gate q = gate(x);
            const float ds = from16<ET>(dy[nb][r >> 2][(r & 3) >> 1] >> (16 * (r & 1)) & 0xffffu) * q.s;
            acc[i][nb][r] = ds * u * (1.0f + x * q.om);
            acc[i][NBH + nb][r] = ds * x;
          }
        put(i, 0, 0);
        put(i, 1, 1);
        wave_lds();
        if (g.C) store(g.C, g.ldc, i, 2);
        store(g.gu, g.ldgu, i, 0);
        store(gu2, g.ldgu, i, 1);
        wave_lds();
      }
    }
  }
}

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
// addresses: 1 x 4097 x 14336 106 us, so 64 (56 since ld16_part's loads overlap; 73
// with weights that no cache holds).
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

// 16 tokens and 16 features a block; its waves share the summed
// dimension, 64 elements a wave and turn, straight from memory into the 16x16x32
// instruction's operands (weights as rows, tokens as columns: lane l holds row l %
// 16 and elements 8 (l / 16) .. + 7), and join their sums in LDS.  16 waves a block
// keep 64 KB of weights a CU in flight: 1 x 4096 x 14336 BF16 43 us = 5.5 TB/s (8
// waves with 128 elements a turn: 46), 1 x 5120 x 20480 72 us = 5.8 TB/s (81).
//
// WHOLE: every row is whole 16-byte pieces.
template <int ET, int OUT, bool WHOLE>
__global__ __launch_bounds__(kFewWaves * 64) void gate_few(ProductArgs g) {
  __shared__ float part[kFewWaves][2][4][64];
  const int lane = threadIdx.x & 63, wave = wave_id(), q = lane >> 4, i16 = lane & 15;
  const int64_t f0 = static_cast<int64_t>(blockIdx.x) * 16, m0 = static_cast<int64_t>(blockIdx.y) * 16;
  const int64_t f = f0 + i16 < g.N ? f0 + i16 : g.N - 1, m = m0 + i16 < g.M ? m0 + i16 : g.M - 1;
  const uint16_t* w = static_cast<const uint16_t*>(g.B) + 8 * q;
  const uint16_t* const px = static_cast<const uint16_t*>(g.A) + m * g.lda + 8 * q;
  const uint16_t* const pw[2] = {w + f * g.ldb, w + (g.N + f) * g.ldb};
  f32x4 acc[2] = {};
  auto load = [&](Piece& v, const uint16_t* p) __attribute__((always_inline)) {
    if constexpr (WHOLE) v.w = ld16(p);
    else v.load(p);
  };
  // (a turn's start is even: a row's pieces are all odd or all even)
  auto value = [&](const Piece& v, const uint16_t* p) __attribute__((always_inline)) {
    if constexpr (WHOLE) return v.w;
    else return v.shifted(8 * Piece::odd(p));
  };
  int64_t k = wave * kFewTurn;
  for (; k + kFewTurn <= g.K; k += kFewWaves * kFewTurn) {
    constexpr int kC = kFewTurn / 32;
    Piece a[2][kC], b[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      load(a[0][c], pw[0] + k + 32 * c);
      load(a[1][c], pw[1] + k + 32 * c);
      load(b[c], px + k + 32 * c);
    }
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
  const int64_t row = m0 + tok, col = f0 + fl;
  if (threadIdx.x >= 256 || col >= g.N || row >= g.M) return;
  float a = 0.0f, u = 0.0f;
#pragma unroll
  for (int v = 0; v < kFewWaves; ++v) {
    a += part[v][0][fl % 4][at];
    u += part[v][1][fl % 4][at];
  }
  const Gate s = gate(a);
  if (g.C) static_cast<uint16_t*>(g.C)[row * g.ldc + col] = static_cast<uint16_t>(to16<ET>(a * s.s * u));
  if constexpr (OUT == kOutGrad) {
    const float ds = from16<ET>(static_cast<const uint16_t*>(g.dy)[row * g.lddy + col]) * s.s;
    const float dg = ds * u * (1.0f + a * s.om);
    u = ds * a;
    a = dg;
  }
  if (g.gu) {
    uint16_t* p = static_cast<uint16_t*>(g.gu) + row * g.ldgu + col;
    p[0] = static_cast<uint16_t>(to16<ET>(a));
    p[g.N] = static_cast<uint16_t>(to16<ET>(u));
  }
}

// Both projections with their gate.  1000 x 4096 x 14336 BF16 188 to 200 us (1.18 to 1.25 PFLOP/s),
// 33 x 5120 x 20480 92 us (4.6 TB/s of weights; 320 tiles of 128 x 128).
template <int ET, int OUT, int MB, int NB, int D, bool FAST>
__global__ __launch_bounds__(256, MB * NB > 8 || D > 2 ? 1 : 2) void gate_tiles(ProductArgs g) {
  __shared__ __align__(16) uint8_t smem[lds_bytes(MB, NB, D)];
  product<ET, true, true, OUT, MB, NB, D, FAST>(g, blockIdx.x, 0, smem);
}

// The two gradient products in one launch, that of the longer sums first: the
// blocks of one fill what the other leaves of the machine (8192 x 4096 x 14336 BF16,
// both 256 x 256: 2850 us for 3.85 TFLOP).  nx: blocks of dx.
template <int ET, int MB, int NB, bool FAST>
__global__ __launch_bounds__(256, MB * NB > 8 ? 1 : 2) void gradient_tiles(ProductArgs gx, ProductArgs gw, uint32_t nx, uint32_t nw, int dx_first) {
  __shared__ __align__(16) uint8_t smem[lds_bytes(MB, NB, 2)];
  const uint32_t before = dx_first ? nx : nw;
  const bool first = blockIdx.x < before, is_dx = first == (dx_first != 0);
  const uint32_t b = first ? blockIdx.x : blockIdx.x - before;
  if (is_dx) {
    const uint32_t tiles = nx / gx.splits;
    product<ET, true, false, kOutC, MB, NB, 2, FAST>(gx, b % tiles, b / tiles, smem);
  } else {
    const uint32_t tiles = nw / gw.splits;
    product<ET, false, false, kOutC, MB, NB, 2, FAST>(gw, b % tiles, b / tiles, smem);
  }
}

// ---- which tile ------------------------------------------------------------

// Operands that the direct loads take: 16-byte rows, windows below 2 GiB and,
// where outputs are contiguous, a whole number of 16-byte pieces of them.
inline bool direct_operand(const void* p, int64_t ld, bool kc, int64_t outs) {
  return aligned(p, 16) && ld % 8 == 0 && ld < (int64_t(1) << 30) / (kc ? 256 : 64) && (kc || outs % 8 == 0);
}

template <int ET, int OUT>
hipError_t launch_gate(const ProductArgs& g, hipStream_t s) {
  const bool fast = direct_operand(g.A, g.lda, true, g.M) && direct_operand(g.B, g.ldb, true, g.N);
  const GateForm form = gate_form(g.M, g.N, g.K, fast, OUT == kOutGrad);
  const dim3 grid(static_cast<unsigned>(tiles_of(g.M, 2 * g.N, form == kLarge ? 256 : 128)));
  switch (form) {
    case kFew: {
      const dim3 groups(static_cast<unsigned>(ceil_div(g.N, 16)), static_cast<unsigned>(ceil_div(g.M, 16)));
      const bool whole = aligned(g.A, 16) && aligned(g.B, 16) && g.lda % 8 == 0 && g.ldb % 8 == 0;
      if (whole) gate_few<ET, OUT, true><<<groups, kFewWaves * 64, 0, s>>>(g);
      else gate_few<ET, OUT, false><<<groups, kFewWaves * 64, 0, s>>>(g);
      break;
    }
    case kLarge: gate_tiles<ET, OUT, 4, 4, 2, true><<<grid, 256, 0, s>>>(g); break;
    case kRing: gate_tiles<ET, OUT, 2, 2, 4, true><<<grid, 256, 0, s>>>(g); break;
    case kSmall: gate_tiles<ET, OUT, 2, 2, 2, true><<<grid, 256, 0, s>>>(g); break;
    case kStaged: gate_tiles<ET, OUT, 2, 2, 2, false><<<grid, 256, 0, s>>>(g); break;
  }
  return hipGetLastError();
}

}  // namespace
}  // namespace amp
