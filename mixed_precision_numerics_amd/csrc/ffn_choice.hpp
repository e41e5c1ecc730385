// Which kernel and which tiles a call of the gated feed-forward block takes, from
// its sizes alone.  Plain C++: tests ask it without a GPU, so that a shape which is
// meant for one kernel is known to reach it.
#pragma once
#include <algorithm>
#include <cstdint>

namespace amp {
namespace {

constexpr int kStepK = 64;                         // elements of a step along the summed dimension
constexpr int kFewWaves = 16, kFewTurn = 64;       // gate_few: waves of a block, elements of a wave's turn

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t tiles_of(int64_t M, int64_t cols, int64_t edge) { return ceil_div(M, edge) * ceil_div(cols, edge); }

// Microseconds of a step of 64 along the summed dimension: a tile of 256 x 256
// has a CU for itself, tiles of 128 x 128 run two to a CU; with fewer than one a
// CU a step of theirs is bound by latency, less with a longer ring.
constexpr double kStepLarge = 1.5, kStepSmall = 1.05, kStepAlone = 0.55, kStepFar = 0.4;
// Of a tile's beginning and end, of the gate and of its gradient.
constexpr double kGateLarge = 11.0, kGateSmall = 6.0, kGradLarge = 25.0, kGradSmall = 8.0;
// Of a turn of gate_few's waves, of which two blocks share a CU, and its ends; and
// the weights' bytes a microsecond.
constexpr double kTurnFew = 2.0, kBlockFew = 3.0, kStream = 5.0e6;

// kFew: gate_few.  Else tiles: kLarge of 256 x 256, kRing of 128 x 128 with a ring of
// four steps, kSmall of 128 x 128, kStaged the same through registers.
enum GateForm : int { kFew = 0, kLarge = 1, kRing = 2, kSmall = 3, kStaged = 4 };

// M tokens, N features, K summed; fast: operands that the direct loads take;
// gradient: with the gate's backward pass in the epilogue.
inline GateForm gate_form(int64_t M, int64_t N, int64_t K, bool fast, bool gradient) {
  const int64_t big = tiles_of(M, 2 * N, 256), small = tiles_of(M, 2 * N, 128), steps = ceil_div(K, kStepK);
  const double large_ends = gradient ? kGradLarge : kGateLarge, small_ends = gradient ? kGradSmall : kGateSmall;
  const double t_large = static_cast<double>(ceil_div(big, 256)) * (kStepLarge * steps + large_ends);
  const double t_small = small <= 256 ? (fast ? kStepFar : 2 * kStepAlone) * steps + small_ends
                                      : static_cast<double>(ceil_div(small, 512)) * (kStepSmall * steps + small_ends);
  const int64_t groups = ceil_div(M, 16), few = groups * ceil_div(N, 16);
  const double weights = 4.0 * static_cast<double>(N) * static_cast<double>(K) / kStream;
  const double t_few = std::max(static_cast<double>(ceil_div(few, 512)) * (kTurnFew * ceil_div(K, kFewWaves * kFewTurn) + kBlockFew),
                                static_cast<double>(groups) * weights);
  // (a launch counts fewer than 2^32 threads)
  if (few < (int64_t(1) << 22) && (groups == 1 || (groups <= 8 && small <= 256 && t_few < std::max(t_small, weights)))) return kFew;
  if (!fast) return kStaged;
  if (t_large <= t_small) return kLarge;
  // up to one block a CU a ring of four steps, 144 KB, keeps more of the weights in
  // flight (65 x 4096 x 14336 BF16 64 -> 52 us, weights from memory)
  return small <= 256 ? kRing : kSmall;
}

// Parts of a product [M, N] over K whose tiles are too few for the machine: about
// `steps` steps each where that at least halves them, their sums within `room`
// numbers of the work area.
inline int parts_of(int64_t M, int64_t N, int64_t K, int64_t steps, int64_t room) {
  const int64_t all = ceil_div(K, kStepK);
  int64_t n = all >= 2 * steps ? all / steps : 1;
  if (M * N > 0 && n > room / (M * N)) n = room / (M * N);
  return n > 1 ? static_cast<int>(n) : 1;
}

// Of the two gradient products, dx [mx, nx] over kx and dw [mw, nw] over kw (one
// that is absent has mx == 0 or mw == 0): tiles of 256 x 256 (wide) or 128 x 128, the
// parts of each, and which product's blocks come first.
struct GradientForm {
  bool wide, dx_first;
  int split_x, split_w;
};
inline GradientForm gradient_form(int64_t mx, int64_t nx, int64_t kx, int64_t mw, int64_t nw, int64_t kw, bool fast, int64_t room) {
  const bool dx = mx > 0 && nx > 0, dw = mw > 0 && nw > 0;
  const int64_t sx = ceil_div(kx, kStepK), sw = ceil_div(kw, kStepK);
  const int64_t tx = tiles_of(mx, nx, 128), tw = tiles_of(mw, nw, 128), bx = tiles_of(mx, nx, 256), bw = tiles_of(mw, nw, 256);
  // 128 x 128 tiles, in parts that share the work out to two blocks a CU
  const int64_t even = (tx * sx + tw * sw) / 512, each = even < 8 ? 8 : even;
  GradientForm f{};
  f.split_x = dx ? parts_of(mx, nx, kx, each, room) : 1;
  f.split_w = dw ? parts_of(mw, nw, kw, each, room - (f.split_x > 1 ? f.split_x * mx * nx : 0)) : 1;
  const double longest = std::max(dx ? static_cast<double>(sx) / f.split_x : 0.0, dw ? static_cast<double>(sw) / f.split_w : 0.0);
  const double small = std::max(kStepSmall * static_cast<double>(tx * sx + tw * sw) / 512, kStepAlone * longest);
  const double large = kStepLarge * std::max(static_cast<double>(bx * sx + bw * sw) / 256, static_cast<double>(std::max(dx ? sx : 0, dw ? sw : 0)));
  f.wide = fast && large <= small;
  if (f.wide) f.split_x = f.split_w = 1;
  f.dx_first = sx * f.split_w >= sw * f.split_x;
  return f;
}

}  // namespace
}  // namespace amp
