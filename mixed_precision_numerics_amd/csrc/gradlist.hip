// Global gradient norm and clipping over a list of tensors (gfx950).
//
//   sumsq = sum_t sum_i (f32(g_t[i]) / S)^2,  coef = min(1, max_norm / (norm + 1e-6))
//   out_t[i] = round(f32(g_t[i]) / S * coef)
//
// HBM-bound: the norm of 0.87 G BF16 elements 293 us (5.95 TB/s), their clipping into
// FP32 1.01 ms (5.2 TB/s); lists of small tensors are bound by launches and by the
// host: the norm of a small net's four tensors 10.6 us, clipping 700 of 2000 elements
// on average 60 us (27 from C).  The list's tensors are cut into chunks, none across
// two tensors, and the chunks dealt out evenly to the blocks in one contiguous run
// each, whatever the tensors' lengths.  The tables travel as kernel arguments:
// nothing is allocated or copied, and a captured graph holds them.
#include "common.hpp"
#include "formats.hpp"

namespace amp {
namespace {

constexpr int kListThreads = 512;
constexpr int kNormTensors = 192, kClipTensors = 128;   // tables of one launch (below 4 KB of arguments)

// n and the types of a table's tensor share a word.
constexpr int kLenBits = 48;
__host__ __device__ inline int64_t length_of(uint64_t nt) { return static_cast<int64_t>(nt & ((uint64_t(1) << kLenBits) - 1)); }

struct NormTable {
  const void* p[kNormTensors];
  uint64_t nt[kNormTensors];      // elements, type << 48
  uint32_t end[kNormTensors];     // chunks up to and with this tensor
  int32_t count;
  uint32_t chunk;                 // elements
};

struct ClipTable {
  const void* p[kClipTensors];
  void* o[kClipTensors];
  uint64_t nt[kClipTensors];      // elements, type << 48, output's type << 56
  uint32_t end[kClipTensors];
  int32_t count;
  uint32_t chunk;
};

// The tensor that holds chunk c: how many tensors end at or before it.  Every
// wave looks at the whole table at once.
template <int N>
__device__ __forceinline__ int tensor_of(const uint32_t (&end)[N], int count, uint32_t c) {
  int t = 0;
#pragma unroll
  for (int i = 0; i < N; i += kWave) {
    const int at = i + static_cast<int>(threadIdx.x & (kWave - 1));
    t += __popcll(__ballot(at < count && end[at < N ? at : 0] <= c));
  }
  return __builtin_amdgcn_readfirstlane(t);
}

// 16 (8) bytes at any element's address.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));

template <int T>
__device__ __forceinline__ float one(const void* p, int64_t i) {
  if constexpr (T == AMP_F32) return static_cast<const float*>(p)[i];
  else if constexpr (T == AMP_BF16) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  else return f16_to_f32(static_cast<const uint16_t*>(p)[i]);
}

template <int T>
__device__ __forceinline__ void widen2(uint32_t w, float* x) {
  if constexpr (T == AMP_BF16) {
    x[0] = bitsf(w << 16);
    x[1] = bitsf(w & 0xffff0000u);
  } else {
    x[0] = f16_to_f32(w & 0xffffu);
    x[1] = f16_to_f32(w >> 16);
  }
}

// E consecutive elements (E elements are 8 or 16 bytes).
template <int T, int E>
__device__ __forceinline__ void several(const void* p, int64_t i, float (&x)[E]) {
  if constexpr (T == AMP_F32) {
    static_assert(E == 4, "16 bytes");
    const u32x4 w = *reinterpret_cast<const u32x4_any*>(static_cast<const float*>(p) + i);
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = bitsf(w[k]);
  } else if constexpr (E == 8) {
    const u32x4 w = *reinterpret_cast<const u32x4_any*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int k = 0; k < 4; ++k) widen2<T>(w[k], x + 2 * k);
  } else {
    const u32x2 w = *reinterpret_cast<const u32x2_any*>(static_cast<const uint16_t*>(p) + i);
    widen2<T>(w[0], x);
    widen2<T>(w[1], x + 2);
  }
}

struct Sum {
  double a[4] = {0.0, 0.0, 0.0, 0.0};   // independent chains, joined in a fixed order
  uint32_t bad = 0;
  __device__ __forceinline__ void add(float x, int c) {
    const uint32_t fin = static_cast<uint32_t>((fbits(x) & 0x7f800000u) != 0x7f800000u);
    bad |= fin ^ 1u;
    const double d = fin ? static_cast<double>(x) : 0.0;
    a[c] = __builtin_fma(d, d, a[c]);
  }
};

template <int T>
__device__ __forceinline__ void sum_range(const void* p, int64_t e0, int64_t e1, Sum& s) {
  constexpr int E = T == AMP_F32 ? 4 : 8, kStep = kListThreads * E;
  int64_t e = e0 + threadIdx.x * E;
  for (; e + 3 * kStep + E <= e1; e += 4 * kStep) {
    float x[4][E];
#pragma unroll
    for (int u = 0; u < 4; ++u) several<T, E>(p, e + u * kStep, x[u]);
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int q = 0; q < E; ++q) s.add(x[u][q], q & 3);
  }
  for (; e + E <= e1; e += kStep) {
    float x[E];
    several<T, E>(p, e, x);
#pragma unroll
    for (int q = 0; q < E; ++q) s.add(x[q], q & 3);
  }
  for (int64_t i = e; i < e1 && i < e + E; ++i) s.add(one<T>(p, i), 0);
}

__global__ __launch_bounds__(kListThreads) void norm_list_kernel(const NormTable tab, amp_scaler_state* __restrict__ st,
                                                                 double* __restrict__ partial) {
  __shared__ double red[kListThreads / kWave];
  __shared__ uint32_t bad_any;
  if (threadIdx.x == 0) bad_any = 0;
  const uint32_t chunks = tab.end[tab.count - 1];
  uint32_t c = static_cast<uint32_t>(static_cast<uint64_t>(chunks) * blockIdx.x / gridDim.x);
  const uint32_t c1 = static_cast<uint32_t>(static_cast<uint64_t>(chunks) * (blockIdx.x + 1) / gridDim.x);
  Sum s;
  for (int t = tensor_of(tab.end, tab.count, c); c < c1; ++t) {
    const uint32_t begin = t ? tab.end[t - 1] : 0u, end = tab.end[t], stop = end < c1 ? end : c1;
    if (stop <= c) continue;              // an empty tensor
    const int64_t n = length_of(tab.nt[t]), e0 = static_cast<int64_t>(c - begin) * tab.chunk;
    const int64_t e1 = static_cast<int64_t>(stop - begin) * tab.chunk < n ? static_cast<int64_t>(stop - begin) * tab.chunk : n;
    switch (tab.nt[t] >> kLenBits) {
      case AMP_F32: sum_range<AMP_F32>(tab.p[t], e0, e1, s); break;
      case AMP_BF16: sum_range<AMP_BF16>(tab.p[t], e0, e1, s); break;
      default: sum_range<AMP_F16>(tab.p[t], e0, e1, s); break;
    }
    c = stop;
  }
  double v = (s.a[0] + s.a[1]) + (s.a[2] + s.a[3]);
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
  __syncthreads();
  if (s.bad) bad_any = 1u;
  if ((threadIdx.x & (kWave - 1)) == 0) red[threadIdx.x / kWave] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    double sum = 0.0;
    for (int w = 0; w < kListThreads / kWave; ++w) sum += red[w];
    partial[blockIdx.x] = sum;
    if (bad_any) st->found_inf = 1;
  }
}

// The partial sums in a fixed order, the sum's scaling by 1/S^2 and the clip
// coefficient.  All latency: every load is on its way before the first is used
// (1024 sums by one wave, one after the other: 7.7 us instead of 4.0).
constexpr int kFinishThreads = 256;
__global__ __launch_bounds__(kFinishThreads) void norm_list_finish(const double* __restrict__ partial, int nb, int first,
                                                                   double* __restrict__ sumsq, const amp_scaler_state* st, float max_norm,
                                                                   float* out) {
  __shared__ double red[kFinishThreads / kWave];
  constexpr int kEach = AMP_NORM_PARTIALS / kFinishThreads;
  static_assert(kEach * kFinishThreads == AMP_NORM_PARTIALS, "every partial sum has a thread");
  double each[kEach], v = 0.0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int b = i * kFinishThreads + threadIdx.x;
    each[i] = b < nb ? partial[b] : 0.0;
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) v += each[i];
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
  if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave] = v;
  __syncthreads();
  if (threadIdx.x != 0) return;
  v = 0.0;
  for (int w = 0; w < kFinishThreads / kWave; ++w) v += red[w];
  const double inv = static_cast<double>(1.0f / st->scale);
  v = (first ? 0.0 : *sumsq) + v * inv * inv;
  *sumsq = v;
  if (!out) return;
  if (st->found_inf) {
    out[0] = 1.0f;
    out[1] = __builtin_inff();
    return;
  }
  const float norm = static_cast<float>(__builtin_sqrt(v));
  const float c = max_norm / (norm + 1e-6f);
  out[0] = c < 1.0f ? c : 1.0f;
  out[1] = norm;
}

template <int T>
__device__ __forceinline__ void put_one(void* p, int64_t i, float x) {
  if constexpr (T == AMP_F32) static_cast<float*>(p)[i] = x;
  else static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(T == AMP_BF16 ? f32_to_bf16(x) : f32_to_f16(x));
}

template <int T, int E>
__device__ __forceinline__ void put_several(void* p, int64_t i, const float (&x)[E]) {
  if constexpr (T == AMP_F32) {
    *reinterpret_cast<u32x4_any*>(static_cast<float*>(p) + i) = u32x4{fbits(x[0]), fbits(x[1]), fbits(x[2]), fbits(x[3])};
  } else {
    uint32_t w[E / 2];
#pragma unroll
    for (int k = 0; k < E / 2; ++k)
      w[k] = T == AMP_BF16 ? f32_to_bf16(x[2 * k]) | f32_to_bf16(x[2 * k + 1]) << 16
                           : f32_to_f16(x[2 * k]) | f32_to_f16(x[2 * k + 1]) << 16;
    uint16_t* q = static_cast<uint16_t*>(p) + i;
    if constexpr (E == 8) *reinterpret_cast<u32x4_any*>(q) = u32x4{w[0], w[1], w[2], w[3]};
    else *reinterpret_cast<u32x2_any*>(q) = u32x2{w[0], w[1]};
  }
}

// The product as the FP32 number that it is: a product whose one use is a
// conversion to FP16 becomes one instruction that rounds once, past FP32.
__device__ __forceinline__ float times(float x, float inv, float coef) {
  float v = (x * inv) * coef;
  asm("" : "+v"(v));
  return v;
}

// Lanes take 16 bytes of the wider side, so that each instruction covers one
// contiguous span on both.
template <int T, int O>
__device__ __forceinline__ void clip_range(const void* p, void* o, int64_t e0, int64_t e1, float inv, float coef) {
  constexpr int E = T == AMP_F32 || O == AMP_F32 ? 4 : 8, kStep = kListThreads * E;
  int64_t e = e0 + threadIdx.x * E;
  for (; e + 3 * kStep + E <= e1; e += 4 * kStep) {
    float x[4][E];
#pragma unroll
    for (int u = 0; u < 4; ++u) several<T, E>(p, e + u * kStep, x[u]);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
#pragma unroll
      for (int q = 0; q < E; ++q) x[u][q] = times(x[u][q], inv, coef);
      put_several<O, E>(o, e + u * kStep, x[u]);
    }
  }
  for (; e + E <= e1; e += kStep) {
    float x[E];
    several<T, E>(p, e, x);
#pragma unroll
    for (int q = 0; q < E; ++q) x[q] = times(x[q], inv, coef);
    put_several<O, E>(o, e, x);
  }
  for (int64_t i = e; i < e1 && i < e + E; ++i) put_one<O>(o, i, times(one<T>(p, i), inv, coef));
}

template <int T>
__device__ __forceinline__ void clip_to(int ot, const void* p, void* o, int64_t e0, int64_t e1, float inv, float coef) {
  switch (ot) {
    case AMP_F32: clip_range<T, AMP_F32>(p, o, e0, e1, inv, coef); break;
    case AMP_BF16: clip_range<T, AMP_BF16>(p, o, e0, e1, inv, coef); break;
    default: clip_range<T, AMP_F16>(p, o, e0, e1, inv, coef); break;
  }
}

__global__ __launch_bounds__(kListThreads) void clip_list_kernel(const ClipTable tab, const amp_scaler_state* __restrict__ st,
                                                                 const float* __restrict__ d_coef) {
  const float inv = st ? 1.0f / st->scale : 1.0f, coef = d_coef ? *d_coef : 1.0f;
  const bool same = inv == 1.0f && coef == 1.0f;
  const uint32_t chunks = tab.end[tab.count - 1];
  uint32_t c = static_cast<uint32_t>(static_cast<uint64_t>(chunks) * blockIdx.x / gridDim.x);
  const uint32_t c1 = static_cast<uint32_t>(static_cast<uint64_t>(chunks) * (blockIdx.x + 1) / gridDim.x);
  for (int t = tensor_of(tab.end, tab.count, c); c < c1; ++t) {
    const uint32_t begin = t ? tab.end[t - 1] : 0u, end = tab.end[t], stop = end < c1 ? end : c1;
    if (stop <= c) continue;
    const int64_t n = length_of(tab.nt[t]), e0 = static_cast<int64_t>(c - begin) * tab.chunk;
    const int64_t e1 = static_cast<int64_t>(stop - begin) * tab.chunk < n ? static_cast<int64_t>(stop - begin) * tab.chunk : n;
    const int it = static_cast<int>(tab.nt[t] >> kLenBits) & 0xff, ot = static_cast<int>(tab.nt[t] >> (kLenBits + 8));
    const void* p = tab.p[t];
    void* o = tab.o[t];
    c = stop;
    if (same && p == o) continue;         // in place, times one
    switch (it) {
      case AMP_F32: clip_to<AMP_F32>(ot, p, o, e0, e1, inv, coef); break;
      case AMP_BF16: clip_to<AMP_BF16>(ot, p, o, e0, e1, inv, coef); break;
      default: clip_to<AMP_F16>(ot, p, o, e0, e1, inv, coef); break;
    }
  }
}

// Elements of a chunk: a block's vectors once over for lists that would
// otherwise leave blocks without work, else four times (all its loads in
// flight), so that the runs that blocks get differ by little.
uint32_t chunk_of(int64_t total) { return total < int64_t(1024) * 16384 ? 4096u : 16384u; }

}  // namespace

hipError_t launch_grad_norm_list(const amp_tensor* grads, int32_t count, int first, amp_scaler_state* st, amp_grad_norm_state* ns,
                                 float max_norm, float* out, hipStream_t s) {
  int64_t total = 0;
  for (int32_t i = 0; i < count; ++i) total += grads[i].n;
  // One partial sum per block, shared out to the launches by their elements:
  // each has one at least, and AMP_LIST_TENSORS tensors are fewer launches than
  // there are partial sums.
  const int64_t launches = (count + kNormTensors - 1) / kNormTensors;
  static_assert((AMP_LIST_TENSORS + kNormTensors - 1) / kNormTensors < AMP_NORM_PARTIALS, "a partial sum for each launch");
  const uint32_t chunk = chunk_of(total);
  int nb = 0;
  for (int32_t i0 = 0; i0 < count; i0 += kNormTensors) {
    NormTable tab;
    tab.count = count - i0 < kNormTensors ? count - i0 : kNormTensors;
    tab.chunk = chunk;
    uint32_t end = 0;
    int64_t here = 0;
    for (int32_t i = 0; i < tab.count; ++i) {
      const amp_tensor& g = grads[i0 + i];
      end += static_cast<uint32_t>((g.n + chunk - 1) / chunk);
      here += g.n;
      tab.p[i] = g.p;
      tab.nt[i] = static_cast<uint64_t>(g.n) | static_cast<uint64_t>(g.type) << kLenBits;
      tab.end[i] = end;
    }
    if (end == 0) continue;
    int64_t blocks = 1 + static_cast<int64_t>(static_cast<double>(AMP_NORM_PARTIALS - launches) * (static_cast<double>(here) / static_cast<double>(total)));
    if (blocks > end) blocks = end;
    if (blocks > AMP_NORM_PARTIALS - nb) blocks = AMP_NORM_PARTIALS - nb;
    norm_list_kernel<<<static_cast<unsigned>(blocks), kListThreads, 0, s>>>(tab, st, ns->partial + nb);
    if (hipError_t e = hipGetLastError()) return e;
    nb += static_cast<int>(blocks);
  }
  norm_list_finish<<<1, kFinishThreads, 0, s>>>(ns->partial, nb, first, &ns->sumsq, st, max_norm, out);
  return hipGetLastError();
}

hipError_t launch_grad_clip_list(const amp_tensor* grads, const amp_tensor* outs, int32_t count, const amp_scaler_state* st,
                                 const float* coef, hipStream_t s) {
  int64_t total = 0;
  for (int32_t i = 0; i < count; ++i) total += grads[i].n;
  const uint32_t chunk = chunk_of(total);
  for (int32_t i0 = 0; i0 < count; i0 += kClipTensors) {
    ClipTable tab;
    tab.count = count - i0 < kClipTensors ? count - i0 : kClipTensors;
    tab.chunk = chunk;
    uint32_t end = 0;
    for (int32_t i = 0; i < tab.count; ++i) {
      const amp_tensor &g = grads[i0 + i], &o = outs[i0 + i];
      end += static_cast<uint32_t>((g.n + chunk - 1) / chunk);
      tab.p[i] = g.p;
      tab.o[i] = o.p;
      tab.nt[i] = static_cast<uint64_t>(g.n) | static_cast<uint64_t>(g.type) << kLenBits | static_cast<uint64_t>(o.type) << (kLenBits + 8);
      tab.end[i] = end;
    }
    if (end == 0) continue;
    clip_list_kernel<<<end < 8192u ? end : 8192u, kListThreads, 0, s>>>(tab, st, coef);
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace amp
