// Matrix-core pieces shared by the GEMM translation units: operand fragments,
// the swizzled LDS stage and direct-to-LDS loads.
#pragma once
#include "common.hpp"

namespace amp {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kRowBytes = 128;                       // LDS bytes per tile row per K-step

__device__ __forceinline__ int swz(int row, int chunk) {
  return row * kRowBytes + ((chunk ^ ((row ^ (row >> 3)) & 7)) << 4);
}

__device__ __forceinline__ u32x4 ld16(const void* p) { return *static_cast<const u32x4*>(p); }

// The wave's index in its block.  It is the same for every lane, but the
// compiler cannot tell from threadIdx; taken through readfirstlane it lives
// in a scalar register, so buffer-load scalar offsets and LDS bases derived
// from it need no per-lane (waterfall) loop.
__device__ __forceinline__ int wave_id() {
  return __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
}

typedef __attribute__((address_space(3))) void lds_void;

// One 16-byte-per-lane direct-to-LDS load (64 lanes fill 1 KB at dst).  With
// ASM set it is written as inline assembly: the compiler then does not track
// it as a pending LDS write.  It has to be kept from tracking it where the
// transposing LDS reads follow: those reads carry no alias information, so
// the compiler would make the first of them wait for every load in flight,
// exposing the whole global-load latency in each K-step.  Every caller makes
// the loads land before their destination is read (s_waitcnt vmcnt(0), then
// a block barrier), which is the ordering the compiler would otherwise add.
template <bool ASM>
__device__ __forceinline__ void d2l16(__amdgpu_buffer_rsrc_t rsrc, uint8_t* dst, uint32_t voff,
                                      uint32_t soff) {
  if constexpr (ASM) {
    const uint32_t m0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_void*)dst));
    asm volatile("buffer_load_dwordx4 %0, %1, %2 offen lds" ::"v"(voff), "s"(rsrc), "s"(soff), "{m0}"(m0)
                 : "memory");
  } else {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void*)dst, 16, voff, soff, 0, 0);
  }
}

typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4i16 lds_v4i16;

// MFMA 32x32x16 operand fragment (lane l: row l%32 of the 32-block, K
// 8*(l/32) .. +7) from an M/N-contiguous stage with two transposing 64-bit
// reads.  ds_read_b64_tr_b16 hands lane i of a 16-lane group element i%4 of
// the 64 bits read by lane 4j + i/4, j = 0..3; so source lane s of group q
// reads the 4 columns 16*(q%2) + 4*(s%4) .. +3 of K-row 8*(q/2) + s/4 (+4 for
// the second read) and every lane receives its own column's 4 K values.
// PITCH: LDS bytes of a K-row.  addr: this lane's byte address for (32-block, K-slice 0, first read);
// slice ks adds 16*ks rows, the second read 4 rows.
template <int PITCH = 512>
__device__ __forceinline__ u32x4 frag_tr(const uint8_t* stage, uint32_t addr, int ks) {
  const uint8_t* p = stage + addr + ks * 16 * PITCH;
  const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (lds_v4i16*)((__attribute__((address_space(3))) uint8_t*)(__attribute__((address_space(3))) void*)p));
  const v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (lds_v4i16*)((__attribute__((address_space(3))) uint8_t*)(__attribute__((address_space(3))) void*)(p + 4 * PITCH)));
  const u32x2 l2 = __builtin_bit_cast(u32x2, lo), h2 = __builtin_bit_cast(u32x2, hi);
  return u32x4{l2[0], l2[1], h2[0], h2[1]};
}

}  // namespace
}  // namespace amp
