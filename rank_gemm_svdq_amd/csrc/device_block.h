// Shared by the kernels of the operators around the layer (norm, FP8 linear,
// rotary positions, attention): vector types, the two 16-bit value types and
// the host-side checks.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "host_internal.h"

namespace svdq {
namespace {

typedef int b4i __attribute__((ext_vector_type(4)));
typedef float b2f __attribute__((ext_vector_type(2)));
typedef float b4f __attribute__((ext_vector_type(4)));
typedef float b16f __attribute__((ext_vector_type(16)));
typedef __bf16 b8bf __attribute__((ext_vector_type(8)));
typedef __bf16 b2bf __attribute__((ext_vector_type(2)));
typedef _Float16 b8h __attribute__((ext_vector_type(8)));
typedef _Float16 b2h __attribute__((ext_vector_type(2)));

// DT: SVDQ_BF16 or SVDQ_FP16.  Two packed 16-bit values <-> two floats; the
// narrowing rounds to nearest even (NaN stays NaN).
template <int DT>
__device__ __forceinline__ b2f widen2(uint32_t w) {
  if constexpr (DT == SVDQ_BF16) {
    return (b2f){__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)};
  } else {
    return __builtin_convertvector(__builtin_bit_cast(b2h, w), b2f);
  }
}
template <int DT>
__device__ __forceinline__ uint32_t narrow2(float a, float b) {
  if constexpr (DT == SVDQ_BF16)
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((b2f){a, b}, b2bf));
  else
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((b2f){a, b}, b2h));
}
template <int DT>
__device__ __forceinline__ void widen8(const b4i& v, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const b2f t = widen2<DT>((uint32_t)v[i]);
    f[2 * i] = t[0];
    f[2 * i + 1] = t[1];
  }
}
template <int DT>
__device__ __forceinline__ b4i narrow8(const float* f) {
  b4i v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = (int)narrow2<DT>(f[2 * i], f[2 * i + 1]);
  return v;
}

#define SVDQ_LDS __attribute__((address_space(3)))

// One wave-wide 1 KB direct-to-LDS copy: lane i's 16 bytes at base + off
// (base wave-uniform, off per lane) land at LDS byte lds + 16 i; inactive
// lanes copy nothing.  Issued from asm so that the compiler does not serialise
// it against unrelated LDS reads: completion is waited for explicitly
// (dma_wait).  Callers keep base and off ready: the scalar arithmetic of
// addresses worked out copy by copy costs more than the copies do.  The load
// needs one wait state after the write of M0.
__device__ __forceinline__ void dma_16(const uint8_t* base, uint32_t off, uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, %2"
      :
      : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(off), "s"(base)
      : "memory", "m0");
}
// The same with 4 bytes a lane (256 bytes).
__device__ __forceinline__ void dma_4(const uint8_t* base, uint32_t off, uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dword %1, %2"
      :
      : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(off), "s"(base)
      : "memory", "m0");
}
__device__ __forceinline__ void dma_wait() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
__device__ __forceinline__ uint32_t lds_address(const void* p) { return (uint32_t)(size_t)(SVDQ_LDS const uint8_t*)p; }

// Blocks are dealt to the 8 XCDs round robin.  xcd_order() maps the block
// index so that each XCD gets one contiguous run of work ids, whose operands
// then share its L2.
__device__ __forceinline__ int xcd_order(int b, int total) {
  const int q = total >> 3, r = total & 7, x = b & 7;
  return x * q + min(x, r) + (b >> 3);
}

// Compute units, for the choice of variants on the host: those of a whole gfx950,
// not the current device's count, as workspace sizes follow from these choices and
// are asked for without a device.
constexpr int kCus = 256;

inline bool on16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
inline bool on4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
inline bool is_dtype(int32_t d) { return d == SVDQ_BF16 || d == SVDQ_FP16; }
inline svdq_status launched() { return hipGetLastError() == hipSuccess ? SVDQ_OK : SVDQ_ERR_DEVICE; }

}  // namespace
}  // namespace svdq
