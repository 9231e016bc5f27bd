// Operand fragments of the 16-bit matrix instructions (bf16 and fp16 in, fp32
// out) and loads of eight 16-bit values from rows of any alignment.
//
// v_mfma_f32_16x16x32: lane l of the first operand holds row l % 16, entries
// k = 8 (l / 16) + j (j = 0..7) of the 32; the second operand holds column
// l % 16 in the same way; the result D[i][j] is in lane j + 16 (i / 4),
// register i % 4.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"

namespace externd {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

template <bool BF>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ float bf16_to_f32(uint32_t lo16) { return __uint_as_float(lo16 << 16); }
// Nearest bf16, ties to even; NaN stays NaN.
__device__ __forceinline__ uint32_t f32_to_bf16(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }
template <bool BF>
__device__ __forceinline__ uint32_t f32_to_16(float f) {
  if constexpr (BF) return f32_to_bf16(f);
  else return __builtin_bit_cast(uint16_t, (_Float16)f);
}
template <bool BF>
__device__ __forceinline__ float f32_from_16(uint32_t lo16) {
  if constexpr (BF) return bf16_to_f32(lo16);
  else return (float)__builtin_bit_cast(_Float16, (uint16_t)lo16);
}

// Eight 16-bit values starting at p, in order.  AL: p is 16-byte aligned.
// Otherwise p is only 2-byte aligned: the dwords that hold the 16 bytes are
// read (five of them when p is odd in halves; only dwords that hold one of
// the eight values are touched) and shifted into place.
template <bool AL>
__device__ __forceinline__ u32x4 load8(const uint16_t* p) {
  if constexpr (AL) {
    return *reinterpret_cast<const u32x4*>(p);
  } else {
    const uint32_t odd = (uint32_t)(reinterpret_cast<uintptr_t>(p) >> 1) & 1u;
    const uint16_t* q = p - odd;
    const u32x4_a4 v = *reinterpret_cast<const u32x4_a4*>(q);
    const uint32_t w = *reinterpret_cast<const uint32_t*>(q + (odd ? 8 : 6));
    const uint32_t sh = odd * 16u;
    u32x4 r;
    r.x = __builtin_amdgcn_alignbit(v.y, v.x, sh);
    r.y = __builtin_amdgcn_alignbit(v.z, v.y, sh);
    r.z = __builtin_amdgcn_alignbit(v.w, v.z, sh);
    r.w = __builtin_amdgcn_alignbit(w, v.w, sh);
    return r;
  }
}

// Loads written before stay before, uses written after stay after: the loads are in
// flight together.  (Left to itself the compiler waits for each of a fragment's narrow
// loads before it makes the next, or gives each a branch.)
__device__ __forceinline__ void loads_made() { asm volatile("" ::: "memory"); }

// Eight 16-bit values into a fragment; those outside first .. end - 1 are 0.
__device__ __forceinline__ u32x4 pack8(const uint16_t (&v)[8], int64_t first, int64_t end) {
  u32x4 r = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int j = 0; j < 8; ++j) r[j / 2] |= (j >= first && j < end ? (uint32_t)v[j] : 0u) << (16 * (j & 1));
  return r;
}

// The first `n` (any sign, may exceed 8) of eight 16-bit values at p, the others 0.
__device__ __forceinline__ u32x4 load8_part(const uint16_t* p, int64_t n) {
  if (n <= 0) return u32x4{0u, 0u, 0u, 0u};
  const int last = (int)(n < 8 ? n : 8) - 1;
  uint16_t v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = p[j < last ? j : last];
  loads_made();
  return pack8(v, 0, n);
}

// 16 bytes per lane from base + offset (bytes, the lane's own) straight to LDS,
// lane l's at dst + 16 l bytes; base and dst the same in all lanes.  (The
// buffer form: after the global form the compiler waits for every LDS
// operation where it would otherwise count them.)
__device__ __forceinline__ void to_lds16(const void* base, uint32_t offset,
                                         __attribute__((address_space(3))) uint16_t* dst) {
  // stride 0, no range limit below 4 GB, raw 32-bit data
  const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, -1, 0x00020000);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 16, offset, 0, 0, 0);
}

// Waits until at most VM of the wave's memory operations (loads to LDS among
// them) and LGKM of its LDS operations are outstanding.
template <int VM, int LGKM>
__device__ __forceinline__ void wait_vm() {
  // vmcnt in bits 3:0 and 15:14, lgkmcnt in 11:8; expcnt (6:4) at its largest: not waited for
  __builtin_amdgcn_s_waitcnt(0x0070 | (VM & 15) | ((VM >> 4) << 14) | (LGKM << 8));
  asm volatile("" ::: "memory");
}

// A workgroup barrier that waits for nothing else: the caller has waited for
// what other waves will read.
__device__ __forceinline__ void block_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

}  // namespace externd
