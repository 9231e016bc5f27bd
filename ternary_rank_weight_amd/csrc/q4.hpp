// The products of 4-bit weights with a few tokens: arguments and kernel, shared by
// the translation units that instantiate it (one per operand type).
#pragma once
#include <algorithm>

#include "activation.hpp"
#include "device_common.hpp"
#include "frag.hpp"
#include "kernels.hpp"

namespace externd {

constexpr int kTile = 16, kChunk = 128;   // rows and columns of a packed tile of a chunk

struct Q4Args {
  const u32x4* codes[2];
  const uint16_t* scales[2];
  const uint16_t* mins[2];
  const uint16_t* x;    // rows of 16-bit entries, or staged
  const float* x32;     // fp32 rows that the kernel splits itself, else null
  void* y;
  int64_t ldx, slice, rows, cols, chunks, tokens;   // slice: entries from one slice of x to the next
  int staged;
  int pieces;           // slots per token: 1, or 3 for fp32
  int act;
};

hipError_t q4_product_bf16(const Q4Args& a, int gpc, int mats, int out_type, hipStream_t s);
hipError_t q4_product_f16(const Q4Args& a, int gpc, int mats, int out_type, hipStream_t s);

// Entries col .. col + 7 of a row as fp32 (0 past the end); n: entries left in the row.
template <int DT>
__device__ inline void load_weights(const void* W, int64_t at, int64_t n, float (&w)[8]) {
  if constexpr (DT == EXTERND_F32) {
    const float* p = static_cast<const float*>(W) + at;
    if (n >= 8) {
      const u32x4_a4 a = *reinterpret_cast<const u32x4_a4*>(p), b = *reinterpret_cast<const u32x4_a4*>(p + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) { w[j] = __uint_as_float(a[j]); w[4 + j] = __uint_as_float(b[j]); }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = j < n ? p[j] : 0.f;
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(W) + at;
    u32x4 v;
    if (n >= 8) v = (reinterpret_cast<uintptr_t>(p) & 15) == 0 ? load8<true>(p) : load8<false>(p);
    else v = load8_part(p, n);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = f32_from_16<DT == EXTERND_BF16>((v[j / 2] >> (16 * (j & 1))) & 0xffffu);
  }
}

// Codes of one word as the operand 16 + c (exact in bf16 and fp16: the code
// sits in the four mantissa bits below 16's units).
template <bool BF>
__device__ __forceinline__ u32x4 unpack_q4(uint32_t w) {
  constexpr uint32_t mask = BF ? 0x00780078u : 0x03C003C0u, base = BF ? 0x41804180u : 0x4C004C00u;
  u32x4 r;
  if constexpr (BF) {
    r.x = ((w << 3) & mask) | base;
    r.y = ((w >> 1) & mask) | base;
    r.z = ((w >> 5) & mask) | base;
    r.w = ((w >> 9) & mask) | base;
  } else {
    r.x = ((w << 6) & mask) | base;
    r.y = ((w << 2) & mask) | base;
    r.z = ((w >> 2) & mask) | base;
    r.w = ((w >> 6) & mask) | base;
  }
  return r;
}

// The high half, the next or the last 8 bits of an fp32 value as bf16, by masks of
// the parts to take off (together they are the value).
__device__ __forceinline__ uint32_t third_of(float v, uint32_t part0, uint32_t part1) {
  const float b = v - __uint_as_float(__float_as_uint(v) & part0);
  const float c = b - __uint_as_float(__float_as_uint(b) & part1);
  return __float_as_uint(c) >> 16;
}

}  // namespace externd
