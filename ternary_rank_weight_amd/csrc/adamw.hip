// An AdamW step over many tensors at once.  Per entry, in fp32 and in this order of roundings:
//   g1 = g scale,  m1 = b1 m + c1 g1,  v1 = b2 v + c2 (g1 g1)           (c = 1 - b)
//   w1 = (1 - lr decay) w - (lr / (1 - b1^t)) (m1 / (sqrt(v1) / sqrt(1 - b2^t) + eps))
// w is the fp32 master weight where there is one (the parameter is its rounding), else the
// parameter itself.  The update takes m1 and v1 as they are; what is kept of them is
// rounded after that.
//
// Moments in 8 bits: blocks of 256 entries share the exponent field b of their largest
// magnitude.  m is an e4m3 number of m 2^(134 - b), whose largest lies in 128 .. 256; v
// has no sign and needs range (it is a square): five bits of exponent and three of
// mantissa of v 2^(141 - b), 2^32 from the largest to the smallest, and what is
// not 0 does not become 0, since a small m over the root of a lost v would be a
// step of any size.  Scales are powers of two: scaling is exact, so a code depends on the fp32
// moment alone.  A moment that is not finite has no part in its block's exponent, and a code of its own:
// NaN, and infinity of v (whose entry then stays as it is, as with 32 bits).
//
// A wave takes a block at a time, four neighbouring entries a lane: whole lines of every
// array, and the block's largest is one reduction over the wave.
#include <algorithm>
#include <type_traits>

#include "adamw.hpp"
#include "device_common.hpp"
#include "frag.hpp"

namespace externd {

namespace {

constexpr int kBlock = kAdamBlock;
constexpr int kWaves = 8, kBlocks = 2;            // waves of a workgroup; blocks that a wave has on their way
constexpr int kAdamChunk = kWaves * kBlocks * kBlock;   // entries of one tensor that a workgroup takes at once

typedef uint32_t u32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));

// Four entries of a type, as they lie in memory.
template <int DT>
struct Four {
  typename std::conditional<DT == EXTERND_F32, u32x4, uint2>::type v;
  __device__ void load(const void* base, int64_t at) {
    if constexpr (DT == EXTERND_F32) {
      v = *reinterpret_cast<const u32x4_a4*>(static_cast<const float*>(base) + at);
    } else {
      const u32x2_a2 w = *reinterpret_cast<const u32x2_a2*>(static_cast<const uint16_t*>(base) + at);
      v = uint2{w.x, w.y};
    }
  }
  // the first `left` of them (any sign), the others 0
  __device__ void load_part(const void* base, int64_t at, int64_t left) {
    uint32_t e[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      e[j] = 0u;
      if (j < left) {
        if constexpr (DT == EXTERND_F32) e[j] = static_cast<const uint32_t*>(base)[at + j];
        else e[j] = static_cast<const uint16_t*>(base)[at + j];
      }
    }
    if constexpr (DT == EXTERND_F32) v = u32x4{e[0], e[1], e[2], e[3]};
    else v = uint2{e[0] | (e[1] << 16), e[2] | (e[3] << 16)};
  }
  __device__ float get(int j) const {
    if constexpr (DT == EXTERND_F32) return __uint_as_float(v[j]);
    else return f32_from_16<DT == EXTERND_BF16>(((j < 2 ? v.x : v.y) >> (16 * (j & 1))) & 0xffffu);
  }
  __device__ void set(const float (&f)[4]) {
    if constexpr (DT == EXTERND_F32) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = __float_as_uint(f[j]);
    } else {
      constexpr bool BF = DT == EXTERND_BF16;
      v = uint2{f32_to_16<BF>(f[0]) | (f32_to_16<BF>(f[1]) << 16), f32_to_16<BF>(f[2]) | (f32_to_16<BF>(f[3]) << 16)};
    }
  }
  __device__ void store(void* base, int64_t at) const {
    if constexpr (DT == EXTERND_F32) *reinterpret_cast<u32x4_a4*>(static_cast<float*>(base) + at) = v;
    else *reinterpret_cast<u32x2_a2*>(static_cast<uint16_t*>(base) + at) = u32x2_a2{v.x, v.y};
  }
  __device__ void store_part(void* base, int64_t at, int64_t left) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j >= left) continue;
      if constexpr (DT == EXTERND_F32) static_cast<uint32_t*>(base)[at + j] = v[j];
      else static_cast<uint16_t*>(base)[at + j] = (uint16_t)((j < 2 ? v.x : v.y) >> (16 * (j & 1)));
    }
  }
};

__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

__device__ __forceinline__ void decode_m(uint32_t codes, int b, float (&m)[4]) {
  const float s = power_of_two(b - 134);
  m[0] = __builtin_amdgcn_cvt_f32_fp8(codes, 0) * s;
  m[1] = __builtin_amdgcn_cvt_f32_fp8(codes, 1) * s;
  m[2] = __builtin_amdgcn_cvt_f32_fp8(codes, 2) * s;
  m[3] = __builtin_amdgcn_cvt_f32_fp8(codes, 3) * s;
}

// A code is the upper byte of the fp16 number's bits below its sign: 0xf8 is infinity, 0xff a NaN.
__device__ __forceinline__ void decode_v(uint32_t codes, int b, float (&v)[4]) {
  const float s = power_of_two(b - 141);
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = f32_from_16<false>(((codes >> (8 * j)) & 0xffu) << 7) * s;
}

// The exponent byte of a wave's block of values.
__device__ __forceinline__ int block_exponent(const float (&x)[4]) {
  uint32_t top = 0u;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t a = __float_as_uint(x[j]) & 0x7fffffffu;
    top = max(top, a < 0x7f800000u ? a : 0u);
  }
  return max(__builtin_amdgcn_readlane((int)wave_umax_to63(top), kWave - 1) >> 23, 15);
}

__device__ __forceinline__ uint32_t encode_m(const float (&m)[4], int b) {
  const float s = power_of_two(134 - b);
  int w = 0;
  w = __builtin_amdgcn_cvt_pk_fp8_f32(m[0] * s, m[1] * s, w, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(m[2] * s, m[3] * s, w, true);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (!__builtin_isfinite(m[j])) w |= 0x7f << (8 * j);
  return (uint32_t)w;
}

__device__ __forceinline__ uint32_t encode_v(const float (&v)[4], int b) {
  const float s = power_of_two(141 - b);
  uint32_t w = 0u;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float x = v[j] * s;
    const uint32_t bits = __float_as_uint(x);
    uint32_t code = x < 0x1p-14f ? max((uint32_t)rintf(x * 0x1p17f), 1u)
                                 : ((bits + 0x7ffffu + ((bits >> 20) & 1u)) >> 20) - (112u << 3);
    if (v[j] == 0.f) code = 0u;
    if (!__builtin_isfinite(v[j])) code = v[j] != v[j] ? 0xffu : 0xf8u;
    w |= code << (8 * j);
  }
  return w;
}

// Bound by HBM: 74.7 million bf16 parameters and gradients with master weights, 417 us with 32-bit moments (28 bytes
// an entry, 5.0 TB/s), 230 to 250 with 8-bit ones (16 bytes, 4.8 to 5.2); with fp32 gradients 442 and 277 (30 and 18 bytes,
// 5.1 and 4.9 TB/s).
template <bool EIGHT, int PT, int GT, bool MASTER>
__global__ __launch_bounds__(kWaves * kWave) void k_adamw(AdamArgs a) {
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  // this step's number and powers of the betas
  const double q1 = a.step[1] * a.b1, q2 = a.step[2] * a.b2, count = a.step[0] + 1.0;
  const double lr = a.lr_device ? (double)*a.lr_device : a.lr;
  const float scale = a.scale_device ? *a.scale_device : a.scale;
  const float b1 = (float)a.b1, c1 = (float)(1.0 - a.b1), b2 = (float)a.b2, c2 = (float)(1.0 - a.b2);
  const float rate = (float)(lr / (1.0 - q1)), root = (float)(1.0 / sqrt(1.0 - q2)), eps = (float)a.eps;

  int i = 0;
  for (uint32_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
    while (i + 1 < a.count && c >= a.t[i + 1].first) ++i;
    const AdamTensor& t = a.t[i];
    const float keep = (float)(1.0 - lr * (double)t.decay);
    const int64_t block0 = (int64_t)(c - t.first) * (kWaves * kBlocks) + wave * kBlocks;
    auto work = [&](auto inside) {   // inside: every entry of the blocks is one of the tensor's
      constexpr bool IN = decltype(inside)::value;
      Four<GT> g[kBlocks];
      Four<PT> p[kBlocks];
      u32x4 w[kBlocks], m[kBlocks], v[kBlocks];   // EIGHT: codes and exponents in the first two
#pragma unroll
      for (int u = 0; u < kBlocks; ++u) {
        const int64_t block = block0 + u, at = block * kBlock + lane * 4, left = t.n - at;
        if (!IN && block * kBlock >= t.n) continue;   // (the same in the whole wave)
        if constexpr (EIGHT) {
          m[u].x = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(t.m) + at);
          v[u].x = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(t.v) + at);
          m[u].y = t.m_exp[block];
          v[u].y = t.v_exp[block];
        } else {
          m[u] = *reinterpret_cast<const u32x4*>(static_cast<const float*>(t.m) + at);
          v[u] = *reinterpret_cast<const u32x4*>(static_cast<const float*>(t.v) + at);
        }
        if constexpr (MASTER) w[u] = *reinterpret_cast<const u32x4*>(t.master + at);
        if constexpr (IN) g[u].load(t.g, at);
        else g[u].load_part(t.g, at, left);
        if constexpr (!MASTER) {
          if constexpr (IN) p[u].load(t.p, at);
          else p[u].load_part(t.p, at, left);
        }
      }
#pragma unroll
      for (int u = 0; u < kBlocks; ++u) {
        const int64_t block = block0 + u, at = block * kBlock + lane * 4, left = t.n - at;
        if (!IN && block * kBlock >= t.n) continue;
        float fm[4], fv[4], fw[4];
        if constexpr (EIGHT) {
          decode_m(m[u].x, (int)m[u].y, fm);
          decode_v(v[u].x, (int)v[u].y, fv);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            fm[j] = __uint_as_float(m[u][j]);
            fv[j] = __uint_as_float(v[u][j]);
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float g1 = g[u].get(j) * scale;
          const float m1 = b1 * fm[j] + c1 * g1;
          const float v1 = b2 * fv[j] + c2 * (g1 * g1);
          const float w0 = MASTER ? __uint_as_float(w[u][j]) : p[u].get(j);
          fm[j] = m1;
          fv[j] = v1;
          fw[j] = keep * w0 - rate * (m1 / (sqrtf(v1) * root + eps));
          if (!IN && j >= left) fm[j] = fv[j] = fw[j] = 0.f;   // (what fills up the last block stays 0)
        }
        p[u].set(fw);
        if constexpr (IN) p[u].store(t.p, at);
        else p[u].store_part(t.p, at, left);
        if constexpr (MASTER) *reinterpret_cast<f32x4*>(t.master + at) = f32x4{fw[0], fw[1], fw[2], fw[3]};
        if constexpr (EIGHT) {
          const int bm = block_exponent(fm), bv = block_exponent(fv);
          *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(t.m) + at) = encode_m(fm, bm);
          *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(t.v) + at) = encode_v(fv, bv);
          if (lane == 0) {
            t.m_exp[block] = (uint8_t)bm;
            t.v_exp[block] = (uint8_t)bv;
          }
        } else {
          *reinterpret_cast<f32x4*>(static_cast<float*>(t.m) + at) = f32x4{fm[0], fm[1], fm[2], fm[3]};
          *reinterpret_cast<f32x4*>(static_cast<float*>(t.v) + at) = f32x4{fv[0], fv[1], fv[2], fv[3]};
        }
      }
    };
    if ((block0 + kBlocks) * kBlock <= t.n) work(std::true_type());
    else work(std::false_type());
  }

  // The last workgroup to get here counts the step: every other has read the old one.  (Counting at the start, past that
  // read, was slower: a wave's loads return behind its atomic.)
  if (a.advance) {
    __syncthreads();
    if (threadIdx.x == 0) {
      uint32_t* arrived = reinterpret_cast<uint32_t*>(a.step + 3);
      if (atomicAdd(arrived, 1u) == gridDim.x - 1) {
        a.step[0] = count;
        a.step[1] = q1;
        a.step[2] = q2;
        *arrived = 0u;
      }
    }
  }
}

// The values of 8-bit moments.  Bound by HBM, mostly what it writes: 74.7 million entries, 147 us (10 bytes an entry, 5.1 TB/s).
__global__ __launch_bounds__(256) void k_adamw_moments(const uint8_t* __restrict__ m, const uint8_t* __restrict__ m_exp,
                                                        const uint8_t* __restrict__ v, const uint8_t* __restrict__ v_exp,
                                                        int64_t blocks, float* __restrict__ m_out, float* __restrict__ v_out) {
  const int64_t total = blocks * (kBlock / 4);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t block = i / (kBlock / 4);
    float f[4];
    decode_m(reinterpret_cast<const uint32_t*>(m)[i], m_exp[block], f);
    reinterpret_cast<f32x4*>(m_out)[i] = f32x4{f[0], f[1], f[2], f[3]};
    decode_v(reinterpret_cast<const uint32_t*>(v)[i], v_exp[block], f);
    reinterpret_cast<f32x4*>(v_out)[i] = f32x4{f[0], f[1], f[2], f[3]};
  }
}

// Few workgroups of many waves: each counts itself at the end, 12 ns one after the other (11 million entries in 8
// bits: 42 us with eight of four waves a compute unit, 33 with four of eight).  With 32 bits no more than are resident
// together, as the kernel's registers allow: three where gradients are fp32 and the weights are too or have masters, whose
// fourth would begin when another ends (74.7 million entries, 16-bit parameters with masters 453 -> 442 us, fp32 415 -> 411; held to
// the registers of four 458 and 421).  With 8 bits a fourth that waits costs nothing (277, 279 with three).
template <bool EIGHT, int PT, int GT, bool MASTER>
hipError_t launch(const AdamArgs& a, int cus, hipStream_t s) {
  const auto kernel = k_adamw<EIGHT, PT, GT, MASTER>;
  static const int resident = [&] {
    int n = 0;
    if (EIGHT || hipOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kWaves * kWave, 0) != hipSuccess) n = 4;
    return std::clamp(n, 1, 4);
  }();
  const unsigned grid = std::max(1u, std::min(a.chunks, (uint32_t)(cus * resident)));
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(kWaves * kWave), 0, s, a);
  return hipGetLastError();
}

template <bool EIGHT, int PT, bool MASTER>
hipError_t pick_grad(const AdamArgs& a, int grad, int cus, hipStream_t s) {
  if (grad == EXTERND_F32) return launch<EIGHT, PT, EXTERND_F32, MASTER>(a, cus, s);
  if (grad == EXTERND_BF16) return launch<EIGHT, PT, EXTERND_BF16, MASTER>(a, cus, s);
  return launch<EIGHT, PT, EXTERND_F16, MASTER>(a, cus, s);
}

template <bool EIGHT>
hipError_t pick(const AdamArgs& a, int kind, int cus, hipStream_t s) {
  const int grad = kind % 3, param = kind / 3 % 3;
  const bool master = kind >= 9;
  if (param == EXTERND_F32) return pick_grad<EIGHT, EXTERND_F32, false>(a, grad, cus, s);
  if (param == EXTERND_BF16)
    return master ? pick_grad<EIGHT, EXTERND_BF16, true>(a, grad, cus, s)
                  : pick_grad<EIGHT, EXTERND_BF16, false>(a, grad, cus, s);
  return master ? pick_grad<EIGHT, EXTERND_F16, true>(a, grad, cus, s)
                : pick_grad<EIGHT, EXTERND_F16, false>(a, grad, cus, s);
}

// Tensors of one kind go through one kernel.
int kind_of(const externd_adamw_tensor& t) { return t.grad_dtype + 3 * t.param_dtype + (t.master ? 9 : 0); }

}  // namespace

// At most kAdamTensors a launch, by kind; the last launch counts the step.
hipError_t run_adamw(const externd_adamw_tensor* tensors, int64_t count, const externd_adamw_opts& o, int cus, hipStream_t s) {
  AdamArgs a = {};
  a.lr = o.lr;
  a.lr_device = o.lr_device;
  a.b1 = o.beta1;
  a.b2 = o.beta2;
  a.eps = o.eps;
  a.scale = o.grad_scale;
  a.scale_device = o.grad_scale_device;
  a.step = o.step;
  int kinds[18], used = 0;   // in order of their first tensor
  int64_t left[18] = {};     // tensors of a kind that have not been taken
  for (int64_t i = 0; i < count; ++i)
    if (tensors[i].n > 0 && left[kind_of(tensors[i])]++ == 0) kinds[used++] = kind_of(tensors[i]);
  auto run = [&](int kind, bool last) {
    a.advance = last;
    const hipError_t e = o.bits == 8 ? pick<true>(a, kind, cus, s) : pick<false>(a, kind, cus, s);
    a.count = 0;
    a.chunks = 0;
    return e;
  };
  for (int q = 0; q < used; ++q)
    for (int64_t i = 0; i < count; ++i) {
      const externd_adamw_tensor& t = tensors[i];
      if (t.n == 0 || kind_of(t) != kinds[q]) continue;
      const int64_t chunks = (t.n + kAdamChunk - 1) / kAdamChunk;
      if (a.count == kAdamTensors || a.chunks + chunks > UINT32_MAX / 2) {
        const hipError_t e = run(kinds[q], false);
        if (e != hipSuccess) return e;
      }
      a.t[a.count++] = {t.param, t.grad, t.master, t.m, t.v, t.m_exp, t.v_exp, t.n, a.chunks, t.decay};
      a.chunks += (uint32_t)chunks;
      if (--left[kinds[q]] == 0) {
        const hipError_t e = run(kinds[q], q + 1 == used);
        if (e != hipSuccess) return e;
      }
    }
  return used ? hipSuccess : run(0, true);   // no entries at all: the step counts
}

hipError_t run_adamw_moments(const uint8_t* m, const uint8_t* m_exp, const uint8_t* v, const uint8_t* v_exp, int64_t blocks,
                             float* m_out, float* v_out, int cus, hipStream_t s) {
  const int64_t grid = std::min<int64_t>((blocks * (kBlock / 4) + 255) / 256, (int64_t)cus * 16);
  hipLaunchKernelGGL(k_adamw_moments, dim3((unsigned)grid), dim3(256), 0, s, m, m_exp, v, v_exp, blocks, m_out, v_out);
  return hipGetLastError();
}

}  // namespace externd
