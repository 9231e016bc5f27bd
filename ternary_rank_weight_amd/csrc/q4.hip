// 4-bit weights with group scales: quantization, the values they stand for,
// and their products with a few tokens.
//
// A group is `group` (32, 64 or 128) neighbouring entries of a row, with a
// bf16 scale s and, asymmetric, a bf16 minimum m:
//
//   symmetric   s = bf16(max|w| / 7),         c = clamp(rint(w / s), -8, 7) + 8,   value s (c - 8)
//   asymmetric  s = bf16((max w - min w) / 15), m = bf16(min w),
//               c = clamp(rint((w - m) / s), 0, 15),                               value s c + m
//
// (all steps in fp32, rounded once to the stored type; a group of scale 0
// has c - 8 = 0 or c = 0).  The scales are bf16 because it has fp32's range:
// no weight matrix overflows or loses its small groups.  Its 8 bits cost
// nothing in the codes, which are chosen for the rounded scale.
//
// Layout: tiles of 16 rows x chunks of 128 columns.  A wave reads one tile
// of one chunk with one 16-byte load per lane, 1 KB of neighbouring bytes:
// lane r + 16 p holds row r, and its word i (0..3) the codes of columns
// 32 i + 8 p + j, which are exactly the entries that lane holds in the i-th
// 16x16x32 product of the chunk.  So nothing is moved between lanes, and each
// product stays inside one group.  Code j = 2 s sits at bits 4 s, code
// j = 2 s + 1 at bits 16 + 4 s: one shift and one and-or give two operand entries.
// The scales (and minima) of a tile of a chunk are 16 x 128 / group
// neighbouring bf16 values.
#include <algorithm>

#include "q4.hpp"

namespace externd {

namespace {

// ---- quantize, pack, reconstruct: one wave per (tile, chunk) ----

struct Place {
  int64_t tile, chunk, row, col;   // col: the lane's first column of word 0
  int r, p;
};
__device__ inline Place place_of(int64_t job, int64_t chunks, int lane) {
  Place q;
  q.tile = job / chunks;
  q.chunk = job - q.tile * chunks;
  q.r = lane & 15;
  q.p = lane >> 4;
  q.row = kTile * q.tile + q.r;
  q.col = kChunk * q.chunk + 8 * q.p;
  return q;
}

// Eight codes as a word of the layout.
__device__ inline uint32_t pack_word(const uint32_t (&c)[8]) {
  uint32_t w = 0u;
#pragma unroll
  for (int j = 0; j < 8; ++j) w |= (c[j] & 15u) << (4 * (j >> 1) + 16 * (j & 1));
  return w;
}

// Max of a value over the four lanes that share a row.
__device__ inline float row_max(float v) {
  v = fmaxf(v, __shfl_xor(v, 16, kWave));
  return fmaxf(v, __shfl_xor(v, 32, kWave));
}

// Minimum and maximum of numbers (not NaN) in one instruction: the median with an
// infinity.  (fminf and fmaxf first quiet both operands.)
__device__ inline float max_of(float a, float b) { return __builtin_amdgcn_fmed3f(a, b, INFINITY); }
__device__ inline float min_of(float a, float b) { return __builtin_amdgcn_fmed3f(a, b, -INFINITY); }

// Bound by HBM: one read of the matrix, one write of 4.5 to 5 bits per entry;
// the arithmetic is kept to about a dozen operations an entry so that it stays
// below that.  Quotients are those of a division, without one: y = 1 / s correctly
// rounded, q = w y, and q + (w - q s) y by two fused operations is the correctly
// rounded w / s (Markstein's theorem).  Scales so small that y may not be a
// normal number are divided by.  9728 x 2559 in bf16 (odd rows, read by shifted
// dwords): 21 us, 3.0 TB/s; 1024 x 2560 in fp32: 6.5 us, mostly latency.
template <int DT, int GPC, bool MINS>
__global__ __launch_bounds__(256) void k_q4_quantize(const void* __restrict__ W, int64_t rows, int64_t cols,
                                                      int64_t ldw, int64_t chunks, int64_t jobs,
                                                      u32x4* __restrict__ codes, uint16_t* __restrict__ scales,
                                                      uint16_t* __restrict__ mins) {
  constexpr int SPG = 4 / GPC;   // words (of 32 columns) per group
  constexpr float lo = MINS ? 0.f : -8.f, hi = MINS ? 15.f : 7.f;
  const int lane = threadIdx.x & (kWave - 1);
  for (int64_t job = (int64_t)blockIdx.x * 4 + threadIdx.x / kWave; job < jobs; job += 4 * (int64_t)gridDim.x) {
    const Place q = place_of(job, chunks, lane);
    float w[4][8];
    int left[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      left[i] = q.row < rows ? (int)min<int64_t>(max<int64_t>(cols - q.col - 32 * i, 0), 8) : 0;
      load_weights<DT>(W, q.row * ldw + q.col + 32 * i, left[i], w[i]);
      if (MINS && left[i] > 0 && left[i] < 8) {   // past the end: entries that change no extreme
#pragma unroll
        for (int j = 1; j < 8; ++j) w[i][j] = j < left[i] ? w[i][j] : w[i][0];
      }
    }
    u32x4 out;
#pragma unroll
    for (int g = 0; g < GPC; ++g) {
      // extremes, and a sum of 0 w that is NaN if any entry is not finite (maxima drop NaN)
      float low = INFINITY, high = MINS ? -INFINITY : 0.f, bad = 0.f;
#pragma unroll
      for (int i = g * SPG; i < (g + 1) * SPG; ++i) {
        if (MINS && left[i] == 0) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          bad = fmaf(w[i][j], 0.f, bad);
          if constexpr (MINS) { low = min_of(low, w[i][j]); high = max_of(high, w[i][j]); }
          else high = max_of(high, fabsf(w[i][j]));
        }
      }
      bad = bad == 0.f ? 0.f : 1.f;
      high = row_max(high);
      float s, m = 0.f;
      if constexpr (MINS) {
        low = -row_max(-low);
        const bool any = low <= high;   // a group past the row's end has scale and minimum 0
        s = any ? bf16_to_f32(f32_to_bf16((high - low) / 15.f)) : 0.f;
        m = any ? bf16_to_f32(f32_to_bf16(low)) : 0.f;
      } else {
        s = bf16_to_f32(f32_to_bf16(high / 7.f));
      }
      if (row_max(bad) != 0.f || !(s < INFINITY) || !(fabsf(m) < INFINITY)) s = m = NAN;
      const float inv = 1.f / s;
      const bool plain = s > 1e-30f;   // (bf16 scales stay below 2^126)
#pragma unroll
      for (int i = g * SPG; i < (g + 1) * SPG; ++i) {
        float c[8];
        if (plain) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float v = MINS ? w[i][j] - m : w[i][j], t = v * inv;
            c[j] = __builtin_amdgcn_fmed3f(rintf(fmaf(fmaf(-t, s, v), inv, t)), lo, hi);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float t = s > 0.f ? rintf((MINS ? w[i][j] - m : w[i][j]) / s) : 0.f;
            c[j] = fminf(fmaxf(t, lo), hi);
          }
        }
        // four codes to a half word, exact in fp32: c0 + 16 c2 + 256 c4 + 4096 c6
        const float bias = MINS ? 0.f : 8.f * 4369.f;
        const uint32_t h0 = (uint32_t)(fmaf(c[6], 4096.f, fmaf(c[4], 256.f, fmaf(c[2], 16.f, c[0]))) + bias);
        const uint32_t h1 = (uint32_t)(fmaf(c[7], 4096.f, fmaf(c[5], 256.f, fmaf(c[3], 16.f, c[1]))) + bias);
        out[i] = h0 | (h1 << 16);
      }
      if (q.p == 0) {
        scales[(job * kTile + q.r) * GPC + g] = (uint16_t)f32_to_bf16(s);
        if constexpr (MINS) mins[(job * kTile + q.r) * GPC + g] = (uint16_t)f32_to_bf16(m);
      }
    }
    codes[job * kWave + lane] = out;
  }
}

// One pass when weights are loaded, not tuned: 56 us for 9728 x 2560, 0.7 TB/s (1.6 bytes an
// entry), bound by its byte loads.
// Codes one byte each and tables row by row (rows x ceil(cols / group)) into
// the layout; padding gets code 0, scale 0, minimum 0.
__global__ __launch_bounds__(256) void k_q4_pack(const uint8_t* __restrict__ src, const uint16_t* __restrict__ ssrc,
                                                  const uint16_t* __restrict__ msrc, int64_t rows, int64_t cols,
                                                  int gpc, int64_t chunks, int64_t jobs, u32x4* __restrict__ codes,
                                                  uint16_t* __restrict__ scales, uint16_t* __restrict__ mins) {
  const int lane = threadIdx.x & (kWave - 1);
  for (int64_t job = (int64_t)blockIdx.x * 4 + threadIdx.x / kWave; job < jobs; job += 4 * (int64_t)gridDim.x) {
    const Place q = place_of(job, chunks, lane);
    u32x4 out;
  #pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t left = q.row < rows ? cols - q.col - 32 * i : 0;
      uint32_t c[8];
  #pragma unroll
      for (int j = 0; j < 8; ++j) c[j] = j < left ? src[q.row * cols + q.col + 32 * i + j] : 0u;
      out[i] = pack_word(c);
    }
    codes[job * kWave + lane] = out;
    const int64_t groups = (cols + kChunk / gpc - 1) / (kChunk / gpc);
    if (q.p < gpc) {   // lane (r, p) moves group p of row r
      const int64_t g = q.chunk * gpc + q.p;
      const bool ok = q.row < rows && g < groups;
      scales[(job * kTile + q.r) * gpc + q.p] = ok ? ssrc[q.row * groups + g] : (uint16_t)0;
      if (msrc) mins[(job * kTile + q.r) * gpc + q.p] = ok ? msrc[q.row * groups + g] : (uint16_t)0;
    }
  }
}

// p + m rounded to fp32, towards the neighbour with an odd last bit where it is inexact:
// rounding that to fewer bits gives what rounding the exact sum would.
__device__ inline float add_to_odd(float p, float m) {
  const float v = p + m, b = v - p, rest = (p - (v - b)) + (m - b);   // v + rest = p + m
  const uint32_t bits = __float_as_uint(v);
  if (!(fabsf(rest) > 0.f) || (bits & 1u)) return v;   // (rest is NaN where v is not finite)
  return __uint_as_float((rest > 0.f) == (v > 0.f) ? bits + 1 : bits - 1);
}

// The values, rounded once to the output's type.  Bound by HBM: the write.  9728 x
// 2559 to fp32: 26 us, 4.4 TB/s.
template <int DT>
__global__ __launch_bounds__(256) void k_q4_reconstruct(const u32x4* __restrict__ codes,
                                                         const uint16_t* __restrict__ scales,
                                                         const uint16_t* __restrict__ mins, int64_t rows, int64_t cols,
                                                         int gpc, int64_t chunks, int64_t jobs, void* __restrict__ out) {
  const int lane = threadIdx.x & (kWave - 1);
  for (int64_t job = (int64_t)blockIdx.x * 4 + threadIdx.x / kWave; job < jobs; job += 4 * (int64_t)gridDim.x) {
    const Place q = place_of(job, chunks, lane);
    if (q.row >= rows) continue;
    const u32x4 cw = codes[job * kWave + lane];
  #pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t col = q.col + 32 * i, left = cols - col;
      if (left <= 0) break;
      const int64_t at = (job * kTile + q.r) * gpc + i * gpc / 4;
      const float s = bf16_to_f32(scales[at]);
      const float m = mins ? bf16_to_f32(mins[at]) : 0.f;
      const float mid = mins ? 0.f : 8.f;
      float v[8];
  #pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t c = (cw[i] >> (4 * (j >> 1) + 16 * (j & 1))) & 15u;
        // (the product is exact, 8 by 4 bits, unless it passes fp32's range, which s c + m may not)
        v[j] = fmaf(s, (float)c - mid, m);
        if constexpr (DT != EXTERND_F32) {
          const float p = s * ((float)c - mid);
          if (mins && __builtin_isfinite(p)) v[j] = add_to_odd(p, m);
        }
      }
      if constexpr (DT == EXTERND_F32) {
        float* p = static_cast<float*>(out) + q.row * cols + col;
        if (left >= 8) {
          u32x4 a, b;
  #pragma unroll
          for (int j = 0; j < 4; ++j) { a[j] = __float_as_uint(v[j]); b[j] = __float_as_uint(v[4 + j]); }
          *reinterpret_cast<u32x4_a4*>(p) = a;
          *reinterpret_cast<u32x4_a4*>(p + 4) = b;
        } else {
  #pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < left) p[j] = v[j];
        }
      } else {
        constexpr bool BF = DT == EXTERND_BF16;
        uint16_t* p = static_cast<uint16_t*>(out) + q.row * cols + col;
        if (left >= 8 && (reinterpret_cast<uintptr_t>(p) & 3) == 0) {
          u32x4 a;
  #pragma unroll
          for (int j = 0; j < 4; ++j) a[j] = f32_to_16<BF>(v[2 * j]) | (f32_to_16<BF>(v[2 * j + 1]) << 16);
          *reinterpret_cast<u32x4_a4*>(p) = a;
        } else {
  #pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < left) p[j] = (uint16_t)f32_to_16<BF>(v[j]);
        }
      }
    }
  }
}

// ---- products ----

// x in the order the products read it: for every tile of 16 slots and slice of 32
// columns the 64 lanes' 16 bytes one after the other, so that a wave reads 1 KB
// of neighbouring bytes; zero past the columns.  A slot is a token, or one of
// the three bf16 parts of an fp32 token that add up to it exactly (8 of its 24
// bits each; 15 slots, 5 tokens, per tile).  3 to 5 us.
template <int DT>
__global__ __launch_bounds__(256) void k_q4_stage_x(const void* __restrict__ x, int64_t tokens, int64_t cols,
                                                     int64_t ldx, int64_t slices, int64_t pieces_of_tiles,
                                                     u32x4* __restrict__ out) {
  constexpr int PIECES = DT == EXTERND_F32 ? 3 : 1, PER = DT == EXTERND_F32 ? 5 : 16;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < pieces_of_tiles; i += (int64_t)gridDim.x * 256) {
    const int lane = (int)(i & 63), r = lane & 15, p = lane >> 4;
    const int64_t tile = (i >> 6) / slices, slice = (i >> 6) - tile * slices;
    const int64_t t = tile * PER + r / PIECES, col = 32 * slice + 8 * p, left = cols - col;
    u32x4 v = {0u, 0u, 0u, 0u};
    if (r < PER * PIECES && t < tokens && left > 0) {
      if constexpr (DT == EXTERND_F32) {
        float f[8];
        load_weights<EXTERND_F32>(x, t * ldx + col, left, f);
        const int piece = r % 3;
        const uint32_t m0 = piece > 0 ? 0xffff0000u : 0u, m1 = piece > 1 ? 0xffff0000u : 0u;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j / 2] |= third_of(f[j], m0, m1) << (16 * (j & 1));
      } else {
        const uint16_t* q = static_cast<const uint16_t*>(x) + t * ldx + col;
        v = left >= 8 ? ((reinterpret_cast<uintptr_t>(q) & 15) == 0 ? load8<true>(q) : load8<false>(q))
                      : load8_part(q, left);
      }
    }
    out[i] = v;
  }
}

int64_t chunks_of(int64_t cols) { return (cols + kChunk - 1) / kChunk; }
int64_t jobs_of(int64_t rows, int64_t cols) { return (rows + kTile - 1) / kTile * chunks_of(cols); }
// Workgroups of four waves, one job each until the grid's limit.
dim3 jobs_grid(int64_t jobs) { return dim3((unsigned)std::min<int64_t>((jobs + 3) / 4, 1 << 22)); }

}  // namespace

// Staged: fp32 of more than five tokens, rows that are not all 16-byte aligned, and large matrices with
// more than one slot tile, where the waves' reads of x outweigh the weights and
// 64-byte pieces of rows come at half the rate of whole kilobytes.  In us, bf16, read in
// place and staged (the copy's launch with it):
//                          17 tokens     32 tokens     48 tokens     64 tokens
//   2560 x 2560 (2^22.6)    9.1 11.4     10.0 11.6     14.6 13.4     17.8 14.6
//   4096 x 4096 (2^24)     14.1 17.0     15.5 17.1     20.8 18.3     24.9 19.7
//   9728 x 2560 (2^24.6)   14.5 16.1     17.1 16.2     16.5 14.9     20.3 16.9
//   32000 x 8192 (2^28)    68.7 66.2     79.3 66.3     74.7 61.0    125.5 88.6
bool q4_stages_x(int64_t rows, int64_t cols, int64_t tokens, int64_t ldx, int dtype, const void* x) {
  if (dtype == EXTERND_F32) return tokens > 5;   // five tokens fill a slot tile, which splits them itself
  return cols % 8 != 0 || ldx % 8 != 0 || (reinterpret_cast<uintptr_t>(x) & 15) != 0 ||
         (tokens > 16 && rows * cols >= (int64_t)1 << 24);
}

static int64_t stage_slots(int64_t tokens, int dtype) {
  return (dtype == EXTERND_F32 ? (tokens + 4) / 5 : (tokens + 15) / 16) * 16;
}
size_t q4_stage_bytes(int64_t cols, int64_t tokens, int dtype) {
  return (size_t)(chunks_of(cols) * kChunk * stage_slots(tokens, dtype)) * 2;
}

hipError_t run_q4_apply(const externd_q4* w, int mats, const void* x, int64_t tokens, int64_t ldx, int dtype, int act,
                        void* y, void* ws, hipStream_t s) {
  Q4Args a;
  for (int q = 0; q < 2; ++q) {
    const externd_q4& m = w[q < mats ? q : 0];
    a.codes[q] = reinterpret_cast<const u32x4*>(m.codes);
    a.scales[q] = m.scales;
    a.mins[q] = m.mins;
  }
  a.rows = w[0].rows;
  a.cols = w[0].cols;
  a.chunks = chunks_of(a.cols);
  a.tokens = tokens;
  a.pieces = dtype == EXTERND_F32 ? 3 : 1;
  a.act = act;
  a.y = y;
  a.staged = ws != nullptr;
  a.x32 = nullptr;
  if (ws) {
    const int64_t items = a.chunks * 16 * stage_slots(tokens, dtype);
    const dim3 grid((unsigned)std::min<int64_t>((items + 255) / 256, 1 << 16));
    u32x4* o = static_cast<u32x4*>(ws);
    if (dtype == EXTERND_F32)
      hipLaunchKernelGGL(k_q4_stage_x<EXTERND_F32>, grid, dim3(256), 0, s, x, tokens, a.cols, ldx, 4 * a.chunks, items, o);
    else
      hipLaunchKernelGGL(k_q4_stage_x<EXTERND_BF16>, grid, dim3(256), 0, s, x, tokens, a.cols, ldx, 4 * a.chunks, items, o);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    a.x = reinterpret_cast<const uint16_t*>(o);
    a.ldx = 0;
    a.slice = 64 * 8;
  } else {
    a.x = static_cast<const uint16_t*>(x);
    if (dtype == EXTERND_F32) a.x32 = static_cast<const float*>(x);
    a.ldx = ldx;
    a.slice = 32;
  }
  const int gpc = kChunk / w[0].group;
  return dtype == EXTERND_F16 ? q4_product_f16(a, gpc, mats, EXTERND_F16, s) : q4_product_bf16(a, gpc, mats, dtype, s);
}

template <int DT>
static hipError_t launch_quantize(const void* W, int64_t rows, int64_t cols, int64_t ldw, int group, void* codes,
                                  uint16_t* scales, uint16_t* mins, hipStream_t s) {
  const int64_t jobs = jobs_of(rows, cols), chunks = chunks_of(cols);
  const dim3 grid = jobs_grid(jobs), block(256);
  u32x4* c = static_cast<u32x4*>(codes);
#define EXTERND_Q4_QUANT(GPC)                                                                                        \
  if (mins)                                                                                                          \
    hipLaunchKernelGGL((k_q4_quantize<DT, GPC, true>), grid, block, 0, s, W, rows, cols, ldw, chunks, jobs, c, scales, mins); \
  else                                                                                                               \
    hipLaunchKernelGGL((k_q4_quantize<DT, GPC, false>), grid, block, 0, s, W, rows, cols, ldw, chunks, jobs, c, scales, mins)
  if (group == 32) { EXTERND_Q4_QUANT(4); }
  else if (group == 64) { EXTERND_Q4_QUANT(2); }
  else { EXTERND_Q4_QUANT(1); }
#undef EXTERND_Q4_QUANT
  return hipGetLastError();
}

hipError_t run_q4_quantize(const void* W, int64_t rows, int64_t cols, int64_t ldw, int dtype, int group, void* codes,
                           uint16_t* scales, uint16_t* mins, hipStream_t s) {
  if (dtype == EXTERND_F32) return launch_quantize<EXTERND_F32>(W, rows, cols, ldw, group, codes, scales, mins, s);
  if (dtype == EXTERND_BF16) return launch_quantize<EXTERND_BF16>(W, rows, cols, ldw, group, codes, scales, mins, s);
  return launch_quantize<EXTERND_F16>(W, rows, cols, ldw, group, codes, scales, mins, s);
}

hipError_t run_q4_pack(const uint8_t* src, const uint16_t* ssrc, const uint16_t* msrc, int64_t rows, int64_t cols,
                       int group, void* codes, uint16_t* scales, uint16_t* mins, hipStream_t s) {
  const int64_t jobs = jobs_of(rows, cols);
  hipLaunchKernelGGL(k_q4_pack, jobs_grid(jobs), dim3(256), 0, s, src, ssrc, msrc, rows, cols,
                     kChunk / group, chunks_of(cols), jobs, static_cast<u32x4*>(codes), scales, mins);
  return hipGetLastError();
}

hipError_t run_q4_reconstruct(const externd_q4& w, int dtype, void* out, hipStream_t s) {
  const int64_t jobs = jobs_of(w.rows, w.cols);
  const dim3 grid = jobs_grid(jobs), block(256);
  const u32x4* c = reinterpret_cast<const u32x4*>(w.codes);
  const int gpc = kChunk / w.group;
#define EXTERND_Q4_RECON(DT)                                                                                          \
  hipLaunchKernelGGL(k_q4_reconstruct<DT>, grid, block, 0, s, c, w.scales, w.mins, w.rows, w.cols, gpc, chunks_of(w.cols), \
                     jobs, out)
  if (dtype == EXTERND_F32) EXTERND_Q4_RECON(EXTERND_F32);
  else if (dtype == EXTERND_BF16) EXTERND_Q4_RECON(EXTERND_BF16);
  else EXTERND_Q4_RECON(EXTERND_F16);
#undef EXTERND_Q4_RECON
  return hipGetLastError();
}

}  // namespace externd
