// The gated feed-forward block: g = x Wg^T, u = x Wu^T, h = act(g) u in one
// kernel, and its backward pass
//   dg = dh u act'(g), du = dh act(g)           (one pass over T x F)
//   dx = dg Wg + du Wu                          (one product over 4 F)
//   dWg = dg^T x, dWu = du^T x                  (one launch, over 2 T)
// for T tokens, K columns (the model's width) and F rows of each weight
// matrix (the hidden width).
//
// All products are one tiled kernel on the bf16/fp16 matrix instructions with
// fp32 sums, k_gated_gemm (gated_gemm.hpp), in three forms that differ in where an
// operand's entries lie along the contraction: neighbours in a row ("rows", forward),
// or one per row ("cols": both operands of dW, the weights of dx), which is read
// from LDS with the transposing 64-bit read.  Both weight matrices share a
// forward tile, gate and up rows of the same hidden units, so that the
// activation and the product are done on the accumulators and neither g nor u
// goes to memory unless the caller keeps them for the backward pass.  They are
// kept in fp32, and dg and du are held in two 16-bit parts each, the rounded value and
// what the rounding took away, which the products take one after the other: the
// gradients then see no rounding to 16 bits but their own.  (With the rounded
// dg and du alone the products take half the matrix instructions and the
// gradients have 1.4 times the error, for few tokens more: a few roundings decide there.)
// In fp16 they are scaled by powers of two, which the sums are divided by again.
#include <algorithm>
#include <type_traits>

#include "activation.hpp"
#include "device_common.hpp"
#include "frag.hpp"
#include "gated.hpp"
#include "kernels.hpp"

namespace externd {

namespace {

struct SlopeArgs {
  const float *g, *u;    // tokens x hidden
  const uint16_t* dh;    // rows lddh apart
  int64_t tokens, hidden, lddh;
};

// dg and du of token t, hidden units c .. c + 7 (0 past the hidden width).  ONCE: g and u are
// not read again soon.
template <bool BF, int ACT, bool ONCE>
__device__ __forceinline__ void slopes_at(const SlopeArgs& a, int64_t t, int64_t c, float (&vg)[8], float (&vu)[8]) {
  typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
  const int64_t at = t * a.hidden + c, left = a.hidden - c;
  const uint16_t* q = a.dh + t * a.lddh + c;
  float gv[8], uv[8];
  u32x4 d;
  if (left >= 8) {
    d = (reinterpret_cast<uintptr_t>(q) & 15) == 0 ? load8<true>(q) : load8<false>(q);
    auto take = [](const float* p) {
      if constexpr (ONCE) return __builtin_nontemporal_load(reinterpret_cast<const f32x4_a4*>(p));
      else return *reinterpret_cast<const f32x4_a4*>(p);
    };
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
      const f32x4 x = take(a.g + at + e), y = take(a.u + at + e);
#pragma unroll
      for (int f = 0; f < 4; ++f) { gv[e + f] = x[f]; uv[e + f] = y[f]; }
    }
  } else {
    // (dg and du are 0 past the end: dh is)
    const int last = (int)max<int64_t>(left, 1) - 1;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      gv[e] = left > 0 ? a.g[at + min(e, last)] : 0.f;
      uv[e] = left > 0 ? a.u[at + min(e, last)] : 0.f;
    }
    d = load8_part(q, left);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e >= left) gv[e] = uv[e] = 0.f;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float v, slope;
    act_both_fast<ACT>(gv[e], v, slope);
    const float dv = f32_from_16<BF>((d[e / 2] >> (16 * (e & 1))) & 0xffffu);
    vg[e] = dv * uv[e] * slope;
    vu[e] = dv * v;
  }
}

template <typename F>
__device__ __forceinline__ void with_act(int act, F&& run) {
  if (act == EXTERND_ACT_SILU) run(std::integral_constant<int, EXTERND_ACT_SILU>());
  else if (act == EXTERND_ACT_GELU) run(std::integral_constant<int, EXTERND_ACT_GELU>());
  else run(std::integral_constant<int, EXTERND_ACT_GELU_TANH>());
}

// fp16 has neither the range of dg and du (a finite gradient can come from a dg past 65504)
// nor that of small ones.  So each is multiplied by a power of two before it is rounded,
// which the products take back on their fp32 sums: the row of an output has a power of its own,
// from the largest finite dg or du that enters it (by token for dx, by hidden unit for
// each weight gradient), and no token or unit loses bits to another.  (bf16 has
// fp32's range and needs none of this.)  These are the largest magnitudes, as the bits of
// fp32: by token (of both dg and du), by hidden unit of dg and ldd entries on of du; zero before.
// One block: `strip` tokens x 256 hidden units, fewer where there would be few blocks (777 x 1001
// with 64: 52 blocks).  Bound by HBM: reads 4 + 4 + 2 bytes per unit and token; 41 us for
// 2048 x 9728, 7 us for 777 x 1001.
__global__ __launch_bounds__(256) void k_gated_tops(SlopeArgs a, int64_t ldd, int act, int strip,
                                                     uint32_t* __restrict__ by_token, uint32_t* __restrict__ by_unit) {
  constexpr int UNITS = 256;
  __shared__ float col[2][8][UNITS];
  const int piece = threadIdx.x & 31, line = threadIdx.x >> 5;   // 8 units; every eighth token
  const int64_t strips = (a.hidden + UNITS - 1) / UNITS;
  const int64_t t0 = (int64_t)blockIdx.x / strips * strip, c0 = (int64_t)blockIdx.x % strips * UNITS, c = c0 + 8 * piece;
  float top_g[8], top_u[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) top_g[e] = top_u[e] = 0.f;
  auto size = [](float v) { return __builtin_isfinite(v) ? fabsf(v) : 0.f; };
  with_act(act, [&](auto kind) {
    for (int64_t t = t0 + line; t < min(t0 + strip, a.tokens); t += 8) {
      float vg[8], vu[8], most = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) vg[e] = vu[e] = 0.f;
      if (c < a.hidden) slopes_at<false, decltype(kind)::value, false>(a, t, c, vg, vu);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        top_g[e] = fmaxf(top_g[e], size(vg[e]));
        top_u[e] = fmaxf(top_u[e], size(vu[e]));
        most = fmaxf(most, fmaxf(size(vg[e]), size(vu[e])));
      }
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) most = fmaxf(most, __shfl_xor(most, w, 32));
      if (piece == 0) atomicMax(by_token + t, __float_as_uint(most));
    }
  });
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    col[0][line][8 * piece + e] = top_g[e];
    col[1][line][8 * piece + e] = top_u[e];
  }
  __syncthreads();
  const int64_t unit = c0 + threadIdx.x;
  if (unit >= a.hidden) return;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    float most = 0.f;
#pragma unroll
    for (int l = 0; l < 8; ++l) most = fmaxf(most, col[q][l][threadIdx.x]);
    atomicMax(by_unit + q * ldd + unit, __float_as_uint(most));
  }
}

// dg and du in rows of ldd entries (a multiple of 8; zero past the hidden width), each
// in two parts of the operands' type: the rounded value, and `rest` entries further on
// what the rounding took away.  Bound by HBM: reads 4 + 4 + 2 bytes, writes
// 4 + 4 per hidden unit and token; 62 us for 2048 x 9728 (5.8 TB/s: part of what
// it writes stays in the last-level cache).  fp16: scaled by the power of two that
// k_gated_tops' bits give for the token, or for the hidden unit of dg and of du (the other null).
template <bool BF>
__global__ __launch_bounds__(256) void k_gated_slopes(SlopeArgs a, int64_t ldd, int act, int64_t rest,
                                                       const uint32_t* __restrict__ by_token,
                                                       const uint32_t* __restrict__ by_unit,
                                                       uint16_t* __restrict__ dg, uint16_t* __restrict__ du) {
  const int64_t per = ldd / 8, total = a.tokens * per;
  with_act(act, [&](auto kind) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
      const int64_t t = i / per, c = (i - t * per) * 8;
      float vg[8], vu[8];
      slopes_at<BF, decltype(kind)::value, BF>(a, t, c, vg, vu);
      if constexpr (!BF) {
        const float all = by_token ? scale_of(by_token[t]) : 0.f;
        u32x4 tg[2], tu[2];
        if (!by_token) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            tg[h] = *reinterpret_cast<const u32x4*>(by_unit + c + 4 * h);
            tu[h] = *reinterpret_cast<const u32x4*>(by_unit + ldd + c + 4 * h);
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          vg[e] *= by_token ? all : scale_of(tg[e / 4][e & 3]);
          vu[e] *= by_token ? all : scale_of(tu[e / 4][e & 3]);
        }
      }
      u32x4 og, ou, rg, ru;
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        uint32_t wg[2], wu[2], lg[2], lu[2];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          wg[f] = f32_to_16<BF>(vg[e + f]);
          wu[f] = f32_to_16<BF>(vu[e + f]);
          const float tg = vg[e + f] - f32_from_16<BF>(wg[f]), tu = vu[e + f] - f32_from_16<BF>(wu[f]);
          lg[f] = __builtin_isfinite(tg) ? f32_to_16<BF>(tg) : 0u;   // (infinite and NaN are in the first part)
          lu[f] = __builtin_isfinite(tu) ? f32_to_16<BF>(tu) : 0u;
        }
        og[e / 2] = wg[0] | (wg[1] << 16);
        ou[e / 2] = wu[0] | (wu[1] << 16);
        rg[e / 2] = lg[0] | (lg[1] << 16);
        ru[e / 2] = lu[0] | (lu[1] << 16);
      }
      *reinterpret_cast<u32x4*>(dg + t * ldd + c) = og;
      *reinterpret_cast<u32x4*>(du + t * ldd + c) = ou;
      *reinterpret_cast<u32x4*>(dg + rest + t * ldd + c) = rg;
      *reinterpret_cast<u32x4*>(du + rest + t * ldd + c) = ru;
    }
  });
}

// Zeros: a weight gradient of no tokens, and k_gated_tops' results before it.
template <typename T>
__global__ void k_fill_zero(T* __restrict__ p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x)
    p[i] = 0;
}

// Up to three matrices of 16-bit entries copied into rows of ldp entries (a
// multiple of 64), zero past their columns: what the 16-byte loads need where
// the caller's rows are not aligned.  (Reading such rows through registers in every
// step instead took 83 us for the forward of 777 tokens at 1001 x 1237; the copies
// take 5 us, and the forward on them 24.)
struct PadArgs {
  const uint16_t* src[3];
  uint16_t* dst[3];
  int64_t rows[3], ld[3];
  int64_t cols, ldp;
};
__global__ __launch_bounds__(256) void k_pad_rows(PadArgs a) {
  const int w = blockIdx.y;
  const int64_t per = a.ldp / 8, total = a.rows[w] * per;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / per, c = (i - row * per) * 8, left = a.cols - c;
    const uint16_t* p = a.src[w] + row * a.ld[w] + c;
    const u32x4 v = left >= 8 ? load8<false>(p) : load8_part(p, left);
    *reinterpret_cast<u32x4*>(a.dst[w] + row * a.ldp + c) = v;
  }
}

unsigned blocks(int64_t items) { return (unsigned)std::max<int64_t>(1, std::min<int64_t>(ceil_div64(items, 256), 1 << 15)); }

hipError_t product(GatedProduct mode, const GatedGemm& g, const GatedPlan& plan, float* part, bool bf, int cus,
                   hipStream_t s) {
  return bf ? gated_product_bf16(mode, g, plan, part, cus, s) : gated_product_f16(mode, g, plan, part, cus, s);
}

bool rows_aligned(const void* p, int64_t ld) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 8 == 0 && ld < (1 << 22);
}

// x, Wg and Wu as the products can read them: the caller's, or padded copies in
// the workspace.
struct Operands {
  const uint16_t *x, *wg, *wu;
  int64_t ldx, ldw, cols;   // cols: padded, when copied
};
bool needs_copies(const GatedArgs& a) {
  return !rows_aligned(a.x, a.ldx) || !rows_aligned(a.wg, a.ldw) || !rows_aligned(a.wu, a.ldw) || a.cols % 8 != 0;
}
int64_t copy_entries(int64_t tokens, int64_t cols, int64_t rows) { return (tokens + 2 * rows) * padded(cols, kBK); }
hipError_t operands(const GatedArgs& a, uint16_t* ws, Operands* o, hipStream_t s) {
  *o = {static_cast<const uint16_t*>(a.x), static_cast<const uint16_t*>(a.wg), static_cast<const uint16_t*>(a.wu),
        a.ldx, a.ldw, a.cols};
  if (!needs_copies(a)) return hipSuccess;
  PadArgs q;
  q.cols = a.cols;
  q.ldp = padded(a.cols, kBK);
  q.src[0] = o->x; q.src[1] = o->wg; q.src[2] = o->wu;
  q.rows[0] = a.tokens; q.rows[1] = q.rows[2] = a.rows;
  q.ld[0] = a.ldx; q.ld[1] = q.ld[2] = a.ldw;
  for (int w = 0; w < 3; ++w) {
    q.dst[w] = ws;
    ws += q.rows[w] * q.ldp;
  }
  hipLaunchKernelGGL(k_pad_rows, dim3(blocks(std::max(a.tokens, a.rows) * (q.ldp / 8)), 3), dim3(256), 0, s, q);
  *o = {q.dst[0], q.dst[1], q.dst[2], q.ldp, q.ldp, q.ldp};
  return hipGetLastError();
}
size_t region(size_t bytes) { return (bytes + 255) / 256 * 256; }

}  // namespace

bool gated_is_aligned(const GatedArgs& a) { return !needs_copies(a); }

// Workspace.  Forward: padded copies unless aligned, then the split sums.  Backward: dg and du,
// the largest magnitudes, then as the forward.
size_t gated_forward_workspace_bytes(int64_t tokens, int64_t cols, int64_t rows, bool aligned, int cus) {
  if (gated_takes_rows(tokens, cols, rows, aligned, cus)) return 0;
  const GatedPlan p = plan_of(kFwd, tokens, rows, steps_of(padded(cols, kBK)), cus);
  return (aligned ? 0 : region(2 * (size_t)copy_entries(tokens, cols, rows))) +
         region(4 * (size_t)part_floats(kFwd, tokens, rows, p));
}

hipError_t run_gated_forward(const GatedArgs& a, void* ws, hipStream_t s) {
  if (gated_takes_rows(a.tokens, a.cols, a.rows, gated_is_aligned(a), a.cus)) return run_gated_rows(a, s);
  const bool bf = a.dtype == EXTERND_BF16;
  char* w = static_cast<char*>(ws);
  Operands o;
  hipError_t e = operands(a, reinterpret_cast<uint16_t*>(w), &o, s);
  if (e != hipSuccess) return e;
  if (needs_copies(a)) w += region(2 * (size_t)copy_entries(a.tokens, a.cols, a.rows));
  GatedGemm g = {};
  g.a = {{o.x, o.x}, o.ldx, a.tokens};
  g.b = {{o.wg, o.wu}, o.ldw, a.rows};
  g.segs = 1;
  g.inner = o.cols;
  g.out[0] = static_cast<uint16_t*>(a.h);
  g.mo = a.tokens;
  g.ldo = a.rows;
  g.save[0] = a.g;
  g.save[1] = a.u;
  g.act = a.act;
  const GatedPlan p = plan_of(kFwd, a.tokens, a.rows, steps_of(padded(a.cols, kBK)), a.cus);
  return product(kFwd, g, p, reinterpret_cast<float*>(w), bf, a.cus, s);
}

size_t gated_backward_workspace_bytes(int64_t tokens, int64_t cols, int64_t rows, bool aligned, int cus) {
  const GatedPlan px = plan_dx(tokens, cols, rows, cus), pw = plan_dw(tokens, cols, rows, cus);
  return region(2 * (size_t)(4 * tokens * padded(rows, 8))) + region(4 * (size_t)(tokens + 2 * padded(rows, 8))) +
         (aligned ? 0 : region(2 * (size_t)copy_entries(tokens, cols, rows))) +
         region(4 * (size_t)std::max(part_floats(kDx, tokens, cols, px), part_floats(kDw, rows, cols, pw)));
}

hipError_t run_gated_backward(const GatedArgs& a, void* ws, hipStream_t s) {
  const bool bf = a.dtype == EXTERND_BF16;
  hipError_t e;
  if (a.tokens == 0) {
    for (void* w : {a.dwg, a.dwu}) {
      if (!w) continue;
      hipLaunchKernelGGL(k_fill_zero<uint16_t>, dim3(1024), dim3(256), 0, s, static_cast<uint16_t*>(w), a.rows * a.cols);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    return hipSuccess;
  }
  // dg, its rest, du, its rest
  const int64_t ldd = padded(a.rows, 8), part_len = a.tokens * ldd;
  char* w = static_cast<char*>(ws);
  uint16_t *dg = reinterpret_cast<uint16_t*>(w), *du = dg + 2 * part_len;
  w += region(2 * (size_t)(4 * part_len));
  uint32_t *by_unit = reinterpret_cast<uint32_t*>(w), *by_token = by_unit + 2 * ldd;
  w += region(4 * (size_t)(a.tokens + 2 * ldd));
  const SlopeArgs sa = {a.g, a.u, static_cast<const uint16_t*>(a.dh), a.tokens, a.rows, a.lddh};
  if (!bf) {
    const int64_t strips = ceil_div64(a.rows, 256);
    const int strip = ceil_div64(a.tokens, 64) * strips >= 2 * a.cus ? 64 : 16;
    hipLaunchKernelGGL(k_fill_zero<uint32_t>, dim3(64), dim3(256), 0, s, by_unit, a.tokens + 2 * ldd);
    hipLaunchKernelGGL(k_gated_tops, dim3((unsigned)(ceil_div64(a.tokens, strip) * strips)), dim3(256), 0, s, sa, ldd,
                       a.act, strip, by_token, by_unit);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  // fp16: for dx scaled by token, for the weight gradients by hidden unit
  auto slopes = [&](const uint32_t* token, const uint32_t* unit) {
    const dim3 grid(blocks(a.tokens * (ldd / 8))), block(256);
    if (bf) hipLaunchKernelGGL(k_gated_slopes<true>, grid, block, 0, s, sa, ldd, a.act, part_len, token, unit, dg, du);
    else hipLaunchKernelGGL(k_gated_slopes<false>, grid, block, 0, s, sa, ldd, a.act, part_len, token, unit, dg, du);
    return hipGetLastError();
  };
  Operands o;
  if ((e = operands(a, reinterpret_cast<uint16_t*>(w), &o, s)) != hipSuccess) return e;
  if (needs_copies(a)) w += region(2 * (size_t)copy_entries(a.tokens, a.cols, a.rows));
  float* part = reinterpret_cast<float*>(w);
  const int64_t cols8 = padded(a.cols, 8);
  if (a.dx) {
    if ((e = slopes(by_token, nullptr)) != hipSuccess) return e;
    const GatedPlan px = plan_dx(a.tokens, a.cols, a.rows, a.cus);
    GatedGemm g = {};
    g.a = {{dg, dg}, ldd, px.stacked * a.tokens};
    g.b = {{o.wg, o.wu}, o.ldw, cols8};
    g.segs = px.stacked == 2 ? 2 : 4;   // stacked: a segment's rows are both parts
    g.rest = px.stacked * part_len;
    g.tops = bf ? nullptr : by_token;
    g.inner = a.rows;
    g.out[0] = static_cast<uint16_t*>(a.dx);
    g.mo = px.stacked * a.tokens;
    g.ldo = a.cols;
    if ((e = product(kDx, g, px, part, bf, a.cus, s)) != hipSuccess) return e;
  }
  if (a.dwg) {
    if ((!bf || !a.dx) && (e = slopes(nullptr, by_unit)) != hipSuccess) return e;
    GatedGemm g = {};
    g.a = {{dg, du}, ldd, ldd};
    g.b = {{o.x, o.x}, o.ldx, cols8};
    g.segs = 2;
    g.rest = part_len;
    g.tops = bf ? nullptr : by_unit;
    g.tops_of_up = ldd;
    g.inner = a.tokens;
    g.out[0] = static_cast<uint16_t*>(a.dwg);
    g.out[1] = static_cast<uint16_t*>(a.dwu);
    g.mo = a.rows;
    g.ldo = a.cols;
    const GatedPlan p = plan_dw(a.tokens, a.cols, a.rows, a.cus);
    if ((e = product(kDw, g, p, part, bf, a.cus, s)) != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace externd
