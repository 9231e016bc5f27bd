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
#include <algorithm>
#include <type_traits>

#include "activation.hpp"
#include "device_common.hpp"
#include "frag.hpp"
#include "gated.hpp"
#include "kernels.hpp"

namespace externd {

namespace {

// dg and du in rows of ldd entries (a multiple of 8; zero past the hidden width), each
// in two parts of the operands' type: the rounded value, and `rest` entries further on
// what the rounding took away.  Bound by HBM: reads 4 + 4 + 2 bytes, writes
// 4 + 4 per hidden unit and token.  VEC: rows of all inputs are 16-byte aligned.
template <bool BF, bool VEC>
__global__ __launch_bounds__(256) void k_gated_slopes(const float* __restrict__ g, const float* __restrict__ u,
                                                       const uint16_t* __restrict__ dh, int64_t tokens, int64_t hidden,
                                                       int64_t lddh, int64_t ldd, int act, int64_t rest,
                                                       uint16_t* __restrict__ dg, uint16_t* __restrict__ du) {
  const int64_t per = ldd / 8, total = tokens * per;
  auto run = [&](auto kind) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
      const int64_t t = i / per, c = (i - t * per) * 8, at = t * hidden + c;
      float gv[8], uv[8], d[8];
      if constexpr (VEC) {   // hidden is a multiple of 8 here
        const u32x4 dv = *reinterpret_cast<const u32x4*>(dh + t * lddh + c);
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const f32x4 a = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(g + at + e));
          const f32x4 b = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(u + at + e));
#pragma unroll
          for (int f = 0; f < 4; ++f) { gv[e + f] = a[f]; uv[e + f] = b[f]; }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = f32_from_16<BF>((dv[e / 2] >> (16 * (e & 1))) & 0xffffu);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const bool ok = c + e < hidden;
          gv[e] = ok ? g[at + e] : 0.f;
          uv[e] = ok ? u[at + e] : 0.f;
          d[e] = ok ? f32_from_16<BF>(dh[t * lddh + c + e]) : 0.f;
        }
      }
      u32x4 og, ou, rg, ru;
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        uint32_t wg[2], wu[2], lg[2], lu[2];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          float a, slope;
          act_both_fast<decltype(kind)::value>(gv[e + f], a, slope);
          const float vg = d[e + f] * uv[e + f] * slope, vu = d[e + f] * a;
          wg[f] = f32_to_16<BF>(vg);
          wu[f] = f32_to_16<BF>(vu);
          const float tg = vg - f32_from_16<BF>(wg[f]), tu = vu - f32_from_16<BF>(wu[f]);
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
  };
  if (act == EXTERND_ACT_SILU) run(std::integral_constant<int, EXTERND_ACT_SILU>());
  else if (act == EXTERND_ACT_GELU) run(std::integral_constant<int, EXTERND_ACT_GELU>());
  else run(std::integral_constant<int, EXTERND_ACT_GELU_TANH>());
}

// Zero outputs (a weight gradient of no tokens).
__global__ void k_fill_u16(uint16_t* __restrict__ p, int64_t n) {
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

int64_t padded(int64_t n, int64_t to) { return ceil_div64(n, to) * to; }
unsigned blocks(int64_t items) { return (unsigned)std::max<int64_t>(1, std::min<int64_t>(ceil_div64(items, 256), 1 << 15)); }

// How a product of m x n outputs (forward: n hidden units; dW: m rows of each of
// the two gradients) over `steps` steps is run: the least of an estimate in
// microseconds, from K = 2560 and F = 9728.
//   big   256 x 256 tiles, one workgroup a CU: 1.4 us a step and 6 a tile;
//   pair  128 x 128 tiles, two a CU: 0.95 us a step and 4 a tile each;
//   deep  128 x 128 tiles, one a CU with loads three steps ahead, where there are
//         no more units than CUs: 0.45 us a step and 8 in all.
// A split costs its sums' way to memory and back.
int64_t tiles_of(int mode, int64_t m, int64_t n, bool big) {
  const int64_t b = big ? 256 : 128;
  return (mode == kDw ? 2 : 1) * ceil_div64(m, b) * ceil_div64(n, mode == kFwd ? b / 2 : b);
}
GatedPlan plan_of(int mode, int64_t m, int64_t n, int64_t steps, int cus) {
  GatedPlan best = {kPair, 1};
  double least = 1e300;
  for (const GatedKind kind : {kBig, kPair, kDeep}) {
    const int64_t tiles = tiles_of(mode, m, n, kind == kBig);
    // (dx is split at 256 x 256 too: its contraction is the longest and its tiles the fewest)
    const int64_t most = kind == kDeep || (kind == kBig && mode == kDx) ? 16 : 1;
    for (int64_t splits = 1; splits <= most && splits <= std::max<int64_t>(1, steps / 4); ++splits) {
      const int64_t units = tiles * splits;
      if (kind == kDeep && units > cus) break;
      const double per = (double)ceil_div64(std::max<int64_t>(steps, 1), splits);
      const double rounds = (double)ceil_div64(units, (int64_t)cus * (kind == kPair ? 2 : 1));
      double us = kind == kBig ? rounds * (per * 1.4 + 6.0) : kind == kPair ? rounds * (per * 0.95 + 4.0) : per * 0.45 + 8.0;
      if (splits > 1) us += 4.0 + (double)(mode == kDx ? 1 : 2) * (double)m * (double)n * 4.0 * (double)(splits * 2) / 4e6;
      if (us < least) {
        least = us;
        best = {kind, splits};
      }
    }
  }
  return best;
}
int64_t steps_of(int64_t inner) { return inner / kBK; }

// dx.  For few tokens the two parts of dg and du are stacked as twice the rows, which are
// added at the end: a 128-row tile has room for both, so the second costs no matrix
// instruction.  Otherwise they follow each other in the contraction.
GatedPlan plan_dx(int64_t tokens, int64_t cols, int64_t rows, int cus) {
  const bool stack = tokens <= 64 && tiles_of(kDx, 2 * tokens, cols, false) <= cus;
  GatedPlan p = plan_of(kDx, stack ? 2 * tokens : tokens, cols, (stack ? 2 : 4) * steps_of(rows), cus);
  if (stack) {
    if (p.kind != kDeep) p = {kDeep, 1};
    p.stacked = 2;
  }
  return p;
}
GatedPlan plan_dw(int64_t tokens, int64_t cols, int64_t rows, int cus) {
  return plan_of(kDw, rows, cols, 2 * steps_of(tokens), cus);
}
int64_t part_floats(int mode, int64_t m, int64_t n, const GatedPlan& p) {
  return p.splits * p.stacked > 1 ? p.splits * p.stacked * (mode == kDx ? 1 : 2) * m * n : 0;
}

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

// Workspace: dg and du, padded copies unless aligned, then the split sums.
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
  return region(2 * (size_t)(4 * tokens * padded(rows, 8))) +
         (aligned ? 0 : region(2 * (size_t)copy_entries(tokens, cols, rows))) +
         region(4 * (size_t)std::max(part_floats(kDx, tokens, cols, px), part_floats(kDw, rows, cols, pw)));
}

hipError_t run_gated_backward(const GatedArgs& a, void* ws, hipStream_t s) {
  const bool bf = a.dtype == EXTERND_BF16;
  hipError_t e;
  if (a.tokens == 0) {
    for (void* w : {a.dwg, a.dwu}) {
      if (!w) continue;
      hipLaunchKernelGGL(k_fill_u16, dim3(1024), dim3(256), 0, s, static_cast<uint16_t*>(w), a.rows * a.cols);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    return hipSuccess;
  }
  // dg, its rest, du, its rest
  const int64_t ldd = padded(a.rows, 8), part_len = a.tokens * ldd;
  char* w = static_cast<char*>(ws);
  uint16_t *dg = reinterpret_cast<uint16_t*>(w), *du = dg + 2 * part_len;
  w += region(2 * (size_t)(4 * part_len));
  {
    const bool vec = a.rows % 8 == 0 && a.lddh % 8 == 0 &&
                     ((reinterpret_cast<uintptr_t>(a.dh) | reinterpret_cast<uintptr_t>(a.g) |
                       reinterpret_cast<uintptr_t>(a.u)) & 15) == 0;
    const dim3 grid(blocks(a.tokens * (ldd / 8))), block(256);
    auto run = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, grid, block, 0, s, a.g, a.u, static_cast<const uint16_t*>(a.dh), a.tokens, a.rows,
                         a.lddh, ldd, a.act, part_len, dg, du);
    };
    if (bf) vec ? run(k_gated_slopes<true, true>) : run(k_gated_slopes<true, false>);
    else vec ? run(k_gated_slopes<false, true>) : run(k_gated_slopes<false, false>);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  Operands o;
  if ((e = operands(a, reinterpret_cast<uint16_t*>(w), &o, s)) != hipSuccess) return e;
  if (needs_copies(a)) w += region(2 * (size_t)copy_entries(a.tokens, a.cols, a.rows));
  float* part = reinterpret_cast<float*>(w);
  const int64_t cols8 = padded(a.cols, 8);
  if (a.dx) {
    const GatedPlan px = plan_dx(a.tokens, a.cols, a.rows, a.cus);
    GatedGemm g = {};
    g.a = {{dg, dg}, ldd, px.stacked * a.tokens};
    g.b = {{o.wg, o.wu}, o.ldw, cols8};
    g.segs = px.stacked == 2 ? 2 : 4;   // stacked: a segment's rows are both parts
    g.rest = px.stacked * part_len;
    g.inner = a.rows;
    g.out[0] = static_cast<uint16_t*>(a.dx);
    g.mo = px.stacked * a.tokens;
    g.ldo = a.cols;
    if ((e = product(kDx, g, px, part, bf, a.cus, s)) != hipSuccess) return e;
  }
  if (a.dwg) {
    GatedGemm g = {};
    g.a = {{dg, du}, ldd, ldd};
    g.b = {{o.x, o.x}, o.ldx, cols8};
    g.segs = 2;
    g.rest = part_len;
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
