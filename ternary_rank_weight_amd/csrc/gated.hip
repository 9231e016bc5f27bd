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
#include "pad.hpp"
#include "slopes.hpp"

namespace externd {

namespace {

hipError_t product(GatedProduct mode, const GatedGemm& g, const GatedPlan& plan, float* part, bool bf, int cus,
                   hipStream_t s) {
  return bf ? gated_product_bf16(mode, g, plan, part, cus, s) : gated_product_f16(mode, g, plan, part, cus, s);
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
  PadArgs q = {};
  const int64_t ldp = padded(a.cols, kBK);
  q.src[0] = o->x; q.src[1] = o->wg; q.src[2] = o->wu;
  q.rows[0] = a.tokens; q.rows[1] = q.rows[2] = a.rows;
  q.ld[0] = a.ldx; q.ld[1] = q.ld[2] = a.ldw;
  for (int w = 0; w < 3; ++w) {
    q.cols[w] = a.cols;
    q.ldp[w] = ldp;
    q.dst[w] = ws;
    ws += q.rows[w] * ldp;
  }
  hipLaunchKernelGGL(k_pad_rows, dim3(blocks(std::max(a.tokens, a.rows) * (ldp / 8)), 3), dim3(256), 0, s, q);
  *o = {q.dst[0], q.dst[1], q.dst[2], ldp, ldp, ldp};
  return hipGetLastError();
}
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
    hipLaunchKernelGGL(k_gated_tops<>, dim3((unsigned)(ceil_div64(a.tokens, strip) * strips)), dim3(256), 0, s, sa, ldd,
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
