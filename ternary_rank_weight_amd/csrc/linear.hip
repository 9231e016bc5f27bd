// The linear layer: z = x W^T + bias, y = act(z) + residual in one kernel, and its
// backward pass
//   dz = dy act'(z)                       (one pass over T x F; without an activation dz is dy)
//   dx = dz W, dW = dz^T x                (a product each)
//   db = the sum of dz over the tokens    (one pass)
// for T tokens, K columns and F rows of W.  The products are the tiled kernel of the gated block
// (gated_gemm.hpp) in forms of one weight matrix; with an activation dz is held in two 16-bit
// parts as dg and du are there, so that each gradient is rounded once.  That doubles dx and dW: bf16, 2048 tokens at 2560 x
// 9728, silu, the whole backward pass 372 us in two parts and 200 in one, whose dx and dW are off by 2.35e-3 of their
// size instead of 1.66e-3, which rounding them leaves (fp16: 400 and 206 us, 2.9e-4 and 2.1e-4).
#include <algorithm>

#include "activation.hpp"
#include "device_common.hpp"
#include "frag.hpp"
#include "gated.hpp"
#include "linear.hpp"
#include "linear_plan.hpp"
#include "pad.hpp"
#include "slopes.hpp"

namespace externd {

namespace {

// db: sums over the tokens of dz in fp32, in an order that does not depend on timing.  A workgroup takes COLS
// columns, a wave's lanes 64 / COLS tokens of them at a time; the lanes' and the waves' sums are joined in order.
// Fewer columns where more would leave compute units without any (777 tokens at 1001 rows: 15 us with 64, 7 with 16),
// but whole lines of z where there are enough (2048 tokens at 9728 rows, with dz: 74 us with 16, 55 with 32).
constexpr int kSumWaves = 16;
struct BiasArgs {
  const uint16_t* dy;
  const float* z;   // null: without an activation
  uint16_t* db;
  int64_t lddy, tokens, rows;
  int act;
};
template <bool BF, int COLS>
__device__ __forceinline__ void sum_bias(const BiasArgs& a, int64_t block) {
  const uint16_t* __restrict__ const dy = a.dy;
  const float* __restrict__ const z = a.z;
  const int64_t tokens = a.tokens, rows = a.rows, lddy = a.lddy;
  constexpr int LINES = kSumWaves * kWave / COLS;   // tokens that the workgroup takes at once
  constexpr int U = 8;                              // times that on their way
  __shared__ float red[LINES][COLS];
  const int col = threadIdx.x % COLS, line = threadIdx.x / COLS;
  const int64_t c = block * COLS + col, at = min(c, rows - 1);
  float sum[2] = {};
  auto add = [&](auto slope) {
    for (int64_t t0 = line; t0 < tokens; t0 += U * LINES) {
      float d[U], v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t t = min(t0 + u * LINES, tokens - 1);
        d[u] = f32_from_16<BF>(dy[t * lddy + at]);
        v[u] = z ? z[t * rows + at] : 0.f;
      }
      loads_made();
#pragma unroll
      for (int u = 0; u < U; ++u) sum[u & 1] += t0 + u * LINES < tokens ? (z ? d[u] * slope(v[u]) : d[u]) : 0.f;
    }
  };
  if (z)
    with_act(a.act, [&](auto kind) {
      add([](float v) {
        float h, s;
        act_both_fast<decltype(kind)::value>(v, h, s);
        return s;
      });
    });
  else add([](float) { return 1.f; });
  red[line][col] = sum[0] + sum[1];
  __syncthreads();
  for (int n = LINES / 2; n > 0; n /= 2) {
    if (line < n) red[line][col] += red[line + n][col];
    __syncthreads();
  }
  if (line == 0 && c < rows) a.db[c] = (uint16_t)f32_to_16<BF>(red[0][col]);
}

template <bool BF, int COLS>
__global__ __launch_bounds__(kSumWaves * kWave) void k_bias_sums(BiasArgs a) { sum_bias<BF, COLS>(a, blockIdx.x); }

// dz in parts, and db by the first workgroups, which are its slowest: together in the time of the longer, and one
// launch.  777 tokens x 1001, fp16: 9.8 us, apart 6.5 and 6.0.  Bound by HBM with many: 2048 x 9728, bf16, 55 us for
// 320 MB, of which dy and z come twice (apart, with 16 columns: 51 and 31).
struct PartsArgs {
  SlopeArgs s;
  int64_t ldd, rest;
  const uint32_t *by_token, *by_unit;
  uint16_t *dz, *dz_by_unit;
  BiasArgs b;
  int bias_blocks;
};
template <bool BF, int COLS>
__global__ __launch_bounds__(kSumWaves * kWave) void k_linear_parts(PartsArgs a) {
  if ((int)blockIdx.x < a.bias_blocks) sum_bias<BF, COLS>(a.b, blockIdx.x);
  else
    put_slopes<BF, false>(a.s, a.ldd, a.b.act, a.rest, a.by_token, a.by_unit, a.dz, a.dz_by_unit,
                          (int64_t)(blockIdx.x - a.bias_blocks) * blockDim.x + threadIdx.x,
                          (int64_t)(gridDim.x - a.bias_blocks) * blockDim.x);
}

// Columns of db a workgroup takes.
int bias_cols(const LinearArgs& a) { return a.rows >= (int64_t)64 * a.cus ? 64 : a.rows >= (int64_t)32 * a.cus ? 32 : 16; }

hipError_t launch_bias_sums(const LinearArgs& a, const BiasArgs& b, hipStream_t s) {
  const int cols = bias_cols(a);
  const auto kernel = a.dtype == EXTERND_BF16 ? (cols == 64 ? k_bias_sums<true, 64> : cols == 32 ? k_bias_sums<true, 32> : k_bias_sums<true, 16>)
                                              : (cols == 64 ? k_bias_sums<false, 64> : cols == 32 ? k_bias_sums<false, 32> : k_bias_sums<false, 16>);
  hipLaunchKernelGGL(kernel, dim3((unsigned)ceil_div64(a.rows, cols)), dim3(kSumWaves * kWave), 0, s, b);
  return hipGetLastError();
}

hipError_t launch_parts(const LinearArgs& a, PartsArgs q, hipStream_t s) {
  const int cols = bias_cols(a);
  constexpr int THREADS = kSumWaves * kWave;
  q.bias_blocks = a.db ? (int)ceil_div64(a.rows, cols) : 0;
  const int64_t most = std::min<int64_t>(ceil_div64(a.tokens * (q.ldd / 8), THREADS), 1 << 15);
  const auto kernel = a.dtype == EXTERND_BF16 ? (cols == 64 ? k_linear_parts<true, 64> : cols == 32 ? k_linear_parts<true, 32> : k_linear_parts<true, 16>)
                                              : (cols == 64 ? k_linear_parts<false, 64> : cols == 32 ? k_linear_parts<false, 32> : k_linear_parts<false, 16>);
  hipLaunchKernelGGL(kernel, dim3((unsigned)(q.bias_blocks + most)), dim3(THREADS), 0, s, q);
  return hipGetLastError();
}

hipError_t product(GatedProduct mode, const GatedGemm& g, const GatedPlan& plan, float* part, bool bf, int cus,
                   hipStream_t s) {
  return bf ? linear_product_bf16(mode, g, plan, part, cus, s) : linear_product_f16(mode, g, plan, part, cus, s);
}

// x, W and dy as the products can read them: the caller's, or padded copies in the workspace.
struct Operands {
  const uint16_t *x, *w, *dy;
  int64_t ldx, ldw, lddy, cols;   // cols: padded, when copied
};
int64_t copy_entries(int64_t tokens, int64_t cols, int64_t rows) { return (tokens + rows) * padded(cols, kBK); }

// ws: room for the copies of x and W, then of dy.  zeros: words to clear on the way, or null.
hipError_t operands(const LinearArgs& a, bool copy_xw, bool copy_dy, uint16_t* ws, uint32_t* zeros, int64_t zeros_n, Operands* o,
                    hipStream_t s) {
  *o = {static_cast<const uint16_t*>(a.x), static_cast<const uint16_t*>(a.w), static_cast<const uint16_t*>(a.dy),
        a.ldx, a.ldw, a.lddy, a.cols};
  PadArgs q = {};
  int n = 0;
  int64_t most = 0;
  auto copy = [&](const uint16_t*& src, int64_t& ld, int64_t rows, int64_t cols) {
    const int64_t ldp = padded(cols, kBK);
    q.src[n] = src;
    q.dst[n] = ws;
    q.rows[n] = rows;
    q.cols[n] = cols;
    q.ld[n] = ld;
    q.ldp[n++] = ldp;
    src = ws;
    ld = ldp;
    ws += rows * ldp;
    most = std::max(most, rows * (ldp / 8));
  };
  if (copy_xw) {
    copy(o->x, o->ldx, a.tokens, a.cols);
    copy(o->w, o->ldw, a.rows, a.cols);
    o->cols = padded(a.cols, kBK);
  }
  if (copy_dy) copy(o->dy, o->lddy, a.tokens, a.rows);
  if (n == 0) {
    if (!zeros) return hipSuccess;
    hipLaunchKernelGGL(k_fill_zero<uint32_t>, dim3(64), dim3(256), 0, s, zeros, zeros_n);
    return hipGetLastError();
  }
  q.zeros = zeros;
  q.zeros_n = zeros_n;
  hipLaunchKernelGGL(k_pad_rows, dim3(blocks(most), n), dim3(256), 0, s, q);
  return hipGetLastError();
}

}  // namespace

bool linear_is_aligned(const LinearArgs& a) { return rows_aligned(a.x, a.ldx) && rows_aligned(a.w, a.ldw) && a.cols % 8 == 0; }
bool linear_reads_dy(const LinearArgs& a) {
  return a.act == EXTERND_ACT_NONE && rows_aligned(a.dy, a.lddy) && a.rows % 8 == 0;
}

size_t linear_forward_workspace_bytes(int64_t tokens, int64_t cols, int64_t rows, bool aligned, int cus) {
  if (linear_takes_rows(tokens, cols, rows, aligned, cus)) return 0;
  const GatedPlan p = plan_linear(kLin, tokens, rows, steps_of(padded(cols, kBK)), cus);
  return (aligned ? 0 : region(2 * (size_t)copy_entries(tokens, cols, rows))) + region(4 * (size_t)part_floats(kLin, tokens, rows, p));
}

hipError_t run_linear_forward(const LinearArgs& a, void* ws, hipStream_t s) {
  const bool al = linear_is_aligned(a);
  if (linear_takes_rows(a.tokens, a.cols, a.rows, al, a.cus)) return run_linear_rows(a, s);
  char* w = static_cast<char*>(ws);
  Operands o;
  const hipError_t e = operands(a, !al, false, reinterpret_cast<uint16_t*>(w), nullptr, 0, &o, s);
  if (e != hipSuccess) return e;
  if (!al) w += region(2 * (size_t)copy_entries(a.tokens, a.cols, a.rows));
  GatedGemm g = {};
  g.a = {{o.x, o.x}, o.ldx, a.tokens};
  g.b = {{o.w, o.w}, o.ldw, a.rows};
  g.segs = 1;
  g.inner = o.cols;
  g.out[0] = static_cast<uint16_t*>(a.y);
  g.mo = a.tokens;
  g.ldo = a.rows;
  g.save[0] = a.z;
  g.act = a.act;
  g.bias = static_cast<const uint16_t*>(a.bias);
  g.residual = static_cast<const uint16_t*>(a.residual);
  g.ldr = a.ldr;
  const GatedPlan p = plan_linear(kLin, a.tokens, a.rows, steps_of(padded(a.cols, kBK)), a.cus);
  return product(kLin, g, p, reinterpret_cast<float*>(w), a.dtype == EXTERND_BF16, a.cus, s);
}

// Workspace: dz in two parts (fp16: with two scales) and its largest magnitudes where there is an activation,
// padded copies, the split sums.
size_t linear_backward_workspace_bytes(int64_t tokens, int64_t cols, int64_t rows, int act, bool aligned, bool reads_dy, int cus) {
  const bool parts = act != EXTERND_ACT_NONE;
  const GatedPlan px = plan_linear_dx(tokens, cols, rows, parts, cus), pw = plan_linear_dw(tokens, cols, rows, parts, cus);
  return (parts ? region(2 * (size_t)(4 * tokens * padded(rows, 8))) + region(4 * (size_t)(tokens + padded(rows, 8))) : 0) +
         region(2 * (size_t)((aligned ? 0 : copy_entries(tokens, cols, rows)) + (parts || reads_dy ? 0 : tokens * padded(rows, kBK)))) +
         region(4 * (size_t)std::max(part_floats(kDx, tokens, cols, px), part_floats(kLinDw, rows, cols, pw)));
}

hipError_t run_linear_backward(const LinearArgs& a, void* ws, hipStream_t s) {
  const bool bf = a.dtype == EXTERND_BF16, parts = a.act != EXTERND_ACT_NONE;
  hipError_t e;
  if (a.tokens == 0) {
    const struct { void* p; int64_t n; } zero[2] = {{a.dw, a.rows * a.cols}, {a.db, a.rows}};
    for (const auto& z : zero) {
      if (!z.p) continue;
      hipLaunchKernelGGL(k_fill_zero<uint16_t>, dim3(1024), dim3(256), 0, s, static_cast<uint16_t*>(z.p), z.n);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    return hipSuccess;
  }
  const BiasArgs bias = {static_cast<const uint16_t*>(a.dy), parts ? a.z : nullptr, static_cast<uint16_t*>(a.db), a.lddy, a.tokens, a.rows, a.act};
  const bool products = a.dx || a.dw;
  if (a.db && !(parts && products) && (e = launch_bias_sums(a, bias, s)) != hipSuccess) return e;
  if (!products) return hipSuccess;
  char* w = static_cast<char*>(ws);
  // dz and its rest; fp16: scaled by token for dx, and again by row of W for dW
  const int64_t ldd = padded(a.rows, 8), part_len = a.tokens * ldd;
  uint16_t *dz = reinterpret_cast<uint16_t*>(w), *dz_by_unit = bf ? dz : dz + 2 * part_len;
  uint32_t *by_unit = nullptr, *by_token = nullptr;
  const SlopeArgs sa = {a.z, nullptr, static_cast<const uint16_t*>(a.dy), a.tokens, a.rows, a.lddy};
  if (parts) {
    w += region(2 * (size_t)(4 * part_len));
    by_unit = reinterpret_cast<uint32_t*>(w);
    by_token = by_unit + ldd;
    w += region(4 * (size_t)(a.tokens + ldd));
  }
  const bool al = linear_is_aligned(a), reads_dy = linear_reads_dy(a), scaled = parts && !bf;
  Operands o;
  e = operands(a, !al, !parts && !reads_dy, reinterpret_cast<uint16_t*>(w), scaled ? by_unit : nullptr, a.tokens + ldd, &o, s);
  if (e != hipSuccess) return e;
  w += region(2 * (size_t)((al ? 0 : copy_entries(a.tokens, a.cols, a.rows)) + (parts || reads_dy ? 0 : a.tokens * padded(a.rows, kBK))));
  if (parts) {
    if (!bf) {
      const int64_t strips = ceil_div64(a.rows, 256);
      const int strip = ceil_div64(a.tokens, 64) * strips >= 2 * a.cus ? 64 : 16;
      hipLaunchKernelGGL(k_gated_tops<false>, dim3((unsigned)(ceil_div64(a.tokens, strip) * strips)), dim3(256), 0, s, sa, ldd,
                         a.act, strip, by_token, by_unit);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    const PartsArgs q = {sa, ldd, part_len, !bf && a.dx ? by_token : nullptr, !bf && a.dw ? by_unit : nullptr, dz, dz_by_unit, bias, 0};
    if ((e = launch_parts(a, q, s)) != hipSuccess) return e;
  }
  float* part = reinterpret_cast<float*>(w);
  const int64_t cols8 = padded(a.cols, 8);
  const uint16_t* d = parts ? dz : o.dy;
  const int64_t ld = parts ? ldd : o.lddy;
  const GatedPlan px = plan_linear_dx(a.tokens, a.cols, a.rows, parts, a.cus), pw = plan_linear_dw(a.tokens, a.cols, a.rows, parts, a.cus);
  GatedGemm x = {}, y = {};   // dx and dW
  x.a = {{d, d}, ld, px.stacked * a.tokens};
  x.b = {{o.w, o.w}, o.ldw, cols8};
  x.segs = parts && px.stacked == 1 ? 2 : 1;   // stacked: a segment's rows are both parts
  x.rest = part_len;
  x.tops = parts && !bf ? by_token : nullptr;
  x.inner = a.rows;
  x.out[0] = static_cast<uint16_t*>(a.dx);
  x.mo = px.stacked * a.tokens;
  x.ldo = a.cols;
  const uint16_t* const du = parts ? dz_by_unit : d;
  y.a = {{du, du}, ld, ldd};
  y.b = {{o.x, o.x}, o.ldx, cols8};
  y.segs = parts ? 2 : 1;
  y.rest = part_len;
  y.tops = parts && !bf ? by_unit : nullptr;
  y.inner = a.tokens;
  y.out[0] = static_cast<uint16_t*>(a.dw);
  y.mo = a.rows;
  y.ldo = a.cols;
  const LinearJoin j = linear_join(a.tokens, a.cols, a.rows, parts, a.cus);
  if (a.dx && a.dw && j.dx > 0) return (bf ? linear_gradients_bf16 : linear_gradients_f16)(x, y, j.dx, j.dw, j.kind, s);
  if (a.dx && (e = product(kDx, x, px, part, bf, a.cus, s)) != hipSuccess) return e;
  if (a.dw && (e = product(kLinDw, y, pw, part, bf, a.cus, s)) != hipSuccess) return e;
  return hipSuccess;
}

}  // namespace externd
