// k_q4_apply and its dispatch; each including unit instantiates one operand type.
#pragma once
#include <type_traits>

#include "q4.hpp"

namespace externd {

namespace {

// y = W x (MATS = 1) or act(Wg x) (Wu x) (MATS = 2) for tiles of 16 slots.
//
// A workgroup of WV waves takes RT row tiles and NT slot tiles; its waves take
// every WV-th chunk, so neighbouring waves read neighbouring kilobytes, and
// their sums are joined in LDS in wave order (the result does not depend on
// timing).  Per chunk a wave makes four 16x16x32 products per row and slot
// tile, with the slots as rows of the first operand and weight rows as columns
// of the second: D[slot][weight row] then has one weight row per lane, and
// the group's scale is one multiplication by the lane's own value.
//
// The operand is 16 + c, not c - 8 or c: its offset is taken off by a product of x
// with the constant -24 (or -16), made once for all row tiles.  With minima that product, scaled by -m / 16, is also the
// m sum(x) term.  Sums are fp32 throughout.
//
// Bound by the weights' latency for a few tokens: 2560 x 9728 with minima, one token, 9.9 us
// where they come from memory (1.6 TB/s of 160 workgroups; reading 1 GiB: 5.3) and 8.1 where
// three layers of them stay in the last-level cache; gate and up of 9728 x 2560, 10.0 us
// (2.8 TB/s) and 8.6.  (The loads keep what they read in that cache; with nontemporal ones, in a
// graph: 9.2 against 9.6 and 9.5 against 9.9 us from memory, 8.8 against 7.7 and 9.0 against 8.2 from the
// cache.)  With 48 tokens on 32000 x 8192, 50 us (2.8 TB/s, 0.50 PFLOP/s): the matrix instructions take
// 14, unpacking 15, x from L2 15 and the weights 27 us, and the two waves per SIMD that the
// accumulators leave room for overlap them only in part.  Past 64 tokens every four slot
// tiles (fp32: 20 tokens) read and unpack the weights again: 512 tokens on 9728 x 2560,
// 86 us in bf16 (0.30 PFLOP/s), 267 in fp32.
template <bool BF, int GPC, bool MINS, int MATS, int RT, int NT, int WV, int SL, bool X32>
__global__ __launch_bounds__(WV * kWave) void k_q4_apply(Q4Args a, int out_type) {
  constexpr int F = MATS * RT;      // row tiles held by a wave, of all matrices
  constexpr int SPG = 4 / GPC;      // products per group
  constexpr int PF = F * NT <= 4 ? 3 : 2;
  static_assert(!X32 || (BF && NT == 1), "fp32 x is read for one slot tile");
  __shared__ float red[WV][F][64 * SL];
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int r = lane & 15, p = lane >> 4;
  const int64_t tiles = (a.rows + kTile - 1) / kTile;
  const int64_t tile0 = (int64_t)blockIdx.x * RT;
  // slots of a slot tile, and the lane's: operand row r, or r / 4 when only every
  // fourth result row is wanted
  const int per = SL == 1 ? 4 : a.pieces == 3 ? 15 : 16;
  const int64_t slots = a.tokens * a.pieces;
  const int slot = SL == 1 ? r >> 2 : r;

  const uint16_t* xp[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    // a slot (or tile) past the end repeats the last one: its sums are not written
    const int64_t tile = (int64_t)blockIdx.y * NT + n;
    if (a.staged) xp[n] = a.x + min(tile, (slots + per - 1) / per - 1) * a.chunks * (4 * 64 * 8) + lane * 8;
    else xp[n] = a.x + min(tile * 16 + slot, slots - 1) * a.ldx + 8 * p;
  }
  // fp32 x read here: the lane's token, and which of its three parts
  const int64_t last_slot = min<int64_t>(slot, slots - 1);
  const float* xf32 = a.x32 + (X32 ? last_slot / 3 * a.ldx + 8 * p : 0);
  const uint32_t part0 = X32 && last_slot % 3 > 0 ? 0xffff0000u : 0u, part1 = X32 && last_slot % 3 > 1 ? 0xffff0000u : 0u;
  // row tile f's blocks of chunks: the same in all lanes
  const u32x4* cp[F];
  const uint16_t* sp[F];
  const uint16_t* mp[F];
#pragma unroll
  for (int f = 0; f < F; ++f) {
    const int64_t tile = min(tile0 + f % RT, tiles - 1);   // as for slots
    cp[f] = a.codes[f / RT] + tile * a.chunks * kWave;
    sp[f] = a.scales[f / RT] + tile * a.chunks * kTile * GPC;
    if constexpr (MINS) mp[f] = a.mins[f / RT] + tile * a.chunks * kTile * GPC;
  }
  float acc[F][NT][SL];   // result rows 4 p + e, e < SL
#pragma unroll
  for (int f = 0; f < F; ++f)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < SL; ++e) acc[f][n][e] = 0.f;

  struct Stage {
    u32x4 c[F];
    uint64_t s[F], m[F];   // GPC bf16 values in the low bits
  };
  auto table = [](const uint16_t* q) -> uint64_t {
    if constexpr (GPC == 4) return *reinterpret_cast<const uint64_t*>(q);
    else if constexpr (GPC == 2) return *reinterpret_cast<const uint32_t*>(q);
    else return *q;
  };
  auto fetch = [&](int64_t c, Stage& st) {
#pragma unroll
    for (int f = 0; f < F; ++f) {
      st.c[f] = cp[f][c * kWave + lane];
      st.s[f] = table(sp[f] + c * kTile * GPC + r * GPC);
      if constexpr (MINS) st.m[f] = table(mp[f] + c * kTile * GPC + r * GPC);
    }
  };
  constexpr uint32_t off2 = MINS ? (BF ? 0xC180C180u : 0xCC00CC00u) : (BF ? 0xC1C0C1C0u : 0xCE00CE00u);
  const u32x4 off = {off2, off2, off2, off2};
  // x of the four slices of a chunk, on its way one chunk ahead: fp32 as it is,
  // split when it is used
  struct Slice {
    u32x4 v[X32 ? 2 : NT];
  };
  Slice xs[4];
  const int64_t full = a.staged ? a.chunks : a.cols / kChunk;   // chunks without a tail
  auto load_x = [&](int64_t c, int i, bool tail) {   // slice i of chunk c
    if constexpr (X32) {
      const int64_t col = kChunk * c + 32 * i;
      float f[8];
      load_weights<EXTERND_F32>(xf32, col, tail ? a.cols - col - 8 * p : 8, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) xs[i].v[j / 4][j & 3] = __float_as_uint(f[j]);
    } else {
      const int64_t at = (4 * c + i) * a.slice;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (!tail || at + 8 * p < a.cols) xs[i].v[n] = *reinterpret_cast<const u32x4*>(xp[n] + at);
        else xs[i].v[n] = u32x4{0u, 0u, 0u, 0u};   // (only unstaged, where `at` is the column)
      }
    }
  };
  auto operand = [&](int i, int n) {
    if constexpr (X32) {
      u32x4 r;
#pragma unroll
      for (int j = 0; j < 8; j += 2)
        r[j / 2] = third_of(__uint_as_float(xs[i].v[j / 4][j & 3]), part0, part1) |
                   (third_of(__uint_as_float(xs[i].v[j / 4][(j & 3) + 1]), part0, part1) << 16);
      return r;
    } else {
      return xs[i].v[n];
    }
  };
  auto add_group = [&](const Stage& st, int g, int f, const f32x4 (&d)[NT], const f32x4 (&xo)[NT]) {
    const float s = bf16_to_f32((uint32_t)(st.s[f] >> (16 * g)) & 0xffffu);
    const float m = MINS ? -0.0625f * bf16_to_f32((uint32_t)(st.m[f] >> (16 * g)) & 0xffffu) : 0.f;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < SL; ++e) {
        acc[f][n][e] = fmaf(s, d[n][e] + xo[n][e], acc[f][n][e]);
        if constexpr (MINS) acc[f][n][e] = fmaf(m, xo[n][e], acc[f][n][e]);
      }
  };
  constexpr f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  constexpr bool MANY = F * NT >= 8;   // accumulators: products started further ahead would spill them
  // One chunk; the x of chunk cn sets out behind each group (with one group: each slice).  (Without conditions, here
  // and in the loop below: with them the compiler moves the sums behind all
  // groups' products, which then spill.)
  auto work_on = [&](const Stage& st, int64_t cn, auto ahead) {
#pragma unroll
    for (int g = 0; g < GPC; ++g) {
      f32x4 xo[NT];
      if constexpr (SPG <= 2) {
        // one row tile's products after the other's
        u32x4 xf[SPG][NT];
#pragma unroll
        for (int i = 0; i < SPG; ++i)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            xf[i][n] = operand(g * SPG + i, n);
            xo[n] = mfma16<BF>(xf[i][n], off, i ? xo[n] : zero);
          }
#pragma unroll
        for (int f = 0; f < F; ++f) {
          f32x4 d[NT];
#pragma unroll
          for (int i = 0; i < SPG; ++i) {
            const u32x4 wf = unpack_q4<BF>(st.c[f][g * SPG + i]);
#pragma unroll
            for (int n = 0; n < NT; ++n) d[n] = mfma16<BF>(xf[i][n], wf, i ? d[n] : zero);
          }
          add_group(st, g, f, d, xo);
          if constexpr (MANY) __builtin_amdgcn_sched_barrier(0);
        }
      } else {
        // one slice after the other, all row tiles' products in registers
        f32x4 d[F][NT];
#pragma unroll
        for (int i = 0; i < SPG; ++i) {
          u32x4 xf[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            xf[n] = operand(i, n);
            xo[n] = mfma16<BF>(xf[n], off, i ? xo[n] : zero);
          }
#pragma unroll
          for (int f = 0; f < F; ++f) {
            const u32x4 wf = unpack_q4<BF>(st.c[f][i]);
#pragma unroll
            for (int n = 0; n < NT; ++n) d[f][n] = mfma16<BF>(xf[n], wf, i ? d[f][n] : zero);
          }
          if (decltype(ahead)::value) load_x(cn, i, false);
          if constexpr (MANY) __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int f = 0; f < F; ++f) add_group(st, g, f, d[f], xo);
        if constexpr (MANY) __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (SPG <= 2 && decltype(ahead)::value) {
#pragma unroll
        for (int i = 0; i < SPG; ++i) load_x(cn, g * SPG + i, false);
      }
    }
  };
  // PF - 1 chunks of codes are on their way while one is worked on (past the
  // end, the last one again)
  Stage st[PF];
  int64_t c = wave;
  if (c < full) {
#pragma unroll
    for (int u = 0; u < PF - 1; ++u) fetch(min(c + u * WV, full - 1), st[u]);
#pragma unroll
    for (int i = 0; i < 4; ++i) load_x(c, i, false);
#pragma unroll 1
    for (; c < full; c += WV) {
      fetch(min(c + (PF - 1) * WV, full - 1), st[PF - 1]);
      work_on(st[0], min(c + WV, full - 1), std::true_type());
#pragma unroll
      for (int u = 0; u + 1 < PF; ++u) st[u] = st[u + 1];
    }
  }
  if (c < a.chunks) {   // the last chunk, which has a tail
    fetch(c, st[0]);
#pragma unroll
    for (int i = 0; i < 4; ++i) load_x(c, i, true);
    work_on(st[0], 0, std::false_type());
  }

  const int rows_here = (int)min<int64_t>(RT * kTile, a.rows - tile0 * kTile);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    if (n) __syncthreads();
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
      for (int e = 0; e < SL; ++e) red[wave][f][(SL * p + e) * kTile + r] = acc[f][n][e];
    __syncthreads();
    const int64_t tok0 = ((int64_t)blockIdx.y * NT + n) * (per / a.pieces);
    for (int o = threadIdx.x; o < RT * 256; o += WV * kWave) {
      const int f = o >> 8, tk = (o >> 4) & 15, row = o & 15;
      if (tk >= per / a.pieces || tok0 + tk >= a.tokens || f * kTile + row >= rows_here) continue;
      float v[MATS];
#pragma unroll
      for (int q = 0; q < MATS; ++q) {
        float sum = 0.f;
        for (int e = 0; e < a.pieces; ++e)
#pragma unroll
          for (int w = 0; w < WV; ++w) sum += red[w][q * RT + f][(tk * a.pieces + e) * kTile + row];
        v[q] = sum;
      }
      float out = v[0];
      if constexpr (MATS == 2) out = act_value(a.act, v[0]) * v[1];
      const int64_t at = (tok0 + tk) * a.rows + (tile0 + f) * kTile + row;
      if (out_type == EXTERND_F32) static_cast<float*>(a.y)[at] = out;
      else static_cast<uint16_t*>(a.y)[at] = (uint16_t)f32_to_16<BF>(out);
    }
  }
}

template <bool BF, int GPC, bool MINS, int MATS, int RT, int NT, int WV, int SL, bool X32>
hipError_t launch_apply(const Q4Args& a, int out_type, hipStream_t s) {
  const int64_t tiles = (a.rows + kTile - 1) / kTile;
  const int64_t tpt = a.pieces == 3 ? 5 : 16;   // tokens of a slot tile (SL = 1: they all fit one)
  const int64_t gy = (a.tokens + tpt * NT - 1) / (tpt * NT);
  const int64_t gx = (tiles + RT - 1) / RT;
  hipLaunchKernelGGL((k_q4_apply<BF, GPC, MINS, MATS, RT, NT, WV, SL, X32>), dim3((unsigned)gx, (unsigned)gy),
                     dim3(WV * kWave), 0, s, a, out_type);
  return hipGetLastError();
}

// One slot tile: few slots or many, x of the operands' type or fp32.
template <bool BF, int GPC, bool MINS, int MATS, int WV>
hipError_t one_tile(const Q4Args& a, int out_type, hipStream_t s) {
  const bool few = a.tokens * a.pieces <= 4;
  if constexpr (BF) {
    if (a.x32)
      return few ? launch_apply<BF, GPC, MINS, MATS, 1, 1, WV, 1, true>(a, out_type, s)
                 : launch_apply<BF, GPC, MINS, MATS, 1, 1, WV, 4, true>(a, out_type, s);
  }
  return few && !a.staged ? launch_apply<BF, GPC, MINS, MATS, 1, 1, WV, 1, false>(a, out_type, s)
                          : launch_apply<BF, GPC, MINS, MATS, 1, 1, WV, 4, false>(a, out_type, s);
}

// Row tiles per wave and waves per workgroup: with one slot tile the weights'
// way from memory counts, and few row tiles get sixteen waves so that a whole
// matrix is on its way at once; with more, x is read again for every row tile that
// a wave does not hold.  In us, weights from memory, one token with 8 and 16 waves:
// 2560 x 9728 (160 row tiles) 10.3, 8.0; 4096 x 4096 (256) 6.2, 5.3; 8000 x 2560 (500) 5.9,
// 5.8; 9728 x 2560 (608) 7.4, 7.7; two matrices of that 8.9, 12.6 (of 2560 x 9728 11.8, 11.3).
// Row tiles a wave, 1, 2 and 4 (64 tokens: 3), bf16, group 32:
//                  32 tokens         48 tokens          64 tokens
//   32000 x 8192   79.8 66.3 50.0    103.4 89.5 61.1    155.8 90.8 87.8
//   9728 x 2560    17.2 16.2 12.8    19.4 21.5 15.0     28.9 22.0 16.8
//   4096 x 4096    11.1 17.1 14.8    13.1 15.4 18.2     21.8 16.0 19.5
// (matrices of few row tiles would rather have one a wave).
template <bool BF, int GPC, bool MINS>
hipError_t pick_apply(const Q4Args& a, int mats, int out_type, hipStream_t s) {
  const int64_t slot_tiles = a.pieces == 3 ? (a.tokens + 4) / 5 : (a.tokens + 15) / 16;
  const int64_t tiles = (a.rows + kTile - 1) / kTile;
  if (mats == 2) {
    if (slot_tiles == 1) return one_tile<BF, GPC, MINS, 2, 8>(a, out_type, s);
    if (slot_tiles == 2) return launch_apply<BF, GPC, MINS, 2, 1, 2, 8, 4, false>(a, out_type, s);
    if (slot_tiles == 3) return launch_apply<BF, GPC, MINS, 2, 2, 3, 8, 4, false>(a, out_type, s);
    return launch_apply<BF, GPC, MINS, 2, 1, 4, 8, 4, false>(a, out_type, s);
  }
  if (slot_tiles == 1)
    return tiles < 512 ? one_tile<BF, GPC, MINS, 1, 16>(a, out_type, s) : one_tile<BF, GPC, MINS, 1, 8>(a, out_type, s);
  if (slot_tiles == 2) return launch_apply<BF, GPC, MINS, 1, 2, 2, 8, 4, false>(a, out_type, s);
  if (slot_tiles == 3) return launch_apply<BF, GPC, MINS, 1, 4, 3, 8, 4, false>(a, out_type, s);
  return launch_apply<BF, GPC, MINS, 1, 3, 4, 8, 4, false>(a, out_type, s);
}

template <bool BF>
hipError_t pick_group(const Q4Args& a, int gpc, int mats, int out_type, hipStream_t s) {
  const bool mins = a.mins[0] != nullptr;
  if (gpc == 4) return mins ? pick_apply<BF, 4, true>(a, mats, out_type, s) : pick_apply<BF, 4, false>(a, mats, out_type, s);
  if (gpc == 2) return mins ? pick_apply<BF, 2, true>(a, mats, out_type, s) : pick_apply<BF, 2, false>(a, mats, out_type, s);
  return mins ? pick_apply<BF, 1, true>(a, mats, out_type, s) : pick_apply<BF, 1, false>(a, mats, out_type, s);
}

}  // namespace

}  // namespace externd
