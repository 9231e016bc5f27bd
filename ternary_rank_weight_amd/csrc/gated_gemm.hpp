// The tiled product of the gated block and the join of its splits; each including
// unit instantiates one operand type.
#pragma once
#include <algorithm>
#include <type_traits>

#include "activation.hpp"
#include "device_common.hpp"
#include "frag.hpp"
#include "gated.hpp"
#include "kernels.hpp"

namespace externd {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) uint16_t* lds16;

// LDS image of an operand tile for one step: O outer entries x 64 contraction
// entries in 16-byte slots.  Slots are permuted so that the 16 rows (or the
// 4 k rows x 32 bytes per lane group) of a fragment read lie in different
// banks; a slot's content is chosen by its source address, since loads to LDS
// write lanes in order.
template <bool COLS, int O>
struct Tile {
  static constexpr int kSlots = O * 8;
  // contraction-major permutation: which 32-byte block of a k row holds block b
  __device__ static int mix(int k) { return k & 3; }
  // (outer, k) of a slot's first entry
  __device__ static void place(int slot, int& o, int& k) {
    if constexpr (!COLS) {
      o = slot >> 3;
      k = ((slot & 7) ^ (o & 7)) * 8;
    } else {
      constexpr int per = O / 8;
      k = slot / per;
      const int s = slot % per;
      o = ((s >> 1) ^ mix(k)) * 16 + (s & 1) * 8;
    }
  }
  // A lane's offsets (entries) into an image for the fragments of a wave whose
  // first outer entry is w0 (a multiple of 64 for COLS): rows, by the half of the
  // step; cols, by the fragment number modulo 4.  Kept as plain values so that
  // a fragment's address is image + offset + constant.
  struct Lane {
    uint32_t at[COLS ? 4 : 2];
    __device__ Lane(int w0, int lane) {
      const int r = lane & 15, p = lane >> 4;
#pragma unroll
      for (int q = 0; q < (COLS ? 4 : 2); ++q) {
        if constexpr (!COLS) at[q] = (w0 + r) * 64 + (((q * 4 + p) ^ (r & 7)) * 8);
        else at[q] = (8 * p + (r >> 2)) * O + ((w0 >> 4) + (q ^ (r >> 2))) * 16 + 4 * (r & 3);
        asm("" : "+v"(at[q]));
      }
    }
  };
  // The wave's fragment i (16 outer entries from 16 i on), contraction entries 32 kk .. + 31.
  __device__ static u32x4 frag(lds16 img, const Lane& l, int i, int kk) {
    if constexpr (!COLS) {
      return *(const lds_u32x4*)(img + l.at[kk] + i * 16 * 64);
    } else {
      // two transposing reads of 4 k rows x 16 outer entries per lane group:
      // lane r of a group supplies k row r / 4, entries 4 (r % 4) .. + 3, and
      // receives entry r of the four rows
      u32x4 v;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const uint64_t t = __builtin_bit_cast(
            uint64_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                          (lds_s16x4*)(img + l.at[i & 3] + ((kk * 32 + 4 * hf) * O + (i >> 2) * 64))));
        v[2 * hf] = (uint32_t)t;
        v[2 * hf + 1] = (uint32_t)(t >> 32);
      }
      return v;
    }
  }
};

// f(0), f(1), ..., f(N - 1) with the index as a compile-time constant.
template <int N, int I = 0, typename F>
__device__ __forceinline__ void for_constants(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>());
    for_constants<N, I + 1>(f);
  }
}

// out tile = sum over k of A[m][k] B[n][k].  BM x BN outputs per workgroup of
// WM x WN waves.  The products take b's fragment as first and a's as second
// operand, so that a lane holds four neighbouring output columns of one row.
//
// Whole steps go from memory to LDS without passing through registers (so every
// row starts 16-byte aligned); the last, partial step of a contraction is read
// through registers, zero past its end.  Rows are read in pieces of 128 bytes: pieces of 64 come
// from L2 at half the rate.
//
// Bound by the matrix instructions: at K = 10240 the forward runs at 1.38
// PFLOP/s (a large library product without the activation: 1.43).  K = 2560, F = 9728,
// bf16: forward of 4096 tokens 330 us (1.24 PFLOP/s; the same two products by the
// library, without activation and product: 428 us); of 2048 tokens with g and u
// kept 234 us; dx, both parts of dg and du, 337 us and its join 16; dW, both parts, 333 us
// (1.23 PFLOP/s).  What is lost is the end of a tile (6 of 62 us a tile of 40 steps) and
// the last round of tiles.
template <bool BF, int MODE, int BM, int BN, int WM, int WN, int NA, int NB, bool SPLIT>
__global__ __launch_bounds__(WM * WN * kWave, BM == 256 || NB == 2 ? 2 : 1) void k_gated_gemm(GatedGemm g) {
  constexpr int NTHR = WM * WN * kWave;
  constexpr bool ACOLS = MODE == kDw, BCOLS = MODE != kFwd;
  constexpr int MI = BM / WM / 16, NI = BN / WN / 16;
  using TA = Tile<ACOLS, BM>;
  using TB = Tile<BCOLS, BN>;
  constexpr int SA = TA::kSlots / NTHR, SB = TB::kSlots / NTHR;
  // separate objects: the compiler then sees that a read of one image need not
  // wait for the loads into another
  constexpr int A3 = NA > 3 ? BM * kBK : 8, B2 = NB > 2 ? BN * kBK : 8;
  __shared__ __align__(16) uint16_t sa0[BM * kBK], sa1[BM * kBK], sa2[BM * kBK], sa3[A3];
  __shared__ __align__(16) uint16_t sb0[BN * kBK], sb1[BN * kBK], sb2[B2], sb3[B2];
  const lds16 la0 = (lds16)sa0, la1 = (lds16)sa1, la2 = (lds16)sa2, la3 = (lds16)sa3;
  const lds16 lb0 = (lds16)sb0, lb1 = (lds16)sb1, lb2 = (lds16)sb2, lb3 = (lds16)sb3;
  auto image_a = [&](auto index) {
    constexpr int I = decltype(index)::value % NA;
    if constexpr (I == 0) return la0;
    else if constexpr (I == 1) return la1;
    else if constexpr (I == 2) return la2;
    else return la3;
  };
  auto image_b = [&](auto index) {
    constexpr int I = decltype(index)::value % NB;
    if constexpr (I == 0) return lb0;
    else if constexpr (I == 1) return lb1;
    else if constexpr (I == 2) return lb2;
    else return lb3;
  };
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int wm = wave / WN, wn = wave % WN;

  constexpr int BNO = MODE == kFwd ? BN / 2 : BN;   // output columns per tile
  constexpr bool SEGS = MODE != kFwd;   // a contraction of several segments
  const int segs = SEGS ? g.segs : 1;

  // A workgroup takes units (one tile, one split) id, id + grid, ...  They are
  // numbered down groups of 8 tile rows, each XCD a run of them, so that the
  // workgroups of an XCD share operand rows in its L2.
  struct Unit {
    int64_t m0, n0;          // first output row and column
    int64_t s_begin, s_end;  // whole steps of all segments in order
    int outsel, split;
    bool last;               // also takes the partial steps
  };
  const uint32_t tiles = (uint32_t)(g.mt * g.nt), units = tiles * (uint32_t)g.splits;
  auto locate = [&](uint32_t at) {
    Unit q;
    const uint32_t x = at & 7, rest = units % 8;
    const uint32_t id = x * (units / 8) + min(x, rest) + (at >> 3);
    const uint32_t split = id / tiles, tile = id % tiles;
    const uint32_t group = 8 * (uint32_t)g.nt, g0 = tile / group * 8, gh = min(8u, (uint32_t)g.mt - g0);
    uint32_t mt = __builtin_amdgcn_readfirstlane(g0 + tile % group % gh);
    const uint32_t ntile = __builtin_amdgcn_readfirstlane(tile % group / gh);
    q.split = __builtin_amdgcn_readfirstlane(split);
    q.outsel = 0;
    if constexpr (MODE == kDw) {   // tile rows: all of dWg, then all of dWu
      const uint32_t half = (uint32_t)g.mt / 2;
      q.outsel = mt >= half;
      mt -= q.outsel * half;
    }
    q.m0 = (int64_t)mt * BM;
    q.n0 = (int64_t)ntile * BNO;
    q.s_begin = q.split * g.split_steps;
    q.s_end = min(segs * g.full, q.s_begin + g.split_steps);
    q.last = q.split == g.splits - 1;
    return q;
  };
  Unit u = locate(blockIdx.x);

  f32x4 acc[MI][NI];
  auto clear = [&] {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  };

  // source of a slot at contraction offset k0
  auto src_a = [&](int slot, int seg, int64_t k0, int64_t& left_o, int64_t& left_k) -> const uint16_t* {
    int o, k;
    TA::place(slot, o, k);
    const uint16_t* base = g.a.p[u.outsel] + seg * g.rest;
    left_o = g.a.outer - (u.m0 + o);
    left_k = g.inner - (k0 + k);
    if constexpr (!ACOLS) return base + min(u.m0 + o, g.a.outer - 1) * g.a.ld + (k0 + k);
    else return base + (k0 + k) * g.a.ld + (u.m0 + o);
  };
  auto src_b = [&](int slot, int seg, int64_t k0, int64_t& left_o, int64_t& left_k) -> const uint16_t* {
    int o, k;
    TB::place(slot, o, k);
    if constexpr (MODE == kFwd) {   // the tile's first half gate rows, its second up rows
      const int which = o >= BNO;
      o -= which * BNO;
      left_o = 8;
      left_k = g.inner - (k0 + k);
      return g.b.p[which] + min(u.n0 + o, g.b.outer - 1) * g.b.ld + (k0 + k);
    } else {
      const uint16_t* base = g.b.p[MODE == kDx && 2 * seg >= segs];
      left_o = g.b.outer - (u.n0 + o);
      left_k = g.inner - (k0 + k);
      return base + (k0 + k) * g.b.ld + (u.n0 + o);
    }
  };
  // A partial step through registers.  A slot's eight entries are all inside or all past
  // an end: rows are padded to 8 entries (with zeros, where they were padded here).
  // A thread's loads are in flight together; a slot past an end loads the operand's first.
  auto stage_operand = [&](auto n, lds16 image, const uint16_t* inside, auto source) {
    constexpr int PER = NA == 4 ? 4 : BM == 128 ? 2 : 1;   // (what each kind has registers for)
    static_assert(decltype(n)::value % (PER * NTHR) == 0);
#pragma unroll 1
    for (int slot = tid; slot < decltype(n)::value; slot += PER * NTHR) {
      u32x4 v[PER];
      bool in[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        int64_t lo, lk;
        const uint16_t* q = source(slot + i * NTHR, lo, lk);
        in[i] = lo > 0 && lk > 0;
        v[i] = load8<true>(in[i] ? q : inside);
      }
      loads_made();
#pragma unroll
      for (int i = 0; i < PER; ++i)
        *(lds_u32x4*)(image + (slot + i * NTHR) * 8) = in[i] ? v[i] : u32x4{0u, 0u, 0u, 0u};
    }
  };
  auto stage_part = [&](int seg, int64_t k0) {
    stage_operand(std::integral_constant<int, TA::kSlots>(), la0, g.a.p[0], [&](int slot, int64_t& lo, int64_t& lk) {
      const uint16_t* q = src_a(slot, seg, k0, lo, lk);
      if constexpr (!ACOLS) lo = 1;   // (a row past the end repeats the last)
      return q;
    });
    stage_operand(std::integral_constant<int, TB::kSlots>(), lb0, g.b.p[0], [&](int slot, int64_t& lo, int64_t& lk) {
      const uint16_t* q = src_b(slot, seg, k0, lo, lk);
      if constexpr (!BCOLS) lo = 1;
      return q;
    });
  };
  // the forward's b: half of a wave's fragments in the gate rows, half in the up rows
  const typename TA::Lane lane_a(wm * MI * 16, lane);
  const typename TB::Lane lane_b(wn * (MODE == kFwd ? NI / 2 : NI) * 16, lane);
  auto read_a = [&](lds16 img, int i, int kk) { return TA::frag(img, lane_a, i, kk); };
  auto read_b = [&](lds16 img, int j, int kk) {
    if constexpr (MODE == kFwd) return TB::frag(img, lane_b, j / (NI / 2) * (BNO / 16) + j % (NI / 2), kk);
    else return TB::frag(img, lane_b, j, kk);
  };
  auto multiply_all = [&]() {   // one step whose image is the first
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      u32x4 b[NI];
#pragma unroll
      for (int j = 0; j < NI; ++j) b[j] = read_b(lb0, j, kk);
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const u32x4 a = read_a(la0, i, kk);
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] = mfma16<BF>(b[j], a, acc[i][j]);
      }
    }
  };
  // Loads to LDS: where the next step of each operand is read.  A wave moves SA or
  // SB pieces of a step, 64 slots each.
  uint32_t va[SA], vb[SB];   // byte offsets of this thread's slots from the tile's first entry
  const uint16_t *pa = nullptr, *pb = nullptr;
  int64_t step_a = 0, step_b = 0;   // within the segment
  int seg_b = 0;
  const int64_t move_a = ACOLS ? kBK * g.a.ld : kBK, move_b = BCOLS ? kBK * g.b.ld : kBK;
  const int64_t to_up = MODE != kDw ? g.b.p[1] - g.b.p[0] : 0;
  const int uwave = __builtin_amdgcn_readfirstlane(wave);
  auto stage_a = [&](lds16 img, int piece) {
    to_lds16(pa, va[piece], img + (piece * NTHR + uwave * kWave) * 8);
    if (piece == SA - 1) {
      pa += move_a;
      if (SEGS && ++step_a == g.full) {
        step_a = 0;
        pa += g.rest - g.full * move_a;
      }
    }
  };
  auto stage_b = [&](lds16 img, int piece) {
    // a wave's 64 slots of the forward's b are 8 rows of one source
    const bool up = MODE == kFwd && (piece * NTHR + uwave * kWave) / 8 >= BNO;
    to_lds16(up ? pb + to_up : pb, vb[piece], img + (piece * NTHR + uwave * kWave) * 8);
    if (piece == SB - 1) {
      pb += move_b;
      if (SEGS && ++step_b == g.full) {
        step_b = 0;
        pb -= g.full * move_b;
        if (MODE == kDx && 2 * ++seg_b == segs) pb += to_up;
      }
    }
  };
  constexpr int R = 2 * MI, T = R - 3, PIECES = SA + SB, EARLY = 3 * PIECES / R;   // see below
  // Sets out the first loads of a unit; every image is free.
  auto begin = [&](const Unit& q) {
#pragma unroll
    for (int i = 0; i < SA; ++i) {
      int o, k;
      TA::place(i * NTHR + tid, o, k);
      if constexpr (!ACOLS) va[i] = (uint32_t)(min<int64_t>(o, g.a.outer - 1 - q.m0) * g.a.ld + k) * 2u;
      else va[i] = (uint32_t)(k * g.a.ld + min<int64_t>(o, g.a.outer - 8 - q.m0)) * 2u;
    }
#pragma unroll
    for (int i = 0; i < SB; ++i) {
      int o, k;
      TB::place(i * NTHR + tid, o, k);
      if constexpr (MODE == kFwd) o -= (o >= BNO) * BNO;
      if constexpr (!BCOLS) vb[i] = (uint32_t)(min<int64_t>(o, g.b.outer - 1 - q.n0) * g.b.ld + k) * 2u;
      else vb[i] = (uint32_t)(k * g.b.ld + min<int64_t>(o, g.b.outer - 8 - q.n0)) * 2u;
    }
    int seg = 0;
    int64_t first = q.s_begin;
    while (SEGS && seg + 1 < segs && first >= g.full) {
      first -= g.full;
      ++seg;
    }
    const int64_t from_a = ACOLS ? q.m0 : q.m0 * g.a.ld, from_b = BCOLS ? q.n0 : q.n0 * g.b.ld;
    pa = g.a.p[q.outsel] + seg * g.rest + from_a + first * move_a;
    pb = g.b.p[MODE == kDx && 2 * seg >= segs] + from_b + first * move_b;
    step_a = step_b = first;
    seg_b = seg;
    // as the barriers of steps -NA .. -1 would: see below
    for_constants<NA - 1>([&](auto index) {
      constexpr int J = decltype(index)::value, JB = J - NA + NB;
      if constexpr (JB >= 0) {
        if (q.s_begin + JB < q.s_end) {
#pragma unroll
          for (int p = 0; p < SB; ++p) stage_b(image_b(std::integral_constant<int, JB>()), p);
        }
      }
      if (q.s_begin + J < q.s_end) {
#pragma unroll
        for (int p = 0; p < SA; ++p) stage_a(image_a(index), p);
      }
    });
    if (q.s_begin + NB - 1 < q.s_end) {
#pragma unroll
      for (int p = 0; p < EARLY; ++p) stage_b(image_b(std::integral_constant<int, NB - 1>()), p);
    }
  };
  auto contract = [&] {
    // A step is 2 MI rows of fragment products.  Row t multiplies fragments that
    // were read from LDS three rows (a) or more (b) before, so that the products
    // of neighbouring rows and steps follow each other without a wait.  There are
    // NA images of a and NB of b.  The only barrier of step s is before row T =
    // 2 MI - 3, when every wave has read all of its fragments (the wait before it
    // says so).  Past it the images of step s are free: the pieces of step s + NB of b
    // and then of s + NA of a set out from memory, spread over the rows up to the next
    // barrier, and the fragments of s + 1 are read, whose images the wait has made
    // sure of.  With NA = 3 and NB = 2 (160 KB at 256 x 256; 80 KB at 128 x 128, two
    // workgroups a CU) b has one step and a two to arrive; NA = NB = 4 (128 KB at 128 x 128)
    // gives both three, for workgroups that have a CU to themselves.
    static_assert(MI % 4 == 0 && NI <= 4 && EARLY <= SB && (NA == NB || NA == NB + 1), "rotation");
    constexpr int ROUND = NA == NB ? NA : NA * NB;   // steps after which the images repeat
    const int64_t n = u.s_end - u.s_begin;
    u32x4 fa[4], fb[2][NI];
    auto step = [&](auto index, auto steady, int64_t s) {
      constexpr int J = decltype(index)::value;   // s modulo ROUND
      constexpr bool ALL = decltype(steady)::value;   // every step that this one moves exists
      constexpr std::integral_constant<int, J + 1> next;
      constexpr std::integral_constant<int, J + NB - 1> later_b;   // what is left of the last barrier's
      constexpr std::integral_constant<int, J + NA - 1> later_a;
      const lds16 ca = image_a(index), na = image_a(next), cb = image_b(index), nb = image_b(next);
#pragma unroll
      for (int t = 0; t < R; ++t) {
        if (t == T) {
          // outstanding at most: what was sent for steps after s + 1 (near the end, less)
          if (ALL || s + NB < n) wait_vm<(NA > NB ? SA : 0) + (NB - 2) * PIECES, 0>();
          else if (NB > 3 && s + 3 < n) wait_vm<PIECES, 0>();
          else wait_vm<0, 0>();
          block_barrier();
        }
        // (past the last step these read images that are not used)
        if (t + 3 < R) fa[(t + 3) & 3] = read_a(ca, (t + 3) % MI, (t + 3) / MI);
        else fa[(t + 3) & 3] = read_a(na, t + 3 - R, 0);
        if (t < NI) fb[1][t] = read_b(cb, t, 1);
        if (t >= T) {
#pragma unroll
          for (int j = (t - T) * 2; j < NI && j < (t - T) * 2 + 2; ++j) fb[0][j] = read_b(nb, j, 0);
        }
        const int d = (t - T + R) % R;
        if (t >= T) {
          if (ALL || s + NB < n) {
#pragma unroll
            for (int q = d * PIECES / R; q < (d + 1) * PIECES / R; ++q) stage_b(cb, q);
          }
        } else {
#pragma unroll
          for (int q = d * PIECES / R; q < (d + 1) * PIECES / R; ++q) {
            if (q < SB) {
              if (ALL || s + NB - 1 < n) stage_b(image_b(later_b), q);
            } else {
              if (ALL || s + NA - 1 < n) stage_a(image_a(later_a), q - SB);
            }
          }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[t % MI][j] = mfma16<BF>(fb[t / MI][j], fa[t & 3], acc[t % MI][j]);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    if (n > 0) {
#pragma unroll
      for (int j = 0; j < NI; ++j) fb[0][j] = read_b(lb0, j, 0);
#pragma unroll
      for (int i = 0; i < 3; ++i) fa[i] = read_a(la0, i, 0);
      int64_t s = 0;
#pragma unroll 1
      for (; s + ROUND - 1 + NB < n; s += ROUND)
        for_constants<ROUND>([&](auto index) { step(index, std::true_type(), s + decltype(index)::value); });
#pragma unroll 1
      for (; s < n; s += ROUND)
        for_constants<ROUND>([&](auto index) {
          if (s + decltype(index)::value < n) step(index, std::false_type(), s + decltype(index)::value);
        });
      __syncthreads();
    }
  };
  // ---- outputs: a lane holds row m, columns n .. n + 3 of each fragment ----
  const int r = lane & 15, p = lane >> 4;
  constexpr int NO = MODE == kFwd ? NI / 2 : NI;   // output fragments per fragment row
  // whole: the fragment's four entries exist and may be stored at once
  auto put16 = [&](uint16_t* q, int64_t left, bool whole, uint2 w) {
    if (whole) {
      *reinterpret_cast<uint2*>(q) = w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < left) q[e] = (uint16_t)((e < 2 ? w.x : w.y) >> (16 * (e & 1)));
    }
  };
  auto put32 = [&](float* q, int64_t left, bool whole, f32x4 v) {
    if (whole) {
      *reinterpret_cast<f32x4*>(q) = v;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < left) q[e] = v[e];
    }
  };
  auto pack = [&](f32x4 v) {
    return uint2{f32_to_16<BF>(v[0]) | (f32_to_16<BF>(v[1]) << 16), f32_to_16<BF>(v[2]) | (f32_to_16<BF>(v[3]) << 16)};
  };
  uint2 packed[MI][NO];   // 16-bit outputs
  auto activate = [&](auto act) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NO; ++j) {
        f32x4 h;
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = act_fast<decltype(act)::value>(acc[i][j][e]) * acc[i][j + NI / 2][e];
        packed[i][j] = pack(h);
      }
  };
  const int64_t n_lane = wn * NO * 16 + 4 * p, m_lane = wm * MI * 16 + r;
  auto round_outputs = [&] {
    if constexpr (MODE == kFwd) {
      if (g.act == EXTERND_ACT_SILU) activate(std::integral_constant<int, EXTERND_ACT_SILU>());
      else if (g.act == EXTERND_ACT_GELU) activate(std::integral_constant<int, EXTERND_ACT_GELU>());
      else activate(std::integral_constant<int, EXTERND_ACT_GELU_TANH>());
    } else {
      float back[MI];   // fp16: what takes the scale of a's row off
#pragma unroll
      for (int i = 0; i < MI; ++i)
        if constexpr (!BF) back[i] = unscale_of(g.tops[u.outsel * g.tops_of_up + min(u.m0 + m_lane + i * 16, g.mo - 1)]);
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NO; ++j) packed[i][j] = pack(BF ? acc[i][j] : acc[i][j] * back[i]);
    }
  };
  const bool aligned = g.ldo % 4 == 0 &&
                       ((reinterpret_cast<uintptr_t>(g.out[0]) | reinterpret_cast<uintptr_t>(g.out[1])) & 7) == 0 &&
                       ((reinterpret_cast<uintptr_t>(g.save[0]) | reinterpret_cast<uintptr_t>(g.save[1])) & 15) == 0;
  auto put_outputs = [&](auto inside) {   // inside: the whole tile is, and its rows are aligned
    constexpr bool IN = decltype(inside)::value;
    constexpr int OUTS = MODE == kDx ? 1 : 2;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int64_t m = u.m0 + m_lane + i * 16, at = m * g.ldo + u.n0 + n_lane;
      if (!IN && m >= g.mo) continue;
#pragma unroll
      for (int j = 0; j < NO; ++j) {
        const int64_t left = g.ldo - (u.n0 + n_lane + j * 16);
        if (!IN && left <= 0) continue;
        const bool whole = IN || (aligned && left >= 4);
        if constexpr (SPLIT) {
          float* q = g.part + ((int64_t)u.split * OUTS + u.outsel) * g.mo * g.ldo + at + j * 16;
          put32(q, left, whole, acc[i][j]);
          if constexpr (MODE == kFwd) put32(q + g.mo * g.ldo, left, whole, acc[i][j + NI / 2]);
        } else {
          put16(g.out[u.outsel] + at + j * 16, left, whole, packed[i][j]);
          if (MODE == kFwd && g.save[0]) {
            put32(g.save[0] + at + j * 16, left, whole, acc[i][j]);
            put32(g.save[1] + at + j * 16, left, whole, acc[i][j + NI / 2]);
          }
        }
      }
    }
  };
  begin(u);
  wait_vm<0, 0>();
#pragma unroll 1
  for (uint32_t at = blockIdx.x;;) {
    clear();
    block_barrier();   // every wave has waited for its first loads
    contract();
    if (u.last && g.full * kBK < g.inner) {
#pragma unroll 1
      for (int seg = 0; seg < segs; ++seg) {
        stage_part(seg, g.full * kBK);
        __syncthreads();
        multiply_all();
        __syncthreads();
      }
    }
    // The next unit's first loads travel while this one's outputs are worked out,
    // and have arrived before the first output is stored: the stores then drain
    // behind the next unit's products.
    at += gridDim.x;
    const bool more = at < units;
    const Unit next = locate(more ? at : blockIdx.x);
    if (more) begin(next);
    if constexpr (!SPLIT) round_outputs();
    wait_vm<0, 0>();
    if (aligned && u.m0 + BM <= g.mo && u.n0 + BNO <= g.ldo) put_outputs(std::true_type());
    else put_outputs(std::false_type());
    if (!more) break;
    u = next;
  }
}

// What the split contractions left: the splits' sums in their order, then the
// outputs as the unsplit kernel makes them.  part: (split, outs, count) fp32, rows of ldo;
// tops: as in GatedGemm.
// Forward: both projections, the activation and the product.  Bound by HBM: 16 us for
// three splits of 2048 x 2560 (4.3 TB/s).
template <bool BF, int MODE>
__global__ __launch_bounds__(256) void k_gated_join(const float* __restrict__ part, int64_t count, int64_t splits,
                                                     uint16_t* __restrict__ out0, uint16_t* __restrict__ out1,
                                                     float* __restrict__ g, float* __restrict__ u, int act,
                                                     const uint32_t* __restrict__ tops, int64_t tops_of_up, int64_t ldo) {
  constexpr int OUTS = MODE == kDx ? 1 : 2;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (int64_t)gridDim.x * 256) {
    float s[OUTS];
#pragma unroll
    for (int o = 0; o < OUTS; ++o) {
      s[o] = part[o * count + i];
      for (int64_t q = 1; q < splits; ++q) s[o] += part[(q * OUTS + o) * count + i];
    }
    if constexpr (MODE == kFwd) {
      out0[i] = (uint16_t)f32_to_16<BF>(act_value(act, s[0]) * s[1]);
      if (g) { g[i] = s[0]; u[i] = s[1]; }
    } else {
      if constexpr (!BF) {
        const int64_t row = i / ldo;
#pragma unroll
        for (int o = 0; o < OUTS; ++o) s[o] *= unscale_of(tops[o * tops_of_up + row]);
      }
      out0[i] = (uint16_t)f32_to_16<BF>(s[0]);
      if constexpr (MODE == kDw) out1[i] = (uint16_t)f32_to_16<BF>(s[1]);
    }
  }
}

// Persistent workgroups: as many as are resident together.
template <bool BF, int MODE, GatedKind KIND, bool SPLIT>
hipError_t launch_tile(GatedGemm g, int cus, hipStream_t s) {
  constexpr int B = KIND == kBig ? 256 : 128, WN = KIND == kBig ? 4 : 2;
  constexpr int NA = KIND == kDeep ? 4 : 3, NB = KIND == kDeep ? 4 : 2;
  g.mt = MODE == kDw ? 2 * ceil_div64(g.a.outer, B) : ceil_div64(g.a.outer, B);
  g.nt = ceil_div64(g.b.outer, MODE == kFwd ? B / 2 : B);
  const int64_t resident = (int64_t)cus * (KIND == kPair ? 2 : 1);
  const dim3 grid((unsigned)std::min<int64_t>(g.mt * g.nt * g.splits, resident)), block(2 * WN * kWave);
  hipLaunchKernelGGL((k_gated_gemm<BF, MODE, B, B, 2, WN, NA, NB, SPLIT>), grid, block, 0, s, g);
  return hipGetLastError();
}

template <bool BF, int MODE>
hipError_t product(GatedGemm g, const GatedPlan& plan, float* part, int cus, hipStream_t s) {
  g.full = g.inner / kBK;
  const int64_t whole = std::max<int64_t>(1, g.segs * g.full);
  g.split_steps = ceil_div64(whole, plan.splits);
  g.splits = ceil_div64(whole, g.split_steps);   // none without steps
  if (plan.splits == 1 && plan.stacked == 1)
    return plan.kind == kBig    ? launch_tile<BF, MODE, kBig, false>(g, cus, s)
           : plan.kind == kPair ? launch_tile<BF, MODE, kPair, false>(g, cus, s)
                                : launch_tile<BF, MODE, kDeep, false>(g, cus, s);
  g.part = part;
  hipError_t e = hipSuccess;
  if constexpr (MODE == kDx)
    if (plan.kind == kBig) e = launch_tile<BF, MODE, kBig, true>(g, cus, s);
  if (plan.kind == kDeep) e = launch_tile<BF, MODE, kDeep, true>(g, cus, s);
  if (e != hipSuccess) return e;
  const int64_t count = g.mo / plan.stacked * g.ldo;   // (a half is as good as a split)
  const dim3 grid((unsigned)std::max<int64_t>(1, std::min<int64_t>(ceil_div64(count, 256), 1 << 15))), block(256);
  hipLaunchKernelGGL((k_gated_join<BF, MODE>), grid, block, 0, s, part, count, g.splits * plan.stacked, g.out[0], g.out[1], g.save[0],
                     g.save[1], g.act, g.tops, g.tops_of_up, g.ldo);
  return hipGetLastError();
}

template <bool BF>
hipError_t any_product(GatedProduct mode, const GatedGemm& g, const GatedPlan& plan, float* part, int cus,
                       hipStream_t s) {
  if (mode == kFwd) return product<BF, kFwd>(g, plan, part, cus, s);
  if (mode == kDx) return product<BF, kDx>(g, plan, part, cus, s);
  return product<BF, kDw>(g, plan, part, cus, s);
}

}  // namespace

}  // namespace externd
