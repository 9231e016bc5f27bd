// C ABI of the ExTernD library: argument validation, device checks,
// workspace management and dispatch to the HIP kernels.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <initializer_list>
#include <mutex>
#include <string>

#include "../../include/externd.h"
#include "kernels.hpp"

namespace {

thread_local std::string g_last_error;

int fail(int status, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return status;
}

int hip_fail(hipError_t e, const char* where) {
  return fail(EXTERND_EHIP, "%s: %s", where, hipGetErrorString(e));
}

struct DeviceInfo {
  bool checked = false;
  bool gfx950 = false;
  int cus = 0;
};
std::mutex g_dev_mu;
DeviceInfo g_dev[64];

// Current device must be a gfx950; remembers its compute-unit count.
int check_device(int* cus) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
  if (dev < 0 || dev >= 64) return fail(EXTERND_EUNSUPPORTED, "device index %d out of range", dev);
  std::lock_guard<std::mutex> lk(g_dev_mu);
  DeviceInfo& d = g_dev[dev];
  if (!d.checked) {
    hipDeviceProp_t prop;
    e = hipGetDeviceProperties(&prop, dev);
    if (e != hipSuccess) return hip_fail(e, "hipGetDeviceProperties");
    d.gfx950 = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
    d.cus = prop.multiProcessorCount;
    d.checked = true;
  }
  if (!d.gfx950) return fail(EXTERND_EUNSUPPORTED, "device %d is not gfx950", dev);
  if (cus) *cus = d.cus;
  return EXTERND_OK;
}

bool bad_size(int64_t m, int64_t n) {
  return m <= 0 || n <= 0 || m > (int64_t(1) << 31) - 1 || n > (int64_t(1) << 31) - 1 ||
         m * n > (int64_t(1) << 40);
}

// The sequential mode a request runs in: AUTO takes the resident kernel when
// the shape fits on chip (not with the projection or an applied safeguard),
// else the persistent streaming kernel when it applies, else the streaming
// kernel chain.  -1 when an explicit mode does not apply to the shape.
int seq_mode(int requested, int64_t m, int64_t n, int cus, bool projection, bool safeguard) {
  const bool res_ok = externd::resident_fits(m, n, cus) && !projection && !safeguard;
  const bool per_ok = externd::persist_fits(m, n, cus) && !projection && !safeguard;
  switch (requested) {
    case EXTERND_MODE_RESIDENT: return res_ok ? EXTERND_MODE_RESIDENT : -1;
    case EXTERND_MODE_PERSISTENT: return per_ok ? EXTERND_MODE_PERSISTENT : -1;
    case EXTERND_MODE_STREAMING: return EXTERND_MODE_STREAMING;
    default: return res_ok ? EXTERND_MODE_RESIDENT : (per_ok ? EXTERND_MODE_PERSISTENT : EXTERND_MODE_STREAMING);
  }
}

// Stream-ordered workspace: allocated on the stream, freed on the stream
// (or borrowed from the caller, then never freed here).
struct Workspace {
  void* ptr = nullptr;
  hipStream_t s = nullptr;
  bool owned = false;
  ~Workspace() {
    if (ptr && owned) (void)hipFreeAsync(ptr, s);
  }
};

int alloc_ws(Workspace& w, size_t bytes, hipStream_t s) {
  w.s = s;
  hipError_t e = hipMallocAsync(&w.ptr, bytes, s);
  if (e != hipSuccess) {
    w.ptr = nullptr;
    return fail(EXTERND_ENOMEM, "hipMallocAsync(%zu): %s", bytes, hipGetErrorString(e));
  }
  w.owned = true;
  return EXTERND_OK;
}

// The caller's workspace when opts provides one (checked against `bytes`),
// else a stream-ordered allocation.
int get_ws(Workspace& w, const externd_opts& o, size_t bytes, hipStream_t s) {
  if (!o.workspace) return alloc_ws(w, bytes, s);
  if (o.workspace_bytes < bytes)
    return fail(EXTERND_ENOMEM, "workspace of %llu bytes < %zu needed",
                (unsigned long long)o.workspace_bytes, bytes);
  w.ptr = o.workspace;
  w.s = s;
  w.owned = false;
  return EXTERND_OK;
}

// The caller's workspace when given (checked), else a stream-ordered one;
// nothing when none is needed.
int op_ws(Workspace& w, void* workspace, size_t workspace_bytes, size_t need, hipStream_t s) {
  if (need == 0) return EXTERND_OK;
  if (!workspace) return alloc_ws(w, need, s);
  if ((reinterpret_cast<uintptr_t>(workspace) & 255) != 0 || workspace_bytes < need)
    return fail(EXTERND_EINVAL, "workspace must be 256-byte aligned and at least %zu bytes", need);
  w.ptr = workspace;
  return EXTERND_OK;
}

// Rows of `width` bytes, `stride` bytes apart; a null pointer is an empty region.
struct Region {
  const void* p;
  int64_t rows, width, stride;
  const char* name;
};
Region packed(const void* p, int64_t bytes, const char* name) { return {p, 1, bytes, bytes, name}; }

// Whether a region of one row has a byte in common with another.
bool overlaps(const Region& one, const Region& r) {
  if (!one.p || !r.p || one.width <= 0 || r.width <= 0 || r.rows <= 0) return false;
  const uintptr_t begin = reinterpret_cast<uintptr_t>(one.p), end = begin + one.width, at = reinterpret_cast<uintptr_t>(r.p);
  if (end <= at) return false;
  // r's first row that ends past `begin`
  const uintptr_t row = begin < at + r.width ? 0 : (begin - at - r.width) / r.stride + 1;
  return row < (uintptr_t)r.rows && at + row * r.stride < end;
}

// What a call writes has no byte in common with what it reads or writes besides: the
// kernels read and write in no set order.
int check_apart(std::initializer_list<Region> written, std::initializer_list<Region> read) {
  for (auto w = written.begin(); w != written.end(); ++w) {
    for (auto o = written.begin(); o != w; ++o)
      if (overlaps(*w, *o)) return fail(EXTERND_EINVAL, "%s overlaps %s", w->name, o->name);
    for (const Region& r : read)
      if (overlaps(*w, r)) return fail(EXTERND_EINVAL, "%s overlaps %s", w->name, r.name);
  }
  return EXTERND_OK;
}

bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
size_t dtype_bytes(int dtype) { return dtype == EXTERND_F32 ? 4 : 2; }
bool bad_dtype(int dtype) { return dtype != EXTERND_F32 && dtype != EXTERND_BF16 && dtype != EXTERND_F16; }
bool bad_act(int act) { return act != EXTERND_ACT_SILU && act != EXTERND_ACT_GELU && act != EXTERND_ACT_GELU_TANH; }
bool bad_group(int group) { return group != 32 && group != 64 && group != 128; }
// Row strides: at least the row, and small enough that offsets fit 63 bits with room.
bool bad_stride(int64_t ld, int64_t cols) { return ld < cols || ld > int64_t(1) << 40; }
constexpr int64_t kMaxTokens = int64_t(1) << 20;   // of the 4-bit products
constexpr int64_t kMaxGated = int64_t(1) << 21;    // widths of the gated block

int check_q4(const externd_q4* w, const char* name) {
  if (!w) return fail(EXTERND_EINVAL, "null %s", name);
  if (bad_size(w->rows, w->cols)) return fail(EXTERND_EINVAL, "%s: bad shape", name);
  if (bad_group(w->group)) return fail(EXTERND_EINVAL, "%s: group must be 32, 64 or 128", name);
  if (!w->codes || !w->scales) return fail(EXTERND_EINVAL, "%s: null codes or scales", name);
  if (!aligned_to(w->codes, 16) || !aligned_to(w->scales, 8) || !aligned_to(w->mins, 8))
    return fail(EXTERND_EINVAL, "%s: codes must be 16-byte and tables 8-byte aligned", name);
  return EXTERND_OK;
}

int64_t q4_blocks(int64_t rows, int64_t cols) { return (rows + 15) / 16 * ((cols + 127) / 128); }
int64_t q4_code_bytes(const externd_q4& w) { return 1024 * q4_blocks(w.rows, w.cols); }
int64_t q4_table_bytes(const externd_q4& w) { return 4096 / w.group * q4_blocks(w.rows, w.cols); }

// The common part of the 4-bit products.
int q4_product(const externd_q4* w, int mats, const void* x, int64_t tokens, int64_t ldx, int dtype, int act,
               void* stream, void* y, void* workspace, size_t workspace_bytes) {
  if (bad_dtype(dtype)) return fail(EXTERND_EINVAL, "unknown dtype %d", dtype);
  if (tokens < 0 || tokens > kMaxTokens) return fail(EXTERND_EINVAL, "tokens must be 0 to 2^20");
  if (bad_stride(ldx, w->cols)) return fail(EXTERND_EINVAL, "ldx must be at least the columns");
  if (tokens == 0) return EXTERND_OK;
  if (!x || !y) return fail(EXTERND_EINVAL, "null x or output pointer");
  if (!aligned_to(x, dtype_bytes(dtype)) || !aligned_to(y, dtype_bytes(dtype)))
    return fail(EXTERND_EINVAL, "x and the output must be aligned to their type");
  const int64_t e_bytes = (int64_t)dtype_bytes(dtype);
  const externd_q4 &a = w[0], &b = w[mats - 1];
  const size_t need = externd::q4_stages_x(w->rows, w->cols, tokens, ldx, dtype, x) ? externd::q4_stage_bytes(w->cols, tokens, dtype) : 0;
  int st = check_apart({packed(y, tokens * w->rows * e_bytes, "the output"), packed(workspace, (int64_t)need, "workspace")},
                       {{x, tokens, w->cols * e_bytes, ldx * e_bytes, "x"},
                        packed(a.codes, q4_code_bytes(a), "codes"), packed(a.scales, q4_table_bytes(a), "scales"),
                        packed(a.mins, q4_table_bytes(a), "mins"), packed(b.codes, q4_code_bytes(b), "codes"),
                        packed(b.scales, q4_table_bytes(b), "scales"), packed(b.mins, q4_table_bytes(b), "mins")});
  if (st != EXTERND_OK) return st;
  if ((st = check_device(nullptr)) != EXTERND_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  Workspace ws;
  if ((st = op_ws(ws, workspace, workspace_bytes, need, s)) != EXTERND_OK) return st;
  hipError_t e = externd::run_q4_apply(w, mats, x, tokens, ldx, dtype, act, y, ws.ptr, s);
  if (e != hipSuccess) return hip_fail(e, "4-bit product");
  return EXTERND_OK;
}

// Checks that both passes of the gated block share.
int check_gated(const externd::GatedArgs& a) {
  if (bad_dtype(a.dtype)) return fail(EXTERND_EINVAL, "unknown dtype %d", a.dtype);
  if (a.dtype == EXTERND_F32) return fail(EXTERND_EUNSUPPORTED, "the gated block takes bf16 or fp16");
  if (bad_act(a.act)) return fail(EXTERND_EINVAL, "unknown activation %d", a.act);
  if (bad_size(a.rows, a.cols)) return fail(EXTERND_EINVAL, "bad weight shape");
  if (a.rows > kMaxGated || a.cols > kMaxGated)   // a tile's offsets are 32 bits
    return fail(EXTERND_EUNSUPPORTED, "the gated block takes at most 2^21 rows and columns of the weights");
  if (a.tokens < 0 || (a.tokens > 0 && (bad_size(a.tokens, a.cols) || bad_size(a.tokens, a.rows))))
    return fail(EXTERND_EINVAL, "bad number of tokens");
  if (bad_stride(a.ldx, a.cols) || bad_stride(a.ldw, a.cols))
    return fail(EXTERND_EINVAL, "ldx and ldw must be at least the columns");
  return EXTERND_OK;
}

}  // namespace

namespace externd {
int report(int status, const char* msg) { return fail(status, "%s", msg); }
thread_local bool g_single_placement = false;
}  // namespace externd

extern "C" {

const char* externd_status_string(int status) {
  switch (status) {
    case EXTERND_OK: return "ok";
    case EXTERND_EINVAL: return "invalid argument";
    case EXTERND_ENOMEM: return "out of device memory";
    case EXTERND_EHIP: return "HIP runtime error";
    case EXTERND_EUNSUPPORTED: return "unsupported device or shape";
    default: return "unknown status";
  }
}

const char* externd_last_error(void) { return g_last_error.c_str(); }

int externd_apply(const uint32_t* B2, const uint32_t* C2, const float* D, int64_t m, int64_t n,
                  int64_t k, const float* x, void* stream, float* y) {
  if (!x || !y) return fail(EXTERND_EINVAL, "null x or y pointer");
  if (bad_size(m, n) || k < 0 || k > (int64_t(1) << 31))
    return fail(EXTERND_EINVAL, "bad shape");
  if (k > 0 && (!B2 || !C2 || !D)) return fail(EXTERND_EINVAL, "null factor pointer");
  int st = check_device(nullptr);
  if (st != EXTERND_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  Workspace w;
  if ((st = alloc_ws(w, externd::apply_workspace_bytes(m, k), s)) != EXTERND_OK) return st;
  hipError_t e = externd::run_apply(B2, C2, D, m, n, k, x, y, w.ptr, s);
  if (e != hipSuccess) return hip_fail(e, "apply");
  return EXTERND_OK;
}

int externd_transpose_codes(const uint32_t* src, int64_t rows, int64_t cols, void* stream, uint32_t* dst) {
  if (rows < 0 || cols < 0 || rows > (int64_t(1) << 40) || cols > (int64_t(1) << 40))
    return fail(EXTERND_EINVAL, "bad shape");
  if (rows > 0 && cols > 0 && (!src || !dst)) return fail(EXTERND_EINVAL, "null code pointer");
  int st = check_device(nullptr);
  if (st != EXTERND_OK) return st;
  hipError_t e = externd::run_codes_transpose(src, rows, cols, dst, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "transpose_codes");
  return EXTERND_OK;
}

size_t externd_apply_rows_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  if (bad_size(m, n) || k < 0 || !externd::apply_rows_fits(m, n, k)) return 0;
  int cus = 0;
  if (check_device(&cus) != EXTERND_OK) return 0;
  return externd::apply_rows_workspace_bytes(m, k, cus);
}

int externd_apply_rows(const uint32_t* BT2, const uint32_t* C2, const float* D, int64_t m, int64_t n, int64_t k,
                       const float* x, void* stream, float* y, void* workspace, size_t workspace_bytes) {
  if (!x || !y) return fail(EXTERND_EINVAL, "null x or y pointer");
  if (bad_size(m, n) || k < 0 || !externd::apply_rows_fits(m, n, k))
    return fail(EXTERND_EINVAL, "bad shape (n and k at most 2^21)");
  if (k > 0 && (!BT2 || !C2 || !D)) return fail(EXTERND_EINVAL, "null factor pointer");
  int cus = 0;
  int st = check_device(&cus);
  if (st != EXTERND_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const size_t need = externd::apply_rows_workspace_bytes(m, k, cus);
  Workspace w;
  if (workspace) {
    if ((reinterpret_cast<uintptr_t>(workspace) & 255) != 0 || workspace_bytes < need)
      return fail(EXTERND_EINVAL, "workspace must be 256-byte aligned and at least %zu bytes", need);
    w.ptr = workspace;
  } else if ((st = alloc_ws(w, need, s)) != EXTERND_OK) {
    return st;
  }
  hipError_t e = externd::run_apply_rows(BT2, C2, D, m, n, k, x, y, w.ptr, cus, s);
  if (e != hipSuccess) return hip_fail(e, "apply_rows");
  return EXTERND_OK;
}

int64_t externd_rank(int64_t m, int64_t n, float mu) {
  if (m <= 0 || n <= 0 || !std::isfinite(mu) || mu < 0.f) return -1;
  const double v = (double)mu * (double)(m < n ? m : n);
  if (v > 9.0e15) return -1;
  const double whole = std::floor(v);
  return (int64_t)whole + ((v - whole) >= 0.5 ? 1 : 0);
}

int64_t externd_rank_for_energy(const double* trace, int64_t len, int64_t total, int32_t step,
                                double norm_a2, double target, double* energy) {
  if (energy) *energy = std::nan("");
  if (len < 0 || total < 0 || step < 1 || (len > 0 && !trace) || !std::isfinite(target) ||
      !std::isfinite(norm_a2) || norm_a2 < 0.0)
    return (fail(EXTERND_EINVAL, "bad arguments to externd_rank_for_energy"), -2);
  if (norm_a2 == 0.0) {
    if (energy) *energy = 1.0;
    return 0;
  }
  for (int64_t j = 0; j < len; ++j) {
    const double e = 1.0 - trace[j] / norm_a2;
    if (e >= target) {
      if (energy) *energy = e;
      const int64_t c = (j + 1) * (int64_t)step;
      return c < total ? c : total;
    }
  }
  return -1;
}

int32_t externd_block_width(int64_t m, int64_t n, int32_t block) {
  if (block <= 1 || m <= 0 || n <= 0) return 1;
  const int64_t cap = (m < n ? m : n) / 8;
  const int64_t b = block < cap ? block : cap;
  return b >= 2 ? (int32_t)b : 1;
}

int32_t externd_resident_fits(int64_t m, int64_t n) {
  int cus = 0;
  if (check_device(&cus) != EXTERND_OK) return 0;
  return externd::resident_fits(m, n, cus) ? 1 : 0;
}

uint64_t externd_workspace_bytes(int64_t m, int64_t n, float mu, int32_t block, int32_t mode) {
  if (bad_size(m, n)) return (fail(EXTERND_EINVAL, "bad shape"), 0);
  if (!std::isfinite(mu) || mu <= 0.f) return (fail(EXTERND_EINVAL, "mu must be finite and > 0"), 0);
  if (mode < -1 || mode > 2) return (fail(EXTERND_EINVAL, "bad mode %d", mode), 0);
  const int b = externd_block_width(m, n, block);
  if (b > 1) return externd::block_workspace_bytes(m, n, b);
  const int64_t k = externd_rank(m, n, mu);
  if (mode == EXTERND_MODE_STREAMING) return externd::stream_workspace_bytes(m, n);
  int cus = 0;
  if (check_device(&cus) != EXTERND_OK) return 0;
  const int md = seq_mode(mode, m, n, cus, false, false);
  if (md < 0) return (fail(EXTERND_EUNSUPPORTED, "%lld x %lld does not fit the %s kernel", (long long)m, (long long)n,
                           mode == EXTERND_MODE_RESIDENT ? "resident" : "persistent streaming"), 0);
  if (md == EXTERND_MODE_RESIDENT)
    return externd::resident_workspace_bytes(m, n, k, externd::resident_place_candidates(m, n, k));
  if (md == EXTERND_MODE_PERSISTENT) return externd::persist_workspace_bytes(m, n, k, cus);
  return externd::stream_workspace_bytes(m, n);
}

int externd_decompose(const float* A, int64_t m, int64_t n, float mu, float tau, int32_t iters,
                      int32_t block, void* stream, uint32_t* B2, uint32_t* C2, float* D,
                      double* energy, const externd_opts* opts) {
  if (!A || !energy) return fail(EXTERND_EINVAL, "null A or energy pointer");
  if (bad_size(m, n)) return fail(EXTERND_EINVAL, "bad shape %lld x %lld", (long long)m, (long long)n);
  if (!std::isfinite(mu) || mu <= 0.f) return fail(EXTERND_EINVAL, "mu must be finite and > 0");
  if (!std::isfinite(tau) || tau < 0.f) return fail(EXTERND_EINVAL, "tau must be finite and >= 0");
  if (iters < 1) return fail(EXTERND_EINVAL, "iters must be >= 1");
  const int64_t k = externd_rank(m, n, mu);
  if (k < 0 || k > (int64_t(1) << 31)) return fail(EXTERND_EINVAL, "rank out of range");
  if (k > 0 && (!B2 || !C2 || !D)) return fail(EXTERND_EINVAL, "null factor pointer");
  externd_opts o{};
  o.struct_size = sizeof(externd_opts);
  o.mode = EXTERND_MODE_AUTO;
  o.capture_component = -1;
  if (opts) {
    if (opts->struct_size != sizeof(externd_opts))
      return fail(EXTERND_EINVAL, "externd_opts.struct_size %u != %zu", opts->struct_size,
                  sizeof(externd_opts));
    o = *opts;
  }
  if (o.mode < -1 || o.mode > 2) return fail(EXTERND_EINVAL, "bad mode %d", o.mode);
  if (o.sweeps < 0) return fail(EXTERND_EINVAL, "sweeps must be >= 0");
  if (!std::isfinite(o.importance_lambda) || o.importance_lambda < 0.f)
    return fail(EXTERND_EINVAL, "importance_lambda must be finite and >= 0");
  if (o.ternarizer != EXTERND_TERN_MEAN && o.ternarizer != EXTERND_TERN_PROJECTION)
    return fail(EXTERND_EINVAL, "bad ternarizer %d", o.ternarizer);
  const bool projection = o.ternarizer == EXTERND_TERN_PROJECTION;
  if (projection && (m > externd::kProjMaxN || n > externd::kProjMaxN))
    return fail(EXTERND_EUNSUPPORTED, "the optimal projection takes vectors of at most %d entries",
                externd::kProjMaxN);
  if (projection && (o.mode == EXTERND_MODE_RESIDENT || o.mode == EXTERND_MODE_PERSISTENT))
    return fail(EXTERND_EUNSUPPORTED, "the optimal projection runs in streaming or block mode");
  if (o.workspace && (reinterpret_cast<uintptr_t>(o.workspace) & 255u) != 0)
    return fail(EXTERND_EINVAL, "workspace must be 256-byte aligned");
  if (o.safeguard != 0 && o.safeguard != 1) return fail(EXTERND_EINVAL, "bad safeguard %d", o.safeguard);
  const int b = externd_block_width(m, n, block);
  if (b > EXTERND_MAX_BLOCK)
    return fail(EXTERND_EUNSUPPORTED, "block width %d exceeds the widest supported block, %d", b,
                EXTERND_MAX_BLOCK);
  if (o.sweeps > 0 && b == 1)
    return fail(EXTERND_EINVAL, "refinement sweeps need block mode (block width %d)", b);
  if (o.safeguard && b > 1)
    return fail(EXTERND_EUNSUPPORTED, "the safeguard's replacement runs in the sequential path only");
  if (o.safeguard && projection)
    return fail(EXTERND_EUNSUPPORTED, "the safeguard is not combined with the optimal projection");
  if (o.safeguard && (o.mode == EXTERND_MODE_RESIDENT || o.mode == EXTERND_MODE_PERSISTENT))
    return fail(EXTERND_EUNSUPPORTED, "the safeguard's replacement runs in streaming mode");
  const externd_block_capture* bc = o.block_capture;
  if (bc && b > 1) {
    const int64_t nblocks = (k + b - 1) / b;
    if (bc->block < 0 || bc->block >= nblocks || bc->iteration < 0 || bc->iteration >= iters)
      return fail(EXTERND_EINVAL, "block capture (block %lld, iteration %d) out of range",
                  (long long)bc->block, bc->iteration);
  }
  int cus = 0;
  int st = check_device(&cus);
  if (st != EXTERND_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);

  if (b > 1) {
    externd::BlockArgs ba{};
    ba.A = A;
    ba.m = m;
    ba.n = n;
    ba.k = k;
    ba.b = b;
    ba.tau = tau;
    ba.iters = iters;
    ba.seed = o.seed;
    ba.B2 = B2;
    ba.C2 = C2;
    ba.D = D;
    ba.energy = energy;
    ba.trace = o.trace;
    ba.stats = reinterpret_cast<long long*>(o.stats);
    ba.norm_a2 = o.norm_a2;
    ba.sweeps = o.sweeps;
    ba.sweep_trace = o.sweep_trace;
    ba.importance = o.importance;
    ba.lambda = o.importance_lambda;
    ba.projection = projection ? 1 : 0;
    ba.cap = bc;
    Workspace w;
    if ((st = get_ws(w, o, externd::block_workspace_bytes(m, n, b), s)) != EXTERND_OK) return st;
    hipError_t e = externd::run_block(ba, w.ptr, s);
    if (e != hipSuccess) return hip_fail(e, "block decomposition");
    return EXTERND_OK;
  }

  externd::SeqArgs sa{};
  sa.A = A;
  sa.m = m;
  sa.n = n;
  sa.k = k;
  sa.tau = tau;
  sa.iters = iters;
  sa.seed = o.seed;
  sa.B2 = B2;
  sa.C2 = C2;
  sa.D = D;
  sa.energy = energy;
  sa.trace = o.trace;
  sa.stats = reinterpret_cast<long long*>(o.stats);
  sa.norm_a2 = o.norm_a2;
  sa.importance = o.importance;
  sa.lambda = o.importance_lambda;
  sa.projection = projection ? 1 : 0;
  sa.safeguard = o.safeguard;
  const bool any_capture = o.capture_R || o.capture_Rcol || o.capture_R_next || o.capture_y ||
                           o.capture_x || o.capture_v || o.capture_u || o.capture_d;
  sa.capture_component = o.capture_component;
  if (o.capture_component >= 0 && any_capture) {
    if (o.capture_component >= k) return fail(EXTERND_EINVAL, "capture_component >= k");
    sa.capture_R = o.capture_R;
    sa.capture_Rcol = o.capture_Rcol;
    sa.capture_R_next = o.capture_R_next;
    sa.capture_y = o.capture_y;
    sa.capture_x = o.capture_x;
    sa.capture_v = o.capture_v;
    sa.capture_u = o.capture_u;
    sa.capture_d = o.capture_d;
  } else {
    sa.capture_component = -1;
  }
  const int mode = seq_mode(o.mode, m, n, cus, projection, o.safeguard != 0);
  if (mode < 0)
    return fail(EXTERND_EUNSUPPORTED, "%lld x %lld does not fit the %s kernel", (long long)m, (long long)n,
                o.mode == EXTERND_MODE_RESIDENT ? "resident" : "persistent streaming");
  Workspace w;
  hipError_t e;
  if (mode == EXTERND_MODE_RESIDENT) {
    const int cands = externd::g_single_placement ? 1 : externd::resident_place_candidates(m, n, k);
    if ((st = get_ws(w, o, externd::resident_workspace_bytes(m, n, k, cands), s)) != EXTERND_OK) return st;
    int grid = 0;
    e = externd::run_resident_seq(sa, w.ptr, cands, cus, s, &grid);
    if (e != hipSuccess) return hip_fail(e, "resident decomposition");
  } else if (mode == EXTERND_MODE_PERSISTENT) {
    if ((st = get_ws(w, o, externd::persist_workspace_bytes(m, n, k, cus), s)) != EXTERND_OK) return st;
    e = externd::run_persist_seq(sa, w.ptr, cus, s);
    if (e != hipSuccess) return hip_fail(e, "persistent streaming decomposition");
  } else {
    if ((st = get_ws(w, o, externd::stream_workspace_bytes(m, n), s)) != EXTERND_OK) return st;
    e = externd::run_stream_seq(sa, w.ptr, s);
    if (e != hipSuccess) return hip_fail(e, "streaming decomposition");
  }
  return EXTERND_OK;
}

int externd_energy(const float* A, int64_t m, int64_t n, const uint32_t* B2, const uint32_t* C2,
                   const float* D, int64_t k, void* stream, double* energy) {
  if (!A || !energy) return fail(EXTERND_EINVAL, "null A or energy pointer");
  if (bad_size(m, n) || k < 0) return fail(EXTERND_EINVAL, "bad shape");
  if (k > 0 && (!B2 || !C2 || !D)) return fail(EXTERND_EINVAL, "null factor pointer");
  int st = check_device(nullptr);
  if (st != EXTERND_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  Workspace w;
  if ((st = alloc_ws(w, externd::energy_workspace_bytes(m, n), s)) != EXTERND_OK) return st;
  hipError_t e = externd::run_energy(A, m, n, B2, C2, D, k, energy, w.ptr, s);
  if (e != hipSuccess) return hip_fail(e, "energy");
  return EXTERND_OK;
}

int externd_reconstruct(const uint32_t* B2, const uint32_t* C2, const float* D, int64_t m,
                        int64_t n, int64_t k, void* stream, float* A_hat) {
  if (!A_hat) return fail(EXTERND_EINVAL, "null output pointer");
  if (bad_size(m, n) || k < 0) return fail(EXTERND_EINVAL, "bad shape");
  if (k > 0 && (!B2 || !C2 || !D)) return fail(EXTERND_EINVAL, "null factor pointer");
  int st = check_device(nullptr);
  if (st != EXTERND_OK) return st;
  hipError_t e = externd::run_reconstruct(B2, C2, D, m, n, k, A_hat, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "reconstruct");
  return EXTERND_OK;
}

int externd_ternarize(const float* x, int64_t N, float tau, void* stream, uint32_t* codes,
                      int32_t* nnz) {
  if (!x || !codes) return fail(EXTERND_EINVAL, "null pointer");
  if (N <= 0 || N > (int64_t(1) << 31) - 1) return fail(EXTERND_EINVAL, "bad length");
  if (!std::isfinite(tau) || tau < 0.f) return fail(EXTERND_EINVAL, "tau must be finite and >= 0");
  int st = check_device(nullptr);
  if (st != EXTERND_OK) return st;
  hipError_t e = externd::launch_ternarize(x, N, tau, codes, nnz, nullptr, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "ternarize");
  return EXTERND_OK;
}

int externd_project(const float* x, int64_t N, void* stream, uint32_t* codes, int32_t* nnz) {
  if (!x || !codes) return fail(EXTERND_EINVAL, "null pointer");
  if (N <= 0) return fail(EXTERND_EINVAL, "bad length");
  if (N > externd::kProjMaxN)
    return fail(EXTERND_EUNSUPPORTED, "the optimal projection takes at most %d entries", externd::kProjMaxN);
  int st = check_device(nullptr);
  if (st != EXTERND_OK) return st;
  hipError_t e = externd::launch_project(x, N, codes, nnz, nullptr, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "project");
  return EXTERND_OK;
}

int externd_gemv_t(const float* R, int64_t m, int64_t n, const uint32_t* u_codes, void* stream,
                   float* y) {
  if (!R || !u_codes || !y) return fail(EXTERND_EINVAL, "null pointer");
  if (bad_size(m, n)) return fail(EXTERND_EINVAL, "bad shape");
  int st = check_device(nullptr);
  if (st != EXTERND_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  Workspace w;
  if ((st = alloc_ws(w, sizeof(float) * (size_t)(externd::gemv_t_chunks(m) * n) + 256, s)) != EXTERND_OK) return st;
  hipError_t e = externd::launch_gemv_t(const_cast<float*>(R), m, n, u_codes,
                                        static_cast<float*>(w.ptr), y, nullptr, nullptr, nullptr, s);
  if (e != hipSuccess) return hip_fail(e, "gemv_t");
  return EXTERND_OK;
}

int externd_gemv_n(const float* R, int64_t m, int64_t n, const uint32_t* v_codes, void* stream,
                   float* x) {
  if (!R || !v_codes || !x) return fail(EXTERND_EINVAL, "null pointer");
  if (bad_size(m, n)) return fail(EXTERND_EINVAL, "bad shape");
  int st = check_device(nullptr);
  if (st != EXTERND_OK) return st;
  hipError_t e = externd::launch_gemv_n(R, m, n, v_codes, x, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "gemv_n");
  return EXTERND_OK;
}

int externd_deflate(float* R, int64_t m, int64_t n, const uint32_t* u_codes,
                    const uint32_t* v_codes, float d, void* stream) {
  if (!R || !u_codes || !v_codes) return fail(EXTERND_EINVAL, "null pointer");
  if (bad_size(m, n)) return fail(EXTERND_EINVAL, "bad shape");
  if (!std::isfinite(d)) return fail(EXTERND_EINVAL, "d must be finite");
  int st = check_device(nullptr);
  if (st != EXTERND_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  Workspace w;
  if ((st = alloc_ws(w, 256, s)) != EXTERND_OK) return st;
  float* dptr = static_cast<float*>(w.ptr);
  hipError_t e = externd::launch_fill_f32(dptr, 1, d, s);
  if (e == hipSuccess) e = externd::launch_deflate(R, m, n, u_codes, v_codes, dptr, s);
  if (e != hipSuccess) return hip_fail(e, "deflate");
  return EXTERND_OK;
}

int64_t externd_q4_code_words(int64_t rows, int64_t cols) {
  if (bad_size(rows, cols)) return -1;
  return 256 * q4_blocks(rows, cols);
}

int64_t externd_q4_table_len(int64_t rows, int64_t cols, int32_t group) {
  if (bad_size(rows, cols) || bad_group(group)) return -1;
  return 2048 / group * q4_blocks(rows, cols);
}

size_t externd_q4_workspace_bytes(int64_t cols, int64_t tokens, int32_t dtype) {
  if (bad_size(1, cols) || tokens < 0 || tokens > kMaxTokens || bad_dtype(dtype)) return 0;
  return externd::q4_stage_bytes(cols, tokens, dtype);
}

int externd_q4_quantize(const void* W, int64_t rows, int64_t cols, int64_t ldw, int32_t dtype, int32_t group,
                        void* stream, uint32_t* codes, uint16_t* scales, uint16_t* mins) {
  if (!W) return fail(EXTERND_EINVAL, "null W");
  if (bad_dtype(dtype)) return fail(EXTERND_EINVAL, "unknown dtype %d", dtype);
  if (bad_size(rows, cols) || bad_stride(ldw, cols)) return fail(EXTERND_EINVAL, "bad shape or stride");
  if (!aligned_to(W, dtype_bytes(dtype))) return fail(EXTERND_EINVAL, "W must be aligned to its type");
  const externd_q4 w = {codes, scales, mins, rows, cols, group, 0};
  int st = check_q4(&w, "output");
  if (st != EXTERND_OK) return st;
  const int64_t e_bytes = (int64_t)dtype_bytes(dtype);
  st = check_apart({packed(codes, q4_code_bytes(w), "codes"), packed(scales, q4_table_bytes(w), "scales"),
                    packed(mins, q4_table_bytes(w), "mins")},
                   {{W, rows, cols * e_bytes, ldw * e_bytes, "W"}});
  if (st != EXTERND_OK) return st;
  if ((st = check_device(nullptr)) != EXTERND_OK) return st;
  hipError_t e = externd::run_q4_quantize(W, rows, cols, ldw, dtype, group, codes, scales, mins,
                                          static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "q4_quantize");
  return EXTERND_OK;
}

int externd_q4_pack(const uint8_t* codes_in, const uint16_t* scales_in, const uint16_t* mins_in, int64_t rows,
                    int64_t cols, int32_t group, void* stream, uint32_t* codes, uint16_t* scales, uint16_t* mins) {
  if (!codes_in || !scales_in) return fail(EXTERND_EINVAL, "null input");
  if ((mins_in == nullptr) != (mins == nullptr)) return fail(EXTERND_EINVAL, "mins_in and mins go together");
  if (!aligned_to(scales_in, 2) || !aligned_to(mins_in, 2)) return fail(EXTERND_EINVAL, "misaligned input");
  const externd_q4 w = {codes, scales, mins, rows, cols, group, 0};
  int st = check_q4(&w, "output");
  if (st != EXTERND_OK) return st;
  const int64_t table_in = 2 * rows * ((cols + group - 1) / group);
  st = check_apart({packed(codes, q4_code_bytes(w), "codes"), packed(scales, q4_table_bytes(w), "scales"),
                    packed(mins, q4_table_bytes(w), "mins")},
                   {packed(codes_in, rows * cols, "codes_in"), packed(scales_in, table_in, "scales_in"),
                    packed(mins_in, table_in, "mins_in")});
  if (st != EXTERND_OK) return st;
  if ((st = check_device(nullptr)) != EXTERND_OK) return st;
  hipError_t e = externd::run_q4_pack(codes_in, scales_in, mins_in, rows, cols, group, codes, scales, mins,
                                      static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "q4_pack");
  return EXTERND_OK;
}

int externd_q4_reconstruct(const externd_q4* w, int32_t dtype, void* stream, void* out) {
  int st = check_q4(w, "weights");
  if (st != EXTERND_OK) return st;
  if (bad_dtype(dtype)) return fail(EXTERND_EINVAL, "unknown dtype %d", dtype);
  if (!out || !aligned_to(out, dtype_bytes(dtype))) return fail(EXTERND_EINVAL, "null or misaligned output");
  st = check_apart({packed(out, w->rows * w->cols * (int64_t)dtype_bytes(dtype), "the output")},
                   {packed(w->codes, q4_code_bytes(*w), "codes"), packed(w->scales, q4_table_bytes(*w), "scales"),
                    packed(w->mins, q4_table_bytes(*w), "mins")});
  if (st != EXTERND_OK) return st;
  if ((st = check_device(nullptr)) != EXTERND_OK) return st;
  hipError_t e = externd::run_q4_reconstruct(*w, dtype, out, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "q4_reconstruct");
  return EXTERND_OK;
}

int externd_q4_apply(const externd_q4* w, const void* x, int64_t tokens, int64_t ldx, int32_t dtype, void* stream,
                     void* y, void* workspace, size_t workspace_bytes) {
  int st = check_q4(w, "weights");
  if (st != EXTERND_OK) return st;
  return q4_product(w, 1, x, tokens, ldx, dtype, EXTERND_ACT_SILU, stream, y, workspace, workspace_bytes);
}

int externd_q4_gated(const externd_q4* wg, const externd_q4* wu, const void* x, int64_t tokens, int64_t ldx,
                     int32_t dtype, int32_t act, void* stream, void* h, void* workspace, size_t workspace_bytes) {
  int st = check_q4(wg, "gate weights");
  if (st != EXTERND_OK) return st;
  if ((st = check_q4(wu, "up weights")) != EXTERND_OK) return st;
  if (wg->rows != wu->rows || wg->cols != wu->cols || wg->group != wu->group ||
      (wg->mins == nullptr) != (wu->mins == nullptr))
    return fail(EXTERND_EINVAL, "gate and up weights differ in shape, group or kind");
  if (bad_act(act)) return fail(EXTERND_EINVAL, "unknown activation %d", act);
  const externd_q4 both[2] = {*wg, *wu};
  return q4_product(both, 2, x, tokens, ldx, dtype, act, stream, h, workspace, workspace_bytes);
}

size_t externd_gated_forward_workspace_bytes(int64_t tokens, int64_t cols, int64_t rows, int32_t aligned) {
  if (bad_size(rows, cols) || tokens < 1 || bad_size(tokens, cols) || bad_size(tokens, rows)) return 0;
  int cus = 0;
  if (check_device(&cus) != EXTERND_OK) return 0;
  const size_t with = externd::gated_forward_workspace_bytes(tokens, cols, rows, true, cus);
  if (aligned) return with;
  // for any alignment: few unaligned tokens may need none where aligned ones have split sums
  return std::max(with, externd::gated_forward_workspace_bytes(tokens, cols, rows, false, cus));
}

int externd_gated_forward(const void* x, int64_t tokens, int64_t cols, int64_t ldx, const void* wg, const void* wu,
                          int64_t rows, int64_t ldw, int32_t dtype, int32_t act, void* stream, void* h, float* g,
                          float* u, void* workspace, size_t workspace_bytes) {
  externd::GatedArgs a = {};
  a.x = x; a.wg = wg; a.wu = wu;
  a.tokens = tokens; a.cols = cols; a.rows = rows;
  a.ldx = ldx; a.ldw = ldw;
  a.dtype = dtype; a.act = act;
  a.h = h; a.g = g; a.u = u;
  int st = check_gated(a);
  if (st != EXTERND_OK) return st;
  if ((g == nullptr) != (u == nullptr)) return fail(EXTERND_EINVAL, "g and u go together");
  if (tokens == 0) return EXTERND_OK;
  if (!x || !wg || !wu || !h) return fail(EXTERND_EINVAL, "null pointer");
  if (!aligned_to(x, 2) || !aligned_to(wg, 2) || !aligned_to(wu, 2) || !aligned_to(h, 2) || !aligned_to(g, 4) ||
      !aligned_to(u, 4))
    return fail(EXTERND_EINVAL, "pointers must be aligned to their type");
  const Region rx = {x, tokens, 2 * cols, 2 * ldx, "x"}, rg = {wg, rows, 2 * cols, 2 * ldw, "wg"},
               ru = {wu, rows, 2 * cols, 2 * ldw, "wu"}, oh = packed(h, 2 * tokens * rows, "h"),
               og = packed(g, 4 * tokens * rows, "g"), ou = packed(u, 4 * tokens * rows, "u");
  if ((st = check_apart({oh, og, ou}, {rx, rg, ru})) != EXTERND_OK) return st;
  if ((st = check_device(&a.cus)) != EXTERND_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  Workspace ws;
  const size_t need =
      externd::gated_forward_workspace_bytes(tokens, cols, rows, externd::gated_is_aligned(a), a.cus);
  if ((st = check_apart({packed(workspace, (int64_t)need, "workspace")}, {rx, rg, ru, oh, og, ou})) != EXTERND_OK) return st;
  if ((st = op_ws(ws, workspace, workspace_bytes, need, s)) != EXTERND_OK) return st;
  hipError_t e = externd::run_gated_forward(a, ws.ptr, s);
  if (e != hipSuccess) return hip_fail(e, "gated forward");
  return EXTERND_OK;
}

size_t externd_gated_backward_workspace_bytes(int64_t tokens, int64_t cols, int64_t rows, int32_t aligned) {
  if (bad_size(rows, cols) || tokens < 1 || bad_size(tokens, cols) || bad_size(tokens, rows)) return 0;
  int cus = 0;
  if (check_device(&cus) != EXTERND_OK) return 0;
  return externd::gated_backward_workspace_bytes(tokens, cols, rows, aligned != 0, cus);
}

int externd_gated_backward(const void* x, int64_t tokens, int64_t cols, int64_t ldx, const void* wg, const void* wu,
                           int64_t rows, int64_t ldw, const float* g, const float* u, const void* dh, int64_t lddh,
                           int32_t dtype, int32_t act, void* stream, void* dx, void* dwg, void* dwu, void* workspace,
                           size_t workspace_bytes) {
  externd::GatedArgs a = {};
  a.x = x; a.wg = wg; a.wu = wu;
  a.tokens = tokens; a.cols = cols; a.rows = rows;
  a.ldx = ldx; a.ldw = ldw;
  a.dtype = dtype; a.act = act;
  a.g = const_cast<float*>(g); a.u = const_cast<float*>(u);
  a.dh = dh; a.lddh = lddh;
  a.dx = dx; a.dwg = dwg; a.dwu = dwu;
  int st = check_gated(a);
  if (st != EXTERND_OK) return st;
  if (bad_stride(lddh, rows)) return fail(EXTERND_EINVAL, "lddh must be at least the rows of the weights");
  if ((dwg == nullptr) != (dwu == nullptr)) return fail(EXTERND_EINVAL, "dwg and dwu go together");
  if (!dx && !dwg) return EXTERND_OK;
  if (tokens > 0 && (!x || !wg || !wu || !g || !u || !dh)) return fail(EXTERND_EINVAL, "null pointer");
  if (tokens == 0 && !dwg) return EXTERND_OK;
  if (!aligned_to(x, 2) || !aligned_to(wg, 2) || !aligned_to(wu, 2) || !aligned_to(dh, 2) || !aligned_to(dx, 2) ||
      !aligned_to(dwg, 2) || !aligned_to(dwu, 2) || !aligned_to(g, 4) || !aligned_to(u, 4))
    return fail(EXTERND_EINVAL, "pointers must be aligned to their type");
  const Region rx = {x, tokens, 2 * cols, 2 * ldx, "x"}, rwg = {wg, rows, 2 * cols, 2 * ldw, "wg"},
               rwu = {wu, rows, 2 * cols, 2 * ldw, "wu"}, rg = packed(g, 4 * tokens * rows, "g"),
               ru = packed(u, 4 * tokens * rows, "u"), rdh = {dh, tokens, 2 * rows, 2 * lddh, "dh"},
               ox = packed(dx, 2 * tokens * cols, "dx"), og = packed(dwg, 2 * rows * cols, "dwg"),
               ou = packed(dwu, 2 * rows * cols, "dwu");
  if ((st = check_apart({ox, og, ou}, {rx, rwg, rwu, rg, ru, rdh})) != EXTERND_OK) return st;
  if ((st = check_device(&a.cus)) != EXTERND_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  Workspace ws;
  const size_t need =
      tokens > 0
          ? externd::gated_backward_workspace_bytes(tokens, cols, rows, externd::gated_is_aligned(a), a.cus)
          : 0;
  if ((st = check_apart({packed(workspace, (int64_t)need, "workspace")}, {rx, rwg, rwu, rg, ru, rdh, ox, og, ou})) != EXTERND_OK)
    return st;
  if ((st = op_ws(ws, workspace, workspace_bytes, need, s)) != EXTERND_OK) return st;
  hipError_t e = externd::run_gated_backward(a, ws.ptr, s);
  if (e != hipSuccess) return hip_fail(e, "gated backward");
  return EXTERND_OK;
}

}  // extern "C"
