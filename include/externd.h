/*
 * externd.h — C ABI of the MI355X (gfx950) ExTernD library.
 *
 * ExTernD ("ExTernD: Expanded-Rank Ternary Decomposition Ternary LLM PTQ with
 * Accuracy Approaching Any Quantization Level") approximates a real matrix
 * A (m x n) by B diag(D) C with ternary B (m x k), ternary C (k x n) and real
 * D (k), k = mu * min(m, n) (§2.1).  Component i is fitted to the residual
 * R = A - sum_{j<i} d_j b_j c_j^T by a fixed number of alternating ternary fits
 * v = T_tau(R^T u), u = T_tau(R v) (§2.3 step 1, T_tau of §2.2), given the
 * least-squares scale d = u^T R v / (|u|^2 |v|^2) (§2.3 step 2) and deflated
 * out of R (§2.3 step 3).  Block mode extracts b components at a time with
 * decorrelated targets and a joint scale solve (§2.4).
 *
 * Conventions for every entry point:
 *  - Pointers named A, R, x, y, B2, C2, D, energy, trace, stats, capture_* and
 *    workspace are DEVICE pointers (hipMalloc'd or equivalent) on the current
 *    HIP device.  The caller owns every buffer; the library never frees them.
 *  - Matrices are row-major and densely packed (leading dimension = columns).
 *  - `stream` is a hipStream_t passed as void* (NULL = the default stream).
 *    All device work is enqueued on it; entry points return without waiting
 *    for it, so device outputs are valid once the stream has completed.
 *  - Argument errors are detected on the host before anything is enqueued
 *    and return EXTERND_EINVAL; device-side failures return EXTERND_EHIP with
 *    a message available from externd_last_error().
 *  - 2-bit ternary codes: a row of length L occupies ceil(L/16) uint32 words;
 *    element j sits in bits 2*(j%16)..2*(j%16)+1 of word j/16 with
 *    00 = 0, 01 = +1, 11 = -1 (10 never produced).  Padding bits are 00.
 *    B2 is component-major: row i (ceil(m/16) words) holds column i of B.
 *    C2 row i (ceil(n/16) words) holds row i of C.
 */
#ifndef EXTERND_H
#define EXTERND_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum externd_status {
  EXTERND_OK = 0,
  EXTERND_EINVAL = 1,       /* bad argument (null pointer, size, non-finite knob) */
  EXTERND_ENOMEM = 2,       /* workspace allocation failed or too small */
  EXTERND_EHIP = 3,         /* HIP runtime error or a failed kernel launch */
  EXTERND_EUNSUPPORTED = 4  /* device is not gfx950 / shape outside a mode's limits */
};

/* Execution modes of the sequential path. */
enum externd_mode {
  EXTERND_MODE_AUTO = -1,      /* resident when the shape fits on chip, else persistent streaming
                                  when it applies, else streaming */
  EXTERND_MODE_STREAMING = 0,  /* R in device memory, a few kernels per ALS half-step */
  EXTERND_MODE_RESIDENT = 1,   /* one cooperative kernel, R kept in LDS/VGPRs */
  EXTERND_MODE_PERSISTENT = 2  /* one cooperative kernel, R in device memory: n % 4 == 0,
                                  m, n <= 10240 and at most 64 rows per CU; not with the
                                  optimal projection or an applied safeguard */
};

enum externd_ternarizer { EXTERND_TERN_MEAN = 0, EXTERND_TERN_PROJECTION = 1 };

/* Indices into the optional int64 statistics array (EXTERND_STATS_LEN entries). */
enum externd_stat {
  EXTERND_STAT_SUM_NNZ_U = 0,   /* sum over components and iterations of nnz(u_t) */
  EXTERND_STAT_SUM_NNZ_V = 1,   /* same for v_t */
  EXTERND_STAT_NNZ_B = 2,       /* nonzeros in the final B */
  EXTERND_STAT_NNZ_C = 3,       /* nonzeros in the final C */
  EXTERND_STAT_FALLBACKS = 4,   /* T_tau calls that fell back to the single largest entry */
  EXTERND_STAT_NONFINITE = 5,   /* non-finite entries found in A (energy is NaN if > 0) */
  EXTERND_STAT_MODE = 6,        /* mode actually run (0 streaming, 1 resident, 2 block,
                                   3 persistent streaming) */
  EXTERND_STAT_GRID = 7,        /* workgroups of the resident or persistent kernel (0 otherwise) */
  EXTERND_STAT_RIDGE_RETRIES = 8, /* block mode: joint scale solves retried with a ridge */
  EXTERND_STAT_TIMEOUTS = 9,    /* waits that ran out (energy is NaN): resident exchange, or
                                   block mode's Gram-before-inverse wait */
  EXTERND_STAT_INVERSE_UNCONVERGED = 10, /* block mode, b <= 64: Gram inverses whose fp64
                                    residual ||I - (G + eps I) X||_F stayed at or above 1e-3
                                    after the fp64 refinement (the inverse is then not known
                                    to 1e-6); wider blocks invert exactly in fp64: always 0 */
  EXTERND_STAT_SWEEP_KEPT_OLD = 11, /* block mode: sweep visits that kept the stored block */
  EXTERND_STAT_NS_ITERATIONS = 12,  /* block mode, b <= 64: Newton-Schulz residual evaluations over all Gram inverses */
  EXTERND_STAT_NS_RESTARTS = 13,    /* block mode, b <= 64: warm starts replaced by another start */
  EXTERND_STAT_ITERATIONS = 14,     /* ALS iterations run, over all components (blocks) */
  EXTERND_STAT_SAFEGUARD = 15,      /* components (sequential) or blocks (block mode) whose
                                       decrease of ||R||^2 fell below the single-entry bound
                                       max_ij w_j R_ij^2 of the residual before them, i.e.
                                       where the §7 safeguard would replace the fit; counted
                                       whether or not opts.safeguard applies it (extraction
                                       only, not refinement sweeps) */
  EXTERND_STATS_LEN = 16
};

/*
 * Test capture of one iteration of one block of the block path (§2.4), for
 * checking every step of it on identical inputs.  Every pointer is a device
 * buffer and may be NULL (that item is not recorded).  Rows are components:
 * a row of P, Vt, Q or Ut holds one column of the paper's n x b or m x b
 * matrix.  bb is the width of the captured block (b, or k mod b for a
 * trailing partial block).  Only the extraction pass is captured, not
 * refinement sweeps.
 */
typedef struct externd_block_capture {
  int64_t block;       /* block index: components [block * b, block * b + bb) */
  int32_t iteration;   /* ALS iteration whose two half-steps are recorded (0-based) */
  int32_t reserved;
  float* R;            /* m x n: the residual the block is fitted to */
  uint32_t* U_in;      /* bb x ceil(m/16) code words: U entering the iteration */
  float* P;            /* bb x n: U^T R, summed over the contraction's splits */
  float* GinvU;        /* bb x bb: (U^T U + eps I)^-1 as applied */
  float* Vt;           /* bb x n: decorrelated V target (P (U^T U + eps I)^-1)^T */
  uint32_t* V;         /* bb x ceil(n/16): T_tau of each row of Vt */
  float* Q;            /* bb x m: (R diag(w) V)^T (w = 1 unless importance weighted) */
  float* GinvV;        /* bb x bb: (V^T diag(w) V + eps I)^-1 as applied */
  float* Ut;           /* bb x m: decorrelated U target */
  uint32_t* U_out;     /* bb x ceil(m/16): T_tau of each row of Ut */
  double* rhs;         /* bb: u_j . q_j of the final iteration (joint-solve right side) */
} externd_block_capture;

/*
 * Optional knobs of externd_decompose.  Zero-initialise, set struct_size to
 * sizeof(externd_opts), then set what you need.  A NULL opts means defaults.
 */
typedef struct externd_opts {
  uint32_t struct_size;   /* sizeof(externd_opts) */
  uint32_t reserved0;
  uint64_t seed;          /* starting-vector seed (default 0) */
  int32_t mode;           /* enum externd_mode; sequential path only (default AUTO) */
  int32_t reserved1;
  double* trace;          /* device, optional: ||R||^2 after each component
                             (sequential: k entries, predicted from the exact
                             per-step decrease) or after each block (block mode:
                             ceil(k/b) entries) */
  int64_t* stats;         /* device, optional: EXTERND_STATS_LEN counters (overwritten) */
  /* Test capture of one component of the sequential path.  It is enabled
   * when capture_component >= 0 and at least one capture pointer is
   * non-NULL (a zero-initialised opts captures nothing); each pointer may be
   * NULL. */
  int64_t capture_component;
  float* capture_R;       /* m*n: residual before the component (row-resident copy) */
  float* capture_Rcol;    /* m*n: the same residual from the column-resident copy */
  float* capture_R_next;  /* m*n: residual after the component's deflation */
  float* capture_y;       /* iters*n: y_t = R^T u_{t-1} */
  float* capture_x;       /* iters*m: x_t = R v_t */
  int8_t* capture_v;      /* iters*n: v_t */
  int8_t* capture_u;      /* iters*m: u_t (u_0 is the seeded start) */
  float* capture_d;       /* 1: the component's scale */
  /* Caller-owned device workspace (optional).  When non-NULL it must be
   * 256-byte aligned and hold at least externd_workspace_bytes(...) bytes for
   * the same arguments; the library then allocates nothing.  Its contents are
   * scratch: nothing is expected in it and nothing is left for the caller.
   * Two calls in flight at once must not share one workspace. */
  void* workspace;
  uint64_t workspace_bytes;
  double* norm_a2;        /* device, optional: receives ||A||_F^2 (fp64) */
  /* Refinement sweeps (§2.4, block mode only; EXTERND_EINVAL when the block
   * width is 1).  After extraction every sweep revisits the blocks in order:
   * the block is added back to R, its iterations run again from its stored U,
   * the scales are solved jointly, and the refit replaces the block when its
   * predicted decrease of ||R||^2 is at least the stored block's (measured
   * exactly while adding it back), else the stored block is deflated again.
   * The energy therefore never falls from sweep to sweep (up to the fp32
   * rounding of the deflations). */
  int32_t sweeps;         /* default 0 */
  /* Ternarizer (§2.2): EXTERND_TERN_MEAN (default) is T_tau; with
   * EXTERND_TERN_PROJECTION every ternarization is the optimal ternary
   * projection (keep the s largest |x| maximising their sum over sqrt(s);
   * tau is unused).  The projection runs in streaming and block mode only
   * (AUTO picks streaming) and needs m, n <= 16384; otherwise
   * EXTERND_EUNSUPPORTED. */
  int32_t ternarizer;
  double* sweep_trace;    /* device, optional: sweeps entries, predicted ||R||^2 after each sweep */
  /* Importance-weighted ALS (§2.5, every mode).  importance: device, n
   * per-input-channel second moments h >= 0 (e.g. from an importance matrix);
   * the column weights are w_j = h_j / max(h) + importance_lambda, computed
   * in fp32 on the device (w = lambda when h is all zero).  The objective is
   * sum_ij w_j (A - B diag(D) C)_ij^2: the u update targets R diag(w) v, the v
   * update keeps the plain R^T u, d = u^T R diag(w) v / (|u|^2 v^T diag(w) v)
   * (0 when v^T diag(w) v = 0), block mode uses the Gram V^T diag(w) V, and
   * energy, trace, sweep_trace and norm_a2 are the weighted sums.  Negative or
   * non-finite entries of h count as non-finite input (energy NaN). */
  const float* importance;
  float importance_lambda; /* >= 0, finite (default 0) */
  /* Single-entry safeguard (appendix §7, monotone residual decrease): when
   * the fitted component lowers ||R||^2 by less than max_ij w_j R_ij^2 (the
   * decrease of the single entry e_r e_c^T with d = R_rc), replace it by that
   * entry; the smallest row-major index r n + c takes a tie.  0 (default)
   * leaves every fit as it is; stats[EXTERND_STAT_SAFEGUARD] counts the
   * would-be replacements either way.  1 applies it: sequential path only,
   * run in streaming mode (AUTO picks streaming; RESIDENT and block mode give
   * EXTERND_EUNSUPPORTED). */
  int32_t safeguard;
  const externd_block_capture* block_capture; /* HOST pointer, optional (block mode) */
} externd_opts;

/*
 * Decompose A (m x n, fp32, row-major) into k = externd_rank(m, n, mu)
 * components.  §2.3 (block <= 1) or §2.4 (block > 1).
 *   mu     > 0, finite: inner-rank multiplier (§2.1).
 *   tau    >= 0, finite: threshold scale of T_tau (§2.2), used as fp32.
 *   iters  >= 1: alternating-fit iterations per component / block (§2.3: 15).
 *   block  <= 1: sequential greedy ALS; otherwise block ALS with
 *          b = externd_block_width(m, n, block) (falls back to sequential if < 2;
 *          EXTERND_EUNSUPPORTED if b > EXTERND_MAX_BLOCK).
 * Outputs (device): B2 [k][ceil(m/16)] u32, C2 [k][ceil(n/16)] u32, D [k] fp32,
 *   energy [1] fp64 = 1 - ||A - B diag(D) C||^2 / ||A||^2 of the fp32 residual
 *   (1 when ||A|| = 0; NaN when A has non-finite entries).
 * A is not modified.  Workspace is opts->workspace when given (EXTERND_ENOMEM if
 * smaller than externd_workspace_bytes, EXTERND_EINVAL if not 256-byte
 * aligned), else allocated and freed stream-ordered on `stream`.
 */
int externd_decompose(const float* A, int64_t m, int64_t n, float mu, float tau,
                      int32_t iters, int32_t block, void* stream,
                      uint32_t* B2, uint32_t* C2, float* D, double* energy,
                      const externd_opts* opts);

/*
 * externd_decompose for callers that cannot allocate device memory (code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * allocation): the same arguments and results, on the resident sequential
 * path only (block widths above 1, EXTERND_MODE_STREAMING and shapes that do
 * not fit on chip give EXTERND_EUNSUPPORTED; opts->workspace must be NULL).
 * Its scratch memory is a static 256 KiB device array per GPU, held until
 * the process ends, so it calls no allocator; it holds one placement of the
 * exchange words (16 KB (ceil(m/1024) + ceil(n/1024)) rounded up to 16 KB,
 * plus 2 KB), so this entry point skips the placement probe that
 * externd_decompose runs for long decompositions (the factors are the
 * same).  A shape needing more scratch (the words, 4 n + k / 8 bytes, and
 * about 40 KB: 146.5 KiB at 2560 x 2560 with k = 5120) gives
 * EXTERND_ENOMEM.  All calls on
 * one GPU share that array (each call clears what it needs first): calls
 * that overlap on one GPU, on any streams, race and must not be issued.
 */
int externd_decompose_noalloc(const float* A, int64_t m, int64_t n, float mu, float tau,
                              int32_t iters, int32_t block, void* stream,
                              uint32_t* B2, uint32_t* C2, float* D, double* energy,
                              const externd_opts* opts);

/* energy = 1 - ||A - B diag(D) C||^2 / ||A||^2 accumulated in fp64 from the
 * 2-bit factors (§2.1).  k may be 0 (energy 0, or 1 for A = 0). */
int externd_energy(const float* A, int64_t m, int64_t n, const uint32_t* B2,
                   const uint32_t* C2, const float* D, int64_t k, void* stream,
                   double* energy);

/* A_hat = B diag(D) C (m x n fp32 row-major), accumulated in fp64 per entry (§2.1). */
int externd_reconstruct(const uint32_t* B2, const uint32_t* C2, const float* D,
                        int64_t m, int64_t n, int64_t k, void* stream, float* A_hat);

/* Inference with the factors (§2.6): y = B (diag(D) (C x)) for x of length n,
 * y of length m.  C x and B w are sums of signed copies (no multiplies; k
 * multiplies for w = D * C x), accumulated in fp32 in a fixed order.  B2, C2,
 * D as produced by externd_decompose; k may be 0 (y = 0).  Workspace of about
 * 4 (k + m k / 64) bytes is allocated and freed stream-ordered. */
int externd_apply(const uint32_t* B2, const uint32_t* C2, const float* D, int64_t m, int64_t n,
                  int64_t k, const float* x, void* stream, float* y);

/* Transpose a 2-bit code matrix (the §2.6 storage: 16 codes per uint32, code
 * j of a word in bits 2j, 2j+1): src holds `rows` rows of `cols` codes,
 * ceil(cols/16) words per row; dst receives `cols` rows of `rows` codes,
 * ceil(rows/16) words per row, zero padding.  externd_transpose_codes(B2, k,
 * m, ...) turns the component-major B2 of externd_decompose into B row by
 * row, the form externd_apply_rows reads (once per factorisation).  Device
 * pointers owned by the caller, dst not overlapping src; enqueued on
 * `stream`.  EXTERND_EINVAL for a negative size or a null pointer with
 * nonzero sizes. */
int externd_transpose_codes(const uint32_t* src, int64_t rows, int64_t cols, void* stream, uint32_t* dst);

/* y = B (diag(D) (C x)) (§2.6) with B given row by row: BT2 holds m rows of
 * ceil(k/16) words (externd_transpose_codes of B2); C2 and D as produced by
 * externd_decompose; x has n entries, y receives m.  Both products run on
 * int8 MFMA: the vector (x, then w = D (C x) in fp32) is rounded to fixed
 * point with 30 bits below its largest magnitude and split into four int8
 * digits, every ternary sum is an exact integer, and each output is
 * converted once.  So the result is the exact one for the rounded vector
 * (each entry moved by at most 2^-30 of the vector's largest magnitude),
 * independent of summation order and bit-reproducible.  n, k <= 2^21
 * (EXTERND_EINVAL beyond).  A non-finite entry of x, D or w makes y all
 * NaN.  k may be 0 (y = 0).  workspace: NULL, and a workspace of
 * externd_apply_rows_workspace_bytes(m, n, k) bytes (4 k plus a few KiB) is
 * allocated and freed stream-ordered; or a caller device buffer, 256-byte
 * aligned, of at least that many bytes (workspace_bytes), used instead, so
 * that a loop of calls allocates nothing (EXTERND_EINVAL if too small or
 * misaligned).  Calls that overlap on one workspace race. */
int externd_apply_rows(const uint32_t* BT2, const uint32_t* C2, const float* D, int64_t m, int64_t n,
                       int64_t k, const float* x, void* stream, float* y, void* workspace,
                       size_t workspace_bytes);

/* Workspace bytes externd_apply_rows needs for this shape on the current
 * device; 0 for an invalid shape or device. */
size_t externd_apply_rows_workspace_bytes(int64_t m, int64_t n, int64_t k);

/* k = mu * min(m, n) rounded half away from zero in fp64 (§2.1); -1 on bad input. */
int64_t externd_rank(int64_t m, int64_t n, float mu);

/* Rank needed for a target energy (§3.3: choosing mu per matrix), read off
 * one decomposition's trace thanks to the greedy prefix property: the run at
 * a smaller rank is the prefix of the run at a larger one (in block mode the
 * smaller rank must be a whole number of blocks).  HOST arrays: trace[j] is
 * ||R||^2 after component j (sequential, step = 1) or after block j (block
 * mode, step = b); total is the decomposition's k; norm_a2 its ||A||^2
 * (externd_opts.norm_a2).  Returns the smallest c = min((j+1) step, total)
 * with 1 - trace[j] / norm_a2 >= target, 0 when norm_a2 = 0, -1 when no
 * prefix reaches the target, and -2 on invalid arguments.  mu = c / min(m, n)
 * reproduces c through externd_rank.  energy (HOST, may be NULL) receives the
 * energy of the returned prefix: 1 - trace[j] / norm_a2, 1 when norm_a2 = 0,
 * NaN when no prefix reaches the target or the arguments are invalid. */
int64_t externd_rank_for_energy(const double* trace, int64_t len, int64_t total, int32_t step,
                                double norm_a2, double target, double* energy);

/* Block width of a request: min(block, floor(min(m,n)/8)), 1 meaning
 * sequential (§2.4).  The block kernels take widths up to
 * EXTERND_MAX_BLOCK: externd_decompose returns EXTERND_EUNSUPPORTED for a
 * wider one (e.g. the pages' default 256 on a matrix with min(m, n) >=
 * 2048), rather than silently narrowing the block. */
#define EXTERND_MAX_BLOCK 128
int32_t externd_block_width(int64_t m, int64_t n, int32_t block);

/* 1 if the resident sequential kernel can hold an m x n residual on chip. */
int32_t externd_resident_fits(int64_t m, int64_t n);

/* Bytes of device workspace externd_decompose needs for these arguments
 * (mode as in externd_opts.mode; it only matters for the sequential path).
 * Without opts->workspace the library allocates this much stream-ordered
 * (hipMallocAsync) and frees it stream-ordered before returning.  For the
 * resident path of a long decomposition (k >= 1024 and m n >= 2^20) it
 * includes 8 placements of the exchange words, which a short probe times
 * before the run to keep the fastest (about 852 KB at 2560 x 2560, k =
 * 5120; one placement otherwise).  Returns 0
 * for invalid arguments, or when the AUTO/RESIDENT choice needs the device
 * and no gfx950 device is current; externd_last_error() says which. */
uint64_t externd_workspace_bytes(int64_t m, int64_t n, float mu, int32_t block, int32_t mode);

/* ---- single-step entry points (the same device routines as the streaming path) ---- */

/* codes = T_tau(x) for a length-N fp32 vector (§2.2); nnz (device int32, may
 * be NULL) receives the number of nonzeros. */
int externd_ternarize(const float* x, int64_t N, float tau, void* stream,
                      uint32_t* codes, int32_t* nnz);

/* codes = the optimal ternary projection of a length-N fp32 vector (§2.2):
 * the s largest |x_j| keep their signs, s maximising their sum over sqrt(s);
 * the sort takes equal magnitudes in index order, and prefixes are compared
 * exactly on the fixed-point magnitudes of T_tau's mean.  1 <= N <= 16384
 * (EXTERND_EUNSUPPORTED above).  nnz as for externd_ternarize. */
int externd_project(const float* x, int64_t N, void* stream, uint32_t* codes, int32_t* nnz);

/* y = R^T u for R (m x n) and u given as 2-bit codes of length m (§2.3 step 1). */
int externd_gemv_t(const float* R, int64_t m, int64_t n, const uint32_t* u_codes,
                   void* stream, float* y);

/* x = R v for v given as 2-bit codes of length n (§2.3 step 1). */
int externd_gemv_n(const float* R, int64_t m, int64_t n, const uint32_t* v_codes,
                   void* stream, float* x);

/* R <- R - d u v^T in place, one fp32 rounding per entry (§2.3 step 3). */
int externd_deflate(float* R, int64_t m, int64_t n, const uint32_t* u_codes,
                    const uint32_t* v_codes, float d, void* stream);

/* ---- 4-bit weights with group scales ----
 *
 * The storage that the ternary factors are weighed against, and its products
 * with a few tokens.  A group is `group` neighbouring entries of a row (32, 64
 * or 128; the last group of a row may be shorter) with a bf16 scale s and,
 * asymmetric, a bf16 minimum m:
 *   symmetric:  s = bf16(max|w| / 7), code c = clamp(rint(w / s), -8, 7) + 8, value s (c - 8);
 *   asymmetric: s = bf16((max w - min w) / 15), m = bf16(min w),
 *               c = clamp(rint((w - m) / s), 0, 15), value s c + m.
 * Steps are fp32, rint takes ties to even, and a group of scale 0 has c = 8
 * (symmetric) or 0.  A group with a non-finite entry, or whose scale overflows,
 * gets a NaN scale: all its values are NaN.
 *
 * Layout: tiles of 16 rows by chunks of 128 columns, tile-major,
 * ceil(rows/16) x ceil(cols/128) of them:
 *   codes:  256 uint32 words per tile of a chunk.  Word 4 l + i, l = r + 16 p
 *           (r < 16, p < 4, i < 4), holds row r's codes of columns
 *           32 i + 8 p + j, j = 0..7: j = 2 e in bits 4 e .. 4 e + 3, j = 2 e + 1
 *           in bits 16 + 4 e .. 19 + 4 e.
 *   scales, mins: bf16, 16 x (128 / group) per tile of a chunk, row r's groups
 *           at r * (128 / group).
 * Padding entries may hold any code; padding scales and minima must be
 * finite.  codes must be 16-byte aligned, scales and mins 8-byte.
 *
 * What these functions and those of the gated block, the linear layer and the experts below write, the workspace
 * included, must have no byte in common with what they read or write besides
 * (EXTERND_EINVAL); what they only read may overlap. */
enum externd_dtype { EXTERND_F32 = 0, EXTERND_BF16 = 1, EXTERND_F16 = 2 };
enum externd_activation {
  EXTERND_ACT_SILU = 0,      /* g / (1 + exp(-g)) */
  EXTERND_ACT_GELU = 1,      /* g (1 + erf(g / sqrt 2)) / 2 */
  EXTERND_ACT_GELU_TANH = 2, /* g (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))) / 2 */
  EXTERND_ACT_NONE = 3       /* g; of the linear layer alone */
};

typedef struct externd_q4 {
  const uint32_t* codes;   /* device */
  const uint16_t* scales;  /* device */
  const uint16_t* mins;    /* device, NULL: symmetric */
  int64_t rows, cols;
  int32_t group;           /* 32, 64 or 128 */
  int32_t reserved;
} externd_q4;

/* Elements of codes (uint32) and of scales or mins (bf16) in the layout above;
 * -1 for a bad shape or group. */
int64_t externd_q4_code_words(int64_t rows, int64_t cols);
int64_t externd_q4_table_len(int64_t rows, int64_t cols, int32_t group);

/* Quantize W (rows x cols of dtype, rows ldw >= cols entries apart).  mins
 * NULL: symmetric.  Padding is written too. */
int externd_q4_quantize(const void* W, int64_t rows, int64_t cols, int64_t ldw, int32_t dtype, int32_t group,
                        void* stream, uint32_t* codes, uint16_t* scales, uint16_t* mins);

/* Bring codes made elsewhere into the layout: codes_in one byte each (rows x
 * cols, low four bits), scales_in and mins_in bf16, rows x ceil(cols/group).
 * mins_in and mins are both NULL or both given. */
int externd_q4_pack(const uint8_t* codes_in, const uint16_t* scales_in, const uint16_t* mins_in, int64_t rows,
                    int64_t cols, int32_t group, void* stream, uint32_t* codes, uint16_t* scales, uint16_t* mins);

/* The values (rows x cols of dtype, packed), each rounded once. */
int externd_q4_reconstruct(const externd_q4* w, int32_t dtype, void* stream, void* out);

/* y[t] = W x[t] for `tokens` rows of x (cols entries of dtype, ldx >= cols
 * entries apart); y is tokens x rows of dtype, packed.  Sums are fp32, in an
 * order that does not depend on timing; fp32 x is split into three bf16 parts
 * that add up to it exactly.  Codes enter as 16 + c, and the 16 (or 24) is taken off
 * again: so the |x| of each group have to add up to less than 2^123, past which
 * a sum may overflow that W x does not, and an infinite entry of x makes its token's
 * outputs NaN, as a NaN does.  tokens may be 0, at most 2^20.
 * workspace: NULL, and where x needs a staged copy (fp32 of more than 5 tokens, rows
 * that are not all 16-byte aligned, more than 16 tokens on a large matrix)
 * externd_q4_workspace_bytes bytes are allocated and freed stream-ordered; or a caller device buffer, 256-byte aligned, of at least
 * that many bytes, used instead.  Calls that overlap on one workspace race. */
int externd_q4_apply(const externd_q4* w, const void* x, int64_t tokens, int64_t ldx, int32_t dtype, void* stream,
                     void* y, void* workspace, size_t workspace_bytes);

/* h[t] = act(Wg x[t]) * (Wu x[t]), both projections in one kernel; wg and wu
 * have one shape, group size and kind.  Everything else as externd_q4_apply. */
int externd_q4_gated(const externd_q4* wg, const externd_q4* wu, const void* x, int64_t tokens, int64_t ldx,
                     int32_t dtype, int32_t act, void* stream, void* h, void* workspace, size_t workspace_bytes);

/* Workspace bytes that covers externd_q4_apply and externd_q4_gated for any
 * alignment of x; 0 for a bad shape or dtype. */
size_t externd_q4_workspace_bytes(int64_t cols, int64_t tokens, int32_t dtype);

/* ---- gated feed-forward block, dense 16-bit weights ----
 *
 * h = act(x Wg^T) * (x Wu^T): x tokens x cols (rows ldx entries apart), Wg and Wu
 * rows x cols (rows ldw entries apart), h tokens x rows, packed; dtype
 * EXTERND_BF16 or EXTERND_F16 (fp32 is EXTERND_EUNSUPPORTED: its matrix rate is
 * a sixteenth).  Sums and the activation are fp32 and h is rounded once.  g and u
 * (both or neither): tokens x rows fp32, the projections, kept for the
 * backward pass.  Strides are in entries, at least cols; rows and cols are at
 * most 2^21 (EXTERND_EUNSUPPORTED beyond).  tokens may be 0.
 * workspace: as for externd_q4_apply, of externd_gated_forward_workspace_bytes
 * bytes (which may be 0).  Its `aligned` says that x, Wg and Wu start on 16 bytes
 * and that cols, ldx and ldw are multiples of 8 (strides below 2^22); the
 * products of more than 32 tokens read padded copies otherwise, kept in the
 * workspace.  aligned = 0 gives what covers any alignment.  The bytes are those of this
 * number of tokens: fewer tokens may need more, as their sums are split. */
int externd_gated_forward(const void* x, int64_t tokens, int64_t cols, int64_t ldx, const void* wg, const void* wu,
                          int64_t rows, int64_t ldw, int32_t dtype, int32_t act, void* stream, void* h, float* g,
                          float* u, void* workspace, size_t workspace_bytes);
size_t externd_gated_forward_workspace_bytes(int64_t tokens, int64_t cols, int64_t rows, int32_t aligned);

/* Gradients of the block from dh (tokens x rows, rows lddh entries apart) and
 * the g and u that the forward pass kept:
 *   dg = dh u act'(g), du = dh act(g)   (held in two parts of dtype, to twice its bits; in
 *     fp16 scaled by a power of two per token for dx and per hidden unit for dWg and dWu, so
 *     that a gradient in fp16's range does not overflow or vanish on its way)
 *   dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x   (fp32 sums, rounded once).
 * dx (tokens x cols) may be NULL; dwg and dwu (rows x cols) are both given or
 * both NULL.  Outputs are packed.  With tokens = 0, dwg and dwu are zero.
 * workspace: as above, of externd_gated_backward_workspace_bytes bytes. */
int externd_gated_backward(const void* x, int64_t tokens, int64_t cols, int64_t ldx, const void* wg, const void* wu,
                           int64_t rows, int64_t ldw, const float* g, const float* u, const void* dh, int64_t lddh,
                           int32_t dtype, int32_t act, void* stream, void* dx, void* dwg, void* dwu, void* workspace,
                           size_t workspace_bytes);
size_t externd_gated_backward_workspace_bytes(int64_t tokens, int64_t cols, int64_t rows, int32_t aligned);

/* ---- linear layer, dense 16-bit weights ----
 *
 * z = x W^T + bias, y = act(z) + residual: x tokens x cols (rows ldx entries apart), W rows x cols
 * (rows ldw entries apart), bias (rows entries) and residual (tokens x rows, rows ldr entries apart)
 * NULL or of dtype, y tokens x rows, packed; dtype EXTERND_BF16 or EXTERND_F16.  Sums, the activation
 * and the residual's sum are fp32, and y is rounded once.  z (or NULL): tokens x rows fp32, kept for the
 * backward pass of an activation.  Limits, workspace and its `aligned` (of x and W) as for
 * externd_gated_forward. */
int externd_linear_forward(const void* x, int64_t tokens, int64_t cols, int64_t ldx, const void* w, int64_t rows,
                           int64_t ldw, const void* bias, const void* residual, int64_t ldr, int32_t dtype, int32_t act,
                           void* stream, void* y, float* z, void* workspace, size_t workspace_bytes);
size_t externd_linear_forward_workspace_bytes(int64_t tokens, int64_t cols, int64_t rows, int32_t aligned);

/* Gradients of the layer from dy (tokens x rows, rows lddy entries apart) and, unless act is
 * EXTERND_ACT_NONE, the z that the forward pass kept:
 *   dz = dy act'(z)   (held in two parts of dtype, in fp16 scaled, as the gated block's dg; without an
 *     activation dz is dy)
 *   dx = dz W, dW = dz^T x, db = the sum of dz over the tokens   (fp32 sums, rounded once).
 * Each of dx (tokens x cols), dw (rows x cols) and db (rows) may be NULL; they are packed.  The
 * residual's gradient is dy.  With tokens = 0, dw and db are zero.  `aligned` says besides that dy starts on 16
 * bytes and that lddy and rows are multiples of 8. */
int externd_linear_backward(const void* x, int64_t tokens, int64_t cols, int64_t ldx, const void* w, int64_t rows,
                            int64_t ldw, const float* z, const void* dy, int64_t lddy, int32_t dtype, int32_t act,
                            void* stream, void* dx, void* dw, void* db, void* workspace, size_t workspace_bytes);
size_t externd_linear_backward_workspace_bytes(int64_t tokens, int64_t cols, int64_t rows, int32_t act, int32_t aligned);

/* ---- mixture-of-experts layer for a few tokens, dense 16-bit weights ----
 *
 * Each token goes through `top` of the experts, gated blocks with a projection back:
 *   y[t] = sum over j of weights[t][j] * Wd_e (act(Wg_e x[t]) * (Wu_e x[t])),  e = ids[t][j].
 * Sums, activations and what lies between the products are fp32 or more (fp16: each slot's hidden values to 2^-39 of its
 * largest), and y is rounded once.  dtype of x, the experts and y: EXTERND_BF16 or EXTERND_F16.  tokens * top at most EXTERND_MOE_SLOTS, experts at most 1024, top at
 * most 64 and at most the experts, rows and cols at most 2^21 (EXTERND_EUNSUPPORTED beyond). */
#define EXTERND_MOE_SLOTS 8192

typedef struct externd_moe_weights {
  const void *wg, *wu;   /* device: experts x rows x cols, rows up_ld and experts up_stride entries apart */
  const void* wd;        /* device: experts x cols x rows, rows down_ld and experts down_stride entries apart */
  int64_t experts, rows, cols;   /* rows: hidden units of an expert; cols: the layer's width */
  int64_t up_ld, up_stride, down_ld, down_stride;
} externd_moe_weights;

/* Routing: logits x Wr^T (Wr experts x cols of wr_dtype, dtype or EXTERND_F32, rows ldr entries apart), summed
 * in 64 bits; ids (tokens x top): the experts of the largest logits, largest first, the lower index where
 * logits are equal, NaN after all others; weights (tokens x top, fp32): exp(logit) over the sum of those of the chosen experts
 * (normalize) or of all.  workspace: NULL, and externd_moe_workspace_bytes(tokens, cols, 0, experts, top) bytes are
 * allocated and freed stream-ordered; or a caller buffer of at least as many, 256-byte aligned. */
int externd_moe_route(const void* x, int64_t tokens, int64_t cols, int64_t ldx, const void* wr, int64_t experts, int64_t ldr,
                      int32_t wr_dtype, int32_t dtype, int32_t top, int32_t normalize, void* stream, int32_t* ids,
                      float* weights, void* workspace, size_t workspace_bytes);

/* The experts' sum for a choice that was made before: ids (tokens x top; one outside the experts adds nothing, one twice adds
 * twice) and weights.  workspace as above, of externd_moe_workspace_bytes(tokens, cols, rows, experts, top) bytes. */
int externd_moe_experts(const void* x, int64_t tokens, int64_t ldx, const int32_t* ids, const float* weights, int32_t top,
                        const externd_moe_weights* w, int32_t dtype, int32_t act, void* stream, void* y, void* workspace,
                        size_t workspace_bytes);

/* Both: the whole layer, ids and weights written too. */
int externd_moe(const void* x, int64_t tokens, int64_t ldx, const void* wr, int64_t ldr, int32_t wr_dtype, int32_t top,
                int32_t normalize, const externd_moe_weights* w, int32_t dtype, int32_t act, void* stream, void* y,
                int32_t* ids, float* weights, void* workspace, size_t workspace_bytes);

/* Workspace that covers the three calls (rows = 0: externd_moe_route alone); 0 for what they refuse. */
size_t externd_moe_workspace_bytes(int64_t tokens, int64_t cols, int64_t rows, int64_t experts, int32_t top);

/* ---- AdamW step over many tensors ----
 *
 * Per entry, steps in fp32:
 *   g1 = g grad_scale, m1 = beta1 m + (1 - beta1) g1, v1 = beta2 v + (1 - beta2) (g1 g1),
 *   w1 = (1 - lr decay) w - lr / (1 - beta1^t) * m1 / (sqrt(v1) / sqrt(1 - beta2^t) + eps)
 * with t the number of this step: one count for all tensors, also for those that earlier steps left
 * out.  w is the tensor's master weight where it has one, and the parameter becomes its rounding; else
 * the parameter.
 *
 * Moments are kept for whole blocks of EXTERND_ADAMW_BLOCK entries (as is the master weight),
 * 0 past the tensor's end.  bits = 32: fp32.  bits = 8: a byte per entry, and a byte b per
 * block, max(15, the exponent field of the largest finite fp32 magnitude in it):
 *   m: the OCP e4m3 number nearest to m 2^(134 - b); 0x7f or 0xff, a NaN, where m is not finite;
 *   v: the number nearest to v 2^(141 - b) with five bits of exponent (bias 15, subnormals)
 *      and three of mantissa, no sign; 1 rather than 0 where v > 0; 0xf8 for infinity and 0xff for a NaN.
 * Ties go to the even code.  All codes 0 and b = 15 are zeros. */
#define EXTERND_ADAMW_BLOCK 256

typedef struct externd_adamw_tensor {
  void* param;             /* device, n entries of param_dtype */
  const void* grad;        /* device, n entries of grad_dtype */
  float* master;           /* device, 16-byte aligned, or NULL; not for fp32 parameters */
  void *m, *v;             /* device: fp32 and 16-byte aligned, or codes, 4-byte aligned */
  uint8_t *m_exp, *v_exp;  /* device, a byte per block; NULL with bits = 32 */
  int64_t n;               /* 0: left out */
  float decay;             /* weight decay */
  int32_t param_dtype, grad_dtype;   /* externd_dtype */
  int32_t reserved;
} externd_adamw_tensor;

typedef struct externd_adamw_opts {
  double lr, beta1, beta2, eps;     /* betas in 0 <= beta < 1, eps >= 0 */
  const float* lr_device;           /* device, read by the kernel instead of lr; or NULL */
  const float* grad_scale_device;   /* device, read instead of grad_scale; or NULL */
  float grad_scale;
  int32_t bits;                     /* 8 or 32 */
  double* step;                     /* device, four: steps taken, beta1 and beta2 to that power, 0 (the
                                       kernel's own).  0, 1, 1, 0 before the first step. */
} externd_adamw_opts;

/* One step of `count` tensors (a HOST array); the step is counted on the device, so that a
 * captured call counts in each replay.  What is written must have no byte in common with
 * anything else that the call reads or writes.  Calls that overlap on one state race. */
int externd_adamw_step(const externd_adamw_tensor* tensors, int64_t count, const externd_adamw_opts* opts, void* stream);

/* The fp32 values of 8-bit moments of `blocks` blocks. */
int externd_adamw_moments(const uint8_t* m, const uint8_t* m_exp, const uint8_t* v, const uint8_t* v_exp, int64_t blocks,
                          void* stream, float* m_out, float* v_out);

/* Status text and the last error message of the calling thread. */
const char* externd_status_string(int status);
const char* externd_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* EXTERND_H */
