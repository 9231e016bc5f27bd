"""Python binding of libexternd.so, the MI355X ExTernD library.

ExTernD ("ExTernD: Expanded-Rank Ternary Decomposition Ternary LLM PTQ with
Accuracy Approaching Any Quantization Level", §2) factors a weight matrix as
A ~ B diag(D) C with ternary B, C.  Every step runs in the HIP kernels behind
the C ABI declared in include/externd.h; this module only marshals torch
tensors (device memory) and the current HIP stream into those calls.  It
raises ImportError when the shared library has not been built; there is no
fallback implementation.
"""
import ctypes
import os

import torch

__all__ = [
    "decompose", "decompose_noalloc", "energy", "reconstruct", "apply", "rank", "block_width", "resident_fits",
    "workspace_bytes",
    "rank_for_energy", "mu_for_energy", "project",
    "ternarize", "gemv_t", "gemv_n", "deflate", "Decomposition", "ExterndError",
    "Q4", "q4_quantize", "q4_pack", "q4_reconstruct", "q4_apply", "q4_gated", "q4_workspace_bytes",
    "gated", "gated_forward", "gated_backward", "gated_forward_workspace_bytes", "gated_backward_workspace_bytes",
    "STAT", "MODE_AUTO", "MODE_STREAMING", "MODE_RESIDENT", "MODE_PERSISTENT", "library_path",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libexternd.so")

MODE_AUTO, MODE_STREAMING, MODE_RESIDENT, MODE_PERSISTENT = -1, 0, 1, 2
STATS_LEN = 16
STAT = {"sum_nnz_u": 0, "sum_nnz_v": 1, "nnz_b": 2, "nnz_c": 3, "fallbacks": 4,
        "nonfinite": 5, "mode": 6, "grid": 7, "ridge_retries": 8, "timeouts": 9,
        "inverse_unconverged": 10, "sweep_kept_old": 11, "ns_iterations": 12, "ns_restarts": 13,
        "iterations": 14, "safeguard": 15}

if not os.path.exists(library_path):
    raise ImportError(f"{library_path} is missing; build it with "
                      "`python ternary_rank_weight_amd/build.py`")
_lib = ctypes.CDLL(library_path)

_p = ctypes.c_void_p
_i64 = ctypes.c_int64
_i32 = ctypes.c_int32
_f32 = ctypes.c_float


class _BlockCapture(ctypes.Structure):
    _fields_ = [
        ("block", ctypes.c_int64), ("iteration", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("R", _p), ("U_in", _p), ("P", _p), ("GinvU", _p), ("Vt", _p), ("V", _p),
        ("Q", _p), ("GinvV", _p), ("Ut", _p), ("U_out", _p), ("rhs", _p),
    ]


class _Opts(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32), ("reserved0", ctypes.c_uint32),
        ("seed", ctypes.c_uint64), ("mode", ctypes.c_int32), ("reserved1", ctypes.c_int32),
        ("trace", _p), ("stats", _p),
        ("capture_component", ctypes.c_int64),
        ("capture_R", _p), ("capture_Rcol", _p), ("capture_R_next", _p),
        ("capture_y", _p), ("capture_x", _p), ("capture_v", _p), ("capture_u", _p),
        ("capture_d", _p),
        ("workspace", _p), ("workspace_bytes", ctypes.c_uint64),
        ("norm_a2", _p),
        ("sweeps", _i32), ("ternarizer", _i32), ("sweep_trace", _p),
        ("importance", _p), ("importance_lambda", ctypes.c_float), ("safeguard", _i32),
        ("block_capture", ctypes.POINTER(_BlockCapture)),
    ]


class _Q4(ctypes.Structure):
    _fields_ = [("codes", _p), ("scales", _p), ("mins", _p), ("rows", _i64), ("cols", _i64),
                ("group", _i32), ("reserved", _i32)]


def _sig(name, res, args):
    f = getattr(_lib, name)
    f.restype = res
    f.argtypes = args
    return f


_decompose = _sig("externd_decompose", ctypes.c_int,
                  [_p, _i64, _i64, _f32, _f32, _i32, _i32, _p, _p, _p, _p, _p, ctypes.POINTER(_Opts)])
_decompose_noalloc = _sig("externd_decompose_noalloc", ctypes.c_int,
                          [_p, _i64, _i64, _f32, _f32, _i32, _i32, _p, _p, _p, _p, _p, ctypes.POINTER(_Opts)])
_energy = _sig("externd_energy", ctypes.c_int, [_p, _i64, _i64, _p, _p, _p, _i64, _p, _p])
_reconstruct = _sig("externd_reconstruct", ctypes.c_int, [_p, _p, _p, _i64, _i64, _i64, _p, _p])
_apply = _sig("externd_apply", ctypes.c_int, [_p, _p, _p, _i64, _i64, _i64, _p, _p, _p])
_apply_rows = _sig("externd_apply_rows", ctypes.c_int, [_p, _p, _p, _i64, _i64, _i64, _p, _p, _p, _p, ctypes.c_size_t])
_apply_rows_ws = _sig("externd_apply_rows_workspace_bytes", ctypes.c_size_t, [_i64, _i64, _i64])
_transpose_codes = _sig("externd_transpose_codes", ctypes.c_int, [_p, _i64, _i64, _p, _p])
_rank = _sig("externd_rank", ctypes.c_int64, [_i64, _i64, _f32])
_block_width = _sig("externd_block_width", ctypes.c_int32, [_i64, _i64, _i32])
_resident_fits = _sig("externd_resident_fits", ctypes.c_int32, [_i64, _i64])
_workspace_bytes = _sig("externd_workspace_bytes", ctypes.c_uint64, [_i64, _i64, _f32, _i32, _i32])
_rank_for_energy = _sig("externd_rank_for_energy", ctypes.c_int64,
                        [ctypes.POINTER(ctypes.c_double), _i64, _i64, _i32, ctypes.c_double, ctypes.c_double,
                         ctypes.POINTER(ctypes.c_double)])
_ternarize = _sig("externd_ternarize", ctypes.c_int, [_p, _i64, _f32, _p, _p, _p])
_project = _sig("externd_project", ctypes.c_int, [_p, _i64, _p, _p, _p])
_gemv_t = _sig("externd_gemv_t", ctypes.c_int, [_p, _i64, _i64, _p, _p, _p])
_gemv_n = _sig("externd_gemv_n", ctypes.c_int, [_p, _i64, _i64, _p, _p, _p])
_deflate = _sig("externd_deflate", ctypes.c_int, [_p, _i64, _i64, _p, _p, _f32, _p])
_pq4 = ctypes.POINTER(_Q4)
_size = ctypes.c_size_t
_q4_quantize = _sig("externd_q4_quantize", ctypes.c_int, [_p, _i64, _i64, _i64, _i32, _i32, _p, _p, _p, _p])
_q4_pack = _sig("externd_q4_pack", ctypes.c_int, [_p, _p, _p, _i64, _i64, _i32, _p, _p, _p, _p])
_q4_reconstruct = _sig("externd_q4_reconstruct", ctypes.c_int, [_pq4, _i32, _p, _p])
_q4_apply = _sig("externd_q4_apply", ctypes.c_int, [_pq4, _p, _i64, _i64, _i32, _p, _p, _p, _size])
_q4_gated = _sig("externd_q4_gated", ctypes.c_int, [_pq4, _pq4, _p, _i64, _i64, _i32, _i32, _p, _p, _p, _size])
_q4_ws = _sig("externd_q4_workspace_bytes", _size, [_i64, _i64, _i32])
_q4_code_words = _sig("externd_q4_code_words", _i64, [_i64, _i64])
_q4_table_len = _sig("externd_q4_table_len", _i64, [_i64, _i64, _i32])
_gated_forward = _sig("externd_gated_forward", ctypes.c_int,
                      [_p, _i64, _i64, _i64, _p, _p, _i64, _i64, _i32, _i32, _p, _p, _p, _p, _p, _size])
_gated_forward_ws = _sig("externd_gated_forward_workspace_bytes", _size, [_i64, _i64, _i64, _i32])
_gated_backward = _sig("externd_gated_backward", ctypes.c_int,
                       [_p, _i64, _i64, _i64, _p, _p, _i64, _i64, _p, _p, _p, _i64, _i32, _i32, _p, _p, _p, _p, _p,
                        _size])
_gated_backward_ws = _sig("externd_gated_backward_workspace_bytes", _size, [_i64, _i64, _i64, _i32])
_status_string = _sig("externd_status_string", ctypes.c_char_p, [ctypes.c_int])
_last_error = _sig("externd_last_error", ctypes.c_char_p, [])

# Every exported symbol of the C ABI, for load checks.
ABI_SYMBOLS = ("externd_decompose", "externd_decompose_noalloc", "externd_energy", "externd_reconstruct", "externd_apply",
               "externd_apply_rows", "externd_apply_rows_workspace_bytes", "externd_transpose_codes", "externd_rank",
               "externd_block_width", "externd_resident_fits", "externd_workspace_bytes",
               "externd_rank_for_energy",
               "externd_ternarize", "externd_project",
               "externd_gemv_t", "externd_gemv_n", "externd_deflate",
               "externd_q4_code_words", "externd_q4_table_len", "externd_q4_quantize", "externd_q4_pack",
               "externd_q4_reconstruct", "externd_q4_apply", "externd_q4_gated", "externd_q4_workspace_bytes",
               "externd_gated_forward", "externd_gated_forward_workspace_bytes",
               "externd_gated_backward", "externd_gated_backward_workspace_bytes",
               "externd_status_string", "externd_last_error")


class ExterndError(RuntimeError):
    def __init__(self, status):
        self.status = status
        super().__init__(f"{_status_string(status).decode()}: {_last_error().decode()}")


def _check(status):
    if status != 0:
        raise ExterndError(status)


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _need(t, dtype, name):
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def rank(m, n, mu):
    """k = mu * min(m, n) rounded half away from zero (§2.1)."""
    return int(_rank(m, n, mu))


def block_width(m, n, block):
    """Block width used for a request (§2.4); 1 means sequential."""
    return int(_block_width(m, n, block))


def resident_fits(m, n):
    return bool(_resident_fits(m, n))


def workspace_bytes(m, n, mu, block=0, mode=MODE_AUTO):
    """Device workspace externd_decompose needs for these arguments (0: invalid)."""
    return int(_workspace_bytes(m, n, mu, block, mode))


class Decomposition:
    """Device outputs of one decomposition.

    B2: (k, ceil(m/16)) int32 words of 2-bit codes (component-major B),
    C2: (k, ceil(n/16)) int32 words (rows of C), D: (k,) float32,
    energy: (1,) float64, trace / stats: optional device tensors,
    capture: dict of captured tensors when requested.
    """

    def __init__(self, m, n, k, B2, C2, D, energy, trace, stats, capture, norm_a2=None, block=1):
        self.m, self.n, self.k = m, n, k
        self.B2, self.C2, self.D, self.energy = B2, C2, D, energy
        self.trace, self.stats, self.capture = trace, stats, capture
        self.norm_a2, self.block = norm_a2, block

    def stat(self, name):
        return int(self.stats[STAT[name]].item())


def decompose(A, mu, tau, iters=15, block=0, seed=0, mode=MODE_AUTO, trace=False, stats=False,
              capture=None, out=None, workspace=None, sweeps=0, importance=None, lam=0.0,
              projection=False, safeguard=False, block_capture=None, _entry=None):
    """Run externd_decompose on the current stream.

    A: (m, n) float32 CUDA tensor.  capture: component index whose
    intermediate vectors and residuals are recorded (sequential path only).
    out: optional Decomposition whose B2/C2/D/energy buffers are reused.
    workspace: optional contiguous CUDA tensor used as the library's scratch
    memory (at least workspace_bytes(...) bytes, 256-byte aligned); the
    library then allocates nothing.
    sweeps: refinement sweeps after extraction (block mode only); with
    trace=True their predicted ||R||^2 values land in .sweep_trace.
    importance: optional (n,) float32 CUDA tensor of per-input-channel second
    moments h; the column weights are h / max(h) + lam (importance-weighted
    ALS), and energy / trace / norm_a2 become weighted.
    projection: use the optimal ternary projection instead of T_tau
    (streaming or block mode; AUTO picks streaming).
    safeguard: apply the single-entry safeguard (sequential path, streaming
    mode); stats["safeguard"] counts the would-be replacements either way.
    block_capture: (block index, iteration) of the block path to record; the
    tensors land in .block_capture (R, U_in, P, GinvU, Vt, V, Q, GinvV, Ut,
    U_out, rhs; rows are components, codes as int32 words).
    """
    _need(A, torch.float32, "A")
    if A.dim() != 2:
        raise ValueError("A must be 2-D")
    m, n = A.shape
    k = rank(m, n, mu)
    if k < 0:
        raise ValueError("bad mu")
    dev = A.device
    if out is not None and (out.m, out.n, out.k) == (m, n, k):
        B2, C2, D, E = out.B2, out.C2, out.D, out.energy
    else:
        B2 = torch.empty((k, (m + 15) // 16), dtype=torch.int32, device=dev)
        C2 = torch.empty((k, (n + 15) // 16), dtype=torch.int32, device=dev)
        D = torch.empty((k,), dtype=torch.float32, device=dev)
        E = torch.empty((1,), dtype=torch.float64, device=dev)
    b = block_width(m, n, block)
    ntrace = ((k + b - 1) // b) if b > 1 else k
    tr = torch.empty((max(ntrace, 1),), dtype=torch.float64, device=dev) if trace else None
    st = torch.zeros((STATS_LEN,), dtype=torch.int64, device=dev) if stats else None
    na2 = torch.empty((1,), dtype=torch.float64, device=dev) if trace else None
    swt = torch.empty((sweeps,), dtype=torch.float64, device=dev) if trace and sweeps > 0 else None
    opts = _Opts()
    opts.struct_size = ctypes.sizeof(_Opts)
    opts.seed = seed
    opts.mode = mode
    opts.trace = _ptr(tr)
    opts.stats = _ptr(st)
    opts.norm_a2 = _ptr(na2)
    opts.sweeps = int(sweeps)
    opts.sweep_trace = _ptr(swt)
    if importance is not None:
        _need(importance, torch.float32, "importance")
        if importance.dim() != 1 or importance.numel() != n:
            raise ValueError("importance must have n entries")
        opts.importance = _ptr(importance)
    opts.importance_lambda = float(lam)
    opts.ternarizer = 1 if projection else 0
    opts.safeguard = 1 if safeguard else 0
    opts.capture_component = -1
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or workspace.device.type != "cuda" \
                or not workspace.is_contiguous():
            raise TypeError("workspace must be a contiguous CUDA tensor")
        opts.workspace = _ptr(workspace)
        opts.workspace_bytes = workspace.numel() * workspace.element_size()
    cap = None
    if capture is not None:
        cap = {
            "R": torch.empty((m, n), dtype=torch.float32, device=dev),
            "Rcol": torch.empty((m, n), dtype=torch.float32, device=dev),
            "R_next": torch.empty((m, n), dtype=torch.float32, device=dev),
            "y": torch.empty((iters, n), dtype=torch.float32, device=dev),
            "x": torch.empty((iters, m), dtype=torch.float32, device=dev),
            "v": torch.empty((iters, n), dtype=torch.int8, device=dev),
            "u": torch.empty((iters, m), dtype=torch.int8, device=dev),
            "d": torch.empty((1,), dtype=torch.float32, device=dev),
        }
        opts.capture_component = int(capture)
        opts.capture_R = _ptr(cap["R"])
        opts.capture_Rcol = _ptr(cap["Rcol"])
        opts.capture_R_next = _ptr(cap["R_next"])
        opts.capture_y = _ptr(cap["y"])
        opts.capture_x = _ptr(cap["x"])
        opts.capture_v = _ptr(cap["v"])
        opts.capture_u = _ptr(cap["u"])
        opts.capture_d = _ptr(cap["d"])
    bcap = None
    if block_capture is not None:
        blk, it = block_capture
        bb = min(b, k - blk * b) if b > 1 else 0
        if b <= 1 or not 0 <= blk * b < k:
            raise ValueError("block_capture needs block mode and a block index below ceil(k/b)")
        wm, wn = (m + 15) // 16, (n + 15) // 16
        f32 = dict(dtype=torch.float32, device=dev)
        i32 = dict(dtype=torch.int32, device=dev)
        bcap = {"R": torch.empty((m, n), **f32), "U_in": torch.empty((bb, wm), **i32),
                "P": torch.empty((bb, n), **f32), "GinvU": torch.empty((bb, bb), **f32),
                "Vt": torch.empty((bb, n), **f32), "V": torch.empty((bb, wn), **i32),
                "Q": torch.empty((bb, m), **f32), "GinvV": torch.empty((bb, bb), **f32),
                "Ut": torch.empty((bb, m), **f32), "U_out": torch.empty((bb, wm), **i32),
                "rhs": torch.empty((bb,), dtype=torch.float64, device=dev)}
        bc = _BlockCapture()
        bc.block, bc.iteration = int(blk), int(it)
        for name, tensor in bcap.items():
            setattr(bc, name, _ptr(tensor))
        opts.block_capture = ctypes.pointer(bc)
    _check((_entry or _decompose)(_ptr(A), m, n, mu, tau, iters, block, _stream(), _ptr(B2), _ptr(C2),
                                  _ptr(D), _ptr(E), ctypes.byref(opts)))
    res = Decomposition(m, n, k, B2, C2, D, E, tr, st, cap, na2, b)
    res.sweep_trace = swt
    res.block_capture = bcap
    return res


def decompose_noalloc(A, mu, tau, iters=15, block=0, seed=0, **kw):
    """Run externd_decompose_noalloc: decompose() on the resident sequential
    path with the library's static scratch, for callers that cannot
    allocate (the outputs here are still allocated by torch).  Takes the
    keyword arguments of decompose() except workspace."""
    if kw.get("workspace") is not None:
        raise ValueError("decompose_noalloc brings its own scratch")
    return decompose(A, mu, tau, iters, block, seed, _entry=_decompose_noalloc, **kw)


def rank_for_energy(trace, total, step, norm_a2, target, with_energy=False):
    """Smallest prefix rank whose energy reaches target (host-side scan of a
    trace; see externd_rank_for_energy).  -1 if none does.  with_energy:
    return (rank, energy of that prefix) instead, the energy NaN for -1."""
    import numpy as np
    tr = np.ascontiguousarray(np.asarray(trace, dtype=np.float64))
    e = ctypes.c_double(0.0)
    r = int(_rank_for_energy(tr.ctypes.data_as(ctypes.POINTER(ctypes.c_double)), tr.size, int(total),
                             int(step), float(norm_a2), float(target), ctypes.byref(e)))
    if r == -2:
        raise ExterndError(1)
    return (r, e.value) if with_energy else r


def mu_for_energy(A, target, mu_max, tau, iters=15, block=0, seed=0):
    """Smallest mu (a multiple of 1/min(m, n), and of b/min(m, n) in block
    mode) whose decomposition reaches energy >= target, from one run at
    mu_max (§3.3).  Returns (mu, k, energy_at_k) or None if mu_max is short."""
    res = decompose(A, mu_max, tau, iters, block, seed, trace=True)
    torch.cuda.synchronize()
    tr = res.trace.cpu().numpy()
    a2 = float(res.norm_a2.item())
    c, e = rank_for_energy(tr, res.k, res.block, a2, target, with_energy=True)
    if c < 0:
        return None
    m, n = A.shape
    return c / min(m, n), c, e


def energy(A, B2, C2, D):
    """E = 1 - ||A - B diag(D) C||^2 / ||A||^2 from 2-bit factors, fp64 (§2.1)."""
    _need(A, torch.float32, "A")
    m, n = A.shape
    k = D.numel()
    E = torch.empty((1,), dtype=torch.float64, device=A.device)
    _check(_energy(_ptr(A), m, n, _ptr(B2), _ptr(C2), _ptr(D), k, _stream(), _ptr(E)))
    return E


def reconstruct(B2, C2, D, m, n):
    """A_hat = B diag(D) C as an (m, n) float32 tensor (§2.1)."""
    k = D.numel()
    out = torch.empty((m, n), dtype=torch.float32, device=D.device)
    _check(_reconstruct(_ptr(B2), _ptr(C2), _ptr(D), m, n, k, _stream(), _ptr(out)))
    return out


def apply(B2, C2, D, m, n, x):
    """y = B (diag(D) (C x)) from the 2-bit factors (§2.6); x: float32 (n,)."""
    _need(x, torch.float32, "x")
    if x.numel() != n:
        raise ValueError("x must have n entries")
    k = D.numel()
    y = torch.empty((m,), dtype=torch.float32, device=x.device)
    _check(_apply(_ptr(B2), _ptr(C2), _ptr(D), m, n, k, _ptr(x), _stream(), _ptr(y)))
    return y


def transpose_codes(src, rows, cols):
    """Transpose a 2-bit code matrix: src holds `rows` rows of `cols` codes
    (ceil(cols/16) int32 words per row); returns `cols` rows of `rows` codes.
    transpose_codes(B2, k, m) gives B row by row, the form apply_rows reads."""
    _need(src, torch.int32, "src")
    if src.numel() != rows * ((cols + 15) // 16):
        raise ValueError("src must hold rows * ceil(cols/16) words")
    dst = torch.empty((cols, (rows + 15) // 16), dtype=torch.int32, device=src.device)
    _check(_transpose_codes(_ptr(src), rows, cols, _stream(), _ptr(dst)))
    return dst


def apply_rows_workspace_bytes(m, n, k):
    """Device workspace apply_rows needs for this shape (0: invalid)."""
    return int(_apply_rows_ws(m, n, k))


def apply_rows(BT2, C2, D, m, n, x, out=None, workspace=None):
    """y = B (diag(D) (C x)) (§2.6) with B row by row (BT2 = transpose_codes(B2,
    k, m)), on int8 MFMA with the vectors in exact fixed point; x: float32 (n,).
    out: optional float32 (m,) CUDA tensor written and returned; workspace:
    optional contiguous CUDA tensor of at least apply_rows_workspace_bytes(m,
    n, k) bytes (256-byte aligned), so that the call allocates nothing."""
    _need(x, torch.float32, "x")
    if x.numel() != n:
        raise ValueError("x must have n entries")
    k = D.numel()
    if out is None:
        out = torch.empty((m,), dtype=torch.float32, device=x.device)
    else:
        _need(out, torch.float32, "out")
        if out.numel() != m:
            raise ValueError("out must have m entries")
    wsb = 0
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or workspace.device.type != "cuda" \
                or not workspace.is_contiguous():
            raise TypeError("workspace must be a contiguous CUDA tensor")
        wsb = workspace.numel() * workspace.element_size()
    _check(_apply_rows(_ptr(BT2), _ptr(C2), _ptr(D), m, n, k, _ptr(x), _stream(), _ptr(out), _ptr(workspace), wsb))
    return out


def ternarize(x, tau):
    """T_tau of a float32 vector (§2.2) -> (2-bit code words, nnz)."""
    _need(x, torch.float32, "x")
    N = x.numel()
    codes = torch.empty(((N + 15) // 16,), dtype=torch.int32, device=x.device)
    nnz = torch.empty((1,), dtype=torch.int32, device=x.device)
    _check(_ternarize(_ptr(x), N, tau, _stream(), _ptr(codes), _ptr(nnz)))
    return codes, nnz


def project(x):
    """Optimal ternary projection of a float32 vector (§2.2) -> (codes, nnz)."""
    _need(x, torch.float32, "x")
    N = x.numel()
    codes = torch.empty(((N + 15) // 16,), dtype=torch.int32, device=x.device)
    nnz = torch.empty((1,), dtype=torch.int32, device=x.device)
    _check(_project(_ptr(x), N, _stream(), _ptr(codes), _ptr(nnz)))
    return codes, nnz


def gemv_t(R, u_codes):
    """y = R^T u with u as 2-bit codes (§2.3)."""
    _need(R, torch.float32, "R")
    m, n = R.shape
    y = torch.empty((n,), dtype=torch.float32, device=R.device)
    _check(_gemv_t(_ptr(R), m, n, _ptr(u_codes), _stream(), _ptr(y)))
    return y


def gemv_n(R, v_codes):
    """x = R v with v as 2-bit codes (§2.3)."""
    _need(R, torch.float32, "R")
    m, n = R.shape
    x = torch.empty((m,), dtype=torch.float32, device=R.device)
    _check(_gemv_n(_ptr(R), m, n, _ptr(v_codes), _stream(), _ptr(x)))
    return x


def deflate(R, u_codes, v_codes, d):
    """R <- R - d u v^T in place (§2.3 step 3)."""
    _need(R, torch.float32, "R")
    m, n = R.shape
    _check(_deflate(_ptr(R), m, n, _ptr(u_codes), _ptr(v_codes), float(d), _stream()))
    return R


# ---- 4-bit weights with group scales, and the gated feed-forward block ----

_DTYPE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_ACT = {"silu": 0, "gelu": 1, "gelu_tanh": 2}


_current_device = torch.cuda.current_device
# torch's current stream as a plain number, without building a Stream object for every call
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _op_device(*tensors):
    """Index of the device that all tensors are on; it has to be the current one, whose stream the call uses."""
    index = tensors[0].get_device()
    for t in tensors:
        if t.get_device() != index or index < 0:
            if not t.is_cuda or index < 0:
                raise TypeError("tensors must be CUDA (HIP) tensors")
            raise ValueError("tensors are on different devices")
    if index != _current_device():
        raise ValueError("tensors are not on the current device")
    return index


def _act_code(act):
    code = _ACT.get(act)
    if code is None:
        raise ValueError(f"act must be one of {', '.join(_ACT)}, got {act!r}")
    return code


def _dtype_code(dtype, name):
    code = _DTYPE.get(dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {dtype}")
    return code


def _rows_of(x, cols, name):
    """x with `cols` entries in its last dimension as (2-D tensor of unit column stride, row stride)."""
    if x.dim() == 2 and x.is_contiguous() and x.shape[1] == cols:
        return x, cols
    if x.dim() == 0 or x.shape[-1] != cols:
        raise ValueError(f"{name} must have {cols} entries in its last dimension, got shape {tuple(x.shape)}")
    if x.dim() != 2:
        x = x.reshape(-1, cols)
    tokens, ld = x.shape[0], x.stride(0)
    if x.stride(1) != 1 and cols != 1 or ld < cols and tokens > 1:   # transposed, expanded or overlapping rows
        x = x.contiguous()
        ld = cols
    return x, max(ld, cols)


def _scratch(workspace, index):
    """(pointer, bytes) of a workspace on the device of that index."""
    if workspace is None:
        return None, 0
    if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous CUDA tensor")
    if workspace.get_device() != index:
        raise ValueError("workspace is on another device than the operands")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _out_or_new(out, shape, dtype, device, name="out"):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _need(out, dtype, name)
    if tuple(out.shape) != tuple(shape) or out.device != device:
        raise ValueError(f"{name} must have shape {tuple(shape)} on {device}")
    return out


class _NoGradient(torch.autograd.Function):
    @staticmethod
    def forward(ctx, message, out, *inputs):
        ctx.message = message
        return out.detach()

    @staticmethod
    def backward(ctx, grad):
        raise RuntimeError(ctx.message)


def _records(out):
    """Whether autograd records a call whose input requires a gradient; an error where it writes into a
    tensor of the caller's."""
    if not torch.is_grad_enabled():
        return False
    if out is not None:
        raise RuntimeError("out cannot be given where an input requires a gradient (torch.no_grad() turns that off)")
    return True


def _q4_part(t, dtype, count, codes, name):
    if t.dtype is not dtype or not t.is_cuda or not t.is_contiguous():
        _need(t, dtype, name)
    if t.numel() != count:
        raise ValueError(f"{name} must hold {count} elements, got {t.numel()}")
    if t.get_device() != codes.get_device():
        raise ValueError(f"{name} is on another device than codes")


class Q4:
    """A weight matrix in 4 bits with group scales, in the library's layout.

    codes: int32 words, scales and mins (None: symmetric): bfloat16, laid out as
    include/externd.h says (tiles of 16 rows by chunks of 128 columns).
    q4_quantize and q4_pack make them.  Its shape is (rows, cols).  It is read only, and
    the tensors are not to be resized or given other storage while it is in use."""

    __slots__ = ("_codes", "_scales", "_mins", "_rows", "_cols", "_group", "_c", "_index")
    # read only: _c holds the tensors' addresses
    codes, scales, mins, rows, cols, group = (
        property(lambda self, name=name: getattr(self, name)) for name in __slots__[:6])

    def __init__(self, codes, scales, mins, rows, cols, group):
        if group not in (32, 64, 128) or not 0 < rows < 1 << 31 or not 0 < cols < 1 << 31:
            raise ValueError("bad shape or group (32, 64 or 128)")
        blocks = -(-rows // 16) * -(-cols // 128)   # tiles of chunks
        _q4_part(codes, torch.int32, 256 * blocks, codes, "codes")
        _q4_part(scales, torch.bfloat16, 2048 // group * blocks, codes, "scales")
        if mins is not None:
            _q4_part(mins, torch.bfloat16, 2048 // group * blocks, codes, "mins")
        self._codes, self._scales, self._mins = codes, scales, mins
        self._rows, self._cols, self._group = rows, cols, group
        self._index = codes.get_device()
        self._c = _Q4(codes.data_ptr(), scales.data_ptr(), None if mins is None else mins.data_ptr(), rows, cols,
                      group, 0)

    @property
    def shape(self):
        return self.rows, self.cols

    @property
    def symmetric(self):
        return self.mins is None

    def __repr__(self):
        return f"Q4({self.rows}x{self.cols}, group={self.group}, {'symmetric' if self.symmetric else 'with minima'})"


def _q4_new(rows, cols, group, symmetric, device):
    if group not in (32, 64, 128):
        raise ValueError("group must be 32, 64 or 128")
    blocks = -(-rows // 16) * -(-cols // 128)
    table = 2048 // group * blocks
    codes = torch.empty((256 * blocks,), dtype=torch.int32, device=device)
    tables = torch.empty((1 if symmetric else 2, table), dtype=torch.bfloat16, device=device)
    return Q4(codes, tables[0], None if symmetric else tables[1], rows, cols, group)


def q4_quantize(W, group=32, symmetric=True):
    """W (rows, cols; float32, bfloat16 or float16, unit column stride) to 4 bits: per group of
    `group` entries of a row a bf16 scale and, unless symmetric, a bf16 minimum."""
    if not isinstance(W, torch.Tensor) or W.dim() != 2:
        raise ValueError("W must be a 2-D tensor")
    dtype = _dtype_code(W.dtype, "W")
    index = _op_device(W)
    W, ldw = _rows_of(W, W.shape[1], "W")
    rows, cols = W.shape
    q = _q4_new(rows, cols, group, symmetric, W.device)
    _check(_q4_quantize(_ptr(W), rows, cols, ldw, dtype, group, _raw_stream(index), q._c.codes, q._c.scales, q._c.mins))
    return q


def q4_pack(codes, scales, mins=None, group=32):
    """4-bit weights made elsewhere into the library's layout: codes uint8 (rows, cols) with values
    0..15, scales and mins bfloat16 (rows, ceil(cols / group)).  Without mins a code c stands for
    scale * (c - 8), with them for scale * c + min."""
    _need(codes, torch.uint8, "codes")
    if codes.dim() != 2:
        raise ValueError("codes must be 2-D")
    rows, cols = codes.shape
    if group not in (32, 64, 128):
        raise ValueError("group must be 32, 64 or 128")
    for t, name in ((scales, "scales"), (mins, "mins")):
        if t is not None or name == "scales":
            _need(t, torch.bfloat16, name)
            if tuple(t.shape) != (rows, -(-cols // group)):
                raise ValueError(f"{name} must have shape {(rows, -(-cols // group))}")
    index = _op_device(*(t for t in (codes, scales, mins) if t is not None))
    q = _q4_new(rows, cols, group, mins is None, codes.device)
    _check(_q4_pack(_ptr(codes), _ptr(scales), _ptr(mins), rows, cols, group, _raw_stream(index), q._c.codes, q._c.scales,
                    q._c.mins))
    return q


def q4_reconstruct(q, dtype=torch.float32):
    """The values that q stands for, as a (rows, cols) tensor, each rounded once."""
    code = _dtype_code(dtype, "dtype")
    index = _op_device(q.codes)
    out = torch.empty((q.rows, q.cols), dtype=dtype, device=q.codes.device)
    _check(_q4_reconstruct(q._c, code, _raw_stream(index), _ptr(out)))
    return out


def q4_workspace_bytes(cols, tokens, dtype):
    """Device workspace that covers q4_apply and q4_gated on `tokens` rows of `cols` entries (0: invalid)."""
    return int(_q4_ws(cols, tokens, _dtype_code(dtype, "dtype")))


def _q4_scratch(workspace, x, ldx, dtype):
    """As _gated_scratch, for the staged copy of x that the 4-bit products may need."""
    if workspace is None:
        tokens, cols = x.shape
        if tokens <= (5 if dtype == 0 else 0) or \
                tokens <= 16 and dtype != 0 and (cols | ldx) & 7 == 0 and x.data_ptr() & 15 == 0:
            return None, 0, None
        workspace = torch.empty((_q4_ws(cols, tokens, dtype),), dtype=torch.uint8, device=x.device)
    return (*_scratch(workspace, x.get_device()), workspace)


def q4_apply(q, x, out=None, workspace=None):
    """y = x W^T with 4-bit W: x (..., cols) float32, bfloat16 or float16, y (..., rows) of its type.
    Rows of x may be strided.  Where x needs a staged copy (float32 of more than 5 tokens, rows that are not
    16-byte aligned, more than 16 tokens on a large matrix) it is made in workspace (at least q4_workspace_bytes(...) bytes, 256-byte aligned), by
    default one from torch's allocator.  There is no gradient: asking for one raises an error."""
    dtype = _DTYPE.get(x.dtype)
    if dtype is None:
        _dtype_code(x.dtype, "x")
    index = q._index
    if x.get_device() != index or index != _current_device():
        _op_device(x, q._codes)
    record = x.requires_grad and _records(out)
    given = x
    y = x.new_empty((*x.shape[:-1], q._rows)) if out is None else \
        _out_or_new(out, (*x.shape[:-1], q._rows), x.dtype, x.device)
    x, ldx = _rows_of(x, q._cols, "x")
    ws, wsb, keep = _q4_scratch(workspace, x, ldx, dtype)
    status = _q4_apply(q._c, x.data_ptr(), x.shape[0], ldx, dtype, _raw_stream(index), y.data_ptr(), ws, wsb)
    if status:
        _check(status)
    return _NoGradient.apply("q4_apply has no gradient", y, given) if record else y


def q4_gated(qg, qu, x, act="silu", out=None, workspace=None):
    """h = act(x Wg^T) * (x Wu^T) with both matrices in 4 bits (one shape, group and kind), in one
    kernel; everything else as q4_apply.  act: "silu", "gelu" (erf) or "gelu_tanh"."""
    dtype = _DTYPE.get(x.dtype)
    if dtype is None:
        _dtype_code(x.dtype, "x")
    index = qg._index
    if x.get_device() != index or qu._index != index or index != _current_device():
        _op_device(x, qg._codes, qu._codes)
    record = x.requires_grad and _records(out)
    given = x
    h = x.new_empty((*x.shape[:-1], qg._rows)) if out is None else \
        _out_or_new(out, (*x.shape[:-1], qg._rows), x.dtype, x.device)
    x, ldx = _rows_of(x, qg._cols, "x")
    ws, wsb, keep = _q4_scratch(workspace, x, ldx, dtype)
    _check(_q4_gated(qg._c, qu._c, x.data_ptr(), x.shape[0], ldx, dtype, _act_code(act), _raw_stream(index), h.data_ptr(), ws,
                     wsb))
    return _NoGradient.apply("q4_gated has no gradient", h, given) if record else h


def _gated_weights(x, Wg, Wu):
    """Checks both weight matrices against x; returns (Wg, Wu, their common row stride, dtype code)."""
    if x.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"x must be bfloat16 or float16, got {x.dtype}")
    for w, name in ((Wg, "Wg"), (Wu, "Wu")):
        if w.dtype != x.dtype:
            raise TypeError(f"{name} must be {x.dtype} like x, got {w.dtype}")
        if w.dim() != 2 or w.shape != Wg.shape:
            raise ValueError("Wg and Wu must be 2-D of one shape")
    cols = Wg.shape[1]
    Wg, ldg = _rows_of(Wg, cols, "Wg")
    Wu, ldu = _rows_of(Wu, cols, "Wu")
    if ldg != ldu:
        Wg, Wu = Wg.contiguous(), Wu.contiguous()
        ldg = cols
    return Wg, Wu, ldg, _DTYPE[x.dtype]


def gated_forward_workspace_bytes(tokens, cols, rows, aligned=True):
    """Device workspace gated_forward needs (may be 0).  aligned: x, Wg and Wu start on 16 bytes, and
    cols and their row strides are multiples of 8; False covers any alignment.  Fewer tokens may need more."""
    return int(_gated_forward_ws(tokens, cols, rows, aligned))


def gated_backward_workspace_bytes(tokens, cols, rows, aligned=True):
    """Device workspace gated_backward needs (0: invalid); aligned as for gated_forward_workspace_bytes."""
    return int(_gated_backward_ws(tokens, cols, rows, aligned))


def _gated_scratch(workspace, bytes_of, x, ldx, Wg, Wu, ldw):
    """(pointer, bytes, the tensor to keep) of the caller's workspace, or of one from torch's allocator
    (whose blocks, unlike a stream-ordered allocation, cost next to nothing from one call to the next)."""
    if workspace is None:
        aligned = (x.data_ptr() | Wg.data_ptr() | Wu.data_ptr()) & 15 == 0 and (ldx | ldw | Wg.shape[1]) & 7 == 0 \
            and max(ldx, ldw) < 1 << 22
        need = bytes_of(x.shape[0], Wg.shape[1], Wg.shape[0], aligned) if x.shape[0] else 0
        if need == 0:
            return None, 0, None
        workspace = torch.empty((need,), dtype=torch.uint8, device=x.device)
    return (*_scratch(workspace, x.get_device()), workspace)


def gated_forward(x, Wg, Wu, act="silu", save=False, out=None, workspace=None):
    """h = act(x Wg^T) * (x Wu^T), the gated feed-forward block's first half, in one kernel.

    x (..., cols) and Wg, Wu (rows, cols) bfloat16 or float16; h (..., rows) of their type.  With
    save, returns (h, g, u): g and u are the projections (tokens, rows) in float32, which
    gated_backward takes.  Rows of x and of the weights may be strided (both weights alike).  act:
    "silu", "gelu" (erf) or "gelu_tanh".  gated() is the differentiable form: asking for a gradient
    of this one raises an error (with save, its result carries none)."""
    act = _act_code(act)
    record = not save and (x.requires_grad or Wg.requires_grad or Wu.requires_grad) and _records(out)
    given = x, Wg, Wu
    index = _op_device(x, Wg, Wu)
    Wg, Wu, ldw, dtype = _gated_weights(x, Wg, Wu)
    rows, cols = Wg.shape
    h = x.new_empty((*x.shape[:-1], rows)) if out is None else \
        _out_or_new(out, (*x.shape[:-1], rows), x.dtype, x.device)
    x, ldx = _rows_of(x, cols, "x")
    tokens = x.shape[0]
    g = u = None
    if save:
        g, u = torch.empty((2, tokens, rows), dtype=torch.float32, device=x.device)
    ws, wsb, keep = _gated_scratch(workspace, _gated_forward_ws, x, ldx, Wg, Wu, ldw)
    _check(_gated_forward(x.data_ptr(), tokens, cols, ldx, Wg.data_ptr(), Wu.data_ptr(), rows, ldw, dtype, act,
                          _raw_stream(index), h.data_ptr(), None if g is None else g.data_ptr(),
                          None if u is None else u.data_ptr(), ws, wsb))
    if record:
        return _NoGradient.apply("gated_forward has no gradient; gated has", h, *given)
    return (h, g, u) if save else h


def gated_backward(x, Wg, Wu, g, u, dh, act="silu", need_dx=True, need_dw=True, workspace=None):
    """(dx, dWg, dWu) of the gated block from dh (..., rows) and the g, u that gated_forward(...,
    save=True) returned; None for what need_dx / need_dw leave out."""
    act = _act_code(act)
    index = _op_device(x, Wg, Wu, g, u, dh)
    Wg, Wu, ldw, dtype = _gated_weights(x, Wg, Wu)
    rows, cols = Wg.shape
    shape = x.shape
    x, ldx = _rows_of(x, cols, "x")
    tokens = x.shape[0]
    if dh.dtype != x.dtype:
        raise TypeError(f"dh must be {x.dtype} like x, got {dh.dtype}")
    if dh.shape[:-1] != shape[:-1]:
        raise ValueError("dh and x must have the same leading dimensions")
    dh, lddh = _rows_of(dh, rows, "dh")
    for t, name in ((g, "g"), (u, "u")):
        _need(t, torch.float32, name)
        if t.numel() != tokens * rows:
            raise ValueError(f"{name} must have {tokens} x {rows} entries")
    dx = torch.empty(shape, dtype=x.dtype, device=x.device) if need_dx else None
    dwg = torch.empty((rows, cols), dtype=x.dtype, device=x.device) if need_dw else None
    dwu = torch.empty_like(dwg) if need_dw else None
    ws, wsb, keep = _gated_scratch(workspace, _gated_backward_ws, x, ldx, Wg, Wu, ldw)
    _check(_gated_backward(x.data_ptr(), tokens, cols, ldx, Wg.data_ptr(), Wu.data_ptr(), rows, ldw, g.data_ptr(),
                           u.data_ptr(), dh.data_ptr(), lddh, dtype, act, _raw_stream(index), _ptr(dx), _ptr(dwg), _ptr(dwu),
                           ws, wsb))
    return dx, dwg, dwu


class _Gated(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, Wg, Wu, act):
        ctx.act = act
        h, g, u = gated_forward(x, Wg, Wu, act, save=True)
        ctx.save_for_backward(x, Wg, Wu, g, u)
        return h

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dh):
        x, Wg, Wu, g, u = ctx.saved_tensors
        need_dx, need_dg, need_du = ctx.needs_input_grad[:3]
        dx, dwg, dwu = gated_backward(x, Wg, Wu, g, u, dh, ctx.act, need_dx, need_dg or need_du)
        return dx, dwg if need_dg else None, dwu if need_du else None, None


def gated(x, Wg, Wu, act="silu"):
    """gated_forward as a differentiable torch operation (gradients of x, Wg and Wu; g and u are kept
    in float32 only where a gradient is needed: not under torch.no_grad())."""
    if not (torch.is_grad_enabled() and (x.requires_grad or Wg.requires_grad or Wu.requires_grad)):
        return gated_forward(x, Wg, Wu, act)
    return _Gated.apply(x, Wg, Wu, act)
