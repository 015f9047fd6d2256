"""Python binding of libqmm: block-quantized (GGUF Q4_0 / Q8_0, and Q4_K
super-blocks) weight matmul on AMD Instinct MI355X.

Argument marshalling only: every step of the computation runs in the
library's gfx950 kernels; PyTorch supplies device memory and the stream.

Two layers:
* ``qmm_gemv_q4_0``, ``qmm_gemv_q8_0``, ``qmm_gemm_q4_0``, ``qmm_gemm_q8_0``,
  ``qmm_ffn_gate_up_q4_0``, ``qmm_gemv_q4_k``, ``qmm_gemm_q4_k`` -- the C-ABI
  entry points of ``include/qmm.h``
  with the same names and arguments (device addresses as integers, a HIP
  stream handle); they return the status code.
* ``gemv_q4_0``, ``gemv_q8_0``, ``gemm_q4_0``, ``gemm_q8_0``,
  ``ffn_gate_up_q4_0``, ``gemv_q4_k``, ``gemm_q4_k`` -- tensor front ends that check dtypes, shapes and
  devices, allocate ``y`` with torch, launch on the current stream and raise
  ``QmmError`` on a non-OK status.

The paged Q4_0 KV cache has both layers too: ``qmm_kv_plan``,
``qmm_kv_append_q4_0``, ``qmm_kv_read_q4_0``, ``qmm_attend_q4_0`` (and
``qmm_kv_chunk_bytes_q4_0``, ``qmm_attend_q4_0_workspace``), and the front ends
``kv_cache_q4_0``, ``kv_plan``, ``kv_append_q4_0``, ``kv_read_q4_0``,
``attend_q4_0``. One serving step of a layer is

    step = kv_plan(want, lens, table, ring, pool, tokens, page_size)
    kv_append_q4_0(k, v, cache, step.slots)
    out = attend_q4_0(q, cache, table, step.lens, step.cu, max_q=1)     # decoding

There is no fallback: if ``libqmm.so`` is missing, every call raises.
Build it with ``python -m block_quantized_matmul_q4_amd._build``.
"""

from __future__ import annotations

import collections
import ctypes
import functools
import pathlib

HERE = pathlib.Path(__file__).resolve().parent
LIBRARY = HERE / "libqmm.so"

QMM_OK, QMM_EINVAL, QMM_EALIGN, QMM_EUNSUPPORTED, QMM_EHIP = range(5)
GEMV_MAX_M = 16
MAX_K = 65536
# format -> (weights per block, bytes per block)
BLOCKS = {"q4_0": (32, 18), "q8_0": (32, 34), "q4_k": (256, 144)}

# Every symbol include/qmm.h declares.
EXPORTS = ("qmm_gemv_q4_0", "qmm_gemv_q8_0", "qmm_gemm_q4_0", "qmm_gemm_q8_0",
           "qmm_ffn_gate_up_q4_0", "qmm_gemv_q4_k", "qmm_gemm_q4_k", "qmm_status_string",
           "qmm_last_error", "qmm_version", "qmm_kv_chunk_bytes_q4_0", "qmm_kv_plan",
           "qmm_kv_append_q4_0", "qmm_kv_read_q4_0", "qmm_attend_q4_0_workspace",
           "qmm_attend_q4_0")

# What kv_plan writes to a request's status
KV_OK, KV_NO_PAGES, KV_BAD_LENGTH, KV_NO_ROWS = range(4)


class KvCache(ctypes.Structure):
    """``qmm_kv_cache`` of include/qmm.h: where a paged cache lies, and its geometry."""

    _fields_ = [("pages", ctypes.c_void_p), ("num_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int64), ("kv_heads", ctypes.c_int64),
                ("head_dim", ctypes.c_int64)]


class QmmError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{status_string(status)}: {message}")
        self.status = status


_lib = None


def library() -> ctypes.CDLL:
    """The loaded ``libqmm.so`` (raises if it has not been built)."""
    global _lib
    if _lib is None:
        # PyTorch owns the device memory and streams we are handed, so the
        # library must bind to the same HIP runtime instance: load torch's
        # first (the loader then resolves libqmm's libamdhip64.so.7 to it).
        import torch  # noqa: F401
        if not LIBRARY.exists():
            raise QmmError(QMM_EHIP, f"{LIBRARY} is not built; run "
                           "`python -m block_quantized_matmul_q4_amd._build`")
        lib = ctypes.CDLL(str(LIBRARY))
        args = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p]
        for name in ("qmm_gemv_q4_0", "qmm_gemv_q8_0", "qmm_gemm_q4_0", "qmm_gemm_q8_0",
                     "qmm_gemv_q4_k", "qmm_gemm_q4_k"):
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        lib.qmm_ffn_gate_up_q4_0.argtypes = [ctypes.c_void_p] * 4 + [ctypes.c_int64] * 3 + [
            ctypes.c_void_p]
        lib.qmm_ffn_gate_up_q4_0.restype = ctypes.c_int
        p, i64, cache = ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(KvCache)
        for name, args, result in (
                ("qmm_kv_chunk_bytes_q4_0", [i64] * 2, i64),
                ("qmm_kv_plan", [p] * 11 + [i64] * 5 + [p], ctypes.c_int),
                ("qmm_kv_append_q4_0", [p, i64, p, i64, cache, p, i64, p], ctypes.c_int),
                ("qmm_kv_read_q4_0", [cache, p, p, p, i64, p], ctypes.c_int),
                ("qmm_attend_q4_0_workspace", [cache] + [i64] * 6, i64),
                ("qmm_attend_q4_0",
                 [p, i64, cache, p, i64, p, p, p, p, p] + [i64] * 6 +
                 [ctypes.c_float, ctypes.c_int, i64, p], ctypes.c_int)):
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = result
        lib.qmm_status_string.argtypes = [ctypes.c_int]
        lib.qmm_status_string.restype = ctypes.c_char_p
        lib.qmm_last_error.argtypes = []
        lib.qmm_last_error.restype = ctypes.c_char_p
        lib.qmm_version.argtypes = []
        lib.qmm_version.restype = ctypes.c_int
        _lib = lib
    return _lib


# ---------------------------------------------------------------------------
# C-ABI mirror
# ---------------------------------------------------------------------------

def qmm_gemv_q4_0(x: int, w: int, y: int, M: int, N: int, K: int, stream: int = 0) -> int:
    return library().qmm_gemv_q4_0(x, w, y, M, N, K, stream)


def qmm_gemv_q8_0(x: int, w: int, y: int, M: int, N: int, K: int, stream: int = 0) -> int:
    return library().qmm_gemv_q8_0(x, w, y, M, N, K, stream)


def qmm_gemm_q4_0(x: int, w: int, y: int, M: int, N: int, K: int, stream: int = 0) -> int:
    return library().qmm_gemm_q4_0(x, w, y, M, N, K, stream)


def qmm_gemm_q8_0(x: int, w: int, y: int, M: int, N: int, K: int, stream: int = 0) -> int:
    return library().qmm_gemm_q8_0(x, w, y, M, N, K, stream)


def qmm_ffn_gate_up_q4_0(x: int, w_gate: int, w_up: int, h: int, M: int, N: int, K: int,
                         stream: int = 0) -> int:
    return library().qmm_ffn_gate_up_q4_0(x, w_gate, w_up, h, M, N, K, stream)


def qmm_gemv_q4_k(x: int, w: int, y: int, M: int, N: int, K: int, stream: int = 0) -> int:
    return library().qmm_gemv_q4_k(x, w, y, M, N, K, stream)


def qmm_gemm_q4_k(x: int, w: int, y: int, M: int, N: int, K: int, stream: int = 0) -> int:
    return library().qmm_gemm_q4_k(x, w, y, M, N, K, stream)


def qmm_kv_chunk_bytes_q4_0(page_size: int, head_dim: int) -> int:
    return library().qmm_kv_chunk_bytes_q4_0(page_size, head_dim)


def qmm_kv_plan(want: int, lens: int, table: int, ring: int, pool: int, new_lens: int,
                new_pool: int, cu: int, slots: int, positions: int, status: int, B: int, T: int,
                width: int, ring_size: int, page_size: int, stream: int = 0) -> int:
    return library().qmm_kv_plan(want, lens, table, ring, pool, new_lens, new_pool, cu, slots,
                                 positions, status, B, T, width, ring_size, page_size, stream)


def qmm_kv_append_q4_0(k: int, k_stride: int, v: int, v_stride: int, cache: KvCache, slots: int,
                       T: int, stream: int = 0) -> int:
    return library().qmm_kv_append_q4_0(k, k_stride, v, v_stride, cache, slots, T, stream)


def qmm_kv_read_q4_0(cache: KvCache, slots: int, k: int, v: int, T: int, stream: int = 0) -> int:
    return library().qmm_kv_read_q4_0(cache, slots, k, v, T, stream)


def qmm_attend_q4_0_workspace(cache: KvCache, T: int, B: int, q_heads: int, max_q: int,
                              max_len: int, window: int) -> int:
    return library().qmm_attend_q4_0_workspace(cache, T, B, q_heads, max_q, max_len, window)


def qmm_attend_q4_0(q: int, q_stride: int, cache: KvCache, table: int, width: int, lens: int,
                    cu: int, out: int, lse: int, workspace: int, workspace_bytes: int, T: int,
                    B: int, q_heads: int, max_q: int, max_len: int, scale: float, causal: int,
                    window: int, stream: int = 0) -> int:
    return library().qmm_attend_q4_0(q, q_stride, cache, table, width, lens, cu, out, lse,
                                     workspace, workspace_bytes, T, B, q_heads, max_q, max_len,
                                     scale, causal, window, stream)


def qmm_status_string(status: int) -> str:
    return library().qmm_status_string(status).decode()


def qmm_last_error() -> str:
    return library().qmm_last_error().decode()


def qmm_version() -> int:
    return library().qmm_version()


def status_string(status: int) -> str:
    try:
        return qmm_status_string(status)
    except Exception:  # library missing: still name the status
        return {0: "QMM_OK", 1: "QMM_EINVAL", 2: "QMM_EALIGN",
                3: "QMM_EUNSUPPORTED", 4: "QMM_EHIP"}.get(status, str(status))


def check(status: int) -> None:
    if status != QMM_OK:
        raise QmmError(status, qmm_last_error())


# ---------------------------------------------------------------------------
# Tensor front ends
# ---------------------------------------------------------------------------

def _call(fn, fmt, x, w, n, k, out):
    import torch

    if not (isinstance(x, torch.Tensor) and isinstance(w, torch.Tensor)):
        raise TypeError("x and w must be torch tensors")
    if x.device.type != "cuda" or w.device != x.device:
        raise ValueError("x and w must be on the same GPU")
    if x.dtype != torch.float32 or x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous float32 [M, K] tensor")
    if w.dtype != torch.uint8 or not w.is_contiguous():
        raise ValueError("w must be a contiguous uint8 tensor of packed blocks")
    m = x.shape[0]
    if x.shape[1] != k:
        raise ValueError(f"x has {x.shape[1]} columns, K={k}")
    per, nbytes = BLOCKS[fmt]
    if k % per or w.numel() != n * (k // per) * nbytes:
        raise ValueError(f"w has {w.numel()} bytes; {fmt} N={n} K={k} needs "
                         f"{n * (k // per) * nbytes} (K a multiple of {per})")
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=x.device)
    elif (out.dtype != torch.float32 or out.shape != (m, n) or not out.is_contiguous()
          or out.device != x.device):
        raise ValueError("out must be a contiguous float32 [M, N] tensor on x's device")
    with torch.cuda.device(x.device):
        stream = torch.cuda.current_stream(x.device).cuda_stream
        check(fn(x.data_ptr(), w.data_ptr(), out.data_ptr(), m, n, k, stream))
    return out


def gemv_q4_0(x, w, n: int, k: int, out=None):
    """y[M, N] = x[M, K] @ W^T for Q4_0 W (1 <= M <= 16)."""
    return _call(qmm_gemv_q4_0, "q4_0", x, w, n, k, out)


def gemv_q8_0(x, w, n: int, k: int, out=None):
    """y[M, N] = x[M, K] @ W^T for Q8_0 W (1 <= M <= 16)."""
    return _call(qmm_gemv_q8_0, "q8_0", x, w, n, k, out)


def gemm_q4_0(x, w, n: int, k: int, out=None):
    """y[M, N] = bf16(x) @ bf16(W)^T with f32 accumulation, Q4_0 W, any M
    (M <= 4, and M <= 16 with N <= 4096: the GEMV result, bit for bit)."""
    return _call(qmm_gemm_q4_0, "q4_0", x, w, n, k, out)


def gemm_q8_0(x, w, n: int, k: int, out=None):
    """y[M, N] = bf16(x) @ bf16(W)^T with f32 accumulation, Q8_0 W, any M
    (M <= 4, and M <= 16 with N <= 4096: the GEMV result, bit for bit)."""
    return _call(qmm_gemm_q8_0, "q8_0", x, w, n, k, out)


def gemv_q4_k(x, w, n: int, k: int, out=None):
    """y[M, N] = x[M, K] @ W^T for Q4_K W (super-blocks of 256; 1 <= M <= 16)."""
    return _call(qmm_gemv_q4_k, "q4_k", x, w, n, k, out)


def gemm_q4_k(x, w, n: int, k: int, out=None):
    """y[M, N] = bf16(x) @ bf16(W)^T with f32 accumulation, Q4_K W, any M
    (M <= 4, and M <= 16 with N <= 4096: the GEMV result, bit for bit)."""
    return _call(qmm_gemm_q4_k, "q4_k", x, w, n, k, out)


def ffn_gate_up_q4_0(x, w_gate, w_up, n: int, k: int, out=None):
    """h[M, N] = gelu_tanh(x @ W_gate^T) * (x @ W_up^T) for Q4_0 W_gate, W_up (1 <= M <= 16)."""
    import torch

    if not isinstance(w_up, torch.Tensor):
        raise TypeError("w_up must be a torch tensor")
    if w_up.device != w_gate.device or w_up.dtype != torch.uint8 or not w_up.is_contiguous():
        raise ValueError("w_up must be a contiguous uint8 tensor on w_gate's device")
    if w_up.numel() != w_gate.numel():
        raise ValueError("w_up and w_gate must have the same size")

    def fn(xp, wp, yp, m, n_, k_, stream):
        return qmm_ffn_gate_up_q4_0(xp, wp, w_up.data_ptr(), yp, m, n_, k_, stream)

    return _call(fn, "q4_0", x, w_gate, n, k, out)


# ---------------------------------------------------------------------------
# Paged KV cache
# ---------------------------------------------------------------------------

def _refuse(name, t, dtype, shape, index):
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on the same GPU as the others")
    sizes = ", ".join("*" if n < 0 else str(n) for n in shape)
    raise ValueError(f"{name} must be a contiguous {str(dtype).split('.')[-1]} tensor [{sizes}], "
                     f"got {str(t.dtype).split('.')[-1]} {list(t.shape)}")


# A launch takes a few microseconds on the GPU, so the checks are kept short:
# one expression each while all is well, the reasons only when it is not.

def _whole(name, t, dtype, shape, index):
    """Address of a contiguous tensor of that type and shape on GPU `index`."""
    try:
        if (t.dtype is dtype and t.get_device() == index and t.shape == shape
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(name, t, dtype, shape, index)


def _sizes(name, t, dtype, dims, index=None):
    """Sizes of a contiguous tensor of that type and number of dimensions on a GPU."""
    try:
        at = t.get_device()
        if (t.dtype is dtype and at >= 0 and (index is None or at == index) and t.dim() == dims
                and t.is_contiguous()):
            return t.shape
    except AttributeError:
        at = 0
    _refuse(name, t, dtype, (-1,) * dims, at if index is None else index)


def _rows(name, t):
    """Stride of the rows of a float32 [T, heads, D] tensor whose rows are contiguous."""
    import torch

    if t.dtype is not torch.float32 or t.dim() != 3:
        raise ValueError(f"{name} must be a float32 [T, heads, head_dim] tensor")
    rows, heads, dim = t.shape
    if rows < 2 and t.is_contiguous():
        return heads * dim
    stride, across, along = t.stride()
    if rows and ((dim > 1 and along != 1) or (heads > 1 and across != dim)):
        raise ValueError(f"{name}: the heads of a row must lie side by side")
    return stride if rows > 1 else heads * dim


def _row_sizes(name, t, index=None):
    """Sizes and row stride of a tensor as _rows takes it, on a GPU."""
    import torch

    if not isinstance(t, torch.Tensor) or t.get_device() < 0 or index not in (None, t.get_device()):
        _refuse(name, t, torch.float32, (-1, -1, -1), index)
    if t.dtype is torch.float32 and t.dim() == 3 and t.is_contiguous():
        rows, heads, dim = t.shape
        return rows, heads, dim, heads * dim
    return (*t.shape, _rows(name, t)) if t.dim() == 3 else _rows(name, t)


_chunk_bytes = functools.lru_cache(maxsize=None)(
    lambda page_size, head_dim: qmm_kv_chunk_bytes_q4_0(page_size, head_dim))


def _geometry(cache, sizes, head_dim):
    pages, heads, chunk = sizes
    page_size = chunk * 8 // (9 * head_dim) if head_dim > 0 else 0
    if chunk == 0 or _chunk_bytes(page_size, head_dim) != chunk:
        raise ValueError(f"cache has chunks of {chunk} bytes: no supported page size gives that "
                         f"for head_dim {head_dim}")
    return KvCache(cache.data_ptr(), pages, page_size, heads, head_dim)


def _launch(index, fn, *args):
    """Call a C-ABI entry point on GPU `index` and its current stream."""
    import torch

    stream = torch._C._cuda_getCurrentRawStream(index)
    if torch._C._cuda_getDevice() == index:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            status = fn(*args, stream)
    if status:
        check(status)


def kv_cache_q4_0(num_pages: int, page_size: int, kv_heads: int, head_dim: int, device="cuda"):
    """A cache of zeros for one layer: uint8 [num_pages, kv_heads, chunk bytes]."""
    import torch

    chunk = _chunk_bytes(page_size, head_dim)
    if not chunk:
        raise ValueError(f"page_size {page_size} or head_dim {head_dim} is not supported")
    return torch.zeros((num_pages, kv_heads, chunk), dtype=torch.uint8, device=device)


KvPlan = collections.namedtuple("KvPlan", "lens pool cu slots positions status")


def kv_plan(want, lens, table, ring, pool, tokens: int, page_size: int, out=None):
    """Pages, slots and positions of one serving step (``qmm_kv_plan``).

    want, lens int32 [B]; table int32 [B, width] and ring int32 [ring size] are
    updated in place; pool int64 [2] holds (head, count) of the ring. Returns a
    KvPlan of new tensors, or fills and returns ``out``, whose lens and pool
    may be the inputs themselves and whose positions may be None. A request
    that is refused (status KV_NO_PAGES or KV_NO_ROWS) keeps its rows in cu, with
    slots of -1: what attention then writes to them means nothing.
    """
    import torch

    int32, int64 = torch.int32, torch.int64
    (batch,) = _sizes("want", want, int32, 1)
    index = want.get_device()
    before = _whole("lens", lens, int32, (batch,), index)
    rows, width = _sizes("table", table, int32, 2, index)
    if rows != batch:
        _refuse("table", table, int32, (batch, -1), index)
    (ring_size,) = _sizes("ring", ring, int32, 1, index)
    state = _whole("pool", pool, int64, (2,), index)
    if tokens < 0:
        raise ValueError(f"tokens must not be negative ({tokens})")
    if out is None:
        # the 64-bit slots and pool first, then the 32-bit arrays
        longs = want.new_empty(2 + tokens, dtype=int64)
        ints = want.new_empty(3 * batch + 1 + tokens)
        after, cu, status, positions = ints.unsafe_split_with_sizes((batch, batch + 1, batch, tokens))
        to, slots = longs.unsafe_split_with_sizes((2, tokens))
        out = KvPlan(after, to, cu, slots, positions, status)
        at, long_at = ints.data_ptr(), longs.data_ptr()
        ends = (at, long_at, at + 4 * batch, long_at + 16, at + 4 * (3 * batch + 1),
                at + 4 * (2 * batch + 1))
    else:
        ends = (_whole("out.lens", out.lens, int32, (batch,), index),
                _whole("out.pool", out.pool, int64, (2,), index),
                _whole("out.cu", out.cu, int32, (batch + 1,), index),
                _whole("out.slots", out.slots, int64, (tokens,), index),
                0 if out.positions is None else
                _whole("out.positions", out.positions, int32, (tokens,), index),
                _whole("out.status", out.status, int32, (batch,), index))
    _launch(index, library().qmm_kv_plan, want.data_ptr(), before, table.data_ptr(),
            ring.data_ptr(), state, *ends, batch, tokens, width, ring_size, page_size)
    return out


def kv_append_q4_0(k, v, cache, slots):
    """Quantize rows k, v float32 [T, kv_heads, head_dim] into the cache at slots int64 [T].

    Rows may be strided (k and v as column ranges of one matrix); a slot of -1
    leaves its row out.
    """
    import torch

    tokens, heads, dim, k_stride = _row_sizes("k", k)
    index = k.get_device()
    *sizes, v_stride = _row_sizes("v", v, index)
    if sizes != [tokens, heads, dim]:
        raise ValueError(f"k {list(k.shape)} and v {list(v.shape)} differ")
    geometry = _geometry(cache, _sizes("cache", cache, torch.uint8, 3, index), dim)
    if geometry.kv_heads != heads:
        raise ValueError(f"cache has {geometry.kv_heads} heads, k has {heads}")
    _launch(index, library().qmm_kv_append_q4_0, k.data_ptr(), k_stride, v.data_ptr(), v_stride,
            geometry, _whole("slots", slots, torch.int64, (tokens,), index), tokens)


def kv_read_q4_0(cache, slots, head_dim: int, out=None):
    """The cached rows at slots int64 [T]: k, v float32 [T, kv_heads, head_dim]."""
    import torch

    sizes = _sizes("cache", cache, torch.uint8, 3)
    index = cache.get_device()
    geometry = _geometry(cache, sizes, head_dim)
    (tokens,) = _sizes("slots", slots, torch.int64, 1, index)
    shape = (tokens, sizes[1], head_dim)
    if out is None:
        k = cache.new_empty(shape, dtype=torch.float32)
        v = torch.empty_like(k)
        ends = k.data_ptr(), v.data_ptr()
    else:
        k, v = out
        ends = (_whole("k", k, torch.float32, shape, index),
                _whole("v", v, torch.float32, shape, index))
    _launch(index, library().qmm_kv_read_q4_0, geometry, slots.data_ptr(), *ends, tokens)
    return k, v


@functools.lru_cache(maxsize=1024)
def _attend_workspace(pages, page_size, kv_heads, dim, tokens, batch, heads, max_q, max_len, window):
    """Bytes of workspace that an attention call of these sizes needs (minus the status of one that
    is refused)."""
    return qmm_attend_q4_0_workspace(KvCache(None, pages, page_size, kv_heads, dim), tokens, batch,
                                     heads, max_q, max_len, window)


def attend_q4_0(q, cache, table, lens, cu, *, scale=None, causal: bool = True, window: int = 0,
                max_q=None, max_len=None, return_lse: bool = False, out=None, lse=None,
                workspace=None):
    """Attention of q float32 [T, q_heads, head_dim] over the cache (``qmm_attend_q4_0``).

    Rows cu[b] .. cu[b + 1] - 1 are the last tokens of request b, which has
    lens[b] tokens in the pages table[b]. scale defaults to head_dim ** -0.5;
    max_q and max_len are the largest number of rows and of tokens expected of
    a request (all rows and the table's width if not given, which is right but
    launched as one long prompt: decoding callers should say max_q=1). Rows
    before cu[0] and from cu[-1] on are left as they are. workspace: a uint8 tensor to use instead of a new one.
    Returns out float32 [T, q_heads, head_dim], with return_lse also lse
    float32 [T, q_heads].
    """
    import torch

    int32, float32 = torch.int32, torch.float32
    tokens, heads, dim, q_stride = _row_sizes("q", q)
    index = q.get_device()
    sizes = _sizes("cache", cache, torch.uint8, 3, index)
    geometry = _geometry(cache, sizes, dim)
    pages, kv_heads, _ = sizes
    page_size = geometry.page_size
    batch, width = _sizes("table", table, int32, 2, index)
    if heads == 0 or kv_heads == 0 or heads % kv_heads:
        raise ValueError(f"q has {heads} heads, not a multiple of the cache's {kv_heads}")
    if out is None:
        out = q.new_empty((tokens, heads, dim))
        to = out.data_ptr()
    else:
        to = _whole("out", out, float32, (tokens, heads, dim), index)
    lse_to = 0
    if lse is not None:
        lse_to = _whole("lse", lse, float32, (tokens, heads), index)
    elif return_lse:
        lse = q.new_empty((tokens, heads))
        lse_to = lse.data_ptr()
    if max_q is None:
        max_q = max(tokens, 1)
    if max_len is None:
        max_len = width * page_size
    need = _attend_workspace(pages, page_size, kv_heads, dim, tokens, batch, heads, max_q, max_len,
                             window)
    if need < 0:                        # refused: once more, for this thread's error string
        check(-qmm_attend_q4_0_workspace(geometry, tokens, batch, heads, max_q, max_len, window))
    if workspace is not None:
        (need,) = _sizes("workspace", workspace, torch.uint8, 1, index)
    elif need:
        workspace = cache.new_empty(need)
    _launch(index, library().qmm_attend_q4_0, q.data_ptr(), q_stride, geometry, table.data_ptr(),
            width, _whole("lens", lens, int32, (batch,), index),
            _whole("cu", cu, int32, (batch + 1,), index), to, lse_to,
            0 if workspace is None else workspace.data_ptr(), need, tokens, batch, heads, max_q,
            max_len, dim ** -0.5 if scale is None else scale, 1 if causal else 0, window)
    return (out, lse) if return_lse else out
