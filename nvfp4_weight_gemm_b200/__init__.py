"""NVFP4 verify GEMM for B200: Y[M,N] = X[M,K] . dequant(W)[N,K]^T, M <= 128.

Thin Python layer over libtl_nvfp4.so (the C ABI in include/tl_nvfp4.h). Torch tensors
are used for device memory and streams only; every step of the computation runs in the
library's CUDA kernels. There is no CPU path.
"""

from __future__ import annotations

import ctypes
import functools

from . import _lib
from ._lib import Matrix, TlError, check

__all__ = ["verify_gemm", "verify_gemm_simt", "set_gemm_path", "get_gemm_path", "gemm_path", "PATH_BLOCK_SCALED",
           "PATH_BF16_EXACT", "PATH_EXACT", "verify_stack", "verify_stack_host", "Plan", "dequant",
           "quantize", "check_device_error", "noalloc_check_error", "fp8_head", "gdn_commit", "KvCache", "kv_slots", "kv_commit",
           "kv_attention", "kv_attention_workspace", "init", "num_sms", "Matrix", "TlError"]


def _stream(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t) -> ctypes.c_void_p:
    return ctypes.c_void_p(t.data_ptr())


def init(device: int = 0) -> None:
    check(_lib.lib().tl_init(device))


def num_sms(device: int = 0) -> int:
    return _lib.lib().tl_num_sms(device)


PATH_BLOCK_SCALED = _lib.TL_PATH_BLOCK_SCALED
PATH_BF16_EXACT = _lib.TL_PATH_BF16_EXACT
PATH_EXACT = _lib.TL_PATH_EXACT


def set_gemm_path(path: int) -> None:
    """Select the tensor-core path of verify_gemm, verify_stack(_host) and new plans:
    PATH_EXACT (default; exact f16 operands: hardware E2M1 decode, X prepared per row),
    PATH_BF16_EXACT (exact bf16 operands, integer decode; slower) or PATH_BLOCK_SCALED
    (approximate: X split into FP4 pieces for the block-scaled MMA)."""
    check(_lib.lib().tl_set_gemm_path(path))


def get_gemm_path() -> int:
    return _lib.lib().tl_get_gemm_path()


class gemm_path:
    """Context manager: `with gemm_path(PATH_BF16_EXACT): ...` restores the previous path on exit."""

    def __init__(self, path: int):
        self.path = path
        self.prev = None

    def __enter__(self):
        self.prev = get_gemm_path()
        set_gemm_path(self.path)
        return self

    def __exit__(self, *exc):
        set_gemm_path(self.prev)
        return False


def _gemm(name, x, codes, scales, global_scale, y=None, stream=None):
    import torch
    M, K = x.shape
    N = codes.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    check(getattr(_lib.lib(), name)(_ptr(x), M, _ptr(codes), _ptr(scales), ctypes.c_float(global_scale),
                                    _ptr(y), N, K, _stream(stream)))
    return y


def verify_gemm(x, codes, scales, global_scale, y=None, stream=None):
    """Tensor-core path. x: bf16 [M, K]; codes: uint8 [N, K/2]; scales: uint8 [N, K/16]."""
    return _gemm("tl_nvfp4_verify_gemm", x, codes, scales, global_scale, y, stream)


def verify_gemm_simt(x, codes, scales, global_scale, y=None, stream=None):
    """CUDA-core path (cross-check)."""
    return _gemm("tl_nvfp4_verify_gemm_simt", x, codes, scales, global_scale, y, stream)


def make_matrices(entries):
    """entries: iterable of (codes, scales, global_scale, x, y) tensors -> ctypes array of Matrix."""
    entries = list(entries)
    arr = (Matrix * len(entries))()
    for i, (c, s, g, x, y) in enumerate(entries):
        arr[i] = Matrix(c.data_ptr(), s.data_ptr(), x.data_ptr() if x is not None else None,
                        y.data_ptr() if y is not None else None, float(g), c.shape[0], c.shape[1] * 2)
    return arr


def verify_stack(mats, M: int, stream=None):
    """mats: ctypes array from make_matrices (x and y set)."""
    check(_lib.lib().tl_nvfp4_verify_stack(mats, len(mats), M, _stream(stream)))


def verify_stack_host(mats, M: int, x_host, x_dev, y_host, y_dev, stream=None):
    """End-to-end stack call: X from host memory in, Y to host memory out (contiguous buffers)."""
    check(_lib.lib().tl_nvfp4_verify_stack_host(mats, len(mats), M, _ptr(x_host), _ptr(x_dev),
                                                _ptr(y_host), _ptr(y_dev), _stream(stream)))


class Plan:
    """A stack whose descriptors are built once (tl_nvfp4_plan_create); run() only launches.

    Keeps the ctypes matrix table and the tensors it points to alive while the plan lives."""

    def __init__(self, entries, M: int):
        self._entries = list(entries)
        self._mats = make_matrices(self._entries)
        self.M = M
        h = ctypes.c_void_p()
        check(_lib.lib().tl_nvfp4_plan_create(self._mats, len(self._mats), M, ctypes.byref(h)))
        self._h = h

    def run(self, stream=None):
        check(_lib.lib().tl_nvfp4_plan_run(self._h, _stream(stream)))

    def run_host(self, x_host, y_host, stream=None):
        check(_lib.lib().tl_nvfp4_plan_run_host(self._h, _ptr(x_host), _ptr(y_host), _stream(stream)))

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            _lib.lib().tl_nvfp4_plan_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def dequant(codes, scales, global_scale, out=None, stream=None):
    import torch
    N, K = codes.shape[0], codes.shape[1] * 2
    if out is None:
        out = torch.empty((N, K), dtype=torch.float32, device=codes.device)
    check(_lib.lib().tl_nvfp4_dequant(_ptr(codes), _ptr(scales), ctypes.c_float(global_scale), _ptr(out), N, K,
                                      _stream(stream)))
    return out


def quantize(w, stream=None):
    """fp32 [N, K] device tensor -> (codes uint8 [N, K/2], scales uint8 [N, K/16], g). Synchronises."""
    import torch
    N, K = w.shape
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
    scales = torch.empty((N, K // 16), dtype=torch.uint8, device=w.device)
    g = ctypes.c_float(0.0)
    check(_lib.lib().tl_nvfp4_quantize(_ptr(w), N, K, _ptr(codes), _ptr(scales), ctypes.byref(g), _stream(stream)))
    return codes, scales, g.value


def check_device_error(stream=None) -> None:
    check(_lib.lib().tl_check_device_error(_stream(stream)))


def noalloc_check_error(stream=None) -> None:
    """Status word of the no-allocation entry point's static scratch (allocation-free)."""
    check(_lib.lib().tl_noalloc_check_error(_stream(stream)))


def fp8_head(x, w_fp8, scale, logits=None, stream=None):
    """FP8 output head: x bf16 [M, K]; w_fp8 uint8 [N, K] (E4M3 bytes); scale a float (per tensor)
    or a float32 device tensor [N] (per row). Returns (logits float32 [M, N], top2 int32/float32
    tensor [M, 4] viewed as (token, top1, top2, gap_ulp): the token as int32 bits in column 0)."""
    import torch
    M, K = x.shape
    N = w_fp8.shape[0]
    if logits is None:
        logits = torch.empty((M, N), dtype=torch.float32, device=x.device)
    top2 = torch.empty((M, 4), dtype=torch.int32, device=x.device)
    if isinstance(scale, (float, int)):
        ts, rs = float(scale), None
    else:
        ts, rs = 0.0, ctypes.c_void_p(scale.data_ptr())
    check(_lib.lib().tl_fp8_head(_ptr(x), M, _ptr(w_fp8), N, K, ctypes.c_float(ts), rs, _ptr(logits), _ptr(top2),
                                 _stream(stream)))
    return logits, top2


def head_top2_fields(top2):
    """(token int64[M], top1, top2, gap float64[M]) from fp8_head's top2 tensor (on the host)."""
    import numpy as np
    t = top2.cpu().numpy()
    return (t[:, 0].astype(np.int64), t[:, 1].view(np.float32).astype(np.float64),
            t[:, 2].view(np.float32).astype(np.float64), t[:, 3].view(np.float32).astype(np.float64))


def gdn_commit(state, k, v, alpha, beta, path, stream=None):
    """Closed-form commit of an accepted draft path through Gated DeltaNet states, in place.

    state float32 [H, d_v, d_k] (device); k float32 [n_nodes, H, d_k]; v float32 [n_nodes, H, d_v];
    alpha, beta float32 [n_nodes, H]; path: the accepted node indices in order (a host sequence
    of at most 32 ints). Returns `state`."""
    H, d_v, d_k = state.shape
    n_nodes = k.shape[0]
    p = [int(t) for t in path]
    arr = (ctypes.c_int * max(1, len(p)))(*p)
    check(_lib.lib().tl_gdn_commit(_ptr(state), H, d_k, d_v, _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), n_nodes, arr,
                                   len(p), _stream(stream)))
    return state


# ---------------------------------------------------------------- 8-bit paged KV cache
#
# What the library cannot see behind a pointer (types, shapes, devices) is checked here, with few Python
# operations: these calls come every decoding round, and a call of a few tokens is bound by the host. So
# the tensors are looked at together, and one by one only to say which is wrong.

def _refuse(what: str):
    raise ValueError(what)


def _ints(name, t, shape, index):
    """Pointer of a contiguous int32 tensor of `shape` on CUDA device `index`."""
    import torch
    if t.dtype is not torch.int32 or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        _refuse(f"{name}: need a contiguous int32 tensor of shape {tuple(shape)} on cuda:{index}, "
                f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _rows(name, t, heads, dim, index):
    """(rows, distance between rows) of bf16 rows [n, heads, dim] whose heads lie side by side."""
    import torch
    n, h, d = t.shape if t.dim() == 3 else (0, -1, -1)
    if h != heads or d != dim or t.dtype is not torch.bfloat16 or t.get_device() != index:
        _refuse(f"{name}: need bf16 [rows, {heads}, {dim}] on cuda:{index}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    a, b, c = t.stride()
    if c != 1 or (b != dim and heads > 1):
        _refuse(f"{name}: the heads of a row must lie side by side")
    return n, (a if n > 1 else heads * dim)


def _stream_of(index, stream):
    import torch
    return torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream


def _empty_on(stream, like, shape):
    """An uninitialised tensor of like's type and device that belongs to `stream`: a block of the current stream's pool may
    still be in use by what is queued there, for which `stream` does not wait."""
    import torch
    with torch.cuda.stream(stream):
        return like.new_empty(shape)


def _call_on(index, fn, args):
    """fn(*args) with CUDA device `index` current."""
    import torch
    if torch._C._cuda_getDevice() == index:
        status = fn(*args)
    else:
        with torch.cuda.device(index):
            status = fn(*args)
    if status:
        check(status)


def _same_rows(a, b):
    """Whether b has a's type, device, shape and strides."""
    return a.dtype is b.dtype and a.shape == b.shape and a.stride() == b.stride() and a.get_device() == b.get_device()


class KvCache:
    """One layer's 8-bit paged KV cache: `pages` uint8 [n_pages, kv_heads, 2, page_tokens * head_dim] (E4M3 bytes; K as
    [dim/16, tokens, 16], V as [tokens/16, dim, 16]) and `scales` float32 [n_pages, kv_heads, 2] (powers of two).
    Holds the two tensors; kv_commit() fills them, kv_attention() reads them."""

    __slots__ = ("pages", "scales", "page_tokens", "n_pages", "kv_heads", "head_dim", "index", "_c")

    def __init__(self, pages, scales, page_tokens: int):
        import torch
        shape = pages.shape
        if pages.dtype is not torch.uint8 or len(shape) != 4 or shape[2] != 2 or not pages.is_contiguous():
            _refuse("pages: need a contiguous uint8 tensor [n_pages, kv_heads, 2, page_tokens * head_dim]")
        n, heads, _, side = shape
        if page_tokens <= 0 or side % page_tokens:
            _refuse("pages: page_tokens does not divide a page's side")
        if scales.dtype is not torch.float32 or scales.shape != shape[:3] or not scales.is_contiguous() or scales.get_device() != pages.get_device():
            _refuse("scales: need a contiguous float32 tensor [n_pages, kv_heads, 2] beside pages")
        self.pages, self.scales, self.page_tokens = pages, scales, page_tokens
        self.n_pages, self.kv_heads, self.head_dim, self.index = n, heads, side // page_tokens, pages.get_device()
        self._c = _lib.KvCacheC(pages.data_ptr(), scales.data_ptr(), n, page_tokens, heads, self.head_dim)

    @classmethod
    def empty(cls, n_pages: int, kv_heads: int, head_dim: int, page_tokens: int = 64, device="cuda"):
        """A pool of uninitialised pages (no page is read before a commit began it)."""
        import torch
        return cls(torch.empty((n_pages, kv_heads, 2, page_tokens * head_dim), dtype=torch.uint8, device=device),
                   torch.empty((n_pages, kv_heads, 2), dtype=torch.float32, device=device), page_tokens)

    def _on_gpu(self):
        return self.index if self.index >= 0 else _refuse("the cache must be on a CUDA device")


def kv_slots(lens, want, table, free_pages, n_free, page_tokens, slots, starts, info, stream=None):
    """Block tables and slot maps from lengths, on the GPU (tl_kv_slots). Requests go from `lens` to `want` tokens: those
    that grow take pages off the stack `free_pages` of height `n_free`, those that shrink (0: ended) return theirs.

    All int32 tensors on one device: lens, want [B]; table [B, width]; free_pages [n_pages]; n_free [1]; outputs
    slots [max_slots] (a slot for every token that requests grow by, then -1), starts [B + 1], info [4]
    (code, pages missing, slots missing, requests refused). lens, table, free_pages and n_free are updated in place.
    Returns (slots, starts, info)."""
    import torch
    index, i32 = lens.get_device(), torch.int32
    if index < 0 or lens.dim() != 1:
        _refuse("lens: need an int32 tensor [B] on a CUDA device")
    B, width, n_pages, room = lens.numel(), table.shape[-1], free_pages.numel(), slots.numel()
    if not (lens.dtype is i32 and want.dtype is i32 and table.dtype is i32 and free_pages.dtype is i32 and n_free.dtype is i32
            and slots.dtype is i32 and starts.dtype is i32 and info.dtype is i32
            and want.get_device() == index and table.get_device() == index and free_pages.get_device() == index
            and n_free.get_device() == index and slots.get_device() == index and starts.get_device() == index
            and info.get_device() == index
            and want.shape == lens.shape and table.shape == (B, width) and free_pages.dim() == 1 and n_free.shape == (1,)
            and slots.dim() == 1 and starts.shape == (B + 1,) and info.shape == (4,)
            and lens.is_contiguous() and want.is_contiguous() and table.is_contiguous() and free_pages.is_contiguous()
            and n_free.is_contiguous() and slots.is_contiguous() and starts.is_contiguous() and info.is_contiguous()):
        for name, t, shape in (("lens", lens, (B,)), ("want", want, (B,)), ("table", table, (B, width)),
                               ("free_pages", free_pages, (n_pages,)), ("n_free", n_free, (1,)), ("slots", slots, (room,)),
                               ("starts", starts, (B + 1,)), ("info", info, (4,))):
            _ints(name, t, shape, index)
    _call_on(index, _lib.lib().tl_kv_slots,
             (lens.data_ptr(), want.data_ptr(), B, page_tokens, table.data_ptr(), width, free_pages.data_ptr(), n_pages,
              n_free.data_ptr(), slots.data_ptr(), room, starts.data_ptr(), info.data_ptr(), _stream_of(index, stream)))
    return slots, starts, info


def kv_commit(cache, k, v, slots, src=None, stream=None):
    """Commit accepted tokens into the cache (tl_kv_commit): token i, row src[i] (or i) of k and v, goes to slots[i].

    k, v bf16 [rows, kv_heads, head_dim] (rows may be slices of the QKV projection's output); slots int32 [n] as
    kv_slots() writes them (negative: nowhere); src int32 [n] or None. The tokens of one page must stand next to one another
    in `slots`, in ascending places, with no negative slot or other page between them (else the page's contents are
    undefined): rows that were not accepted are left out by `src`, not marked by -1. Returns `cache`."""
    index = cache._on_gpu()
    rows = _rows("k", k, cache.kv_heads, cache.head_dim, index)
    if not _same_rows(k, v) and _rows("v", v, cache.kv_heads, cache.head_dim, index) != rows:
        _refuse("k and v must have the same rows and row stride")
    n = slots.numel()
    _call_on(index, _lib.lib().tl_kv_commit,
             (cache._c, k.data_ptr(), v.data_ptr(), rows[1], rows[0], None if src is None else _ints("src", src, (n,), index),
              _ints("slots", slots, (n,), index), n, _stream_of(index, stream)))
    return cache


def kv_attention_workspace(cache, n_q_heads: int, batch: int, max_rows: int) -> int:
    """Bytes of workspace kv_attention() needs for these sizes."""
    return _kv_workspace(cache.page_tokens, cache.kv_heads, cache.head_dim, n_q_heads, batch, max_rows)


@functools.lru_cache(maxsize=1024)
def _kv_workspace(page_tokens, kv_heads, head_dim, n_q_heads, batch, max_rows):
    # a function of the sizes alone
    c, n = _lib.KvCacheC(None, None, 1, page_tokens, kv_heads, head_dim), ctypes.c_size_t()
    check(_lib.lib().tl_kv_attention_workspace(c, n_q_heads, batch, max_rows, ctypes.byref(n)))
    return n.value


def kv_attention(q, cache, table, lens, k_new=None, v_new=None, mask=None, row_start=None, max_rows=None, scale=None,
                 out=None, workspace=None, stream=None):
    """Attention of one token or of a draft tree's rows over the cache (tl_kv_attention).

    q bf16 [R, q_heads, head_dim]; table int32 [B, width], lens int32 [B]: each request's pages and cached tokens;
    k_new, v_new bf16 [R, kv_heads, head_dim]: the rows' own keys and values, not in the cache yet (None: rows see
    cached tokens only). mask int32 [R]: bit j, the row sees node j of its request (None: the nodes up to itself).
    row_start int32 [B + 1]: request b has rows row_start[b]..row_start[b+1]-1, at most max_rows (<= 32) of them
    (None: R / B rows each). scale defaults to head_dim ** -0.5. out bf16 [R, q_heads, head_dim]; workspace uint8 of
    kv_attention_workspace() bytes (both allocated when None, on the stream that the call runs on). Rows of no request, and
    those of a request whose offsets do not fit, are left as they are in `out`: uninitialised, where it is allocated here.
    Returns `out`."""
    import torch
    index, heads, dim, i32 = cache._on_gpu(), cache.kv_heads, cache.head_dim, torch.int32
    hq = q.shape[1] if q.dim() == 3 else -1
    R, q_stride = _rows("q", q, hq, dim, index)
    B, width = lens.numel(), table.shape[-1]
    if row_start is not None:
        if max_rows is None:
            _refuse("row_start needs max_rows, the most rows of one request")
    elif max_rows is None:
        max_rows = R // B if B and R % B == 0 else _refuse(f"{R} rows do not go round {B} requests: give row_start")
    new_stride, k_ptr, v_ptr = 0, None, None
    if k_new is not None or v_new is not None:
        if k_new is None or v_new is None:
            _refuse("k_new and v_new go together")
        new = _rows("k_new", k_new, heads, dim, index)
        if new[0] != R or (not _same_rows(k_new, v_new) and _rows("v_new", v_new, heads, dim, index) != new):
            _refuse("k_new and v_new must have q's rows and one row stride")
        new_stride, k_ptr, v_ptr = new[1], k_new.data_ptr(), v_new.data_ptr()
    made = out is None
    if made:
        if stream is not None:
            out = _empty_on(stream, q, (R, hq, dim))
        else:
            out = torch.empty_like(q) if q.is_contiguous() else q.new_empty((R, hq, dim))
        out_stride = hq * dim
    else:
        n, out_stride = _rows("out", out, hq, dim, index)
        if n != R:
            _refuse("out must have q's rows")
    if R == 0:
        return out
    if workspace is None:
        size = kv_attention_workspace(cache, hq, B, max_rows)
        n = (size + 1) // 2      # bf16, as q is: two bytes an element
        workspace = q.new_empty(n) if stream is None else _empty_on(stream, q, n)
    elif workspace.dtype is not torch.uint8 or workspace.get_device() != index or not workspace.is_contiguous():
        _refuse(f"workspace: need a contiguous uint8 tensor on cuda:{index}")
    else:
        size = workspace.numel()
    mask_ptr = start_ptr = None
    if not (table.dtype is i32 and lens.dtype is i32 and table.shape == (B, width) and lens.dim() == 1
            and table.get_device() == index and lens.get_device() == index and table.is_contiguous() and lens.is_contiguous()):
        _ints("table", table, (B, width), index)
        _ints("lens", lens, (B,), index)
    if mask is not None:
        if not (mask.dtype is i32 and mask.shape == (R,) and mask.get_device() == index and mask.is_contiguous()):
            _ints("mask", mask, (R,), index)
        mask_ptr = mask.data_ptr()
    if row_start is not None:
        if not (row_start.dtype is i32 and row_start.shape == (B + 1,) and row_start.get_device() == index and row_start.is_contiguous()):
            _ints("row_start", row_start, (B + 1,), index)
        start_ptr = row_start.data_ptr()
    _call_on(index, _lib.lib().tl_kv_attention,
             (q.data_ptr(), q_stride, hq, cache._c, table.data_ptr(), width, lens.data_ptr(), B, k_ptr, v_ptr, new_stride,
              mask_ptr, start_ptr, R, max_rows, dim ** -0.5 if scale is None else scale, out.data_ptr(), out_stride, workspace.data_ptr(), size,
              _stream_of(index, stream)))
    if made and stream is not None:   # the caller may use it on the current stream, after waiting for the other one
        out.record_stream(torch.cuda.current_stream(index))
    return out
