"""Python binding of libkin.so: block top-k sparse decode attention on B200.

Argument marshalling only.  Every function has the name of the C entry point
it wraps (see include/kin.h for the exact semantics, layouts and errors),
takes CUDA tensors, passes their device pointers and the current CUDA stream,
and raises KinError when the library returns a non-OK status.  All
arithmetic runs in the library's CUDA kernels; there is no fallback: if
libkin.so is missing or cannot be loaded, the first call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkin.so")

KIN_OK = 0
STATUS_NAMES = {
    0: "KIN_OK", 1: "KIN_ERR_INVALID_ARG", 2: "KIN_ERR_WORKSPACE", 3: "KIN_ERR_CAPACITY",
    4: "KIN_ERR_CUDA", 5: "KIN_ERR_DEVICE_DATA", 6: "KIN_ERR_TIMEOUT",
}
EXPORTED = (
    "kin_status_string", "kin_workspace_bytes", "kin_block_means_build",
    "kin_block_means_update", "kin_block_topk_select", "kin_sparse_decode_attn",
    "kin_block_topk_select_noalloc", "kin_block_means_build_paged", "kin_block_means_update_paged",
    "kin_sparse_decode_attn_paged", "kin_block_means_build_ex", "kin_block_means_update_ex",
    "kin_block_topk_select_ex", "kin_token_topk_workspace_bytes", "kin_token_topk_decode_attn",
    "kin_block_topk_select_paged", "kin_dual_means_bytes", "kin_dual_page_means_bytes",
    "kin_kv4_store", "kin_kv4_append", "kin_kv4_load", "kin_kv_attn_workspace_bytes", "kin_kv_decode_attn",
    "kin_kv_evict_workspace_bytes", "kin_kv_evict",
)
KIN_MEANS_F32, KIN_MEANS_BF16, KIN_MEANS_DUAL = 0, 1, 2
KIN_MEANS_PER_PAGE = 0x100
KIN_KV_BF16, KIN_KV_INT4 = 0, 1
NOALLOC_SCRATCH_FLOATS = 1 << 21  # KIN_NOALLOC_SCRATCH_FLOATS in include/kin.h


class KinError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")


class kin_dims(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("max_seq_len", ctypes.c_int32),
    ]

    def __repr__(self):
        return "kin_dims(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


class kin_kv(ctypes.Structure):
    _fields_ = [
        ("format", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("block_table", ctypes.c_void_p),
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("k_scales", ctypes.c_void_p),
        ("v_scales", ctypes.c_void_p),
    ]


def make_dims(batch, num_kv_heads, num_q_heads, head_dim, block_size, max_seq_len) -> kin_dims:
    return kin_dims(batch, num_kv_heads, num_q_heads, head_dim, block_size, max_seq_len)


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libkin.so (once) and declare the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"libkin.so not found at {path}: build it with "
            "`python -m block_top_sparse_kin_b200.build` (nvcc, sm_100a)")
    lib = ctypes.CDLL(path)
    vp, i32, sz, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
    dp = ctypes.POINTER(kin_dims)
    lib.kin_status_string.argtypes = [ctypes.c_int]
    lib.kin_status_string.restype = ctypes.c_char_p
    lib.kin_workspace_bytes.argtypes = [dp, i32]
    lib.kin_workspace_bytes.restype = sz
    lib.kin_block_means_build.argtypes = [dp, vp, vp, vp, vp, vp]
    lib.kin_block_means_build.restype = ctypes.c_int
    lib.kin_block_means_update.argtypes = [dp, vp, vp, vp, vp, vp, vp, i32, vp, vp]
    lib.kin_block_means_update.restype = ctypes.c_int
    lib.kin_block_topk_select.argtypes = [dp, vp, vp, vp, i32, vp, vp, vp, sz, vp, vp]
    lib.kin_block_topk_select.restype = ctypes.c_int
    lib.kin_sparse_decode_attn.argtypes = [dp, vp, vp, vp, vp, vp, vp, i32, f32, vp, vp, vp, sz,
                                           vp, vp]
    lib.kin_sparse_decode_attn.restype = ctypes.c_int
    lib.kin_block_topk_select_noalloc.argtypes = [dp, vp, vp, vp, i32, vp, vp, vp, vp]
    lib.kin_block_topk_select_noalloc.restype = ctypes.c_int
    lib.kin_block_means_build_paged.argtypes = [dp, vp, i32, vp, vp, vp, vp, vp]
    lib.kin_block_means_build_paged.restype = ctypes.c_int
    lib.kin_block_means_update_paged.argtypes = [dp, vp, vp, i32, vp, vp, vp, vp, vp, i32, vp, vp]
    lib.kin_block_means_update_paged.restype = ctypes.c_int
    lib.kin_sparse_decode_attn_paged.argtypes = [dp, vp, vp, vp, i32, vp, vp, vp, vp, i32, f32, vp, vp, vp,
                                                 sz, vp, vp]
    lib.kin_sparse_decode_attn_paged.restype = ctypes.c_int
    lib.kin_block_means_build_ex.argtypes = [dp, vp, i32, vp, vp, vp, i32, vp, vp]
    lib.kin_block_means_build_ex.restype = ctypes.c_int
    lib.kin_block_means_update_ex.argtypes = [dp, vp, vp, i32, vp, vp, i32, vp, vp, vp, i32, vp, vp]
    lib.kin_block_means_update_ex.restype = ctypes.c_int
    lib.kin_block_topk_select_ex.argtypes = [dp, vp, vp, i32, vp, i32, vp, vp, vp, sz, vp, vp]
    lib.kin_block_topk_select_ex.restype = ctypes.c_int
    lib.kin_token_topk_workspace_bytes.argtypes = [dp, i32]
    lib.kin_token_topk_workspace_bytes.restype = sz
    lib.kin_token_topk_decode_attn.argtypes = [dp, vp, vp, vp, vp, i32, f32, vp, vp, vp, vp, sz, vp, vp]
    lib.kin_token_topk_decode_attn.restype = ctypes.c_int
    lib.kin_block_topk_select_paged.argtypes = [dp, vp, vp, i32, i32, vp, vp, i32, vp, vp, vp, sz, vp, vp]
    lib.kin_block_topk_select_paged.restype = ctypes.c_int
    lib.kin_dual_means_bytes.argtypes = [dp]
    lib.kin_dual_means_bytes.restype = sz
    lib.kin_dual_page_means_bytes.argtypes = [dp, i32]
    lib.kin_dual_page_means_bytes.restype = sz
    kp = ctypes.POINTER(kin_kv)
    lib.kin_kv4_store.argtypes = [dp, kp, kp, vp, vp, i32, vp, vp]
    lib.kin_kv4_store.restype = ctypes.c_int
    lib.kin_kv4_append.argtypes = [dp, kp, vp, i32, vp, vp, vp, vp, i32, vp, vp]
    lib.kin_kv4_append.restype = ctypes.c_int
    lib.kin_kv4_load.argtypes = [dp, kp, vp, vp, i32, vp, vp, vp, vp]
    lib.kin_kv4_load.restype = ctypes.c_int
    lib.kin_kv_attn_workspace_bytes.argtypes = [dp, i32, i32]
    lib.kin_kv_attn_workspace_bytes.restype = sz
    lib.kin_kv_decode_attn.argtypes = [dp, vp, kp, vp, vp, vp, i32, f32, vp, vp, vp, vp, sz, vp, vp]
    lib.kin_kv_decode_attn.restype = ctypes.c_int
    lib.kin_kv_evict_workspace_bytes.argtypes = [dp, i32]
    lib.kin_kv_evict_workspace_bytes.restype = sz
    lib.kin_kv_evict.argtypes = [dp, kp, vp, vp, i32, i32, i32, dp, kp, vp, vp, vp, i32, vp, vp, sz, vp, vp]
    lib.kin_kv_evict.restype = ctypes.c_int
    _lib = lib
    return lib


# a CUDA tensor at hand means that CUDA is initialised: the raw queries are enough
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # where torch has none, by its public call


def _dev(t: Optional[torch.Tensor], name: str, dtype=None, nullable=False, count: Optional[int] = None):
    """The device pointer of t after checking that it is a contiguous CUDA
    tensor on the current device, of an accepted dtype and, when count is
    given, of at least count elements (what the library reads or writes
    through it): a short tensor is refused here, on the host, because the C
    ABI receives bare pointers and could not see it."""
    if t is None:
        if nullable:
            return None
        raise ValueError(f"{name} is required")
    if (t.is_cuda and t.get_device() == _current_device() and t.is_contiguous()
            and (dtype is None or t.dtype is dtype or (dtype.__class__ is tuple and t.dtype in dtype))
            and (count is None or t.numel() >= count)):
        return t.data_ptr()
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != _current_device():
        raise ValueError(f"{name} is on {t.device}; the calls run on the current device "
                         f"cuda:{torch.cuda.current_device()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype is not dtype and (not isinstance(dtype, tuple) or t.dtype not in dtype):
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    raise ValueError(f"{name} holds {t.numel()} elements; the dims need {count}")


def _ptr(t, name: str, dtype, count, dev: int):
    """_dev for the common case, at a third of its cost: a contiguous tensor
    of one dtype on the current device `dev`."""
    if (t is not None and count is not None and t.get_device() == dev and t.dtype is dtype and t.numel() >= count
            and t.is_contiguous()):
        return t.data_ptr()
    return _dev(t, name, _BF16 if dtype is torch.bfloat16 else dtype, count=count)


class _Counts:
    """Element counts of every buffer a call touches, from the dims (all
    None when the dims are invalid: the call then returns the library's
    own status for them)."""

    def __init__(self, dims: kin_dims):
        ok = load_library().kin_workspace_bytes(ctypes.byref(dims), 2) > 0
        B, Hkv, Hq, D = dims.batch, dims.num_kv_heads, dims.num_q_heads, dims.head_dim
        bs, L = dims.block_size, dims.max_seq_len
        nbcap = -(-L // bs) if ok else 0
        self.ok = ok
        self.q = B * Hq * D if ok else None            # q, out
        self.lse = B * Hq if ok else None
        self.cache = B * Hkv * L * D if ok else None   # k_cache, v_cache
        self.means = B * Hkv * nbcap * D if ok else None
        self.table = B * nbcap if ok else None
        self.lens = B if ok else None
        self.pairs = B * Hkv if ok else None           # sel_cnt
        self.page = Hkv * bs * D if ok else None       # one page of a pool
        self.page_mean = Hkv * D if ok else None       # one per-page mean
        self.bkd = B * Hkv * D if ok else None         # one appended row per (b, h)
        self.rows = B * Hkv * L if ok else None        # tokens of the cache (accumulated weights)

    def times(self, n, per):
        return None if per is None else int(n) * per


@functools.lru_cache(maxsize=256)
def _counts_of(*fields) -> _Counts:
    return _Counts(kin_dims(*fields))


def _counts(d: kin_dims) -> _Counts:
    """The counts of these dims' values (kept: a decode loop asks for the same ones each step)."""
    return _counts_of(d.batch, d.num_kv_heads, d.num_q_heads, d.head_dim, d.block_size, d.max_seq_len)


def _status(dev_status):
    return None if dev_status is None else _dev(dev_status, "dev_status", torch.int32, nullable=True, count=1)


def _stream(stream):
    if stream is None:
        if _current_stream is None:
            return torch.cuda.current_stream().cuda_stream
        return _current_stream(_current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(rc: int, where: str):
    if rc != KIN_OK:
        raise KinError(rc, where)


_BF16 = (torch.bfloat16, torch.uint16, torch.int16)


def kin_status_string(status: int) -> str:
    return load_library().kin_status_string(status).decode()


def kin_workspace_bytes(dims: kin_dims, k_blocks: int) -> int:
    return int(load_library().kin_workspace_bytes(ctypes.byref(dims), k_blocks))


def alloc_workspace(dims: kin_dims, k_blocks: int, device="cuda") -> torch.Tensor:
    """A zero-filled workspace tensor of kin_workspace_bytes (torch allocations are 256-B aligned)."""
    n = kin_workspace_bytes(dims, k_blocks)
    if n == 0:
        raise KinError(1, "kin_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def kin_block_means_build(dims, k_cache, seq_lens, block_means, dev_status=None, stream=None):
    c = _counts(dims)
    rc = load_library().kin_block_means_build(
        ctypes.byref(dims), _dev(k_cache, "k_cache", _BF16, count=c.cache),
        _dev(seq_lens, "seq_lens", torch.int32, count=c.lens),
        _dev(block_means, "block_means", torch.float32, count=c.means), _status(dev_status), _stream(stream))
    _check(rc, "kin_block_means_build")


def kin_block_means_update(dims, k_cache, v_cache, block_means, seq_lens, k_new, v_new, n_new,
                           dev_status=None, stream=None):
    c = _counts(dims)
    new_rows = c.times(max(int(n_new), 0), c.bkd)
    rc = load_library().kin_block_means_update(
        ctypes.byref(dims), _dev(k_cache, "k_cache", _BF16, count=c.cache),
        _dev(v_cache, "v_cache", _BF16, count=c.cache), _dev(block_means, "block_means", torch.float32, count=c.means),
        _dev(seq_lens, "seq_lens", torch.int32, count=c.lens), _dev(k_new, "k_new", _BF16, count=new_rows),
        _dev(v_new, "v_new", _BF16, count=new_rows), int(n_new), _status(dev_status), _stream(stream))
    _check(rc, "kin_block_means_update")


def kin_block_topk_select(dims, q, block_means, seq_lens, k_blocks, sel_idx, sel_cnt, workspace,
                          dev_status=None, stream=None):
    c = _counts(dims)
    rc = load_library().kin_block_topk_select(
        ctypes.byref(dims), _dev(q, "q", _BF16, count=c.q), _dev(block_means, "block_means", torch.float32, count=c.means),
        _dev(seq_lens, "seq_lens", torch.int32, count=c.lens), int(k_blocks),
        _dev(sel_idx, "sel_idx", torch.int32, count=c.times(max(int(k_blocks), 0), c.pairs)),
        _dev(sel_cnt, "sel_cnt", torch.int32, count=c.pairs), _dev(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _status(dev_status), _stream(stream))
    _check(rc, "kin_block_topk_select")


def kin_sparse_decode_attn(dims, q, k_cache, v_cache, seq_lens, sel_idx, sel_cnt, k_blocks,
                           softmax_scale, out, lse, workspace, dev_status=None, stream=None):
    c = _counts(dims)
    rc = load_library().kin_sparse_decode_attn(
        ctypes.byref(dims), _dev(q, "q", _BF16, count=c.q), _dev(k_cache, "k_cache", _BF16, count=c.cache),
        _dev(v_cache, "v_cache", _BF16, count=c.cache), _dev(seq_lens, "seq_lens", torch.int32, count=c.lens),
        _dev(sel_idx, "sel_idx", torch.int32, count=c.times(max(int(k_blocks), 0), c.pairs)),
        _dev(sel_cnt, "sel_cnt", torch.int32, count=c.pairs), int(k_blocks), float(softmax_scale),
        _dev(out, "out", _BF16, count=c.q), _dev(lse, "lse", torch.float32, nullable=True, count=c.lse),
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(), _status(dev_status),
        _stream(stream))
    _check(rc, "kin_sparse_decode_attn")


def kin_block_topk_select_noalloc(dims, q, block_means, seq_lens, k_blocks, sel_idx, sel_cnt,
                                  dev_status=None, stream=None):
    """kin_block_topk_select without a workspace, for callers that may not
    allocate device memory: the scratch lives in a fixed array inside
    libkin.so (see include/kin.h for its limit and its sharing rules)."""
    c = _counts(dims)
    rc = load_library().kin_block_topk_select_noalloc(
        ctypes.byref(dims), _dev(q, "q", _BF16, count=c.q), _dev(block_means, "block_means", torch.float32, count=c.means),
        _dev(seq_lens, "seq_lens", torch.int32, count=c.lens), int(k_blocks),
        _dev(sel_idx, "sel_idx", torch.int32, count=c.times(max(int(k_blocks), 0), c.pairs)),
        _dev(sel_cnt, "sel_cnt", torch.int32, count=c.pairs), _status(dev_status), _stream(stream))
    _check(rc, "kin_block_topk_select_noalloc")


# ---------------------------------------------------------------- paged KV
# k_pages / v_pages [num_pages, Hkv, bs, D] bf16; block_table [B, ceil(Lcap / bs)]
# int32 (page of each logical block).  See include/kin.h.

def kin_block_means_build_paged(dims, k_pages, block_table, seq_lens, block_means, dev_status=None,
                                stream=None):
    c = _counts(dims)
    pages = int(k_pages.shape[0])
    rc = load_library().kin_block_means_build_paged(
        ctypes.byref(dims), _dev(k_pages, "k_pages", _BF16, count=c.times(pages, c.page)), pages,
        _dev(block_table, "block_table", torch.int32, count=c.table),
        _dev(seq_lens, "seq_lens", torch.int32, count=c.lens),
        _dev(block_means, "block_means", torch.float32, count=c.means), _status(dev_status), _stream(stream))
    _check(rc, "kin_block_means_build_paged")


def kin_block_means_update_paged(dims, k_pages, v_pages, block_table, block_means, seq_lens, k_new, v_new,
                                 n_new, dev_status=None, stream=None):
    c = _counts(dims)
    pages = int(k_pages.shape[0])
    new_rows = c.times(max(int(n_new), 0), c.bkd)
    rc = load_library().kin_block_means_update_paged(
        ctypes.byref(dims), _dev(k_pages, "k_pages", _BF16, count=c.times(pages, c.page)),
        _dev(v_pages, "v_pages", _BF16, count=c.times(pages, c.page)), pages,
        _dev(block_table, "block_table", torch.int32, count=c.table),
        _dev(block_means, "block_means", torch.float32, count=c.means),
        _dev(seq_lens, "seq_lens", torch.int32, count=c.lens), _dev(k_new, "k_new", _BF16, count=new_rows),
        _dev(v_new, "v_new", _BF16, count=new_rows), int(n_new), _status(dev_status), _stream(stream))
    _check(rc, "kin_block_means_update_paged")


def kin_sparse_decode_attn_paged(dims, q, k_pages, v_pages, block_table, seq_lens, sel_idx, sel_cnt, k_blocks,
                                 softmax_scale, out, lse, workspace, dev_status=None, stream=None):
    c = _counts(dims)
    pages = int(k_pages.shape[0])
    rc = load_library().kin_sparse_decode_attn_paged(
        ctypes.byref(dims), _dev(q, "q", _BF16, count=c.q), _dev(k_pages, "k_pages", _BF16, count=c.times(pages, c.page)),
        _dev(v_pages, "v_pages", _BF16, count=c.times(pages, c.page)), pages,
        _dev(block_table, "block_table", torch.int32, count=c.table),
        _dev(seq_lens, "seq_lens", torch.int32, count=c.lens),
        _dev(sel_idx, "sel_idx", torch.int32, count=c.times(max(int(k_blocks), 0), c.pairs)),
        _dev(sel_cnt, "sel_cnt", torch.int32, count=c.pairs), int(k_blocks), float(softmax_scale),
        _dev(out, "out", _BF16, count=c.q), _dev(lse, "lse", torch.float32, nullable=True, count=c.lse),
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(), _status(dev_status),
        _stream(stream))
    _check(rc, "kin_sparse_decode_attn_paged")


# ------------------------------------------------ extended: bf16 block means
# The means dtype follows the block_means tensor (float32 or bfloat16);
# block_table None selects the contiguous cache.  See include/kin.h.

def _means(block_means, count=None, name="block_means", dims=None, pages=None):
    """The means pointer and its dtype code, from the tensor: float32 rows,
    bfloat16 rows, or a uint8 buffer of dual means (fp32 rows, their bf16
    rounding and the rows' error radii: see kin_dual_means_bytes; per page
    when `pages` is given, see kin_dual_page_means_bytes)."""
    if block_means is not None and block_means.dtype == torch.float32:
        return _dev(block_means, name, torch.float32, count=count), KIN_MEANS_F32
    if block_means is not None and block_means.dtype == torch.uint8:
        if dims is None:
            nbytes = None
        elif pages is not None:
            nbytes = kin_dual_page_means_bytes(dims, pages)
        else:
            nbytes = kin_dual_means_bytes(dims)
        return _dev(block_means, name, torch.uint8, count=nbytes or None), KIN_MEANS_DUAL
    return _dev(block_means, name, torch.bfloat16, count=count), KIN_MEANS_BF16


def kin_dual_means_bytes(dims: kin_dims) -> int:
    """Bytes of a dual block-means buffer (KIN_MEANS_DUAL) for these dims."""
    return int(load_library().kin_dual_means_bytes(ctypes.byref(dims)))


def kin_dual_page_means_bytes(dims: kin_dims, num_pages: int) -> int:
    """Bytes of a dual block-means buffer stored per page (KIN_MEANS_DUAL |
    KIN_MEANS_PER_PAGE) for a pool of num_pages pages."""
    return int(load_library().kin_dual_page_means_bytes(ctypes.byref(dims), int(num_pages)))


def alloc_dual_page_means(dims: kin_dims, num_pages: int, device="cuda") -> torch.Tensor:
    """A dual block-means buffer per page (uint8), filled by the build/update
    calls with per_page=True and read by kin_block_topk_select_paged."""
    n = kin_dual_page_means_bytes(dims, num_pages)
    if n == 0:
        raise KinError(1, "kin_dual_page_means_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def alloc_dual_means(dims: kin_dims, device="cuda") -> torch.Tensor:
    """A dual block-means buffer (uint8, 256-byte aligned as torch allocates),
    filled by kin_block_means_build_ex / _update_ex and read by
    kin_block_topk_select_ex."""
    n = kin_dual_means_bytes(dims)
    if n == 0:
        raise KinError(1, "kin_dual_means_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def _layout(rows, block_table, c: _Counts):
    """(num_pages, table pointer, rows per K/V tensor): the contiguous cache
    without a table, else the page pool it indexes."""
    if block_table is None:
        return 0, None, c.cache
    pages = int(rows.shape[0])
    return pages, _dev(block_table, "block_table", torch.int32, count=c.table), c.times(pages, c.page)


def kin_block_means_build_ex(dims, k_rows, seq_lens, block_means, block_table=None, dev_status=None,
                             stream=None, per_page=False):
    """per_page: block_means is [num_pages, Hkv, D] (one mean per page; needs block_table)."""
    c = _counts(dims)
    pages, table, rows = _layout(k_rows, block_table, c)
    means, dtype = _means(block_means, c.times(pages, c.page_mean) if per_page else c.means, dims=dims,
                          pages=pages if per_page else None)
    dtype |= KIN_MEANS_PER_PAGE if per_page else 0
    rc = load_library().kin_block_means_build_ex(
        ctypes.byref(dims), _dev(k_rows, "k_rows", _BF16, count=rows), pages, table,
        _dev(seq_lens, "seq_lens", torch.int32, count=c.lens), means, dtype, _status(dev_status), _stream(stream))
    _check(rc, "kin_block_means_build_ex")


def kin_block_means_update_ex(dims, k_rows, v_rows, block_means, seq_lens, k_new, v_new, n_new,
                              block_table=None, dev_status=None, stream=None, per_page=False):
    c = _counts(dims)
    pages, table, rows = _layout(k_rows, block_table, c)
    means, dtype = _means(block_means, c.times(pages, c.page_mean) if per_page else c.means, dims=dims,
                          pages=pages if per_page else None)
    dtype |= KIN_MEANS_PER_PAGE if per_page else 0
    new_rows = c.times(max(int(n_new), 0), c.bkd)
    rc = load_library().kin_block_means_update_ex(
        ctypes.byref(dims), _dev(k_rows, "k_rows", _BF16, count=rows), _dev(v_rows, "v_rows", _BF16, count=rows),
        pages, table, means, dtype, _dev(seq_lens, "seq_lens", torch.int32, count=c.lens),
        _dev(k_new, "k_new", _BF16, count=new_rows), _dev(v_new, "v_new", _BF16, count=new_rows), int(n_new),
        _status(dev_status), _stream(stream))
    _check(rc, "kin_block_means_update_ex")


def kin_block_topk_select_ex(dims, q, block_means, seq_lens, k_blocks, sel_idx, sel_cnt, workspace,
                             dev_status=None, stream=None):
    c = _counts(dims)
    means, dtype = _means(block_means, c.means, dims=dims)
    rc = load_library().kin_block_topk_select_ex(
        ctypes.byref(dims), _dev(q, "q", _BF16, count=c.q), means, dtype,
        _dev(seq_lens, "seq_lens", torch.int32, count=c.lens), int(k_blocks),
        _dev(sel_idx, "sel_idx", torch.int32, count=c.times(max(int(k_blocks), 0), c.pairs)),
        _dev(sel_cnt, "sel_cnt", torch.int32, count=c.pairs), _dev(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _status(dev_status), _stream(stream))
    _check(rc, "kin_block_topk_select_ex")


# --------------------------------------------------- token-level top-k attention

def kin_token_topk_workspace_bytes(dims: kin_dims, k_tokens: int) -> int:
    return int(load_library().kin_token_topk_workspace_bytes(ctypes.byref(dims), k_tokens))


def alloc_token_workspace(dims: kin_dims, k_tokens: int, device="cuda") -> torch.Tensor:
    n = kin_token_topk_workspace_bytes(dims, k_tokens)
    if n == 0:
        raise KinError(1, "kin_token_topk_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def kin_token_topk_decode_attn(dims, q, k_cache, v_cache, seq_lens, k_tokens, softmax_scale, out, lse, workspace,
                               sel_tokens=None, dev_status=None, stream=None):
    c = _counts(dims)
    rc = load_library().kin_token_topk_decode_attn(
        ctypes.byref(dims), _dev(q, "q", _BF16, count=c.q), _dev(k_cache, "k_cache", _BF16, count=c.cache),
        _dev(v_cache, "v_cache", _BF16, count=c.cache), _dev(seq_lens, "seq_lens", torch.int32, count=c.lens),
        int(k_tokens), float(softmax_scale), _dev(out, "out", _BF16, count=c.q),
        _dev(lse, "lse", torch.float32, nullable=True, count=c.lse),
        _dev(sel_tokens, "sel_tokens", torch.int32, nullable=True, count=c.times(max(int(k_tokens), 0), c.lse)),
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(), _status(dev_status),
        _stream(stream))
    _check(rc, "kin_token_topk_decode_attn")


def kin_block_topk_select_paged(dims, q, page_means, block_table, seq_lens, k_blocks, sel_idx, sel_cnt, workspace,
                                dev_status=None, stream=None, num_pages=None):
    """The select over per-page block means [num_pages, Hkv, D] (fp32 or bf16),
    or a per-page dual buffer (uint8; num_pages then required), found through
    block_table: the shared-prompt layout (see include/kin.h)."""
    c = _counts(dims)
    if page_means is not None and page_means.dtype == torch.uint8:
        if num_pages is None:
            raise ValueError("page_means: a dual buffer needs num_pages")
        pages = int(num_pages)
        means, dtype = _means(page_means, None, "page_means", dims=dims, pages=pages)
    else:
        pages = int(page_means.shape[0])
        means, dtype = _means(page_means, c.times(pages, c.page_mean), "page_means")
    rc = load_library().kin_block_topk_select_paged(
        ctypes.byref(dims), _dev(q, "q", _BF16, count=c.q), means, dtype, pages,
        _dev(block_table, "block_table", torch.int32, count=c.table),
        _dev(seq_lens, "seq_lens", torch.int32, count=c.lens), int(k_blocks),
        _dev(sel_idx, "sel_idx", torch.int32, count=c.times(max(int(k_blocks), 0), c.pairs)),
        _dev(sel_cnt, "sel_cnt", torch.int32, count=c.pairs), _dev(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _status(dev_status), _stream(stream))
    _check(rc, "kin_block_topk_select_paged")


# ------------------------------------- 4-bit caches, attention weights, eviction

class KvCache:
    """A KV cache as the kin_kv_* calls take it: bf16 rows (no scales), or
    4-bit codes (uint8) with their bf16 scales; contiguous, or a page pool
    with its block_table.  Holds the tensors it is made of; their types,
    device and layout are checked at the first call that takes it, their
    places (they must stay where they are) and sizes at every one."""

    __slots__ = ("_k", "_v", "_k_scales", "_v_scales", "_block_table", "_c", "_at", "_device")

    def __init__(self, k, v, k_scales=None, v_scales=None, block_table=None):
        if (k_scales is None) != (v_scales is None):
            raise ValueError("a 4-bit cache has k_scales and v_scales")
        self._k, self._v, self._k_scales, self._v_scales, self._block_table = k, v, k_scales, v_scales, block_table
        self._c = None

    k = property(lambda self: self._k)
    v = property(lambda self: self._v)
    k_scales = property(lambda self: self._k_scales)
    v_scales = property(lambda self: self._v_scales)
    block_table = property(lambda self: self._block_table)

    @property
    def int4(self) -> bool:
        return self._k_scales is not None

    def _tensors(self):
        return [t for t in (self._k, self._v, self._k_scales, self._v_scales, self._block_table) if t is not None]

    def _struct(self, c: "_Counts", name: str):
        """The C descriptor and the pool's pages, after the checks every call makes of its tensors."""
        if self._c is None:
            pages = 0 if self._block_table is None else int(self._k.shape[0])
            rows = torch.uint8 if self.int4 else _BF16
            table = None if self._block_table is None else _dev(self._block_table, f"{name}.block_table", torch.int32)
            scales = (_dev(self._k_scales, f"{name}.k_scales", _BF16), _dev(self._v_scales, f"{name}.v_scales", _BF16)) \
                if self.int4 else (None, None)
            self._c = kin_kv(KIN_KV_INT4 if self.int4 else KIN_KV_BF16, pages, table, _dev(self._k, f"{name}.k", rows),
                             _dev(self._v, f"{name}.v", rows), *scales)
            self._at = [t.data_ptr() for t in self._tensors()]
            self._device = _current_device()
        k, v, ks, vs, table, at = self._k, self._v, self._k_scales, self._v_scales, self._block_table, self._at
        if self._device != _current_device():
            raise ValueError(f"{name} is on cuda:{self._device}; the calls run on the current device")
        if (k.data_ptr() != at[0] or v.data_ptr() != at[1] or (ks is not None and (ks.data_ptr() != at[2] or vs.data_ptr() != at[3]))
                or (table is not None and table.data_ptr() != at[-1])):
            raise ValueError(f"{name}: a tensor of the cache has moved since its first call")
        if c.ok:
            need = c.cache if table is None else self._c.num_pages * c.page
            if ks is None:
                fits = k.numel() >= need and v.numel() >= need
            else:
                codes, scales = need >> 1, need >> 5
                fits = k.numel() >= codes and v.numel() >= codes and ks.numel() >= scales and vs.numel() >= scales
            if not fits or (table is not None and table.numel() < c.table):
                raise ValueError(f"{name}: a tensor of the cache is smaller than the dims need ({need} channels in k and in v"
                                 + (f", {c.table} table entries)" if table is not None else ")"))
        return self._c, self._c.num_pages


def alloc_kv4(dims: kin_dims, num_pages: Optional[int] = None, block_table=None, device="cuda") -> KvCache:
    """A zero-filled 4-bit cache for these dims: contiguous, or a pool of
    num_pages pages found through block_table."""
    if (num_pages is None) != (block_table is None):
        raise ValueError("a page pool needs num_pages and block_table")
    if num_pages is None:
        shape = (dims.batch, dims.num_kv_heads, dims.max_seq_len)
    else:
        shape = (int(num_pages), dims.num_kv_heads, dims.block_size)
    codes = [torch.zeros(shape + (dims.head_dim // 2,), dtype=torch.uint8, device=device) for _ in range(2)]
    scales = [torch.zeros(shape + (dims.head_dim // 32,), dtype=torch.bfloat16, device=device) for _ in range(2)]
    return KvCache(*codes, *scales, block_table=block_table)


def _kv_means(block_means, c: _Counts, dims, pages, per_page):
    """The optional block means beside a cache: pointer and dtype code."""
    if block_means is None:
        return None, KIN_MEANS_F32
    means, dtype = _means(block_means, c.times(pages, c.page_mean) if per_page else c.means, dims=dims,
                          pages=pages if per_page else None)
    return means, dtype | (KIN_MEANS_PER_PAGE if per_page else 0)


def kin_kv4_store(dims, src: KvCache, dst: KvCache, seq_lens, block_means=None, dev_status=None, stream=None,
                  per_page=False):
    """A prefilled bf16 cache into a 4-bit one, with its block means."""
    c = _counts(dims)
    s, _ = src._struct(c, "src")
    d, pages = dst._struct(c, "dst")
    means, dtype = _kv_means(block_means, c, dims, pages, per_page)
    rc = load_library().kin_kv4_store(
        ctypes.byref(dims), ctypes.byref(s), ctypes.byref(d), _dev(seq_lens, "seq_lens", torch.int32, count=c.lens),
        means, dtype, _status(dev_status), _stream(stream))
    _check(rc, "kin_kv4_store")


def kin_kv4_append(dims, kv: KvCache, block_means, seq_lens, new_lens, k_new, v_new, n_new, dev_status=None,
                   stream=None, per_page=False):
    """n_new tokens onto a 4-bit cache; new_lens may be seq_lens (in place)."""
    c = _counts(dims)
    d, pages = kv._struct(c, "kv")
    dev = _current_device()
    means, dtype = _kv_means(block_means, c, dims, pages, per_page)
    n = int(n_new)
    new_rows = c.times(max(n, 0), c.bkd)
    i32, bf16 = torch.int32, torch.bfloat16
    rc = load_library().kin_kv4_append(
        ctypes.byref(dims), ctypes.byref(d), means, dtype, _ptr(seq_lens, "seq_lens", i32, c.lens, dev),
        _ptr(new_lens, "new_lens", i32, c.lens, dev), _ptr(k_new, "k_new", bf16, new_rows, dev),
        _ptr(v_new, "v_new", bf16, new_rows, dev), n, _status(dev_status), _stream(stream))
    _check(rc, "kin_kv4_append")


def kin_kv4_load(dims, kv: KvCache, seq_lens, k_out, v_out, starts=None, n=None, dev_status=None, stream=None):
    """Rows of a 4-bit cache as bf16: n tokens a sequence from starts (0 when
    not given) into k_out / v_out [B, Hkv, n, D]; n defaults to k_out's."""
    c = _counts(dims)
    d, _ = kv._struct(c, "kv")
    dev = _current_device()
    n = int(k_out.shape[2]) if n is None else int(n)
    rows = c.times(max(n, 0), c.bkd)
    i32, bf16 = torch.int32, torch.bfloat16
    rc = load_library().kin_kv4_load(
        ctypes.byref(dims), ctypes.byref(d), _ptr(seq_lens, "seq_lens", i32, c.lens, dev),
        None if starts is None else _ptr(starts, "starts", i32, c.lens, dev), n, _ptr(k_out, "k_out", bf16, rows, dev),
        _ptr(v_out, "v_out", bf16, rows, dev), _status(dev_status), _stream(stream))
    _check(rc, "kin_kv4_load")


def kin_kv_attn_workspace_bytes(dims: kin_dims, k_blocks: int, with_acc: bool = False) -> int:
    return int(load_library().kin_kv_attn_workspace_bytes(ctypes.byref(dims), int(k_blocks), int(with_acc)))


def alloc_kv_attn_workspace(dims: kin_dims, k_blocks: int, acc: bool = False, device="cuda") -> torch.Tensor:
    """A zero-filled workspace of kin_kv_attn_workspace_bytes."""
    n = kin_kv_attn_workspace_bytes(dims, k_blocks, acc)
    if n == 0:
        raise KinError(1, "kin_kv_attn_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def kin_kv_decode_attn(dims, q, kv: KvCache, seq_lens, sel_idx, sel_cnt, k_blocks, softmax_scale, out, lse, workspace,
                       acc=None, dev_status=None, stream=None):
    """Decode attention over a bf16 or 4-bit cache; sel_idx and sel_cnt None
    with k_blocks 0 attend to every block; acc [B, Hkv, Lcap] fp32 takes the
    attention weights on top of what it holds."""
    c = _counts(dims)
    d, _ = kv._struct(c, "kv")
    dev = _current_device()
    k = int(k_blocks)
    i32, f32, bf16 = torch.int32, torch.float32, torch.bfloat16
    rc = load_library().kin_kv_decode_attn(
        ctypes.byref(dims), _ptr(q, "q", bf16, c.q, dev), ctypes.byref(d), _ptr(seq_lens, "seq_lens", i32, c.lens, dev),
        None if sel_idx is None else _ptr(sel_idx, "sel_idx", i32, c.times(max(k, 0), c.pairs), dev),
        None if sel_cnt is None else _ptr(sel_cnt, "sel_cnt", i32, c.pairs, dev), k, float(softmax_scale),
        _ptr(out, "out", bf16, c.q, dev), None if lse is None else _ptr(lse, "lse", f32, c.lse, dev),
        None if acc is None else _ptr(acc, "acc", f32, c.rows, dev), _dev(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _status(dev_status), _stream(stream))
    _check(rc, "kin_kv_decode_attn")


def kin_kv_evict_workspace_bytes(dims: kin_dims, n_keep: int) -> int:
    return int(load_library().kin_kv_evict_workspace_bytes(ctypes.byref(dims), int(n_keep)))


def alloc_kv_evict_workspace(dims: kin_dims, n_keep: int, device="cuda") -> torch.Tensor:
    n = kin_kv_evict_workspace_bytes(dims, n_keep)
    if n == 0:
        raise KinError(1, "kin_kv_evict_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def kin_kv_evict(dims, kv: KvCache, acc, seq_lens, n_keep, n_sink, n_recent, dst_dims, dst: KvCache, dst_acc, dst_lens,
                 workspace, block_means=None, sel_tokens=None, dev_status=None, stream=None, per_page=False):
    """The n_keep tokens of every (sequence, KV head) that stay (first n_sink,
    last n_recent, then by acc), moved in order to the cache dst."""
    c, cd = _counts(dims), _counts(dst_dims)
    s, _ = kv._struct(c, "kv")
    d, pages = dst._struct(cd, "dst")
    dev = _current_device()
    means, dtype = _kv_means(block_means, cd, dst_dims, pages, per_page)
    i32, f32, keep = torch.int32, torch.float32, int(n_keep)
    rc = load_library().kin_kv_evict(
        ctypes.byref(dims), ctypes.byref(s), _ptr(acc, "acc", f32, c.rows, dev), _ptr(seq_lens, "seq_lens", i32, c.lens, dev),
        keep, int(n_sink), int(n_recent), ctypes.byref(dst_dims), ctypes.byref(d),
        None if dst_acc is None else _ptr(dst_acc, "dst_acc", f32, cd.rows, dev), _ptr(dst_lens, "dst_lens", i32, c.lens, dev),
        means, dtype,
        None if sel_tokens is None else _ptr(sel_tokens, "sel_tokens", i32, c.times(max(keep, 0), c.pairs), dev),
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(), _status(dev_status), _stream(stream))
    _check(rc, "kin_kv_evict")
