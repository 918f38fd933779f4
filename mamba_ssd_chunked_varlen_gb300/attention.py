"""Python binding of the C ABI in include/ssd_attn.h (ctypes): the paged
key/value cache and the attention over it.

Argument marshalling only, as in ``binding``: the work runs in the CUDA kernels
of libssd_scan.so on torch's current stream (or `stream`), and there is no CPU
fallback.  The cache is a pair of tensors (num_pages, nheads_kv, page_size,
head_dim) in bfloat16, float8_e4m3fn or int8; the 8-bit types go with a pair of
fp32 scales (num_pages, nheads_kv, page_size).
"""
from __future__ import annotations

import ctypes

from . import binding
from .binding import SSD_OK, SSDError

# Every symbol include/ssd_attn.h declares.
EXPORTED_SYMBOLS = (
    "ssd_kv_cache_write",
    "ssd_kv_cache_read",
    "ssd_attn_varlen_workspace_size",
    "ssd_attn_varlen_fwd",
)

DEVERR_BAD_KV_LEN = 0x8
DEVERR_BAD_PAGE = 0x10

_fn = None


class _Functions:
    def __init__(self):
        import torch
        lib = binding.library()
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        # num_pages, page_size, table_width, table_stride, cache_type
        cache = [i64, i32, i32, i64, i32]
        self.write = lib.ssd_kv_cache_write
        self.read = lib.ssd_kv_cache_read
        for f in (self.write, self.read):
            f.restype = ctypes.c_int
            f.argtypes = [vp] * 9 + [i64, i32, i32, i32] + cache + [i64, i64, vp, vp]
        self.workspace_size = lib.ssd_attn_varlen_workspace_size
        self.workspace_size.restype = sz
        self.workspace_size.argtypes = [i64, i32, i32, i32, i32]
        self.attn = lib.ssd_attn_varlen_fwd
        self.attn.restype = ctypes.c_int
        self.attn.argtypes = ([vp] * 10 + [i64, i32, i32, i32, i32] + cache
                              + [i64, i64, ctypes.c_float, i32, vp, sz, vp, vp])
        self.types = {torch.bfloat16: 0, torch.float8_e4m3fn: 1, torch.int8: 2}
        self.bf16, self.f32, self.i32, self.u8 = (torch.bfloat16, torch.float32, torch.int32,
                                                  torch.uint8)
        self.u32 = torch.uint32
        self.current_stream = torch.cuda.current_stream


def _functions() -> _Functions:
    global _fn
    if _fn is None:
        _fn = _Functions()
    return _fn


def _ptr(t, what: str, dtype, device):
    """Address of a contiguous tensor of that type on that device."""
    if t.dtype != dtype:
        raise ValueError(f"{what} must have dtype {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{what} must be on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _rows(t, what: str, f, device):
    """Address and row pitch (elements) of a (rows, heads, head_dim) bf16 tensor
    whose rows are contiguous."""
    if t.dtype != f.bf16:
        raise ValueError(f"{what} must have dtype {f.bf16}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{what} must be on {device}, got {t.device}")
    n, h, d = t.shape
    s = t.stride()
    if (s[2] != 1 and d != 1) or (s[1] != d and h != 1):
        raise ValueError(f"{what}: each token's row must be contiguous")
    return t.data_ptr(), (s[0] if n > 1 else h * d)


def _cache(f, k_cache, v_cache, k_scale, v_scale, query_start_loc, kv_lens, block_table, device):
    """The arguments that all calls share: (nine pointers' tail, sizes)."""
    kind = f.types.get(k_cache.dtype)
    if kind is None:
        raise ValueError(f"k_cache must be bfloat16, float8_e4m3fn or int8, got {k_cache.dtype}")
    if not k_cache.is_cuda:
        raise ValueError("k_cache must be a CUDA tensor")
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must both have shape "
                         "(num_pages, nheads_kv, page_size, head_dim)")
    ks = vs = None
    if kind:
        if k_scale is None or v_scale is None:
            raise ValueError("an 8-bit cache needs k_scale and v_scale")
        if k_scale.shape != shape[:3] or v_scale.shape != shape[:3]:
            raise ValueError(f"k_scale and v_scale must have shape {tuple(shape[:3])}")
        ks, vs = _ptr(k_scale, "k_scale", f.f32, device), _ptr(v_scale, "v_scale", f.f32, device)
    elif k_scale is not None or v_scale is not None:
        raise ValueError("a bfloat16 cache has no scales")
    batch = query_start_loc.shape[0] - 1
    if kv_lens.shape != (batch,):
        raise ValueError(f"kv_lens must have shape ({batch},)")
    if block_table.dtype != f.i32 or block_table.device != device or block_table.dim() != 2 \
            or block_table.shape[0] != batch:
        raise ValueError(f"block_table must be an int32 tensor ({batch}, pages) on {device}")
    width = block_table.shape[1]
    if width > 1 and block_table.stride(1) != 1:
        raise ValueError("block_table: each sequence's entries must be contiguous")
    stride = block_table.stride(0) if batch > 1 else width
    return ((_ptr(k_cache, "k_cache", k_cache.dtype, device),
             _ptr(v_cache, "v_cache", k_cache.dtype, device), ks, vs,
             _ptr(query_start_loc, "query_start_loc", f.i32, device),
             _ptr(kv_lens, "kv_lens", f.i32, device), block_table.data_ptr()),
            batch, shape[1], shape[3], (shape[0], shape[2], width, stride, kind))


def _errors(f, errors, device):
    if errors is None:
        return None
    if errors.dtype not in (f.i32, f.u32) or errors.device != device or errors.numel() < 1:
        raise ValueError(f"errors must be an int32 or uint32 tensor on {device}")
    return errors.data_ptr()


def _copy(f, fn, what, k, v, k_cache, v_cache, k_scale, v_scale, query_start_loc, kv_lens,
          block_table, errors, stream):
    device = k_cache.device
    ptrs, batch, heads, dim, sizes = _cache(f, k_cache, v_cache, k_scale, v_scale,
                                            query_start_loc, kv_lens, block_table, device)
    if k.shape != v.shape or len(k.shape) != 3 or k.shape[1:] != (heads, dim):
        raise ValueError(f"k and v must both have shape (rows, {heads}, {dim})")
    pk, k_stride = _rows(k, "k", f, device)
    pv, v_stride = _rows(v, "v", f, device)
    s = f.current_stream(device) if stream is None else stream
    st = fn(pk, pv, *ptrs, k.shape[0], batch, heads, dim, *sizes, k_stride, v_stride,
            _errors(f, errors, device), s.cuda_stream)
    if st != SSD_OK:
        raise SSDError(st, what)


def ssd_kv_cache_write(k, v, k_cache, v_cache, k_scale, v_scale, query_start_loc, kv_lens,
                       block_table, *, errors=None, stream=None) -> None:
    """Write the new tokens' keys and values into the paged cache, quantised
    row by row when the cache is 8-bit.

    k, v (rows, nheads_kv, head_dim) bf16, each row contiguous, any row pitch
    that is a multiple of 8 elements; query_start_loc (batch + 1,) int32;
    kv_lens (batch,) int32, the tokens of each sequence with the new ones
    counted; block_table (batch, pages) int32.  errors: an int32 tensor of one
    element that collects the SSD_DEVERR_* flags, or None."""
    f = _functions()
    _copy(f, f.write, "ssd_kv_cache_write", k, v, k_cache, v_cache, k_scale, v_scale,
          query_start_loc, kv_lens, block_table, errors, stream)


def ssd_kv_cache_read(k, v, k_cache, v_cache, k_scale, v_scale, query_start_loc, kv_lens,
                      block_table, *, errors=None, stream=None) -> None:
    """Read cache rows back into k and v (bf16): row t gets the token that
    ssd_kv_cache_write would write from it.  Arguments as there; with
    query_start_loc the running sum of kv_lens it reads whole contexts."""
    f = _functions()
    _copy(f, f.read, "ssd_kv_cache_read", k, v, k_cache, v_cache, k_scale, v_scale,
          query_start_loc, kv_lens, block_table, errors, stream)


def ssd_attn_varlen_workspace_size(total_len: int, batch: int, nheads: int, nheads_kv: int,
                                   head_dim: int) -> int:
    return int(_functions().workspace_size(total_len, batch, nheads, nheads_kv, head_dim))


def alloc_attn_workspace(total_len: int, batch: int, nheads: int, nheads_kv: int, head_dim: int,
                         device="cuda"):
    """A uint8 torch tensor of the size the C ABI asks for; it serves every call
    of at most these sizes, whatever the contexts' lengths."""
    import torch
    n = ssd_attn_varlen_workspace_size(total_len, batch, nheads, nheads_kv, head_dim)
    if n == 0:
        raise SSDError(2, "ssd_attn_varlen_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def ssd_attn_varlen_fwd(o, lse, q, k_cache, v_cache, k_scale, v_scale, query_start_loc, kv_lens,
                        block_table, *, softmax_scale: float, window: int = 0, workspace=None,
                        errors=None, stream=None) -> None:
    """Causal grouped-query attention of the new tokens over the paged cache,
    which already holds them (ssd_kv_cache_write).

    o, q (rows, nheads, head_dim) bf16, each row contiguous, any row pitch that
    is a multiple of 8 elements; lse (rows, nheads) fp32 or None; the cache and
    the batch as for ssd_kv_cache_write; window 0 or the number of keys a query
    sees; workspace: a uint8 tensor of at least ssd_attn_varlen_workspace_size
    bytes (alloc_attn_workspace)."""
    f = _functions()
    device = k_cache.device
    ptrs, batch, heads_kv, dim, sizes = _cache(f, k_cache, v_cache, k_scale, v_scale,
                                               query_start_loc, kv_lens, block_table, device)
    if o.shape != q.shape or len(q.shape) != 3 or q.shape[2] != dim:
        raise ValueError(f"o and q must both have shape (rows, nheads, {dim})")
    total, heads = q.shape[0], q.shape[1]
    if workspace is None:
        raise ValueError("workspace is required (see alloc_attn_workspace)")
    plse = None
    if lse is not None:
        if lse.shape != (total, heads):
            raise ValueError(f"lse must have shape ({total}, {heads})")
        plse = _ptr(lse, "lse", f.f32, device)
    po, o_stride = _rows(o, "o", f, device)
    pq, q_stride = _rows(q, "q", f, device)
    s = f.current_stream(device) if stream is None else stream
    st = f.attn(po, plse, pq, *ptrs, total, batch, heads, heads_kv, dim, *sizes, o_stride, q_stride,
                softmax_scale, window, _ptr(workspace, "workspace", f.u8, device),
                workspace.numel(), _errors(f, errors, device), s.cuda_stream)
    if st != SSD_OK:
        raise SSDError(st, "ssd_attn_varlen_fwd")
