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
        # the current stream's handle alone, where torch has that (an order of
        # magnitude less time than a Stream object)
        self.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda device: torch.cuda.current_stream(device).cuda_stream)


def _functions() -> _Functions:
    global _fn
    if _fn is None:
        _fn = _Functions()
    return _fn


def _tensor(t, what: str, dtype, device: int, contiguous: bool = True):
    """Raise what is wrong with a tensor that should be of that type and device."""
    if t.dtype != dtype:
        raise ValueError(f"{what} must have dtype {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if t.get_device() != device:
        raise ValueError(f"{what} must be on device {device}, got {t.get_device()}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")


def _refuse(f, k_cache, v_cache, k_scale, v_scale, query_start_loc, kv_lens, block_table, errors):
    """Raise what is wrong with the arguments that all calls share."""
    if k_cache.dtype not in f.types:
        raise ValueError(f"k_cache must be bfloat16, float8_e4m3fn or int8, got {k_cache.dtype}")
    if not k_cache.is_cuda:
        raise ValueError("k_cache must be a CUDA tensor")
    device, shape = k_cache.get_device(), k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must both have shape "
                         "(num_pages, nheads_kv, page_size, head_dim)")
    _tensor(k_cache, "k_cache", k_cache.dtype, device)
    _tensor(v_cache, "v_cache", k_cache.dtype, device)
    if f.types[k_cache.dtype]:
        if k_scale is None or v_scale is None:
            raise ValueError("an 8-bit cache needs k_scale and v_scale")
        for t, what in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t.shape != shape[:3]:
                raise ValueError(f"{what} must have shape {tuple(shape[:3])}")
            _tensor(t, what, f.f32, device)
    elif k_scale is not None or v_scale is not None:
        raise ValueError("a bfloat16 cache has no scales")
    _tensor(query_start_loc, "query_start_loc", f.i32, device)
    _tensor(kv_lens, "kv_lens", f.i32, device)
    if query_start_loc.dim() != 1 or query_start_loc.shape[0] < 1:
        raise ValueError("query_start_loc must have shape (batch + 1,)")
    batch = query_start_loc.shape[0] - 1
    if kv_lens.shape != (batch,):
        raise ValueError(f"kv_lens must have shape ({batch},)")
    _tensor(block_table, "block_table", f.i32, device, contiguous=False)
    if block_table.dim() != 2 or block_table.shape[0] != batch:
        raise ValueError(f"block_table must have shape ({batch}, pages)")
    if block_table.shape[1] > 1 and block_table.stride(1) != 1:
        raise ValueError("block_table: each sequence's entries must be contiguous")
    if block_table.stride(0) < block_table.shape[1] and batch > 1:
        raise ValueError("block_table: sequences' rows must not overlap (an expanded table has to "
                         "be made contiguous)")
    if errors is not None:
        if errors.numel() < 1 or errors.dtype not in (f.i32, f.u32):
            raise ValueError("errors must be an int32 or uint32 tensor of one element")
        _tensor(errors, "errors", errors.dtype, device)
    raise ValueError("invalid arguments")


def _cache(f, k_cache, v_cache, k_scale, v_scale, query_start_loc, kv_lens, block_table, errors):
    """The arguments that all calls share: pointers, batch, nheads_kv, head_dim, sizes,
    the errors' pointer and the device.  One pass of cheap tests; what fails one
    is looked at again for its message."""
    shape, dtype, device, i32 = k_cache.shape, k_cache.dtype, k_cache.get_device(), f.i32
    kind = f.types.get(dtype)
    tshape, ks, vs, pe = block_table.shape, None, None, None
    good = (kind is not None and device >= 0 and len(shape) == 4 and v_cache.shape == shape
            and v_cache.dtype is dtype and v_cache.get_device() == device
            and k_cache.is_contiguous() and v_cache.is_contiguous()
            and query_start_loc.dtype is i32 and query_start_loc.get_device() == device
            and query_start_loc.is_contiguous()
            and kv_lens.dtype is i32 and kv_lens.get_device() == device and kv_lens.is_contiguous()
            and block_table.dtype is i32 and block_table.get_device() == device
            and len(tshape) == 2)
    if good:
        batch, width = tshape
        tstride = block_table.stride()
        good = (query_start_loc.shape == (batch + 1,) and kv_lens.shape == (batch,)
                and (tstride[1] == 1 or width <= 1) and (tstride[0] >= width or batch <= 1))
    if good and kind:
        if k_scale is None or v_scale is None:
            good = False
        else:
            ks, vs = k_scale.data_ptr(), v_scale.data_ptr()
            good = (k_scale.dtype is f.f32 and v_scale.dtype is f.f32
                    and k_scale.shape == shape[:3] and v_scale.shape == shape[:3]
                    and k_scale.get_device() == device and v_scale.get_device() == device
                    and k_scale.is_contiguous() and v_scale.is_contiguous())
    elif k_scale is not None or v_scale is not None:
        good = False
    if good and errors is not None:
        pe = errors.data_ptr()
        good = ((errors.dtype is i32 or errors.dtype is f.u32) and errors.get_device() == device
                and errors.numel() >= 1)
    if not good:
        _refuse(f, k_cache, v_cache, k_scale, v_scale, query_start_loc, kv_lens, block_table, errors)
    return ((k_cache.data_ptr(), v_cache.data_ptr(), ks, vs, query_start_loc.data_ptr(),
             kv_lens.data_ptr(), block_table.data_ptr()),
            batch, shape[1], shape[3],
            (shape[0], shape[2], width, tstride[0] if batch > 1 else width, kind), pe, device)


def _pitch(t, what: str, f, device: int):
    """Row pitch (elements) of a (rows, heads, head_dim) bf16 tensor whose rows are
    contiguous and do not overlap (an expanded tensor's do: its pitch of 0 would
    say "contiguous" in the C ABI)."""
    n, h, d = t.shape
    s = t.stride()
    if t.dtype is not f.bf16 or t.get_device() != device:
        _tensor(t, what, f.bf16, device, contiguous=False)
    if (s[2] != 1 and d != 1) or (s[1] != d and h != 1):
        raise ValueError(f"{what}: each token's row must be contiguous")
    if n <= 1:
        return h * d
    if s[0] < h * d:
        raise ValueError(f"{what}: tokens' rows must not overlap (an expanded tensor has to be "
                         "made contiguous)")
    return s[0]


def _copy(f, fn, what, k, v, k_cache, v_cache, k_scale, v_scale, query_start_loc, kv_lens,
          block_table, errors, stream):
    ptrs, batch, heads, dim, sizes, pe, device = _cache(f, k_cache, v_cache, k_scale, v_scale,
                                                        query_start_loc, kv_lens, block_table, errors)
    shape = k.shape
    if v.shape != shape or len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"k and v must both have shape (rows, {heads}, {dim})")
    st = fn(k.data_ptr(), v.data_ptr(), *ptrs, shape[0], batch, heads, dim, *sizes,
            _pitch(k, "k", f, device), _pitch(v, "v", f, device), pe,
            f.raw_stream(device) if stream is None else stream.cuda_stream)
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
    if not 0 <= window <= 0x7fffffff:    # (ctypes would cut it to 32 bits)
        raise ValueError(f"window must be in [0, 2^31), got {window}")
    f = _functions()
    ptrs, batch, heads_kv, dim, sizes, pe, device = _cache(f, k_cache, v_cache, k_scale, v_scale,
                                                           query_start_loc, kv_lens, block_table,
                                                           errors)
    shape = q.shape
    if o.shape != shape or len(shape) != 3 or shape[2] != dim:
        raise ValueError(f"o and q must both have shape (rows, nheads, {dim})")
    total, heads, _ = shape
    if workspace is None:
        raise ValueError("workspace is required (see alloc_attn_workspace)")
    if workspace.dtype is not f.u8 or workspace.get_device() != device \
            or not workspace.is_contiguous():
        _tensor(workspace, "workspace", f.u8, device)
    plse = None
    if lse is not None:
        if lse.shape != (total, heads):
            raise ValueError(f"lse must have shape ({total}, {heads})")
        if lse.dtype is not f.f32 or lse.get_device() != device or not lse.is_contiguous():
            _tensor(lse, "lse", f.f32, device)
        plse = lse.data_ptr()
    st = f.attn(o.data_ptr(), plse, q.data_ptr(), *ptrs, total, batch, heads, heads_kv, dim, *sizes,
                _pitch(o, "o", f, device), _pitch(q, "q", f, device), softmax_scale, window,
                workspace.data_ptr(), workspace.numel(), pe,
                f.raw_stream(device) if stream is None else stream.cuda_stream)
    if st != SSD_OK:
        raise SSDError(st, "ssd_attn_varlen_fwd")
