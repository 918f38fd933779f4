"""Python binding of the C ABI in include/ssd_layers.h (ctypes): the operators
around the scan and the attention in a hybrid model's layers.

Argument marshalling only, as in ``binding``: the work runs in the CUDA kernels
of libssd_scan.so on torch's current stream (or `stream`), and there is no CPU
fallback.  Calls run on the device of their tensors.
"""
from __future__ import annotations

import ctypes

import math

from . import attention, binding
from .binding import SSD_OK, SSDError

# Every symbol include/ssd_layers.h declares.
EXPORTED_SYMBOLS = (
    "ssd_causal_conv_varlen_fwd",
    "ssd_selective_scan_varlen_workspace_size",
    "ssd_selective_scan_varlen_fwd",
    "ssd_rms_norm_fwd",
    "ssd_rope_table",
    "ssd_rope_varlen_fwd",
    "ssd_rope_kv_cache_write",
)

NO_SLOT = 0xffffffff   # SSD_NO_SLOT (-1 in an int32 tensor of cache_indices)

_fn = None


class SelectiveStrides(ctypes.Structure):
    """ssd_selective_strides_t: elements between consecutive tokens (0: contiguous)."""
    _fields_ = [(n, ctypes.c_int64) for n in ("y", "x", "dt", "B", "C", "z")]


class _Functions:
    def __init__(self):
        import torch
        lib = binding.library()
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        self.conv = lib.ssd_causal_conv_varlen_fwd
        self.conv.restype = ctypes.c_int
        self.conv.argtypes = [vp] * 8 + [i64, i32, i32, i32, i64, i64, i64, i32, vp, vp]
        self.scan_workspace_size = lib.ssd_selective_scan_varlen_workspace_size
        self.scan_workspace_size.restype = sz
        self.scan_workspace_size.argtypes = [i64, i32, i32, i32]
        self.scan = lib.ssd_selective_scan_varlen_fwd
        self.scan.restype = ctypes.c_int
        self.scan.argtypes = ([vp] * 13 + [i64, i32, i32, i32, i64, i32, i32]
                              + [ctypes.POINTER(SelectiveStrides), vp, sz, vp, vp])
        self.norm = lib.ssd_rms_norm_fwd
        self.norm.restype = ctypes.c_int
        self.norm.argtypes = [vp] * 6 + [i64, i32, i32, i32, ctypes.c_float] + [i64] * 4 + [vp]
        self.rope_table = lib.ssd_rope_table
        self.rope_table.restype = ctypes.c_int
        self.rope_table.argtypes = [vp, vp, i32]
        # total_len, batch, nheads, nheads_kv, head_dim, rotary_dim, interleaved, magnitude
        rotary = [i64, i32, i32, i32, i32, i32, i32, ctypes.c_float]
        self.rope = lib.ssd_rope_varlen_fwd
        self.rope.restype = ctypes.c_int
        self.rope.argtypes = [vp] * 7 + rotary + [i64] * 4 + [vp, vp]
        self.rope_write = lib.ssd_rope_kv_cache_write
        self.rope_write.restype = ctypes.c_int
        self.rope_write.argtypes = ([vp] * 12 + rotary + [i64, i32, i32, i64, i32] + [i64] * 4 + [vp, vp])
        self.types = {torch.bfloat16: 0, torch.float8_e4m3fn: 1, torch.int8: 2}
        self.bf16, self.f32, self.i32, self.u32 = torch.bfloat16, torch.float32, torch.int32, torch.uint32
        self.u8, self.bool, self.i64 = torch.uint8, torch.bool, torch.int64
        # the current stream's handle alone, where torch has that (an order of
        # magnitude less time than a Stream object)
        self.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda device: torch.cuda.current_stream(device).cuda_stream)
        self.current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _functions() -> _Functions:
    global _fn
    if _fn is None:
        _fn = _Functions()
    return _fn


def _call(f, fn, what: str, device: int, stream, *args):
    """Call into the library on the tensors' device and stream."""
    if f.current_device() != device:
        import torch
        with torch.cuda.device(device):
            return _call(f, fn, what, device, stream, *args)
    st = fn(*args, f.raw_stream(device) if stream is None else stream.cuda_stream)
    if st != SSD_OK:
        raise SSDError(st, what)


def _device(t, what: str) -> int:
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    return t.get_device()


def _ptr(t, what: str, dtype, shape, device: int):
    """Pointer of a contiguous tensor of exactly that type and shape."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == device:
        return t.data_ptr()
    if t.dtype is not dtype:
        raise ValueError(f"{what} must have dtype {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    raise ValueError(f"{what} must be on device {device}, got {t.device}")


def _rows(t, what: str, dtype, shape, device: int):
    """Pointer and row pitch (elements; 0: contiguous) of a token-major tensor whose rows
    are contiguous and do not overlap (an expanded tensor's do: its pitch of 0 would
    say "contiguous" in the C ABI)."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == device:
        return t.data_ptr(), 0
    if t.dtype is not dtype:
        raise ValueError(f"{what} must have dtype {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{what} must be on device {device}, got {t.device}")
    row = 1
    stride = t.stride()
    for d in range(len(shape) - 1, 0, -1):
        if stride[d] != row and shape[d] != 1:
            raise ValueError(f"{what}: each token's row must be contiguous")
        row *= shape[d]
    if shape[0] <= 1:
        return t.data_ptr(), 0
    if stride[0] < row:
        raise ValueError(f"{what}: tokens' rows must not overlap (an expanded tensor has to be "
                         "made contiguous)")
    return t.data_ptr(), stride[0]


def _errors(f, errors, device: int):
    if errors is None:
        return None
    if (errors.dtype is not f.i32 and errors.dtype is not f.u32) or errors.numel() < 1:
        raise ValueError("errors must be an int32 or uint32 tensor of one element")
    if errors.get_device() != device:
        raise ValueError(f"errors must be on device {device}, got {errors.device}")
    return errors.data_ptr()


def _slots(f, query_start_loc, has_initial_state, cache_indices, device: int):
    """Pointers of the batch and its slots, and the batch size."""
    if query_start_loc.dim() != 1 or query_start_loc.shape[0] < 1:
        raise ValueError("query_start_loc must have shape (batch + 1,)")
    batch = query_start_loc.shape[0] - 1
    has = None
    if has_initial_state is not None:
        has = _ptr(has_initial_state, "has_initial_state",
                   f.bool if has_initial_state.dtype is f.bool else f.u8, (batch,), device)
    return (_ptr(query_start_loc, "query_start_loc", f.i32, (batch + 1,), device), has,
            _ptr(cache_indices, "cache_indices", f.u32 if cache_indices.dtype is f.u32 else f.i32,
                 (batch,), device)), batch


def _slots_fast(f, query_start_loc, has_initial_state, cache_indices, errors, device: int):
    """Pointers of the batch, its slots and the errors, and the batch size; None where
    anything is not as it should be (_slots and _errors say what).  One pass of cheap
    tests: a step's calls are short."""
    shape, dtype = query_start_loc.shape, cache_indices.dtype
    if (len(shape) != 1 or shape[0] < 1 or query_start_loc.dtype is not f.i32
            or query_start_loc.get_device() != device or not query_start_loc.is_contiguous()
            or cache_indices.shape != (shape[0] - 1,) or (dtype is not f.i32 and dtype is not f.u32)
            or cache_indices.get_device() != device or not cache_indices.is_contiguous()):
        return None, 0
    batch, has, pe = shape[0] - 1, None, None
    if has_initial_state is not None:
        dtype = has_initial_state.dtype
        if (has_initial_state.shape != (batch,) or (dtype is not f.bool and dtype is not f.u8)
                or has_initial_state.get_device() != device or not has_initial_state.is_contiguous()):
            return None, 0
        has = has_initial_state.data_ptr()
    if errors is not None:
        dtype = errors.dtype
        if (dtype is not f.i32 and dtype is not f.u32) or errors.get_device() != device or errors.numel() < 1:
            return None, 0
        pe = errors.data_ptr()
    return (query_start_loc.data_ptr(), has, cache_indices.data_ptr(), pe), batch


def _vector(f, t, n: int, device: int) -> bool:
    return t.dtype is f.f32 and t.shape == (n,) and t.get_device() == device and t.is_contiguous()


def ssd_causal_conv_varlen_fwd(y, x, weight, bias, conv_pool, query_start_loc, has_initial_state,
                               cache_indices, *, silu: bool = True, errors=None, stream=None) -> None:
    """The short causal convolution of every channel, for prompts and single tokens,
    with the last inputs of every sequence kept in a pool of slots.

    y, x (rows, channels) bf16, each row contiguous, any row pitch that is a
    multiple of 8 elements; weight (channels, width) fp32, width 2 to 4; bias
    (channels,) fp32 or None; conv_pool (slots, width - 1, channels) bf16, updated
    in place; query_start_loc (batch + 1,) int32; has_initial_state (batch,)
    uint8/bool or None; cache_indices (batch,) int32/uint32 (same bits; -1 is no
    slot); silu: y is silu of the sum; y must not overlap x.  errors: an int32 tensor of one
    element that collects the SSD_DEVERR_* flags, or None."""
    f = _functions()
    shape, wshape, bf16, f32 = x.shape, weight.shape, f.bf16, f.f32
    device = x.get_device()
    if len(shape) == 2 and len(wshape) == 2 and conv_pool.dim() == 3 and device >= 0:
        total, channels = shape
        width, max_slots = wshape[1], conv_pool.shape[0]
        where, batch = _slots_fast(f, query_start_loc, has_initial_state, cache_indices, errors, device)
        if (where is not None and x.dtype is bf16 and y.dtype is bf16 and y.shape == shape
                and y.get_device() == device and x.is_contiguous() and y.is_contiguous()
                and weight.dtype is f32 and wshape[0] == channels and weight.get_device() == device
                and weight.is_contiguous() and conv_pool.dtype is bf16
                and conv_pool.shape == (max_slots, width - 1, channels)
                and conv_pool.get_device() == device and conv_pool.is_contiguous()
                and (bias is None or _vector(f, bias, channels, device))):
            return _call(f, f.conv, "ssd_causal_conv_varlen_fwd", device, stream, y.data_ptr(), x.data_ptr(),
                         weight.data_ptr(), None if bias is None else bias.data_ptr(), conv_pool.data_ptr(),
                         *where[:3], total, batch, channels, width, max_slots, 0, 0, bool(silu), where[3])
    # rows with a pitch of their own, or something is wrong
    device = _device(x, "x")
    if x.dim() != 2 or weight.dim() != 2 or conv_pool.dim() != 3:
        raise ValueError("x must have shape (rows, channels), weight (channels, width) and conv_pool "
                         "(slots, width - 1, channels)")
    total, channels = shape
    width = weight.shape[1]
    slots, batch = _slots(f, query_start_loc, has_initial_state, cache_indices, device)
    py, sy = _rows(y, "y", f.bf16, shape, device)
    px, sx = _rows(x, "x", f.bf16, shape, device)
    max_slots = conv_pool.shape[0]
    _call(f, f.conv, "ssd_causal_conv_varlen_fwd", device, stream,
          py, px, _ptr(weight, "weight", f.f32, (channels, width), device),
          None if bias is None else _ptr(bias, "bias", f.f32, (channels,), device),
          _ptr(conv_pool, "conv_pool", f.bf16, (max_slots, width - 1, channels), device),
          *slots, total, batch, channels, width, max_slots, sy, sx, bool(silu),
          _errors(f, errors, device))


def ssd_selective_scan_varlen_workspace_size(total_len: int, batch: int, channels: int, dstate: int) -> int:
    return int(_functions().scan_workspace_size(total_len, batch, channels, dstate))


def alloc_selective_scan_workspace(total_len: int, batch: int, channels: int, dstate: int, device="cuda"):
    """A uint8 torch tensor of the size the C ABI asks for; it serves every call of at
    most these sizes."""
    import torch
    n = ssd_selective_scan_varlen_workspace_size(total_len, batch, channels, dstate)
    if n == 0:
        raise SSDError(2, "ssd_selective_scan_varlen_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def ssd_selective_scan_varlen_fwd(y, x, dt, A, B, C, D, z, dt_bias, ssm_pool, query_start_loc,
                                  has_initial_state, cache_indices, *, dt_softplus: bool = True,
                                  workspace=None, errors=None, stream=None) -> None:
    """The selective scan whose step and decay are each channel's own, for prompts and
    single tokens.

    y, x, dt (rows, channels) and z (the gate) likewise or None, B, C (rows, dstate) bf16,
    each row contiguous, any row pitch that is a multiple of 8 elements; A (channels,
    dstate) fp32; D, dt_bias (channels,) fp32 or None; ssm_pool (slots, channels, dstate)
    fp32 or bf16, updated in place; the batch and errors as for
    ssd_causal_conv_varlen_fwd; y must not overlap another tensor; workspace: a uint8 tensor of
    at least ssd_selective_scan_varlen_workspace_size bytes (alloc_selective_scan_workspace)."""
    f = _functions()
    if workspace is None:
        raise ValueError("workspace is required (see alloc_selective_scan_workspace)")
    shape, ashape, bf16, f32 = x.shape, A.shape, f.bf16, f.f32
    device = x.get_device()
    if len(shape) == 2 and len(ashape) == 2 and ssm_pool.dim() == 3 and device >= 0:
        total, channels = shape
        dstate, max_slots, kind = ashape[1], ssm_pool.shape[0], ssm_pool.dtype
        bc = (total, dstate)
        where, batch = _slots_fast(f, query_start_loc, has_initial_state, cache_indices, errors, device)
        if (where is not None and x.dtype is bf16 and y.dtype is bf16 and dt.dtype is bf16 and B.dtype is bf16
                and C.dtype is bf16 and A.dtype is f32 and y.shape == shape and dt.shape == shape
                and B.shape == bc and C.shape == bc and ashape[0] == channels
                and y.get_device() == device and dt.get_device() == device and A.get_device() == device
                and B.get_device() == device and C.get_device() == device
                and x.is_contiguous() and y.is_contiguous() and dt.is_contiguous() and A.is_contiguous()
                and B.is_contiguous() and C.is_contiguous()
                and (z is None or (z.dtype is bf16 and z.shape == shape and z.get_device() == device
                                   and z.is_contiguous()))
                and (D is None or _vector(f, D, channels, device))
                and (dt_bias is None or _vector(f, dt_bias, channels, device))
                and (kind is f32 or kind is bf16) and ssm_pool.shape == (max_slots, channels, dstate)
                and ssm_pool.get_device() == device and ssm_pool.is_contiguous()
                and workspace.dtype is f.u8 and workspace.get_device() == device and workspace.is_contiguous()):
            return _call(f, f.scan, "ssd_selective_scan_varlen_fwd", device, stream, y.data_ptr(), x.data_ptr(),
                         dt.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(),
                         None if D is None else D.data_ptr(), None if z is None else z.data_ptr(),
                         None if dt_bias is None else dt_bias.data_ptr(), ssm_pool.data_ptr(), *where[:3], total,
                         batch, channels, dstate, max_slots, kind is bf16, bool(dt_softplus), None,
                         workspace.data_ptr(), workspace.numel(), where[3])
    # rows with a pitch of their own, or something is wrong
    device = _device(x, "x")
    if x.dim() != 2 or A.dim() != 2 or ssm_pool.dim() != 3:
        raise ValueError("x must have shape (rows, channels), A (channels, dstate) and ssm_pool "
                         "(slots, channels, dstate)")
    total, channels = shape
    dstate = A.shape[1]
    slots, batch = _slots(f, query_start_loc, has_initial_state, cache_indices, device)
    py, sy = _rows(y, "y", f.bf16, shape, device)
    px, sx = _rows(x, "x", f.bf16, shape, device)
    pd, sd = _rows(dt, "dt", f.bf16, shape, device)
    pb, sb = _rows(B, "B", f.bf16, (total, dstate), device)
    pc, sc = _rows(C, "C", f.bf16, (total, dstate), device)
    pz, sz = (None, 0) if z is None else _rows(z, "z", f.bf16, shape, device)
    max_slots, narrow = ssm_pool.shape[0], ssm_pool.dtype is f.bf16
    _call(f, f.scan, "ssd_selective_scan_varlen_fwd", device, stream, py, px, pd,
          _ptr(A, "A", f.f32, (channels, dstate), device), pb, pc,
          None if D is None else _ptr(D, "D", f.f32, (channels,), device), pz,
          None if dt_bias is None else _ptr(dt_bias, "dt_bias", f.f32, (channels,), device),
          _ptr(ssm_pool, "ssm_pool", f.bf16 if narrow else f.f32, (max_slots, channels, dstate), device),
          *slots, total, batch, channels, dstate, max_slots, narrow, bool(dt_softplus),
          ctypes.byref(SelectiveStrides(sy, sx, sd, sb, sc, sz)),
          _ptr(workspace, "workspace", f.u8, (workspace.numel(),), device), workspace.numel(),
          _errors(f, errors, device))


def ssd_rms_norm_fwd(y, x, weight, *, residual=None, gate=None, scale=None, ngroups: int = 1,
                     eps: float = 1e-5, stream=None) -> None:
    """Root-mean-square norm over each row's groups of dim / ngroups columns, of
    x, of x + residual (updated in place) or of x silu(gate).

    x, residual, gate (rows, dim) bf16, each row contiguous, any row pitch that is a
    multiple of 8 elements; weight (dim,) fp32 or None; y (rows, dim) bf16 (it may
    be x or gate), or float8_e4m3fn or int8 codes with scale (rows, ngroups) fp32; eps
    from 2^-80 to 1."""
    f = _functions()
    device = _device(x, "x")
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("x must have shape (rows, dim)")
    rows, dim = shape
    kind = f.types.get(y.dtype)
    if kind is None:
        raise ValueError(f"y must be bfloat16, float8_e4m3fn or int8, got {y.dtype}")
    if (kind != 0) != (scale is not None):
        raise ValueError("8-bit codes need a scale" if kind else "a bfloat16 output has no scale")
    if ngroups < 1 or dim % ngroups:
        raise ValueError(f"ngroups must divide {dim}, got {ngroups}")
    py, sy = _rows(y, "y", y.dtype, shape, device)
    px, sx = _rows(x, "x", f.bf16, shape, device)
    pr, sr = (None, 0) if residual is None else _rows(residual, "residual", f.bf16, shape, device)
    pg, sg = (None, 0) if gate is None else _rows(gate, "gate", f.bf16, shape, device)
    _call(f, f.norm, "ssd_rms_norm_fwd", device, stream, py,
          None if scale is None else _ptr(scale, "scale", f.f32, (rows, ngroups), device), px, pr, pg,
          None if weight is None else _ptr(weight, "weight", f.f32, (dim,), device),
          rows, dim, ngroups, kind, eps, sy, sx, sr, sg)


def rope_frequencies(rotary_dim: int, base: float = 10000.0, *, scaling: str = "none", factor: float = 1.0,
                     original_len: int = 8192, low_turns: float = 1.0, high_turns: float = 32.0):
    """Frequencies (radians per position, rotary_dim / 2 of them, in 64 bits) and the
    magnitude for alloc_rope_table and the rotary calls.

    f_i = base^(-2 i / rotary_dim), for contexts `factor` times original_len changed by
    `scaling`:

      "none"        as they are
      "linear"      all divided by factor
      "base"        the base times factor^(rotary_dim / (rotary_dim - 2)): the highest stays,
                    the lowest is divided by factor
      "ramp"        divided where a pair makes at most low_turns turns in original_len
                    positions, kept from high_turns on, blended linearly in the pair's
                    index between (from whole index to whole index, outwards, within 0 and
                    rotary_dim - 1: the ramp may end behind the last pair); magnitude
                    0.1 ln(factor) + 1
      "wavelength"  the same blended linearly in the number of turns; magnitude 1"""
    if rotary_dim < 4 or rotary_dim % 2:
        raise ValueError(f"rotary_dim must be even and at least 4, got {rotary_dim}")
    if not (base > 1.0 and math.isfinite(base) and factor >= 1.0 and math.isfinite(factor)):
        raise ValueError("base must be above 1 and factor at least 1")
    half = rotary_dim // 2
    if scaling == "base":
        base *= factor ** (rotary_dim / (rotary_dim - 2))
    f = [base ** (-i / half) for i in range(half)]
    if scaling in ("none", "base"):
        return f, 1.0
    if scaling == "linear":
        return [x / factor for x in f], 1.0
    if scaling not in ("ramp", "wavelength"):
        raise ValueError(f"scaling must be none, linear, base, ramp or wavelength, got {scaling!r}")
    if not 0.0 < low_turns < high_turns or original_len < 1:
        raise ValueError("0 < low_turns < high_turns and original_len >= 1 are needed")
    if scaling == "ramp":
        def pair_of(turns):    # the (fractional) pair that makes so many turns in original_len positions
            return half * math.log(original_len / (turns * 2 * math.pi)) / math.log(base)
        low = max(math.floor(pair_of(high_turns)), 0)
        high = min(math.ceil(pair_of(low_turns)), rotary_dim - 1)
        # (high <= 0: even the first pair makes at most low_turns)
        keep = [1.0 - min(max((i - low) / max(high - low, 0.001), 0.0), 1.0) if high > 0 else 0.0
                for i in range(half)]
    else:
        keep = [min(max((x * original_len / (2 * math.pi) - low_turns) / (high_turns - low_turns), 0.0), 1.0)
                for x in f]
    return ([x / factor * (1.0 - k) + x * k for x, k in zip(f, keep)],
            0.1 * math.log(factor) + 1.0 if scaling == "ramp" else 1.0)


def alloc_rope_table(frequencies, device="cuda"):
    """The table of turns that the rotary calls take: an int64 tensor of one element per
    frequency (the bits of the C ABI's uint64)."""
    import torch
    values = [float(x) for x in frequencies]
    if not values:
        raise ValueError("at least one frequency is needed")
    turns = (ctypes.c_uint64 * len(values))()
    st = _functions().rope_table(turns, (ctypes.c_double * len(values))(*values), len(values))
    if st != SSD_OK:
        raise SSDError(st, "ssd_rope_table")
    return torch.tensor([t - (1 << 64) if t >> 63 else t for t in turns], dtype=torch.int64, device=device)


def _rotary(f, table, device: int):
    shape = table.shape
    if len(shape) != 1:
        raise ValueError("table must have shape (rotary_dim / 2,)")
    return _ptr(table, "table", f.i64, shape, device), 2 * shape[0]


def _same_rows(out, x, what: str, f, shape, device: int):
    """Pointers and pitches of an output and its input, of shape (rows, heads, head_dim)."""
    bf16 = f.bf16
    if (out.dtype is bf16 and x.dtype is bf16 and out.shape == shape and out.get_device() == device
            and x.get_device() == device and out.is_contiguous() and x.is_contiguous()):
        return out.data_ptr(), 0, x.data_ptr(), 0
    return *_rows(out, f"{what}_out", bf16, shape, device), *_rows(x, what, bf16, shape, device)


def ssd_rope_varlen_fwd(q_out, q, k_out, k, table, query_start_loc, kv_lens, *, interleaved: bool = False,
                        magnitude: float = 1.0, errors=None, stream=None) -> None:
    """Rotate the new tokens' queries and keys by their positions (k and k_out may
    both be None, or q and q_out).

    q_out, q (rows, nheads, head_dim) and k_out, k (rows, nheads_kv, head_dim) bf16, each
    row contiguous, any row pitch that is a multiple of 8 elements, an output may be
    its input; table: alloc_rope_table's, of rotary_dim / 2 pairs; query_start_loc
    (batch + 1,) and kv_lens (batch,) int32 as for ssd_kv_cache_write; interleaved: pairs
    of neighbours and not of halves."""
    f = _functions()
    if (q is None) != (q_out is None) or (k is None) != (k_out is None) or (q is None and k is None):
        raise ValueError("q and q_out, or k and k_out, or both are needed")
    device = _device(k if q is None else q, "k" if q is None else "q")
    turns, rotary_dim = _rotary(f, table, device)
    if query_start_loc.dim() != 1 or query_start_loc.shape[0] < 1:
        raise ValueError("query_start_loc must have shape (batch + 1,)")
    batch = query_start_loc.shape[0] - 1
    qo = qi = ko = ki = None
    sqo = sq = sko = sk = heads = heads_kv = 0
    for t, what in ((q, "q"), (k, "k")):
        if t is not None and t.dim() != 3:
            raise ValueError(f"{what} must have shape (rows, heads, head_dim)")
    if q is not None:
        total, heads, dim = q.shape
        qo, sqo, qi, sq = _same_rows(q_out, q, "q", f, q.shape, device)
    if k is not None:
        shape = k.shape
        if q is not None and (shape[0] != total or shape[2] != dim):
            raise ValueError(f"k must have shape ({total}, nheads_kv, {dim}), got {tuple(shape)}")
        total, heads_kv, dim = shape
        ko, sko, ki, sk = _same_rows(k_out, k, "k", f, shape, device)
    _call(f, f.rope, "ssd_rope_varlen_fwd", device, stream, qo, qi, ko, ki, turns,
          _ptr(query_start_loc, "query_start_loc", f.i32, (batch + 1,), device),
          _ptr(kv_lens, "kv_lens", f.i32, (batch,), device), total, batch, heads, heads_kv, dim, rotary_dim,
          bool(interleaved), magnitude, sqo, sq, sko, sk, _errors(f, errors, device))


def ssd_rope_kv_cache_write(q_out, q, k, v, table, k_cache, v_cache, k_scale, v_scale, query_start_loc,
                            kv_lens, block_table, *, interleaved: bool = False, magnitude: float = 1.0,
                            errors=None, stream=None) -> None:
    """Rotate the new tokens' queries into q_out, and write their rotated keys and their
    values into the paged cache, in one launch: ssd_rope_varlen_fwd and
    ssd_kv_cache_write, with their arguments."""
    f = _functions()
    ptrs, batch, heads_kv, dim, sizes, pe, device = attention._cache(
        attention._functions(), k_cache, v_cache, k_scale, v_scale, query_start_loc, kv_lens, block_table,
        errors)
    turns, rotary_dim = _rotary(f, table, device)
    shape = q.shape
    if len(shape) != 3 or shape[2] != dim:
        raise ValueError(f"q must have shape (rows, nheads, {dim}), got {tuple(shape)}")
    total, heads, _ = shape
    qo, sqo, qi, sq = _same_rows(q_out, q, "q", f, shape, device)
    kv = (total, heads_kv, dim)
    pk, sk = _rows(k, "k", f.bf16, kv, device)
    pv, sv = _rows(v, "v", f.bf16, kv, device)
    _call(f, f.rope_write, "ssd_rope_kv_cache_write", device, stream, qo, qi, pk, pv, turns, *ptrs, total,
          batch, heads, heads_kv, dim, rotary_dim, bool(interleaved), magnitude, *sizes, sqo, sq, sk, sv, pe)
