"""Python binding of libsgemv.so: argument marshalling only.

Every step of the GEMV runs in the HIP library; this module converts torch
tensors and NumPy arrays to pointers and sizes, passes the current HIP
stream, and turns status codes into exceptions.  PyTorch is used for device
memory and streams only.  The names match the C entry points.
"""
from __future__ import annotations

import ctypes
import os
import struct

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libsgemv.so")

SGEMV_OK = 0
SGEMV_EINVAL = -1
SGEMV_ESIZE = -2
SGEMV_EALIGN = -3
SGEMV_EUNSUPPORTED = -4
SGEMV_EHIP = -5
SGEMV_OUT_F32 = 1
SGEMV_GROUP = 128
SGEMV_TILE_N = 512
SGEMV_LAYOUT_PAIRS = 1    # layout version 1: (s, z) fp16 pairs
SGEMV_LAYOUT_Z4 = 2       # layout version 2: fp16 scales, 4-bit zero-points
SGEMV_LAYOUT_NG = 3       # layout version 3: groups along N, (s, z) per column and 128 outputs
SGEMV_MAX_BATCH = 16
SGEMV_MAX_K = 65536
SGEMV_MAX_N = 1 << 20
SGEMV_F16, SGEMV_BF16, SGEMV_F32 = 0, 1, 2
SGEMV_ACT_SILU, SGEMV_ACT_GELU, SGEMV_ACT_RELU = 0, 1, 2
SGEMV_Q4_GATED, SGEMV_Q4_ZEROS, SGEMV_Q4_BF16_SCALES = 1, 2, 4
SGEMV_NORM_POST, SGEMV_NORM_CENTER, SGEMV_NORM_PLUS_ONE = 1, 2, 4
SGEMV_E4M3 = 3
SGEMV_ROTARY_ADJACENT, SGEMV_ROTARY_STRIPED = 1, 2
SGEMV_MAX_HEADS, SGEMV_MAX_DIM, SGEMV_MAX_AXES = 1024, 256, 4
SGEMV_MAX_BEAMS, SGEMV_MAX_CHOICES = 32, 64
SGEMV_MAX_LAYERS, SGEMV_MAX_ROWS = 128, 8192

EXPORTED = ["sgemv_pack_layout", "sgemv_pack_layout_z4", "sgemv_pack_layout_ng", "sgemv_pack_layout_parts",
            "sgemv_desc_from_header",
            "sgemv_gather_indices",
            "sgemv_run", "sgemv_run_batched", "sgemv_run_fused", "sgemv_run_fused_static", "sgemv_workspace_bytes",
            "sgemv_q4_pack", "sgemv_q4_pack_gated", "sgemv_q4_pack_device",
            "sgemv_q4_desc_from_header", "sgemv_q4_run", "sgemv_q4_run_gated",
            "sgemv_block_norm",
            "sgemv_rotary", "sgemv_attn_paged", "sgemv_attn_workspace_bytes",
            "sgemv_beam_select", "sgemv_beam_workspace_bytes",
            "sgemv_pages_fork", "sgemv_pages_compact", "sgemv_pages_copy", "sgemv_pages_workspace_bytes",
            "sgemv_strerror", "sgemv_last_hip_error"]


class SgemvError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {strerror(status)} ({status})")


class Desc(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int32), ("K", ctypes.c_int32), ("group", ctypes.c_int32),
                ("tile_n", ctypes.c_int32), ("w_off", ctypes.c_uint64),
                ("w_bytes", ctypes.c_uint64), ("m_off", ctypes.c_uint64),
                ("m_bytes", ctypes.c_uint64), ("total_bytes", ctypes.c_uint64),
                ("version", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]

    def as_dict(self) -> dict:
        return {f: getattr(self, f) for f, _ in self._fields_}


class Q4Desc(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int32), ("K", ctypes.c_int32), ("group", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("w_off", ctypes.c_uint64), ("w_bytes", ctypes.c_uint64),
                ("s_off", ctypes.c_uint64), ("s_bytes", ctypes.c_uint64), ("z_off", ctypes.c_uint64),
                ("z_bytes", ctypes.c_uint64), ("total_bytes", ctypes.c_uint64)]

    def as_dict(self) -> dict:
        return {f: getattr(self, f) for f, _ in self._fields_}


_lib = None


def lib():
    """Load libsgemv.so; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -c 'import __graft_entry__ as g; g.build()'`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, u32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint32, ctypes.c_size_t
    pd = ctypes.POINTER(Desc)
    L.sgemv_pack_layout.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp, sz, pd]
    L.sgemv_pack_layout.restype = ctypes.c_int
    L.sgemv_pack_layout_z4.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp, sz, pd]
    L.sgemv_pack_layout_z4.restype = ctypes.c_int
    L.sgemv_pack_layout_ng.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp, sz, pd]
    L.sgemv_pack_layout_ng.restype = ctypes.c_int
    L.sgemv_pack_layout_parts.argtypes = [i32, vp, vp, vp, vp, i32, i32, i32, u32, vp, sz, pd]
    L.sgemv_pack_layout_parts.restype = ctypes.c_int
    L.sgemv_desc_from_header.argtypes = [vp, sz, pd]
    L.sgemv_desc_from_header.restype = ctypes.c_int
    L.sgemv_gather_indices.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp]
    L.sgemv_gather_indices.restype = ctypes.c_int
    L.sgemv_run.argtypes = [pd, vp, vp, vp, vp, vp, u32, vp, vp]
    L.sgemv_run.restype = ctypes.c_int
    L.sgemv_run_batched.argtypes = [pd, vp, vp, i32, i32, vp, vp, vp, vp, i32, u32, vp, vp]
    L.sgemv_run_batched.restype = ctypes.c_int
    L.sgemv_run_fused.argtypes = [pd, vp, vp, i32, i32, vp, vp, vp, vp, i32, u32, vp, vp]
    L.sgemv_run_fused.restype = ctypes.c_int
    L.sgemv_run_fused_static.argtypes = [pd, vp, vp, i32, i32, vp, vp, vp, vp, i32, u32, vp]
    L.sgemv_run_fused_static.restype = ctypes.c_int
    L.sgemv_workspace_bytes.argtypes = [pd, i32]
    L.sgemv_workspace_bytes.restype = sz
    pq = ctypes.POINTER(Q4Desc)
    L.sgemv_q4_pack.argtypes = [vp, vp, vp, i32, i32, i32, u32, vp, sz, pq]
    L.sgemv_q4_pack.restype = ctypes.c_int
    L.sgemv_q4_pack_gated.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, u32, vp, sz, pq]
    L.sgemv_q4_pack_gated.restype = ctypes.c_int
    L.sgemv_q4_pack_device.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, u32, vp, sz, pq, vp]
    L.sgemv_q4_pack_device.restype = ctypes.c_int
    L.sgemv_q4_desc_from_header.argtypes = [vp, sz, pq]
    L.sgemv_q4_desc_from_header.restype = ctypes.c_int
    L.sgemv_q4_run.argtypes = [pq, vp, vp, i32, i32, i32, vp, vp, i32, i32, vp]
    L.sgemv_q4_run.restype = ctypes.c_int
    L.sgemv_q4_run_gated.argtypes = [pq, vp, vp, i32, i32, i32, vp, vp, i32, vp, i32, i32, vp]
    L.sgemv_q4_run_gated.restype = ctypes.c_int
    L.sgemv_block_norm.argtypes = [ctypes.c_char_p, vp]
    L.sgemv_block_norm.restype = ctypes.c_int
    raw = ctypes.c_char_p   # a packed struct
    for name in ("sgemv_rotary", "sgemv_attn_paged", "sgemv_pages_fork", "sgemv_pages_compact"):
        getattr(L, name).argtypes = [raw, raw, vp]
        getattr(L, name).restype = ctypes.c_int
    L.sgemv_beam_select.argtypes = [raw, vp]
    L.sgemv_beam_select.restype = ctypes.c_int
    L.sgemv_pages_copy.argtypes = [raw, i32, vp, vp, i32, vp]
    L.sgemv_pages_copy.restype = ctypes.c_int
    for name, n in (("sgemv_attn_workspace_bytes", 4), ("sgemv_beam_workspace_bytes", 4),
                    ("sgemv_pages_workspace_bytes", 3)):
        getattr(L, name).argtypes = [i32] * n
        getattr(L, name).restype = sz
    L.sgemv_strerror.argtypes = [ctypes.c_int]
    L.sgemv_strerror.restype = ctypes.c_char_p
    L.sgemv_last_hip_error.argtypes = []
    L.sgemv_last_hip_error.restype = ctypes.c_int
    _lib = L
    return L


def strerror(status: int) -> str:
    return lib().sgemv_strerror(int(status)).decode()


def _check(status: int, what: str):
    if status != SGEMV_OK:
        raise SgemvError(status, what)


def _ptr(t):
    """Address of a torch tensor, a NumPy array, or None."""
    if t is None:
        return None
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    import torch
    return torch.cuda.current_stream().cuda_stream


def _require(t, what: str, dtypes, min_numel: int, rows: int | None = None):
    """Check a device buffer before its address crosses the ABI: a torch
    tensor of one of `dtypes` holding at least `min_numel` elements, its last
    dimension contiguous (and, for `rows`, 1-D or 2-D with that many rows),
    (the device is checked by _require_gpu, after every other check of a
    call).  A plain integer is taken as a raw device address and passed
    through unchecked.  Raises ValueError on the first failed check, before
    any library call."""
    if isinstance(t, int):
        return
    import torch
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{what}: expected a torch tensor, got {type(t).__name__}")
    if t.dtype not in dtypes:
        names = ", ".join(str(d).replace("torch.", "") for d in dtypes)
        raise ValueError(f"{what}: dtype {str(t.dtype).replace('torch.', '')}, expected {names}")
    if rows is not None:
        if t.dim() not in (1, 2) or (t.dim() == 2 and t.shape[0] != rows) or (t.dim() == 1 and rows != 1):
            raise ValueError(f"{what}: shape {tuple(t.shape)}, expected [{rows}][...] rows")
    if t.dim() >= 1 and t.numel() > 0 and t.stride(-1) != 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    if t.dim() == 2 and t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{what}: rows overlap (stride {t.stride(0)} < {t.shape[1]})")
    if rows is None and t.dim() > 1 and not t.is_contiguous():
        raise ValueError(f"{what}: must be contiguous")
    if t.numel() < min_numel:
        raise ValueError(f"{what}: {t.numel()} elements, at least {min_numel} needed")


def _require_gpu(**bufs):
    """Every tensor among `bufs` (name=tensor; None and raw addresses are
    skipped) lives on a GPU."""
    import torch
    for what, t in bufs.items():
        if isinstance(t, torch.Tensor) and not t.is_cuda:
            raise ValueError(f"{what}: must be a GPU tensor")


def _f16():
    import torch
    return (torch.float16,)


def _i32():
    import torch
    return (torch.int32,)


def _u8():
    import torch
    return (torch.uint8,)


def _yt():
    import torch
    return (torch.float16, torch.float32)


def _require_matrix(desc: "Desc", packed, workspace, M: int):
    _require(packed, "packed", _u8(), int(desc.total_bytes))
    if workspace is None:   # the library says whether the call needs one (SGEMV_EINVAL)
        return
    _require(workspace, "workspace", _u8(), sgemv_workspace_bytes(desc, M))


def _thresholds(t, M):
    if t is None:
        return None
    arr = np.ascontiguousarray(np.asarray(t, dtype=np.float32).reshape(-1))
    if arr.size == 1 and M > 1:
        arr = np.repeat(arr, M)
    if arr.size != M:
        raise ValueError("one threshold per row")
    return arr


# ---------------------------------------------------------------------------
# the device and host calls
# ---------------------------------------------------------------------------
def sgemv_pack_layout(q, scales_f16, zeros_f16, tile_n: int = SGEMV_TILE_N, _which: str = "sgemv_pack_layout"):
    """Pack int4 codes q (uint8 [N][K]) and fp16 bit patterns of scales and
    zero-points (uint16 [N][K/128]) into a blob.  Returns (Desc, uint8 blob)."""
    q = np.ascontiguousarray(q, dtype=np.uint8)
    s = np.ascontiguousarray(scales_f16)
    z = np.ascontiguousarray(zeros_f16)
    if s.dtype == np.float16:
        s = s.view(np.uint16)
    if z.dtype == np.float16:
        z = z.view(np.uint16)
    s = np.ascontiguousarray(s, dtype=np.uint16)
    z = np.ascontiguousarray(z, dtype=np.uint16)
    N, K = q.shape
    if _which == "sgemv_pack_layout_ng":
        if s.shape != (N // SGEMV_GROUP, K) or z.shape != (N // SGEMV_GROUP, K) or N % SGEMV_GROUP:
            raise ValueError("scales/zeros must be [N/128][K] (groups along N)")
    elif s.shape != (N, K // SGEMV_GROUP) or z.shape != (N, K // SGEMV_GROUP):
        raise ValueError("scales/zeros must be [N][K/128]")
    d = Desc()
    fn = getattr(lib(), _which)
    _check(fn(None, None, None, N, K, SGEMV_GROUP, tile_n, None, 0, ctypes.byref(d)), f"{_which}(size)")
    blob = np.empty(d.total_bytes, dtype=np.uint8)
    _check(fn(_ptr(q), _ptr(s), _ptr(z), N, K, SGEMV_GROUP, tile_n, _ptr(blob), blob.nbytes, ctypes.byref(d)),
           _which)
    return d, blob


def sgemv_pack_layout_z4(q, scales_f16, zeros_f16, tile_n: int = SGEMV_TILE_N):
    """As sgemv_pack_layout, with the compact metadata of layout version 2
    (fp16 scales, then the integer zero-points in 4 bits)."""
    return sgemv_pack_layout(q, scales_f16, zeros_f16, tile_n, _which="sgemv_pack_layout_z4")


def sgemv_pack_layout_ng(q, scales_f16, zeros_f16, tile_n: int = SGEMV_TILE_N):
    """Layout version 3, for weights quantized with groups along N: scales
    and zero-points are uint16 [N/128][K] (one per input column and 128
    outputs)."""
    return sgemv_pack_layout(q, scales_f16, zeros_f16, tile_n, _which="sgemv_pack_layout_ng")


def sgemv_pack_layout_parts(parts, tile_n: int = SGEMV_TILE_N, version: int = SGEMV_LAYOUT_PAIRS):
    """One blob for several projections sharing their input, rows stacked in
    the order given.  `parts` is a list of (q, scales_f16, zeros_f16), each
    with a row count that is a multiple of tile_n and the same K.  Returns
    (Desc, uint8 blob)."""
    qs, ss, zs, ns = [], [], [], []
    for q, s_, z in parts:
        q = np.ascontiguousarray(q, dtype=np.uint8)
        s_ = np.asarray(s_)
        z = np.asarray(z)
        s_ = np.ascontiguousarray(s_.view(np.uint16) if s_.dtype == np.float16 else s_, dtype=np.uint16)
        z = np.ascontiguousarray(z.view(np.uint16) if z.dtype == np.float16 else z, dtype=np.uint16)
        want = ((q.shape[0] // SGEMV_GROUP, q.shape[1]) if version == SGEMV_LAYOUT_NG
                else (q.shape[0], q.shape[1] // SGEMV_GROUP))
        if s_.shape != want or z.shape != s_.shape:
            raise ValueError("scales/zeros of a part must be " +
                             ("[N/128][K]" if version == SGEMV_LAYOUT_NG else "[N][K/128]"))
        qs.append(q); ss.append(s_); zs.append(z); ns.append(q.shape[0])
    Ks = {q.shape[1] for q in qs}
    if len(Ks) != 1:
        raise ValueError("parts must share K")
    K = Ks.pop()
    n = len(qs)
    qa = (ctypes.c_void_p * n)(*[a.ctypes.data for a in qs])
    sa = (ctypes.c_void_p * n)(*[a.ctypes.data for a in ss])
    za = (ctypes.c_void_p * n)(*[a.ctypes.data for a in zs])
    na = np.ascontiguousarray(ns, dtype=np.int32)
    d = Desc()
    L = lib()
    _check(L.sgemv_pack_layout_parts(n, None, None, None, na.ctypes.data, K, SGEMV_GROUP, tile_n, version,
                                     None, 0, ctypes.byref(d)), "sgemv_pack_layout_parts(size)")
    blob = np.empty(d.total_bytes, dtype=np.uint8)
    _check(L.sgemv_pack_layout_parts(n, qa, sa, za, na.ctypes.data, K, SGEMV_GROUP, tile_n, version,
                                     blob.ctypes.data, blob.nbytes, ctypes.byref(d)), "sgemv_pack_layout_parts")
    return d, blob


def sgemv_desc_from_header(blob) -> Desc:
    b = np.ascontiguousarray(np.asarray(blob, dtype=np.uint8)[:64])
    d = Desc()
    _check(lib().sgemv_desc_from_header(_ptr(b), b.nbytes, ctypes.byref(d)),
           "sgemv_desc_from_header")
    return d


def sgemv_gather_indices(x, thresholds, idx, count, K: int | None = None, stream=None):
    """x: fp16 device tensor [K] or [M][ldx]; writes idx (int32 [K]) and
    count (int32 [1]) on the device."""
    M = 1 if x.dim() == 1 else x.shape[0]
    ldx = x.shape[-1] if x.dim() == 1 else x.stride(0)
    K = x.shape[-1] if K is None else K
    _require(x, "x", _f16(), K, rows=M)
    if K > x.shape[-1]:
        raise ValueError(f"x: {x.shape[-1]} columns, K = {K}")
    _require(idx, "idx", _i32(), K)
    _require(count, "count", _i32(), 1)
    _require_gpu(x=x, idx=idx, count=count)
    t = _thresholds(thresholds, M)
    _check(lib().sgemv_gather_indices(_ptr(x), M, K, ldx, _ptr(t), _ptr(idx), _ptr(count),
                                      _stream(stream)), "sgemv_gather_indices")


def _flags(y):
    import torch
    if y.dtype == torch.float32:
        return SGEMV_OUT_F32
    if y.dtype == torch.float16:
        return 0
    raise TypeError("y must be float16 or float32")


def sgemv_run(desc: Desc, packed, x, idx, count, y, workspace, stream=None):
    """y = W . x over idx[:count] (idx None: all columns)."""
    _require_matrix(desc, packed, workspace, 1)
    _require(x, "x", _f16(), desc.K)
    if idx is not None or count is not None:
        _require(idx, "idx", _i32(), desc.K)
        _require(count, "count", _i32(), 1)
    _require(y, "y", _yt(), desc.N)
    _require_gpu(packed=packed, workspace=workspace, x=x, idx=idx, count=count, y=y)
    _check(lib().sgemv_run(ctypes.byref(desc), _ptr(packed), _ptr(x), _ptr(idx), _ptr(count),
                           _ptr(y), _flags(y), _ptr(workspace), _stream(stream)), "sgemv_run")


def sgemv_run_batched(desc: Desc, packed, x, thresholds, idx, count, y, workspace, stream=None):
    """y[m] = W . xe[m] over the union list; x is [M][ldx], y is [M][ldy]."""
    M = x.shape[0]
    _require_matrix(desc, packed, workspace, M)
    _require(x, "x", _f16(), desc.K, rows=M)
    _require(y, "y", _yt(), desc.N, rows=M)
    if x.shape[-1] < desc.K or y.shape[-1] < desc.N:
        raise ValueError(f"x/y: rows of {x.shape[-1]}/{y.shape[-1]}, need K = {desc.K} and N = {desc.N}")
    if idx is not None or count is not None:
        _require(idx, "idx", _i32(), desc.K)
        _require(count, "count", _i32(), 1)
    _require_gpu(packed=packed, workspace=workspace, x=x, idx=idx, count=count, y=y)
    t = _thresholds(thresholds, M)
    _check(lib().sgemv_run_batched(ctypes.byref(desc), _ptr(packed), _ptr(x), M, x.stride(0),
                                   _ptr(t), _ptr(idx), _ptr(count), _ptr(y), y.stride(0),
                                   _flags(y), _ptr(workspace), _stream(stream)),
           "sgemv_run_batched")


def sgemv_run_fused(desc: Desc, packed, x, thresholds, y, workspace, idx=None, count=None,
                    stream=None):
    """Threshold + compact + GEMV in one launch; x is [K] or [M][ldx] with
    M <= 16, y matches; idx/count (optional) receive the active list (the
    union over the rows)."""
    M = 1 if x.dim() == 1 else x.shape[0]
    ldx = desc.K if x.dim() == 1 else x.stride(0)
    ldy = desc.N if y.dim() == 1 else y.stride(0)
    _require_matrix(desc, packed, workspace, M)
    _require(x, "x", _f16(), desc.K, rows=M)
    _require(y, "y", _yt(), desc.N, rows=M)
    if x.shape[-1] < desc.K or y.shape[-1] < desc.N:
        raise ValueError(f"x/y: rows of {x.shape[-1]}/{y.shape[-1]}, need K = {desc.K} and N = {desc.N}")
    if (idx is None) != (count is None):
        raise ValueError("idx and count: both or neither")
    if idx is not None:
        _require(idx, "idx", _i32(), desc.K)
        _require(count, "count", _i32(), 1)
    _require_gpu(packed=packed, workspace=workspace, x=x, idx=idx, count=count, y=y)
    t = _thresholds(thresholds, M)
    _check(lib().sgemv_run_fused(ctypes.byref(desc), _ptr(packed), _ptr(x), M, ldx, _ptr(t),
                                 _ptr(idx), _ptr(count), _ptr(y), ldy, _flags(y),
                                 _ptr(workspace), _stream(stream)), "sgemv_run_fused")


def sgemv_run_fused_static(desc: Desc, packed, x, thresholds, y, idx=None, count=None, stream=None):
    """sgemv_run_fused without a workspace: the library's fixed device array
    holds the scratch (for callers that cannot allocate); no call may overlap
    another such call on the same GPU."""
    M = 1 if x.dim() == 1 else x.shape[0]
    ldx = desc.K if x.dim() == 1 else x.stride(0)
    ldy = desc.N if y.dim() == 1 else y.stride(0)
    _require(packed, "packed", _u8(), int(desc.total_bytes))
    _require(x, "x", _f16(), desc.K, rows=M)
    _require(y, "y", _yt(), desc.N, rows=M)
    if x.shape[-1] < desc.K or y.shape[-1] < desc.N:
        raise ValueError(f"x/y: rows of {x.shape[-1]}/{y.shape[-1]}, need K = {desc.K} and N = {desc.N}")
    if (idx is None) != (count is None):
        raise ValueError("idx and count: both or neither")
    if idx is not None:
        _require(idx, "idx", _i32(), desc.K)
        _require(count, "count", _i32(), 1)
    _require_gpu(packed=packed, x=x, idx=idx, count=count, y=y)
    t = _thresholds(thresholds, M)
    _check(lib().sgemv_run_fused_static(ctypes.byref(desc), _ptr(packed), _ptr(x), M, ldx, _ptr(t),
                                        _ptr(idx), _ptr(count), _ptr(y), ldy, _flags(y), _stream(stream)),
           "sgemv_run_fused_static")


# ---------------------------------------------------------------------------
# 4-bit products that read every weight, and the norms around a block
# ---------------------------------------------------------------------------
_TYPES: dict = {}     # torch dtype -> SGEMV_F16 / BF16 / F32, filled on the first call
_CACHE_TYPES: dict = {}
_torch = None
_raw_stream = None    # device index -> handle of its current stream
_device_now = None    # -> index of the current device


def _load_torch():
    global _torch, _raw_stream, _device_now
    import torch
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream)
    _device_now = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    _torch = torch
    _CACHE_TYPES.update({torch.float16: SGEMV_F16, torch.bfloat16: SGEMV_BF16, torch.float8_e4m3fn: SGEMV_E4M3})
    # last: a thread that finds its type here uses the others without a check
    _TYPES.update({torch.float16: SGEMV_F16, torch.bfloat16: SGEMV_BF16, torch.float32: SGEMV_F32})


def _type_code(t, what: str) -> int:
    try:
        return _TYPES[t.dtype]
    except (KeyError, AttributeError):
        if not _TYPES:
            _load_torch()
        code = _TYPES.get(getattr(t, "dtype", None))   # again: another thread may have filled the table meanwhile
        if code is not None:
            return code
    if not isinstance(t, _torch.Tensor):
        raise ValueError(f"{what}: expected a torch tensor, got {type(t).__name__}")
    raise ValueError(f"{what}: dtype {str(t.dtype).replace('torch.', '')}, expected float16, bfloat16, float32")


def _row_stride(t, what: str, M: int, n: int) -> int:
    """Row stride of a [M][n] operand given as [n] (one row) or [M][>= n]."""
    shape, stride = t.shape, t.stride()
    if len(shape) == 2 and shape[0] == M and shape[1] >= n:
        if shape[1] > 1 and stride[1] != 1:
            raise ValueError(f"{what}: the last dimension must be contiguous")
        if M <= 1:
            return max(shape[1], n)
        if stride[0] < shape[1]:
            raise ValueError(f"{what}: rows overlap (stride {stride[0]} < {shape[1]})")
        return stride[0]
    if len(shape) == 1:
        if M != 1:
            raise ValueError(f"{what}: one row, {M} needed")
        if shape[0] < n:
            raise ValueError(f"{what}: {shape[0]} elements, at least {n} needed")
        if shape[0] > 1 and stride[0] != 1:
            raise ValueError(f"{what}: the last dimension must be contiguous")
        return max(shape[0], n)
    raise ValueError(f"{what}: shape {tuple(shape)}, expected [{M}][>= {n}]")


def _fits_int32(what: str, **sizes):
    """Refuse sizes that the C call's int32 arguments would cut off."""
    for name, v in sizes.items():
        if not -1 << 31 <= v < 1 << 31:
            raise SgemvError(SGEMV_ESIZE, f"{what}: {name} = {v}")


def _vector(t, what: str, n: int, code: int) -> int:
    """Address of an optional contiguous vector of at least n elements."""
    if t is None:
        return 0
    if getattr(t, "shape", None) == (n,) and _TYPES.get(t.dtype) == code and t.is_contiguous():
        return t.data_ptr()
    if _type_code(t, what) != code:
        raise ValueError(f"{what}: dtype {str(t.dtype).replace('torch.', '')} differs from the operands it goes with")
    if t.dim() != 1 or t.shape[0] < n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected [{n}], contiguous")
    return t.data_ptr()


def _stream_on(device, stream):
    """Handle of `stream`, or of the current stream of `device`."""
    if stream is None:
        return _raw_stream(device.index)
    on = getattr(stream, "device", None)
    if on is not None and on.index is not None and on.index != device.index:
        raise ValueError(f"stream: on {on}, the buffers on {device}")
    return stream if isinstance(stream, int) else stream.cuda_stream


def _on_one_gpu(device, names, tensors):
    """Every tensor (None is skipped) lives on `device`, a GPU."""
    if device.type == "cuda":
        index = device.index
        for t in tensors:
            if t is not None and t.get_device() != index:   # -1 for a host tensor
                break
        else:
            return
    for what, t in zip(names, tensors):
        if t is not None and t.device.type != "cuda":
            raise ValueError(f"{what}: must be a GPU tensor")
    for what, t in zip(names, tensors):
        if t is not None and t.device != device:
            raise ValueError(f"{what}: on {t.device}, other buffers on {device}")


def _call(fn, device, args, what: str):
    """fn(*args) with `device` current; a bad status becomes SgemvError."""
    if _device_now() == device.index:
        status = fn(*args)
    else:
        with _torch.cuda.device(device):
            status = fn(*args)
    if status != SGEMV_OK:
        raise SgemvError(status, what)


def _host_codes(a, what: str, dtype, view=None):
    """A contiguous NumPy array of `dtype` from a NumPy array or a torch
    tensor (any device); 16-bit floats become their bit patterns."""
    if not isinstance(a, np.ndarray) and hasattr(a, "detach"):
        import torch
        if a.dtype in (torch.float16, torch.bfloat16):
            a = a.detach().contiguous().cpu().view(torch.int16).numpy().view(np.uint16)
        else:
            a = a.detach().cpu().numpy()
    a = np.asarray(a)
    if a.dtype == np.float16:
        a = a.view(np.uint16) if a.flags.c_contiguous else np.ascontiguousarray(a).view(np.uint16)
    if a.dtype != dtype:
        raise ValueError(f"{what}: dtype {a.dtype}, expected {np.dtype(dtype).name}")
    return np.ascontiguousarray(a)


def _q4_part(part, group: int, what: str):
    q, s, z = part
    q = _host_codes(q, f"{what} codes", np.uint8)
    s = _host_codes(s, f"{what} scales", np.uint16)
    z = None if z is None else _host_codes(z, f"{what} zeros", np.uint8)
    if q.ndim != 2:
        raise ValueError(f"{what} codes: shape {q.shape}, expected [N][K]")
    _fits_int32(what, N=q.shape[0], K=q.shape[1], group=group)
    want = (q.shape[0], -(-q.shape[1] // group)) if group > 0 else None
    for name, a in (("scales", s), ("zeros", z)):
        if a is not None and want is not None and a.shape != want:
            raise ValueError(f"{what} {name}: shape {a.shape}, expected {want}")
    return q, s, z


def _is_bf16(s) -> bool:
    return "bfloat16" in str(getattr(s, "dtype", ""))


def _bf16_scales(said: bool | None, **scales) -> bool:
    """Whether the scales (of one matrix or of a pair, by name) are bf16: by
    their own type, or for uint16 bits as `said` (None: fp16).  Types that
    contradict `said` or each other are refused, never reinterpreted."""
    own = {what: _is_bf16(s) for what, s in scales.items()
           if str(getattr(s, "dtype", "")).endswith("float16")}   # float16 and bfloat16
    if len(set(own.values())) > 1:
        raise ValueError("gate and up scales must have one type")
    for what, bf16 in own.items():
        if said is not None and bf16 != bool(said):
            raise ValueError(f"{what} scales are {'bfloat16' if bf16 else 'float16'}, bf16_scales = {said}")
    if said is not None:
        return bool(said)
    if 0 < len(own) < len(scales) and any(own.values()):   # bits beside bf16 scales
        raise ValueError("gate and up scales must have one type")
    return any(own.values())


def sgemv_q4_pack(q, scales, zeros=None, group: int = SGEMV_GROUP, bf16_scales: bool | None = None):
    """Lay int4 codes q (uint8 [N][K]) with scales [N][ceil(K/group)] (float16,
    bfloat16 or their bits as uint16) and zero-points uint8 (None: symmetric,
    every zero-point 8) out for sgemv_q4_run.  bf16_scales says what uint16
    scales hold (None: fp16); it is refused where scales of a type of their
    own contradict it.  NumPy arrays or torch tensors.  Returns (Q4Desc, uint8
    blob)."""
    bf16 = _bf16_scales(bf16_scales, weight=scales)
    q, s, z = _q4_part((q, scales, zeros), group, "weight")
    flags = (SGEMV_Q4_ZEROS if z is not None else 0) | (SGEMV_Q4_BF16_SCALES if bf16 else 0)
    d = Q4Desc()
    fn, (N, K) = lib().sgemv_q4_pack, q.shape
    _check(fn(None, None, None, N, K, group, flags, None, 0, ctypes.byref(d)), "sgemv_q4_pack(size)")
    blob = np.empty(d.total_bytes, dtype=np.uint8)
    _check(fn(_ptr(q), _ptr(s), _ptr(z), N, K, group, flags, _ptr(blob), blob.nbytes, ctypes.byref(d)),
           "sgemv_q4_pack")
    return d, blob


def sgemv_q4_pack_gated(gate, up, group: int = SGEMV_GROUP, bf16_scales: bool | None = None):
    """The same for a gate and an up projection, each (q, scales, zeros) of
    one shape and format, for sgemv_q4_run_gated."""
    bf16 = _bf16_scales(bf16_scales, gate=gate[1], up=up[1])
    qg, sg, zg = _q4_part(gate, group, "gate")
    qu, su, zu = _q4_part(up, group, "up")
    if qg.shape != qu.shape or (zg is None) != (zu is None):
        raise ValueError("gate and up must have one shape, and both zero-points or neither")
    flags = (SGEMV_Q4_ZEROS if zg is not None else 0) | (SGEMV_Q4_BF16_SCALES if bf16 else 0)
    d = Q4Desc()
    fn, (N, K) = lib().sgemv_q4_pack_gated, qg.shape
    _check(fn(None, None, None, None, None, None, N, K, group, flags, None, 0, ctypes.byref(d)),
           "sgemv_q4_pack_gated(size)")
    blob = np.empty(d.total_bytes, dtype=np.uint8)
    _check(fn(_ptr(qg), _ptr(sg), _ptr(zg), _ptr(qu), _ptr(su), _ptr(zu), N, K, group, flags, _ptr(blob), blob.nbytes,
              ctypes.byref(d)), "sgemv_q4_pack_gated")
    return d, blob


def sgemv_q4_pack_device(q, scales, zeros=None, up=None, group: int = SGEMV_GROUP):
    """sgemv_q4_pack (or, with up = (q, scales, zeros), sgemv_q4_pack_gated)
    of torch tensors that are on one GPU, on that GPU and its current stream;
    scales are float16 or bfloat16.  Codes, scales and zero-points are
    checked, which waits for the GPU.  Returns (Q4Desc, uint8 GPU tensor)."""
    _type_code(scales, "scales")
    torch, parts = _torch, [(q, scales, zeros)] + ([] if up is None else [tuple(up)])
    for name, part in zip(("weight", "up"), parts):
        for kind, t in zip(("codes", "scales", "zeros"), part):
            if not isinstance(t, torch.Tensor) and (kind != "zeros" or t is not None):
                raise ValueError(f"{name} {kind}: expected a torch tensor, got {type(t).__name__}")
    if q.dim() != 2:
        raise ValueError(f"weight codes: shape {tuple(q.shape)}, expected [N][K]")
    N, K = q.shape
    _fits_int32("sgemv_q4_pack_device", N=N, K=K, group=group)
    flags = (SGEMV_Q4_ZEROS if zeros is not None else 0) | (SGEMV_Q4_GATED if up is not None else 0) | \
        (SGEMV_Q4_BF16_SCALES if scales.dtype == torch.bfloat16 else 0)
    d, fn = Q4Desc(), lib().sgemv_q4_pack if up is None else lib().sgemv_q4_pack_gated
    _check(fn(*[None] * (3 * len(parts)), N, K, group, flags, None, 0, ctypes.byref(d)), "sgemv_q4_pack_device(size)")
    device, G, operands = q.device, -(-K // group), []
    for name, (pq, ps, pz) in zip(("weight", "up"), parts):
        if (pz is None) != (zeros is None):
            raise ValueError("gate and up must both have zero-points, or neither")
        for what, t, dtypes, shape in ((f"{name} codes", pq, (torch.uint8,), (N, K)),
                                       (f"{name} scales", ps, (scales.dtype,) if name == "up" else
                                        (torch.float16, torch.bfloat16), (N, G)),
                                       (f"{name} zeros", pz, (torch.uint8,), (N, G))):
            if t is not None and (t.dtype not in dtypes or tuple(t.shape) != shape):
                raise ValueError(f"{what}: {str(t.dtype).replace('torch.', '')} {tuple(t.shape)}, expected "
                                 f"{' or '.join(str(x).replace('torch.', '') for x in dtypes)} {shape}")
            operands.append((what, t))
    _on_one_gpu(device, *zip(*operands))
    for what, t in operands:
        if t is not None and not (bool(torch.isfinite(t).all()) if t.is_floating_point() else int(t.max()) <= 15):
            raise SgemvError(SGEMV_EINVAL, f"sgemv_q4_pack_device: {what}")
    kept = [None if t is None else t.contiguous() for _, t in operands]
    blob = torch.empty(d.total_bytes, dtype=torch.uint8, device=device)
    ptrs = [0 if t is None else t.data_ptr() for t in kept] + [0] * (6 - len(kept))
    _call(lib().sgemv_q4_pack_device, device, (*ptrs, N, K, group, flags, blob.data_ptr(), blob.numel(), d,
                                               _stream_on(device, None)), "sgemv_q4_pack_device")
    return d, blob


def sgemv_q4_desc_from_header(blob) -> Q4Desc:
    b = np.ascontiguousarray(np.asarray(blob, dtype=np.uint8)[:256])
    d = Q4Desc()
    _check(lib().sgemv_q4_desc_from_header(_ptr(b), b.nbytes, ctypes.byref(d)), "sgemv_q4_desc_from_header")
    return d


def _q4_operands(desc, packed, x, y, call, out):
    """Checked (x type, rows, ldx, y type, ldy) of `call`, whose output is named `out`."""
    try:   # what nearly every call brings: two-dimensional operands, checked in few steps
        xt, yt = _TYPES[x.dtype], _TYPES[y.dtype]
        (M, k), (ldx, ex), (rows, n), (ldy, ey) = x.shape, x.stride(), y.shape, y.stride()
        if (rows == M >= 1 and ex == 1 == ey and ldx >= k >= desc.K and ldy >= n >= desc.N and xt < SGEMV_F32
                and ldx | ldy | M < 1 << 31
                and (yt == xt or yt == SGEMV_F32) and packed.dtype is _torch.uint8 and packed.is_contiguous()
                and packed.numel() >= desc.total_bytes):
            return xt, M, ldx, yt, ldy
    except (AttributeError, KeyError, TypeError, ValueError):
        pass
    xt, yt = _type_code(x, "x"), _type_code(y, out)
    if xt == SGEMV_F32:
        raise ValueError("x: dtype float32, expected float16, bfloat16")
    if yt != xt and yt != SGEMV_F32:
        raise ValueError(f"{out}: dtype {str(y.dtype).replace('torch.', '')}, expected x's or float32")
    if not (type(packed) is _torch.Tensor and packed.dtype is _torch.uint8 and packed.is_contiguous()
            and packed.numel() >= desc.total_bytes):
        if isinstance(packed, int):
            raise ValueError("packed: expected a torch tensor, got int")
        _require(packed, "packed", _u8(), int(desc.total_bytes))
    M = 1 if x.dim() < 2 else x.shape[0]
    ldx, ldy = _row_stride(x, "x", M, desc.K), _row_stride(y, out, M, desc.N)
    _fits_int32(call, rows=M, ldx=ldx, **{"ld" + out: ldy})
    return xt, M, ldx, yt, ldy


def sgemv_q4_run(desc: Q4Desc, packed, x, y, bias=None, stream=None):
    """y = W . x + bias over 4-bit weights packed by sgemv_q4_pack: x is [K]
    or [M][>= K] with M <= 16, float16 or bfloat16; y is [N] or [M][>= N], of
    x's type or float32; bias is [N] of x's type.  Runs on `stream`, or on the
    current stream of the tensors' device."""
    xt, M, ldx, yt, ldy = _q4_operands(desc, packed, x, y, "sgemv_q4_run", "y")
    b = None if bias is None else _vector(bias, "bias", desc.N, xt)
    device = x.device
    _on_one_gpu(device, ("packed", "x", "y", "bias"), (packed, x, y, bias))
    _call(lib().sgemv_q4_run, device, (desc, packed.data_ptr(), x.data_ptr(), xt, M, ldx, b, y.data_ptr(), yt, ldy,
                                       _stream_on(device, stream)), "sgemv_q4_run")


_ACTS = {"silu": SGEMV_ACT_SILU, "gelu": SGEMV_ACT_GELU, "relu": SGEMV_ACT_RELU}


def sgemv_q4_run_gated(desc: Q4Desc, packed, x, h, act: str = "silu", bias_gate=None, bias_up=None, stream=None):
    """h = act(gate . x + bias_gate) * (up . x + bias_up) over 4-bit weights
    packed by sgemv_q4_pack_gated; act is "silu", "gelu" (error function) or
    "relu".  Operands as for sgemv_q4_run.  h goes on to sgemv_q4_run, or, as
    float16, to sgemv_run_fused."""
    if act not in _ACTS:
        raise ValueError(f"act: {act!r}, expected one of {', '.join(_ACTS)}")
    xt, M, ldx, ht, ldh = _q4_operands(desc, packed, x, h, "sgemv_q4_run_gated", "h")
    bg = None if bias_gate is None else _vector(bias_gate, "bias_gate", desc.N, xt)
    bu = None if bias_up is None else _vector(bias_up, "bias_up", desc.N, xt)
    device = x.device
    _on_one_gpu(device, ("packed", "x", "h", "bias_gate", "bias_up"), (packed, x, h, bias_gate, bias_up))
    _call(lib().sgemv_q4_run_gated, device, (desc, packed.data_ptr(), x.data_ptr(), xt, M, ldx, bg, bu, _ACTS[act],
                                             h.data_ptr(), ht, ldh, _stream_on(device, stream)), "sgemv_q4_run_gated")


# struct sgemv_norm of the C header, field by field
_NORM = struct.Struct("@qiI9P5q2f4i")


def _norm_operands(x, residual, y, residual_out, weight, bias, post_weight, post_bias, gate):
    """Checked (rows, D, addresses, strides, types) of a sgemv_block_norm call."""
    rt, xt = _type_code(residual, "residual"), _type_code(x, "x")
    rows = 1 if residual.dim() < 2 else residual.shape[0]
    D = residual.shape[-1] if residual.dim() else 0
    _fits_int32("sgemv_block_norm", D=D)
    ldr, ldx = _row_stride(residual, "residual", rows, D), _row_stride(x, "x", rows, D)
    device = residual.device
    yt, ldy, yp, ldg, gp, ldo, op = rt, 0, 0, 0, 0, 0, 0
    if y is not None:
        yt, ldy, yp = _type_code(y, "y"), _row_stride(y, "y", rows, D), y.data_ptr()
    if residual_out is not None:
        if _type_code(residual_out, "residual_out") != rt:
            raise ValueError("residual_out: must have residual's type")
        ldo, op = _row_stride(residual_out, "residual_out", rows, D), residual_out.data_ptr()
    if gate is not None:
        if y is None or _type_code(gate, "gate") != yt:
            raise ValueError("gate: needs y, and y's type")
        if gate.dim() == 1:
            gp = _vector(gate, "gate", D, yt)
        elif gate.dim() == 2 and gate.shape[0] == rows >= 1 and gate.stride(0) == 0:   # one vector, expanded
            gp = _vector(gate[0], "gate", D, yt)
        else:
            ldg, gp = _row_stride(gate, "gate", rows, D), gate.data_ptr()
    wt, w0, w1, w2, w3 = -1, 0, 0, 0, 0
    if weight is not None:
        wt = _type_code(weight, "weight")
        w2 = _vector(weight, "weight", D, wt)
    if bias is not None:
        wt = _type_code(bias, "bias") if wt < 0 else wt
        w3 = _vector(bias, "bias", D, wt)
    if post_weight is not None:
        wt = _type_code(post_weight, "post_weight") if wt < 0 else wt
        w0 = _vector(post_weight, "post_weight", D, wt)
    if post_bias is not None:
        wt = _type_code(post_bias, "post_bias") if wt < 0 else wt
        w1 = _vector(post_bias, "post_bias", D, wt)
    _on_one_gpu(device, ("residual", "x", "y", "residual_out", "gate", "weight", "bias", "post_weight", "post_bias"),
                (residual, x, y, residual_out, gate, weight, bias, post_weight, post_bias))
    return (rows, D, (residual.data_ptr(), yp, gp, w0, w1, w2, w3, op, x.data_ptr()), (ldr, ldy, ldg, ldo, ldx),
            (rt, yt, wt if wt >= 0 else xt, xt))


def _norm_operands_quick(x, residual, y, residual_out, vectors, gate):
    """The same in few steps for what nearly every call brings (matrices of
    two dimensions, vectors of D elements), or None."""
    rt, xt = _TYPES[residual.dtype], _TYPES[x.dtype]
    (rows, D), (ldr, e), device = residual.shape, residual.stride(), residual.device
    (r, n), (ldx, ex) = x.shape, x.stride()
    if not (e == 1 == ex and r == rows and ldr >= D < 1 << 31 and ldx >= n >= D and x.device == device
            and device.type == "cuda"):
        return None
    yt, ldy, yp, gp, ldg, ldo, op, wt, wp = rt, 0, 0, 0, 0, 0, 0, xt, []
    if y is not None:
        (r, n), (ldy, e), yt, yp = y.shape, y.stride(), _TYPES[y.dtype], y.data_ptr()
        if not (e == 1 and r == rows and ldy >= n >= D and y.device == device):
            return None
    if residual_out is not None:
        (r, n), (ldo, e), op = residual_out.shape, residual_out.stride(), residual_out.data_ptr()
        if not (e == 1 and r == rows and ldo >= n >= D and residual_out.device == device
                and residual_out.dtype is residual.dtype):
            return None
    if gate is not None:
        if y is None or gate.dtype is not y.dtype or not gate.is_contiguous() or gate.device != device:
            return None
        gp = gate.data_ptr()
        if gate.shape == (rows, D):
            ldg = D
        elif gate.shape != (D,):
            return None
    dtype = None
    for w in vectors:
        if w is None:
            wp.append(0)
            continue
        if dtype is None:
            dtype, wt = w.dtype, _TYPES[w.dtype]
        if w.dtype is not dtype or w.shape != (D,) or not w.is_contiguous() or w.device != device:
            return None
        wp.append(w.data_ptr())
    return (rows, D, (residual.data_ptr(), yp, gp, *wp, op, x.data_ptr()), (ldr, ldy, ldg, ldo, ldx), (rt, yt, wt, xt))


def sgemv_block_norm(x, residual, y=None, residual_out=None, *, weight=None, bias=None, post_weight=None,
                     post_bias=None, gate=None, scale: float = 1.0, eps: float = 1e-6, post_norm: bool | None = None,
                     center: bool = False, plus_one: bool = False, stream=None):
    """From a block's output y to the next block's input, in one launch:
    r = residual + scale * gate * u with u = y, or norm(y; post_weight,
    post_bias) when post_norm (by default: when either is given);
    residual_out (optional) receives r, x receives norm(r; weight, bias).
    The norm is the root mean square norm, or layer norm with center;
    plus_one takes weights stored around zero.  x, residual, y, residual_out
    are [D] or [rows][>= D] in float16, bfloat16 or float32 (residual_out of
    residual's type); gate is [D] or [rows][D] of y's type; the vectors share
    one type.  D is residual's last dimension; residual_out may be residual
    and x may be y."""
    flags = 0
    if post_norm is None:
        post_norm = post_weight is not None or post_bias is not None
    if post_norm:
        flags |= SGEMV_NORM_POST
        if y is None:
            raise ValueError("post_norm: needs y")
    elif post_weight is not None or post_bias is not None:
        raise ValueError("post_weight, post_bias: given without post_norm")
    if center:
        flags |= SGEMV_NORM_CENTER
    if plus_one:
        flags |= SGEMV_NORM_PLUS_ONE
    try:
        found = _norm_operands_quick(x, residual, y, residual_out, (post_weight, post_bias, weight, bias), gate)
    except (AttributeError, KeyError, TypeError, ValueError):
        found = None
    if found is None:
        found = _norm_operands(x, residual, y, residual_out, weight, bias, post_weight, post_bias, gate)
    rows, D, addresses, strides, types = found
    device = residual.device
    args = _NORM.pack(rows, D, flags, *addresses, *strides, scale, eps, *types)
    _call(lib().sgemv_block_norm, device, (args, _stream_on(device, stream)), "sgemv_block_norm")


# ---------------------------------------------------------------------------
# rotary positions, a paged cache, attention over it, beams, pages
# ---------------------------------------------------------------------------
# the C header's structs, field by field
_KV = struct.Struct("@4P6q6i")
_ROTARY = struct.Struct("@8P12q10iIf")
_ATTN = struct.Struct("@6PN5q5i2fi")
_BEAM = struct.Struct("@7PN2q6i")
_PAGES = struct.Struct("@13PN2q6i")


_NO_SECTIONS = (0,) * SGEMV_MAX_AXES


class KVCache:
    """One layer's paged cache over the caller's tensors: k and v are
    [pages][page_size][heads][dim] in float16, bfloat16 or float8_e4m3fn, any
    strides with the last dimension contiguous (a [pages][heads][page_size][dim]
    buffer is passed as buffer.transpose(1, 2), keys and values of one buffer as
    its slices).  k_scale and v_scale, float32 [heads], say what a stored 1 of
    an 8-bit cache stands for (None: 1).  Addresses, shape and strides are those
    of the tensors when the KVCache is made: one whose storage is replaced later
    (resize_, set_, .data) needs a new KVCache."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if not _TYPES:
            _load_torch()
        for what, t in (("k", k), ("v", v)):
            if not isinstance(t, _torch.Tensor) or t.dim() != 4:
                raise ValueError(f"{what}: expected a torch tensor [pages][page_size][heads][dim]")
            if t.dtype not in _CACHE_TYPES:
                raise ValueError(f"{what}: dtype {str(t.dtype).replace('torch.', '')}, expected float16, bfloat16, "
                                 "float8_e4m3fn")
            if t.shape[3] > 1 and t.stride(3) != 1:
                raise ValueError(f"{what}: the last dimension must be contiguous")
        if k.shape != v.shape or k.dtype != v.dtype:
            raise ValueError("k and v: must have one shape and type")
        self.pages, self.page_size, self.heads, self.dim = k.shape
        _fits_int32("KVCache", pages=self.pages, page_size=self.page_size, heads=self.heads, dim=self.dim)
        self.type = _CACHE_TYPES[k.dtype]
        at = []
        for what, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t is not None and self.type != SGEMV_E4M3:
                raise ValueError(f"{what}: for float8_e4m3fn caches only")
            at.append(0 if t is None else _vector(t, what, self.heads, SGEMV_F32))
        self.k, self.v, self.k_scale, self.v_scale, self.device = k, v, k_scale, v_scale, k.device
        for t in (v, k_scale, v_scale):
            if t is not None and t.device != self.device:
                raise ValueError("k, v and their scales: must be on one device")
        self.args = _KV.pack(k.data_ptr(), v.data_ptr(), *at, *k.stride()[:3], *v.stride()[:3], self.type, self.pages,
                             self.page_size, self.heads, self.dim, 0)


def _cache(cache) -> KVCache:
    if not isinstance(cache, KVCache):
        raise ValueError(f"cache: expected a KVCache, got {type(cache).__name__}")
    return cache


def _heads_of(t, what: str, code: int, like=None):
    """(address, row stride, head stride) of a [rows][heads][dim] tensor of
    type `code`, of the shape `like` where that is given."""
    try:
        if _TYPES[t.dtype] == code:
            shape, (row, head, one) = t.shape, t.stride()
            if (one == 1 or shape[2] <= 1) and (like is None or shape == like):
                return t.data_ptr(), row, head
    except (AttributeError, KeyError, TypeError, ValueError):
        pass
    if _type_code(t, what) != code:
        raise ValueError(f"{what}: dtype {str(t.dtype).replace('torch.', '')} differs from the operands it goes with")
    if t.dim() != 3 or (like is not None and t.shape != like):
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {'[rows][heads][dim]' if like is None else tuple(like)}")
    raise ValueError(f"{what}: the last dimension must be contiguous")


def _ints(t, what: str, *shape) -> int:
    """Address of a contiguous int32 tensor of `shape`."""
    try:
        if t.dtype is _torch.int32 and t.shape == shape and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, _torch.Tensor):
        raise ValueError(f"{what}: expected a torch tensor, got {type(t).__name__}")
    if t.dtype is not _torch.int32:
        raise ValueError(f"{what}: dtype {str(t.dtype).replace('torch.', '')}, expected int32")
    if t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {''.join(f'[{n}]' for n in shape)}")
    raise ValueError(f"{what}: must be contiguous")


def _table_of(t, what: str, rows: int):
    """(address, row stride, columns) of an int32 [rows][max_pages] table."""
    try:
        if t.dtype is _torch.int32 and t.is_contiguous():
            n, columns = t.shape
            if n == rows:
                return t.data_ptr(), columns, columns
    except (AttributeError, ValueError):
        pass
    if not isinstance(t, _torch.Tensor):
        raise ValueError(f"{what}: expected a torch tensor, got {type(t).__name__}")
    if t.dtype is not _torch.int32:
        raise ValueError(f"{what}: dtype {str(t.dtype).replace('torch.', '')}, expected int32")
    if t.dim() != 2 or t.shape[0] != rows:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected [{rows}][max_pages]")
    (ld, one), columns = t.stride(), t.shape[1]
    if columns > 1 and one != 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    return t.data_ptr(), max(ld, columns) if rows <= 1 else ld, columns


def _space(t):
    """(address, bytes) of a workspace."""
    if not isinstance(t, _torch.Tensor) or t.dtype is not _torch.uint8 or not t.is_contiguous():
        raise ValueError("workspace: expected a contiguous uint8 tensor")
    return t.data_ptr(), t.numel()


def sgemv_rotary(q, q_out, positions, inv_freq, *, k=None, k_out=None, v=None, cache: KVCache | None = None, slots=None,
                 sections=None, adjacent: bool = False, striped: bool = False, scale: float = 1.0, stream=None):
    """Turn q (and k) by their positions, write k and v into a paged cache.
    q, q_out are [tokens][heads][dim], k, k_out, v [tokens][kv heads][dim], of
    one type (float16, bfloat16, float32), any strides with the last dimension
    contiguous (views of one projection's output); q and q_out may be None, and
    an output may be its input.  positions is int32 [tokens] or [axes][tokens],
    inv_freq float32 [pairs]; sections gives each axis its number of pairs
    (None: one axis), dealt in turn when `striped`.  Pairs are (i, pairs + i)
    of a head, or (2i, 2i + 1) when `adjacent`.  With a cache, slots is int32
    [tokens] (page * page_size + place; negative: not written)."""
    first = q if q is not None else k
    code = _type_code(first, "q" if q is not None else "k")
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out: both or neither")
    if first.dim() != 3:
        raise ValueError(f"{'q' if q is not None else 'k'}: shape {tuple(first.shape)}, expected [tokens][heads][dim]")
    tokens, _, dim = first.shape
    at, strides = [0] * 8, [0] * 11
    if q is not None:
        at[0], strides[0], strides[1] = _heads_of(q, "q", code)
        at[1], strides[2], strides[3] = _heads_of(q_out, "q_out", code, q.shape)
    if k is not None:
        at[2], strides[4], strides[5] = _heads_of(k, "k", code)
        if k.shape[0] != tokens or k.shape[2] != dim:
            raise ValueError(f"k: shape {tuple(k.shape)}, expected [{tokens}][kv heads][{dim}]")
        if k_out is not None:
            at[3], strides[6], strides[7] = _heads_of(k_out, "k_out", code, k.shape)
        elif cache is None:
            raise ValueError("k: needs k_out or a cache")
    elif k_out is not None:
        raise ValueError("k_out: needs k")
    if cache is None:
        if v is not None or slots is not None:
            raise ValueError("v, slots: need a cache")
    else:
        if k is None:
            raise ValueError("cache: needs k")
        if (_cache(cache).heads, cache.dim) != (k.shape[1], dim):
            raise ValueError(f"cache: {cache.heads} heads of {cache.dim}, k has {k.shape[1]} of {dim}")
        if v is not None:
            at[4], strides[8], strides[9] = _heads_of(v, "v", code, k.shape)
        at[7] = _ints(slots, "slots", tokens)
    shape = getattr(positions, "shape", ())
    if len(shape) not in (1, 2) or positions.dtype is not _torch.int32 or shape[-1] != tokens \
            or (tokens > 1 and positions.stride(-1) != 1):
        raise ValueError(f"positions: expected int32 [{tokens}] or [axes][{tokens}], the last dimension contiguous")
    axes = 1 if len(shape) == 1 else shape[0]
    at[5], strides[10] = positions.data_ptr(), tokens if axes == 1 else positions.stride(0)
    shape = getattr(inv_freq, "shape", ())
    if len(shape) != 1 or inv_freq.dtype is not _torch.float32 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq: expected float32 [pairs], contiguous")
    at[6], pairs = inv_freq.data_ptr(), shape[0]
    sections = (pairs,) if sections is None else tuple(sections)
    if len(sections) != axes or axes > SGEMV_MAX_AXES or sum(sections) != pairs or min(sections) < 0:
        raise ValueError(f"sections: {sections}, expected {axes} numbers that sum to {pairs} (up to {SGEMV_MAX_AXES})")
    device = first.device
    _on_one_gpu(device, ("q", "q_out", "k", "k_out", "v", "positions", "inv_freq", "slots", "cache"),
                (q, q_out, k, k_out, v, positions, inv_freq, slots, None if cache is None else cache.k))
    args = _ROTARY.pack(*at, *strides, tokens, code, 0 if q is None else q.shape[1], 0 if k is None else k.shape[1], dim,
                        pairs, axes, *sections, *_NO_SECTIONS[axes:],
                        (SGEMV_ROTARY_ADJACENT if adjacent else 0) | (SGEMV_ROTARY_STRIPED if striped else 0), scale)
    _call(lib().sgemv_rotary, device, (args, None if cache is None else cache.args, _stream_on(device, stream)),
          "sgemv_rotary")


def sgemv_attn_workspace_bytes(batch: int, heads: int, heads_kv: int, dim: int) -> int:
    return int(lib().sgemv_attn_workspace_bytes(batch, heads, heads_kv, dim))


def sgemv_attn_paged(q, cache: KVCache, table, lengths, out, workspace, *, scale: float | None = None, window: int = 0,
                     softcap: float = 0.0, lse=None, stream=None):
    """Attention of one new token per sequence over its paged cache: q and out
    are [batch][heads][dim] in float16 or bfloat16, heads a multiple of the
    cache's; table is int32 [batch][max_pages], lengths int32 [batch], both on
    the device; workspace is uint8, zero-filled once, of
    sgemv_attn_workspace_bytes(batch, heads, kv heads, dim).  scale defaults
    to 1 / sqrt(dim); window: only the last tokens are seen (0: all), and
    table entries whose tokens all lie before it may be anything;
    softcap * tanh(z / softcap) of every score (0: none); lse (optional)
    float32 [batch][heads] receives the logarithm of the sum of exponentials."""
    code = _type_code(q, "q")
    if code == SGEMV_F32:
        raise ValueError("q: dtype float32, expected float16, bfloat16")
    qp, q_row, q_head = _heads_of(q, "q", code)
    op, out_row, out_head = _heads_of(out, "out", code, q.shape)
    batch, heads, dim = q.shape
    if _cache(cache).dim != dim or heads % cache.heads:
        raise ValueError(f"cache: {cache.heads} heads of {cache.dim}, q has {heads} of {dim}")
    if cache.type not in (code, SGEMV_E4M3):
        raise ValueError("cache: must have q's type, or float8_e4m3fn")
    if softcap and not softcap >= 2.0 ** -126:   # smaller ones would be none as a float
        raise ValueError(f"softcap: {softcap}, expected 0 or a normal float above it")
    tp, ld, columns = _table_of(table, "table", batch)
    lp, zp = _ints(lengths, "lengths", batch), 0
    if lse is not None:
        if _type_code(lse, "lse") != SGEMV_F32 or lse.shape != (batch, heads) or not lse.is_contiguous():
            raise ValueError(f"lse: expected float32 [{batch}][{heads}], contiguous")
        zp = lse.data_ptr()
    wp, size = _space(workspace)
    try:
        args = _ATTN.pack(qp, op, zp, tp, lp, wp, size, q_row, q_head, out_row, out_head, ld, code, batch, heads, columns,
                          window, dim ** -0.5 if scale is None else scale, softcap, 0)
    except struct.error:
        _fits_int32("sgemv_attn_paged", batch=batch, heads=heads, max_pages=columns, window=window)
        raise
    device = q.device
    _on_one_gpu(device, ("q", "cache", "table", "lengths", "out", "workspace", "lse"),
                (q, cache.k, table, lengths, out, workspace, lse))
    _call(lib().sgemv_attn_paged, device, (args, cache.args, _stream_on(device, stream)), "sgemv_attn_paged")


def sgemv_beam_workspace_bytes(batch: int, beams: int, vocab: int, choices: int) -> int:
    return int(lib().sgemv_beam_workspace_bytes(batch, beams, vocab, choices))


def sgemv_beam_select(logits, scores, tokens, parents, scores_out, workspace, *, finished=None, end_token: int = 0,
                      stream=None):
    """The best continuations of a batch of beam searches: logits
    [batch][beams][vocab] (float16, bfloat16, float32, any strides with the
    last dimension contiguous), scores float32 [batch][beams]; tokens and
    parents int32 and scores_out float32 [batch][choices] receive the largest
    score + log softmax(logits), largest first; where there are fewer, token and
    parent are -1.  sgemv_pages_fork takes rows, -1 for those: torch.where(parents < 0,
    -1, parents + beams * arange(batch)[:, None]), and no growth.  finished (optional) uint8
    [batch][beams]: such a beam goes on with end_token at its own score.
    workspace is uint8, zero-filled once, of sgemv_beam_workspace_bytes(batch,
    beams, vocab, choices)."""
    code = _type_code(logits, "logits")
    lp, ld_batch, ld_beam = _heads_of(logits, "logits", code)
    batch, beams, vocab = logits.shape
    if not isinstance(scores_out, _torch.Tensor) or scores_out.dim() != 2:
        raise ValueError(f"scores_out: expected float32 [{batch}][choices]")
    choices = scores_out.shape[1]
    for what, t, shape in (("scores", scores, (batch, beams)), ("scores_out", scores_out, (batch, choices))):
        if _type_code(t, what) != SGEMV_F32 or t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{what}: expected float32 {shape}, contiguous")
    fp = 0
    if finished is not None:
        if not isinstance(finished, _torch.Tensor) or finished.dtype not in (_torch.uint8, _torch.bool) \
                or finished.shape != (batch, beams) or not finished.is_contiguous():
            raise ValueError(f"finished: expected uint8 or bool [{batch}][{beams}], contiguous")
        fp = finished.data_ptr()
    wp, size = _space(workspace)
    device = logits.device
    tp, pp = _ints(tokens, "tokens", batch, choices), _ints(parents, "parents", batch, choices)
    try:
        args = _BEAM.pack(lp, scores.data_ptr(), fp, tp, pp, scores_out.data_ptr(), wp, size, ld_batch, ld_beam, code,
                          batch, beams, vocab, choices, end_token)
    except struct.error:
        _fits_int32("sgemv_beam_select", batch=batch, beams=beams, vocab=vocab, choices=choices, end_token=end_token)
        raise
    _on_one_gpu(device, ("logits", "scores", "tokens", "parents", "scores_out", "workspace", "finished"),
                (logits, scores, tokens, parents, scores_out, workspace, finished))
    _call(lib().sgemv_beam_select, device, (args, _stream_on(device, stream)), "sgemv_beam_select")


def sgemv_pages_workspace_bytes(rows: int, max_pages: int, pages: int) -> int:
    return int(lib().sgemv_pages_workspace_bytes(rows, max_pages, pages))


def _caches(caches) -> tuple:
    caches = [_cache(c) for c in caches]
    if len(caches) > SGEMV_MAX_LAYERS:
        raise SgemvError(SGEMV_ESIZE, f"caches: {len(caches)}, at most {SGEMV_MAX_LAYERS} a call")
    return caches, b"".join([c.args for c in caches]) if caches else None


def _pages_call(name, table, lengths, refs, table_out, lengths_out, refs_out, workspace, page_size, parents, grow, slots,
                pairs, count, status, caches, stream):
    if not _TYPES:
        _load_torch()
    if not isinstance(table, _torch.Tensor) or table.dim() != 2:
        raise ValueError("table: expected int32 [rows][max_pages]")
    rows = table.shape[0]
    tp, ld, columns = _table_of(table, "table", rows)
    op, ld_out, columns_out = _table_of(table_out, "table_out", rows)
    if columns_out != columns:
        raise ValueError(f"table_out: {columns_out} columns, table has {columns}")
    if not isinstance(refs, _torch.Tensor) or refs.dim() != 1:
        raise ValueError("refs: expected int32 [pages]")
    pages = refs.shape[0]
    if slots is not None and (not isinstance(slots, _torch.Tensor) or slots.dim() != 2):
        raise ValueError(f"slots: expected int32 [{rows}][most]")
    lp, rp = _ints(lengths, "lengths", rows), _ints(refs, "refs", pages)
    fork = name == "sgemv_pages_fork"
    at = [tp, lp, rp, op, _ints(lengths_out, "lengths_out", rows) if fork else 0, _ints(refs_out, "refs_out", pages),
          0 if parents is None else _ints(parents, "parents", rows), 0 if grow is None else _ints(grow, "grow", rows),
          0 if slots is None else _ints(slots, "slots", rows, slots.shape[1]), _ints(pairs, "pairs", rows if fork else pages, 3),
          _ints(count, "count", 1), _ints(status, "status", 2) if fork else 0]
    wp, size = _space(workspace)
    max_grow = 0 if slots is None else slots.shape[1]
    caches, packed = _caches(caches)
    try:
        args = _PAGES.pack(*at, wp, size, ld, ld_out, rows, columns, pages, page_size, max_grow, len(caches))
    except struct.error:
        _fits_int32(name, rows=rows, max_pages=columns, pages=pages, page_size=page_size, max_grow=max_grow)
        raise
    device = table.device
    _on_one_gpu(device, ("table", "lengths", "refs", "table_out", "lengths_out", "refs_out", "parents", "grow", "slots",
                         "pairs", "count", "status", "workspace") + ("caches",) * len(caches),
                (table, lengths, refs, table_out, lengths_out, refs_out, parents, grow, slots, pairs, count, status,
                 workspace) + tuple(c.k for c in caches))
    _call(getattr(lib(), name), device, (args, packed, _stream_on(device, stream)), name)


def sgemv_pages_fork(table, lengths, refs, table_out, lengths_out, refs_out, workspace, *, page_size: int, pairs, count,
                     status, parents=None, grow=None, slots=None, caches=(), stream=None):
    """One step of a batch's pages, all int32 on the device: table
    [rows][max_pages], lengths [rows], refs [pages] (how many rows' entries name
    a page; 0: free).  Row r takes over the pages of row parents[r] (None: its
    own; outside 0 .. rows - 1: it ends), then grows by grow[r] tokens (None: by
    none), whose places go to slots [rows][most]; a shared last page is copied
    for a row that grows, in every KVCache of `caches`, and listed in pairs
    [rows][3], count [1].  status [2]: pages missing, rows that cannot grow
    that far; where either is not 0, no row grows.  Outputs may be their inputs.
    workspace is uint8, zero-filled once, of sgemv_pages_workspace_bytes."""
    _pages_call("sgemv_pages_fork", table, lengths, refs, table_out, lengths_out, refs_out, workspace, page_size, parents,
                grow, slots, pairs, count, status, caches, stream)


def sgemv_pages_compact(table, lengths, refs, table_out, refs_out, workspace, *, page_size: int, pairs, count, caches=(),
                        stream=None):
    """Move the pages in use to the lowest ids, in tables, counts and every
    KVCache of `caches`; pairs [pages][3] and count [1] say which went where."""
    _pages_call("sgemv_pages_compact", table, lengths, refs, table_out, None, refs_out, workspace, page_size, None, None,
                None, pairs, count, None, caches, stream)


def sgemv_pages_copy(caches, pairs, count=None, stream=None):
    """Copy pages within every KVCache of `caches`: pairs int32 [n][3] of
    (source, target, tokens), the first count[0] of them (None: all)."""
    if not _TYPES:
        _load_torch()
    caches, packed = _caches(caches)
    if not caches:
        raise ValueError("caches: at least one")
    if not isinstance(pairs, _torch.Tensor) or pairs.dim() != 2:
        raise ValueError("pairs: expected int32 [n][3]")
    pp, cp = _ints(pairs, "pairs", pairs.shape[0], 3), 0 if count is None else _ints(count, "count", 1)
    _fits_int32("sgemv_pages_copy", pairs=pairs.shape[0])
    device = caches[0].device
    _on_one_gpu(device, ("caches",) * len(caches) + ("pairs", "count"), tuple(c.k for c in caches) + (pairs, count))
    _call(lib().sgemv_pages_copy, device, (packed, len(caches), pp, cp, pairs.shape[0], _stream_on(device, stream)),
          "sgemv_pages_copy")


def sgemv_workspace_bytes(desc: Desc, M: int = 1) -> int:
    return int(lib().sgemv_workspace_bytes(ctypes.byref(desc), M))


def sgemv_last_hip_error() -> int:
    return int(lib().sgemv_last_hip_error())


# ---------------------------------------------------------------------------
# convenience: device buffers for one matrix
# ---------------------------------------------------------------------------
class PackedMatrix:
    """A packed matrix on the device with its workspace (torch tensors)."""

    def __init__(self, q, scales_f16, zeros_f16, device="cuda", max_batch: int = SGEMV_MAX_BATCH,
                 z4: bool = False, _packed=None, ng: bool = False):
        import torch
        if _packed is None:
            pack = sgemv_pack_layout_ng if ng else sgemv_pack_layout_z4 if z4 else sgemv_pack_layout
            _packed = pack(q, scales_f16, zeros_f16)
        self.desc, blob = _packed
        self.blob = torch.from_numpy(blob).to(device)
        self.workspace = torch.zeros(max(sgemv_workspace_bytes(self.desc, max_batch), 256),
                                     dtype=torch.uint8, device=device)
        self.N, self.K = self.desc.N, self.desc.K

    @classmethod
    def from_parts(cls, parts, device="cuda", max_batch: int = SGEMV_MAX_BATCH, z4: bool = False,
                   ng: bool = False):
        """Several projections sharing their input as one matrix (rows
        stacked in order), packed by sgemv_pack_layout_parts (ng: parts
        quantized with groups along N, layout version 3)."""
        version = SGEMV_LAYOUT_NG if ng else SGEMV_LAYOUT_Z4 if z4 else SGEMV_LAYOUT_PAIRS
        packed = sgemv_pack_layout_parts(parts, version=version)
        return cls(None, None, None, device=device, max_batch=max_batch, z4=z4, _packed=packed, ng=ng)


class FusedProjections:
    """Projections that read the same activations (q/k/v, gate/up), packed
    as one matrix with their rows concatenated, so that one call of
    sgemv_run_fused thresholds x once and computes all of them.  Each
    projection's N must be a multiple of 512 (the layout tile), so every
    tile belongs to one projection.  `split(y)` returns the per-projection
    views of the concatenated output."""

    def __init__(self, parts, device="cuda", max_batch: int = 2, z4: bool = False, ng: bool = False):
        names = [p[0] for p in parts]
        if len(set(names)) != len(names):
            raise ValueError("projection names must be unique")
        Ks = {np.asarray(p[1]).shape[1] for p in parts}
        if len(Ks) != 1:
            raise ValueError("fused projections must share K")
        self.offsets = {}
        start = 0
        for name, q, _, _ in parts:
            n = np.asarray(q).shape[0]
            if n % SGEMV_TILE_N:
                raise ValueError(f"{name}: N = {n} is not a multiple of {SGEMV_TILE_N}")
            self.offsets[name] = (start, n)
            start += n
        self.matrix = PackedMatrix.from_parts([p[1:] for p in parts], device=device, max_batch=max_batch, z4=z4,
                                              ng=ng)
        self.N, self.K = self.matrix.N, self.matrix.K

    def split(self, y):
        return {name: y[..., a:a + n] for name, (a, n) in self.offsets.items()}


class Q4Matrix:
    """A matrix (or gate/up pair) packed for sgemv_q4_run (sgemv_q4_run_gated)
    on the device: codes q uint8 [N][K], scales [N][ceil(K/group)], zeros
    uint8 or None (symmetric).  GPU tensors are packed on their GPU, host
    arrays on the host."""

    def __init__(self, q, scales, zeros=None, group: int = SGEMV_GROUP, device="cuda", bf16_scales=None, _up=None):
        import torch
        if isinstance(q, torch.Tensor) and q.is_cuda:
            if bf16_scales not in (None, _is_bf16(scales)):
                raise ValueError("scales on a GPU are float16 or bfloat16 tensors, which say their type themselves")
            self.desc, blob = sgemv_q4_pack_device(q, scales, zeros, _up, group)
        else:
            if _up is None:
                self.desc, blob = sgemv_q4_pack(q, scales, zeros, group, bf16_scales)
            else:
                self.desc, blob = sgemv_q4_pack_gated((q, scales, zeros), _up, group, bf16_scales)
            blob = torch.from_numpy(blob)
        self.blob = blob.to(device)
        self.N, self.K = self.desc.N, self.desc.K

    @classmethod
    def gated(cls, gate, up, group: int = SGEMV_GROUP, device="cuda", bf16_scales=None):
        """A gate and an up projection, each (q, scales, zeros)."""
        return cls(*gate, group=group, device=device, bf16_scales=bf16_scales, _up=tuple(up))
