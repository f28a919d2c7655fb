"""Paged GQA verify attention over an FP8 E4M3 KV cache, for GB300 (sm_103a).

Thin Python binding of the C ABI in ``include/verify_attn_e4m3.h``: it turns
torch tensors into ``vae4_tensor`` descriptors and passes torch's current CUDA
stream.  Every step of the computation runs in the library's CUDA kernels;
this module does argument marshalling only and has no fallback: if the
library cannot be built or loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

ABI_VERSION = 3

VAE4_U8, VAE4_I32, VAE4_F16, VAE4_F32, VAE4_BF16 = 1, 2, 3, 4, 5

FLAG_WARP_MMA = 0x1
FLAG_KV_E5M2 = 0x2
FLAG_BRIDGE_RAW = 0x4
FLAG_TEST_SHORT_WAITS = 0x8

STATUS_BAD_BLOCK = 0x1
STATUS_BAD_LENGTH = 0x2
STATUS_BAD_QLEN = 0x4
STATUS_TIMEOUT = 0x8
STATUS_PLAN = 0x10
STATUS_BAD_SCALE = 0x20
STATUS_BAD_VALUE = 0x40

ERRORS = {
    0: "VAE4_OK", -1: "VAE4_ERR_NULL", -2: "VAE4_ERR_DTYPE", -3: "VAE4_ERR_SHAPE",
    -4: "VAE4_ERR_STRIDE", -5: "VAE4_ERR_MISALIGNED", -6: "VAE4_ERR_UNSUPPORTED",
    -7: "VAE4_ERR_GQA", -8: "VAE4_ERR_WORKSPACE", -9: "VAE4_ERR_CUDA",
    -10: "VAE4_ERR_PARTITION", -11: "VAE4_ERR_OPTIONS",
}

# Every symbol include/verify_attn_e4m3.h declares.
EXPORTS = (
    "verify_attn_e4m3", "verify_attn_e4m3_ex", "verify_attn_e4m3_partials",
    "verify_attn_e4m3_combine", "verify_attn_e4m3_plan",
    "verify_attn_e4m3_workspace_bytes", "verify_attn_e4m3_abi_version",
    "verify_attn_e4m3_strerror", "verify_attn_e4m3_read_status",
    "verify_attn_e4m3_clear_status", "verify_attn_e4m3_decode_table",
    "verify_attn_e4m3_noalloc", "verify_attn_e4m3_kv_read",
    "verify_attn_e4m3_bridge_fp16", "verify_attn_e4m3_kv",
    "verify_attn_e4m3_append", "verify_attn_e4m3_block_scaled",
    "verify_attn_e4m3_block_scores", "verify_attn_e4m3_select_blocks",
    "verify_attn_e4m3_sparse", "verify_attn_e4m3_block_scaled_workspace_bytes",
    "verify_attn_e4m3_sparse_workspace_bytes",
)

NOALLOC_SCRATCH_BYTES = 8 << 20


class Tensor(ctypes.Structure):
    """vae4_tensor"""
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32),
                ("ndim", ctypes.c_int32), ("shape", ctypes.c_int64 * 5),
                ("stride", ctypes.c_int64 * 5)]


class Options(ctypes.Structure):
    """vae4_options"""
    _fields_ = [("softmax_scale", ctypes.c_float), ("partition_tokens", ctypes.c_int32),
                ("max_seq_len", ctypes.c_int32), ("num_sms", ctypes.c_int32),
                ("flags", ctypes.c_int32), ("hilo_pv", ctypes.c_int32)]


class Vae4Error(RuntimeError):
    def __init__(self, code: int, where: str = ""):
        self.code = code
        super().__init__(f"{where}: {ERRORS.get(code, code)} ({strerror(code)})")


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    from . import _build
    return _build.LIB


def load(build_if_stale: bool = True):
    """Load libvae4.so (building it first if it is missing or stale) and check
    its ABI revision; raises if either step fails."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        from . import _build
        if build_if_stale and not _build.up_to_date():
            _build.build()
        if not os.path.exists(_build.LIB):
            raise RuntimeError(f"{_build.LIB} is missing; build it with "
                               "fp8_paged_attention_e4m3_gb300._build.build()")
        lib = ctypes.CDLL(_build.LIB)
        P = ctypes.POINTER(Tensor)
        for name in ("verify_attn_e4m3",):
            getattr(lib, name).argtypes = [P] * 7 + [ctypes.c_void_p]
            getattr(lib, name).restype = ctypes.c_int
        for name in ("verify_attn_e4m3_ex", "verify_attn_e4m3_partials",
                     "verify_attn_e4m3_combine", "verify_attn_e4m3_kv_read"):
            getattr(lib, name).argtypes = [P] * 7 + [ctypes.c_void_p, ctypes.POINTER(Options)]
            getattr(lib, name).restype = ctypes.c_int
        lib.verify_attn_e4m3_kv.argtypes = [P] * 8 + [ctypes.c_void_p, ctypes.POINTER(Options)]
        lib.verify_attn_e4m3_kv.restype = ctypes.c_int
        lib.verify_attn_e4m3_bridge_fp16.argtypes = [P] * 6 + [ctypes.c_void_p, ctypes.c_int32,
                                                               ctypes.c_void_p]
        lib.verify_attn_e4m3_bridge_fp16.restype = ctypes.c_int
        lib.verify_attn_e4m3_plan.argtypes = [ctypes.c_int] * 5 + [
            ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32)]
        lib.verify_attn_e4m3_plan.restype = ctypes.c_int
        lib.verify_attn_e4m3_workspace_bytes.argtypes = [ctypes.c_int] * 8
        lib.verify_attn_e4m3_workspace_bytes.restype = ctypes.c_int64
        lib.verify_attn_e4m3_abi_version.argtypes = []
        lib.verify_attn_e4m3_abi_version.restype = ctypes.c_int
        lib.verify_attn_e4m3_strerror.argtypes = [ctypes.c_int]
        lib.verify_attn_e4m3_strerror.restype = ctypes.c_char_p
        lib.verify_attn_e4m3_read_status.argtypes = [P, ctypes.POINTER(ctypes.c_int32),
                                                     ctypes.c_void_p]
        lib.verify_attn_e4m3_read_status.restype = ctypes.c_int
        lib.verify_attn_e4m3_clear_status.argtypes = [P, ctypes.c_void_p]
        lib.verify_attn_e4m3_clear_status.restype = ctypes.c_int
        lib.verify_attn_e4m3_decode_table.argtypes = [ctypes.c_void_p,
                                                      ctypes.POINTER(ctypes.c_int32),
                                                      ctypes.c_int32, ctypes.c_void_p]
        lib.verify_attn_e4m3_decode_table.restype = ctypes.c_int
        lib.verify_attn_e4m3_noalloc.argtypes = [P] * 6 + [ctypes.c_void_p,
                                                           ctypes.POINTER(Options)]
        lib.verify_attn_e4m3_noalloc.restype = ctypes.c_int
        v = lib.verify_attn_e4m3_abi_version()
        if v != ABI_VERSION:
            raise RuntimeError(f"stale library: ABI revision {v}, binding expects "
                               f"{ABI_VERSION}; rebuild it")
        VP, I, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float
        O = ctypes.POINTER(Options)
        for name, args in (("append", [VP] * 9 + [I, VP]),
                           ("block_scaled", [VP] * 9 + [O]),
                           ("sparse", [VP] * 10 + [O]),
                           ("block_scores", [VP] * 6 + [I, F, VP, I, VP]),
                           ("select_blocks", [VP] * 3 + [I, I, I, VP, VP])):
            fn = getattr(lib, "verify_attn_e4m3_" + name)
            fn.argtypes, fn.restype = args, ctypes.c_int
        lib.verify_attn_e4m3_block_scaled_workspace_bytes.argtypes = [ctypes.c_int] * 7
        lib.verify_attn_e4m3_block_scaled_workspace_bytes.restype = ctypes.c_int64
        lib.verify_attn_e4m3_sparse_workspace_bytes.argtypes = [ctypes.c_int] * 9
        lib.verify_attn_e4m3_sparse_workspace_bytes.restype = ctypes.c_int64
        _lib = lib
        return lib


def strerror(code: int) -> str:
    try:
        return load().verify_attn_e4m3_strerror(int(code)).decode()
    except Exception:  # library unavailable
        return ERRORS.get(code, "unknown")


# ----------------------------------------------------------------------------
# torch tensor -> vae4_tensor
# ----------------------------------------------------------------------------
def _dtype_code(t) -> int:
    import torch
    m = {torch.uint8: VAE4_U8, torch.int32: VAE4_I32, torch.float16: VAE4_F16,
         torch.float32: VAE4_F32}
    if t.dtype == getattr(torch, "float8_e4m3fn", None):
        return VAE4_U8
    if t.dtype not in m:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return m[t.dtype]


def describe(t) -> Tensor:
    """A vae4_tensor view of a torch tensor (no copy)."""
    if t.dim() > 5:
        raise ValueError("at most 5 dimensions")
    d = Tensor()
    d.data = t.data_ptr() if t.numel() > 0 or t.data_ptr() else None
    d.dtype = _dtype_code(t)
    d.ndim = t.dim()
    for k in range(t.dim()):
        d.shape[k] = t.shape[k]
        d.stride[k] = t.stride(k)
    return d


def _stream_handle(stream) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _check(rc: int, where: str):
    if rc != 0:
        raise Vae4Error(rc, where)


# ----------------------------------------------------------------------------
# public API (same names as the C ABI)
# ----------------------------------------------------------------------------
def verify_attn_e4m3(q, kv_pages, block_table, seq_lens, kv_scales, out, workspace, *,
                     softmax_scale: float = 0.0, partition_tokens: int = 0,
                     max_seq_len: int = 0, num_sms: int = 0, flags: int = 0,
                     hilo_pv: bool = False, stream=None):
    """Run the verify step into ``out``.  All tensors on the current device;
    see include/verify_attn_e4m3.h for layouts.  Asynchronous on ``stream``
    (torch's current stream by default).  ``partition_tokens=0`` selects the
    automatic plan, made on the device from the lengths of each call (a
    captured graph stays balanced as they change); a positive multiple of 16
    fixes T.  ``hilo_pv=True`` carries P into the value product as an FP16
    high part plus a residual scaled by 2^11 (about 22 significant bits)."""
    lib = load()
    opt = Options(float(softmax_scale), int(partition_tokens), int(max_seq_len),
                  int(num_sms), int(flags), int(bool(hilo_pv)))
    descs = [describe(t) for t in (q, kv_pages, block_table, seq_lens, kv_scales, out,
                                   workspace)]
    rc = lib.verify_attn_e4m3_ex(*[ctypes.byref(x) for x in descs],
                                 ctypes.c_void_p(_stream_handle(stream)), ctypes.byref(opt))
    _check(rc, "verify_attn_e4m3")
    return out


verify = verify_attn_e4m3


def verify_attn_e4m3_kv(q, k_cache, v_cache, block_table, seq_lens, kv_scales, out, workspace,
                        *, softmax_scale: float = 0.0, partition_tokens: int = 0,
                        max_seq_len: int = 0, num_sms: int = 0, flags: int = 0,
                        hilo_pv: bool = False, stream=None):
    """The verify step over separate K and V caches uint8 [n_pages][page]
    [Hkv][D] in any strided layout (token-major, padded token strides that
    are multiples of 8 bytes); see the header.  Other arguments as
    verify_attn_e4m3."""
    lib = load()
    opt = Options(float(softmax_scale), int(partition_tokens), int(max_seq_len),
                  int(num_sms), int(flags), int(bool(hilo_pv)))
    descs = [describe(t) for t in (q, k_cache, v_cache, block_table, seq_lens, kv_scales,
                                   out, workspace)]
    rc = lib.verify_attn_e4m3_kv(*[ctypes.byref(x) for x in descs],
                                 ctypes.c_void_p(_stream_handle(stream)), ctypes.byref(opt))
    _check(rc, "verify_attn_e4m3_kv")
    return out


def _stage(name, q, kv_pages, block_table, seq_lens, kv_scales, out, workspace, *,
           softmax_scale=0.0, partition_tokens=0, max_seq_len=0, num_sms=0, flags=0,
           hilo_pv=False, stream=None):
    lib = load()
    opt = Options(float(softmax_scale), int(partition_tokens), int(max_seq_len),
                  int(num_sms), int(flags), int(bool(hilo_pv)))
    descs = [describe(t) for t in (q, kv_pages, block_table, seq_lens, kv_scales, out,
                                   workspace)]
    rc = getattr(lib, name)(*[ctypes.byref(x) for x in descs],
                            ctypes.c_void_p(_stream_handle(stream)), ctypes.byref(opt))
    _check(rc, name)
    return out


def verify_attn_e4m3_partials(*args, **kw):
    """Split stage only (see the header)."""
    return _stage("verify_attn_e4m3_partials", *args, **kw)


def verify_attn_e4m3_combine(*args, **kw):
    """Combine stage only (see the header)."""
    return _stage("verify_attn_e4m3_combine", *args, **kw)


def verify_attn_e4m3_bridge_fp16(kv_pages, block_table, seq_lens, kv_scales, k_out, v_out,
                                 *, status=None, flags: int = 0, stream=None):
    """Paged FP8 -> dense FP16 K and V (see the header): k_out / v_out are
    fp16 [B][Hkv][cap][D]; status is an optional int32 device tensor whose
    first element receives the status bits."""
    lib = load()
    descs = [describe(t) for t in (kv_pages, block_table, seq_lens, kv_scales, k_out, v_out)]
    st = ctypes.c_void_p(status.data_ptr()) if status is not None else ctypes.c_void_p(None)
    rc = lib.verify_attn_e4m3_bridge_fp16(*[ctypes.byref(x) for x in descs], st,
                                          ctypes.c_int32(int(flags)),
                                          ctypes.c_void_p(_stream_handle(stream)))
    _check(rc, "verify_attn_e4m3_bridge_fp16")
    return k_out, v_out


def verify_attn_e4m3_kv_read(*args, **kw):
    """Streaming read of the step's KV bytes, no compute (see the header):
    the gather floor the step is measured against."""
    return _stage("verify_attn_e4m3_kv_read", *args, **kw)


def verify_attn_e4m3_noalloc(q, kv_pages, block_table, seq_lens, kv_scales, out, *,
                             softmax_scale: float = 0.0, partition_tokens: int = 0,
                             max_seq_len: int = 0, num_sms: int = 0, hilo_pv: bool = False,
                             stream=None):
    """The verify step without a workspace, for callers that cannot allocate
    device memory: the library's own fixed 8 MiB scratch holds the partials.
    Calls on one device share that scratch, so they must not overlap on the
    GPU; the first call on a device must precede any stream capture."""
    lib = load()
    opt = Options(float(softmax_scale), int(partition_tokens), int(max_seq_len),
                  int(num_sms), 0, int(bool(hilo_pv)))
    descs = [describe(t) for t in (q, kv_pages, block_table, seq_lens, kv_scales, out)]
    rc = lib.verify_attn_e4m3_noalloc(*[ctypes.byref(x) for x in descs],
                                      ctypes.c_void_p(_stream_handle(stream)),
                                      ctypes.byref(opt))
    _check(rc, "verify_attn_e4m3_noalloc")
    return out


def verify_attn_e4m3_plan(B: int, Hkv: int, max_seq_len: int, partition_tokens: int = 0,
                          num_sms: int = 0):
    """(T, P) of the split-K plan for sequences at the capacity (with
    partition_tokens == 0 a call refines it on the device from the lengths it
    reads); num_sms == 0 uses the current device."""
    lib = load()
    if num_sms == 0:
        import torch
        num_sms = torch.cuda.get_device_properties(torch.cuda.current_device()) \
            .multi_processor_count
    T, P = ctypes.c_int32(), ctypes.c_int32()
    _check(lib.verify_attn_e4m3_plan(B, Hkv, max_seq_len, partition_tokens, num_sms,
                                     ctypes.byref(T), ctypes.byref(P)), "plan")
    return T.value, P.value


plan = verify_attn_e4m3_plan


def verify_attn_e4m3_workspace_bytes(B, Hq, Hkv, Qmax, D, max_seq_len,
                                     partition_tokens=0, num_sms=0) -> int:
    n = load().verify_attn_e4m3_workspace_bytes(B, Hq, Hkv, Qmax, D, max_seq_len,
                                                 partition_tokens, num_sms)
    if n < 0:
        raise Vae4Error(int(n), "workspace_bytes")
    return int(n)


workspace_bytes = verify_attn_e4m3_workspace_bytes


def verify_attn_e4m3_read_status(workspace, stream=None) -> int:
    """Status word of ``workspace`` (synchronises the stream)."""
    import torch
    lib = load()
    host = ctypes.c_int32(0)
    st = stream or torch.cuda.current_stream()
    _check(lib.verify_attn_e4m3_read_status(ctypes.byref(describe(workspace)),
                                            ctypes.byref(host),
                                            ctypes.c_void_p(_stream_handle(st))),
           "read_status")
    st.synchronize()
    return host.value & 0xFFFFFFFF


read_status = verify_attn_e4m3_read_status


def verify_attn_e4m3_clear_status(workspace, stream=None):
    _check(load().verify_attn_e4m3_clear_status(ctypes.byref(describe(workspace)),
                                                ctypes.c_void_p(_stream_handle(stream))),
           "clear_status")


clear_status = verify_attn_e4m3_clear_status


def verify_attn_e4m3_decode_table(flags: int = 0, stream=None):
    """(fp16 bit patterns of the 256 decoded codes as a device uint16-in-int16
    tensor, scale exponent): code b decodes to dec(b) * 2^scale_log2.  flags
    picks the kernel whose decoder runs (0 = tcgen05 path)."""
    import torch
    out = torch.empty(256, dtype=torch.int16, device="cuda")
    e = ctypes.c_int32(0)
    _check(load().verify_attn_e4m3_decode_table(ctypes.c_void_p(out.data_ptr()),
                                                ctypes.byref(e), int(flags),
                                                ctypes.c_void_p(_stream_handle(stream))),
           "decode_table")
    return out, e.value


decode_table = verify_attn_e4m3_decode_table


def alloc_workspace(B, Hq, Hkv, Qmax, D, max_seq_len, partition_tokens=0, device=None):
    """A zeroed workspace of the right size (torch allocation, 256-B aligned),
    for the head-scaled calls and verify_attn_e4m3_block_scaled alike (for the
    head-scaled calls alone where the other refuses the batch as too large)."""
    import torch
    n = workspace_bytes(B, Hq, Hkv, Qmax, D, max_seq_len, partition_tokens)
    try:
        n = max(n, block_scaled_workspace_bytes(B, Hq, Hkv, Qmax, D, max_seq_len))
    except Vae4Error as e:
        if ERRORS.get(e.code) != "VAE4_ERR_SHAPE":
            raise
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


# ----------------------------------------------------------------------------
# the block-scaled cache
# ----------------------------------------------------------------------------
def cache_views(kv_pages):
    """(K, V) views [n_pages][page][Hkv][D] of a pool [n_pages][2][Hkv][page][D]
    (no copy): the form the block-scaled cache's calls take."""
    return kv_pages[:, 0].transpose(1, 2), kv_pages[:, 1].transpose(1, 2)


def alloc_block_scales(n_pages, Hkv, page, block_tokens, device=None):
    """Block scales f32 [n_pages][2][Hkv][page / block_tokens] of an empty
    cache (torch allocation)."""
    import torch
    if block_tokens < 16 or block_tokens % 16 or page % block_tokens:
        raise ValueError("block_tokens: a multiple of 16 that divides the page")
    return torch.ones(n_pages, 2, Hkv, page // block_tokens, dtype=torch.float32,
                      device=device or "cuda")


def alloc_k_bounds(n_pages, Hkv, page, block_tokens, D, device=None):
    """Block bounds uint8 [n_pages][Hkv][page / block_tokens][2][D] of an empty
    cache (torch allocation)."""
    import torch
    if block_tokens < 16 or block_tokens % 16 or page % block_tokens:
        raise ValueError("block_tokens: a multiple of 16 that divides the page")
    return torch.zeros(n_pages, Hkv, page // block_tokens, 2, D, dtype=torch.uint8,
                       device=device or "cuda")


# What the calls below need of torch, looked up on first use (torch is imported
# lazily): these calls run once per layer and step, so their host time counts.
_torch = None
_CODES = {}      # torch dtype -> vae4_dtype, where the cache's bytes are E4M3
_CODES_E5M2 = {}  # and where they are E5M2
_raw_stream = None
_device = None
# a vae4_tensor of n dimensions: data, dtype | ndim << 32, shape[5], stride[5]
_PACK = [struct.Struct(f"=2q{n}q{40 - 8 * n}x{n}q{40 - 8 * n}x").pack for n in range(6)]


def _setup():
    global _torch, _raw_stream, _device
    import torch
    for codes, fp8 in ((_CODES, torch.float8_e4m3fn), (_CODES_E5M2, torch.float8_e5m2)):
        codes.update({torch.uint8: VAE4_U8, torch.int32: VAE4_I32, torch.float16: VAE4_F16,
                      torch.float32: VAE4_F32, torch.bfloat16: VAE4_BF16, fp8: VAE4_U8})
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda dev: torch.cuda.current_stream(dev).cuda_stream)
    _device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _torch = torch


def _call(name, tensors, rest, stream, flags=0, opt=None):
    """lib.verify_attn_e4m3_<name>(tensors..., rest..., stream[, opt]), the
    tensors (None: a null pointer) as packed vae4_tensor structures.  Every
    tensor has to be on the current device, and one of an FP8 type of the
    format that ``flags`` gives the cache (uint8 is either)."""
    if _torch is None:
        _setup()
    codes = _CODES_E5M2 if flags & FLAG_KV_E5M2 else _CODES
    args, dev = [], None
    for t in tensors:
        if t is None:
            args.append(None)
            continue
        code = codes.get(t.dtype)
        if code is None:
            if t.dtype in _CODES or t.dtype in _CODES_E5M2:
                raise TypeError(f"{t.dtype} beside flags of the other FP8 format")
            raise TypeError(f"unsupported dtype {t.dtype}")
        d = t.get_device()
        if d != dev:
            dev = d if dev is None else -1
        shape = t.shape
        n = len(shape)
        if n > 5:
            raise ValueError("at most 5 dimensions")
        args.append(_PACK[n](t.data_ptr(), code | n << 32, *shape, *t.stride()))
    if dev is None or dev < 0:
        raise ValueError("tensors have to be on one CUDA device")
    if dev != _device():
        raise ValueError("tensors have to be on the current device")
    st = _raw_stream(dev) if stream is None else _stream_handle(stream)
    fn = getattr(_lib or load(), name)
    rc = fn(*args, *rest, st) if opt is None else fn(*args, *rest, st, ctypes.byref(opt))
    if rc != 0:
        raise Vae4Error(rc, name)


def _status_pointer(status):
    if status is None:
        return None
    if _torch is None:
        _setup()
    dev = status.get_device()
    if status.dtype != _torch.int32 or status.numel() < 1 or dev < 0 or dev != _device():
        raise ValueError("status: an int32 tensor on the current device")
    return status.data_ptr()


def verify_attn_e4m3_append(k_new, v_new, k_cache, v_cache, block_table, seq_lens, block_scales, *,
                            k_bounds=None, status=None, flags: int = 0, stream=None):
    """Quantise new K and V rows (f16 or bf16 [B][Qmax][Hkv][D]) into the
    block-scaled cache, its scales and (optionally) its bounds, in place; see
    the header.  ``status``: an optional int32 device tensor whose first
    element receives the status bits."""
    _call("verify_attn_e4m3_append", (k_new, v_new, k_cache, v_cache, block_table, seq_lens,
                                      block_scales, k_bounds),
          (_status_pointer(status), flags), stream, flags)


def verify_attn_e4m3_block_scaled(q, k_cache, v_cache, block_table, seq_lens, block_scales, out,
                                  workspace, *, softmax_scale: float = 0.0,
                                  max_seq_len: int = 0, num_sms: int = 0, flags: int = 0,
                                  stream=None):
    """The verify step over a cache with one scale per block of tokens and KV
    head (f32 [n_pages][2][Hkv][page / block]) into ``out``; other arguments
    as verify_attn_e4m3_kv.  ``workspace`` from alloc_workspace."""
    opt = Options(softmax_scale, 0, max_seq_len, num_sms, flags, 0)
    _call("verify_attn_e4m3_block_scaled", (q, k_cache, v_cache, block_table, seq_lens,
                                            block_scales, out, workspace), (), stream, flags, opt)
    return out


def verify_attn_e4m3_sparse(q, k_cache, v_cache, block_table, seq_lens, block_scales, block_ids,
                            out, workspace, *, softmax_scale: float = 0.0, max_seq_len: int = 0,
                            num_sms: int = 0, flags: int = 0, stream=None):
    """Block-scaled attention in which each query attends only to the blocks
    that ``block_ids`` (int32 [B][Qmax][Hkv][k]) lists for it; see the header.
    ``workspace`` from alloc_sparse_workspace."""
    opt = Options(softmax_scale, 0, max_seq_len, num_sms, flags, 0)
    _call("verify_attn_e4m3_sparse", (q, k_cache, v_cache, block_table, seq_lens, block_scales,
                                      block_ids, out, workspace), (), stream, flags, opt)
    return out


def verify_attn_e4m3_block_scores(q, k_bounds, block_table, seq_lens, block_scales, scores, *,
                                  block_tokens: int, softmax_scale: float = 0.0, status=None,
                                  flags: int = 0, stream=None):
    """Scores (f32 [B][Qmax][Hkv][columns]) of every block for every query: an
    upper bound of the group's logits in the block; see the header."""
    _call("verify_attn_e4m3_block_scores", (q, k_bounds, block_table, seq_lens, block_scales,
                                            scores),
          (block_tokens, softmax_scale, _status_pointer(status), flags), stream, flags)
    return scores


def verify_attn_e4m3_select_blocks(scores, seq_lens, block_ids, *, block_tokens: int,
                                   sink_blocks: int = 0, local_blocks: int = 1, status=None,
                                   stream=None):
    """Fill ``block_ids`` (int32 [B][Qmax][Hkv][k]) with the k blocks each
    query attends to: the first ``sink_blocks`` and last ``local_blocks`` it
    sees, then the highest scores, equal ones by the lowest number; ascending,
    -1 padded.  See the header."""
    _call("verify_attn_e4m3_select_blocks", (scores, seq_lens, block_ids),
          (block_tokens, sink_blocks, local_blocks, _status_pointer(status)), stream)
    return block_ids


def verify_attn_e4m3_block_scaled_workspace_bytes(B, Hq, Hkv, Qmax, D, max_seq_len,
                                                  num_sms=0) -> int:
    n = load().verify_attn_e4m3_block_scaled_workspace_bytes(B, Hq, Hkv, Qmax, D, max_seq_len,
                                                             num_sms)
    if n < 0:
        raise Vae4Error(int(n), "block_scaled_workspace_bytes")
    return int(n)


block_scaled_workspace_bytes = verify_attn_e4m3_block_scaled_workspace_bytes


def verify_attn_e4m3_sparse_workspace_bytes(B, Hq, Hkv, Qmax, D, max_seq_len, block_tokens, blocks,
                                            num_sms=0) -> int:
    n = load().verify_attn_e4m3_sparse_workspace_bytes(B, Hq, Hkv, Qmax, D, max_seq_len,
                                                       block_tokens, blocks, num_sms)
    if n < 0:
        raise Vae4Error(int(n), "sparse_workspace_bytes")
    return int(n)


sparse_workspace_bytes = verify_attn_e4m3_sparse_workspace_bytes


def alloc_sparse_workspace(B, Hq, Hkv, Qmax, D, max_seq_len, block_tokens, blocks, device=None):
    """A zeroed workspace for verify_attn_e4m3_sparse (torch allocation,
    256-B aligned)."""
    import torch
    n = sparse_workspace_bytes(B, Hq, Hkv, Qmax, D, max_seq_len, block_tokens, blocks)
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")
