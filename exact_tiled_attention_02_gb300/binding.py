"""Python binding of libfa.so (the C ABI in include/fa.h).

Argument marshalling only: torch tensors become device pointers and sizes,
the ``stream`` keyword (a torch CUDA stream; by default the current one)
becomes the library's stream argument, and non-OK status codes become
``FaError``.  Every step of attention runs in the library's CUDA kernels;
there is no other code path.  PyTorch supplies device memory (outputs and
workspaces, allocated on the stream the call runs on) and streams.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfa.so")

FA_OK, FA_ERR_INVALID, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_TIMEOUT = range(5)
FA_DTYPE_F32, FA_DTYPE_BF16 = 0, 1

EXPORTS = ("fa_fwd", "fa_bwd", "fa_bwd_workspace_bytes", "fa_bwd_static_workspace", "fa_fwd_key_major",
           "fa_fwd_key_major_workspace_bytes", "fa_fwd_f32_3xtf32", "fa_fwd_f32_3xtf32_workspace_bytes",
           "fa_fwd_shared_prefix", "fa_fwd_shared_prefix_workspace_bytes", "fa_fwd_latent_absorbed",
           "fa_fwd_latent_absorbed_workspace_bytes", "fa_fwd_latent", "fa_bwd_latent", "fa_bwd_latent_workspace_bytes",
           "fa_last_device_status", "fa_set_wait_limit_us", "fa_selftest_wait_timeout", "fa_status_string",
           "fa_version")


class FaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {lib.fa_status_string(status).decode()}")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m exact_tiled_attention_02_gb300.build` "
                          "(or __graft_entry__.build()); there is no fallback implementation")
    L = ctypes.CDLL(LIB_PATH)
    vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    L.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, i, vp]
    L.fa_fwd.restype = i
    L.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, i, vp, sz, vp]
    L.fa_bwd.restype = i
    L.fa_bwd_static_workspace.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, i, vp]
    L.fa_bwd_static_workspace.restype = i
    L.fa_bwd_workspace_bytes.argtypes = [i, i, i, i]
    L.fa_bwd_workspace_bytes.restype = sz
    L.fa_fwd_key_major.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, i, vp, sz, vp]
    L.fa_fwd_key_major.restype = i
    L.fa_fwd_key_major_workspace_bytes.argtypes = [i, i, i, i]
    L.fa_fwd_key_major_workspace_bytes.restype = sz
    L.fa_fwd_f32_3xtf32.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp, sz, vp]
    L.fa_fwd_f32_3xtf32.restype = i
    L.fa_fwd_f32_3xtf32_workspace_bytes.argtypes = [i, i, i, i]
    L.fa_fwd_f32_3xtf32_workspace_bytes.restype = sz
    L.fa_fwd_shared_prefix.argtypes = [vp] * 8 + [i] * 7 + [f, i, vp, sz, vp]
    L.fa_fwd_shared_prefix.restype = i
    L.fa_fwd_shared_prefix_workspace_bytes.argtypes = [i] * 7
    L.fa_fwd_shared_prefix_workspace_bytes.restype = sz
    L.fa_fwd_latent_absorbed.argtypes = [vp] * 6 + [i] * 8 + [f, i, vp, sz, vp]
    L.fa_fwd_latent_absorbed.restype = i
    L.fa_fwd_latent_absorbed_workspace_bytes.argtypes = [i] * 6
    L.fa_fwd_latent_absorbed_workspace_bytes.restype = sz
    L.fa_fwd_latent.argtypes = [vp] * 6 + [i] * 7 + [f, i, i, vp]
    L.fa_fwd_latent.restype = i
    L.fa_bwd_latent.argtypes = [vp] * 11 + [i] * 7 + [f, i, i, vp, sz, vp]
    L.fa_bwd_latent.restype = i
    L.fa_bwd_latent_workspace_bytes.argtypes = [i] * 7
    L.fa_bwd_latent_workspace_bytes.restype = sz
    L.fa_last_device_status.argtypes = [vp]
    L.fa_last_device_status.restype = i
    L.fa_set_wait_limit_us.argtypes = [ctypes.c_longlong]
    L.fa_set_wait_limit_us.restype = ctypes.c_longlong
    L.fa_selftest_wait_timeout.argtypes = [i, vp]
    L.fa_selftest_wait_timeout.restype = i
    L.fa_status_string.argtypes = [i]
    L.fa_status_string.restype = ctypes.c_char_p
    L.fa_version.argtypes = []
    L.fa_version.restype = i
    return L


lib = _load()


@functools.lru_cache(maxsize=None)
def _torch():
    import torch
    return torch


def _stream_ptr(stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _alloc_on(stream):
    """Context for the tensors a call allocates (outputs, workspace): on the
    stream its kernels run on.  The caching allocator hands a freed block out
    again in the order of the stream it was allocated on; a workspace
    allocated on the current stream and dropped on return, while the kernels
    still run on another stream, could otherwise be reused at once."""
    torch = _torch()
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return FA_DTYPE_BF16
    if t.dtype == torch.float32:
        return FA_DTYPE_F32
    raise TypeError(f"unsupported dtype {t.dtype}: use torch.bfloat16 or torch.float32")


def _check_qkv(*ts):
    ref = ts[0]
    if ref.dim() != 4:
        raise ValueError("tensors must be [B, H, N, d]")
    for t in ts:
        if not t.is_cuda:
            raise ValueError("tensors must live on a CUDA device")
        if t.shape != ref.shape or t.dtype != ref.dtype or t.device != ref.device:
            raise ValueError("q, k, v (and o, dO, grads) must share shape, dtype and device")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous [B, H, N, d]")


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def fa_status_string(status: int) -> str:
    return lib.fa_status_string(int(status)).decode()


def fa_version() -> int:
    return lib.fa_version()


def fa_set_wait_limit_us(limit_us: int) -> int:
    return lib.fa_set_wait_limit_us(int(limit_us))


def fa_bwd_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return lib.fa_bwd_workspace_bytes(B, H, N, d)


def fa_fwd_key_major_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return lib.fa_fwd_key_major_workspace_bytes(B, H, N, d)


def fa_fwd_f32_3xtf32_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return lib.fa_fwd_f32_3xtf32_workspace_bytes(B, H, N, d)


def fa_last_device_status(stream=None) -> int:
    return lib.fa_last_device_status(_stream_ptr(stream))


def fa_selftest_wait_timeout(limit_us: int, stream=None) -> int:
    return lib.fa_selftest_wait_timeout(int(limit_us), _stream_ptr(stream))


def fa_fwd(q, k, v, scale: float | None = None, window: int = 0, o=None, lse=None, want_lse: bool = True,
           stream=None):
    """O = softmax(Q K^T * scale) V on the GPU; returns ``(o, lse)``.

    ``q, k, v``: contiguous [B, H, N, d] bf16 (d in {64, 96, 128, 256}) or float32
    (d <= 128) CUDA tensors.  ``scale`` defaults to 1/sqrt(d).  ``window``:
    0 = unmasked, else the odd full width of the local window.  ``o``/``lse``
    may be given to write into existing buffers; ``lse`` is float32 [B, H, N]
    (None when ``want_lse`` is false and none is given).
    """
    torch = _torch()
    _check_qkv(q, k, v)
    B, H, N, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    with _alloc_on(stream):
        if o is None:
            o = torch.empty_like(q)
        if lse is None and want_lse:
            lse = torch.empty((B, H, N), device=q.device, dtype=torch.float32)
    _check_qkv(q, o)
    if lse is not None and (lse.dtype != torch.float32 or not lse.is_contiguous() or lse.numel() != B * H * N):
        raise ValueError("lse must be a contiguous float32 [B, H, N] tensor")
    st = lib.fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d, float(scale), int(window),
                    _dtype_code(q), _stream_ptr(stream))
    if st != FA_OK:
        raise FaError(st, "fa_fwd")
    return o, lse


def fa_fwd_key_major(q, k, v, scale: float | None = None, window: int = 0, o=None, lse=None, want_lse: bool = True,
                     workspace=None, stream=None):
    """The forward pass in the key-major loop order (a comparison schedule,
    bf16 with d = 64 or 128); same results as ``fa_fwd``.  The fp32 workspace
    for the running statistics is taken from ``workspace`` (a CUDA uint8
    tensor of at least ``fa_fwd_key_major_workspace_bytes`` bytes) or
    allocated here with torch."""
    torch = _torch()
    _check_qkv(q, k, v)
    B, H, N, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    with _alloc_on(stream):
        if o is None:
            o = torch.empty_like(q)
        if lse is None and want_lse:
            lse = torch.empty((B, H, N), device=q.device, dtype=torch.float32)
        if workspace is None:
            workspace = torch.empty(fa_fwd_key_major_workspace_bytes(B, H, N, d), device=q.device, dtype=torch.uint8)
    _check_qkv(q, o)
    if lse is not None and (lse.dtype != torch.float32 or not lse.is_contiguous() or lse.numel() != B * H * N):
        raise ValueError("lse must be a contiguous float32 [B, H, N] tensor")
    st = lib.fa_fwd_key_major(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d, float(scale), int(window),
                              _dtype_code(q), _ptr(workspace), workspace.numel() * workspace.element_size(),
                              _stream_ptr(stream))
    if st != FA_OK:
        raise FaError(st, "fa_fwd_key_major")
    return o, lse


def fa_fwd_f32_3xtf32(q, k, v, scale: float | None = None, window: int = 0, o=None, lse=None, want_lse: bool = True,
                      workspace=None, stream=None):
    """float32 forward on the tensor cores by the 3xTF32 split (d <= 64);
    same operation and outputs as ``fa_fwd`` on float32 tensors.  The
    workspace (split copies of Q, K, V) is taken from ``workspace`` (a CUDA
    uint8 tensor of at least ``fa_fwd_f32_3xtf32_workspace_bytes`` bytes) or
    allocated here with torch."""
    torch = _torch()
    _check_qkv(q, k, v)
    if q.dtype != torch.float32:
        raise TypeError("fa_fwd_f32_3xtf32 takes float32 tensors")
    B, H, N, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    with _alloc_on(stream):
        if o is None:
            o = torch.empty_like(q)
        if lse is None and want_lse:
            lse = torch.empty((B, H, N), device=q.device, dtype=torch.float32)
        if workspace is None:
            workspace = torch.empty(fa_fwd_f32_3xtf32_workspace_bytes(B, H, N, d), device=q.device, dtype=torch.uint8)
    _check_qkv(q, o)
    if lse is not None and (lse.dtype != torch.float32 or not lse.is_contiguous() or lse.numel() != B * H * N):
        raise ValueError("lse must be a contiguous float32 [B, H, N] tensor")
    st = lib.fa_fwd_f32_3xtf32(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d, float(scale), int(window),
                               _ptr(workspace), workspace.numel() * workspace.element_size(), _stream_ptr(stream))
    if st != FA_OK:
        raise FaError(st, "fa_fwd_f32_3xtf32")
    return o, lse


def fa_bwd(q, k, v, o, lse, do, scale: float | None = None, window: int = 0, dq=None, dk=None, dv=None,
           workspace=None, stream=None):
    """Gradients (dQ, dK, dV) of the forward above, by recomputation.

    ``o`` and ``lse`` are the forward's outputs; ``do`` is dL/dO.  The
    workspace (float32 dQ accumulator + row sums) is taken from ``workspace``
    (a CUDA uint8 tensor of at least ``fa_bwd_workspace_bytes`` bytes) or
    allocated here with torch.
    """
    torch = _torch()
    _check_qkv(q, k, v, o, do)
    B, H, N, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if lse.dtype != torch.float32 or not lse.is_contiguous() or lse.numel() != B * H * N:
        raise ValueError("lse must be a contiguous float32 [B, H, N] tensor")
    need = fa_bwd_workspace_bytes(B, H, N, d)
    with _alloc_on(stream):
        dq = torch.empty_like(q) if dq is None else dq
        dk = torch.empty_like(q) if dk is None else dk
        dv = torch.empty_like(q) if dv is None else dv
        if workspace is None:
            workspace = torch.empty(need, device=q.device, dtype=torch.uint8)
    _check_qkv(q, dq, dk, dv)
    st = lib.fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk), _ptr(dv),
                    B, H, N, d, float(scale), int(window), _dtype_code(q), _ptr(workspace),
                    workspace.numel() * workspace.element_size(), _stream_ptr(stream))
    if st != FA_OK:
        raise FaError(st, "fa_bwd")
    return dq, dk, dv


def fa_bwd_static_workspace(q, k, v, o, lse, do, dq, dk, dv, scale: float | None = None, window: int = 0,
                            stream=None):
    """fa_bwd without a workspace argument, for callers that cannot allocate
    device memory: the library's fixed 64 MiB scratch array stands in for the
    workspace, and neither this wrapper nor the library allocates anything
    (the caller passes the dq, dk, dv outputs).  Calls that overlap on the GPU
    share that array and race; problems needing more than 64 MiB of workspace
    raise FaError(FA_ERR_UNSUPPORTED)."""
    torch = _torch()
    _check_qkv(q, k, v, o, do, dq, dk, dv)
    B, H, N, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if lse.dtype != torch.float32 or not lse.is_contiguous() or lse.numel() != B * H * N:
        raise ValueError("lse must be a contiguous float32 [B, H, N] tensor")
    st = lib.fa_bwd_static_workspace(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk),
                                     _ptr(dv), B, H, N, d, float(scale), int(window), _dtype_code(q),
                                     _stream_ptr(stream))
    if st != FA_OK:
        raise FaError(st, "fa_bwd_static_workspace")
    return dq, dk, dv


@functools.lru_cache(maxsize=256)
def fa_fwd_shared_prefix_workspace_bytes(B: int, Hq: int, Hkv: int, Nq: int, Np: int, Ns: int, d: int) -> int:
    return lib.fa_fwd_shared_prefix_workspace_bytes(B, Hq, Hkv, Nq, Np, Ns, d)


@functools.lru_cache(maxsize=256)
def fa_fwd_latent_absorbed_workspace_bytes(B: int, H: int, Nq: int, page_size: int, max_pages: int, dc: int) -> int:
    return lib.fa_fwd_latent_absorbed_workspace_bytes(B, H, Nq, page_size, max_pages, dc)


@functools.lru_cache(maxsize=256)
def fa_bwd_latent_workspace_bytes(B: int, H: int, Nq: int, Nk: int, dn: int, dr: int, dv: int) -> int:
    return lib.fa_bwd_latent_workspace_bytes(B, H, Nq, Nk, dn, dr, dv)


def _at(t):
    return 0 if t is None else t.data_ptr()


def _need(name, t, shape, dtype, device):
    if t.shape == shape and t.dtype == dtype and t.device == device and t.is_contiguous():
        return t
    raise ValueError(f"{name} must be a contiguous {dtype} {tuple(shape)} tensor on {device}, "
                     f"not {t.dtype} {tuple(t.shape)} on {t.device}")


def _first(name, t, dims):
    """The tensor that sets a call's dtype and device: its dtype code."""
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, not {t.dim()}")
    code = _dtype_code(t)
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return code


def _current_stream(device, stream):
    """The handle of the stream a call runs on where nothing has to be made
    current for it: no stream given, the tensors on the current device."""
    torch = _torch()
    if stream is not None or torch._C._cuda_getDevice() != device.index:
        return None
    return torch._C._cuda_getCurrentRawStream(device.index)


@contextlib.contextmanager
def _made_current(device, stream):
    """The tensors' device, and the stream if one is given, made current: the
    call's work and the tensors it allocates go there (see _alloc_on)."""
    torch = _torch()
    if stream is not None and stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {device}")
    with torch.cuda.device(device), _alloc_on(stream):
        yield


class _Workspace:
    """A call's workspace: the tensor given, or a block of torch's caching
    allocator on the call's stream, handed back on leaving (calls queued later
    on that stream may reuse it in order).  Taken without a tensor around it: a
    tensor costs 6 us more beside a kernel launch."""

    __slots__ = ("at", "bytes", "block")

    def __init__(self, workspace, need, device, stream_ptr):
        self.block = None
        if workspace is None:
            self.block = self.at = _torch()._C._cuda_cudaCachingAllocator_raw_alloc(need, stream_ptr)
            self.bytes = need
        else:
            if workspace.device != device or not workspace.is_contiguous():
                raise ValueError(f"workspace must be a contiguous tensor on {device}")
            self.at, self.bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        if self.block:
            _torch()._C._cuda_cudaCachingAllocator_raw_delete(self.block)


def fa_fwd_shared_prefix(q, k_prefix, v_prefix, k, v, lens, scale: float | None = None, o=None, lse=None,
                         want_lse: bool = True, workspace=None, stream=None):
    """Attention of a decoding batch whose sequences share one prefix; returns ``(o, lse)``.

    ``q``: [B, Hq, Nq, d], each sequence's Nq new tokens; ``k_prefix,
    v_prefix``: [Hkv, Np, d], seen by every row and read once for the batch;
    ``k, v``: [B, Hkv, Ns, d], each sequence's own keys and values (the new
    tokens' included), of which ``lens[b]`` (int32 [B]) are valid.  Query
    token t sees the prefix and its own keys j < lens[b] - (Nq - 1 - t).  bf16
    (d in {64, 96, 128}) or float32 (d <= 128), contiguous, on one device.
    ``scale`` defaults to 1/sqrt(d).  ``workspace``: a CUDA uint8 tensor of at
    least ``fa_fwd_shared_prefix_workspace_bytes`` bytes, or allocated here.
    """
    torch = _torch()
    code = _first("q", q, 4)
    dev = q.device
    sp = _current_stream(dev, stream)
    if sp is None:
        with _made_current(dev, stream):
            return fa_fwd_shared_prefix(q, k_prefix, v_prefix, k, v, lens, scale, o, lse, want_lse, workspace)
    if k_prefix.dim() != 3 or k.dim() != 4:
        raise ValueError("k_prefix must be [Hkv, Np, d] and k [B, Hkv, Ns, d]")
    B, Hq, Nq, d = q.shape
    Hkv, Np, _ = k_prefix.shape
    Ns, t = k.shape[2], q.dtype
    _need("k_prefix", k_prefix, (Hkv, Np, d), t, dev)
    _need("v_prefix", v_prefix, (Hkv, Np, d), t, dev)
    _need("k", k, (B, Hkv, Ns, d), t, dev)
    _need("v", v, (B, Hkv, Ns, d), t, dev)
    _need("lens", lens, (B,), torch.int32, dev)
    o = torch.empty_like(q) if o is None else _need("o", o, (B, Hq, Nq, d), t, dev)
    if lse is not None:
        _need("lse", lse, (B, Hq, Nq), torch.float32, dev)
    elif want_lse:
        lse = q.new_empty((B, Hq, Nq), dtype=torch.float32)
    with _Workspace(workspace, fa_fwd_shared_prefix_workspace_bytes(B, Hq, Hkv, Nq, Np, Ns, d), dev, sp) as ws:
        st = lib.fa_fwd_shared_prefix(_at(q), _at(k_prefix), _at(v_prefix), _at(k), _at(v), _at(lens), _at(o), _at(lse),
                                      B, Hq, Hkv, Nq, Np, Ns, d, 1.0 / math.sqrt(d) if scale is None else scale, code,
                                      ws.at, ws.bytes, sp)
    if st != FA_OK:
        raise FaError(st, "fa_fwd_shared_prefix")
    return o, lse


def fa_fwd_latent_absorbed(q, cache, lens, dc: int, scale: float, block_table=None, o=None, lse=None,
                           want_lse: bool = True, workspace=None, stream=None):
    """Latent attention, absorbed form, over a paged cache; returns ``(o, lse)``.

    ``q``: [B, H, Nq, dc+dr], each sequence's Nq new tokens; ``cache``:
    [pages, page_size, dc+dr], one vector a token, whose first ``dc`` entries
    are also the value; ``block_table``: int32 [B, max_pages], or None when
    sequence b is page b; ``lens``: int32 [B], tokens in the cache, the new
    ones included.  ``o`` is [B, H, Nq, dc].  bf16 (dc 256 or 512, dr 64, pages
    of a multiple of 16 tokens) or float32 (dc <= 512, dr <= 128).  ``scale``
    is the expanded head's.  ``workspace``: at least
    ``fa_fwd_latent_absorbed_workspace_bytes`` bytes, or allocated here.
    """
    torch = _torch()
    code = _first("q", q, 4)
    dev = q.device
    sp = _current_stream(dev, stream)
    if sp is None:
        with _made_current(dev, stream):
            return fa_fwd_latent_absorbed(q, cache, lens, dc, scale, block_table, o, lse, want_lse, workspace)
    B, H, Nq, dk = q.shape
    if cache.dim() != 3 or not 0 < dc < dk:
        raise ValueError("cache must be [pages, page_size, dc + dr], with 0 < dc < dc + dr")
    pages, page_size, _ = cache.shape
    _need("cache", cache, (pages, page_size, dk), q.dtype, dev)
    _need("lens", lens, (B,), torch.int32, dev)
    max_pages = 1
    if block_table is not None:
        if block_table.dim() != 2:
            raise ValueError("block_table must be [B, max_pages]")
        max_pages = block_table.shape[1]
        _need("block_table", block_table, (B, max_pages), torch.int32, dev)
    o = q.new_empty((B, H, Nq, dc)) if o is None else _need("o", o, (B, H, Nq, dc), q.dtype, dev)
    if lse is not None:
        _need("lse", lse, (B, H, Nq), torch.float32, dev)
    elif want_lse:
        lse = q.new_empty((B, H, Nq), dtype=torch.float32)
    need = fa_fwd_latent_absorbed_workspace_bytes(B, H, Nq, page_size, max_pages, dc)
    with _Workspace(workspace, need, dev, sp) as ws:
        st = lib.fa_fwd_latent_absorbed(_at(q), _at(cache), _at(block_table), _at(lens), _at(o), _at(lse), B, H, Nq,
                                        pages, page_size, max_pages, dc, dk - dc, scale, code, ws.at, ws.bytes, sp)
    if st != FA_OK:
        raise FaError(st, "fa_fwd_latent_absorbed")
    return o, lse


def _check_latent(q, k_nope, k_rope, v):
    code = _first("q", q, 4)
    if k_nope.dim() != 4 or v.dim() != 4:
        raise ValueError("k_nope and v must be [B, H, Nk, d]")
    B, H, Nq, dk = q.shape
    Nk, dn, dv = k_nope.shape[2], k_nope.shape[3], v.shape[3]
    if not 0 < dn < dk:
        raise ValueError("q must be [B, H, Nq, dn + dr]")
    _need("k_nope", k_nope, (B, H, Nk, dn), q.dtype, q.device)
    _need("k_rope", k_rope, (B, Nk, dk - dn), q.dtype, q.device)
    _need("v", v, (B, H, Nk, dv), q.dtype, q.device)
    return code, (B, H, Nq, Nk, dn, dk - dn, dv)


def fa_fwd_latent(q, k_nope, k_rope, v, scale: float | None = None, causal: bool = True, o=None, lse=None,
                  want_lse: bool = True, stream=None):
    """Latent attention, expanded form; returns ``(o, lse)``.

    ``q``: [B, H, Nq, dn+dr]; ``k_nope``: [B, H, Nk, dn]; ``k_rope``: [B, Nk,
    dr], shared by the heads; ``v``: [B, H, Nk, dv]; ``o``: [B, H, Nq, dv].
    ``causal``: row i sees keys j <= i + Nk - Nq (sequences padded on the right
    may share a call where their pasts, keys less queries, are equal).  bf16
    (dn = 128, dr = 64, dv = 128) or float32 (dn + dr <= 256, dv <= 128).
    ``scale`` defaults to 1/sqrt(dn + dr).
    """
    torch = _torch()
    code, (B, H, Nq, Nk, dn, dr, dv) = _check_latent(q, k_nope, k_rope, v)
    dev = q.device
    sp = _current_stream(dev, stream)
    if sp is None:
        with _made_current(dev, stream):
            return fa_fwd_latent(q, k_nope, k_rope, v, scale, causal, o, lse, want_lse)
    o = q.new_empty((B, H, Nq, dv)) if o is None else _need("o", o, (B, H, Nq, dv), q.dtype, dev)
    if lse is not None:
        _need("lse", lse, (B, H, Nq), torch.float32, dev)
    elif want_lse:
        lse = q.new_empty((B, H, Nq), dtype=torch.float32)
    st = lib.fa_fwd_latent(_at(q), _at(k_nope), _at(k_rope), _at(v), _at(o), _at(lse), B, H, Nq, Nk, dn, dr, dv,
                           1.0 / math.sqrt(dn + dr) if scale is None else scale, bool(causal), code, sp)
    if st != FA_OK:
        raise FaError(st, "fa_fwd_latent")
    return o, lse


def fa_bwd_latent(q, k_nope, k_rope, v, o, lse, do, scale: float | None = None, causal: bool = True, dq=None,
                  dk_nope=None, dk_rope=None, dv=None, workspace=None, stream=None):
    """Gradients ``(dq, dk_nope, dk_rope, dv)`` of ``fa_fwd_latent``, by
    recomputation from its outputs ``o`` and ``lse`` and ``do`` = dL/dO.  The
    workspace (at least ``fa_bwd_latent_workspace_bytes`` bytes) is taken from
    ``workspace`` or allocated here."""
    torch = _torch()
    code, (B, H, Nq, Nk, dn, dr, dvw) = _check_latent(q, k_nope, k_rope, v)
    dev = q.device
    sp = _current_stream(dev, stream)
    if sp is None:
        with _made_current(dev, stream):
            return fa_bwd_latent(q, k_nope, k_rope, v, o, lse, do, scale, causal, dq, dk_nope, dk_rope, dv, workspace)
    _need("o", o, (B, H, Nq, dvw), q.dtype, dev)
    _need("do", do, (B, H, Nq, dvw), q.dtype, dev)
    _need("lse", lse, (B, H, Nq), torch.float32, dev)
    dq, dk_nope, dk_rope, dv = (torch.empty_like(t) if g is None else _need(name, g, t.shape, q.dtype, dev)
                                for name, g, t in (("dq", dq, q), ("dk_nope", dk_nope, k_nope),
                                                   ("dk_rope", dk_rope, k_rope), ("dv", dv, v)))
    with _Workspace(workspace, fa_bwd_latent_workspace_bytes(B, H, Nq, Nk, dn, dr, dvw), dev, sp) as ws:
        st = lib.fa_bwd_latent(_at(q), _at(k_nope), _at(k_rope), _at(v), _at(o), _at(lse), _at(do), _at(dq),
                               _at(dk_nope), _at(dk_rope), _at(dv), B, H, Nq, Nk, dn, dr, dvw,
                               1.0 / math.sqrt(dn + dr) if scale is None else scale, bool(causal), code, ws.at,
                               ws.bytes, sp)
    if st != FA_OK:
        raise FaError(st, "fa_bwd_latent")
    return dq, dk_nope, dk_rope, dv
