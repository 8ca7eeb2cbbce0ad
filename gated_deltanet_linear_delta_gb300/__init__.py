"""GB300 (sm_103a) gated delta rule layer: thin Python binding of the C ABI.

Every function here only marshals arguments (shapes, dtypes, device pointers,
the current CUDA stream) and calls the entry point of the same name in
``libgdn_gb300.so`` (declared in ``include/gdn.h``). All arithmetic runs in
the library's CUDA kernels. There is no CPU fallback: if the library is not
built, every call raises.

Tensors are torch CUDA tensors, contiguous, in the layouts of ``gdn.h``:
q, k [Ttot, Hk, dk]; v, out [Ttot, Hv, dv]; g, b [Ttot, Hv] (bf16 or fp32,
all the same dtype); states [B, Hv, dv, dk] fp32; cu_seqlens int32 [B+1];
paged caches [num_pages, Hkv, page_size, d] (the packed rows of the cache calls
may have a token stride of their own).

The per-call host cost is kept small because a decode step of a few
sequences runs in a few microseconds on the GPU: the library handle and its
function objects are looked up once, pointers go to ctypes as plain integers,
and the current stream is read as a raw handle. Size and alignment checks are
the C library's (it returns an error before queueing anything). The paged cache
calls and the calls on trees, which have the most tensors, are marshalled in C++
(csrc/binding.cpp).
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import threading

import torch

from . import _build

__all__ = ["GDNError", "gdn_prefill", "gdn_prefill_ws", "gdn_prefill_workspace_size", "gdn_prefill_static",
           "gdn_prefill_from_host",
           "gdn_decode_step", "gdn_decode_step_slots", "gdn_prepass", "gdn_prefill_path",
           "gdn_kv_write", "gdn_kv_read", "gdn_paged_attn", "gdn_paged_attn_workspace_size",
           "gdn_tree_attn", "gdn_tree_scan", "gdn_tree_verify", "gdn_tree_advance", "gdn_kv_keep",
           "gdn_get_device_status", "gdn_status_string", "library", "library_path",
           "GDN_OK", "GDN_ERR_INVALID_ARG", "GDN_ERR_UNSUPPORTED", "GDN_ERR_CUDA",
           "GDN_ERR_DEVICE_CHECK", "GDN_BF16", "GDN_F32", "GDN_FP8", "GDN_INT8"]

GDN_OK, GDN_ERR_INVALID_ARG, GDN_ERR_UNSUPPORTED, GDN_ERR_CUDA, GDN_ERR_DEVICE_CHECK = 0, -1, -2, -3, -4
GDN_BF16, GDN_F32, GDN_FP8, GDN_INT8 = 0, 1, 2, 3

_lock = threading.Lock()
_lib: ctypes.CDLL | None = None

_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_int64
_calls = None
_DTYPE = {torch.bfloat16: GDN_BF16, torch.float32: GDN_F32}
# the current stream of a device as a raw cudaStream_t (falls back to the Stream object)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


class GDNError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where} returned {gdn_status_string(status)} ({status})")


def library_path() -> str:
    return _build.lib_path()


def library() -> ctypes.CDLL:
    """Load libgdn_gb300.so (built by ``__graft_entry__.build()``); raise if it is missing."""
    global _lib
    lib = _lib
    if lib is not None:
        return lib
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise RuntimeError(f"the CUDA library {path} is not built; run __graft_entry__.build()")
            lib = ctypes.CDLL(path)
            lib.gdn_prefill.argtypes = [_P] * 9 + [_I] * 8 + [_P]
            lib.gdn_prefill.restype = _I
            lib.gdn_prefill_static.argtypes = [_P] * 9 + [_I] * 8 + [_P]
            lib.gdn_prefill_static.restype = _I
            lib.gdn_prefill_ws.argtypes = [_P] * 9 + [_I] * 8 + [_P, ctypes.c_size_t, _P]
            lib.gdn_prefill_ws.restype = _I
            lib.gdn_prefill_workspace_size.argtypes = [_I] * 8
            lib.gdn_prefill_workspace_size.restype = ctypes.c_size_t
            lib.gdn_decode_step.argtypes = [_P] * 7 + [_I] * 6 + [_P]
            lib.gdn_decode_step.restype = _I
            lib.gdn_prefill_from_host.argtypes = [_P] * 15 + [_I] * 8 + [_P]
            lib.gdn_prefill_from_host.restype = _I
            lib.gdn_decode_step_slots.argtypes = [_P] * 8 + [_I] * 7 + [_P]
            lib.gdn_decode_step_slots.restype = _I
            lib.gdn_prepass.argtypes = [_P] * 5 + [_I] * 7 + [_P] * 4 + [_P]
            lib.gdn_prepass.restype = _I
            lib.gdn_prefill_path.argtypes = [_I] * 8
            lib.gdn_prefill_path.restype = _I
            lib.gdn_kv_write.argtypes = [_P] * 9 + [_I] * 7 + [_L] * 2 + [_I] * 2 + [_P]
            lib.gdn_kv_write.restype = _I
            lib.gdn_kv_read.argtypes = [_P] * 9 + [_I] * 7 + [_L] * 2 + [_I] * 2 + [_P]
            lib.gdn_kv_read.restype = _I
            lib.gdn_paged_attn.argtypes = [_P] * 9 + [_I] * 8 + [_L, ctypes.c_float] + [_I] * 2 + \
                [_P, ctypes.c_size_t, _P]
            lib.gdn_paged_attn.restype = _I
            lib.gdn_paged_attn_workspace_size.argtypes = [_I] * 6
            lib.gdn_paged_attn_workspace_size.restype = ctypes.c_size_t
            lib.gdn_tree_attn.argtypes = [_P] * 10 + [_I] * 8 + [_L, ctypes.c_float] + [_I] * 2 + \
                [_P, ctypes.c_size_t, _P]
            lib.gdn_tree_attn.restype = _I
            lib.gdn_kv_keep.argtypes = [_P] * 9 + [_I] * 9 + [_P]
            lib.gdn_kv_keep.restype = _I
            lib.gdn_tree_scan.argtypes = [_P] * 10 + [_I] * 8 + [_P]
            lib.gdn_tree_scan.restype = _I
            lib.gdn_tree_advance.argtypes = [_P] * 10 + [_I] * 9 + [_P]
            lib.gdn_tree_advance.restype = _I
            lib.gdn_tree_verify.argtypes = [_P] * 10 + [_I] * 3 + [_L] * 2 + [_I, _P]
            lib.gdn_tree_verify.restype = _I
            lib.gdn_get_device_status.argtypes = [_P]
            lib.gdn_get_device_status.restype = _I
            lib.gdn_status_string.argtypes = [_I]
            lib.gdn_status_string.restype = ctypes.c_char_p
            _lib = lib
        return _lib


def gdn_status_string(status: int) -> str:
    return library().gdn_status_string(int(status)).decode()


def _dtype_code(t: torch.Tensor) -> int:
    code = _DTYPE.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}: use bfloat16 or float32")
    return code


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not (t.is_cuda and t.is_contiguous()):
        raise ValueError("tensors must be contiguous CUDA tensors")
    return t.data_ptr()


def _current_device() -> int:
    """The current CUDA device. The first call replaces this function by the quickest one that tells (of one device: 0)."""
    global _current_device
    _current_device = int if torch.cuda.device_count() == 1 else getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    return _current_device()


def _stream(stream, t: torch.Tensor | None = None):
    """cudaStream_t of `stream`, or of the current stream. The library launches on the current device, so a call
    whose tensor t lies on another one is refused here (its kernels would run where the tensors are not)."""
    device = _current_device()
    if t is not None and t.get_device() != device:
        raise ValueError("tensors must be on the current CUDA device (torch.cuda.set_device)")
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(device)
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _torch_stream(stream, t: torch.Tensor):
    """The torch stream object of `stream` (memory taken under it is not handed on before its work is done)."""
    if stream is None:
        return torch.cuda.current_stream(t.device)
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(_stream(stream), device=t.device)


def _check(rc: int, where: str) -> None:
    if rc != GDN_OK:
        raise GDNError(rc, where)


def _prefill_sizes(q, v, g, b, out, state_in, state_out, cu_seqlens, B, T):
    Ttot, Hk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int32:
            raise TypeError("cu_seqlens must be int32")
        B, T = cu_seqlens.numel() - 1, Ttot
    else:
        B = 1 if B is None else B
        T = Ttot // B if T is None else T
    for t in (v, g, b, out):
        if t.dtype != q.dtype:
            raise TypeError("q, k, v, g, b and out must share one dtype")
    for t in (state_in, state_out):
        if t is not None and t.dtype != torch.float32:
            raise TypeError("states are fp32")
    return B, T, Hk, Hv, dk, dv


def gdn_prefill(q, k, v, g, b, state_in, state_out, out, cu_seqlens=None, B=None, T=None, chunk=64,
                stream=None) -> None:
    """Chunked prefill over packed sequences; writes `out` and `state_out` (may alias state_in)."""
    lib = _lib or library()
    if k.dtype != q.dtype:
        raise TypeError("q, k, v, g, b and out must share one dtype")
    B, T, Hk, Hv, dk, dv = _prefill_sizes(q, v, g, b, out, state_in, state_out, cu_seqlens, B, T)
    rc = lib.gdn_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(b), _ptr(state_in), _ptr(state_out), _ptr(out),
                         _ptr(cu_seqlens), B, T, Hk, Hv, dk, dv, chunk, _dtype_code(q), _stream(stream, q))
    _check(rc, "gdn_prefill")


def gdn_prefill_static(q, k, v, g, b, state_in, state_out, out, cu_seqlens=None, B=None, T=None, chunk=64,
                       stream=None) -> None:
    """gdn_prefill that allocates nothing at call time: the tensor-core path's scratch is a fixed
    array in the library's device image, shared by all calls on a device (overlapping calls race)."""
    lib = _lib or library()
    if k.dtype != q.dtype:
        raise TypeError("q, k, v, g, b and out must share one dtype")
    B, T, Hk, Hv, dk, dv = _prefill_sizes(q, v, g, b, out, state_in, state_out, cu_seqlens, B, T)
    rc = lib.gdn_prefill_static(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(b), _ptr(state_in), _ptr(state_out),
                                _ptr(out), _ptr(cu_seqlens), B, T, Hk, Hv, dk, dv, chunk, _dtype_code(q),
                                _stream(stream, q))
    _check(rc, "gdn_prefill_static")


def gdn_prefill_workspace_size(B, T, Hk, Hv, dk, dv, chunk, dtype) -> int:
    """Bytes of device workspace gdn_prefill_ws needs for these sizes (0: none)."""
    if isinstance(dtype, torch.dtype):
        dtype = _DTYPE[dtype]
    return int(library().gdn_prefill_workspace_size(B, T, Hk, Hv, dk, dv, chunk, int(dtype)))


def gdn_prefill_ws(q, k, v, g, b, state_in, state_out, out, workspace, cu_seqlens=None, B=None, T=None, chunk=64,
                   stream=None) -> None:
    """gdn_prefill with a caller-owned device workspace (a uint8 CUDA tensor, or None when none is needed)."""
    lib = _lib or library()
    if k.dtype != q.dtype:
        raise TypeError("q, k, v, g, b and out must share one dtype")
    B, T, Hk, Hv, dk, dv = _prefill_sizes(q, v, g, b, out, state_in, state_out, cu_seqlens, B, T)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib.gdn_prefill_ws(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(b), _ptr(state_in), _ptr(state_out), _ptr(out),
                            _ptr(cu_seqlens), B, T, Hk, Hv, dk, dv, chunk, _dtype_code(q), _ptr(workspace), nbytes,
                            _stream(stream, q))
    _check(rc, "gdn_prefill_ws")


def _host_ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if t.is_cuda or not t.is_contiguous():
        raise ValueError("host arrays must be contiguous CPU tensors")
    return t.data_ptr()


def gdn_prefill_from_host(q, k, v, g, b, state_in, state_out, out, dev, chunk=64, fragment=1024,
                          stream=None) -> None:
    """Prefill of one sequence from host tensors (pinned for overlap): q..b, state_in (or None),
    state_out and out are CPU tensors; `dev` holds the device buffers of the same shapes (keys
    q, k, v, g, b, out, state). Copies overlap the computation fragment by fragment."""
    T, Hk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    for t in (state_in, state_out):
        if t is not None and t.dtype != torch.float32:
            raise TypeError("states are fp32")
    rc = library().gdn_prefill_from_host(
        _host_ptr(q), _host_ptr(k), _host_ptr(v), _host_ptr(g), _host_ptr(b), _host_ptr(state_in),
        _host_ptr(state_out), _host_ptr(out), _ptr(dev["q"]), _ptr(dev["k"]), _ptr(dev["v"]), _ptr(dev["g"]),
        _ptr(dev["b"]), _ptr(dev["state"]), _ptr(dev["out"]), T, Hk, Hv, dk, dv, chunk, _dtype_code(q),
        fragment, _stream(stream, dev["q"]))
    _check(rc, "gdn_prefill_from_host")


def gdn_decode_step(q, k, v, g, b, state, out, stream=None) -> None:
    """One decode step for N sequences; updates `state` in place and writes `out`."""
    lib = _lib or library()
    N, Hk, dk = q.shape
    _, Hv, dv = v.shape
    if state.dtype != torch.float32:
        raise TypeError("the state is fp32")
    rc = lib.gdn_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(b), _ptr(state), _ptr(out),
                             N, Hk, Hv, dk, dv, _dtype_code(q), _stream(stream, q))
    if rc:
        raise GDNError(rc, "gdn_decode_step")


def gdn_decode_step_slots(q, k, v, g, b, state_pool, slots, out, stream=None) -> None:
    """One decode step; sequence n updates state_pool[slots[n]] in place (slots[n] < 0: padding)."""
    lib = _lib or library()
    N, Hk, dk = q.shape
    _, Hv, dv = v.shape
    if state_pool.dtype != torch.float32:
        raise TypeError("the state pool is fp32")
    if slots.dtype != torch.int32 or slots.numel() != N:
        raise TypeError("slots must be int32 with one entry per sequence")
    rc = lib.gdn_decode_step_slots(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(b), _ptr(state_pool), _ptr(slots),
                                   _ptr(out), N, state_pool.shape[0], Hk, Hv, dk, dv, _dtype_code(q),
                                   _stream(stream, q))
    if rc:
        raise GDNError(rc, "gdn_decode_step_slots")


def gdn_prepass(q, k, g, b, rq, rk, beta, gcum, cu_seqlens=None, B=None, T=None, chunk=64,
                stream=None) -> None:
    """Per-token inverse norms, beta and in-block cumulative gate (fp32 outputs)."""
    Ttot, Hk, dk = q.shape
    Hv = g.shape[1]
    if cu_seqlens is not None:
        B, T = cu_seqlens.numel() - 1, Ttot
    else:
        B = 1 if B is None else B
        T = Ttot // B if T is None else T
    rc = library().gdn_prepass(_ptr(q), _ptr(k), _ptr(g), _ptr(b), _ptr(cu_seqlens), B, T, Hk, Hv, dk,
                               chunk, _dtype_code(q), _ptr(rq), _ptr(rk), _ptr(beta), _ptr(gcum),
                               _stream(stream, q))
    _check(rc, "gdn_prepass")


def _load_calls():
    """The CPython module with the paged cache calls and those on trees (it checks their tensors; built beside the library)."""
    global _calls
    library()  # the module is linked against it
    with _lock:
        if _calls is None:
            path = _build.calls_path()
            if not os.path.exists(path):
                raise RuntimeError(f"the binding {path} is not built; run __graft_entry__.build()")
            loader = importlib.machinery.ExtensionFileLoader("_calls", path)
            spec = importlib.util.spec_from_file_location("_calls", path, loader=loader)
            _calls = importlib.util.module_from_spec(spec)
            loader.exec_module(_calls)
        return _calls


def gdn_kv_write(k, v, k_cache, v_cache, block_table, kv_lens, k_scale=None, v_scale=None, cu_seqlens=None,
                 B=None, T=None, stream=None) -> None:
    """Store new tokens' k, v [Ttot, Hkv, d] in paged caches [num_pages, Hkv, page_size, d] (of k's dtype,
    float8_e4m3fn or int8; 8-bit caches with fp32 scales [num_pages, Hkv, page_size]). kv_lens counts the
    new tokens in: token t of sequence n's T_n goes to position kv_lens[n] - T_n + t (negative: skipped)."""
    rc = (_calls or _load_calls()).kv_write(k, v, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens,
                                            B, T, _stream(stream, k) if k.is_cuda else 0)
    if rc:
        raise GDNError(rc, "gdn_kv_write")


def gdn_kv_read(k_cache, v_cache, block_table, kv_lens, k, v, k_scale=None, v_scale=None, cu_seqlens=None,
                B=None, T=None, stream=None) -> None:
    """The last T_n cached rows of every sequence as values, into k, v [Ttot, Hkv, d] (padding: zeros)."""
    rc = (_calls or _load_calls()).kv_read(k, v, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens,
                                           B, T, _stream(stream, k) if k.is_cuda else 0)
    if rc:
        raise GDNError(rc, "gdn_kv_read")


def gdn_paged_attn_workspace_size(B, T, Hq, Hkv, d, packed=False) -> int:
    """Bytes of device workspace gdn_paged_attn needs (packed: cu_seqlens is given, T the packed total)."""
    return int(library().gdn_paged_attn_workspace_size(B, T, int(packed), Hq, Hkv, d))


def gdn_paged_attn(q, k_cache, v_cache, block_table, kv_lens, out, k_scale=None, v_scale=None, cu_seqlens=None,
                   B=None, T=None, scale=None, workspace=None, stream=None) -> None:
    """Causal attention of the new tokens' q [Ttot, Hq, d] over their sequences' paged caches, into `out`.
    `scale` is d**-0.5 unless given. `workspace`: a uint8 CUDA tensor of gdn_paged_attn_workspace_size(...)
    bytes that a program keeps; without one the call takes it from torch's allocator."""
    on = _stream(stream, q) if q.is_cuda else 0
    if workspace is None:
        workspace = _attn_workspace(q, k_cache, kv_lens, cu_seqlens, B, stream)
    rc = (_calls or _load_calls()).paged_attn(q, out, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens,
                                              B, T, scale, workspace, on)
    if rc:
        raise GDNError(rc, "gdn_paged_attn")


def _attn_workspace(q, k_cache, kv_lens, cu_seqlens, B, stream):
    """A workspace for one call, from torch's allocator (None for tensors that the call is going to refuse)."""
    if not q.is_cuda:
        return None
    packed = cu_seqlens is not None
    n = kv_lens.numel() if B is None else B
    need = gdn_paged_attn_workspace_size(n, q.shape[0] if packed else (q.shape[0] // n if n else 0), q.shape[1],
                                         k_cache.shape[1], k_cache.shape[-1], packed)
    with torch.cuda.stream(_torch_stream(stream, q)):
        return torch.empty(need, dtype=torch.uint8, device=q.device)


def gdn_tree_attn(q, k_cache, v_cache, block_table, kv_lens, parents, out, k_scale=None, v_scale=None, cu_seqlens=None,
                  B=None, T=None, scale=None, workspace=None, stream=None) -> None:
    """gdn_paged_attn of trees of at most 64 nodes a sequence: parents int32 [Ttot] names each node's parent by its
    index within its sequence (-1: a root; below: padding). A node sees the context (the positions before the
    sequence's last T_n) and the nodes on its path from the root."""
    on = _stream(stream, q) if q.is_cuda else 0
    if workspace is None:
        workspace = _attn_workspace(q, k_cache, kv_lens, cu_seqlens, B, stream)
    rc = (_calls or _load_calls()).tree_attn(q, out, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens,
                                             B, T, scale, workspace, on, parents)
    if rc:
        raise GDNError(rc, "gdn_tree_attn")


def gdn_kv_keep(k_cache, v_cache, block_table, kv_lens, path, counts, k_scale=None, v_scale=None, cu_seqlens=None,
                T=None, stream=None) -> None:
    """The accepted paths' cache rows (path int32 [B, P], counts int32 [B]: as gdn_tree_verify leaves them) move right
    after their contexts. The step's nodes follow cu_seqlens, or T gives those of each sequence."""
    rc = (_calls or _load_calls()).kv_keep(k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens, None, T,
                                           path, counts, _stream(stream, k_cache) if k_cache.is_cuda else 0)
    if rc:
        raise GDNError(rc, "gdn_kv_keep")


def gdn_tree_scan(q, k, v, g, b, state, parents, out, slots=None, cu_seqlens=None, B=None, T=None, stream=None) -> None:
    """The gated delta rule over trees of at most 64 nodes a sequence (parents as for gdn_tree_attn): out of each node
    is what the recurrence over its path gives, from the sequence's state, which is left as it is."""
    rc = (_calls or _load_calls()).tree_scan(q, k, v, g, b, state, slots, parents, cu_seqlens, out, B, T,
                                             _stream(stream, k) if k.is_cuda else 0)
    if rc:
        raise GDNError(rc, "gdn_tree_scan")


def gdn_tree_advance(k, v, g, b, state_in, state_out, path, counts, slots=None, cu_seqlens=None, B=None, T=None,
                     stream=None) -> None:
    """The states after the recurrence over the accepted paths (path int32 [B, P], counts int32 [B]); state_out may be
    state_in. With slots both are pools, of which sequence n's entry is slots[n]."""
    rc = (_calls or _load_calls()).tree_advance(k, v, g, b, state_in, state_out, slots, path, counts, cu_seqlens, B, T,
                                                _stream(stream, k) if k.is_cuda else 0)
    if rc:
        raise GDNError(rc, "gdn_tree_advance")


def gdn_tree_verify(target_probs, draft_probs, tokens, parents, r, r_last, path, counts, next, cu_seqlens=None, B=None,
                    T=None, stream=None) -> None:
    """Which drafted tokens stand: walks each sequence's tree from node 0 by the target's and the draft's probabilities
    [Ttot, V] fp32 (draft_probs None: each child was proposed for certain) and the random numbers r [Ttot], r_last [B].
    Writes the accepted nodes, node 0 first, to path int32 [B, P] (-1 after them), their number to counts int32 [B]
    and the token after them to next int32 [B]."""
    rc = (_calls or _load_calls()).tree_verify(target_probs, draft_probs, tokens, parents, r, r_last, cu_seqlens, path, counts,
                                               next, B, T, _stream(stream, target_probs) if target_probs.is_cuda else 0)
    if rc:
        raise GDNError(rc, "gdn_tree_verify")


def gdn_prefill_path(B, T, Hk, Hv, dk, dv, chunk, dtype) -> int:
    """2 = token scan, 1 = tensor-core kernel, 0 = CUDA-core kernel, <0 = the status gdn_prefill would return."""
    if isinstance(dtype, torch.dtype):
        dtype = GDN_BF16 if dtype == torch.bfloat16 else GDN_F32
    return library().gdn_prefill_path(B, T, Hk, Hv, dk, dv, chunk, int(dtype))


def gdn_get_device_status(stream=None) -> int:
    """Synchronise the stream, return and clear the device status word."""
    return library().gdn_get_device_status(_stream(stream))
