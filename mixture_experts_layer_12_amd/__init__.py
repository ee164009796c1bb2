"""Python binding of the MoE layer C ABI (``include/moe.h``).

Argument marshalling only: every step of the layer runs in the HIP kernels of
``lib/libmoe.so``.  Functions carry the C names (``moe_workspace_size``,
``moe_dispatch_dims``, ``moe_route``, ``moe_forward``, ``moe_strerror``) and
accept torch tensors (their ``data_ptr()`` is passed) or raw integer device
addresses.  The separate operators (``moe_grouped_matmul`` and its gradients,
``moe_quantize_rows``, ``moe_grouped_matmul_i8``, ``moe_combine`` and its
gradients) also check that the tensors they are given are dense, on one GPU
and of the type and size that the shape says, and run on the current stream of
that GPU unless they are given one.  PyTorch only provides device memory and
the current stream.

There is no fallback: if the library is missing the calls raise.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

LIB_DIR = os.path.join(os.path.dirname(os.path.abspath(__file__)), "lib")
LIB_PATH = os.path.join(LIB_DIR, "libmoe.so")

# enums of moe.h
MOE_F32, MOE_BF16, MOE_Q4_0, MOE_Q8_0, MOE_FP8_E4M3, MOE_I8 = 0, 1, 2, 3, 4, 5
MOE_PATH_AUTO, MOE_PATH_DECODE, MOE_PATH_PREFILL, MOE_PATH_DECODE_FUSED = 0, 1, 2, 3
MOE_OK, MOE_ERR_NULL, MOE_ERR_SHAPE, MOE_ERR_DTYPE, MOE_ERR_ALIGN, MOE_ERR_WORKSPACE, MOE_ERR_HIP = (
    0, -1, -2, -3, -4, -5, -6)
MOE_ERR_TOO_LARGE = -7
MOE_ERR_NOT_PINNED = -8
MOE_ERR_HOST_ALLOC = -9
MOE_NOALLOC_SCRATCH_BYTES = 64 << 20

DTYPES = {"f32": MOE_F32, "bf16": MOE_BF16, "q4_0": MOE_Q4_0, "q8_0": MOE_Q8_0, "fp8_e4m3": MOE_FP8_E4M3,
          "i8": MOE_I8}
EXPORTED = ("moe_workspace_size", "moe_dispatch_dims", "moe_route", "moe_forward", "moe_forward_profiled",
            "moe_last_hip_error", "moe_strerror", "moe_resolve_path", "moe_sparse_workspace_size",
            "moe_forward_channel_sparse", "moe_forward_tables", "moe_route_workspace_size",
            "moe_probe_read", "moe_probe_mfma_bf16", "moe_forward_noalloc", "moe_cache_region_bytes",
            "moe_cache_create", "moe_cache_destroy", "moe_forward_cached", "moe_cache_stats", "moe_cache_flush",
            "moe_grouped_workspace_size", "moe_grouped_matmul", "moe_grouped_matmul_backward", "moe_quantize_rows",
            "moe_grouped_matmul_i8", "moe_combine", "moe_combine_backward")


class moe_shape_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "T", "H", "E", "I", "top_k", "n_shared", "I_shared", "x_dtype", "w_dtype", "router_dtype", "path")]


class moe_route_out_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "topk_ids", "topk_w", "counts", "offsets", "sorted_ids", "tile_expert", "inv", "active")]


class moe_forward_tables_t(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("path", "tokens", "tile_m", "capacity", "n_tiles")] +
                [(n, ctypes.c_size_t) for n in ("topk_ids", "topk_w", "counts", "offsets", "sorted_ids",
                                                "tile_expert", "inv", "active", "status")] +
                [(n, ctypes.c_int32) for n in ("route_in_gateup", "shared_in_router")])


class moe_host_experts_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("w_gate", "w_up", "w_down")]


class moe_cache_stats_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint64) for n in (
        "lookups", "hits", "misses", "prefetches", "prefetch_hits", "bytes_copied")]


class moe_grouped_shape_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "N", "K", "E", "x_rows", "row_div", "x_dtype", "out_dtype")]


class moe_combine_shape_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "top_k", "H", "rows", "y_dtype", "out_dtype")]


class MoeError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        msg = f"{where}: {moe_strerror(code)} ({code})"
        if code == MOE_ERR_HIP:
            msg += f"; {hip_error_name(moe_last_hip_error())}"
        super().__init__(msg)


_lib: Optional[ctypes.CDLL] = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libmoe.so (once).  Raises FileNotFoundError when it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise FileNotFoundError(f"{path} is missing: build it with __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER
    vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32
    lib.moe_workspace_size.argtypes = [P(moe_shape_t), P(sz)]
    lib.moe_workspace_size.restype = ctypes.c_int
    lib.moe_dispatch_dims.argtypes = [P(moe_shape_t), P(i32), P(i32), P(i32)]
    lib.moe_dispatch_dims.restype = ctypes.c_int
    lib.moe_route.argtypes = [P(moe_shape_t), vp, vp, vp, P(moe_route_out_t), vp, sz, vp]
    lib.moe_route.restype = ctypes.c_int
    lib.moe_forward.argtypes = [P(moe_shape_t), vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_forward.restype = ctypes.c_int
    lib.moe_forward_profiled.argtypes = [P(moe_shape_t), vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp,
                                         P(vp), ctypes.c_int]
    lib.moe_forward_profiled.restype = ctypes.c_int
    lib.moe_last_hip_error.argtypes = []
    lib.moe_last_hip_error.restype = ctypes.c_int
    lib.moe_sparse_workspace_size.argtypes = [P(moe_shape_t), i32, P(sz)]
    lib.moe_sparse_workspace_size.restype = ctypes.c_int
    lib.moe_forward_channel_sparse.argtypes = [P(moe_shape_t), i32] + [vp] * 12 + [sz, vp]
    lib.moe_forward_channel_sparse.restype = ctypes.c_int
    lib.moe_forward_tables.argtypes = [P(moe_shape_t), P(moe_forward_tables_t)]
    lib.moe_forward_tables.restype = ctypes.c_int
    lib.moe_route_workspace_size.argtypes = [P(moe_shape_t), P(sz)]
    lib.moe_route_workspace_size.restype = ctypes.c_int
    lib.moe_forward_noalloc.argtypes = [P(moe_shape_t), vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.moe_forward_noalloc.restype = ctypes.c_int
    lib.moe_probe_read.argtypes = [vp, sz, vp, vp]
    lib.moe_probe_read.restype = ctypes.c_int
    lib.moe_probe_mfma_bf16.argtypes = [i32, vp, P(ctypes.c_double), vp]
    lib.moe_probe_mfma_bf16.restype = ctypes.c_int
    lib.moe_cache_region_bytes.argtypes = [P(moe_shape_t), i32, i32, P(sz)]
    lib.moe_cache_region_bytes.restype = ctypes.c_int
    lib.moe_cache_create.argtypes = [P(moe_shape_t), i32, P(moe_host_experts_t), vp, sz, i32, i32, i32, vp,
                                     P(vp)]
    lib.moe_cache_create.restype = ctypes.c_int
    lib.moe_cache_destroy.argtypes = [vp]
    lib.moe_cache_destroy.restype = ctypes.c_int
    lib.moe_forward_cached.argtypes = [vp, i32, P(moe_shape_t), vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_forward_cached.restype = ctypes.c_int
    lib.moe_cache_stats.argtypes = [vp, P(moe_cache_stats_t), i32]
    lib.moe_cache_stats.restype = ctypes.c_int
    lib.moe_cache_flush.argtypes = [vp]
    lib.moe_cache_flush.restype = ctypes.c_int
    lib.moe_resolve_path.argtypes = [P(moe_shape_t)]
    lib.moe_resolve_path.restype = ctypes.c_int
    lib.moe_grouped_workspace_size.argtypes = [P(moe_grouped_shape_t), P(sz)]
    lib.moe_grouped_workspace_size.restype = ctypes.c_int
    lib.moe_grouped_matmul.argtypes = [P(moe_grouped_shape_t)] + [vp] * 7 + [sz, vp]
    lib.moe_grouped_matmul.restype = ctypes.c_int
    lib.moe_grouped_matmul_backward.argtypes = [P(moe_grouped_shape_t)] + [vp] * 9 + [sz, vp]
    lib.moe_grouped_matmul_backward.restype = ctypes.c_int
    lib.moe_quantize_rows.argtypes = [i32, i32, i32, vp, vp, vp, vp]
    lib.moe_quantize_rows.restype = ctypes.c_int
    lib.moe_grouped_matmul_i8.argtypes = [P(moe_grouped_shape_t)] + [vp] * 9 + [sz, vp]
    lib.moe_grouped_matmul_i8.restype = ctypes.c_int
    lib.moe_combine.argtypes = [P(moe_combine_shape_t)] + [vp] * 5
    lib.moe_combine.restype = ctypes.c_int
    lib.moe_combine_backward.argtypes = [P(moe_combine_shape_t)] + [vp] * 7
    lib.moe_combine_backward.restype = ctypes.c_int
    lib.moe_strerror.argtypes = [ctypes.c_int]
    lib.moe_strerror.restype = ctypes.c_char_p
    _lib = lib
    return lib


def make_shape(T, H, E, I, top_k, n_shared=0, I_shared=0, x_dtype="bf16", w_dtype="bf16",
               router_dtype="bf16", path=MOE_PATH_AUTO) -> moe_shape_t:
    conv = lambda d: DTYPES[d] if isinstance(d, str) else int(d)
    return moe_shape_t(int(T), int(H), int(E), int(I), int(top_k), int(n_shared), int(I_shared),
                       conv(x_dtype), conv(w_dtype), conv(router_dtype), int(path))


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


def moe_strerror(code: int) -> str:
    return load_library().moe_strerror(int(code)).decode()


def moe_last_hip_error() -> int:
    return int(load_library().moe_last_hip_error())


def hip_error_name(err: int) -> str:
    """hipGetErrorName of a hipError_t value (from the HIP runtime)."""
    try:
        hip = ctypes.CDLL("libamdhip64.so")
        hip.hipGetErrorName.restype = ctypes.c_char_p
        hip.hipGetErrorName.argtypes = [ctypes.c_int]
        return f"hipError {err} ({hip.hipGetErrorName(err).decode()})"
    except OSError:
        return f"hipError {err}"


def moe_sparse_workspace_size(shape: moe_shape_t, budget: int) -> int:
    n = ctypes.c_size_t(0)
    rc = load_library().moe_sparse_workspace_size(ctypes.byref(shape), int(budget), ctypes.byref(n))
    if rc:
        raise MoeError(rc, "moe_sparse_workspace_size")
    return n.value


def moe_forward_channel_sparse(shape: moe_shape_t, budget: int, channel_scores, x, router_w, router_b, w_gate, w_up,
                               w_down_t, ws_gate, ws_up, ws_down, out, workspace, ws_bytes=None, stream=None,
                               check=True) -> int:
    nb = _nbytes(workspace) if ws_bytes is None else ws_bytes
    rc = load_library().moe_forward_channel_sparse(
        ctypes.byref(shape), int(budget), _ptr(channel_scores), _ptr(x), _ptr(router_w), _ptr(router_b),
        _ptr(w_gate), _ptr(w_up), _ptr(w_down_t), _ptr(ws_gate), _ptr(ws_up), _ptr(ws_down), _ptr(out),
        _ptr(workspace), nb, _stream(stream))
    if check and rc:
        raise MoeError(rc, "moe_forward_channel_sparse")
    return rc


def moe_resolve_path(shape: moe_shape_t) -> int:
    """MOE_PATH_DECODE / _PREFILL / _DECODE_FUSED that moe_forward takes for ``shape``."""
    rc = load_library().moe_resolve_path(ctypes.byref(shape))
    if rc < 0:
        raise MoeError(rc, "moe_resolve_path")
    return rc


def moe_workspace_size(shape: moe_shape_t) -> int:
    n = ctypes.c_size_t(0)
    rc = load_library().moe_workspace_size(ctypes.byref(shape), ctypes.byref(n))
    if rc:
        raise MoeError(rc, "moe_workspace_size")
    return n.value


def moe_probe_read(buf, nbytes: int, sink, stream=None) -> None:
    """Measurement probe (include/moe_probe.h): read ``nbytes`` of ``buf`` once."""
    rc = load_library().moe_probe_read(_ptr(buf), int(nbytes), _ptr(sink), _stream(stream))
    if rc:
        raise MoeError(rc, "moe_probe_read")


def moe_probe_mfma_bf16(iters: int, sink, stream=None) -> float:
    """Measurement probe: back-to-back bf16 MFMAs on every compute unit; returns the launch's flops."""
    fl = ctypes.c_double(0.0)
    rc = load_library().moe_probe_mfma_bf16(int(iters), _ptr(sink), ctypes.byref(fl), _stream(stream))
    if rc:
        raise MoeError(rc, "moe_probe_mfma_bf16")
    return fl.value


def moe_route_workspace_size(shape: moe_shape_t) -> int:
    n = ctypes.c_size_t(0)
    rc = load_library().moe_route_workspace_size(ctypes.byref(shape), ctypes.byref(n))
    if rc:
        raise MoeError(rc, "moe_route_workspace_size")
    return n.value


def moe_forward_tables(shape: moe_shape_t) -> dict:
    """Where moe_forward leaves the routing of its last pass in the workspace:
    path, tokens, tile_m, capacity, n_tiles and the byte offsets of the arrays."""
    t = moe_forward_tables_t()
    rc = load_library().moe_forward_tables(ctypes.byref(shape), ctypes.byref(t))
    if rc:
        raise MoeError(rc, "moe_forward_tables")
    return {n: getattr(t, n) for n, _ in moe_forward_tables_t._fields_}


def fused_status_ok(shape: moe_shape_t, workspace) -> bool:
    """After a completed call whose shape has status words (the single-launch
    decode, or a decode pass whose selection runs inside the logits launch):
    True unless a wait gave up (the two status words of moe_forward_tables_t
    are equal).  Reads 16 bytes of the workspace back to the host; the caller
    synchronises first."""
    import torch
    o = moe_forward_tables(shape)["status"]
    if o == 0:
        raise ValueError("no status words for this shape and path")
    w = workspace[o:o + 16].view(torch.int64).cpu()
    return int(w[0]) != int(w[1])


def moe_dispatch_dims(shape: moe_shape_t):
    """(tile_m, capacity, n_tiles) of the expert-sorted order."""
    a, b, c = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    rc = load_library().moe_dispatch_dims(ctypes.byref(shape), ctypes.byref(a), ctypes.byref(b), ctypes.byref(c))
    if rc:
        raise MoeError(rc, "moe_dispatch_dims")
    return a.value, b.value, c.value


def moe_route(shape: moe_shape_t, x, router_w, router_b, out: dict, workspace, ws_bytes=None, stream=None,
              check=True) -> int:
    """``out`` maps moe_route_out_t field names to int32/float32 device tensors (or None)."""
    ro = moe_route_out_t(*[_ptr(out.get(n)) for n, _ in moe_route_out_t._fields_])
    nb = _nbytes(workspace) if ws_bytes is None else ws_bytes
    rc = load_library().moe_route(ctypes.byref(shape), _ptr(x), _ptr(router_w), _ptr(router_b), ctypes.byref(ro),
                                  _ptr(workspace), nb, _stream(stream))
    if check and rc:
        raise MoeError(rc, "moe_route")
    return rc


def moe_forward(shape: moe_shape_t, x, router_w, router_b, w_gate, w_up, w_down, ws_gate, ws_up, ws_down,
                out, workspace, ws_bytes=None, stream=None, check=True) -> int:
    nb = _nbytes(workspace) if ws_bytes is None else ws_bytes
    rc = load_library().moe_forward(ctypes.byref(shape), _ptr(x), _ptr(router_w), _ptr(router_b),
                                    _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(ws_gate), _ptr(ws_up),
                                    _ptr(ws_down), _ptr(out), _ptr(workspace), nb, _stream(stream))
    if check and rc:
        raise MoeError(rc, "moe_forward")
    return rc


def moe_forward_noalloc(shape: moe_shape_t, x, router_w, router_b, w_gate, w_up, w_down, ws_gate, ws_up, ws_down,
                        out, stream=None, check=True) -> int:
    """moe_forward with the library's static device scratch as its workspace (allocates nothing)."""
    rc = load_library().moe_forward_noalloc(ctypes.byref(shape), _ptr(x), _ptr(router_w), _ptr(router_b),
                                            _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(ws_gate), _ptr(ws_up),
                                            _ptr(ws_down), _ptr(out), _stream(stream))
    if check and rc:
        raise MoeError(rc, "moe_forward_noalloc")
    return rc


def moe_forward_profiled(shape: moe_shape_t, x, router_w, router_b, w_gate, w_up, w_down, ws_gate, ws_up,
                         ws_down, out, workspace, events, ws_bytes=None, stream=None, check=True) -> int:
    """``events``: sequence of raw hipEvent_t handles (ints) recorded at stage boundaries."""
    nb = _nbytes(workspace) if ws_bytes is None else ws_bytes
    arr = (ctypes.c_void_p * len(events))(*events)
    rc = load_library().moe_forward_profiled(ctypes.byref(shape), _ptr(x), _ptr(router_w), _ptr(router_b),
                                             _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(ws_gate), _ptr(ws_up),
                                             _ptr(ws_down), _ptr(out), _ptr(workspace), nb, _stream(stream),
                                             arr, len(events))
    if check and rc:
        raise MoeError(rc, "moe_forward_profiled")
    return rc


def moe_cache_region_bytes(shape: moe_shape_t, n_layers: int, n_slots: int) -> int:
    n = ctypes.c_size_t(0)
    rc = load_library().moe_cache_region_bytes(ctypes.byref(shape), n_layers, n_slots, ctypes.byref(n))
    if rc:
        raise MoeError(rc, "moe_cache_region_bytes")
    return n.value


def moe_cache_create(shape: moe_shape_t, layers, region, n_slots: int, prefetch_depth: int, prefetch_shift: int,
                     copy_stream, region_bytes=None, check=True):
    """``layers``: sequence of (w_gate, w_up, w_down) pinned host buffers per layer.  Returns the
    handle (an int), or the error code when ``check`` is false and the call fails."""
    arr = (moe_host_experts_t * len(layers))(*[moe_host_experts_t(_ptr(g), _ptr(u), _ptr(d)) for g, u, d in layers])
    h = ctypes.c_void_p(None)
    nb = _nbytes(region) if region_bytes is None else region_bytes
    rc = load_library().moe_cache_create(ctypes.byref(shape), len(layers), arr, _ptr(region), nb, n_slots,
                                         prefetch_depth, prefetch_shift, _stream(copy_stream), ctypes.byref(h))
    if rc:
        if check:
            raise MoeError(rc, "moe_cache_create")
        return rc
    return h.value


def moe_cache_destroy(cache) -> None:
    rc = load_library().moe_cache_destroy(cache)
    if rc:
        raise MoeError(rc, "moe_cache_destroy")


def moe_forward_cached(cache, layer: int, shape: moe_shape_t, x, router_w, router_b, ws_gate, ws_up, ws_down, out,
                       workspace, ws_bytes=None, stream=None, check=True) -> int:
    nb = _nbytes(workspace) if ws_bytes is None else ws_bytes
    rc = load_library().moe_forward_cached(cache, layer, ctypes.byref(shape), _ptr(x), _ptr(router_w),
                                           _ptr(router_b), _ptr(ws_gate), _ptr(ws_up), _ptr(ws_down), _ptr(out),
                                           _ptr(workspace), nb, _stream(stream))
    if check and rc:
        raise MoeError(rc, "moe_forward_cached")
    return rc


def moe_cache_stats(cache, reset: bool = False) -> dict:
    st = moe_cache_stats_t()
    rc = load_library().moe_cache_stats(cache, ctypes.byref(st), 1 if reset else 0)
    if rc:
        raise MoeError(rc, "moe_cache_stats")
    return {n: getattr(st, n) for n, _ in moe_cache_stats_t._fields_}


def moe_cache_flush(cache) -> None:
    rc = load_library().moe_cache_flush(cache)
    if rc:
        raise MoeError(rc, "moe_cache_flush")


def alloc_sparse_workspace(shape: moe_shape_t, budget: int, device="cuda"):
    """A workspace of moe_sparse_workspace_size(shape, budget) bytes (contents irrelevant)."""
    import torch
    return torch.empty(max(moe_sparse_workspace_size(shape, budget), 256), dtype=torch.uint8, device=device)


def alloc_workspace(shape: moe_shape_t, device="cuda"):
    """A workspace of moe_workspace_size(shape) bytes (torch uint8 tensor; contents irrelevant)."""
    import torch
    return torch.empty(max(moe_workspace_size(shape), 256), dtype=torch.uint8, device=device)


# ------------------------------------------------- the layer's parts as operators --

def make_grouped_shape(rows, N, K, E, x_rows=None, row_div=1, x_dtype="bf16", out_dtype="bf16") -> moe_grouped_shape_t:
    """Shape of the grouped expert products; ``x_rows`` defaults to ``rows`` (no row lookup)."""
    conv = lambda d: DTYPES[d] if isinstance(d, str) else int(d)
    return moe_grouped_shape_t(int(rows), int(N), int(K), int(E), int(rows if x_rows is None else x_rows),
                               int(row_div), conv(x_dtype), conv(out_dtype))


def make_combine_shape(T, top_k, H, rows, y_dtype="bf16", out_dtype="bf16") -> moe_combine_shape_t:
    conv = lambda d: DTYPES[d] if isinstance(d, str) else int(d)
    return moe_combine_shape_t(int(T), int(top_k), int(H), int(rows), conv(y_dtype), conv(out_dtype))


def moe_grouped_workspace_size(shape: moe_grouped_shape_t) -> int:
    n = ctypes.c_size_t(0)
    rc = load_library().moe_grouped_workspace_size(ctypes.byref(shape), ctypes.byref(n))
    if rc:
        raise MoeError(rc, "moe_grouped_workspace_size")
    return n.value


def alloc_grouped_workspace(shape: moe_grouped_shape_t, device="cuda"):
    """A workspace of moe_grouped_workspace_size(shape) bytes (contents irrelevant)."""
    import torch
    return torch.empty(max(moe_grouped_workspace_size(shape), 256), dtype=torch.uint8, device=device)


_types = None      # torch dtypes of the element codes


def _torch_types():
    """The torch dtype of each element code (None for those that no tensor has), looked up once."""
    global _types
    if _types is None:
        import torch
        _types = {MOE_F32: torch.float32, MOE_BF16: torch.bfloat16, MOE_I8: torch.int8, "i32": torch.int32}
    return _types


def _device_of(*tensors) -> int:
    """Index of the GPU that the first tensor lies on (-1: on none); None if all are addresses."""
    for t in tensors:
        if t is not None and type(t) is not int:
            return t.get_device()
    return None


def _checked(where: str, name: str, t, dtype, n: int, device):
    """The address of operand ``t``: dense, of the type and at least the size that the shape says, on GPU ``device``.
    Raw addresses and None pass as they are."""
    if t is None or type(t) is int:
        return t
    on = t.get_device()
    if t.dtype is not dtype or t.numel() < n or on < 0 or (on != device and device is not None) or not t.is_contiguous():
        if t.dtype is not dtype:
            why = f"has type {t.dtype}, the shape says {dtype}"
        elif not t.is_contiguous():
            why = "is not contiguous"
        elif t.numel() < n:
            why = f"has {t.numel()} elements, the shape needs {n}"
        elif on < 0:
            why = "is not on a GPU"
        else:
            why = "is on another GPU than the operands before it"
        raise ValueError(f"{where}: {name} {why}")
    return t.data_ptr()


def _launch(where: str, function, device, stream, check: bool, *args) -> int:
    """function(*args, stream) with GPU ``device`` current; ``stream`` None is that GPU's current stream."""
    import torch
    if device is None or device == torch.cuda.current_device():
        if stream is None and device is not None:
            st = torch._C._cuda_getCurrentRawStream(device)
        else:
            st = _stream(stream)
        rc = function(*args, st)
    else:
        with torch.cuda.device(device):
            rc = function(*args, _stream(stream))
    if check and rc:
        raise MoeError(rc, where)
    return rc


def _grouped(where, function, shape, x_name, x, x_scale, dy, row_ids, offsets, counts, w, w_scale, outs, workspace,
             ws_bytes, stream, check):
    """The three grouped products: checks the operands and calls ``function`` with those that it takes."""
    types = _torch_types()
    rows, N, K, E, x_rows = shape.rows, shape.N, shape.K, shape.E, shape.x_rows
    dt, i32 = types.get(shape.x_dtype), types["i32"]
    dev = _device_of(x, dy, w, offsets)
    px = _checked(where, x_name, x, dt, x_rows * K, dev)
    ids = _checked(where, "row_ids", row_ids, i32, rows, dev)
    off = _checked(where, "offsets", offsets, i32, E + (counts is None), dev)
    cnt = _checked(where, "counts", counts, i32, E, dev)
    pw = _checked(where, "w", w, dt, E * N * K, dev)
    po = [_checked(where, name, t, types.get(code), n, dev) for name, t, code, n in outs]
    if x_name == "xq":
        f32 = types[MOE_F32]
        args = (px, _checked(where, "x_scale", x_scale, f32, x_rows, dev), ids, off, cnt, pw,
                _checked(where, "w_scale", w_scale, f32, E * N, dev))
    elif len(po) == 2:
        args = (_checked(where, "dy", dy, dt, rows * N, dev), px, ids, off, cnt, pw)
    else:
        args = (px, ids, off, cnt, pw)
    nb = _nbytes(workspace) if ws_bytes is None else ws_bytes
    if workspace is not None and type(workspace) is not int and dev is not None and workspace.get_device() != dev:
        raise ValueError(f"{where}: workspace is not on the operands' GPU")
    return _launch(where, function, dev, stream, check, ctypes.byref(shape), *args, *po, _ptr(workspace), nb)


def moe_grouped_matmul(shape: moe_grouped_shape_t, x, row_ids, offsets, counts, w, y, workspace, ws_bytes=None,
                       stream=None, check=True) -> int:
    """y[r] = x[row(r)] . w[e]^T over the segments; ``row_ids`` and ``counts`` may be None."""
    return _grouped("moe_grouped_matmul", load_library().moe_grouped_matmul, shape, "x", x, None, None, row_ids, offsets,
                    counts, w, None, (("y", y, shape.out_dtype, shape.rows * shape.N),), workspace, ws_bytes, stream,
                    check)


def moe_grouped_matmul_backward(shape: moe_grouped_shape_t, dy, x, row_ids, offsets, counts, w, dx, dw, workspace,
                                ws_bytes=None, stream=None, check=True) -> int:
    """The gradients dx (sorted order) and dw of moe_grouped_matmul; either may be None."""
    return _grouped("moe_grouped_matmul_backward", load_library().moe_grouped_matmul_backward, shape, "x", x, None, dy,
                    row_ids, offsets, counts, w, None,
                    (("dx", dx, shape.x_dtype, shape.rows * shape.K),
                     ("dw", dw, shape.out_dtype, shape.E * shape.N * shape.K)), workspace, ws_bytes, stream, check)


def moe_grouped_matmul_i8(shape: moe_grouped_shape_t, xq, x_scale, row_ids, offsets, counts, wq, w_scale, y, workspace,
                          ws_bytes=None, stream=None, check=True) -> int:
    """The forward product on 8-bit codes with scales for each row of ``xq`` and each output channel of ``wq``."""
    return _grouped("moe_grouped_matmul_i8", load_library().moe_grouped_matmul_i8, shape, "xq", xq, x_scale, None, row_ids,
                    offsets, counts, wq, w_scale, (("y", y, shape.out_dtype, shape.rows * shape.N),), workspace, ws_bytes,
                    stream, check)


def moe_quantize_rows(x, q, scale, stream=None, check=True) -> int:
    """8-bit codes ``q`` and fp32 ``scale`` of each row of the matrix ``x`` (float32 or bfloat16, two dimensions)."""
    types = _torch_types()
    dt = MOE_F32 if x.dtype is types[MOE_F32] else MOE_BF16
    if x.dim() != 2 or x.dtype is not types[dt]:
        raise ValueError("moe_quantize_rows: x is not a float32 or bfloat16 matrix")
    rows, cols = x.shape
    dev, where = x.get_device(), "moe_quantize_rows"
    return _launch(where, load_library().moe_quantize_rows, dev, stream, check, rows, cols, dt,
                   _checked(where, "x", x, types[dt], rows * cols, dev),
                   _checked(where, "q", q, types[MOE_I8], rows * cols, dev),
                   _checked(where, "scale", scale, types[MOE_F32], rows, dev))


def moe_combine(shape: moe_combine_shape_t, y, inv, weights, out, stream=None, check=True) -> int:
    """out[t] = sum_j weights[t, j] * y[inv[t, j]]; ``weights`` None means 1."""
    types, where = _torch_types(), "moe_combine"
    T, H = shape.T, shape.H
    n, dev = T * shape.top_k, _device_of(y, inv, out)
    return _launch(where, load_library().moe_combine, dev, stream, check, ctypes.byref(shape),
                   _checked(where, "y", y, types.get(shape.y_dtype), shape.rows * H, dev),
                   _checked(where, "inv", inv, types["i32"], n, dev),
                   _checked(where, "weights", weights, types[MOE_F32], n, dev),
                   _checked(where, "out", out, types.get(shape.out_dtype), T * H, dev))


def moe_combine_backward(shape: moe_combine_shape_t, dout, y, inv, weights, dy, dweights, stream=None,
                         check=True) -> int:
    """The gradients dy and dweights of moe_combine; either may be None (``y`` is read for dweights only)."""
    types, where = _torch_types(), "moe_combine_backward"
    T, H = shape.T, shape.H
    n, dev, yt = T * shape.top_k, _device_of(dout, y, inv), types.get(shape.y_dtype)
    return _launch(where, load_library().moe_combine_backward, dev, stream, check, ctypes.byref(shape),
                   _checked(where, "dout", dout, types.get(shape.out_dtype), T * H, dev),
                   _checked(where, "y", y, yt, shape.rows * H, dev),
                   _checked(where, "inv", inv, types["i32"], n, dev),
                   _checked(where, "weights", weights, types[MOE_F32], n, dev),
                   _checked(where, "dy", dy, yt, shape.rows * H, dev),
                   _checked(where, "dweights", dweights, types[MOE_F32], n, dev))
