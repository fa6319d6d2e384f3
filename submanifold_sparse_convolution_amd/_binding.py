"""ctypes binding of libsubmconv.so: argument marshalling only.

Every function here has the name of the C entry point it calls.  Tensors are
device tensors; PyTorch supplies their memory (data_ptr) and the current HIP
stream.  No arithmetic of the method happens in Python, and there is no
fallback: when the shared library is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import operator
import os
import threading

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "lib", "libsubmconv.so")

SUBM_F32, SUBM_F16, SUBM_BF16 = 0, 1, 2
SUBM_MAP_AUTO, SUBM_MAP_HASH, SUBM_MAP_GRID, SUBM_MAP_SUBDIVIDED = 0, 1, 2, 3
SUBM_POOL_MAX, SUBM_POOL_MEAN = 1, 2
SUBM_COARSE, SUBM_FINE, SUBM_PARENT = 0, 1, 2
SUBM_SUBDIVIDE, SUBM_DOWNSAMPLE, SUBM_UPSAMPLE_MASKED = 0, 1, 2
SUBM_ACT_NONE, SUBM_ACT_SILU, SUBM_ACT_RELU = 0, 1, 2
SUBM_ROPE_INTERLEAVED, SUBM_ROPE_HALF = 0, 1
SUBM_ROPE_PLAIN, SUBM_ROPE_LINEAR, SUBM_ROPE_BASE, SUBM_ROPE_PARTS = 0, 1, 2, 3
_DTYPE_CODES = {torch.float32: SUBM_F32, torch.float16: SUBM_F16, torch.bfloat16: SUBM_BF16}
TAPS = 27

# Exported C symbols (kept equal to the declarations in include/*.h).  Every one but the last
# two returns an int status.
C_FUNCTIONS = (
    "sparse_indice_map_build",
    "sparse_indice_map_build_ex",
    "sparse_indice_map_build_async",
    "sparse_indice_map_status",
    "sparse_indice_map_mode",
    "sparse_indice_map_free",
    "sparse_indice_map_info",
    "sparse_indice_map_offset_counts",
    "sparse_indice_map_copy_nbr",
    "sparse_indice_map_plan_state",
    "sparse_indice_map_row_order_state",
    "subm_release_cached_memory",
    "subm_timing_events",
    "subm_mfma_rate",
    "subm_conv3d_forward",
    "subm_conv3d_forward_noalloc",
    "subm_conv3d_forward_per_offset",
    "sparse_subdivide",
    "sparse_downsample_build",
    "sparse_upsample_masked_build",
    "sparse_subdivision_info",
    "sparse_subdivision_kind",
    "sparse_subdivision_coords",
    "sparse_subdivision_parent",
    "sparse_subdivision_copy",
    "sparse_subdivision_free",
    "sparse_downsample_forward",
    "sparse_upsample_forward",
    "sparse_indice_map_subdivide",
    "sparse_group_norm_act",
    "subm_conv3d_forward_group_norm_act",
    "sparse_layer_norm_forward",
    "sparse_layer_norm_backward",
    "sparse_rms_norm_forward",
    "sparse_rms_norm_quantize_forward",
    "sparse_rms_norm_backward",
    "sparse_embedding_forward",
    "sparse_embedding_backward",
    "sparse_rope_frequencies",
    "sparse_rope_forward",
    "sparse_rope_backward",
    "sparse_attention_forward",
    "sparse_attention_backward",
    "sparse_window_attention_forward",
    "sparse_window_attention_backward",
    "subm_status_string",
    "subm_last_error",
)


class _HeadsArg(ctypes.Structure):
    """subm_heads_t of include/sparse_transformer.h."""

    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


_lib = None
_lib_lock = threading.Lock()


class SubmError(RuntimeError):
    """A non-zero status returned by the library."""

    def __init__(self, func: str, status: int, name: str, detail: str):
        super().__init__(f"{func} failed: {name} ({status}): {detail}")
        self.status = status
        self.name = name
        self.detail = detail


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load (once) and return the shared library.  Raises if it has not been built."""
    global _lib
    with _lib_lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(
                f"HIP library not found at {p}; build it with "
                "`python -m submanifold_sparse_convolution_amd.build` (there is no CPU fallback)")
        lib = ctypes.CDLL(p)
        vp, i64, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        lib.sparse_indice_map_build.argtypes = [vp, i64, vp, ctypes.POINTER(vp)]
        lib.sparse_indice_map_build_ex.argtypes = [vp, i64, ci, vp, ctypes.POINTER(vp)]
        lib.sparse_indice_map_build_async.argtypes = [vp, i64, ci, vp, ctypes.POINTER(vp)]
        lib.sparse_indice_map_status.argtypes = [vp]
        lib.sparse_indice_map_mode.argtypes = [vp, ctypes.POINTER(ci)]
        lib.sparse_indice_map_free.argtypes = [vp]
        lib.sparse_indice_map_info.argtypes = [vp, ctypes.POINTER(i64), ctypes.POINTER(i64)]
        lib.sparse_indice_map_offset_counts.argtypes = [vp, ctypes.POINTER(i64)]
        lib.sparse_indice_map_copy_nbr.argtypes = [vp, vp, vp]
        lib.sparse_indice_map_plan_state.argtypes = [vp, ctypes.POINTER(ci)]
        lib.sparse_indice_map_row_order_state.argtypes = [vp, ctypes.POINTER(ci)]
        lib.subm_release_cached_memory.argtypes = []
        lib.subm_timing_events.argtypes = [vp, vp]
        lib.subm_mfma_rate.argtypes = [i64, ci, vp, vp, vp]
        lib.subm_conv3d_forward.argtypes = [vp, i64, ci, ci, ci, ci, vp, vp, vp, vp, vp]
        lib.subm_conv3d_forward_noalloc.argtypes = [vp, i64, ci, ci, ci, ci, vp, vp, vp, vp, vp]
        lib.subm_conv3d_forward_per_offset.argtypes = [vp, i64, ci, ci, ci, vp, vp, vp, vp, vp]
        lib.sparse_subdivide.argtypes = [vp, i64, vp, ctypes.POINTER(vp)]
        lib.sparse_downsample_build.argtypes = [vp, i64, vp, ctypes.POINTER(vp)]
        lib.sparse_upsample_masked_build.argtypes = [vp, vp, i64, vp, ctypes.POINTER(vp)]
        lib.sparse_subdivision_info.argtypes = [vp, ctypes.POINTER(i64), ctypes.POINTER(i64)]
        lib.sparse_subdivision_kind.argtypes = [vp, ctypes.POINTER(ci)]
        lib.sparse_subdivision_coords.argtypes = [vp, ci, ctypes.POINTER(vp)]
        lib.sparse_subdivision_parent.argtypes = [vp, ctypes.POINTER(vp)]
        lib.sparse_subdivision_copy.argtypes = [vp, ci, vp, vp]
        lib.sparse_subdivision_free.argtypes = [vp]
        lib.sparse_downsample_forward.argtypes = [vp, ci, ci, ci, vp, vp, vp]
        lib.sparse_upsample_forward.argtypes = [vp, ci, ci, vp, vp, vp]
        lib.sparse_indice_map_subdivide.argtypes = [vp, vp, vp, ctypes.POINTER(vp)]
        lib.sparse_group_norm_act.argtypes = [vp, i64, ci, ci, vp, ci, ci, vp, vp, ctypes.c_float, ci, vp, vp]
        lib.subm_conv3d_forward_group_norm_act.argtypes = [vp, i64, ci, ci, ci, ci, vp, vp, vp, vp, ci, ci, vp, vp,
                                                           ctypes.c_float, ci, vp, vp]
        cf, cd, hp = ctypes.c_float, ctypes.c_double, ctypes.POINTER(_HeadsArg)
        lib.sparse_layer_norm_forward.argtypes = [vp, i64, ci, ci, vp, vp, cf, vp, vp, vp, vp]
        lib.sparse_layer_norm_backward.argtypes = [vp, vp, i64, ci, ci, vp, vp, vp, vp, vp, vp, vp]
        lib.sparse_rms_norm_forward.argtypes = [vp, vp, i64, ci, ci, vp, cf, vp, vp, vp, vp]
        lib.sparse_rms_norm_quantize_forward.argtypes = [vp, vp, i64, ci, ci, vp, cf, ci, vp, vp, vp, vp, vp]
        lib.sparse_rms_norm_backward.argtypes = [vp, vp, vp, i64, ci, ci, vp, vp, vp, vp, vp]
        lib.sparse_embedding_forward.argtypes = [vp, ci, ci, ci, vp, ci, i64, cf, vp, vp]
        lib.sparse_embedding_backward.argtypes = [vp, ci, ci, ci, vp, ci, i64, cf, vp, vp]
        lib.sparse_rope_frequencies.argtypes = [ci, cd, ci, cd, cd, ctypes.POINTER(cf), ctypes.POINTER(cf)]
        for rope in (lib.sparse_rope_forward, lib.sparse_rope_backward):
            rope.argtypes = [hp, i64, ci, ci, ci, vp, i64, ci, vp, ci, ci, cf, hp, vp]
        lib.sparse_attention_forward.argtypes = [hp, hp, hp, i64, i64, vp, vp, ci, ci, ci, ci, ci, cf, hp, vp, vp]
        lib.sparse_attention_backward.argtypes = [hp, hp, hp, hp, hp, vp, i64, i64, vp, vp, ci, ci, ci, ci, ci, cf, hp,
                                                  hp, hp, vp]
        lib.sparse_window_attention_forward.argtypes = [hp, hp, hp, i64, i64, vp, vp, vp, ci, ci, ci, ci, ci, cf, i64, i64,
                                                        ci, hp, vp, vp]
        lib.sparse_window_attention_backward.argtypes = [hp, hp, hp, hp, hp, vp, i64, i64, vp, vp, ci, ci, ci, ci, ci, cf,
                                                         i64, i64, ci, hp, hp, hp, vp]
        for name in C_FUNCTIONS[:-2]:
            getattr(lib, name).restype = ci
        lib.subm_status_string.argtypes = [ci]
        lib.subm_status_string.restype = ctypes.c_char_p
        lib.subm_last_error.argtypes = []
        lib.subm_last_error.restype = ctypes.c_char_p
        if path is None:
            _lib = lib
        return lib


def _check(lib, func: str, status: int) -> None:
    if status != 0:
        name = lib.subm_status_string(status).decode()
        detail = lib.subm_last_error().decode()
        raise SubmError(func, status, name, detail)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_ptr(stream, device) -> int:
    if stream is None:
        if _raw_stream is not None:  # the current stream's handle without building a Stream object
            return _raw_stream(device.index if device.index is not None else torch.cuda.current_device())
        return torch.cuda.current_stream(device).cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


class _Current:
    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


_CURRENT = _Current()


def _on_device(device):
    """Make `device` current for a call, skipping the switch when it already is."""
    if device.index is None or device.index == torch.cuda.current_device():
        return _CURRENT
    return torch.cuda.device(device)


def _device_tensor(t: torch.Tensor, what: str) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{what} must be a device tensor (got {t.device})")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")


class IndiceMap:
    """Owner of one built indice map (submconv_map_t) for one coordinate set."""

    def __init__(self, handle: int, device: torch.device, n: int):
        self._handle = handle
        self.device = device
        self.n = n
        self._pairs = None

    @property
    def pairs(self) -> int:
        """Total pair count (rulebook entries >= 0, centre included)."""
        if self._pairs is None:
            self._pairs = sparse_indice_map_info(self)[1]
        return self._pairs

    @property
    def mode(self) -> int:
        """SUBM_MAP_HASH or SUBM_MAP_GRID: the structure the build used."""
        return sparse_indice_map_mode(self)

    @property
    def handle(self) -> int:
        if self._handle is None:
            raise ValueError("indice map already freed")
        return self._handle

    def check(self) -> None:
        """Raise the build's coordinate error, if any (waits for an asynchronous build's insert)."""
        sparse_indice_map_status(self)

    def free(self) -> None:
        """Release the map.  No work using it may still be in flight."""
        if self._handle is not None:
            lib = load_library()
            h, self._handle = self._handle, None
            _check(lib, "sparse_indice_map_free", lib.sparse_indice_map_free(h))

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.free()

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def sparse_indice_map_build(coords: torch.Tensor, stream=None, sync: bool = True) -> IndiceMap:
    """Build the indice map of int32 device coordinates [N, 4] = (b, z, y, x).

    sync=False enqueues the build without any host wait (sparse_indice_map_build_async):
    coordinate errors are then raised by IndiceMap.check() or by the first call that reads the
    map on the host."""
    if not sync:
        return sparse_indice_map_build_async(coords, SUBM_MAP_AUTO, stream)
    return sparse_indice_map_build_ex(coords, SUBM_MAP_AUTO, stream)


def sparse_indice_map_build_async(coords: torch.Tensor, mode: int = SUBM_MAP_AUTO, stream=None) -> IndiceMap:
    """Enqueue the build with no host wait; see IndiceMap.check for its coordinate status."""
    return _build(coords, mode, stream, "sparse_indice_map_build_async")


def sparse_indice_map_status(m: IndiceMap) -> None:
    """Raise SubmError with the build's coordinate error, if any."""
    lib = load_library()
    _check(lib, "sparse_indice_map_status", lib.sparse_indice_map_status(m.handle))


def sparse_indice_map_build_ex(coords: torch.Tensor, mode: int, stream=None) -> IndiceMap:
    """Build the indice map with an explicit structure request (SUBM_MAP_AUTO / _HASH / _GRID)."""
    return _build(coords, mode, stream, "sparse_indice_map_build_ex")


def _build(coords: torch.Tensor, mode: int, stream, func: str) -> IndiceMap:
    _device_tensor(coords, "coords")
    if coords.dtype != torch.int32 or coords.dim() != 2 or coords.shape[1] != 4:
        raise ValueError("coords must be int32 [N, 4]")
    lib = load_library()
    out = ctypes.c_void_p()
    with _on_device(coords.device):
        st = getattr(lib, func)(coords.data_ptr(), coords.shape[0], int(mode), _stream_ptr(stream, coords.device),
                                ctypes.byref(out))
    _check(lib, func, st)
    return IndiceMap(out.value, coords.device, coords.shape[0])


def sparse_indice_map_mode(m: IndiceMap) -> int:
    lib = load_library()
    mode = ctypes.c_int()
    _check(lib, "sparse_indice_map_mode", lib.sparse_indice_map_mode(m.handle, ctypes.byref(mode)))
    return mode.value


SUBM_PLAN_NONE, SUBM_PLAN_PENDING, SUBM_PLAN_READY, SUBM_PLAN_OVERFLOW = 0, 1, 2, 3
SUBM_ORDER_NONE, SUBM_ORDER_ON, SUBM_ORDER_OFF = 0, 1, 2


def subm_release_cached_memory(device=None) -> None:
    """Free the library's cached device memory on `device` (default: torch's current device),
    after waiting for that device; see subm_release_cached_memory in include/submconv.h."""
    lib = load_library()
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with _on_device(dev):
        _check(lib, "subm_release_cached_memory", lib.subm_release_cached_memory())


def subm_timing_events(start, stop) -> None:
    """Bind two timing events (torch.cuda.Event, already recorded once so that they exist) to the
    next convolution kernel this thread launches: start.elapsed_time(stop) is then that kernel's
    own duration.  None, None cancels.  See subm_timing_events in include/submconv.h."""
    lib = load_library()
    h = lambda e: None if e is None else ctypes.c_void_p(e.cuda_event)
    _check(lib, "subm_timing_events", lib.subm_timing_events(h(start), h(stop)))


def subm_mfma_rate(iters: int, blocks: int, device=None, stream=None):
    """Launch the matrix-core rate loop (see subm_mfma_rate in include/submconv.h) on `stream`
    (default: torch's current stream).  Returns (sink, clocks) device tensors; the caller times
    the launch.  FLOP = blocks * 4 waves * iters * 8 * 32768."""
    lib = load_library()
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    sink = torch.empty(blocks * 256, dtype=torch.float32, device=dev)
    clocks = torch.empty(2 * blocks, dtype=torch.int64, device=dev)
    s = torch.cuda.current_stream(dev) if stream is None else stream
    with _on_device(dev):
        _check(lib, "subm_mfma_rate", lib.subm_mfma_rate(int(iters), int(blocks), ctypes.c_void_p(sink.data_ptr()),
                                                           ctypes.c_void_p(clocks.data_ptr()),
                                                           ctypes.c_void_p(s.cuda_stream)))
    return sink, clocks


def sparse_indice_map_row_order_state(m: IndiceMap) -> int:
    """State of the map's sparse-row order: SUBM_ORDER_NONE / _ON / _OFF (waits for its kernels)."""
    lib = load_library()
    state = ctypes.c_int()
    _check(lib, "sparse_indice_map_row_order_state",
           lib.sparse_indice_map_row_order_state(m.handle, ctypes.byref(state)))
    return state.value


def sparse_indice_map_plan_state(m: IndiceMap) -> int:
    """State of the map's neighbour-pool plan: SUBM_PLAN_NONE / _PENDING / _READY / _OVERFLOW."""
    lib = load_library()
    state = ctypes.c_int()
    _check(lib, "sparse_indice_map_plan_state", lib.sparse_indice_map_plan_state(m.handle, ctypes.byref(state)))
    return state.value


def sparse_indice_map_free(m: IndiceMap) -> None:
    m.free()


def sparse_indice_map_info(m: IndiceMap) -> tuple[int, int]:
    """(voxel count, pair count) of a built map."""
    lib = load_library()
    n = ctypes.c_int64()
    pairs = ctypes.c_int64()
    _check(lib, "sparse_indice_map_info", lib.sparse_indice_map_info(m.handle, ctypes.byref(n), ctypes.byref(pairs)))
    return n.value, pairs.value


def sparse_indice_map_offset_counts(m: IndiceMap) -> list[int]:
    """Pairs per tap k (27 values)."""
    lib = load_library()
    arr = (ctypes.c_int64 * TAPS)()
    _check(lib, "sparse_indice_map_offset_counts", lib.sparse_indice_map_offset_counts(m.handle, arr))
    return list(arr)


def sparse_indice_map_copy_nbr(m: IndiceMap, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The rulebook nbr [N, 27] int32 (input row of the neighbour, or -1) as a device tensor."""
    if out is None:
        out = torch.empty((m.n, TAPS), dtype=torch.int32, device=m.device)
    _device_tensor(out, "out")
    if out.dtype != torch.int32 or tuple(out.shape) != (m.n, TAPS):
        raise ValueError("out must be int32 [N, 27]")
    lib = load_library()
    with _on_device(out.device):
        st = lib.sparse_indice_map_copy_nbr(m.handle, out.data_ptr(), _stream_ptr(stream, out.device))
    _check(lib, "sparse_indice_map_copy_nbr", st)
    return out


def _conv_args(feats, weight, bias, out, need_out=False):
    _device_tensor(feats, "feats")
    _device_tensor(weight, "weight")
    if feats.dim() != 2 or weight.dim() != 5:
        raise ValueError("feats must be [N, Cin] and weight KRSC [Cout, k, k, k, Cin]")
    k = weight.shape[1]
    if weight.shape[2] != k or weight.shape[3] != k:
        raise ValueError("weight spatial dims must be equal (KRSC [Cout, k, k, k, Cin])")
    if weight.shape[4] != feats.shape[1]:
        raise ValueError("weight Cin does not match feats")
    if feats.dtype not in _DTYPE_CODES or weight.dtype != feats.dtype:
        raise ValueError("feats and weight must share one of float32 / float16 / bfloat16")
    n, cout = feats.shape[0], weight.shape[0]
    bias_ptr = None
    if bias is not None:
        _device_tensor(bias, "bias")
        if bias.dtype != feats.dtype or tuple(bias.shape) != (cout,):
            raise ValueError("bias must be [Cout] in the feats dtype")
        bias_ptr = bias.data_ptr()
    if out is None:
        if need_out:
            raise ValueError("out must be given (this call allocates nothing)")
        out = torch.empty((n, cout), dtype=feats.dtype, device=feats.device)
    _device_tensor(out, "out")
    if out.dtype != feats.dtype or tuple(out.shape) != (n, cout):
        raise ValueError("out must be [N, Cout] in the feats dtype")
    return k, bias_ptr, out


def subm_conv3d_forward_per_offset(m: IndiceMap, feats: torch.Tensor, weight: torch.Tensor,
                                   bias: torch.Tensor | None = None, out: torch.Tensor | None = None,
                                   stream=None) -> torch.Tensor:
    """SubMConv3d (k = 3) computed as a per-offset gather -> GEMM -> scatter-add loop."""
    k, bias_ptr, out = _conv_args(feats, weight, bias, out)
    if k != 3:
        raise ValueError("the per-offset path is the k = 3 convolution")
    lib = load_library()
    with _on_device(feats.device):
        st = lib.subm_conv3d_forward_per_offset(m.handle, feats.shape[0], feats.shape[1], weight.shape[0],
                                                _DTYPE_CODES[feats.dtype], feats.data_ptr(), weight.data_ptr(),
                                                bias_ptr, out.data_ptr(), _stream_ptr(stream, feats.device))
    _check(lib, "subm_conv3d_forward_per_offset", st)
    return out


def subm_conv3d_forward(m: IndiceMap | None, feats: torch.Tensor, weight: torch.Tensor,
                        bias: torch.Tensor | None = None, out: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """SubMConv3d forward: feats [N, Cin], KRSC weight [Cout, k, k, k, Cin] (k = 3 or 1), bias [Cout]."""
    k, bias_ptr, out = _conv_args(feats, weight, bias, out)
    n, cin, cout = feats.shape[0], feats.shape[1], weight.shape[0]
    lib = load_library()
    handle = None if m is None else m.handle
    with _on_device(feats.device):
        st = lib.subm_conv3d_forward(handle, n, k, cin, cout, _DTYPE_CODES[feats.dtype], feats.data_ptr(),
                                     weight.data_ptr(), bias_ptr, out.data_ptr(), _stream_ptr(stream, feats.device))
    _check(lib, "subm_conv3d_forward", st)
    return out


def subm_conv3d_forward_noalloc(m: IndiceMap | None, feats: torch.Tensor, weight: torch.Tensor,
                                bias: torch.Tensor | None, out: torch.Tensor, stream=None) -> torch.Tensor:
    """subm_conv3d_forward with no device allocation (out must be given); see subm_conv3d_forward_noalloc
    in include/submconv.h."""
    k, bias_ptr, out = _conv_args(feats, weight, bias, out, need_out=True)
    n, cin, cout = feats.shape[0], feats.shape[1], weight.shape[0]
    lib = load_library()
    handle = None if m is None else m.handle
    with _on_device(feats.device):
        st = lib.subm_conv3d_forward_noalloc(handle, n, k, cin, cout, _DTYPE_CODES[feats.dtype], feats.data_ptr(),
                                             weight.data_ptr(), bias_ptr, out.data_ptr(),
                                             _stream_ptr(stream, feats.device))
    _check(lib, "subm_conv3d_forward_noalloc", st)
    return out


# --------------------------------------------------------------------------- structure ops

class Subdivision:
    """Owner of one coarse / fine relation (sparse_subdivision_t): subdivide, downsample or masked
    upsample structure."""

    def __init__(self, handle: int, device: torch.device):
        self._handle = handle
        self.device = device
        self.n_coarse, self.n_fine = sparse_subdivision_info(self)
        self.kind = sparse_subdivision_kind(self)

    @property
    def handle(self) -> int:
        if self._handle is None:
            raise ValueError("subdivision already freed")
        return self._handle

    def coarse_coords(self, stream=None) -> torch.Tensor:
        return sparse_subdivision_copy(self, SUBM_COARSE, stream=stream)

    def fine_coords(self, stream=None) -> torch.Tensor:
        return sparse_subdivision_copy(self, SUBM_FINE, stream=stream)

    def parent(self, stream=None) -> torch.Tensor:
        return sparse_subdivision_copy(self, SUBM_PARENT, stream=stream)

    def free(self) -> None:
        if self._handle is not None:
            lib = load_library()
            h, self._handle = self._handle, None
            _check(lib, "sparse_subdivision_free", lib.sparse_subdivision_free(h))

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.free()

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def _coords_arg(coords: torch.Tensor) -> None:
    _device_tensor(coords, "coords")
    if coords.dtype != torch.int32 or coords.dim() != 2 or coords.shape[1] != 4:
        raise ValueError("coords must be int32 [N, 4]")


def _build_subdivision(func: str, coords: torch.Tensor, args: tuple, stream) -> Subdivision:
    lib = load_library()
    out = ctypes.c_void_p()
    with _on_device(coords.device):
        st = getattr(lib, func)(*args, _stream_ptr(stream, coords.device), ctypes.byref(out))
    _check(lib, func, st)
    return Subdivision(out.value, coords.device)


def sparse_subdivide(coords: torch.Tensor, stream=None) -> Subdivision:
    """The 8 children of every voxel of int32 [N, 4] (b, z, y, x), C order, parent-major."""
    _coords_arg(coords)
    return _build_subdivision("sparse_subdivide", coords, (coords.data_ptr(), coords.shape[0]), stream)


def sparse_downsample_build(coords: torch.Tensor, stream=None) -> Subdivision:
    """The 2x coarse cells of int32 [N, 4] coordinates and the fine-to-coarse relation."""
    _coords_arg(coords)
    return _build_subdivision("sparse_downsample_build", coords, (coords.data_ptr(), coords.shape[0]), stream)


def sparse_upsample_masked_build(coords: torch.Tensor, mask: torch.Tensor, stream=None) -> Subdivision:
    """Masked 2x expansion of int32 [N, 4] coordinates by a uint8 [N, 8] child mask."""
    _coords_arg(coords)
    _device_tensor(mask, "mask")
    if mask.dtype != torch.uint8 or tuple(mask.shape) != (coords.shape[0], 8):
        raise ValueError("mask must be uint8 [N, 8]")
    return _build_subdivision("sparse_upsample_masked_build", coords,
                              (coords.data_ptr(), mask.data_ptr(), coords.shape[0]), stream)


def sparse_subdivision_info(s: Subdivision) -> tuple[int, int]:
    """(n_coarse, n_fine)."""
    lib = load_library()
    a, b = ctypes.c_int64(), ctypes.c_int64()
    _check(lib, "sparse_subdivision_info", lib.sparse_subdivision_info(s.handle, ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


def sparse_subdivision_kind(s: Subdivision) -> int:
    lib = load_library()
    k = ctypes.c_int()
    _check(lib, "sparse_subdivision_kind", lib.sparse_subdivision_kind(s.handle, ctypes.byref(k)))
    return k.value


def sparse_subdivision_coords(s: Subdivision, level: int) -> int:
    """Raw device address of the handle-owned coarse / fine coordinates (0 when empty)."""
    lib = load_library()
    p = ctypes.c_void_p()
    _check(lib, "sparse_subdivision_coords", lib.sparse_subdivision_coords(s.handle, int(level), ctypes.byref(p)))
    return p.value or 0


def sparse_subdivision_parent(s: Subdivision) -> int:
    """Raw device address of the handle-owned parent index (0 when empty)."""
    lib = load_library()
    p = ctypes.c_void_p()
    _check(lib, "sparse_subdivision_parent", lib.sparse_subdivision_parent(s.handle, ctypes.byref(p)))
    return p.value or 0


def sparse_subdivision_copy(s: Subdivision, what: int, out: torch.Tensor | None = None,
                            stream=None) -> torch.Tensor:
    """Copy of the coarse coords (SUBM_COARSE), fine coords (SUBM_FINE) or parent index (SUBM_PARENT)."""
    shape = {SUBM_COARSE: (s.n_coarse, 4), SUBM_FINE: (s.n_fine, 4), SUBM_PARENT: (s.n_fine,)}
    if what not in shape:
        raise ValueError("what must be SUBM_COARSE, SUBM_FINE or SUBM_PARENT")
    if out is None:
        out = torch.empty(shape[what], dtype=torch.int32, device=s.device)
    _device_tensor(out, "out")
    if out.dtype != torch.int32 or tuple(out.shape) != shape[what]:
        raise ValueError(f"out must be int32 {shape[what]}")
    lib = load_library()
    with _on_device(out.device):
        st = lib.sparse_subdivision_copy(s.handle, int(what), out.data_ptr(), _stream_ptr(stream, out.device))
    _check(lib, "sparse_subdivision_copy", st)
    return out


def sparse_subdivision_free(s: Subdivision) -> None:
    s.free()


def _feature_pair(inp: torch.Tensor, rows_in: int, out: torch.Tensor | None, rows_out: int, what: str):
    _device_tensor(inp, what)
    if inp.dim() != 2 or inp.shape[0] != rows_in or inp.dtype not in _DTYPE_CODES:
        raise ValueError(f"{what} must be [{rows_in}, C] float32 / float16 / bfloat16")
    if out is None:
        out = torch.empty((rows_out, inp.shape[1]), dtype=inp.dtype, device=inp.device)
    _device_tensor(out, "out")
    if out.dtype != inp.dtype or tuple(out.shape) != (rows_out, inp.shape[1]):
        raise ValueError(f"out must be [{rows_out}, {inp.shape[1]}] in the input dtype")
    return out


def sparse_downsample_forward(s: Subdivision, fine: torch.Tensor, mode: int, out: torch.Tensor | None = None,
                              stream=None) -> torch.Tensor:
    """Pool fine features [n_fine, C] onto the coarse rows: mode SUBM_POOL_MAX or SUBM_POOL_MEAN."""
    out = _feature_pair(fine, s.n_fine, out, s.n_coarse, "fine")
    lib = load_library()
    with _on_device(fine.device):
        st = lib.sparse_downsample_forward(s.handle, fine.shape[1], _DTYPE_CODES[fine.dtype], int(mode),
                                           fine.data_ptr(), out.data_ptr(), _stream_ptr(stream, fine.device))
    _check(lib, "sparse_downsample_forward", st)
    return out


def sparse_upsample_forward(s: Subdivision, coarse: torch.Tensor, out: torch.Tensor | None = None,
                            stream=None) -> torch.Tensor:
    """Fine features [n_fine, C]: every fine row a copy of its parent's coarse row."""
    out = _feature_pair(coarse, s.n_coarse, out, s.n_fine, "coarse")
    lib = load_library()
    with _on_device(coarse.device):
        st = lib.sparse_upsample_forward(s.handle, coarse.shape[1], _DTYPE_CODES[coarse.dtype], coarse.data_ptr(),
                                         out.data_ptr(), _stream_ptr(stream, coarse.device))
    _check(lib, "sparse_upsample_forward", st)
    return out


def sparse_indice_map_subdivide(parent: IndiceMap, s: Subdivision, stream=None) -> IndiceMap:
    """Indice map of a subdivide's fine set, derived from the map of its coarse set."""
    lib = load_library()
    out = ctypes.c_void_p()
    with _on_device(s.device):
        st = lib.sparse_indice_map_subdivide(parent.handle, s.handle, _stream_ptr(stream, s.device),
                                             ctypes.byref(out))
    _check(lib, "sparse_indice_map_subdivide", st)
    return IndiceMap(out.value, s.device, s.n_fine)


# --------------------------------------------------------------------------- normalisation

def _norm_affine(c, dtype, gamma, beta):
    ptrs = []
    for t, name in ((gamma, "gamma"), (beta, "beta")):
        if t is None:
            ptrs.append(None)
            continue
        _device_tensor(t, name)
        if t.dtype != dtype or tuple(t.shape) != (c,):
            raise ValueError(f"{name} must be [C] in the activation dtype")
        ptrs.append(t.data_ptr())
    return ptrs


def _offsets_arg(item_offsets):
    _device_tensor(item_offsets, "item_offsets")
    if item_offsets.dtype != torch.int64 or item_offsets.dim() != 1 or item_offsets.shape[0] < 2:
        raise ValueError("item_offsets must be int64 [num_items + 1]")


def subm_conv3d_forward_group_norm_act(m: IndiceMap | None, feats: torch.Tensor, weight: torch.Tensor,
                                       bias: torch.Tensor | None, item_offsets: torch.Tensor, groups: int,
                                       gamma: torch.Tensor | None = None, beta: torch.Tensor | None = None,
                                       eps: float = 1e-5, act: int = SUBM_ACT_NONE,
                                       out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """act(group_norm(SubMConv3d(feats))) with the group statistics taken in the conv epilogue."""
    k, bias_ptr, out = _conv_args(feats, weight, bias, out)
    _offsets_arg(item_offsets)
    ptrs = _norm_affine(weight.shape[0], feats.dtype, gamma, beta)
    lib = load_library()
    handle = None if m is None else m.handle
    with _on_device(feats.device):
        st = lib.subm_conv3d_forward_group_norm_act(
            handle, feats.shape[0], k, feats.shape[1], weight.shape[0], _DTYPE_CODES[feats.dtype], feats.data_ptr(),
            weight.data_ptr(), bias_ptr, item_offsets.data_ptr(), item_offsets.shape[0] - 1, int(groups), ptrs[0],
            ptrs[1], float(eps), int(act), out.data_ptr(), _stream_ptr(stream, feats.device))
    _check(lib, "subm_conv3d_forward_group_norm_act", st)
    return out


def sparse_group_norm_act(x: torch.Tensor, item_offsets: torch.Tensor, groups: int,
                          gamma: torch.Tensor | None = None, beta: torch.Tensor | None = None,
                          eps: float = 1e-5, act: int = SUBM_ACT_NONE, out: torch.Tensor | None = None,
                          stream=None) -> torch.Tensor:
    """Group normalisation per batch item (rows item_offsets[b] .. item_offsets[b+1] - 1, int64
    device tensor) then an activation (SUBM_ACT_NONE / _SILU / _RELU).  out may be x (in place)."""
    _device_tensor(x, "x")
    if x.dim() != 2 or x.dtype not in _DTYPE_CODES:
        raise ValueError("x must be [N, C] float32 / float16 / bfloat16")
    _offsets_arg(item_offsets)
    c = x.shape[1]
    ptrs = _norm_affine(c, x.dtype, gamma, beta)
    if out is None:
        out = torch.empty_like(x)
    _device_tensor(out, "out")
    if out.dtype != x.dtype or out.shape != x.shape:
        raise ValueError("out must match x")
    lib = load_library()
    with _on_device(x.device):
        st = lib.sparse_group_norm_act(x.data_ptr(), x.shape[0], c, _DTYPE_CODES[x.dtype], item_offsets.data_ptr(),
                                       item_offsets.shape[0] - 1, int(groups), ptrs[0], ptrs[1], float(eps), int(act),
                                       out.data_ptr(), _stream_ptr(stream, x.device))
    _check(lib, "sparse_group_norm_act", st)
    return out


# --------------------------------------------------------------------------- transformer block
#
# (The smallest calls here take as long on the host as on the device, so these functions test the
# common case with few attribute reads and leave naming the fault to the helpers.)

_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _empty(shape, dtype, device, stream):
    """A new tensor that belongs to the stream the call runs on (its memory is then reused in that
    stream's order)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    s = torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream
    with torch.cuda.stream(s):
        return torch.empty(shape, dtype=dtype, device=device)


def _empty_like(t, stream):
    """_empty of a tensor's shape, contiguous."""
    if stream is None and t.is_contiguous():
        return torch.empty_like(t)
    return _empty(t.shape, t.dtype, t.device, stream)


def _run(func: str, device: int, stream, *args) -> None:
    """Call the library on a device (made current for it) and stream; raise its error."""
    lib = _lib or load_library()
    s = _stream_ptr(stream, torch.device("cuda", device)) if stream is not None or _raw_stream is None else _raw_stream(device)
    if device == _current_device():
        st = getattr(lib, func)(*args, s)
    else:
        with torch.cuda.device(device):
            st = getattr(lib, func)(*args, s)
    if st != 0:
        _check(lib, func, st)


def _matrix(t, what):
    """(rows, columns, dtype code) of a contiguous device matrix."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous():
        _device_tensor(t, what)
    code = _DTYPE_CODES.get(t.dtype)
    if t.dim() != 2 or code is None:
        raise ValueError(f"{what} must be [N, C] float32 / float16 / bfloat16")
    n, c = t.shape
    return n, c, code


def _vector(t, shape, dtype, device, what):
    """data_ptr of an optional contiguous device tensor of that shape and dtype."""
    if t is None:
        return None
    _device_tensor(t, what)
    if t.dtype != dtype or tuple(t.shape) != shape or t.device != device:
        raise ValueError(f"{what} must be {list(shape)} {dtype} on {device}")
    return t.data_ptr()


def sparse_layer_norm_forward(x: torch.Tensor, gamma: torch.Tensor | None = None, beta: torch.Tensor | None = None,
                              eps: float = 1e-5, stats: bool = False, out: torch.Tensor | None = None, stream=None):
    """Layer norm of the rows of x [N, C]: (y, mean, rstd), the float32 statistics [N] only with
    stats=True (else None), which the backward pass needs.  out may be x (in place)."""
    n, c, code = _matrix(x, "x")
    g = None if gamma is None else _vector(gamma, (c,), x.dtype, x.device, "gamma")
    b = None if beta is None else _vector(beta, (c,), x.dtype, x.device, "beta")
    if out is None:
        out = _empty_like(x, stream)
        y = out.data_ptr()
    else:
        y = _vector(out, (n, c), x.dtype, x.device, "out")
    mean = rstd = mean_ptr = rstd_ptr = None
    if stats:
        mean, rstd = _empty((n,), torch.float32, x.device, stream), _empty((n,), torch.float32, x.device, stream)
        mean_ptr = mean.data_ptr()
        rstd_ptr = rstd.data_ptr()
    _run("sparse_layer_norm_forward", x.get_device(), stream, x.data_ptr(), n, c, code, g, b, eps, y, mean_ptr, rstd_ptr)
    return out, mean, rstd


def sparse_layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                               gamma: torch.Tensor | None = None, weight_grads: bool = True,
                               out: torch.Tensor | None = None, stream=None):
    """Gradients of sparse_layer_norm_forward: (dx, dgamma, dbeta), the last two None with
    weight_grads=False.  mean, rstd: the forward pass's.  out may be dy (in place)."""
    n, c, code = _matrix(x, "x")
    if dy is None or mean is None or rstd is None:
        raise ValueError("dy, mean and rstd are required")
    dy_ptr = _vector(dy, (n, c), x.dtype, x.device, "dy")
    m = _vector(mean, (n,), torch.float32, x.device, "mean")
    r = _vector(rstd, (n,), torch.float32, x.device, "rstd")
    g = None if gamma is None else _vector(gamma, (c,), x.dtype, x.device, "gamma")
    if out is None:
        out = _empty_like(x, stream)
        dx = out.data_ptr()
    else:
        dx = _vector(out, (n, c), x.dtype, x.device, "out")
    dgamma = dbeta = dg_ptr = db_ptr = None
    if weight_grads:
        dgamma, dbeta = _empty((c,), x.dtype, x.device, stream), _empty((c,), x.dtype, x.device, stream)
        dg_ptr, db_ptr = dgamma.data_ptr(), dbeta.data_ptr()
    _run("sparse_layer_norm_backward", x.get_device(), stream, dy_ptr, x.data_ptr(), n, c, code, g, m, r, dx, dg_ptr, db_ptr)
    return out, dgamma, dbeta


def _alike(t, shape, like, what):
    """_vector of a tensor's dtype and device, with few attribute reads."""
    if isinstance(t, torch.Tensor) and t.dtype is like.dtype and t.shape == shape and t.get_device() == like.get_device() and t.is_contiguous():
        return t.data_ptr()
    return _vector(t, tuple(shape), like.dtype, like.device, what)


def _rms_norm_args(x, gamma, residual, total, stats, stream):
    """(rows, channels, dtype code, pointers of gamma and residual, total and its pointer, rstd and its)."""
    n, c, code = _matrix(x, "x")
    g = r = t = rstd = rstd_ptr = None
    if gamma is not None:
        g = _alike(gamma, (c,), x, "gamma")
    if residual is not None:
        r = _alike(residual, x.shape, x, "residual")
        if total is None:
            total = _empty_like(x, stream)
            t = total.data_ptr()
    if total is not None and t is None:
        t = _alike(total, x.shape, x, "total")
    if stats:
        rstd = _empty((n,), torch.float32, x.device, stream)
        rstd_ptr = rstd.data_ptr()
    return n, c, code, g, r, total, t, rstd, rstd_ptr


def sparse_rms_norm_forward(x: torch.Tensor, gamma: torch.Tensor | None = None, residual: torch.Tensor | None = None,
                            eps: float = 1e-6, stats: bool = False, out: torch.Tensor | None = None,
                            total: torch.Tensor | None = None, stream=None):
    """Root-mean-square norm of the rows of x + residual [N, C]: (y, total, rstd).  total is x + residual (None
    without a residual), rstd float32 [N] only with stats=True; the backward pass needs both.  out and total
    may be x or residual (in place)."""
    n, c, code, g, r, total, t, rstd, rstd_ptr = _rms_norm_args(x, gamma, residual, total, stats, stream)
    if out is None:
        out = _empty_like(x, stream)
        y = out.data_ptr()
    else:
        y = _alike(out, x.shape, x, "out")
    _run("sparse_rms_norm_forward", x.get_device(), stream, x.data_ptr(), r, n, c, code, g, eps, y, t, rstd_ptr)
    return out, total, rstd


def sparse_rms_norm_quantize_forward(x: torch.Tensor, gamma: torch.Tensor | None = None, residual: torch.Tensor | None = None,
                                     eps: float = 1e-6, group: int = 128, stats: bool = False,
                                     total: torch.Tensor | None = None, stream=None):
    """sparse_rms_norm_forward with y in 8 bits: (q float8_e4m3fn [N, C], scales float32 [N, groups], total, rstd),
    y = q * scale with a scale each `group` channels (32, 64, 128; 0: a row)."""
    n, c, code, g, r, total, t, rstd, rstd_ptr = _rms_norm_args(x, gamma, residual, total, stats, stream)
    q = _empty((n, c), torch.float8_e4m3fn, x.device, stream)
    scales = _empty((n, -(-c // group) if group > 0 else 1), torch.float32, x.device, stream)
    _run("sparse_rms_norm_quantize_forward", x.get_device(), stream, x.data_ptr(), r, n, c, code, g, eps, group, q.data_ptr(),
         scales.data_ptr(), t, rstd_ptr)
    return q, scales, total, rstd


def sparse_rms_norm_backward(dy: torch.Tensor, total: torch.Tensor, rstd: torch.Tensor, gamma: torch.Tensor | None = None,
                             dtotal: torch.Tensor | None = None, weight_grads: bool = True,
                             out: torch.Tensor | None = None, stream=None):
    """Gradients of sparse_rms_norm_forward: (dx, dgamma), dx that of x and of residual alike, dgamma None with
    weight_grads=False.  total, rstd: the forward pass's (total is x without a residual); dtotal: the gradient
    of total.  out may be dy or dtotal (in place)."""
    n, c, code = _matrix(total, "total")
    if dy is None or rstd is None:
        raise ValueError("dy and rstd are required")
    dy_ptr = _alike(dy, total.shape, total, "dy")
    r = _vector(rstd, (n,), torch.float32, total.device, "rstd")
    g = None if gamma is None else _alike(gamma, (c,), total, "gamma")
    dt = None if dtotal is None else _alike(dtotal, total.shape, total, "dtotal")
    if out is None:
        out = _empty_like(total, stream)
        dx = out.data_ptr()
    else:
        dx = _alike(out, total.shape, total, "out")
    dgamma = _empty((c,), total.dtype, total.device, stream) if weight_grads else None
    _run("sparse_rms_norm_backward", total.get_device(), stream, dy_ptr, total.data_ptr(), dt, n, c, code, g, r, dx,
         None if dgamma is None else dgamma.data_ptr())
    return out, dgamma


def _tokens_arg(tokens, device):
    """(data_ptr, bytes of a token, count)."""
    if not isinstance(tokens, torch.Tensor) or not tokens.is_cuda or not tokens.is_contiguous():
        _device_tensor(tokens, "tokens")
    if tokens.dim() != 1 or tokens.dtype not in (torch.int32, torch.int64) or tokens.get_device() != device:
        raise ValueError("tokens must be int32 or int64 [N] on the same device")
    return tokens.data_ptr(), tokens.element_size(), tokens.shape[0]


def sparse_embedding_forward(table: torch.Tensor, tokens: torch.Tensor, scale: float = 1.0,
                             out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """scale * table[tokens]: table [rows, C], tokens int32 / int64 [N]; zeros for a token outside the table."""
    rows, c, code = _matrix(table, "table")
    t, size, n = _tokens_arg(tokens, table.get_device())
    if out is None:
        out = _empty((n, c), table.dtype, table.device, stream)
        y = out.data_ptr()
    else:
        y = _alike(out, (n, c), table, "out")
    _run("sparse_embedding_forward", table.get_device(), stream, table.data_ptr(), rows, c, code, t, size, n, scale, y)
    return out


def sparse_embedding_backward(dout: torch.Tensor, tokens: torch.Tensor, rows: int, scale: float = 1.0,
                              out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gradient of sparse_embedding_forward's table: [rows, C], every row written."""
    n, c, code = _matrix(dout, "dout")
    t, size, count = _tokens_arg(tokens, dout.get_device())
    if count != n:
        raise ValueError("dout and tokens must have the same rows")
    if not 0 < rows < 2 ** 31:
        raise ValueError("rows must be 1 .. 2^31 - 1")
    if out is None:
        out = _empty((rows, c), dout.dtype, dout.device, stream)
        d = out.data_ptr()
    else:
        d = _alike(out, (rows, c), dout, "out")
    _run("sparse_embedding_backward", dout.get_device(), stream, dout.data_ptr(), rows, c, code, t, size, n, scale, d)
    return out


def _heads_arg(t, what, like=None):
    """subm_heads_t of a [N, heads, head_dim] view whose channels are contiguous; `like`: the
    tensor whose dtype and device it must share."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{what} must be a device tensor (got {t.device})")
    shape = t.shape
    if len(shape) != 3 or t.dtype not in _DTYPE_CODES:
        raise ValueError(f"{what} must be [N, heads, head_dim] float32 / float16 / bfloat16")
    row, head, channel = t.stride()
    if channel != 1 and shape[2] > 1:
        raise ValueError(f"{what}: the channels of a head must be contiguous")
    if like is not None and (t.dtype != like.dtype or t.get_device() != like.get_device()):
        raise ValueError(f"{what} must be {like.dtype} on {like.device}")
    # (a stride that no step takes is free: torch reports any value for it)
    return _HeadsArg(t.data_ptr(), row if shape[0] > 1 else shape[1] * shape[2], head if shape[1] > 1 else shape[2])


def sparse_rope_frequencies(count: int, base: float = 10000.0, scaling: int = SUBM_ROPE_PLAIN, factor: float = 1.0,
                            trained_length: float = 1.0):
    """(float32 CPU tensor [count], magnitude): the frequencies of one axis and the factor of the
    rotated channels; scaling is one of SUBM_ROPE_PLAIN / _LINEAR / _BASE / _PARTS."""
    freq = torch.empty(max(int(count), 1), dtype=torch.float32)
    magnitude = ctypes.c_float()
    lib = load_library()
    st = lib.sparse_rope_frequencies(int(count), float(base), int(scaling), float(factor), float(trained_length),
                                     ctypes.cast(freq.data_ptr(), ctypes.POINTER(ctypes.c_float)),
                                     ctypes.byref(magnitude))
    _check(lib, "sparse_rope_frequencies", st)
    return freq, magnitude.value


def _rope(func, x, positions, freq, layout, magnitude, out, stream):
    xa = _heads_arg(x, "x")
    n, heads, dim = x.shape
    device = x.get_device()
    if not isinstance(positions, torch.Tensor) or positions.dtype != torch.int32 or positions.dim() != 2 or \
            positions.shape[0] != n or not positions.is_cuda or positions.get_device() != device or \
            (positions.shape[1] > 1 and positions.stride(1) != 1):
        raise ValueError("positions must be int32 [N, axes] on x's device, the axes contiguous")
    _device_tensor(freq, "freq")
    if freq.dtype != torch.float32 or freq.dim() != 1 or freq.get_device() != device:
        raise ValueError("freq must be float32 [num_freq] on x's device")
    if out is None:
        out = _empty((n, heads, dim), x.dtype, x.device, stream)
        ya = _HeadsArg(out.data_ptr(), heads * dim, dim)
    else:
        ya = _heads_arg(out, "out", x)
        if out.shape != x.shape:
            raise ValueError("out must have x's shape")
    _run(func, device, stream, xa, n, heads, dim, _DTYPE_CODES[x.dtype], positions.data_ptr(), positions.stride(0),
         positions.shape[1], freq.data_ptr(), freq.shape[0], layout, magnitude, ya)
    return out


def sparse_rope_forward(x: torch.Tensor, positions: torch.Tensor, freq: torch.Tensor, layout: int,
                        magnitude: float = 1.0, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Rotary positions of x [N, heads, head_dim] (any row and head strides): positions int32
    [N, axes] (voxel coordinates: coords[:, 1:]), freq float32 [num_freq] of each axis, layout
    SUBM_ROPE_INTERLEAVED or SUBM_ROPE_HALF.  out may be x (in place)."""
    return _rope("sparse_rope_forward", x, positions, freq, layout, magnitude, out, stream)


def sparse_rope_backward(dy: torch.Tensor, positions: torch.Tensor, freq: torch.Tensor, layout: int,
                         magnitude: float = 1.0, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gradient of sparse_rope_forward: the rotation the other way."""
    return _rope("sparse_rope_backward", dy, positions, freq, layout, magnitude, out, stream)


def _attention_args(q, k, v, q_offsets, k_offsets, scale):
    qa, ka, va = _heads_arg(q, "q"), _heads_arg(k, "k", q), _heads_arg(v, "v", q)
    if k.shape != v.shape or k.shape[2] != q.shape[2]:
        raise ValueError("q must be [Nq, heads, head_dim], k and v [Nk, kv_heads, head_dim]")
    _offsets_arg(q_offsets)
    if k_offsets is None:
        if k.shape[0] != q.shape[0]:
            raise ValueError("k_offsets is required when q and k have different rows")
        k_offsets = q_offsets
    elif k_offsets is not q_offsets:
        _offsets_arg(k_offsets)
        if k_offsets.shape != q_offsets.shape:
            raise ValueError("q_offsets and k_offsets must have the same items")
    device = q.get_device()
    if q_offsets.get_device() != device or k_offsets.get_device() != device:
        raise ValueError("offsets must be on q's device")
    if scale is None:
        scale = q.shape[2] ** -0.5
    return qa, ka, va, k_offsets, scale


def _attention_out(q, out, lse, stream):
    """(out, its argument, lse, its data_ptr), new ones where not given."""
    nq, heads, dim = q.shape
    if out is None:
        out = _empty((nq, heads, dim), q.dtype, q.device, stream)
        oa = _HeadsArg(out.data_ptr(), heads * dim, dim)
    else:
        oa = _heads_arg(out, "out", q)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    if lse is None:
        lse = _empty((nq, heads), torch.float32, q.device, stream)
        lse_ptr = lse.data_ptr()
    else:
        lse_ptr = _vector(lse, (nq, heads), torch.float32, q.device, "lse")
    return out, oa, lse, lse_ptr


def sparse_attention_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_offsets: torch.Tensor,
                             k_offsets: torch.Tensor | None = None, scale: float | None = None,
                             out: torch.Tensor | None = None, lse: torch.Tensor | None = None, stream=None):
    """Attention within items: (out [Nq, heads, head_dim], lse float32 [Nq, heads]).

    q [Nq, heads, head_dim], k and v [Nk, kv_heads, head_dim] with any row and head strides;
    q_offsets, k_offsets int64 [items + 1] on the device (k_offsets None: self attention); scale
    defaults to head_dim ** -0.5.  A query whose item has no keys gets out 0, lse -infinity."""
    qa, ka, va, k_offsets, scale = _attention_args(q, k, v, q_offsets, k_offsets, scale)
    nq, heads, dim = q.shape
    out, oa, lse, lse_ptr = _attention_out(q, out, lse, stream)
    _run("sparse_attention_forward", q.get_device(), stream, qa, ka, va, nq, k.shape[0], q_offsets.data_ptr(),
         k_offsets.data_ptr(), q_offsets.shape[0] - 1, heads, k.shape[1], dim, _DTYPE_CODES[q.dtype], scale, oa, lse_ptr)
    return out, lse


def _attention_grads(dout, q, k, out, lse, dq, dk, dv, stream):
    """(arguments of dout and out, lse's data_ptr, dq, dk, dv and their arguments), new gradients where not given."""
    dq = _empty(q.shape, q.dtype, q.device, stream) if dq is None else dq
    dk = _empty(k.shape, q.dtype, q.device, stream) if dk is None else dk
    dv = _empty(k.shape, q.dtype, q.device, stream) if dv is None else dv
    ga, oa = _heads_arg(dout, "dout", q), _heads_arg(out, "out", q)
    dqa, dka, dva = _heads_arg(dq, "dq", q), _heads_arg(dk, "dk", q), _heads_arg(dv, "dv", q)
    if not (dout.shape == out.shape == dq.shape == q.shape) or not (dk.shape == dv.shape == k.shape):
        raise ValueError("dout, out and dq must have q's shape, dk and dv k's")
    if lse is None:
        raise ValueError("lse is required")
    lse_ptr = _vector(lse, tuple(q.shape[:2]), torch.float32, q.device, "lse")
    return ga, oa, lse_ptr, dq, dk, dv, dqa, dka, dva


def sparse_attention_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                              out: torch.Tensor, lse: torch.Tensor, q_offsets: torch.Tensor,
                              k_offsets: torch.Tensor | None = None, scale: float | None = None,
                              dq: torch.Tensor | None = None, dk: torch.Tensor | None = None,
                              dv: torch.Tensor | None = None, stream=None):
    """(dq, dk, dv) of sparse_attention_forward from dout and the forward pass's out and lse.  dq,
    dk and dv may be given as views of a packed buffer."""
    qa, ka, va, k_offsets, scale = _attention_args(q, k, v, q_offsets, k_offsets, scale)
    nq, heads, dim = q.shape
    ga, oa, lse_ptr, dq, dk, dv, *da = _attention_grads(dout, q, k, out, lse, dq, dk, dv, stream)
    _run("sparse_attention_backward", q.get_device(), stream, ga, qa, ka, va, oa, lse_ptr, nq, k.shape[0],
         q_offsets.data_ptr(), k_offsets.data_ptr(), q_offsets.shape[0] - 1, heads, k.shape[1], dim, _DTYPE_CODES[q.dtype],
         scale, *da)
    return dq, dk, dv


def _window_args(left, right, sinks):
    """left, right (None: open) and sinks as the library takes them."""
    ends = []
    for end, what in ((left, "left"), (right, "right")):
        end = 2 ** 31 if end is None else operator.index(end)  # (whole numbers: 2.5 is refused)
        if end < 0:
            raise ValueError(f"{what} must not be negative (None leaves it open)")
        ends.append(min(end, 2 ** 31))
    sinks = operator.index(sinks)
    if not 0 <= sinks < 2 ** 31:
        raise ValueError("sinks must not be negative")
    return (*ends, sinks)


def sparse_window_attention_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_offsets: torch.Tensor,
                                    k_offsets: torch.Tensor | None = None, left: int | None = None,
                                    right: int | None = None, sinks: int = 0, k_lengths: torch.Tensor | None = None,
                                    scale: float | None = None, out: torch.Tensor | None = None,
                                    lse: torch.Tensor | None = None, stream=None):
    """sparse_attention_forward within a sliding window: (out, lse).  Query i of an item with nq queries and nk
    keys stands at p = i + nk - nq and sees key j if j <= p + right and (j >= p - left or j < sinks); None
    leaves that end open (right=0: causal).  k_lengths int64 [items]: how many of an item's key rows are
    there (a cache with room behind its tokens)."""
    qa, ka, va, k_offsets, scale = _attention_args(q, k, v, q_offsets, k_offsets, scale)
    left, right, sinks = _window_args(left, right, sinks)
    nq, heads, dim = q.shape
    items = q_offsets.shape[0] - 1
    lengths = None if k_lengths is None else _vector(k_lengths, (items,), torch.int64, q.device, "k_lengths")
    out, oa, lse, lse_ptr = _attention_out(q, out, lse, stream)
    _run("sparse_window_attention_forward", q.get_device(), stream, qa, ka, va, nq, k.shape[0], q_offsets.data_ptr(),
         k_offsets.data_ptr(), lengths, items, heads, k.shape[1], dim, _DTYPE_CODES[q.dtype], scale, left, right, sinks, oa,
         lse_ptr)
    return out, lse


def sparse_window_attention_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                                     out: torch.Tensor, lse: torch.Tensor, q_offsets: torch.Tensor,
                                     k_offsets: torch.Tensor | None = None, left: int | None = None,
                                     right: int | None = None, sinks: int = 0, scale: float | None = None,
                                     dq: torch.Tensor | None = None, dk: torch.Tensor | None = None,
                                     dv: torch.Tensor | None = None, stream=None):
    """(dq, dk, dv) of sparse_window_attention_forward (without k_lengths) from dout and the forward pass's out
    and lse.  dq, dk and dv may be given as views of a packed buffer."""
    qa, ka, va, k_offsets, scale = _attention_args(q, k, v, q_offsets, k_offsets, scale)
    left, right, sinks = _window_args(left, right, sinks)
    nq, heads, dim = q.shape
    ga, oa, lse_ptr, dq, dk, dv, *da = _attention_grads(dout, q, k, out, lse, dq, dk, dv, stream)
    _run("sparse_window_attention_backward", q.get_device(), stream, ga, qa, ka, va, oa, lse_ptr, nq, k.shape[0],
         q_offsets.data_ptr(), k_offsets.data_ptr(), q_offsets.shape[0] - 1, heads, k.shape[1], dim, _DTYPE_CODES[q.dtype],
         scale, left, right, sinks, *da)
    return dq, dk, dv
