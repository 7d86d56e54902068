"""ctypes binding of libgsr.so: argument checks and marshalling only.

Every step of binning, forward and backward runs in the library's CUDA
kernels.  PyTorch provides device memory and streams.  When libgsr.so is
missing, importing this module raises: there is no CPU path.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# GSR_LIBRARY selects another build of the same library (A/B of build flags).
LIB_PATH = os.environ.get("GSR_LIBRARY") or os.path.join(_PKG, "lib", "libgsr.so")

GSR_OK, GSR_ERR_INVALID_ARG, GSR_ERR_CUDA, GSR_ERR_OOM, GSR_ERR_TOO_MANY_PAIRS = range(5)
GSR_PAIRS_ON_DEVICE = 0xFFFFFFFF
OPTIONS = {"bwd_warp_skip": 1, "bwd_last_contrib": 2, "warp_cull": 3, "pdl": 4, "fail_next_alloc": 5,
           "deterministic": 6, "bwd_per_splat": 7, "split": 8, "split_forward": 9}


class GsrError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"gsr error {code}: {msg}")
        self.code = code


class _Bins(ctypes.Structure):
    _fields_ = [("keys", ctypes.c_void_p), ("sorted_idx", ctypes.c_void_p),
                ("tile_ranges", ctypes.c_void_p), ("tile_order", ctypes.c_void_p),
                ("num_pairs_dev", ctypes.c_void_p), ("num_pairs", ctypes.c_uint32),
                ("n", ctypes.c_int32), ("width", ctypes.c_int32), ("height", ctypes.c_int32),
                ("tiles_x", ctypes.c_int32), ("tiles_y", ctypes.c_int32)]


GAUSSIAN_FIELDS = 14   # mean xyz, log_scale xyz, quat wxyz, logit_opacity, rgb
CAMERA_FIELDS = 18     # W row-major (9), t (3), fx, fy, cx, cy, z_near, eps


class _Camera(ctypes.Structure):
    _fields_ = [("v", ctypes.c_float * CAMERA_FIELDS)]


# gsr_group_norm, gsr_heads, gsr_rotary, gsr_attention, gsr_layer_norm and gsr_recurrence, packed per call: an
# order of magnitude quicker than filling ctypes structures, which these calls of
# a few microseconds would notice.
MAX_AXES = 4
GROUP_NORM = struct.Struct("@4iqif")   # dtype, samples, channels, groups, positions, activation, eps
HEADS = struct.Struct("@P3q")          # data, batch, token and head strides
ROTARY = struct.Struct("@12iq")        # dtype, batch, tokens, heads, head_dim, interleaved, axes, sections[4],
                                       # positions_int, positions_batch_stride
ATTENTION = struct.Struct("@7if2P")    # dtype, batch, q_len, kv_len, q_heads, kv_heads, head_dim, scale,
                                       # kv_lengths, key_mask
LAYER_NORM = struct.Struct("@5if")     # dtype, batch, tokens, heads, channels, eps
RECURRENCE = struct.Struct("@5iP")     # dtype, batch, tokens, channels, reverse, lengths
RECURRENCE_BLOCK = 64                  # GSR_RECURRENCE_BLOCK


class _BinStats(ctypes.Structure):
    _fields_ = [("num_pairs", ctypes.c_uint32), ("emitting", ctypes.c_uint32),
                ("radix_passes", ctypes.c_int32), ("depth_pass_mask", ctypes.c_uint32),
                ("tile_pass_mask", ctypes.c_uint32), ("tile_digit_bits", ctypes.c_int32),
                ("tile_digits", ctypes.c_int32), ("capacity", ctypes.c_uint64)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(LIB_PATH)
    P, i32 = ctypes.c_void_p, ctypes.c_int32
    lib.gsr_create.argtypes = [ctypes.POINTER(P), ctypes.c_int]
    lib.gsr_create.restype = ctypes.c_int
    lib.gsr_destroy.argtypes = [P]
    lib.gsr_destroy.restype = None
    lib.gsr_last_error.argtypes = [P]
    lib.gsr_last_error.restype = ctypes.c_char_p
    lib.gsr_set_option.argtypes = [P, ctypes.c_int, ctypes.c_int]
    lib.gsr_set_option.restype = ctypes.c_int
    lib.gsr_launch_count.argtypes = [P]
    lib.gsr_launch_count.restype = ctypes.c_uint64
    lib.gsr_bin_splats.argtypes = [P, P, P, i32, i32, i32, P, ctypes.POINTER(_Bins)]
    lib.gsr_bin_splats.restype = ctypes.c_int
    lib.gsr_rasterize_forward.argtypes = [P, P, i32, ctypes.POINTER(_Bins), P, P, P, P]
    lib.gsr_rasterize_forward.restype = ctypes.c_int
    lib.gsr_rasterize_backward.argtypes = [P, P, i32, ctypes.POINTER(_Bins), P, P, P, P, P]
    lib.gsr_rasterize_backward.restype = ctypes.c_int
    lib.gsr_reserve_pairs.argtypes = [P, ctypes.c_uint64]
    lib.gsr_reserve_pairs.restype = ctypes.c_int
    lib.gsr_num_pairs.argtypes = [P, ctypes.POINTER(ctypes.c_uint32)]
    lib.gsr_num_pairs.restype = ctypes.c_int
    lib.gsr_get_bin_stats.argtypes = [P, ctypes.POINTER(_BinStats)]
    lib.gsr_get_bin_stats.restype = ctypes.c_int
    lib.gsr_project_forward.argtypes = [P, P, i32, ctypes.POINTER(_Camera), P, P, P]
    lib.gsr_project_forward.restype = ctypes.c_int
    lib.gsr_project_backward.argtypes = [P, P, i32, ctypes.POINTER(_Camera), P, P, P]
    lib.gsr_project_backward.restype = ctypes.c_int
    lib.gsr_synchronize.argtypes = [P, P]
    lib.gsr_synchronize.restype = ctypes.c_int
    lib.gsr_exp_neg.argtypes = [P, P, P, i32, P]
    lib.gsr_exp_neg.restype = ctypes.c_int
    lib.gsr_peak_kernel.argtypes = [P, ctypes.c_int, i32, P, ctypes.POINTER(ctypes.c_uint64), P]
    lib.gsr_peak_kernel.restype = ctypes.c_int
    for name, pointers in (("gsr_group_norm_forward", 9), ("gsr_group_norm_backward", 12), ("gsr_rotary_forward", 7),
                           ("gsr_rotary_backward", 7), ("gsr_cross_attention_forward", 8),
                           ("gsr_cross_attention_backward", 12), ("gsr_layer_norm_forward", 11),
                           ("gsr_layer_norm_backward", 12), ("gsr_gated_recurrence_forward", 10),
                           ("gsr_gated_recurrence_backward", 13)):
        getattr(lib, name).argtypes = [P] * pointers
        getattr(lib, name).restype = ctypes.c_int
    return lib


lib = _load()


class _DeviceArray:
    """Minimal __cuda_array_interface__ holder for a view of arena memory."""

    def __init__(self, ptr, shape, typestr):
        self.__cuda_array_interface__ = {"data": (int(ptr or 0), False), "shape": tuple(shape),
                                         "typestr": typestr, "version": 3, "strides": None}


class Context:
    """Owns a libgsr context (the grow-only binning arena) on one CUDA device."""

    def __init__(self, device: int = 0):
        h = ctypes.c_void_p()
        rc = lib.gsr_create(ctypes.byref(h), int(device))
        if rc != GSR_OK:
            raise GsrError(rc, "gsr_create failed")
        self._h = h
        self.device = int(device)
        # Bumped by every bin_splats: bins from an earlier call may point into
        # arena buffers that call freed or overwrote.
        self._bin_generation = 0

    def _check(self, rc):
        if rc != GSR_OK:
            raise GsrError(rc, lib.gsr_last_error(self._h).decode())

    def set_option(self, name: str, value: bool):
        """Sets a GSR_OPT_* switch by its name in OPTIONS (the header documents
        each): "split" (backward segments of crowded tiles, on by default),
        "split_forward" (the forward's chunks past a head, off by default),
        "deterministic", "bwd_per_splat", and the A/B switches."""
        self._check(lib.gsr_set_option(self._h, OPTIONS[name], int(bool(value))))

    def launch_count(self) -> int:
        return int(lib.gsr_launch_count(self._h))

    def reserve_pairs(self, max_pairs: int):
        """Sizes the arena for max_pairs tile pairs; later bin_splats calls
        read nothing back to the host (0: back to reading the count)."""
        self._check(lib.gsr_reserve_pairs(self._h, int(max_pairs)))

    def num_pairs(self) -> int:
        """The last binning's pair count (waits for it); GsrError with code
        GSR_ERR_TOO_MANY_PAIRS when it exceeded the reservation."""
        out = ctypes.c_uint32()
        self._check(lib.gsr_num_pairs(self._h, ctypes.byref(out)))
        return int(out.value)

    def bin_stats(self) -> dict:
        st = _BinStats()
        self._check(lib.gsr_get_bin_stats(self._h, ctypes.byref(st)))
        return {name: (int(getattr(st, name))) for name, _ in _BinStats._fields_}

    def synchronize(self, stream=None):
        """Waits for the work on `stream` (default: the current stream); GsrError if a
        kernel of the decoder's operators gave up waiting, so that what it and later
        calls wrote is not valid.  Call it where their results leave the GPU, and
        after a graph's replays."""
        self._check(lib.gsr_synchronize(self._h, _stream_ptr(stream, self.device)))

    def close(self):
        if getattr(self, "_h", None):
            lib.gsr_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Bins:
    """Result of bin_splats: device views into the context's arena (valid until
    the next bin_splats on the same context, which may free or overwrite the
    buffers; later use raises ValueError)."""

    def __init__(self, ctx: Context, raw: _Bins, device, generation: int):
        self.ctx, self.raw, self._device, self.generation = ctx, raw, device, generation

    def _check_current(self):
        if getattr(self.ctx, "_h", None) is None:
            raise ValueError("the context these bins belong to is closed")
        if self.generation != self.ctx._bin_generation:
            raise ValueError("these bins were replaced by a later bin_splats on the same context")

    @property
    def num_pairs(self) -> int:
        """The pair count; for bins whose count stayed on the device this waits
        for the binning and reads it."""
        if int(self.raw.num_pairs) == GSR_PAIRS_ON_DEVICE:
            self._check_current()
            return self.ctx.num_pairs()
        return int(self.raw.num_pairs)

    @property
    def tiles(self):
        return int(self.raw.tiles_x), int(self.raw.tiles_y)

    def _view(self, ptr, shape, typestr):
        self._check_current()
        if shape[0] == 0:
            return torch.empty(shape, dtype={"<i8": torch.int64, "<i4": torch.int32}[typestr],
                               device=self._device)
        return torch.as_tensor(_DeviceArray(ptr, shape, typestr), device=self._device)

    def keys(self) -> torch.Tensor:
        """Sorted keys as int64 (bit pattern of the uint64 keys)."""
        return self._view(self.raw.keys, (self.num_pairs,), "<i8")

    def sorted_idx(self) -> torch.Tensor:
        return self._view(self.raw.sorted_idx, (self.num_pairs,), "<i4")

    def tile_order(self) -> torch.Tensor:
        """Launch order of the tiles (longest lists first)."""
        tx, ty = self.tiles
        return self._view(self.raw.tile_order, (tx * ty,), "<i4")

    def tile_ranges(self) -> torch.Tensor:
        tx, ty = self.tiles
        return self._view(self.raw.tile_ranges, (tx * ty, 2), "<i4")


def exp_neg(ctx: Context, s: torch.Tensor, out=None, stream=None) -> torch.Tensor:
    """The raster kernels' exp(-s) on a device array (diagnostic)."""
    _need(s, "s", torch.float32)
    if out is None:
        out = torch.empty_like(s)
    _need(out, "out", torch.float32, tuple(s.shape))
    ctx._check(lib.gsr_exp_neg(ctx._h, ctypes.c_void_p(s.data_ptr()), ctypes.c_void_p(out.data_ptr()),
                               int(s.numel()), _stream_ptr(stream, s.device)))
    return out


PEAK_KINDS = {"ffma": 0, "ex2": 1}


def peak_kernel(ctx: Context, kind: str, iters: int, sink: torch.Tensor, stream=None) -> int:
    """Enqueues one launch of the FP32 ("ffma") or SFU ("ex2") rate kernel;
    returns the number of lane operations it performs (time it with events)."""
    _need(sink, "sink", torch.float32)
    ops = ctypes.c_uint64()
    ctx._check(lib.gsr_peak_kernel(ctx._h, PEAK_KINDS[kind], int(iters), ctypes.c_void_p(sink.data_ptr()),
                                   ctypes.byref(ops), _stream_ptr(stream, sink.device)))
    return int(ops.value)


def _stream_ptr(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t: torch.Tensor, name, dtype, shape=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def bin_splats(ctx: Context, splats: torch.Tensor, depths: torch.Tensor, width: int, height: int,
               stream=None) -> Bins:
    n = splats.shape[0] if splats.dim() == 2 else -1
    _need(splats, "splats", torch.float32, (n, 9))
    _need(depths, "depths", torch.float32, (n,))
    raw = _Bins()
    ctx._bin_generation += 1   # even a failed call may have regrown the arena
    ctx._check(lib.gsr_bin_splats(ctx._h, ctypes.c_void_p(splats.data_ptr()),
                                  ctypes.c_void_p(depths.data_ptr()), n, int(width), int(height),
                                  _stream_ptr(stream, splats.device), ctypes.byref(raw)))
    return Bins(ctx, raw, splats.device, ctx._bin_generation)


def rasterize_forward(ctx: Context, splats: torch.Tensor, bins: Bins, out_rgbw=None, final_T=None,
                      last_contrib=None, stream=None):
    """Returns (out_rgbw [H*W, 4] f32, final_T [H*W] f32, last_contrib [H*W] int32)."""
    bins._check_current()
    n = splats.shape[0]
    _need(splats, "splats", torch.float32, (n, 9))
    npx = int(bins.raw.width) * int(bins.raw.height)
    dev = splats.device
    if out_rgbw is None:
        out_rgbw = torch.empty((npx, 4), dtype=torch.float32, device=dev)
    if final_T is None:
        final_T = torch.empty((npx,), dtype=torch.float32, device=dev)
    if last_contrib is None:
        last_contrib = torch.empty((npx,), dtype=torch.int32, device=dev)
    _need(out_rgbw, "out_rgbw", torch.float32, (npx, 4))
    _need(final_T, "final_T", torch.float32, (npx,))
    _need(last_contrib, "last_contrib", torch.int32, (npx,))
    ctx._check(lib.gsr_rasterize_forward(
        ctx._h, ctypes.c_void_p(splats.data_ptr()), n, ctypes.byref(bins.raw),
        ctypes.c_void_p(out_rgbw.data_ptr()), ctypes.c_void_p(final_T.data_ptr()),
        ctypes.c_void_p(last_contrib.data_ptr()), _stream_ptr(stream, dev)))
    return out_rgbw, final_T, last_contrib


def rasterize_backward(ctx: Context, splats: torch.Tensor, bins: Bins, dl_dout: torch.Tensor,
                       final_T: torch.Tensor, last_contrib: torch.Tensor, grad=None, stream=None):
    """Returns grad [N, 9] f32 (d/d of each Splat2D field)."""
    bins._check_current()
    n = splats.shape[0]
    _need(splats, "splats", torch.float32, (n, 9))
    npx = int(bins.raw.width) * int(bins.raw.height)
    dev = splats.device
    if grad is None:
        grad = torch.empty((n, 9), dtype=torch.float32, device=dev)
    _need(dl_dout, "dl_dout", torch.float32, (npx, 4))
    _need(final_T, "final_T", torch.float32, (npx,))
    _need(last_contrib, "last_contrib", torch.int32, (npx,))
    _need(grad, "grad", torch.float32, (n, 9))
    ctx._check(lib.gsr_rasterize_backward(
        ctx._h, ctypes.c_void_p(splats.data_ptr()), n, ctypes.byref(bins.raw),
        ctypes.c_void_p(dl_dout.data_ptr()), ctypes.c_void_p(final_T.data_ptr()),
        ctypes.c_void_p(last_contrib.data_ptr()), ctypes.c_void_p(grad.data_ptr()),
        _stream_ptr(stream, dev)))
    return grad


def _camera(camera) -> _Camera:
    vals = [float(v) for v in (camera.tolist() if hasattr(camera, "tolist") else camera)]
    if len(vals) != CAMERA_FIELDS:
        raise ValueError(f"camera must hold {CAMERA_FIELDS} numbers (W row-major, t, fx, fy, cx, cy, "
                         "z_near, eps)")
    cam = _Camera()
    cam.v[:] = vals
    return cam


def project_forward(ctx: Context, gauss: torch.Tensor, camera, splats=None, depths=None, stream=None):
    """Projects 3-D Gaussians [n, 14] f32 through `camera` (18 numbers).
    Returns (splats [n, 9] f32, depths [n] f32)."""
    n = gauss.shape[0] if gauss.dim() == 2 else -1
    _need(gauss, "gauss", torch.float32, (n, GAUSSIAN_FIELDS))
    dev = gauss.device
    if splats is None:
        splats = torch.empty((n, 9), dtype=torch.float32, device=dev)
    if depths is None:
        depths = torch.empty((n,), dtype=torch.float32, device=dev)
    _need(splats, "splats", torch.float32, (n, 9))
    _need(depths, "depths", torch.float32, (n,))
    cam = _camera(camera)
    ctx._check(lib.gsr_project_forward(ctx._h, ctypes.c_void_p(gauss.data_ptr()), n, ctypes.byref(cam),
                                       ctypes.c_void_p(splats.data_ptr()), ctypes.c_void_p(depths.data_ptr()),
                                       _stream_ptr(stream, dev)))
    return splats, depths


def project_backward(ctx: Context, gauss: torch.Tensor, camera, dl_dsplat: torch.Tensor, dl_dgauss=None,
                     stream=None) -> torch.Tensor:
    """Returns dL/dgauss [n, 14] f32 for dL/dsplat [n, 9] f32."""
    n = gauss.shape[0] if gauss.dim() == 2 else -1
    _need(gauss, "gauss", torch.float32, (n, GAUSSIAN_FIELDS))
    _need(dl_dsplat, "dl_dsplat", torch.float32, (n, 9))
    dev = gauss.device
    if dl_dgauss is None:
        dl_dgauss = torch.empty((n, GAUSSIAN_FIELDS), dtype=torch.float32, device=dev)
    _need(dl_dgauss, "dl_dgauss", torch.float32, (n, GAUSSIAN_FIELDS))
    cam = _camera(camera)
    ctx._check(lib.gsr_project_backward(ctx._h, ctypes.c_void_p(gauss.data_ptr()), n, ctypes.byref(cam),
                                        ctypes.c_void_p(dl_dsplat.data_ptr()),
                                        ctypes.c_void_p(dl_dgauss.data_ptr()), _stream_ptr(stream, dev)))
    return dl_dgauss


# -- the operators of an image-to-Gaussians decoder ---------------------------
#
# The smallest of these calls are bound by the host, so the checks test the usual
# case in one condition and look for the reason only when it fails.

DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2}
_F32 = torch.float32
_HALVES = (torch.bfloat16, torch.float16)


def _first(t, name, among):
    """Checks the tensor that decides a call's dtype and device; returns the device's index."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in among:
        raise ValueError(f"{name} must be one of {', '.join(map(str, among))}, got {t.dtype}")
    return t.get_device()


def _on(ctx, t, name, among):
    """_first of a call on `ctx`, whose device the tensors have to be on: the kernels run there."""
    index = _first(t, name, among)
    if index != ctx.device:
        raise ValueError(f"{name} is on cuda:{index}, the context on cuda:{ctx.device}")
    return index


def _refuse(t, name, dtype, shape, index):
    if not isinstance(t, torch.Tensor) or t.get_device() != index:
        raise ValueError(f"{name} must be a CUDA tensor on cuda:{index}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _array(t, name, dtype, shape, index):
    """The address of a contiguous tensor."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == index):
        _refuse(t, name, dtype, shape, index)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _heads(t, name, dtype, shape, index):
    """A packed gsr_heads of a [batch, tokens, heads, head_dim] tensor, any strides
    but a contiguous last dimension."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == index):
        _refuse(t, name, dtype, shape, index)
    return _strides(t, name)


def _strides(t, name):
    batch, token, head, last = t.stride()
    if last != 1 and t.shape[3] > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return HEADS.pack(t.data_ptr(), batch, token, head)


def _heads_out(t, name, dtype, shape, index, device, stream, like=None):
    """An output [batch, tokens, heads, head_dim], made if None, and its packed gsr_heads."""
    if t is not None:
        return t, _heads(t, name, dtype, shape, index)
    t = _new(shape, dtype, device, stream, like)
    _, tokens, heads, dim = shape
    return t, HEADS.pack(t.data_ptr(), tokens * heads * dim, heads * dim, dim)


def _array_out(t, name, dtype, shape, index, device, stream, like=None):
    """A contiguous output, made if None, and its address."""
    if t is not None:
        return t, _array(t, name, dtype, shape, index)
    t = _new(shape, dtype, device, stream, like)
    return t, t.data_ptr()


def _new(shape, dtype, device, stream, like=None):
    """A contiguous output of this call, allocated for the stream that writes it;
    the caller's stream, which will read it, is recorded on it as well.  `like`: a
    tensor of the same shape and type (the quicker way, if it is contiguous)."""
    if stream is None:
        if like is not None and like.is_contiguous():
            return torch.empty_like(like)
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


# The current stream's handle without a Stream object around it, where torch has it.
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _raw_stream(stream, index):
    return _current_raw_stream(index) if stream is None else stream.cuda_stream


def _norm_desc(x, groups, eps, activation):
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, got {activation!r}")
    shape = x.shape
    if len(shape) < 2:
        raise ValueError(f"x must have shape [samples, ..., channels], got {tuple(shape)}")
    positions = 1
    for extent in shape[1:-1]:
        positions *= extent
    return GROUP_NORM.pack(DTYPES[x.dtype], shape[0], shape[-1], groups, positions, ACTIVATIONS[activation], eps)


def group_norm_forward(ctx: Context, x: torch.Tensor, groups: int, weight=None, bias=None, eps: float = 1e-5,
                       activation: str = "silu", out=None, mean=None, rstd=None, stream=None):
    """act(group norm(x) * weight + bias) over channels-last x [samples, ..., channels]
    (f32, bf16 or f16; weight and bias [channels] f32 or None).  `activation` is
    "none", "silu" or "gelu".  Returns (out, mean, rstd), the last two
    [samples, groups] f32 for the backward.  out may be x."""
    index = _on(ctx, x, "x", DTYPES)
    dtype, shape, dev = x.dtype, x.shape, x.device
    desc = _norm_desc(x, groups, eps, activation)
    channels, stats = shape[-1:], (shape[0], max(int(groups), 0))
    out, at_out = _array_out(out, "out", dtype, shape, index, dev, stream, x)
    mean, at_mean = _array_out(mean, "mean", _F32, stats, index, dev, stream)
    rstd, at_rstd = _array_out(rstd, "rstd", _F32, stats, index, dev, stream)
    ctx._check(lib.gsr_group_norm_forward(
        ctx._h, desc, _array(x, "x", dtype, shape, index),
        None if weight is None else _array(weight, "weight", _F32, channels, index),
        None if bias is None else _array(bias, "bias", _F32, channels, index), at_out, at_mean, at_rstd,
        _raw_stream(stream, index)))
    return out, mean, rstd


def group_norm_backward(ctx: Context, dl_dout: torch.Tensor, x: torch.Tensor, groups: int, weight, bias,
                        mean: torch.Tensor, rstd: torch.Tensor, activation: str = "silu", dl_dx=None,
                        dl_dweight=None, dl_dbias=None, stream=None):
    """Returns (dL/dx as x, dL/dweight [channels] f32, dL/dbias [channels] f32) for
    dL/dout, with the forward's x, weight, bias, mean and rstd.  dl_dx may be dl_dout."""
    index = _on(ctx, x, "x", DTYPES)
    dtype, shape, dev = x.dtype, x.shape, x.device
    desc = _norm_desc(x, groups, 1.0, activation)
    channels, stats = shape[-1:], (shape[0], int(groups))
    dl_dx, at_dx = _array_out(dl_dx, "dl_dx", dtype, shape, index, dev, stream, x)
    dl_dweight, at_dweight = _array_out(dl_dweight, "dl_dweight", _F32, channels, index, dev, stream)
    dl_dbias, at_dbias = _array_out(dl_dbias, "dl_dbias", _F32, channels, index, dev, stream)
    ctx._check(lib.gsr_group_norm_backward(
        ctx._h, desc, _array(dl_dout, "dl_dout", dtype, shape, index), _array(x, "x", dtype, shape, index),
        None if weight is None else _array(weight, "weight", _F32, channels, index),
        None if bias is None else _array(bias, "bias", _F32, channels, index),
        _array(mean, "mean", _F32, stats, index), _array(rstd, "rstd", _F32, stats, index), at_dx, at_dweight,
        at_dbias, _raw_stream(stream, index)))
    return dl_dx, dl_dweight, dl_dbias


def rotary_frequencies(sections, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """The usual frequencies of rotary_forward, one progression per axis: pair j of
    a section of s pairs turns by base^(-j / s) per unit of its axis' position."""
    parts = [base ** (-torch.arange(int(s), dtype=torch.float64) / max(int(s), 1)) for s in sections]
    return torch.cat(parts).float().to(device)


def _rotary(call, name, ctx, x, positions, frequencies, sections, interleaved, out, out_name, stream):
    index = _on(ctx, x, name, DTYPES)
    dtype, shape = x.dtype, x.shape
    if len(shape) != 4:
        raise ValueError(f"{name} must have shape [batch, tokens, heads, head_dim], got {tuple(shape)}")
    batch, tokens, heads, dim = shape
    axes = len(sections)
    if not 1 <= axes <= MAX_AXES:
        raise ValueError(f"sections must hold 1 to {MAX_AXES} numbers of pairs, got {axes}")
    at_frequencies = _array(frequencies, "frequencies", _F32, (sum(sections),), index)
    _first(positions, "positions", (torch.int32, torch.float32))
    each = len(positions.shape) == 3
    if positions.shape != ((batch, tokens, axes) if each else (tokens, axes)):
        raise ValueError(f"positions must have shape {(tokens, axes)} or {(batch, tokens, axes)}, "
                         f"got {tuple(positions.shape)}")
    at_positions = _array(positions, "positions", positions.dtype, positions.shape, index)
    out, at_out = _heads_out(out, out_name, dtype, shape, index, x.device, stream, x)
    desc = ROTARY.pack(DTYPES[dtype], batch, tokens, heads, dim, bool(interleaved), axes, *sections,
                       *(0,) * (MAX_AXES - axes), positions.dtype is torch.int32, tokens * axes if each else 0)
    ctx._check(call(ctx._h, desc, _strides(x, name), at_positions, at_frequencies, at_out,
                    _raw_stream(stream, index)))
    return out


def rotary_forward(ctx: Context, x: torch.Tensor, positions: torch.Tensor, frequencies: torch.Tensor, sections,
                   interleaved: bool = False, out=None, stream=None) -> torch.Tensor:
    """Turns the pairs of x [batch, tokens, heads, head_dim] (f32, bf16 or f16; any
    strides with a contiguous last dimension) by positions [tokens, axes] or
    [batch, tokens, axes] (f32 or int32) times frequencies [sum(sections)] f32;
    sections[a] pairs turn by axis a.  Pairs are dimensions (i, i + sum(sections)),
    or (2i, 2i + 1) when interleaved.  out may be x."""
    return _rotary(lib.gsr_rotary_forward, "x", ctx, x, positions, frequencies, sections, interleaved, out, "out",
                   stream)


def rotary_backward(ctx: Context, dl_dout: torch.Tensor, positions: torch.Tensor, frequencies: torch.Tensor,
                    sections, interleaved: bool = False, dl_dx=None, stream=None) -> torch.Tensor:
    """dL/dx of rotary_forward for dL/dout.  dl_dx may be dl_dout."""
    return _rotary(lib.gsr_rotary_backward, "dl_dout", ctx, dl_dout, positions, frequencies, sections, interleaved,
                   dl_dx, "dl_dx", stream)


def _attention(ctx, q, k, v, kv_lengths, key_mask, scale):
    """The packed description and q, k, v; the device's index and k's shape."""
    index = _on(ctx, q, "q", _HALVES)
    dtype, shape = q.dtype, q.shape
    if len(shape) != 4 or not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("q, k and v must have shape [batch, tokens, heads, head_dim]")
    batch, q_len, q_heads, dim = shape
    kv_len, kv_heads = k.shape[1:3]
    keys = (batch, kv_len, kv_heads, dim)
    at_lengths = at_mask = 0
    if kv_lengths is not None:
        at_lengths = _array(kv_lengths, "kv_lengths", torch.int32, (batch,), index)
    if key_mask is not None:
        _first(key_mask, "key_mask", (torch.bool, torch.uint8))
        at_mask = _array(key_mask, "key_mask", key_mask.dtype, (batch, kv_len), index)
    desc = ATTENTION.pack(DTYPES[dtype], batch, q_len, kv_len, q_heads, kv_heads, dim,
                          dim ** -0.5 if scale is None else scale, at_lengths, at_mask)
    return index, keys, desc, _strides(q, "q"), _heads(k, "k", dtype, keys, index), \
        _heads(v, "v", dtype, keys, index)


def cross_attention_forward(ctx: Context, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, kv_lengths=None,
                            key_mask=None, scale=None, out=None, lse=None, stream=None):
    """Attention of q [batch, q_len, q_heads, head_dim] to k, v [batch, kv_len,
    kv_heads, head_dim] (bf16 or f16; views with a contiguous last dimension).
    Keys at or behind kv_lengths [batch] int32, or whose key_mask [batch, kv_len]
    (bool or uint8) is 0, take no part; a row without any gives 0 and lse -inf.
    `scale` defaults to head_dim ** -0.5.  Returns (out as q, lse [batch, q_heads,
    q_len] f32)."""
    index, _, desc, at_q, at_k, at_v = _attention(ctx, q, k, v, kv_lengths, key_mask, scale)
    dtype, shape = q.dtype, q.shape
    rows = (shape[0], shape[2], shape[1])
    out, at_out = _heads_out(out, "out", dtype, shape, index, q.device, stream, q)
    lse, at_lse = _array_out(lse, "lse", _F32, rows, index, q.device, stream)
    ctx._check(lib.gsr_cross_attention_forward(ctx._h, desc, at_q, at_k, at_v, at_out, at_lse,
                                               _raw_stream(stream, index)))
    return out, lse


def cross_attention_backward(ctx: Context, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                             lse: torch.Tensor, dl_dout: torch.Tensor, kv_lengths=None, key_mask=None, scale=None,
                             dl_dq=None, dl_dk=None, dl_dv=None, stream=None):
    """Returns (dL/dq, dL/dk, dL/dv) for dL/dout, with the forward's arguments, out
    and lse.  Keys that took no part get zeros."""
    index, keys, desc, at_q, at_k, at_v = _attention(ctx, q, k, v, kv_lengths, key_mask, scale)
    dtype, shape, dev = q.dtype, q.shape, q.device
    dl_dq, at_dq = _heads_out(dl_dq, "dl_dq", dtype, shape, index, dev, stream, q)
    dl_dk, at_dk = _heads_out(dl_dk, "dl_dk", dtype, keys, index, dev, stream, k)
    dl_dv, at_dv = _heads_out(dl_dv, "dl_dv", dtype, keys, index, dev, stream, v)
    ctx._check(lib.gsr_cross_attention_backward(
        ctx._h, desc, at_q, at_k, at_v, _heads(out, "out", dtype, shape, index),
        _array(lse, "lse", _F32, (shape[0], shape[2], shape[1]), index),
        _heads(dl_dout, "dl_dout", dtype, shape, index), at_dq, at_dk, at_dv, _raw_stream(stream, index)))
    return dl_dq, dl_dk, dl_dv


def _rows(t, name, dtype, shape, index):
    """A packed gsr_heads of a tensor [..., channels] with one to three leading
    dimensions, any strides but a contiguous last dimension."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == index):
        _refuse(t, name, dtype, shape, index)
    strides = t.stride()
    if strides[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    n = len(strides)
    return HEADS.pack(t.data_ptr(), strides[0] if n > 2 else 0, strides[1] if n > 2 else strides[0],
                      strides[2] if n > 3 else 0)


def _rows_out(t, name, dtype, shape, index, device, stream, like=None):
    """An output [..., channels], made if None, and its packed gsr_heads."""
    if t is None:
        t = _new(shape, dtype, device, stream, like)
    return t, _rows(t, name, dtype, shape, index)


def _layer_desc(x, eps):
    shape = x.shape
    n = len(shape)
    if not 2 <= n <= 4:
        raise ValueError("x must have shape [tokens, channels], [batch, tokens, channels] or [batch, tokens, heads, "
                         f"channels], got {tuple(shape)}")
    return LAYER_NORM.pack(DTYPES[x.dtype], shape[0] if n > 2 else 1, shape[1] if n > 2 else shape[0],
                           shape[2] if n > 3 else 1, shape[-1], eps)


def layer_norm_forward(ctx: Context, x: torch.Tensor, weight=None, bias=None, residual=None, eps: float = 1e-5,
                       out=None, total=None, mean=None, rstd=None, stream=None):
    """Layer norm over the channels of x [tokens, channels], [batch, tokens, channels]
    or [batch, tokens, heads, channels] (f32, bf16 or f16; any strides with a
    contiguous last dimension; weight and bias [channels] f32 or None), or of
    total = x + residual.  Returns (out, total, mean, rstd), total being x without a
    residual and the last two [...] f32, for the backward.  out and total may be x or
    residual, but not each other."""
    index = _on(ctx, x, "x", DTYPES)
    dtype, shape, dev = x.dtype, x.shape, x.device
    desc = _layer_desc(x, eps)
    channels, stats = shape[-1:], shape[:-1]
    at_x = _rows(x, "x", dtype, shape, index)
    out, at_out = _rows_out(out, "out", dtype, shape, index, dev, stream, x)
    at_residual = at_total = None
    if residual is not None:
        at_residual = _rows(residual, "residual", dtype, shape, index)
        total, at_total = _rows_out(total, "total", dtype, shape, index, dev, stream, x)
    elif total is not None:
        raise ValueError("total is x itself without a residual")
    else:
        total = x
    mean, at_mean = _array_out(mean, "mean", _F32, stats, index, dev, stream)
    rstd, at_rstd = _array_out(rstd, "rstd", _F32, stats, index, dev, stream)
    ctx._check(lib.gsr_layer_norm_forward(
        ctx._h, desc, at_x, at_residual, None if weight is None else _array(weight, "weight", _F32, channels, index),
        None if bias is None else _array(bias, "bias", _F32, channels, index), at_out, at_total, at_mean, at_rstd,
        _raw_stream(stream, index)))
    return out, total, mean, rstd


def layer_norm_backward(ctx: Context, dl_dout: torch.Tensor, total: torch.Tensor, weight, mean: torch.Tensor,
                        rstd: torch.Tensor, dl_dtotal=None, dl_dx=None, dl_dweight=None, dl_dbias=None, stream=None):
    """Returns (dL/dx as total, dL/dweight [channels] f32, dL/dbias [channels] f32) for
    dL/dout and, where total goes on past the norm, dL/dtotal; with the forward's
    total, weight, mean and rstd.  dL/dx is the residual's gradient too.  dl_dx may be
    dl_dout or dl_dtotal."""
    index = _on(ctx, total, "total", DTYPES)
    dtype, shape, dev = total.dtype, total.shape, total.device
    desc = _layer_desc(total, 1.0)
    channels, stats = shape[-1:], shape[:-1]
    dl_dx, at_dx = _rows_out(dl_dx, "dl_dx", dtype, shape, index, dev, stream, total)
    dl_dweight, at_dweight = _array_out(dl_dweight, "dl_dweight", _F32, channels, index, dev, stream)
    dl_dbias, at_dbias = _array_out(dl_dbias, "dl_dbias", _F32, channels, index, dev, stream)
    ctx._check(lib.gsr_layer_norm_backward(
        ctx._h, desc, _rows(dl_dout, "dl_dout", dtype, shape, index), _rows(total, "total", dtype, shape, index),
        None if weight is None else _array(weight, "weight", _F32, channels, index),
        _array(mean, "mean", _F32, stats, index), _array(rstd, "rstd", _F32, stats, index),
        None if dl_dtotal is None else _rows(dl_dtotal, "dl_dtotal", dtype, shape, index), at_dx, at_dweight, at_dbias,
        _raw_stream(stream, index)))
    return dl_dx, dl_dweight, dl_dbias


def _recurrence(ctx, x, forget, gate, lengths, reverse):
    """The packed description and x, forget and gate; the device's index."""
    index = _on(ctx, x, "x", DTYPES)
    dtype, shape = x.dtype, x.shape
    if len(shape) != 3:
        raise ValueError(f"x must have shape [batch, tokens, channels], got {tuple(shape)}")
    batch, tokens, channels = shape
    at_lengths = 0 if lengths is None else _array(lengths, "lengths", torch.int32, (batch,), index)
    desc = RECURRENCE.pack(DTYPES[dtype], batch, tokens, channels, bool(reverse), at_lengths)
    return index, desc, _rows(x, "x", dtype, shape, index), _rows(forget, "forget", dtype, shape, index), \
        None if gate is None else _rows(gate, "gate", dtype, shape, index)


def gated_recurrence_forward(ctx: Context, x: torch.Tensor, forget: torch.Tensor, gate=None, initial=None,
                             lengths=None, reverse: bool = False, keep: bool = True, out=None, final=None, states=None,
                             stream=None):
    """h_t = a_t h_(t-1) + (1 - a_t) x_t with a = sigmoid(forget) over the tokens of
    x, forget [batch, tokens, channels] (f32, bf16 or f16; views with a contiguous
    last dimension), and out = h silu(gate), or h without a gate.  `reverse` runs from
    the last token to the first; item b has lengths[b] tokens (int32, all if None),
    and out is 0 behind them.  h starts at initial [batch, channels] f32 (0 if None).
    Returns (out, final [batch, channels] f32, states): the last h, to go on from,
    and what the backward needs (None with keep=False).  out may be x, final may be
    initial."""
    index, desc, at_x, at_forget, at_gate = _recurrence(ctx, x, forget, gate, lengths, reverse)
    dtype, shape, dev = x.dtype, x.shape, x.device
    batch, tokens, channels = shape
    state = (batch, channels)
    out, at_out = _rows_out(out, "out", dtype, shape, index, dev, stream)
    final, at_final = _array_out(final, "final", _F32, state, index, dev, stream)
    at_states = None
    if keep:
        blocks = (batch, -(-tokens // RECURRENCE_BLOCK), channels)
        states, at_states = _array_out(states, "states", _F32, blocks, index, dev, stream)
    elif states is not None:
        raise ValueError("states are written with keep=True only")
    ctx._check(lib.gsr_gated_recurrence_forward(
        ctx._h, desc, at_x, at_forget, at_gate, None if initial is None else _array(initial, "initial", _F32, state, index),
        at_out, at_final, at_states, _raw_stream(stream, index)))
    return out, final, states


def gated_recurrence_backward(ctx: Context, dl_dout: torch.Tensor, x: torch.Tensor, forget: torch.Tensor, gate,
                              states: torch.Tensor, dl_dfinal=None, lengths=None, reverse: bool = False, dl_dx=None,
                              dl_dforget=None, dl_dgate=None, dl_dinitial=None, stream=None):
    """Returns (dL/dx, dL/dforget, dL/dgate, dL/dinitial [batch, channels] f32) for
    dL/dout and, where the last state went on, dL/dfinal; with the forward's arguments
    and states.  dL/dgate is None without a gate.  dl_dx may be dl_dout."""
    index, desc, at_x, at_forget, at_gate = _recurrence(ctx, x, forget, gate, lengths, reverse)
    dtype, shape, dev = x.dtype, x.shape, x.device
    batch, tokens, channels = shape
    state = (batch, channels)
    dl_dx, at_dx = _rows_out(dl_dx, "dl_dx", dtype, shape, index, dev, stream)
    dl_dforget, at_dforget = _rows_out(dl_dforget, "dl_dforget", dtype, shape, index, dev, stream)
    at_dgate = None
    if gate is not None:
        dl_dgate, at_dgate = _rows_out(dl_dgate, "dl_dgate", dtype, shape, index, dev, stream)
    elif dl_dgate is not None:
        raise ValueError("dl_dgate has no gate")
    dl_dinitial, at_dinitial = _array_out(dl_dinitial, "dl_dinitial", _F32, state, index, dev, stream)
    ctx._check(lib.gsr_gated_recurrence_backward(
        ctx._h, desc, _rows(dl_dout, "dl_dout", dtype, shape, index), at_x, at_forget, at_gate,
        _array(states, "states", _F32, (batch, -(-tokens // RECURRENCE_BLOCK), channels), index),
        None if dl_dfinal is None else _array(dl_dfinal, "dl_dfinal", _F32, state, index), at_dx, at_dforget, at_dgate,
        at_dinitial, _raw_stream(stream, index)))
    return dl_dx, dl_dforget, dl_dgate, dl_dinitial
