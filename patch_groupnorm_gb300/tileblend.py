"""Python binding of libtileblend (include/tileblend.h).

Argument marshalling only: every step of the stitch, of PatchGroupNorm (channels
first and last) and of the training calls (layer norm, gradient clipping,
PatchGroupNorm's backward pass, dropout) runs in the library's CUDA kernels.  Tensors must be CUDA tensors on the
current device, contiguous (the layer norm and dropout take strided rows), of one dtype
(float32, float16 or bfloat16).
Calls are asynchronous on the current torch stream unless ``stream`` (a
``torch.cuda.Stream`` or a raw ``cudaStream_t`` integer) is given.

There is no fallback: if the compiled library is missing, importing this
module raises.
"""
import ctypes
import functools
import os
from array import array
from dataclasses import dataclass
from typing import List, Optional, Sequence, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# TILEBLEND_LIB selects another build of the same library (a variant built by
# build.build(variant=...), e.g. with in-kernel bounds checks).
LIB_PATH = os.environ.get("TILEBLEND_LIB") or os.path.join(_HERE, "_build", "libtileblend.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        "libtileblend.so is not built (expected at %s); run "
        "`python -c 'import __graft_entry__ as g; g.build()'` or "
        "`python patch_groupnorm_gb300/build.py`" % LIB_PATH)

_lib = ctypes.CDLL(LIB_PATH)

# ---------------------------------------------------------------------------
# C declarations
# ---------------------------------------------------------------------------

TB_OK, TB_ERR_NULL, TB_ERR_DTYPE, TB_ERR_SHAPE, TB_ERR_GEOMETRY, TB_ERR_UNSUPPORTED, TB_ERR_CUDA = range(7)
TB_F32, TB_F16, TB_BF16 = 0, 1, 2
TB_MAX_TILES_PER_AXIS = 64
TB_MAX_TILES = 1024
TB_GN_PARTS = 8

_DTYPES = {torch.float32: TB_F32, torch.float16: TB_F16, torch.bfloat16: TB_BF16}


class tb_axis(ctypes.Structure):
    _fields_ = [("latent_extent", ctypes.c_int32), ("latent_tile", ctypes.c_int32), ("overlap", ctypes.c_double),
                ("scale", ctypes.c_int32), ("blend_extent", ctypes.c_int32), ("row_limit", ctypes.c_int32)]


class tb_ramp_axis(ctypes.Structure):
    _fields_ = [("n_tiles", ctypes.c_int32), ("tile_extent", ctypes.c_int32), ("out_extent", ctypes.c_int32),
                ("zero", ctypes.c_int32), ("ramp", ctypes.c_int32), ("origins", ctypes.POINTER(ctypes.c_int64))]


class tb_gn_partial(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("mean", ctypes.c_float), ("m2", ctypes.c_float)]


class tb_shard_layout(ctypes.Structure):
    _fields_ = [("row_begin", ctypes.c_int32), ("row_end", ctypes.c_int32), ("out_row_begin", ctypes.c_int64),
                ("out_rows", ctypes.c_int64), ("halo_rows", ctypes.c_int32), ("halo_elems", ctypes.c_int64),
                ("send_elems", ctypes.c_int64)]


_vp, _i32, _i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
_P_vp = ctypes.POINTER(ctypes.c_void_p)
_P_i32 = ctypes.POINTER(ctypes.c_int32)
_P_i64 = ctypes.POINTER(ctypes.c_int64)
_P_axis = ctypes.POINTER(tb_axis)

_lib.tb_version.restype = ctypes.c_size_t
_lib.tb_version.argtypes = []
_lib.tb_status_string.restype = ctypes.c_char_p
_lib.tb_status_string.argtypes = [ctypes.c_int]
_lib.tb_last_cuda_error.restype = ctypes.c_int
_lib.tb_last_cuda_error.argtypes = []
_lib.tb_axis_layout.restype = ctypes.c_int
_lib.tb_axis_layout.argtypes = [_P_axis, _i32, _P_i32, _P_i64, _P_i32, _P_i32, _P_i32, _P_i64]
_lib.tb_stitch2d.restype = ctypes.c_int
_lib.tb_stitch2d.argtypes = [_P_vp, ctypes.c_int, _i64, _i64, _P_axis, _P_axis, _vp, _i64, _i64, _vp]
_lib.tb_stitch3d.restype = ctypes.c_int
_lib.tb_stitch3d.argtypes = [_P_vp, ctypes.c_int, _i64, _i64, _P_axis, _P_axis, _P_axis, _vp, _i64, _i64, _i64, _vp]
_lib.tb_patch_gn_stats.restype = ctypes.c_int
_lib.tb_patch_gn_stats.argtypes = [_P_vp, _i32, ctypes.c_int, _i64, _i64, _P_i64, _i32, _vp, _vp]
_lib.tb_patch_gn_apply.restype = ctypes.c_int
_lib.tb_patch_gn_apply.argtypes = [_P_vp, _P_vp, _i32, ctypes.c_int, _i64, _i64, _P_i64, _i32, _vp, _vp, _vp,
                                   ctypes.c_float, _i32, _vp]

_lib.tb_patch_gn_apply_gathered.restype = ctypes.c_int
_lib.tb_patch_gn_apply_gathered.argtypes = [_P_vp, _P_vp, _i32, ctypes.c_int, _i64, _i64, _P_i64, _i32, _vp, _i32,
                                            _vp, _vp, ctypes.c_float, _i32, _vp]
_lib.tb_stitch_shard_layout.restype = ctypes.c_int
_lib.tb_stitch_shard_layout.argtypes = [_P_axis, _P_axis, _P_axis, _i64, _i64, _i32, _i32,
                                        ctypes.POINTER(tb_shard_layout)]
_lib.tb_stitch_halo_pack.restype = ctypes.c_int
_lib.tb_stitch_halo_pack.argtypes = [_P_vp, ctypes.c_int, _i64, _i64, _P_axis, _P_axis, _P_axis, _i32, _vp, _vp]
_lib.tb_stitch2d_shard.restype = ctypes.c_int
_lib.tb_stitch2d_shard.argtypes = [_P_vp, _vp, ctypes.c_int, _i64, _i64, _P_axis, _P_axis, _i32, _i32, _vp, _i64,
                                   _i64, _vp]
_lib.tb_stitch_shard_frames_layout.restype = ctypes.c_int
_lib.tb_stitch_shard_frames_layout.argtypes = [_P_axis, _P_axis, _P_axis, _i64, _i64, _i32, _i32,
                                               ctypes.POINTER(tb_shard_layout)]
_lib.tb_stitch_halo_pack_frames.restype = ctypes.c_int
_lib.tb_stitch_halo_pack_frames.argtypes = [_P_vp, ctypes.c_int, _i64, _i64, _P_axis, _P_axis, _P_axis, _i32, _vp,
                                            _vp]
_lib.tb_stitch3d_shard_frames.restype = ctypes.c_int
_lib.tb_stitch3d_shard_frames.argtypes = [_P_vp, _vp, ctypes.c_int, _i64, _i64, _P_axis, _P_axis, _P_axis, _i32,
                                          _i32, _vp, _i64, _i64, _i64, _vp]
_lib.tb_stitch3d_shard.restype = ctypes.c_int
_lib.tb_stitch3d_shard.argtypes = [_P_vp, _vp, ctypes.c_int, _i64, _i64, _P_axis, _P_axis, _P_axis, _i32, _i32, _vp,
                                   _i64, _i64, _i64, _vp]

_lib.tb_device_status.restype = ctypes.c_int
_lib.tb_device_status.argtypes = [ctypes.POINTER(ctypes.c_uint32), _i32]
TB_DEV_OK, TB_DEV_WAIT_TIMEOUT, TB_DEV_OUT_OF_BOUNDS = 0, 1, 2

_lib.tb_ramp_axis_spread.restype = ctypes.c_int
_lib.tb_ramp_axis_spread.argtypes = [_i32, _i32, _i32, _i32, _i32, _i32, _P_i64, ctypes.POINTER(tb_ramp_axis)]
_lib.tb_stitch2d_ramp.restype = ctypes.c_int
_lib.tb_stitch2d_ramp.argtypes = [_P_vp, ctypes.c_int, _i64, _i64, ctypes.POINTER(tb_ramp_axis),
                                  ctypes.POINTER(tb_ramp_axis), _vp, _vp]
_lib.tb_patch_group_norm_noalloc.restype = ctypes.c_int
_lib.tb_patch_group_norm_noalloc.argtypes = [_P_vp, _P_vp, _i32, ctypes.c_int, _i64, _i64, _P_i64, _i32, _vp, _vp,
                                             ctypes.c_float, _i32, _vp]
TB_NOALLOC_MAX_PARTIALS = 65536
_lib.tb_patchify_layout.restype = ctypes.c_int
_lib.tb_patchify_layout.argtypes = [_i64, _i32, _i32, _P_i64, _P_i64]
_lib.tb_patchify.restype = ctypes.c_int
_lib.tb_patchify.argtypes = [_vp, ctypes.c_int, _i32, _P_i64, _i32, _i32, _i32, _i64, _P_vp, _vp]
_lib.tb_gather_patches.restype = ctypes.c_int
_lib.tb_gather_patches.argtypes = [_P_vp, _i32, _P_i64, ctypes.c_int, _i32, _P_i64, _i32, _i64, _vp, _vp]
TB_MAX_PATCHES = 64


_lib.tb_layer_norm.restype = ctypes.c_int
_lib.tb_layer_norm.argtypes = [_vp, _i64, _vp, _i64, ctypes.c_int, _i64, _i64, _vp, _vp, ctypes.c_int, ctypes.c_float,
                               _vp, _i64, _vp, _i64, _vp, _vp, _vp]
_lib.tb_layer_norm_workspace.restype = _i64
_lib.tb_layer_norm_workspace.argtypes = [_i64, _i64]
_lib.tb_layer_norm_backward.restype = ctypes.c_int
_lib.tb_layer_norm_backward.argtypes = [_vp, _i64, _vp, _i64, ctypes.c_int, _i64, _i64, _vp, _vp, _vp, ctypes.c_int,
                                        _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _vp]
_lib.tb_grad_records.restype = _i64
_lib.tb_grad_records.argtypes = [_i32]
_lib.tb_grad_stats.restype = ctypes.c_int
_lib.tb_grad_stats.argtypes = [_P_vp, _P_i64, _P_i32, _i32, _vp, _vp]
_lib.tb_grad_norm.restype = ctypes.c_int
_lib.tb_grad_norm.argtypes = [_vp, _i64, _vp, _vp]
_lib.tb_grad_clip.restype = ctypes.c_int
_lib.tb_grad_clip.argtypes = [_P_vp, _P_vp, _P_i64, _P_i32, _i32, _vp, _i64, ctypes.c_float, _vp, _vp]
_lib.tb_patch_gn_grad_stats.restype = ctypes.c_int
_lib.tb_patch_gn_grad_stats.argtypes = [_P_vp, _P_vp, _i32, ctypes.c_int, _i64, _i64, _P_i64, _i32, _vp, _i32, _vp,
                                        _vp, ctypes.c_float, _i32, _vp, _vp]
_lib.tb_patch_gn_grad_apply.restype = ctypes.c_int
_lib.tb_patch_gn_grad_apply.argtypes = [_P_vp, _P_vp, _P_vp, _i32, ctypes.c_int, _i64, _i64, _P_i64, _i32, _vp, _vp,
                                        _i32, _vp, _vp, ctypes.c_float, _i32, _vp, _vp, _vp]
# the channels-last calls take the addresses of their tables (parts of one array)
_int, _f32 = ctypes.c_int, ctypes.c_float
for _name, _args in {
        "tb_patch_gn_stats_cl": [_vp, _i32, _int, _i64, _i64, _vp, _i32, _vp, _vp],
        "tb_patch_gn_apply_cl": [_vp, _vp, _i32, _int, _i64, _i64, _vp, _i32, _vp, _i32, _vp, _vp, _f32, _i32, _vp],
        "tb_patch_group_norm_cl": [_vp, _vp, _i32, _int, _i64, _i64, _vp, _i32, _vp, _vp, _vp, _f32, _i32, _vp],
        "tb_patch_gn_grad_stats_cl": [_vp, _vp, _i32, _int, _i64, _i64, _vp, _i32, _vp, _i32, _vp, _vp, _f32, _i32, _vp,
                                      _vp],
        "tb_patch_gn_grad_apply_cl": [_vp, _vp, _vp, _i32, _int, _i64, _i64, _vp, _i32, _vp, _vp, _i32, _vp, _vp, _f32,
                                      _i32, _vp, _vp, _vp, _i64, _vp],
        "tb_patch_group_norm_backward_cl": [_vp, _vp, _vp, _i32, _int, _i64, _i64, _vp, _i32, _vp, _vp, _vp, _vp, _f32,
                                            _i32, _vp, _vp, _vp, _i64, _vp]}.items():
    getattr(_lib, _name).restype = _int
    getattr(_lib, _name).argtypes = _args
_lib.tb_patch_gn_workspace_cl.restype = _i64
_lib.tb_patch_gn_workspace_cl.argtypes = [_i64, _i32]
_lib.tb_dropout.restype = ctypes.c_int
_lib.tb_dropout.argtypes = [_vp, _i64, _vp, _i64, ctypes.c_int, _i64, _i64, ctypes.c_double, ctypes.c_uint64,
                            ctypes.c_uint64, _vp, _vp, _i64, _vp]
TB_GN_CL_MAX_CHANNELS = 8192
TB_LN_PARTS = 512
TB_MAX_GRADS, TB_GRAD_TABLE, TB_GRAD_PARTS = 65536, 1024, 1024

EXPORTED = ("tb_version", "tb_status_string", "tb_last_cuda_error", "tb_axis_layout", "tb_stitch2d",
            "tb_stitch3d", "tb_stitch_shard_layout", "tb_stitch_halo_pack", "tb_stitch2d_shard",
            "tb_stitch3d_shard", "tb_stitch2d_ramp", "tb_patch_gn_stats", "tb_patch_gn_apply",
            "tb_patch_gn_apply_gathered", "tb_patch_group_norm_noalloc", "tb_patchify_layout", "tb_patchify",
            "tb_gather_patches", "tb_device_status", "tb_ramp_axis_spread", "tb_stitch_shard_frames_layout",
            "tb_stitch_halo_pack_frames", "tb_stitch3d_shard_frames", "tb_layer_norm", "tb_layer_norm_workspace",
            "tb_layer_norm_backward", "tb_grad_records", "tb_grad_stats", "tb_grad_norm", "tb_grad_clip",
            "tb_patch_gn_grad_stats", "tb_patch_gn_grad_apply", "tb_patch_gn_stats_cl", "tb_patch_gn_apply_cl",
            "tb_patch_group_norm_cl", "tb_patch_gn_workspace_cl", "tb_patch_gn_grad_stats_cl",
            "tb_patch_gn_grad_apply_cl", "tb_patch_group_norm_backward_cl", "tb_dropout")


class TileBlendError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = "%s: %s" % (where, _lib.tb_status_string(status).decode())
        if status == TB_ERR_CUDA:
            msg += " (cudaError %d)" % _lib.tb_last_cuda_error()
        super().__init__(msg)
        self.status = status


def _check(status: int, where: str) -> None:
    if status != TB_OK:
        raise TileBlendError(status, where)


def tb_version() -> int:
    return int(_lib.tb_version())


def tb_device_status(clear: bool = False) -> int:
    """The device status word (0 = no kernel reported a problem); synchronises."""
    v = ctypes.c_uint32(0)
    _check(_lib.tb_device_status(ctypes.byref(v), 1 if clear else 0), "tb_device_status")
    return int(v.value)


# ---------------------------------------------------------------------------
# geometry
# ---------------------------------------------------------------------------

@dataclass(frozen=True)
class Axis:
    """Tile-grid parameters of one axis (see tb_axis in tileblend.h)."""
    latent_extent: int
    latent_tile: int
    overlap: float
    scale: int
    blend_extent: int = -1   # < 0: stock value
    row_limit: int = 0       # <= 0: stock value

    def c(self) -> tb_axis:
        return tb_axis(self.latent_extent, self.latent_tile, float(self.overlap), self.scale,
                       self.blend_extent, self.row_limit)


@dataclass(frozen=True)
class Layout:
    n: int
    origins: List[int]     # in decoded samples
    extents: List[int]
    blends: List[int]
    kept: List[int]
    out_extent: int


@functools.lru_cache(maxsize=256)
def tb_axis_layout(axis: Axis) -> Layout:
    """The library's derived geometry of one axis (host only; cached per
    parameter set)."""
    a = axis.c()
    n = ctypes.c_int32(0)
    cap = TB_MAX_TILES_PER_AXIS
    org = (ctypes.c_int64 * cap)()
    ext, bl, kp = (ctypes.c_int32 * cap)(), (ctypes.c_int32 * cap)(), (ctypes.c_int32 * cap)()
    out = ctypes.c_int64(0)
    _check(_lib.tb_axis_layout(ctypes.byref(a), cap, ctypes.byref(n), org, ext, bl, kp, ctypes.byref(out)),
           "tb_axis_layout")
    k = n.value
    return Layout(k, list(org[:k]), list(ext[:k]), list(bl[:k]), list(kp[:k]), out.value)


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------

def _stream_handle(stream) -> Optional[int]:
    if stream is None:
        # the current stream's handle without making a Stream object (2.9 us)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype not in _DTYPES:
        raise TypeError("unsupported dtype %s" % t.dtype)
    return _DTYPES[t.dtype]


def _cuda_contig(t: torch.Tensor, what: str) -> None:
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % what)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % what)


def _ptr_array(ptrs: Sequence[int]):
    return (ctypes.c_void_p * max(1, len(ptrs)))(*ptrs)


# ---------------------------------------------------------------------------
# stitch
# ---------------------------------------------------------------------------

def tb_stitch2d(tiles: Sequence[Sequence[torch.Tensor]], ay: Axis, ax: Axis, out: torch.Tensor, stream=None) -> torch.Tensor:
    """Stitch ``tiles[i][j]`` ([B, C, L_y(i), L_x(j)]) into ``out`` ([B, C, H, W])."""
    _cuda_contig(out, "out")
    B, C, H, W = out.shape
    ly, lx = tb_axis_layout(ay), tb_axis_layout(ax)
    ptrs = []
    if len(tiles) != ly.n:
        raise ValueError("expected %d tile rows, got %d" % (ly.n, len(tiles)))
    dt = out.dtype
    for i, row in enumerate(tiles):
        if len(row) != lx.n:
            raise ValueError("expected %d tiles in row %d, got %d" % (lx.n, i, len(row)))
        Ly = ly.extents[i]
        for j, t in enumerate(row):
            if t.dtype != dt or t.shape != (B, C, Ly, lx.extents[j]) or not t.is_cuda or not t.is_contiguous():
                _cuda_contig(t, "tile (%d,%d)" % (i, j))
                raise ValueError("tile (%d,%d) has %s %s, expected %s %s" % (
                    i, j, t.dtype, tuple(t.shape), dt, (B, C, Ly, lx.extents[j])))
            ptrs.append(t.data_ptr())
    a_y, a_x = ay.c(), ax.c()
    _check(_lib.tb_stitch2d(_ptr_array(ptrs), _dtype_code(out), B, C, ctypes.byref(a_y), ctypes.byref(a_x),
                            out.data_ptr(), H, W, _stream_handle(stream)), "tb_stitch2d")
    return out


def tb_stitch3d(tiles, at: Axis, ay: Axis, ax: Axis, out: torch.Tensor, stream=None) -> torch.Tensor:
    """Stitch ``tiles[k][i][j]`` ([B, C, L_t(k), L_y(i), L_x(j)]) into ``out``
    ([B, C, T, H, W])."""
    _cuda_contig(out, "out")
    B, C, T, H, W = out.shape
    lt, ly, lx = tb_axis_layout(at), tb_axis_layout(ay), tb_axis_layout(ax)
    ptrs = []
    if len(tiles) != lt.n:
        raise ValueError("expected %d frame tiles, got %d" % (lt.n, len(tiles)))
    for k, plane in enumerate(tiles):
        if len(plane) != ly.n:
            raise ValueError("expected %d tile rows" % ly.n)
        for i, row in enumerate(plane):
            if len(row) != lx.n:
                raise ValueError("expected %d tiles per row" % lx.n)
            for j, t in enumerate(row):
                _cuda_contig(t, "tile (%d,%d,%d)" % (k, i, j))
                exp = (B, C, lt.extents[k], ly.extents[i], lx.extents[j])
                if t.dtype != out.dtype or tuple(t.shape) != exp:
                    raise ValueError("tile (%d,%d,%d) has %s %s, expected %s %s" % (
                        k, i, j, t.dtype, tuple(t.shape), out.dtype, exp))
                ptrs.append(t.data_ptr())
    a_t, a_y, a_x = at.c(), ay.c(), ax.c()
    _check(_lib.tb_stitch3d(_ptr_array(ptrs), _dtype_code(out), B, C, ctypes.byref(a_t), ctypes.byref(a_y),
                            ctypes.byref(a_x), out.data_ptr(), T, H, W, _stream_handle(stream)), "tb_stitch3d")
    return out


def tb_stitch2d_raw(tile_ptrs: Sequence[int], dtype: int, B: int, C: int, ay: Axis, ax: Axis, out_ptr: int,
                    H: int, W: int, stream=None) -> None:
    """Pointer-level call (no tensor checks), for timing the bare C ABI."""
    a_y, a_x = ay.c(), ax.c()
    _check(_lib.tb_stitch2d(_ptr_array(tile_ptrs), dtype, B, C, ctypes.byref(a_y), ctypes.byref(a_x), out_ptr,
                            H, W, _stream_handle(stream)), "tb_stitch2d")


# ---------------------------------------------------------------------------
# row-sharded stitch
# ---------------------------------------------------------------------------

@dataclass(frozen=True)
class ShardLayout:
    row_begin: int
    row_end: int
    out_row_begin: int
    out_rows: int
    halo_rows: int
    halo_elems: int
    send_elems: int


def _axis_ref(a: Optional[Axis]):
    if a is None:
        return None, None
    c = a.c()
    return c, ctypes.byref(c)


def tb_stitch_shard_layout(at: Optional[Axis], ay: Axis, ax: Axis, B: int, C: int, world: int,
                           rank: int) -> ShardLayout:
    """Rank ``rank``'s share of a stitch whose tile rows are split over
    ``world`` ranks (host only)."""
    _, pt = _axis_ref(at)
    _, py = _axis_ref(ay)
    _, px = _axis_ref(ax)
    out = tb_shard_layout()
    _check(_lib.tb_stitch_shard_layout(pt, py, px, B, C, world, rank, ctypes.byref(out)), "tb_stitch_shard_layout")
    return ShardLayout(out.row_begin, out.row_end, out.out_row_begin, out.out_rows, out.halo_rows, out.halo_elems,
                       out.send_elems)


def _flat_tiles(tiles, ndim: int) -> List[torch.Tensor]:
    if ndim == 2:
        return [t for row in tiles for t in row]
    return [t for plane in tiles for row in plane for t in row]


def tb_stitch_halo_pack(row_tiles, at: Optional[Axis], ay: Axis, ax: Axis, row: int, halo: torch.Tensor,
                        stream=None) -> torch.Tensor:
    """Pack the last e_y(row + 1) rows of every tile of tile row ``row`` into
    ``halo`` (1D, ``send_elems`` elements).  ``row_tiles`` is the list of the
    row's tiles: ``[t_j]`` for a 2D grid, ``[[t_kj]]`` (frame tile major) for
    a 3D grid."""
    flat = list(row_tiles) if at is None else [t for per_k in row_tiles for t in per_k]
    for q, t in enumerate(flat):
        _cuda_contig(t, "tile %d" % q)
    _cuda_contig(halo, "halo")
    B, C = flat[0].shape[:2]
    _, pt = _axis_ref(at)
    _, py = _axis_ref(ay)
    _, px = _axis_ref(ax)
    _check(_lib.tb_stitch_halo_pack(_ptr_array([t.data_ptr() for t in flat]), _dtype_code(halo), B, C, pt, py, px,
                                    row, halo.data_ptr(), _stream_handle(stream)), "tb_stitch_halo_pack")
    return halo


def tb_stitch2d_shard(tiles, halo: Optional[torch.Tensor], ay: Axis, ax: Axis, row_begin: int, row_end: int,
                      out: torch.Tensor, stream=None) -> torch.Tensor:
    """Stitch tile rows [row_begin, row_end) (``tiles[i - row_begin][j]``)
    with the band ``halo`` of the row above into ``out`` ([B, C, out_rows,
    W])."""
    _cuda_contig(out, "out")
    B, C, H, W = out.shape
    flat = _flat_tiles(tiles, 2)
    for q, t in enumerate(flat):
        _cuda_contig(t, "tile %d" % q)
        if t.dtype != out.dtype:
            raise ValueError("tile %d has dtype %s, out %s" % (q, t.dtype, out.dtype))
    hp = None
    if halo is not None:
        _cuda_contig(halo, "halo")
        hp = halo.data_ptr()
    a_y, a_x = ay.c(), ax.c()
    _check(_lib.tb_stitch2d_shard(_ptr_array([t.data_ptr() for t in flat]), hp, _dtype_code(out), B, C,
                                  ctypes.byref(a_y), ctypes.byref(a_x), row_begin, row_end, out.data_ptr(), H, W,
                                  _stream_handle(stream)), "tb_stitch2d_shard")
    return out


def tb_stitch3d_shard(tiles, halo: Optional[torch.Tensor], at: Axis, ay: Axis, ax: Axis, row_begin: int,
                      row_end: int, out: torch.Tensor, stream=None) -> torch.Tensor:
    """3D form of ``tb_stitch2d_shard``: ``tiles[k][i - row_begin][j]``,
    ``out`` [B, C, T, out_rows, W]."""
    _cuda_contig(out, "out")
    B, C, T, H, W = out.shape
    flat = _flat_tiles(tiles, 3)
    for q, t in enumerate(flat):
        _cuda_contig(t, "tile %d" % q)
        if t.dtype != out.dtype:
            raise ValueError("tile %d has dtype %s, out %s" % (q, t.dtype, out.dtype))
    hp = None
    if halo is not None:
        _cuda_contig(halo, "halo")
        hp = halo.data_ptr()
    a_t, a_y, a_x = at.c(), ay.c(), ax.c()
    _check(_lib.tb_stitch3d_shard(_ptr_array([t.data_ptr() for t in flat]), hp, _dtype_code(out), B, C,
                                  ctypes.byref(a_t), ctypes.byref(a_y), ctypes.byref(a_x), row_begin, row_end,
                                  out.data_ptr(), T, H, W, _stream_handle(stream)), "tb_stitch3d_shard")
    return out


def tb_stitch_shard_frames_layout(at: Axis, ay: Axis, ax: Axis, B: int, C: int, world: int,
                                  rank: int) -> ShardLayout:
    """Rank ``rank``'s share of a video stitch whose frame tiles are split
    over ``world`` ranks (host only; the fields count frame tiles and output
    frames)."""
    a_t, a_y, a_x = at.c(), ay.c(), ax.c()
    out = tb_shard_layout()
    _check(_lib.tb_stitch_shard_frames_layout(ctypes.byref(a_t), ctypes.byref(a_y), ctypes.byref(a_x), B, C, world,
                                              rank, ctypes.byref(out)), "tb_stitch_shard_frames_layout")
    return ShardLayout(out.row_begin, out.row_end, out.out_row_begin, out.out_rows, out.halo_rows, out.halo_elems,
                       out.send_elems)


def tb_stitch_halo_pack_frames(frame_tiles, at: Axis, ay: Axis, ax: Axis, frame_tile: int, halo: torch.Tensor,
                               stream=None) -> torch.Tensor:
    """Pack the last e_t(frame_tile + 1) frames of every tile of frame tile
    ``frame_tile`` (``frame_tiles[i][j]``) into ``halo``."""
    flat = [t for row in frame_tiles for t in row]
    for q, t in enumerate(flat):
        _cuda_contig(t, "tile %d" % q)
    _cuda_contig(halo, "halo")
    B, C = flat[0].shape[:2]
    a_t, a_y, a_x = at.c(), ay.c(), ax.c()
    _check(_lib.tb_stitch_halo_pack_frames(_ptr_array([t.data_ptr() for t in flat]), _dtype_code(halo), B, C,
                                           ctypes.byref(a_t), ctypes.byref(a_y), ctypes.byref(a_x), frame_tile,
                                           halo.data_ptr(), _stream_handle(stream)), "tb_stitch_halo_pack_frames")
    return halo


def tb_stitch3d_shard_frames(tiles, halo: Optional[torch.Tensor], at: Axis, ay: Axis, ax: Axis, frame_begin: int,
                             frame_end: int, out: torch.Tensor, stream=None) -> torch.Tensor:
    """Stitch frame tiles [frame_begin, frame_end) (``tiles[k - frame_begin][i][j]``)
    with the band ``halo`` of the frame tile before into ``out``
    ([B, C, out_frames, H, W])."""
    _cuda_contig(out, "out")
    B, C, T, H, W = out.shape
    flat = _flat_tiles(tiles, 3)
    for q, t in enumerate(flat):
        _cuda_contig(t, "tile %d" % q)
        if t.dtype != out.dtype:
            raise ValueError("tile %d has dtype %s, out %s" % (q, t.dtype, out.dtype))
    hp = None
    if halo is not None:
        _cuda_contig(halo, "halo")
        hp = halo.data_ptr()
    a_t, a_y, a_x = at.c(), ay.c(), ax.c()
    _check(_lib.tb_stitch3d_shard_frames(_ptr_array([t.data_ptr() for t in flat]), hp, _dtype_code(out), B, C,
                                         ctypes.byref(a_t), ctypes.byref(a_y), ctypes.byref(a_x), frame_begin,
                                         frame_end, out.data_ptr(), T, H, W, _stream_handle(stream)),
           "tb_stitch3d_shard_frames")
    return out


# ---------------------------------------------------------------------------
# normalised-ramp stitch
# ---------------------------------------------------------------------------

@dataclass(frozen=True)
class RampAxis:
    """One axis of a normalised-ramp tile layout (see tb_ramp_axis)."""
    origins: Tuple[int, ...]   # output samples, ascending, first 0, last + tile_extent == out_extent
    tile_extent: int
    out_extent: int
    zero: int                  # samples of zero weight next to a shared edge
    ramp: int                  # samples over which the weight rises to 1

    @staticmethod
    def spread(latent_extent: int, latent_tile: int, n_tiles: int, scale: int, zero_latents: int = 4,
               ramp_latents: int = 8) -> "RampAxis":
        """The library's layout of n_tiles tiles spread edge to edge
        (tb_ramp_axis_spread)."""
        org = (ctypes.c_int64 * max(1, n_tiles))()
        a = tb_ramp_axis()
        _check(_lib.tb_ramp_axis_spread(latent_extent, latent_tile, n_tiles, scale, zero_latents, ramp_latents, org,
                                        ctypes.byref(a)), "tb_ramp_axis_spread")
        return RampAxis(tuple(org[:n_tiles]), a.tile_extent, a.out_extent, a.zero, a.ramp)

    def c(self):
        arr = (ctypes.c_int64 * len(self.origins))(*self.origins)
        st = tb_ramp_axis(len(self.origins), self.tile_extent, self.out_extent, self.zero, self.ramp,
                          ctypes.cast(arr, ctypes.POINTER(ctypes.c_int64)))
        st._keep = arr  # the struct points into this array
        return st


def tb_stitch2d_ramp(tiles: Sequence[Sequence[torch.Tensor]], ay: RampAxis, ax: RampAxis, out: torch.Tensor,
                     stream=None) -> torch.Tensor:
    """Normalised-ramp stitch of ``tiles[i][j]`` ([B, C, ay.tile_extent,
    ax.tile_extent]) into ``out`` ([B, C, ay.out_extent, ax.out_extent])."""
    _cuda_contig(out, "out")
    B, C, H, W = out.shape
    if (H, W) != (ay.out_extent, ax.out_extent):
        raise ValueError("out must be [B, C, %d, %d]" % (ay.out_extent, ax.out_extent))
    if len(tiles) != len(ay.origins) or any(len(r) != len(ax.origins) for r in tiles):
        raise ValueError("expected a %d x %d tile grid" % (len(ay.origins), len(ax.origins)))
    shape = (B, C, ay.tile_extent, ax.tile_extent)
    ptrs = []
    for i, row in enumerate(tiles):
        for j, t in enumerate(row):
            if t.dtype != out.dtype or t.shape != shape or not t.is_cuda or not t.is_contiguous():
                _cuda_contig(t, "tile (%d,%d)" % (i, j))
                raise ValueError("tile (%d,%d) has %s %s, expected %s %s" % (i, j, t.dtype, tuple(t.shape),
                                                                            out.dtype, shape))
            ptrs.append(t.data_ptr())
    a_y, a_x = ay.c(), ax.c()
    _check(_lib.tb_stitch2d_ramp(_ptr_array(ptrs), _dtype_code(out), B, C, ctypes.byref(a_y), ctypes.byref(a_x),
                                 out.data_ptr(), _stream_handle(stream)), "tb_stitch2d_ramp")
    return out


# ---------------------------------------------------------------------------
# PatchGroupNorm
# ---------------------------------------------------------------------------

def _gn_args(patches: Sequence[torch.Tensor]) -> Tuple[int, int, int, list, list]:
    if len(patches) == 0:
        raise ValueError("at least one patch")
    N, C = patches[0].shape[:2]
    spatial = []
    ptrs = []
    for q, t in enumerate(patches):
        _cuda_contig(t, "patch %d" % q)
        if t.dtype != patches[0].dtype or tuple(t.shape[:2]) != (N, C):
            raise ValueError("patch %d: dtype/leading dims differ from patch 0" % q)
        s = 1
        for d in t.shape[2:]:
            s *= d
        spatial.append(s)
        ptrs.append(t.data_ptr())
    return N, C, _dtype_code(patches[0]), spatial, ptrs


def new_partials(P: int, N: int, G: int, device=None) -> torch.Tensor:
    """Device buffer for the P * N * G * TB_GN_PARTS tb_gn_partial records
    (16 bytes each) that tb_patch_gn_stats writes."""
    return torch.empty((P, N, G, TB_GN_PARTS, 2), dtype=torch.int64, device=device or torch.device("cuda"))


def tb_patch_gn_stats(patches: Sequence[torch.Tensor], G: int, partials: torch.Tensor, stream=None) -> torch.Tensor:
    """(count, mean, M2) of every part of every (patch, sample, group) into
    ``partials`` (a [P, N, G, TB_GN_PARTS, 2] int64 buffer from
    ``new_partials``)."""
    N, C, dt, spatial, ptrs = _gn_args(patches)
    P = len(patches)
    _cuda_contig(partials, "partials")
    if partials.numel() * partials.element_size() != P * N * G * TB_GN_PARTS * 16:
        raise ValueError("partials must hold P*N*G*TB_GN_PARTS 16-byte records")
    sp = (ctypes.c_int64 * P)(*spatial)
    _check(_lib.tb_patch_gn_stats(_ptr_array(ptrs), P, dt, N, C, sp, G, partials.data_ptr(), _stream_handle(stream)),
           "tb_patch_gn_stats")
    return partials


def tb_patch_gn_apply(patches: Sequence[torch.Tensor], outs: Sequence[torch.Tensor], G: int, partials: torch.Tensor,
                      gamma: Optional[torch.Tensor], beta: Optional[torch.Tensor], eps: float, silu: bool = True,
                      stream=None) -> Sequence[torch.Tensor]:
    """Normalise every patch with the pooled statistics of ``partials``;
    ``outs[p]`` may be ``patches[p]``."""
    N, C, dt, spatial, ptrs = _gn_args(patches)
    P = len(patches)
    if len(outs) != P:
        raise ValueError("one output per patch")
    optrs = []
    for q, (o, t) in enumerate(zip(outs, patches)):
        _cuda_contig(o, "out %d" % q)
        if o.shape != t.shape or o.dtype != t.dtype:
            raise ValueError("out %d must match patch %d" % (q, q))
        optrs.append(o.data_ptr())
    for name, v in (("gamma", gamma), ("beta", beta)):
        if v is not None:
            _cuda_contig(v, name)
            if v.numel() != C or v.dtype != patches[0].dtype:
                raise ValueError("%s must be [C] of the patches' dtype" % name)
    _cuda_contig(partials, "partials")
    if partials.numel() * partials.element_size() != P * N * G * TB_GN_PARTS * 16:
        raise ValueError("partials must hold P*N*G*TB_GN_PARTS 16-byte records")
    sp = (ctypes.c_int64 * P)(*spatial)
    _check(_lib.tb_patch_gn_apply(_ptr_array(ptrs), _ptr_array(optrs), P, dt, N, C, sp, G, partials.data_ptr(),
                                  gamma.data_ptr() if gamma is not None else None,
                                  beta.data_ptr() if beta is not None else None, float(eps), 1 if silu else 0,
                                  _stream_handle(stream)), "tb_patch_gn_apply")
    return outs


def tb_patch_gn_apply_gathered(patches: Sequence[torch.Tensor], outs: Sequence[torch.Tensor], G: int,
                               partials: torch.Tensor, R: int, gamma: Optional[torch.Tensor],
                               beta: Optional[torch.Tensor], eps: float, silu: bool = True,
                               stream=None) -> Sequence[torch.Tensor]:
    """Normalise the local ``patches`` with the pooled statistics of ``R``
    record sets (``partials``: [R, N, G, TB_GN_PARTS, 2] int64, e.g. every
    rank's records after an all-gather)."""
    N, C, dt, spatial, ptrs = _gn_args(patches)
    P = len(patches)
    if len(outs) != P:
        raise ValueError("one output per patch")
    optrs = []
    for q, (o, t) in enumerate(zip(outs, patches)):
        _cuda_contig(o, "out %d" % q)
        if o.shape != t.shape or o.dtype != t.dtype:
            raise ValueError("out %d must match patch %d" % (q, q))
        optrs.append(o.data_ptr())
    for name, v in (("gamma", gamma), ("beta", beta)):
        if v is not None:
            _cuda_contig(v, name)
            if v.numel() != C or v.dtype != patches[0].dtype:
                raise ValueError("%s must be [C] of the patches' dtype" % name)
    _cuda_contig(partials, "partials")
    if partials.numel() * partials.element_size() != R * N * G * TB_GN_PARTS * 16:
        raise ValueError("partials must hold R*N*G*TB_GN_PARTS 16-byte records")
    sp = (ctypes.c_int64 * P)(*spatial)
    _check(_lib.tb_patch_gn_apply_gathered(_ptr_array(ptrs), _ptr_array(optrs), P, dt, N, C, sp, G,
                                           partials.data_ptr(), R, gamma.data_ptr() if gamma is not None else None,
                                           beta.data_ptr() if beta is not None else None, float(eps),
                                           1 if silu else 0, _stream_handle(stream)), "tb_patch_gn_apply_gathered")
    return outs


def patch_group_norm(patches: Sequence[torch.Tensor], G: int, gamma, beta, eps: float, silu: bool = True,
                     outs: Optional[Sequence[torch.Tensor]] = None, partials: Optional[torch.Tensor] = None,
                     stream=None) -> Sequence[torch.Tensor]:
    """Both steps: statistics of every patch, then the pooled normalisation."""
    N = patches[0].shape[0]
    if partials is None:
        partials = new_partials(len(patches), N, G, patches[0].device)
    if outs is None:
        outs = [torch.empty_like(p) for p in patches]
    tb_patch_gn_stats(patches, G, partials, stream)
    return tb_patch_gn_apply(patches, outs, G, partials, gamma, beta, eps, silu, stream)


def tb_patch_group_norm_noalloc(patches: Sequence[torch.Tensor], outs: Sequence[torch.Tensor], G: int,
                                gamma: Optional[torch.Tensor], beta: Optional[torch.Tensor], eps: float,
                                silu: bool = True, stream=None) -> Sequence[torch.Tensor]:
    """PatchGroupNorm for callers that cannot allocate device memory: the
    partial statistics live in the library's own fixed scratch array (room
    for P * N * G * TB_GN_PARTS <= TB_NOALLOC_MAX_PARTIALS records), so the
    call needs no buffer besides the inputs and outputs.  Calls share that array: order
    them on one stream.  The first call on a device looks the array's
    address up."""
    N, C, dt, spatial, ptrs = _gn_args(patches)
    P = len(patches)
    if len(outs) != P:
        raise ValueError("one output per patch")
    optrs = []
    for q, (o, t) in enumerate(zip(outs, patches)):
        _cuda_contig(o, "out %d" % q)
        if o.shape != t.shape or o.dtype != t.dtype:
            raise ValueError("out %d must match patch %d" % (q, q))
        optrs.append(o.data_ptr())
    for name, v in (("gamma", gamma), ("beta", beta)):
        if v is not None:
            _cuda_contig(v, name)
            if v.numel() != C or v.dtype != patches[0].dtype:
                raise ValueError("%s must be [C] of the patches' dtype" % name)
    sp = (ctypes.c_int64 * P)(*spatial)
    _check(_lib.tb_patch_group_norm_noalloc(_ptr_array(ptrs), _ptr_array(optrs), P, dt, N, C, sp, G,
                                            gamma.data_ptr() if gamma is not None else None,
                                            beta.data_ptr() if beta is not None else None, float(eps),
                                            1 if silu else 0, _stream_handle(stream)),
           "tb_patch_group_norm_noalloc")
    return outs


# ---------------------------------------------------------------------------
# Patchify split / patch gather
# ---------------------------------------------------------------------------

def tb_patchify_layout(extent: int, factor: int, P: int) -> Tuple[List[int], List[int]]:
    """(starts, sizes) of the P ranks' bands of an axis of ``extent``
    positions: whole bands of ``factor``, the first ranks one band more."""
    starts, sizes = (ctypes.c_int64 * max(1, P))(), (ctypes.c_int64 * max(1, P))()
    _check(_lib.tb_patchify_layout(extent, factor, P, starts, sizes), "tb_patchify_layout")
    return list(starts[:P]), list(sizes[:P])


def _shape_arr(shape) -> ctypes.Array:
    return (ctypes.c_int64 * max(1, len(shape)))(*shape)


def tb_patchify(x: torch.Tensor, axis: int, factor: int, P: int, patches: Optional[Sequence[torch.Tensor]] = None,
                slot: int = 0, stream=None) -> List[torch.Tensor]:
    """The P ranks' patches of ``x`` along ``axis``.  With ``slot`` > 0 every
    patch buffer has ``slot`` positions along the axis (the band fills the
    first ones; the rest are not written)."""
    _cuda_contig(x, "x")
    axis = axis % x.dim()
    _, sizes = tb_patchify_layout(x.shape[axis], factor, P)
    shapes = []
    for sz in sizes:
        sh = list(x.shape)
        sh[axis] = slot if slot > 0 else sz
        shapes.append(tuple(sh))
    if patches is None:
        patches = [torch.empty(sh, dtype=x.dtype, device=x.device) for sh in shapes]
    if len(patches) != P:
        raise ValueError("one patch buffer per rank")
    for q, (t, sh) in enumerate(zip(patches, shapes)):
        _cuda_contig(t, "patch %d" % q)
        if tuple(t.shape) != sh or t.dtype != x.dtype:
            raise ValueError("patch %d must be %s %s" % (q, x.dtype, sh))
    _check(_lib.tb_patchify(x.data_ptr(), _dtype_code(x), x.dim(), _shape_arr(x.shape), axis, factor, P, slot,
                            _ptr_array([t.data_ptr() for t in patches]), _stream_handle(stream)), "tb_patchify")
    return list(patches)


def tb_gather_patches(patches: Sequence[torch.Tensor], sizes: Sequence[int], axis: int,
                      out: Optional[torch.Tensor] = None, slot: int = 0, stream=None) -> torch.Tensor:
    """Concatenate the first ``sizes[p]`` positions along ``axis`` of every
    patch, in rank order.  With ``slot`` > 0 every patch buffer has ``slot``
    positions along the axis."""
    if len(patches) == 0 or len(sizes) != len(patches):
        raise ValueError("one size per patch, at least one patch")
    ref = patches[0]
    axis = axis % ref.dim()
    shape = list(ref.shape)
    shape[axis] = sum(sizes)
    for q, (t, sz) in enumerate(zip(patches, sizes)):
        _cuda_contig(t, "patch %d" % q)
        want = list(ref.shape)
        want[axis] = slot if slot > 0 else sz
        if list(t.shape) != want or t.dtype != ref.dtype:
            raise ValueError("patch %d must be %s %s" % (q, ref.dtype, tuple(want)))
    if out is None:
        out = torch.empty(shape, dtype=ref.dtype, device=ref.device)
    _cuda_contig(out, "out")
    if list(out.shape) != shape or out.dtype != ref.dtype:
        raise ValueError("out must be %s %s" % (ref.dtype, tuple(shape)))
    sz = (ctypes.c_int64 * len(sizes))(*sizes)
    _check(_lib.tb_gather_patches(_ptr_array([t.data_ptr() for t in patches]), len(patches), sz, _dtype_code(out),
                                  out.dim(), _shape_arr(shape), axis, slot, out.data_ptr(), _stream_handle(stream)),
           "tb_gather_patches")
    return out


# ---------------------------------------------------------------------------
# training: layer norm
# ---------------------------------------------------------------------------

def _on_stream(make, stream):
    """Tensors made by ``make()`` for work on ``stream``: allocated with that
    stream current, so that the allocator reuses their memory in its order."""
    if stream is None:
        return make()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream))
    with torch.cuda.stream(stream):
        return make()


_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _stream_of(stream, device: int) -> int:
    """The stream's handle, for a launch that takes tensors of ``device``: the
    library launches on the current device."""
    if device != _current_device():
        raise ValueError("the tensors are on CUDA device %d, the current device is %d" % (device, _current_device()))
    return _raw_stream(device) if stream is None else _stream_handle(stream)


def _row_ld(t: torch.Tensor, shape, dtype, device: int, what: str) -> int:
    """The row stride (elements) of a tensor seen as rows of its last axis."""
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError("%s has %s %s, expected %s %s" % (what, t.dtype, tuple(t.shape), dtype, tuple(shape)))
    if t.get_device() != device:
        raise ValueError("%s must be on the CUDA device of the other tensors" % what)
    if t.is_contiguous():
        return shape[-1]
    if shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError("%s: the elements of a row must be contiguous" % what)
    ld, span = None, 1  # stride of the innermost row axis, and the rows inside the axis at hand
    for size, st in zip(reversed(shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if ld is None:
            ld = st
        elif st != ld * span:
            raise ValueError("%s: the rows must have one stride" % what)
        span *= size
    if ld is None:
        return shape[-1]
    if ld < shape[-1] and t.numel() > 0:
        raise ValueError("%s: the rows overlap" % what)
    return ld


def _vec(t: Optional[torch.Tensor], n: int, dtype, device: int, what: str):
    """Address of a contiguous tensor of n elements, or None."""
    if t is None:
        return None
    if t.numel() != n or t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
        raise ValueError("%s must be a contiguous [%d] %s tensor on the same device" % (what, n, dtype))
    return t.data_ptr()


def _ln_head(x: torch.Tensor, weight: Optional[torch.Tensor]) -> Tuple[torch.Size, int, int, int, torch.dtype]:
    """(shape, rows, cols, device, weights' dtype) of a layer norm of x."""
    shape, dev = x.shape, x.get_device()
    if dev < 0:
        raise ValueError("the rows must be CUDA tensors")
    if not shape or shape[-1] < 1:
        raise ValueError("rows of at least one element")
    cols = shape[-1]
    wdtype = x.dtype if weight is None else weight.dtype
    if wdtype is not x.dtype and wdtype is not torch.float32:
        raise ValueError("the weights must have the rows' dtype or float32, got %s" % wdtype)
    return shape, x.numel() // cols, cols, dev, wdtype


def tb_layer_norm(x: torch.Tensor, y: torch.Tensor, gamma: Optional[torch.Tensor], beta: Optional[torch.Tensor],
                  eps: float, mean: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None,
                  residual: Optional[torch.Tensor] = None, total: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """Layer norm of x (or x + residual, which goes to ``total``) over the
    last axis into ``y``.  ``x``, ``residual``, ``total`` and ``y`` are
    [..., cols] with any row stride; ``gamma`` / ``beta`` [cols] of x's dtype
    or float32; ``mean`` / ``rstd`` float32, one per row, for the backward
    pass.  ``y`` may be ``x``; ``total`` may be ``x`` or ``residual``."""
    shape, rows, cols, dev, wdt = _ln_head(x, beta if gamma is None else gamma)
    dt = x.dtype
    rp = tp = None
    r_ld = t_ld = 0
    if residual is not None:
        if total is None:
            raise ValueError("a residual needs a total to write the sum to")
        r_ld, t_ld = _row_ld(residual, shape, dt, dev, "residual"), _row_ld(total, shape, dt, dev, "total")
        rp, tp = residual.data_ptr(), total.data_ptr()
    elif total is not None:
        raise ValueError("total without a residual")
    status = _lib.tb_layer_norm(x.data_ptr(), _row_ld(x, shape, dt, dev, "x"), rp, r_ld, _dtype_code(x), rows, cols,
                                _vec(gamma, cols, wdt, dev, "gamma"), _vec(beta, cols, wdt, dev, "beta"),
                                _DTYPES[wdt], eps, tp, t_ld, y.data_ptr(), _row_ld(y, shape, dt, dev, "y"),
                                _vec(mean, rows, torch.float32, dev, "mean"),
                                _vec(rstd, rows, torch.float32, dev, "rstd"), _stream_of(stream, dev))
    if status:
        raise TileBlendError(status, "tb_layer_norm")
    return y


def layer_norm(x: torch.Tensor, gamma: Optional[torch.Tensor], beta: Optional[torch.Tensor], eps: float,
               residual: Optional[torch.Tensor] = None, stream=None):
    """``(y, mean, rstd)`` of tb_layer_norm in new tensors; with a residual
    ``(y, mean, rstd, total)``."""
    def make():
        stats = torch.empty((2,) + tuple(x.shape[:-1]), dtype=torch.float32, device=x.device)
        out = [torch.empty(x.shape, dtype=x.dtype, device=x.device), stats[0], stats[1]]
        return out if residual is None else out + [torch.empty(x.shape, dtype=x.dtype, device=x.device)]
    out = _on_stream(make, stream)
    tb_layer_norm(x, out[0], gamma, beta, eps, out[1], out[2], residual, out[3] if residual is not None else None,
                  stream)
    return tuple(out)


def ln_workspace(rows: int, cols: int, device=None) -> torch.Tensor:
    """The device workspace of tb_layer_norm_backward for these sizes; it may
    serve any number of calls in turn on one stream."""
    n = int(_lib.tb_layer_norm_workspace(rows, cols))
    if n < 0:
        raise ValueError("no layer norm of %d rows of %d elements" % (rows, cols))
    return torch.empty(n, dtype=torch.uint8, device=device or torch.device("cuda"))


def tb_layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                           gamma: Optional[torch.Tensor], dx: Optional[torch.Tensor], dgamma: Optional[torch.Tensor],
                           dbeta: Optional[torch.Tensor], workspace: Optional[torch.Tensor],
                           dtotal: Optional[torch.Tensor] = None, stream=None) -> None:
    """Gradients of tb_layer_norm: ``dx`` (rows like ``x``; ``x`` is what was
    normalised, the total where there was a residual), ``dgamma`` / ``dbeta``
    ([cols]; the sums over all rows).  ``dtotal`` is added to dx.  Any output
    may be None; ``workspace`` comes from ``ln_workspace`` (None without
    weight gradients)."""
    weight = gamma if gamma is not None else dgamma if dgamma is not None else dbeta
    shape, rows, cols, dev, wdt = _ln_head(x, weight)
    dt = x.dtype
    dy_ld, x_ld = _row_ld(dy, shape, dt, dev, "dy"), _row_ld(x, shape, dt, dev, "x")
    dxp = dtp = None
    dx_ld = dt_ld = 0
    if dx is not None:
        dx_ld, dxp = _row_ld(dx, shape, dt, dev, "dx"), dx.data_ptr()
    if dtotal is not None:
        dt_ld, dtp = _row_ld(dtotal, shape, dt, dev, "dtotal"), dtotal.data_ptr()
    wp, wb = None, 0
    if workspace is not None:
        if not workspace.is_contiguous() or workspace.get_device() != dev:
            raise ValueError("workspace must be contiguous, on the same device")
        wp, wb = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _check(_lib.tb_layer_norm_backward(dy.data_ptr(), dy_ld, x.data_ptr(), x_ld, _dtype_code(x), rows, cols,
                                       _vec(mean, rows, torch.float32, dev, "mean"),
                                       _vec(rstd, rows, torch.float32, dev, "rstd"),
                                       _vec(gamma, cols, wdt, dev, "gamma"), _DTYPES[wdt], dtp, dt_ld, dxp, dx_ld,
                                       _vec(dgamma, cols, wdt, dev, "dgamma"), _vec(dbeta, cols, wdt, dev, "dbeta"),
                                       wp, wb, _stream_of(stream, dev)), "tb_layer_norm_backward")


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        gamma: Optional[torch.Tensor], dtotal: Optional[torch.Tensor] = None, wdtype=None,
                        stream=None, needs=(True, True, True)
                        ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor], Optional[torch.Tensor]]:
    """``(dx, dgamma, dbeta)`` in new tensors (the weights' dtype is gamma's,
    or ``wdtype``).  ``needs``: which of the three are wanted; the others are
    None and not computed."""
    cols = x.shape[-1]
    wdt = gamma.dtype if gamma is not None else wdtype or x.dtype

    def make():
        return (torch.empty(x.shape, dtype=x.dtype, device=x.device) if needs[0] else None,
                torch.empty(cols, dtype=wdt, device=x.device) if needs[1] else None,
                torch.empty(cols, dtype=wdt, device=x.device) if needs[2] else None,
                ln_workspace(x.numel() // max(1, cols), cols, x.device) if needs[1] or needs[2] else None)
    dx, dgamma, dbeta, ws = _on_stream(make, stream)
    tb_layer_norm_backward(dy, x, mean, rstd, gamma, dx, dgamma, dbeta, ws, dtotal, stream)
    return dx, dgamma, dbeta


# ---------------------------------------------------------------------------
# training: gradient norm and clip
# ---------------------------------------------------------------------------

class GradTable:
    """The gradients of a program's parameters (``grads``), and where their
    clipped values go (``outs``; None: in place), as the library takes them.
    It holds the tensors and their addresses, none of their contents: make it
    once, and again when a gradient tensor is replaced.  Every output is
    separate from the others and from the other gradients."""

    def __init__(self, grads: Sequence[torch.Tensor], outs: Optional[Sequence[torch.Tensor]] = None):
        self.grads = list(grads)
        self.outs = self.grads if outs is None else list(outs)
        if len(self.outs) != len(self.grads):
            raise ValueError("one output per gradient")
        n = len(self.grads)
        for q, (g, o) in enumerate(zip(self.grads, self.outs)):
            _cuda_contig(g, "gradient %d" % q)
            if o is not g:
                _cuda_contig(o, "output %d" % q)
                if o.shape != g.shape or o.dtype != g.dtype:
                    raise ValueError("output %d must match gradient %d" % (q, q))
            if g.device != self.grads[0].device or o.device != g.device:
                raise ValueError("all gradients and outputs must be on one device")
        self.device = self.grads[0].device if n else None
        self._index = self.grads[0].get_device() if n else None
        self._refuse_overlaps()
        self._in = _ptr_array([g.data_ptr() for g in self.grads])
        self._out = _ptr_array([o.data_ptr() for o in self.outs])
        self._numel = (ctypes.c_int64 * max(1, n))(*[g.numel() for g in self.grads])
        self._dtypes = (ctypes.c_int32 * max(1, n))(*[_dtype_code(g) for g in self.grads])
        self._records = int(_lib.tb_grad_records(n))

    def __len__(self) -> int:
        return len(self.grads)

    def _refuse_overlaps(self) -> None:
        """Outputs must not share elements with one another, nor with any
        gradient but their own, in place (a shared parameter's gradient is
        listed once)."""
        ranges = []
        for g, o in zip(self.grads, self.outs):
            at, to, n = g.data_ptr(), o.data_ptr(), g.numel() * g.element_size()
            if n:
                ranges.append((to, to + n, True))
                if at != to:
                    ranges.append((at, at + n, False))
        read_to = written_to = 0
        for first, last, written in sorted(ranges):
            if first < written_to or (written and first < read_to):
                raise ValueError("outputs overlap one another, or gradients of other outputs")
            if written:
                written_to = max(written_to, last)
            else:
                read_to = max(read_to, last)


def new_grad_records(T: int, device=None) -> torch.Tensor:
    """Device buffer (float64) for the records tb_grad_stats writes for T
    tensors."""
    n = int(_lib.tb_grad_records(T))
    if n < 0:
        raise ValueError("at most %d gradients in one call" % TB_MAX_GRADS)
    return torch.empty(n, dtype=torch.float64, device=device or torch.device("cuda"))


def _records(records: torch.Tensor, table: Optional[GradTable] = None) -> int:
    if records.get_device() < 0 or records.dtype is not torch.float64 or not records.is_contiguous():
        raise ValueError("records must be a contiguous float64 CUDA tensor")
    if table is not None and table._index not in (None, records.get_device()):
        raise ValueError("records must be on the gradients' device")
    return records.data_ptr()


def _own_records(records: torch.Tensor, table: GradTable) -> int:
    at = _records(records, table)
    if records.numel() != table._records and table._records >= 0:
        raise ValueError("records must hold exactly %d values for %d gradients" % (table._records, len(table)))
    return at


def tb_grad_stats(table: GradTable, records: torch.Tensor, stream=None) -> torch.Tensor:
    """Sums of squares of the table's gradients into ``records`` (from
    ``new_grad_records``)."""
    at = _own_records(records, table)
    _check(_lib.tb_grad_stats(table._in, table._numel, table._dtypes, len(table), at,
                              _stream_of(stream, records.get_device())), "tb_grad_stats")
    return records


def _norm_ptr(norm: Optional[torch.Tensor], device: int):
    if norm is None:
        return None
    if norm.get_device() != device or norm.dtype is not torch.float32 or norm.numel() != 1:
        raise ValueError("norm must be one float32 on the records' device")
    return norm.data_ptr()


def tb_grad_norm(records: torch.Tensor, norm: torch.Tensor, stream=None) -> torch.Tensor:
    """The global norm that ``records`` (one or more record sets) describe."""
    at, dev = _records(records), records.get_device()
    _check(_lib.tb_grad_norm(at, records.numel(), _norm_ptr(norm, dev), _stream_of(stream, dev)), "tb_grad_norm")
    return norm


def tb_grad_clip(table: GradTable, records: torch.Tensor, max_norm: float, norm: Optional[torch.Tensor] = None,
                 stream=None) -> None:
    """Every gradient of the table times min(1, max_norm / (norm + 1e-6)), into
    its output; the norm is that of all ``records``."""
    at, dev = _records(records, table), records.get_device()
    _check(_lib.tb_grad_clip(table._in, table._out, table._numel, table._dtypes, len(table), at, records.numel(),
                             max_norm, _norm_ptr(norm, dev), _stream_of(stream, dev)), "tb_grad_clip")


def clip_grad_norm(grads, max_norm: float, records: Optional[torch.Tensor] = None,
                   norm: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Both steps: the global norm of ``grads`` (a GradTable, or tensors to be
    clipped in place), then the clip.  Returns the norm before it (a [1]
    float32 tensor)."""
    table = grads if isinstance(grads, GradTable) else GradTable(grads)
    if records is None:
        records = _on_stream(lambda: new_grad_records(len(table), table.device), stream)
    if norm is None:
        norm = _on_stream(lambda: torch.empty(1, dtype=torch.float32, device=records.device), stream)
    # one check of the arguments for both calls
    at, dev = _own_records(records, table), records.get_device()
    out, handle, T = _norm_ptr(norm, dev), _stream_of(stream, dev), len(table)
    _check(_lib.tb_grad_stats(table._in, table._numel, table._dtypes, T, at, handle), "tb_grad_stats")
    _check(_lib.tb_grad_clip(table._in, table._out, table._numel, table._dtypes, T, at, records.numel(), max_norm, out,
                             handle), "tb_grad_clip")
    return norm


# ---------------------------------------------------------------------------
# training: PatchGroupNorm backward
# ---------------------------------------------------------------------------

def new_grad_partials(P: int, N: int, C: int, device=None) -> torch.Tensor:
    """Device buffer for the P * N * C * TB_GN_PARTS tb_gn_grad_partial records
    (8 bytes each) that tb_patch_gn_grad_stats writes."""
    return torch.empty((P, N, C, TB_GN_PARTS, 2), dtype=torch.float32, device=device or torch.device("cuda"))


_PTRS = {n: ctypes.c_void_p * n for n in range(1, 65)}
_COUNTS = {n: ctypes.c_int64 * n for n in range(1, 65)}


def _like_patches(ts, patches, what: str):
    """Addresses of one tensor per patch, each like its patch."""
    P = len(patches)
    if len(ts) != P:
        raise ValueError("one %s per patch" % what)
    for q in range(P):
        t, x = ts[q], patches[q]
        if t.shape != x.shape or t.dtype is not x.dtype or t.get_device() != x.get_device() or not t.is_contiguous():
            raise ValueError("%s %d must be contiguous and match patch %d" % (what, q, q))
    return _PTRS[P](*[t.data_ptr() for t in ts])


def _gn_grad_args(grads, patches, G, partials, R, gamma, beta):
    P = len(patches)
    if not 1 <= P <= 64:
        raise ValueError("1 to 64 patches")
    first = patches[0]
    dt, dev = first.dtype, first.get_device()
    N, C = first.shape[:2]
    spatial = []
    for q, x in enumerate(patches):
        if x.get_device() != dev or dev < 0 or not x.is_contiguous():
            raise ValueError("patch %d must be a contiguous CUDA tensor, on the device of patch 0" % q)
        if x.dtype is not dt or x.shape[0] != N or x.shape[1] != C:
            raise ValueError("patch %d: dtype/leading dims differ from patch 0" % q)
        spatial.append(x.numel() // (N * C) if N * C else 0)
    xs = _PTRS[P](*[x.data_ptr() for x in patches])
    ds = _like_patches(grads, patches, "gradient")
    _vec(gamma, C, dt, dev, "gamma")
    _vec(beta, C, dt, dev, "beta")
    if partials.get_device() != dev or not partials.is_contiguous() or \
            partials.numel() * partials.element_size() != R * N * G * TB_GN_PARTS * 16:
        raise ValueError("partials must hold R*N*G*TB_GN_PARTS 16-byte records")
    return N, C, _dtype_code(first), _COUNTS[P](*spatial), xs, ds


def _gn_grad_outs(dxs, patches, C, dgamma, dbeta):
    dt, dev = patches[0].dtype, patches[0].get_device()
    return _like_patches(dxs, patches, "dx"), _vec(dgamma, C, dt, dev, "dgamma"), _vec(dbeta, C, dt, dev, "dbeta")


def _grad_partials(t: torch.Tensor, R: int, N: int, C: int, device: int) -> int:
    if t.get_device() != device or not t.is_contiguous() or t.numel() * t.element_size() != R * N * C * TB_GN_PARTS * 8:
        raise ValueError("grad_partials must hold R*N*C*TB_GN_PARTS 8-byte records on the patches' device")
    return t.data_ptr()


def tb_patch_gn_grad_stats(grads: Sequence[torch.Tensor], patches: Sequence[torch.Tensor], G: int,
                           partials: torch.Tensor, R: int, gamma: Optional[torch.Tensor],
                           beta: Optional[torch.Tensor], eps: float, grad_partials: torch.Tensor, silu: bool = True,
                           stream=None) -> torch.Tensor:
    """Sums of dz and dz * xhat of every part of every (patch, sample,
    channel) into ``grad_partials`` (from ``new_grad_partials``).  ``grads``
    are the gradients of the norm's outputs, ``patches`` its inputs,
    ``partials`` the forward pass's ``R`` record sets."""
    N, C, dt, sp, xs, ds = _gn_grad_args(grads, patches, G, partials, R, gamma, beta)
    P = len(patches)
    _check(_lib.tb_patch_gn_grad_stats(xs, ds, P, dt, N, C, sp, G, partials.data_ptr(), R,
                                       gamma.data_ptr() if gamma is not None else None,
                                       beta.data_ptr() if beta is not None else None, float(eps), 1 if silu else 0,
                                       _grad_partials(grad_partials, P, N, C, patches[0].get_device()),
                                       _stream_of(stream, patches[0].get_device())), "tb_patch_gn_grad_stats")
    return grad_partials


def tb_patch_gn_grad_apply(grads: Sequence[torch.Tensor], patches: Sequence[torch.Tensor],
                           dxs: Sequence[torch.Tensor], G: int, partials: torch.Tensor, grad_partials: torch.Tensor,
                           R: int, gamma: Optional[torch.Tensor], beta: Optional[torch.Tensor], eps: float,
                           dgamma: Optional[torch.Tensor] = None, dbeta: Optional[torch.Tensor] = None,
                           silu: bool = True, stream=None) -> Sequence[torch.Tensor]:
    """The gradients of the patches into ``dxs`` (``dxs[p]`` may be
    ``grads[p]`` or ``patches[p]``), and of the weights into ``dgamma`` /
    ``dbeta`` ([C] of the patches' dtype), from the ``R`` record sets of both
    passes."""
    N, C, dt, sp, xs, ds = _gn_grad_args(grads, patches, G, partials, R, gamma, beta)
    P, dev = len(patches), patches[0].get_device()
    os_, gp, bp = _gn_grad_outs(dxs, patches, C, dgamma, dbeta)
    _check(_lib.tb_patch_gn_grad_apply(xs, ds, os_, P, dt, N, C, sp, G,
                                       partials.data_ptr(), _grad_partials(grad_partials, R, N, C, dev), R,
                                       gamma.data_ptr() if gamma is not None else None,
                                       beta.data_ptr() if beta is not None else None, float(eps), 1 if silu else 0,
                                       gp, bp, _stream_of(stream, dev)),
           "tb_patch_gn_grad_apply")
    return dxs


def patch_group_norm_backward(grads: Sequence[torch.Tensor], patches: Sequence[torch.Tensor], G: int,
                              partials: torch.Tensor, gamma: Optional[torch.Tensor], beta: Optional[torch.Tensor],
                              eps: float, silu: bool = True, dxs: Optional[Sequence[torch.Tensor]] = None,
                              dgamma: Optional[torch.Tensor] = None, dbeta: Optional[torch.Tensor] = None,
                              grad_partials: Optional[torch.Tensor] = None, stream=None):
    """Both steps of the backward pass of ``patch_group_norm``: ``(dxs, dgamma,
    dbeta)``.  ``partials`` are the forward pass's records of these patches;
    outputs that are not given are made."""
    P = len(patches)
    if P == 0:
        raise ValueError("at least one patch")
    _cuda_contig(patches[0], "patch 0")
    N, C = patches[0].shape[:2]

    def make():
        w = torch.empty((2, C), dtype=patches[0].dtype, device=patches[0].device)
        return ([torch.empty_like(p) for p in patches] if dxs is None else dxs,
                torch.empty_like(w[0]) if dgamma is None else dgamma,
                torch.empty_like(w[1]) if dbeta is None else dbeta,
                new_grad_partials(P, N, C, patches[0].device) if grad_partials is None else grad_partials)
    if dxs is None or dgamma is None or dbeta is None or grad_partials is None:
        dxs, dgamma, dbeta, grad_partials = _on_stream(make, stream)
    # one check and one set of argument arrays for both calls
    N, C, dt, sp, xs, ds = _gn_grad_args(grads, patches, G, partials, P, gamma, beta)
    os_, gp, bp = _gn_grad_outs(dxs, patches, C, dgamma, dbeta)
    dev = patches[0].get_device()
    rec, grec = partials.data_ptr(), _grad_partials(grad_partials, P, N, C, dev)
    ga = gamma.data_ptr() if gamma is not None else None
    be = beta.data_ptr() if beta is not None else None
    handle, act = _stream_of(stream, dev), 1 if silu else 0
    _check(_lib.tb_patch_gn_grad_stats(xs, ds, P, dt, N, C, sp, G, rec, P, ga, be, eps, act, grec, handle),
           "tb_patch_gn_grad_stats")
    _check(_lib.tb_patch_gn_grad_apply(xs, ds, os_, P, dt, N, C, sp, G, rec, grec, P, ga, be, eps, act, gp, bp, handle),
           "tb_patch_gn_grad_apply")
    return dxs, dgamma, dbeta


# ---------------------------------------------------------------------------
# channels last: PatchGroupNorm forward and backward
# ---------------------------------------------------------------------------

def _cl_args(patches, gamma, beta, *likes):
    """(N, C, dtype, device, P, table, addresses of its parts, gamma's and beta's
    address) of channels-last patches [N, *spatial_p, C] and lists of tensors like
    them.  The table is one array: each patch's positions, the patches' addresses,
    then those of each list."""
    P = len(patches)
    if not 1 <= P <= 64:
        raise ValueError("1 to 64 patches")
    x = patches[0]
    dt, dev, shape = x.dtype, x.get_device(), x.shape
    if len(shape) < 2 or dev < 0:
        raise ValueError("patches are CUDA tensors [N, *spatial, C]")
    N, C = shape[0], shape[-1]
    NC = N * C or 1
    for ts in likes:
        if len(ts) != P:
            raise ValueError("one output, and one gradient, per patch")
    spatial, ptrs, shapes = [], [], []
    for x in patches:
        s = x.shape
        if x.dtype is not dt or x.get_device() != dev or len(s) < 2 or s[0] != N or s[-1] != C:
            raise ValueError("the patches' dtypes, devices, samples or channels differ")
        if not x.is_contiguous():
            raise ValueError("the patches must be contiguous")
        spatial.append(x.numel() // NC)
        ptrs.append(x.data_ptr())
        shapes.append(s)
    for ts in likes:
        for t, s in zip(ts, shapes):
            if t.shape != s or t.dtype is not dt or t.get_device() != dev or not t.is_contiguous():
                raise ValueError("outputs and gradients must be contiguous and match their patches")
            ptrs.append(t.data_ptr())
    table = array("q", spatial + ptrs)
    at = table.buffer_info()[0]
    return (N, C, _DTYPES[dt] if dt in _DTYPES else _dtype_code(x), dev, P, table,
            range(at, at + 8 * len(table), 8 * P), None if gamma is None else _vec(gamma, C, dt, dev, "gamma"),
            None if beta is None else _vec(beta, C, dt, dev, "beta"))


def _cl_records(partials: torch.Tensor, R: int, N: int, G: int, device: int) -> int:
    if partials.get_device() != device or not partials.is_contiguous() or \
            partials.numel() * partials.element_size() != R * N * G * TB_GN_PARTS * 16:
        raise ValueError("partials must hold R*N*G*TB_GN_PARTS 16-byte records on the patches' device")
    return partials.data_ptr()


def _cl_workspace(workspace: torch.Tensor, device: int) -> Tuple[int, int]:
    if workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous, on the patches' device")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def gn_workspace_cl(N: int, G: int, device=None) -> torch.Tensor:
    """The device workspace of tb_patch_gn_grad_apply_cl for these sizes; it
    may serve any number of calls in turn on one stream."""
    n = int(_lib.tb_patch_gn_workspace_cl(N, G))
    if n < 0:
        raise ValueError("no group norm of %d samples in %d groups" % (N, G))
    return torch.empty(n, dtype=torch.uint8, device=device or torch.device("cuda"))


def tb_patch_gn_stats_cl(patches: Sequence[torch.Tensor], G: int, partials: torch.Tensor, stream=None) -> torch.Tensor:
    """``tb_patch_gn_stats`` of channels-last patches [N, *spatial_p, C]: the
    same records, in the same places."""
    N, C, dt, dev, P, table, (sp, xs), _, _ = _cl_args(patches, None, None)
    _check(_lib.tb_patch_gn_stats_cl(xs, P, dt, N, C, sp, G, _cl_records(partials, P, N, G, dev),
                                     _stream_of(stream, dev)), "tb_patch_gn_stats_cl")
    return partials


def tb_patch_gn_apply_cl(patches: Sequence[torch.Tensor], outs: Sequence[torch.Tensor], G: int, partials: torch.Tensor,
                         R: int, gamma: Optional[torch.Tensor], beta: Optional[torch.Tensor], eps: float,
                         silu: bool = True, stream=None) -> Sequence[torch.Tensor]:
    """Normalise (+ SiLU) channels-last patches [N, *spatial_p, C] into
    ``outs`` (``outs[p]`` may be ``patches[p]``) with the statistics pooled
    over the ``R`` record sets in ``partials``."""
    N, C, dt, dev, P, table, (sp, xs, os_), ga, be = _cl_args(patches, gamma, beta, outs)
    _check(_lib.tb_patch_gn_apply_cl(xs, os_, P, dt, N, C, sp, G,
                                     _cl_records(partials, R, N, G, dev), R, ga, be, eps, 1 if silu else 0,
                                     _stream_of(stream, dev)), "tb_patch_gn_apply_cl")
    return outs


def patch_group_norm_cl(patches: Sequence[torch.Tensor], G: int, gamma: Optional[torch.Tensor],
                        beta: Optional[torch.Tensor], eps: float, silu: bool = True,
                        outs: Optional[Sequence[torch.Tensor]] = None, partials: Optional[torch.Tensor] = None,
                        stream=None) -> Sequence[torch.Tensor]:
    """Both steps for channels-last patches [N, *spatial_p, C]: GroupNorm (+
    SiLU) of the whole tensor over its patches.  ``partials`` receives records
    that describe the patches together.  Outputs that are not given are made."""
    if outs is None or partials is None:
        if len(patches) == 0 or patches[0].dim() < 2:
            raise ValueError("at least one patch, [N, *spatial, C]")
        outs, partials = _on_stream(lambda: (
            [torch.empty(x.shape, dtype=x.dtype, device=x.device) for x in patches] if outs is None else outs,
            new_partials(len(patches), patches[0].shape[0], G, patches[0].device) if partials is None else partials),
            stream)
    N, C, dt, dev, P, table, (sp, xs, os_), ga, be = _cl_args(patches, gamma, beta, outs)
    status = _lib.tb_patch_group_norm_cl(xs, os_, P, dt, N, C, sp, G, _cl_records(partials, P, N, G, dev), ga, be, eps,
                                         1 if silu else 0, _stream_of(stream, dev))
    if status:
        raise TileBlendError(status, "tb_patch_group_norm_cl")
    return outs


def tb_patch_gn_grad_stats_cl(grads: Sequence[torch.Tensor], patches: Sequence[torch.Tensor], G: int,
                              partials: torch.Tensor, R: int, gamma: Optional[torch.Tensor],
                              beta: Optional[torch.Tensor], eps: float, grad_partials: torch.Tensor,
                              silu: bool = True, stream=None) -> torch.Tensor:
    """``tb_patch_gn_grad_stats`` of channels-last patches and gradients: the
    same records, in the same places."""
    N, C, dt, dev, P, table, (sp, xs, ds), ga, be = _cl_args(patches, gamma, beta, grads)
    _check(_lib.tb_patch_gn_grad_stats_cl(xs, ds, P, dt, N, C, sp, G,
                                          _cl_records(partials, R, N, G, dev), R, ga, be, eps, 1 if silu else 0,
                                          _grad_partials(grad_partials, P, N, C, dev), _stream_of(stream, dev)),
           "tb_patch_gn_grad_stats_cl")
    return grad_partials


def tb_patch_gn_grad_apply_cl(grads: Sequence[torch.Tensor], patches: Sequence[torch.Tensor],
                              dxs: Sequence[torch.Tensor], G: int, partials: torch.Tensor,
                              grad_partials: torch.Tensor, R: int, gamma: Optional[torch.Tensor],
                              beta: Optional[torch.Tensor], eps: float, workspace: torch.Tensor,
                              dgamma: Optional[torch.Tensor] = None, dbeta: Optional[torch.Tensor] = None,
                              silu: bool = True, stream=None) -> Sequence[torch.Tensor]:
    """The gradients of channels-last patches into ``dxs`` (``dxs[p]`` may be
    ``grads[p]`` or ``patches[p]``), and of the weights into ``dgamma`` /
    ``dbeta``, from the ``R`` record sets of both passes.  ``workspace`` comes
    from ``gn_workspace_cl``."""
    N, C, dt, dev, P, table, (sp, xs, ds, os_), ga, be = _cl_args(patches, gamma, beta, grads, dxs)
    gp, bp = _vec(dgamma, C, patches[0].dtype, dev, "dgamma"), _vec(dbeta, C, patches[0].dtype, dev, "dbeta")
    _check(_lib.tb_patch_gn_grad_apply_cl(xs, ds, os_, P, dt, N, C, sp, G,
                                          _cl_records(partials, R, N, G, dev),
                                          _grad_partials(grad_partials, R, N, C, dev), R, ga, be, eps,
                                          1 if silu else 0, gp, bp, *_cl_workspace(workspace, dev),
                                          _stream_of(stream, dev)), "tb_patch_gn_grad_apply_cl")
    return dxs


def patch_group_norm_backward_cl(grads: Sequence[torch.Tensor], patches: Sequence[torch.Tensor], G: int,
                                 partials: torch.Tensor, gamma: Optional[torch.Tensor], beta: Optional[torch.Tensor],
                                 eps: float, silu: bool = True, dxs: Optional[Sequence[torch.Tensor]] = None,
                                 dgamma: Optional[torch.Tensor] = None, dbeta: Optional[torch.Tensor] = None,
                                 grad_partials: Optional[torch.Tensor] = None,
                                 workspace: Optional[torch.Tensor] = None, stream=None):
    """Both steps of the backward pass of ``patch_group_norm_cl``: ``(dxs,
    dgamma, dbeta)``.  ``partials`` are the forward pass's records of these
    patches; outputs and workspaces that are not given are made."""
    P = len(patches)
    if dxs is None or dgamma is None or dbeta is None or grad_partials is None or workspace is None:
        if P == 0 or patches[0].dim() < 2:
            raise ValueError("at least one patch, [N, *spatial, C]")
        N, C, dt, dev = patches[0].shape[0], patches[0].shape[-1], patches[0].dtype, patches[0].device

        def make():
            return ([torch.empty(x.shape, dtype=x.dtype, device=x.device) for x in patches] if dxs is None else dxs,
                    torch.empty(C, dtype=dt, device=dev) if dgamma is None else dgamma,
                    torch.empty(C, dtype=dt, device=dev) if dbeta is None else dbeta,
                    new_grad_partials(P, N, C, dev) if grad_partials is None else grad_partials,
                    gn_workspace_cl(N, G, dev) if workspace is None else workspace)
        dxs, dgamma, dbeta, grad_partials, workspace = _on_stream(make, stream)
    N, C, dt, dev, P, table, (sp, xs, ds, os_), ga, be = _cl_args(patches, gamma, beta, grads, dxs)
    wdt = patches[0].dtype
    status = _lib.tb_patch_group_norm_backward_cl(xs, ds, os_, P, dt, N, C, sp, G, _cl_records(partials, P, N, G, dev),
                                                  _grad_partials(grad_partials, P, N, C, dev), ga, be, eps,
                                                  1 if silu else 0, _vec(dgamma, C, wdt, dev, "dgamma"),
                                                  _vec(dbeta, C, wdt, dev, "dbeta"), *_cl_workspace(workspace, dev),
                                                  _stream_of(stream, dev))
    if status:
        raise TileBlendError(status, "tb_patch_group_norm_backward_cl")
    return dxs, dgamma, dbeta


# ---------------------------------------------------------------------------
# dropout
# ---------------------------------------------------------------------------

def tb_dropout(x: torch.Tensor, y: torch.Tensor, p: float, seed: int, offset: int = 0,
               residual: Optional[torch.Tensor] = None, state: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """Dropout of x, plus ``residual``, into ``y``; ``y`` may be ``x`` or
    ``residual``.  All are [..., cols] with any row stride.  The mask belongs
    to (seed, offset) and the element's number, so the same call on the
    gradient, without a residual, is the backward pass.  ``seed`` and
    ``offset`` are taken modulo 2^64; ``state``, a contiguous int64 tensor of
    two, is added to them when the kernel runs."""
    shape, dev, dt = x.shape, x.get_device(), x.dtype
    if dev < 0:
        raise ValueError("the rows must be CUDA tensors")
    if not shape:
        raise ValueError("rows of elements")
    cols, rp, r_ld = shape[-1], None, 0
    if residual is not None:
        rp, r_ld = residual.data_ptr(), _row_ld(residual, shape, dt, dev, "residual")
    status = _lib.tb_dropout(x.data_ptr(), cols if x.is_contiguous() else _row_ld(x, shape, dt, dev, "x"), rp, r_ld,
                             _DTYPES[dt] if dt in _DTYPES else _dtype_code(x), x.numel() // cols if cols else 0, cols, p,
                             int(seed) & 0xFFFFFFFFFFFFFFFF, int(offset) & 0xFFFFFFFFFFFFFFFF,
                             None if state is None else _vec(state, 2, torch.int64, dev, "state"), y.data_ptr(),
                             _row_ld(y, shape, dt, dev, "y"), _stream_of(stream, dev))
    if status:
        raise TileBlendError(status, "tb_dropout")
    return y


def dropout(x: torch.Tensor, p: float, seed: int, offset: int = 0, residual: Optional[torch.Tensor] = None,
            state: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """tb_dropout into a new tensor."""
    y = _on_stream(lambda: torch.empty(x.shape, dtype=x.dtype, device=x.device), stream)
    return tb_dropout(x, y, p, seed, offset, residual, state, stream)
