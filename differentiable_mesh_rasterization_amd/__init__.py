"""MI355X-native K-nearest-face mesh rasterizer (forward and backward).

A thin ctypes binding over libdmr.so, whose C ABI is declared in
include/dmr.h. The functions below only marshal torch tensors (device
memory) and the current HIP stream into that ABI: every step of the
computation runs in the library's HIP kernels. There is no CPU fallback: if
libdmr.so is missing, every call raises.

    rasterize_meshes_fwd / rasterize_meshes_bwd   the two C-ABI entry points
    rasterize_meshes_fwd_ex                       the forward with rasterizer settings
    dmr_blend_fwd / dmr_blend_bwd                 the second stage
    dmr_project_fwd / dmr_project_bwd             the upstream projection
    rasterize_points_fwd / rasterize_points_bwd   point clouds
    dmr_grouped_linear_fwd / _bwd                 linear layers, one weight per mesh (or other group)
    dmr_orthogonalize                             orthogonalised updates of their weights
    dmr_grouped_layer_norm_fwd / _bwd             layer norms, one scale and shift per mesh
    dmr_grouped_gated_linear_fwd / _bwd           gated layers, one pair of weights per mesh
    dmr_clip_norm                                 norms of gradients over many tensors, and clipping
    rasterize_meshes, project_meshes,
    rasterize_points, grouped_linear,
    grouped_layer_norm, grouped_gated_linear      autograd-aware conveniences
    orthogonalize, clip_grad_norm                 dmr_orthogonalize and dmr_clip_norm with their buffers allocated
"""

from __future__ import annotations

import ctypes
import os
import struct
from typing import List, Optional, Sequence, Tuple

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdmr.so")

DMR_MAX_K = 64
DMR_BWD_REUSE_FORWARD_WORKSPACE = 0x1
DMR_RASTER_PERSPECTIVE_CORRECT = 0x2
DMR_RASTER_CULL_BACKFACES = 0x4
DMR_RASTER_UNCLIPPED_BARY = 0x8
STATUS = {0: "DMR_SUCCESS", 1: "DMR_ERROR_INVALID_VALUE", 2: "DMR_ERROR_WORKSPACE_TOO_SMALL",
          3: "DMR_ERROR_HIP", 4: "DMR_ERROR_UNSUPPORTED"}
EXPORTED = [
    "rasterize_meshes_fwd", "rasterize_meshes_fwd_ex", "rasterize_meshes_bwd", "dmr_workspace_min_size", "dmr_workspace_size_hint",
    "dmr_workspace_stats", "dmr_status_string", "dmr_kernel_count",
    "dmr_kernel_name", "dmr_set_kernel_timing", "dmr_set_kernel_timing_mask", "dmr_kernel_timing",
    "dmr_reset_kernel_timing", "dmr_blend_fwd", "dmr_blend_bwd", "dmr_project_fwd", "dmr_project_bwd",
    "rasterize_points_fwd", "rasterize_points_bwd", "dmr_points_workspace_min_size", "dmr_points_workspace_size_hint",
    "rasterize_meshes_fwd_noalloc", "dmr_grouped_linear_fwd", "dmr_grouped_linear_bwd", "dmr_grouped_linear_workspace_size",
    "dmr_grouped_linear_plan", "dmr_orthogonalize", "dmr_orthogonalize_workspace_size", "dmr_orthogonalize_tile",
    "dmr_grouped_layer_norm_fwd", "dmr_grouped_layer_norm_bwd", "dmr_grouped_layer_norm_workspace_size",
    "dmr_clip_norm", "dmr_clip_norm_workspace_size", "dmr_grouped_gated_linear_fwd", "dmr_grouped_gated_linear_bwd",
    "dmr_grouped_gated_linear_workspace_size", "dmr_grouped_gated_linear_plan",
]
DMR_NOALLOC_SCRATCH_BYTES = 128 << 20
DMR_MAX_LINEAR_WIDTH = 1 << 20
DMR_MAX_ORTHOGONALIZE_STEPS = 64
DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}   # dmr_dtype
ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "sigmoid": 3}         # dmr_activation


class DmrError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {STATUS.get(status, status)} ({status_string(status)})")


class dmr_blend_params(ctypes.Structure):
    _fields_ = [("sigma", ctypes.c_float), ("gamma", ctypes.c_float), ("znear", ctypes.c_float),
                ("zfar", ctypes.c_float), ("eps", ctypes.c_float), ("background", ctypes.c_float * 3)]


class dmr_stats(ctypes.Structure):
    _fields_ = [("required_bytes", ctypes.c_int64), ("bin_entries", ctypes.c_int64),
                ("bin_capacity", ctypes.c_int64), ("bins", ctypes.c_int64),
                ("overflow_bins", ctypes.c_int64), ("live_faces", ctypes.c_int64),
                ("flags", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


class dmr_linear_plan(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int32) for f in ("y_columns", "y_rows", "grad_x_columns", "grad_x_rows", "grad_weight_side",
                                              "piece_rows", "together")]


class dmr_gated_plan(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int32) for f in ("columns", "rows", "one_kernel", "piece_rows")]


_lib = None


def lib(path: Optional[str] = None):
    """Loads libdmr.so (once) and declares the C signatures."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is not built; run `python -m differentiable_mesh_rasterization_amd.build`")
    L = ctypes.CDLL(p)
    P, I64, I32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    L.rasterize_meshes_fwd.restype = ctypes.c_int
    L.rasterize_meshes_fwd.argtypes = [P, I64, P, I64, P, I64, I32, I32, I32, ctypes.c_float,
                                       P, P, P, P, P, SZ, P]
    L.rasterize_meshes_fwd_ex.restype = ctypes.c_int
    L.rasterize_meshes_fwd_ex.argtypes = [P, I64, P, I64, P, I64, I32, I32, I32, ctypes.c_float,
                                          P, P, P, P, P, SZ, ctypes.c_uint32, P]
    L.rasterize_meshes_fwd_noalloc.restype = ctypes.c_int
    L.rasterize_meshes_fwd_noalloc.argtypes = [P, I64, P, I64, P, I64, I32, I32, I32, ctypes.c_float, P, P, P, P, P]
    L.rasterize_meshes_bwd.restype = ctypes.c_int
    L.rasterize_meshes_bwd.argtypes = [P, I64, P, I64, P, I64, I32, I32, I32, ctypes.c_float, P, P, P, P, P, P, SZ,
                                       ctypes.c_uint32, P]
    L.dmr_workspace_min_size.restype = SZ
    L.dmr_workspace_min_size.argtypes = [I64, I64, I32, I32]
    L.dmr_workspace_size_hint.restype = SZ
    L.dmr_workspace_size_hint.argtypes = [I64, I64, I32, I32, I32, ctypes.c_float]
    L.dmr_workspace_stats.restype = ctypes.c_int
    L.dmr_workspace_stats.argtypes = [P, ctypes.POINTER(dmr_stats), P]
    L.dmr_status_string.restype = ctypes.c_char_p
    L.dmr_status_string.argtypes = [ctypes.c_int]
    L.dmr_kernel_count.restype = I32
    L.dmr_kernel_count.argtypes = []
    L.dmr_kernel_name.restype = ctypes.c_char_p
    L.dmr_kernel_name.argtypes = [I32]
    L.dmr_set_kernel_timing.restype = ctypes.c_int
    L.dmr_set_kernel_timing.argtypes = [I32]
    L.dmr_set_kernel_timing_mask.restype = ctypes.c_int
    L.dmr_set_kernel_timing_mask.argtypes = [ctypes.c_uint32]
    L.dmr_kernel_timing.restype = ctypes.c_int
    L.dmr_kernel_timing.argtypes = [I32, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int64)]
    L.dmr_reset_kernel_timing.restype = ctypes.c_int
    L.dmr_reset_kernel_timing.argtypes = []
    BP = ctypes.POINTER(dmr_blend_params)
    L.dmr_blend_fwd.restype = ctypes.c_int
    L.dmr_blend_fwd.argtypes = [P, P, P, I64, I32, P, I64, BP, P, P]
    L.dmr_blend_bwd.restype = ctypes.c_int
    L.dmr_blend_bwd.argtypes = [P, P, P, I64, I32, P, I64, BP, P, P, P, P]
    L.dmr_project_fwd.restype = ctypes.c_int
    L.dmr_project_fwd.argtypes = [P, I64, P, I64, P, P, P]
    L.dmr_project_bwd.restype = ctypes.c_int
    L.dmr_project_bwd.argtypes = [P, I64, P, I64, P, P, P, P, P]
    L.rasterize_points_fwd.restype = ctypes.c_int
    L.rasterize_points_fwd.argtypes = [P, I64, P, I64, I32, I32, I32, ctypes.c_float, P, P, P, P, SZ, P]
    L.rasterize_points_bwd.restype = ctypes.c_int
    L.rasterize_points_bwd.argtypes = [P, I64, P, I64, I32, I32, I32, P, P, P, P, P]
    L.dmr_points_workspace_min_size.restype = SZ
    L.dmr_points_workspace_min_size.argtypes = [I64, I64, I32, I32]
    L.dmr_points_workspace_size_hint.restype = SZ
    L.dmr_points_workspace_size_hint.argtypes = [I64, I64, I32, I32, I32, ctypes.c_float]
    L.dmr_grouped_linear_fwd.restype = ctypes.c_int
    L.dmr_grouped_linear_fwd.argtypes = [P, I64, I32, P, I64, P, P, I32, ctypes.c_int, P, P]
    L.dmr_grouped_linear_bwd.restype = ctypes.c_int
    L.dmr_grouped_linear_bwd.argtypes = [P, I64, I32, P, I64, P, I32, ctypes.c_int, P, P, P, P, P, SZ, P]
    L.dmr_grouped_linear_workspace_size.restype = SZ
    L.dmr_grouped_linear_workspace_size.argtypes = [I64, I64, I32, I32, ctypes.c_int]
    L.dmr_grouped_linear_plan.restype = ctypes.c_int
    L.dmr_grouped_linear_plan.argtypes = [I64, I64, I32, I32, ctypes.c_int, I32, P]
    L.dmr_orthogonalize_tile.restype = I32
    L.dmr_orthogonalize_tile.argtypes = [I64, I32, I32]
    L.dmr_orthogonalize.restype = ctypes.c_int
    L.dmr_orthogonalize.argtypes = [P, I64, I32, I32, ctypes.c_int, I32, ctypes.c_float, P, P, SZ, P]
    L.dmr_orthogonalize_workspace_size.restype = SZ
    L.dmr_orthogonalize_workspace_size.argtypes = [I64, I32, I32, ctypes.c_int]
    F32, INT = ctypes.c_float, ctypes.c_int
    L.dmr_grouped_layer_norm_fwd.restype = INT
    L.dmr_grouped_layer_norm_fwd.argtypes = [P, I64, I32, P, I64, P, P, F32, INT, P, P]
    L.dmr_grouped_layer_norm_bwd.restype = INT
    L.dmr_grouped_layer_norm_bwd.argtypes = [P, I64, I32, P, I64, P, F32, INT, P, P, P, P, P, SZ, P]
    L.dmr_grouped_layer_norm_workspace_size.restype = SZ
    L.dmr_grouped_layer_norm_workspace_size.argtypes = [I64, I64, I32, INT]
    L.dmr_grouped_gated_linear_fwd.restype = INT
    L.dmr_grouped_gated_linear_fwd.argtypes = [P, I64, I32, P, I64, P, P, I32, INT, INT, P, P]
    L.dmr_grouped_gated_linear_bwd.restype = INT
    L.dmr_grouped_gated_linear_bwd.argtypes = [P, I64, I32, P, I64, P, P, I32, INT, INT, P, P, P, P, P, SZ, P]
    L.dmr_grouped_gated_linear_workspace_size.restype = SZ
    L.dmr_grouped_gated_linear_workspace_size.argtypes = [I64, I64, I32, I32, INT]
    L.dmr_grouped_gated_linear_plan.restype = INT
    L.dmr_grouped_gated_linear_plan.argtypes = [I64, I64, I32, I32, INT, I32, P]
    L.dmr_clip_norm.restype = INT
    L.dmr_clip_norm.argtypes = [P, I32, I64, F32, F32, P, P, SZ, P]
    L.dmr_clip_norm_workspace_size.restype = SZ
    L.dmr_clip_norm_workspace_size.argtypes = [P, I32, I64]
    if path is None:
        _lib = L
    return L


def status_string(status: int) -> str:
    return lib().dmr_status_string(int(status)).decode()


dmr_status_string = status_string


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(device: torch.device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _check(t: torch.Tensor, name: str, dtype, device, shape=None, optional=False):
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


# ----------------------------------------------------------------------------
# workspace sizes and statistics
# ----------------------------------------------------------------------------

def dmr_workspace_min_size(N: int, F: int, H: int, W: int) -> int:
    return int(lib().dmr_workspace_min_size(N, F, H, W))


def dmr_workspace_size_hint(N: int, F: int, H: int, W: int, K: int, blur_radius: float) -> int:
    return int(lib().dmr_workspace_size_hint(N, F, H, W, K, blur_radius))


def dmr_workspace_stats(workspace: torch.Tensor) -> dict:
    s = dmr_stats()
    rc = lib().dmr_workspace_stats(_ptr(workspace), ctypes.byref(s), _stream_handle(workspace.device))
    if rc != 0:
        raise DmrError("dmr_workspace_stats", rc)
    return {f: getattr(s, f) for f, _ in dmr_stats._fields_ if f != "reserved"}


# ----------------------------------------------------------------------------
# the two entry points
# ----------------------------------------------------------------------------

def rasterize_meshes_fwd(verts: torch.Tensor, faces: torch.Tensor, mesh_face_offsets: torch.Tensor,
                         H: int, W: int, K: int, blur_radius: float,
                         pix_to_face: torch.Tensor, zbuf: torch.Tensor, bary: torch.Tensor,
                         dists: torch.Tensor, workspace: torch.Tensor) -> None:
    """C-ABI forward call on preallocated device tensors (include/dmr.h)."""
    _forward(verts, faces, mesh_face_offsets, H, W, K, blur_radius, pix_to_face, zbuf, bary, dists, workspace,
             None)


def rasterize_meshes_fwd_ex(verts: torch.Tensor, faces: torch.Tensor, mesh_face_offsets: torch.Tensor,
                            H: int, W: int, K: int, blur_radius: float,
                            pix_to_face: torch.Tensor, zbuf: torch.Tensor, bary: torch.Tensor,
                            dists: torch.Tensor, workspace: torch.Tensor, flags: int) -> None:
    """C-ABI forward call with rasterizer settings (a mask of the
    DMR_RASTER_* bits; include/dmr.h)."""
    _forward(verts, faces, mesh_face_offsets, H, W, K, blur_radius, pix_to_face, zbuf, bary, dists, workspace,
             int(flags))


def rasterize_meshes_fwd_noalloc(verts: torch.Tensor, faces: torch.Tensor, mesh_face_offsets: torch.Tensor,
                                 H: int, W: int, K: int, blur_radius: float,
                                 pix_to_face: torch.Tensor, zbuf: torch.Tensor, bary: torch.Tensor,
                                 dists: torch.Tensor) -> None:
    """C-ABI forward call that allocates nothing: the library's per-device
    scratch array stands in for the workspace (include/dmr.h). Calls that
    overlap on one device race."""
    dev = verts.device
    N = mesh_face_offsets.shape[0] - 1
    _check(verts, "verts", torch.float32, dev)
    _check(faces, "faces", torch.int64, dev)
    _check(mesh_face_offsets, "mesh_face_offsets", torch.int64, dev)
    shape = (N, H, W, K)
    _check(pix_to_face, "pix_to_face", torch.int64, dev, shape)
    _check(zbuf, "zbuf", torch.float32, dev, shape)
    _check(bary, "bary", torch.float32, dev, shape + (3,))
    _check(dists, "dists", torch.float32, dev, shape)
    rc = lib().rasterize_meshes_fwd_noalloc(_ptr(verts), verts.shape[0], _ptr(faces), faces.shape[0],
                                            _ptr(mesh_face_offsets), N, H, W, K, float(blur_radius),
                                            _ptr(pix_to_face), _ptr(zbuf), _ptr(bary), _ptr(dists),
                                            _stream_handle(dev))
    if rc != 0:
        raise DmrError("rasterize_meshes_fwd_noalloc", rc)


def _forward(verts, faces, mesh_face_offsets, H, W, K, blur_radius, pix_to_face, zbuf, bary, dists, workspace,
             flags):
    dev = verts.device
    N = mesh_face_offsets.shape[0] - 1
    _check(verts, "verts", torch.float32, dev)
    _check(faces, "faces", torch.int64, dev)
    _check(mesh_face_offsets, "mesh_face_offsets", torch.int64, dev)
    shape = (N, H, W, K)
    _check(pix_to_face, "pix_to_face", torch.int64, dev, shape)
    _check(zbuf, "zbuf", torch.float32, dev, shape)
    _check(bary, "bary", torch.float32, dev, shape + (3,))
    _check(dists, "dists", torch.float32, dev, shape)
    _check(workspace, "workspace", torch.uint8, dev)
    args = (_ptr(verts), verts.shape[0], _ptr(faces), faces.shape[0], _ptr(mesh_face_offsets), N,
            H, W, K, float(blur_radius), _ptr(pix_to_face), _ptr(zbuf), _ptr(bary), _ptr(dists),
            _ptr(workspace), workspace.numel())
    if flags is None:
        rc = lib().rasterize_meshes_fwd(*args, _stream_handle(dev))
        if rc != 0:
            raise DmrError("rasterize_meshes_fwd", rc)
    else:
        rc = lib().rasterize_meshes_fwd_ex(*args, flags, _stream_handle(dev))
        if rc != 0:
            raise DmrError("rasterize_meshes_fwd_ex", rc)


def rasterize_meshes_bwd(verts: torch.Tensor, faces: torch.Tensor, mesh_face_offsets: torch.Tensor,
                         H: int, W: int, K: int, blur_radius: float, pix_to_face: torch.Tensor,
                         grad_zbuf: Optional[torch.Tensor], grad_bary: Optional[torch.Tensor],
                         grad_dists: Optional[torch.Tensor], grad_verts: torch.Tensor,
                         workspace: Optional[torch.Tensor] = None, reuse_forward_workspace: bool = False,
                         settings: int = 0) -> None:
    """C-ABI backward call on preallocated device tensors (include/dmr.h).

    With reuse_forward_workspace=True, `workspace` must be the forward call's
    workspace for these same inputs, unmodified since. `settings` are the
    DMR_RASTER_* bits the forward call was given."""
    dev = verts.device
    N = mesh_face_offsets.shape[0] - 1
    shape = (N, H, W, K)
    _check(verts, "verts", torch.float32, dev)
    _check(faces, "faces", torch.int64, dev)
    _check(mesh_face_offsets, "mesh_face_offsets", torch.int64, dev)
    _check(pix_to_face, "pix_to_face", torch.int64, dev, shape)
    _check(grad_zbuf, "grad_zbuf", torch.float32, dev, shape, optional=True)
    _check(grad_bary, "grad_bary", torch.float32, dev, shape + (3,), optional=True)
    _check(grad_dists, "grad_dists", torch.float32, dev, shape, optional=True)
    _check(grad_verts, "grad_verts", torch.float32, dev, tuple(verts.shape))
    _check(workspace, "workspace", torch.uint8, dev, optional=not reuse_forward_workspace)
    flags = (DMR_BWD_REUSE_FORWARD_WORKSPACE if reuse_forward_workspace else 0) | int(settings)
    rc = lib().rasterize_meshes_bwd(
        _ptr(verts), verts.shape[0], _ptr(faces), faces.shape[0], _ptr(mesh_face_offsets), N,
        H, W, K, float(blur_radius), _ptr(pix_to_face), _ptr(grad_zbuf), _ptr(grad_bary), _ptr(grad_dists),
        _ptr(grad_verts), _ptr(workspace), 0 if workspace is None else workspace.numel(), flags,
        _stream_handle(dev))
    if rc != 0:
        raise DmrError("rasterize_meshes_bwd", rc)


def blend_params(sigma: float = 1e-4, gamma: float = 1e-4, znear: float = 1.0, zfar: float = 100.0,
                 eps: float = 1e-10, background=(1.0, 1.0, 1.0)) -> dmr_blend_params:
    return dmr_blend_params(sigma, gamma, znear, zfar, eps, (ctypes.c_float * 3)(*background))


def _blend_inputs(pix_to_face, zbuf, dists, face_colors):
    dev = pix_to_face.device
    K = pix_to_face.shape[-1]
    _check(pix_to_face, "pix_to_face", torch.int64, dev)
    _check(zbuf, "zbuf", torch.float32, dev, tuple(pix_to_face.shape))
    _check(dists, "dists", torch.float32, dev, tuple(pix_to_face.shape))
    _check(face_colors, "face_colors", torch.float32, dev)
    if face_colors.dim() != 2 or face_colors.shape[1] != 3:
        raise ValueError("face_colors must be [F, 3]")
    return dev, pix_to_face.numel() // K, K


def dmr_blend_fwd(pix_to_face: torch.Tensor, zbuf: torch.Tensor, dists: torch.Tensor, face_colors: torch.Tensor,
                  params: dmr_blend_params, rgba: torch.Tensor) -> None:
    """C-ABI second-stage blend on preallocated device tensors (include/dmr.h):
    rgba [..., 4] from the forward pass's [..., K] outputs."""
    dev, P, K = _blend_inputs(pix_to_face, zbuf, dists, face_colors)
    _check(rgba, "rgba", torch.float32, dev, tuple(pix_to_face.shape[:-1]) + (4,))
    rc = lib().dmr_blend_fwd(_ptr(pix_to_face), _ptr(zbuf), _ptr(dists), P, K, _ptr(face_colors),
                             face_colors.shape[0], ctypes.byref(params), _ptr(rgba), _stream_handle(dev))
    if rc != 0:
        raise DmrError("dmr_blend_fwd", rc)


def dmr_blend_bwd(pix_to_face: torch.Tensor, zbuf: torch.Tensor, dists: torch.Tensor, face_colors: torch.Tensor,
                  params: dmr_blend_params, grad_rgba: torch.Tensor, grad_zbuf: torch.Tensor,
                  grad_dists: torch.Tensor) -> None:
    """C-ABI backward of the blend: grad_zbuf, grad_dists [..., K] from grad_rgba [..., 4]."""
    dev, P, K = _blend_inputs(pix_to_face, zbuf, dists, face_colors)
    _check(grad_rgba, "grad_rgba", torch.float32, dev, tuple(pix_to_face.shape[:-1]) + (4,))
    _check(grad_zbuf, "grad_zbuf", torch.float32, dev, tuple(pix_to_face.shape))
    _check(grad_dists, "grad_dists", torch.float32, dev, tuple(pix_to_face.shape))
    rc = lib().dmr_blend_bwd(_ptr(pix_to_face), _ptr(zbuf), _ptr(dists), P, K, _ptr(face_colors),
                             face_colors.shape[0], ctypes.byref(params), _ptr(grad_rgba), _ptr(grad_zbuf),
                             _ptr(grad_dists), _stream_handle(dev))
    if rc != 0:
        raise DmrError("dmr_blend_bwd", rc)


def _project_inputs(verts_world, mesh_vert_offsets, cameras):
    dev = verts_world.device
    _check(verts_world, "verts_world", torch.float32, dev)
    if verts_world.dim() != 2 or verts_world.shape[1] != 3:
        raise ValueError("verts_world must be [V, 3]")
    _check(mesh_vert_offsets, "mesh_vert_offsets", torch.int64, dev)
    N = mesh_vert_offsets.shape[0] - 1
    _check(cameras, "cameras", torch.float32, dev, (N, 4, 4))
    return dev, verts_world.shape[0], N


def dmr_project_fwd(verts_world: torch.Tensor, mesh_vert_offsets: torch.Tensor, cameras: torch.Tensor,
                    verts_ndc: torch.Tensor) -> None:
    """C-ABI projection on preallocated device tensors (include/dmr.h)."""
    dev, V, N = _project_inputs(verts_world, mesh_vert_offsets, cameras)
    _check(verts_ndc, "verts_ndc", torch.float32, dev, (V, 3))
    rc = lib().dmr_project_fwd(_ptr(verts_world), V, _ptr(mesh_vert_offsets), N, _ptr(cameras), _ptr(verts_ndc),
                               _stream_handle(dev))
    if rc != 0:
        raise DmrError("dmr_project_fwd", rc)


def dmr_project_bwd(verts_world: torch.Tensor, mesh_vert_offsets: torch.Tensor, cameras: torch.Tensor,
                    grad_verts_ndc: torch.Tensor, grad_verts_world: torch.Tensor,
                    grad_cameras: Optional[torch.Tensor] = None) -> None:
    """C-ABI backward of the projection (grad_cameras optional)."""
    dev, V, N = _project_inputs(verts_world, mesh_vert_offsets, cameras)
    _check(grad_verts_ndc, "grad_verts_ndc", torch.float32, dev, (V, 3))
    _check(grad_verts_world, "grad_verts_world", torch.float32, dev, (V, 3))
    _check(grad_cameras, "grad_cameras", torch.float32, dev, (N, 4, 4), optional=True)
    rc = lib().dmr_project_bwd(_ptr(verts_world), V, _ptr(mesh_vert_offsets), N, _ptr(cameras),
                               _ptr(grad_verts_ndc), _ptr(grad_verts_world), _ptr(grad_cameras),
                               _stream_handle(dev))
    if rc != 0:
        raise DmrError("dmr_project_bwd", rc)


def dmr_points_workspace_min_size(N: int, P: int, H: int, W: int) -> int:
    return int(lib().dmr_points_workspace_min_size(N, P, H, W))


def dmr_points_workspace_size_hint(N: int, P: int, H: int, W: int, K: int, radius: float) -> int:
    return int(lib().dmr_points_workspace_size_hint(N, P, H, W, K, radius))


def rasterize_points_fwd(points: torch.Tensor, cloud_offsets: torch.Tensor, H: int, W: int, K: int, radius: float,
                         idx: torch.Tensor, zbuf: torch.Tensor, dists: torch.Tensor, workspace: torch.Tensor) -> None:
    """C-ABI point rasterization on preallocated device tensors (include/dmr.h)."""
    dev = points.device
    N = cloud_offsets.shape[0] - 1
    _check(points, "points", torch.float32, dev)
    _check(cloud_offsets, "cloud_offsets", torch.int64, dev)
    shape = (N, H, W, K)
    _check(idx, "idx", torch.int64, dev, shape)
    _check(zbuf, "zbuf", torch.float32, dev, shape)
    _check(dists, "dists", torch.float32, dev, shape)
    _check(workspace, "workspace", torch.uint8, dev)
    rc = lib().rasterize_points_fwd(_ptr(points), points.shape[0], _ptr(cloud_offsets), N, H, W, K, float(radius),
                                    _ptr(idx), _ptr(zbuf), _ptr(dists), _ptr(workspace), workspace.numel(),
                                    _stream_handle(dev))
    if rc != 0:
        raise DmrError("rasterize_points_fwd", rc)


def rasterize_points_bwd(points: torch.Tensor, cloud_offsets: torch.Tensor, H: int, W: int, K: int,
                         idx: torch.Tensor, grad_zbuf: Optional[torch.Tensor], grad_dists: Optional[torch.Tensor],
                         grad_points: torch.Tensor) -> None:
    """C-ABI backward of the point rasterization (include/dmr.h)."""
    dev = points.device
    N = cloud_offsets.shape[0] - 1
    shape = (N, H, W, K)
    _check(points, "points", torch.float32, dev)
    _check(cloud_offsets, "cloud_offsets", torch.int64, dev)
    _check(idx, "idx", torch.int64, dev, shape)
    _check(grad_zbuf, "grad_zbuf", torch.float32, dev, shape, optional=True)
    _check(grad_dists, "grad_dists", torch.float32, dev, shape, optional=True)
    _check(grad_points, "grad_points", torch.float32, dev, tuple(points.shape))
    rc = lib().rasterize_points_bwd(_ptr(points), points.shape[0], _ptr(cloud_offsets), N, H, W, K, _ptr(idx),
                                    _ptr(grad_zbuf), _ptr(grad_dists), _ptr(grad_points), _stream_handle(dev))
    if rc != 0:
        raise DmrError("rasterize_points_bwd", rc)


def _dtype(t: torch.Tensor, name: str) -> int:
    code = DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    return code


def _alike(t: torch.Tensor, dtype, device, shape) -> bool:
    # what _check asks, without its messages (these calls can be short)
    return t.dtype is dtype and t.device == device and t.shape == shape and t.is_contiguous()


def _grouped_inputs(x, row_offsets, weight):
    dev, dt = x.device, x.dtype
    if x.dim() != 2 or weight.dim() != 3:
        raise ValueError("x must be [R, in_features] and weight [N, out_features, in_features]")
    R, cin = x.shape
    N, cout, _ = weight.shape
    if not (x.is_contiguous() and _alike(weight, dt, dev, (N, cout, cin)) and _alike(row_offsets, torch.int64, dev, (N + 1,))):
        _check(x, "x", dt, dev)
        _check(row_offsets, "row_offsets", torch.int64, dev, (N + 1,))
        _check(weight, "weight", dt, dev, (N, cout, cin))
    return dev, dt, R, cin, N, cout, _dtype(x, "x")


def _address(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _raw_stream(device: torch.device) -> int:
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a GPU, got {device}")
    return torch._C._cuda_getCurrentRawStream(device.index)


def dmr_grouped_linear_fwd(x: torch.Tensor, row_offsets: torch.Tensor, weight: torch.Tensor,
                           bias: Optional[torch.Tensor], y: torch.Tensor) -> None:
    """C-ABI layer with one weight per group of rows, on preallocated device
    tensors (include/dmr.h): y [R, out] from x [R, in], row_offsets [N + 1]
    int64, weight [N, out, in] and bias [N, out] or None."""
    dev, dt, R, cin, N, cout, code = _grouped_inputs(x, row_offsets, weight)
    if not (_alike(y, dt, dev, (R, cout)) and (bias is None or _alike(bias, dt, dev, (N, cout)))):
        _check(bias, "bias", dt, dev, (N, cout), optional=True)
        _check(y, "y", dt, dev, (R, cout))
    _launch_grouped(x, R, cin, row_offsets, N, weight, bias, cout, code, y, dev)


def _launch_grouped(x, R, cin, row_offsets, N, weight, bias, cout, code, y, dev):
    rc = lib().dmr_grouped_linear_fwd(x.data_ptr(), R, cin, row_offsets.data_ptr(), N, weight.data_ptr(), _address(bias),
                                      cout, code, y.data_ptr(), _raw_stream(dev))
    if rc != 0:
        raise DmrError("dmr_grouped_linear_fwd", rc)


def dmr_grouped_linear_workspace_size(R: int, N: int, in_features: int, out_features: int, dtype: torch.dtype) -> int:
    return int(lib().dmr_grouped_linear_workspace_size(R, N, in_features, out_features, DTYPES.get(dtype, -1)))


def dmr_grouped_linear_bwd(x: torch.Tensor, row_offsets: torch.Tensor, weight: torch.Tensor, grad_y: torch.Tensor,
                           grad_x: Optional[torch.Tensor], grad_weight: Optional[torch.Tensor],
                           grad_bias: Optional[torch.Tensor], workspace: Optional[torch.Tensor] = None) -> None:
    """C-ABI backward of the layer (include/dmr.h); each of the three
    gradients may be None. grad_weight and grad_bias need a workspace of
    dmr_grouped_linear_workspace_size() bytes."""
    dev, dt, R, cin, N, cout, code = _grouped_inputs(x, row_offsets, weight)
    sums = grad_weight is not None or grad_bias is not None
    if not (_alike(grad_y, dt, dev, (R, cout)) and (grad_x is None or _alike(grad_x, dt, dev, (R, cin)))
            and (grad_weight is None or _alike(grad_weight, dt, dev, (N, cout, cin)))
            and (grad_bias is None or _alike(grad_bias, dt, dev, (N, cout)))
            and (workspace is not None or not sums)):
        _check(grad_y, "grad_y", dt, dev, (R, cout))
        _check(grad_x, "grad_x", dt, dev, (R, cin), optional=True)
        _check(grad_weight, "grad_weight", dt, dev, (N, cout, cin), optional=True)
        _check(grad_bias, "grad_bias", dt, dev, (N, cout), optional=True)
        _check(workspace, "workspace", torch.uint8, dev, optional=not sums)
    if workspace is not None:
        _check(workspace, "workspace", torch.uint8, dev)
    rc = lib().dmr_grouped_linear_bwd(x.data_ptr(), R, cin, row_offsets.data_ptr(), N, weight.data_ptr(), cout, code,
                                      grad_y.data_ptr(), _address(grad_x), _address(grad_weight), _address(grad_bias),
                                      _address(workspace), 0 if workspace is None else workspace.numel(), _raw_stream(dev))
    if rc != 0:
        raise DmrError("dmr_grouped_linear_bwd", rc)


def dmr_grouped_linear_plan(R: int, N: int, in_features: int, out_features: int, dtype: torch.dtype,
                            aligned: bool = True) -> dict:
    """What calls of these sizes are computed by (include/dmr.h)."""
    plan = dmr_linear_plan()
    rc = lib().dmr_grouped_linear_plan(R, N, in_features, out_features, DTYPES.get(dtype, -1), int(aligned),
                                       ctypes.byref(plan))
    if rc != 0:
        raise DmrError("dmr_grouped_linear_plan", rc)
    return {f: getattr(plan, f) for f, _ in dmr_linear_plan._fields_}


def dmr_orthogonalize_tile(B: int, m: int, n: int) -> int:
    return int(lib().dmr_orthogonalize_tile(B, m, n))


def dmr_orthogonalize_workspace_size(B: int, m: int, n: int, dtype: torch.dtype) -> int:
    return int(lib().dmr_orthogonalize_workspace_size(B, m, n, DTYPES.get(dtype, -1)))


def dmr_orthogonalize(update: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor, steps: int = 5,
                      eps: float = 1e-7) -> None:
    """C-ABI orthogonalised update on preallocated device tensors
    (include/dmr.h): update and out [B, m, n]."""
    dev, dt = update.device, update.dtype
    if update.dim() != 3:
        raise ValueError("update must be [B, m, n]")
    B, m, n = update.shape
    _check(update, "update", dt, dev)
    _check(out, "out", dt, dev, (B, m, n))
    _check(workspace, "workspace", torch.uint8, dev)
    rc = lib().dmr_orthogonalize(update.data_ptr(), B, m, n, _dtype(update, "update"), int(steps), float(eps), out.data_ptr(),
                                 workspace.data_ptr(), workspace.numel(), _raw_stream(dev))
    if rc != 0:
        raise DmrError("dmr_orthogonalize", rc)


def _launch(fn, dev, *args) -> None:
    """Calls the library's `fn` on the current stream of `dev`, with that device current."""
    stream = _raw_stream(dev)
    if torch._C._cuda_getDevice() == dev.index:
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, stream)
    if rc != 0:
        raise DmrError(fn.__name__, rc)


def _layer_norm_inputs(x, row_offsets, weight):
    dev, dt = x.device, x.dtype
    if x.dim() != 2 or row_offsets.dim() != 1 or row_offsets.shape[0] < 1:
        raise ValueError("x must be [R, features] and row_offsets [N + 1]")
    R, C = x.shape
    N = row_offsets.shape[0] - 1
    if not (x.is_contiguous() and _alike(row_offsets, torch.int64, dev, (N + 1,))
            and (weight is None or _alike(weight, dt, dev, (N, C)))):
        _check(x, "x", dt, dev)
        _check(row_offsets, "row_offsets", torch.int64, dev, (N + 1,))
        _check(weight, "weight", dt, dev, (N, C), optional=True)
    return dev, dt, R, C, N, _dtype(x, "x")


def dmr_grouped_layer_norm_fwd(x: torch.Tensor, row_offsets: torch.Tensor, weight: Optional[torch.Tensor],
                               bias: Optional[torch.Tensor], y: torch.Tensor, eps: float = 1e-5) -> None:
    """C-ABI layer norm with one scale and shift per group of rows, on
    preallocated device tensors (include/dmr.h): y [R, C] from x [R, C],
    row_offsets [N + 1] int64, weight and bias [N, C] or None."""
    dev, dt, R, C, N, code = _layer_norm_inputs(x, row_offsets, weight)
    if not (_alike(y, dt, dev, (R, C)) and (bias is None or _alike(bias, dt, dev, (N, C)))):
        _check(bias, "bias", dt, dev, (N, C), optional=True)
        _check(y, "y", dt, dev, (R, C))
    _launch(lib().dmr_grouped_layer_norm_fwd, dev, x.data_ptr(), R, C, row_offsets.data_ptr(), N, _address(weight),
            _address(bias), float(eps), code, y.data_ptr())


def dmr_grouped_layer_norm_workspace_size(R: int, N: int, features: int, dtype: torch.dtype) -> int:
    return int(lib().dmr_grouped_layer_norm_workspace_size(R, N, features, DTYPES.get(dtype, -1)))


def dmr_grouped_layer_norm_bwd(x: torch.Tensor, row_offsets: torch.Tensor, weight: Optional[torch.Tensor],
                               grad_y: torch.Tensor, grad_x: Optional[torch.Tensor],
                               grad_weight: Optional[torch.Tensor], grad_bias: Optional[torch.Tensor],
                               workspace: Optional[torch.Tensor] = None, eps: float = 1e-5) -> None:
    """C-ABI backward of the layer norm (include/dmr.h); each of the three
    gradients may be None. grad_weight and grad_bias need a workspace of
    dmr_grouped_layer_norm_workspace_size() bytes."""
    dev, dt, R, C, N, code = _layer_norm_inputs(x, row_offsets, weight)
    sums = grad_weight is not None or grad_bias is not None
    if not (_alike(grad_y, dt, dev, (R, C)) and (grad_x is None or _alike(grad_x, dt, dev, (R, C)))
            and (grad_weight is None or _alike(grad_weight, dt, dev, (N, C)))
            and (grad_bias is None or _alike(grad_bias, dt, dev, (N, C)))):
        _check(grad_y, "grad_y", dt, dev, (R, C))
        _check(grad_x, "grad_x", dt, dev, (R, C), optional=True)
        _check(grad_weight, "grad_weight", dt, dev, (N, C), optional=True)
        _check(grad_bias, "grad_bias", dt, dev, (N, C), optional=True)
    _check(workspace, "workspace", torch.uint8, dev, optional=not sums)
    _launch(lib().dmr_grouped_layer_norm_bwd, dev, x.data_ptr(), R, C, row_offsets.data_ptr(), N, _address(weight), float(eps),
            code, grad_y.data_ptr(), _address(grad_x), _address(grad_weight), _address(grad_bias), _address(workspace),
            0 if workspace is None else workspace.numel())


def _gated_inputs(x, row_offsets, weight, bias, activation):
    dev, dt = x.device, x.dtype
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, got {activation!r}")
    if x.dim() != 2 or weight.dim() != 4:
        raise ValueError("x must be [R, in_features] and weight [N, 2, out_features, in_features]")
    R, C = x.shape
    N, _, F, _ = weight.shape
    if not (x.is_contiguous() and _alike(weight, dt, dev, (N, 2, F, C)) and _alike(row_offsets, torch.int64, dev, (N + 1,))
            and (bias is None or _alike(bias, dt, dev, (N, 2, F)))):
        _check(x, "x", dt, dev)
        _check(row_offsets, "row_offsets", torch.int64, dev, (N + 1,))
        _check(weight, "weight", dt, dev, (N, 2, F, C))
        _check(bias, "bias", dt, dev, (N, 2, F), optional=True)
    return dev, dt, R, C, N, F, act, _dtype(x, "x")


def dmr_grouped_gated_linear_fwd(x: torch.Tensor, row_offsets: torch.Tensor, weight: torch.Tensor,
                                 bias: Optional[torch.Tensor], y: torch.Tensor, activation: str = "silu") -> None:
    """C-ABI gated layer with one pair of weights per group of rows, on
    preallocated device tensors (include/dmr.h): y [R, out] from x [R, in],
    row_offsets [N + 1] int64, weight [N, 2, out, in] and bias [N, 2, out] or
    None; activation one of ACTIVATIONS."""
    dev, dt, R, C, N, F, act, code = _gated_inputs(x, row_offsets, weight, bias, activation)
    if not _alike(y, dt, dev, (R, F)):
        _check(y, "y", dt, dev, (R, F))
    _launch(lib().dmr_grouped_gated_linear_fwd, dev, x.data_ptr(), R, C, row_offsets.data_ptr(), N, weight.data_ptr(),
            _address(bias), F, act, code, y.data_ptr())


def dmr_grouped_gated_linear_workspace_size(R: int, N: int, in_features: int, out_features: int, dtype: torch.dtype) -> int:
    return int(lib().dmr_grouped_gated_linear_workspace_size(R, N, in_features, out_features, DTYPES.get(dtype, -1)))


def dmr_grouped_gated_linear_bwd(x: torch.Tensor, row_offsets: torch.Tensor, weight: torch.Tensor,
                                 bias: Optional[torch.Tensor], grad_y: torch.Tensor, grad_x: Optional[torch.Tensor],
                                 grad_weight: Optional[torch.Tensor], grad_bias: Optional[torch.Tensor],
                                 workspace: torch.Tensor, activation: str = "silu") -> None:
    """C-ABI backward of the gated layer (include/dmr.h); each of the three
    gradients may be None. workspace of
    dmr_grouped_gated_linear_workspace_size() bytes."""
    dev, dt, R, C, N, F, act, code = _gated_inputs(x, row_offsets, weight, bias, activation)
    if not (_alike(grad_y, dt, dev, (R, F)) and (grad_x is None or _alike(grad_x, dt, dev, (R, C)))
            and (grad_weight is None or _alike(grad_weight, dt, dev, (N, 2, F, C)))
            and (grad_bias is None or _alike(grad_bias, dt, dev, (N, 2, F)))):
        _check(grad_y, "grad_y", dt, dev, (R, F))
        _check(grad_x, "grad_x", dt, dev, (R, C), optional=True)
        _check(grad_weight, "grad_weight", dt, dev, (N, 2, F, C), optional=True)
        _check(grad_bias, "grad_bias", dt, dev, (N, 2, F), optional=True)
    _check(workspace, "workspace", torch.uint8, dev)
    _launch(lib().dmr_grouped_gated_linear_bwd, dev, x.data_ptr(), R, C, row_offsets.data_ptr(), N, weight.data_ptr(),
            _address(bias), F, act, code, grad_y.data_ptr(), _address(grad_x), _address(grad_weight), _address(grad_bias),
            workspace.data_ptr(), workspace.numel())


def dmr_grouped_gated_linear_plan(R: int, N: int, in_features: int, out_features: int, dtype: torch.dtype,
                                  aligned: bool = True) -> dict:
    """What calls of these sizes are computed by (include/dmr.h)."""
    plan = dmr_gated_plan()
    rc = lib().dmr_grouped_gated_linear_plan(R, N, in_features, out_features, DTYPES.get(dtype, -1), int(aligned),
                                             ctypes.byref(plan))
    if rc != 0:
        raise DmrError("dmr_grouped_gated_linear_plan", rc)
    return {f: getattr(plan, f) for f, _ in dmr_gated_plan._fields_}


_tensor_address, _tensor_values, _tensor_contiguous, _tensor_device = (
    torch.Tensor.data_ptr, torch.Tensor.numel, torch.Tensor.is_contiguous, torch.Tensor.get_device)


def _spans(tensors, outs, groups, alike=False) -> Tuple[torch.device, bytes]:
    """The device of `tensors` and the library's table of them. alike: outs
    were made like tensors."""
    n = len(tensors)
    if n == 0:
        raise ValueError("there must be a tensor")
    # lists at a time: these calls can be short, and the tensors many
    dev, values, codes = tensors[0].device, list(map(_tensor_values, tensors)), [DTYPES.get(t.dtype) for t in tensors]
    if None in codes or not all(map(_tensor_contiguous, tensors)) or len(set(map(_tensor_device, tensors))) > 1:
        for t in tensors:
            _dtype(t, "tensors")
            _check(t, "tensors", t.dtype, dev)
    if groups != 1:
        if groups < 0 or (groups > 0 and any(v % groups for v in values)):
            raise ValueError(f"tensors of {values} values cannot be shared by {groups} groups")
        values = [v // groups for v in values] if groups else [0] * n
    if not alike:
        for t, o in zip(tensors, outs):
            if o is not t and not _alike(o, t.dtype, dev, t.shape):
                _check(o, "outs", t.dtype, dev, tuple(t.shape))
    table = [0] * (5 * n)
    table[0::5] = map(_tensor_address, tensors)
    table[1::5] = map(_tensor_address, outs)
    table[2::5] = values
    table[3::5] = codes
    return dev, struct.pack("QQqii" * n, *table)


def dmr_clip_norm_workspace_size(tensors: Sequence[torch.Tensor], groups: int = 1) -> int:
    return int(lib().dmr_clip_norm_workspace_size(_spans(tensors, tensors, groups)[1], len(tensors), groups))


def dmr_clip_norm(tensors: Sequence[torch.Tensor], outs: Sequence[torch.Tensor], norms: torch.Tensor,
                  workspace: Optional[torch.Tensor], max_norm: float, groups: int = 1, eps: float = 1e-6) -> None:
    """C-ABI norms and clipping on preallocated device tensors
    (include/dmr.h): outs may be tensors themselves; norms [groups] float32;
    workspace of dmr_clip_norm_workspace_size() bytes."""
    if len(outs) != len(tensors):
        raise ValueError(f"{len(tensors)} tensors, but {len(outs)} outs")
    dev, table = _spans(tensors, outs, groups)
    _check_overlap(tensors, outs)
    _check(norms, "norms", torch.float32, dev, (groups,))
    _check(workspace, "workspace", torch.uint8, dev, optional=True)
    _launch(lib().dmr_clip_norm, dev, table, len(tensors), groups, float(max_norm), float(eps), norms.data_ptr(),
            _address(workspace), 0 if workspace is None else workspace.numel())


def _check_overlap(tensors, outs) -> None:
    """An output may be its own tensor; it may not share memory with another, or with another output."""
    pieces = []
    for t, o in zip(tensors, outs):
        for is_out, v in ((False, t), (True, o)):
            if v.numel() and not (is_out and v.data_ptr() == t.data_ptr()):
                written = is_out or o.data_ptr() == t.data_ptr()
                pieces.append((v.data_ptr(), v.data_ptr() + v.numel() * v.element_size(), written))
    pieces.sort()
    end, written = 0, 0     # of all pieces so far, and of those that are written
    for lo, hi, out in pieces:
        if lo < (end if out else written):
            raise ValueError("an output shares memory with another tensor")
        end = max(end, hi)
        if out:
            written = max(written, hi)


# ----------------------------------------------------------------------------
# convenience: allocation + autograd
# ----------------------------------------------------------------------------

class Workspace:
    """Grow-only forward workspace for one device. The first call on a shape
    uses the library's size hint; calls made with too small a workspace stay
    exact (overflowing bins take the slow path), and `grow()` reads the size
    the last call needed."""

    def __init__(self, device):
        self.device = torch.device(device)
        self.buf = torch.empty(0, dtype=torch.uint8, device=self.device)

    def ensure(self, nbytes: int) -> torch.Tensor:
        if self.buf.numel() < nbytes:
            self.buf = torch.empty(int(nbytes), dtype=torch.uint8, device=self.device)
        return self.buf

    def grow(self) -> dict:
        stats = dmr_workspace_stats(self.buf)
        self.ensure(stats["required_bytes"])
        return stats


_workspaces = {}


def workspace_for(device) -> Workspace:
    device = torch.device(device)
    if device not in _workspaces:
        _workspaces[device] = Workspace(device)
    return _workspaces[device]


def _alloc_outputs(N, H, W, K, device):
    return (torch.empty((N, H, W, K), dtype=torch.int64, device=device),
            torch.empty((N, H, W, K), dtype=torch.float32, device=device),
            torch.empty((N, H, W, K, 3), dtype=torch.float32, device=device),
            torch.empty((N, H, W, K), dtype=torch.float32, device=device))


class _RasterizeMeshes(torch.autograd.Function):
    @staticmethod
    def forward(ctx, verts, faces, offsets, H, W, K, blur_radius, settings):
        N = offsets.shape[0] - 1
        out = _alloc_outputs(N, H, W, K, verts.device)
        # Each call owns its workspace: the backward pass reuses its face
        # records and bin lists, so it must survive until then.
        ws = torch.empty(dmr_workspace_size_hint(N, faces.shape[0], H, W, K, blur_radius), dtype=torch.uint8,
                         device=verts.device)
        rasterize_meshes_fwd_ex(verts, faces, offsets, H, W, K, blur_radius, *out, ws, settings)
        ctx.save_for_backward(verts, faces, offsets, out[0], ws)
        ctx.dims = (H, W, K, blur_radius, settings)
        ctx.mark_non_differentiable(out[0])
        return out

    @staticmethod
    def backward(ctx, g_p2f, g_zbuf, g_bary, g_dists):
        verts, faces, offsets, p2f, ws = ctx.saved_tensors
        H, W, K, blur_radius, settings = ctx.dims
        grad_verts = torch.empty_like(verts)

        def c(g):
            return None if g is None else g.contiguous()

        rasterize_meshes_bwd(verts, faces, offsets, H, W, K, blur_radius, p2f, c(g_zbuf), c(g_bary), c(g_dists),
                             grad_verts, ws, reuse_forward_workspace=True, settings=settings)
        return grad_verts, None, None, None, None, None, None, None


def rasterize_meshes(verts: torch.Tensor, faces: torch.Tensor, mesh_face_offsets: torch.Tensor,
                     image_size: Tuple[int, int], faces_per_pixel: int = 1, blur_radius: float = 0.0,
                     perspective_correct: bool = False, cull_backfaces: bool = False,
                     clip_barycentric_coords: bool = True):
    """Rasterizes a packed batch of meshes on the GPU.

    verts [V,3] float32 (x, y NDC, z depth), faces [F,3] int64, mesh_face_offsets
    [N+1] int64. Returns (pix_to_face, zbuf, bary, dists); zbuf, bary and dists
    are differentiable with respect to verts. The three settings map to the
    DMR_RASTER_* bits of include/dmr.h."""
    H, W = image_size
    settings = ((DMR_RASTER_PERSPECTIVE_CORRECT if perspective_correct else 0)
                | (DMR_RASTER_CULL_BACKFACES if cull_backfaces else 0)
                | (0 if clip_barycentric_coords else DMR_RASTER_UNCLIPPED_BARY))
    return _RasterizeMeshes.apply(verts, faces, mesh_face_offsets, int(H), int(W), int(faces_per_pixel),
                                  float(blur_radius), settings)


class _ProjectMeshes(torch.autograd.Function):
    @staticmethod
    def forward(ctx, verts_world, mesh_vert_offsets, cameras):
        out = torch.empty_like(verts_world)
        dmr_project_fwd(verts_world, mesh_vert_offsets, cameras, out)
        ctx.save_for_backward(verts_world, mesh_vert_offsets, cameras)
        return out

    @staticmethod
    def backward(ctx, g):
        verts_world, offs, cameras = ctx.saved_tensors
        gv = torch.empty_like(verts_world)
        gc = torch.empty_like(cameras) if ctx.needs_input_grad[2] else None
        dmr_project_bwd(verts_world, offs, cameras, g.contiguous(), gv, gc)
        return gv, None, gc


def project_meshes(verts_world: torch.Tensor, mesh_vert_offsets: torch.Tensor, cameras: torch.Tensor):
    """Projects a packed batch of meshes (one 4x4 camera per mesh) to the
    rasterizer's screen space; differentiable with respect to verts_world
    and cameras."""
    return _ProjectMeshes.apply(verts_world, mesh_vert_offsets, cameras)


class _RasterizePoints(torch.autograd.Function):
    @staticmethod
    def forward(ctx, points, offsets, H, W, K, radius):
        N = offsets.shape[0] - 1
        dev = points.device
        idx = torch.empty((N, H, W, K), dtype=torch.int64, device=dev)
        zbuf = torch.empty((N, H, W, K), dtype=torch.float32, device=dev)
        dists = torch.empty((N, H, W, K), dtype=torch.float32, device=dev)
        ws = torch.empty(dmr_points_workspace_size_hint(N, points.shape[0], H, W, K, radius), dtype=torch.uint8,
                         device=dev)
        rasterize_points_fwd(points, offsets, H, W, K, radius, idx, zbuf, dists, ws)
        ctx.save_for_backward(points, offsets, idx)
        ctx.dims = (H, W, K)
        ctx.mark_non_differentiable(idx)
        return idx, zbuf, dists

    @staticmethod
    def backward(ctx, g_idx, g_zbuf, g_dists):
        points, offsets, idx = ctx.saved_tensors
        H, W, K = ctx.dims
        grad = torch.empty_like(points)

        def c(g):
            return None if g is None else g.contiguous()

        rasterize_points_bwd(points, offsets, H, W, K, idx, c(g_zbuf), c(g_dists), grad)
        return grad, None, None, None, None, None


def rasterize_points(points: torch.Tensor, cloud_offsets: torch.Tensor, image_size: Tuple[int, int],
                     points_per_pixel: int = 1, radius: float = 0.01):
    """Rasterizes a packed batch of point clouds on the GPU: (idx, zbuf,
    dists), zbuf and dists differentiable with respect to points."""
    H, W = image_size
    return _RasterizePoints.apply(points, cloud_offsets, int(H), int(W), int(points_per_pixel), float(radius))


class _GroupedLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, row_offsets, weight, bias):
        _grouped_inputs(x, row_offsets, weight)
        y = torch.empty((x.shape[0], weight.shape[1]), dtype=x.dtype, device=x.device)
        dmr_grouped_linear_fwd(x, row_offsets, weight, bias, y)
        ctx.save_for_backward(x, row_offsets, weight)
        return y

    @staticmethod
    def backward(ctx, g):
        x, row_offsets, weight = ctx.saved_tensors
        need_x, _, need_w, need_b = ctx.needs_input_grad
        grads = _GroupedLinearGrads.apply if torch.is_grad_enabled() else _grouped_grads   # create_graph, or not
        gx, gw, gb = grads(x, row_offsets, weight, g.contiguous(), (need_x, need_w, need_b))
        return gx, None, gw, gb


def _grouped_grads(x, row_offsets, weight, g, needs):
    N, cout, cin = weight.shape
    gx = torch.empty_like(x) if needs[0] else None
    gw = torch.empty_like(weight) if needs[1] else None
    gb = torch.empty((N, cout), dtype=weight.dtype, device=weight.device) if needs[2] else None
    ws = None
    if needs[1] or needs[2]:
        ws = torch.empty(dmr_grouped_linear_workspace_size(x.shape[0], N, cin, cout, x.dtype), dtype=torch.uint8,
                         device=x.device)
    dmr_grouped_linear_bwd(x, row_offsets, weight, g, gx, gw, gb, ws)
    return gx, gw, gb


class _GroupedLinearGrads(torch.autograd.Function):
    """The layer's backward pass as a function of x, weight and grad_y: each
    result is a product of two of them (or a sum of grad_y), so its own
    gradients are the layer's three products again."""

    @staticmethod
    def forward(ctx, x, row_offsets, weight, g, needs):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x, row_offsets, weight, g)
        return _grouped_grads(x, row_offsets, weight, g, needs)

    @staticmethod
    def backward(ctx, hx, hw, hb):
        x, off, weight, g = ctx.saved_tensors
        hx, hw, hb = (None if h is None else h.contiguous() for h in (hx, hw, hb))
        need_x, _, need_w, need_g, _ = ctx.needs_input_grad
        grads = _GroupedLinearGrads.apply if torch.is_grad_enabled() else _grouped_grads
        # grad_x_r = W_n^T g_r, grad_W_n = sum_r g_r x_r^T, grad_b_n = sum_r g_r
        dx = grads(x, off, hw, g, (True, False, False))[0] if need_x and hw is not None else None
        dw = grads(hx, off, weight, g, (False, True, False))[1] if need_w and hx is not None else None
        dg = None
        if need_g:
            parts, bias = [], hb
            for rows, w in ((hx, weight), (x, hw)):
                if rows is not None and w is not None:
                    parts.append(grouped_linear(rows, off, w, bias))
                    bias = None
            if bias is not None:
                parts.append(grouped_linear(g.new_ones((g.shape[0], 1)), off, bias.unsqueeze(2)))   # b_n for every row
            dg = sum(parts[1:], parts[0]) if parts else None
        return dx, None, dw, dg, None


def grouped_linear(x: torch.Tensor, row_offsets: torch.Tensor, weight: torch.Tensor,
                   bias: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y_r = W_n x_r + b_n for the rows r of every group n (a mesh's
    vertices, an image's pixels): x [R, in], row_offsets [N + 1] int64,
    weight [N, out, in], bias [N, out], all of one type (float32, float16 or
    bfloat16). Differentiable any number of times with respect to x, weight and
    bias (in reverse mode; forward mode raises)."""
    if forward_ad._current_level >= 0 or torch.is_grad_enabled() and (
            x.requires_grad or weight.requires_grad or (bias is not None and bias.requires_grad)):
        return _GroupedLinear.apply(x, row_offsets, weight, bias)
    dev, dt, R, cin, N, cout, code = _grouped_inputs(x, row_offsets, weight)
    if bias is not None and not _alike(bias, dt, dev, (N, cout)):
        _check(bias, "bias", dt, dev, (N, cout))
    y = torch.empty((R, cout), dtype=dt, device=dev)
    _launch_grouped(x, R, cin, row_offsets, N, weight, bias, cout, code, y, dev)
    return y


class _GroupedLayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, row_offsets, weight, bias, eps):
        y = torch.empty_like(x)
        dmr_grouped_layer_norm_fwd(x, row_offsets, weight, bias, y, eps)
        ctx.eps = eps
        ctx.save_for_backward(x, row_offsets, weight)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        x, row_offsets, weight = ctx.saved_tensors
        need_x, _, need_w, need_b, _ = ctx.needs_input_grad
        N, C = row_offsets.shape[0] - 1, x.shape[1]
        gx = torch.empty_like(x) if need_x else None
        gw, gb = (torch.empty((N, C), dtype=x.dtype, device=x.device) if need else None for need in (need_w, need_b))
        ws = None
        if need_w or need_b:
            ws = torch.empty(dmr_grouped_layer_norm_workspace_size(x.shape[0], N, C, x.dtype), dtype=torch.uint8,
                             device=x.device)
        dmr_grouped_layer_norm_bwd(x, row_offsets, weight, g.contiguous(), gx, gw, gb, ws, ctx.eps)
        return gx, None, gw, gb, None


def _wants_grad(*tensors) -> bool:
    return forward_ad._current_level >= 0 or torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


def grouped_layer_norm(x: torch.Tensor, row_offsets: torch.Tensor, weight: Optional[torch.Tensor] = None,
                       bias: Optional[torch.Tensor] = None, eps: float = 1e-5) -> torch.Tensor:
    """The rows of every group n (a mesh's vertices, an image's pixels) with
    mean 0 and variance 1, times weight_n, plus bias_n: x [R, C], row_offsets
    [N + 1] int64 from 0 to R, weight and bias [N, C] or None, all of one type
    (float32, float16 or bfloat16). Differentiable once with respect to x, weight and
    bias (in reverse mode; second derivatives and forward mode raise)."""
    if _wants_grad(x, weight, bias):
        return _GroupedLayerNorm.apply(x, row_offsets, weight, bias, float(eps))
    y = torch.empty_like(x)
    dmr_grouped_layer_norm_fwd(x, row_offsets, weight, bias, y, eps)
    return y


class _GroupedGatedLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, row_offsets, weight, bias, activation):
        y = _gated(x, row_offsets, weight, bias, activation)
        ctx.activation = activation
        ctx.save_for_backward(x, row_offsets, weight, bias)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        x, row_offsets, weight, bias = ctx.saved_tensors
        need_x, _, need_w, need_b, _ = ctx.needs_input_grad
        N, _, F, C = weight.shape
        gx, gw, gb = (torch.empty_like(t) if need else None for t, need in ((x, need_x), (weight, need_w), (bias, need_b)))
        ws = torch.empty(dmr_grouped_gated_linear_workspace_size(x.shape[0], N, C, F, x.dtype), dtype=torch.uint8,
                         device=x.device)
        dmr_grouped_gated_linear_bwd(x, row_offsets, weight, bias, g.contiguous(), gx, gw, gb, ws, ctx.activation)
        return gx, None, gw, gb, None


def _gated(x, row_offsets, weight, bias, activation):
    dev, dt, R, C, N, F, act, code = _gated_inputs(x, row_offsets, weight, bias, activation)
    y = torch.empty((R, F), dtype=dt, device=dev)
    _launch(lib().dmr_grouped_gated_linear_fwd, dev, x.data_ptr(), R, C, row_offsets.data_ptr(), N, weight.data_ptr(),
            _address(bias), F, act, code, y.data_ptr())
    return y


def grouped_gated_linear(x: torch.Tensor, row_offsets: torch.Tensor, weight: torch.Tensor,
                         bias: Optional[torch.Tensor] = None, activation: str = "silu") -> torch.Tensor:
    """y_r = act(A_n x_r + a_n) * (U_n x_r + u_n) for the rows r of every
    group n (a mesh's vertices, an image's pixels), both products in one
    kernel: x [R, in], row_offsets [N + 1] int64 from 0 to R, weight [N, 2, out,
    in] (A and U), bias [N, 2, out] (a and u) or None, all of one type (float32, float16
    or bfloat16); activation "silu", "gelu", "gelu_tanh" or "sigmoid".
    Differentiable once with respect to x, weight and bias (in reverse mode;
    second derivatives and forward mode raise); the backward pass keeps only
    the inputs and computes both products again."""
    if _wants_grad(x, weight, bias):
        return _GroupedGatedLinear.apply(x, row_offsets, weight, bias, activation)
    return _gated(x, row_offsets, weight, bias, activation)


def clip_grad_norm(grads: Sequence[torch.Tensor], max_norm: float, groups: Optional[int] = None, eps: float = 1e-6,
                   out: Optional[Sequence[torch.Tensor]] = None) -> Tuple[List[torch.Tensor], torch.Tensor]:
    """(grads times min(1, max_norm / (norm + eps)), norms): the norm of all
    values of all tensors together, norms [1]; or, with `groups`, one norm for
    each slice of the tensors' first dimension (each mesh's own decoder), norms
    [groups]. The tensors may be of different types. `out`: where the results
    go (the same list: in place); new tensors if not given. Not
    differentiable."""
    grads = list(grads)
    count = 1 if groups is None else int(groups)
    if groups is not None:
        for g in grads:
            if g.dim() < 1 or g.shape[0] != count:
                raise ValueError(f"grads of {count} groups must be [{count}, ...], got {tuple(g.shape)}")
    outs = list(map(torch.empty_like, grads)) if out is None else list(out)
    if len(outs) != len(grads):
        raise ValueError(f"{len(grads)} grads, but {len(outs)} out")
    dev, table = _spans(grads, outs, count, alike=out is None)
    if out is not None:
        _check_overlap(grads, outs)
    L = lib()
    size = L.dmr_clip_norm_workspace_size(table, len(grads), count)
    norms = torch.empty(count, dtype=torch.float32, device=dev)
    ws = torch.empty(size, dtype=torch.uint8, device=dev) if size > 256 else None   # the least: none is used
    _launch(L.dmr_clip_norm, dev, table, len(grads), count, float(max_norm), float(eps), norms.data_ptr(), _address(ws), size)
    if out is not None:
        for o in outs:      # what autograd saved of them is not what they hold now
            torch.autograd.graph.increment_version(o)
    return outs, norms


def orthogonalize(update: torch.Tensor, steps: int = 5, eps: float = 1e-7) -> torch.Tensor:
    """The nearest thing to an orthogonal matrix in the direction of each
    matrix of `update` [B, m, n] (or [m, n]), by `steps` Newton-Schulz
    products: what an optimiser applies in place of a weight's momentum. Not
    differentiable."""
    u = update.detach()
    if u.dim() == 2:
        u = u.unsqueeze(0)
    if u.dim() != 3:
        raise ValueError("update must be [B, m, n] or [m, n]")
    _dtype(u, "update")
    _check(u, "update", u.dtype, u.device)
    out = torch.empty_like(u)
    ws = torch.empty(dmr_orthogonalize_workspace_size(*u.shape, u.dtype), dtype=torch.uint8, device=u.device)
    dmr_orthogonalize(u, out, ws, steps, eps)
    return out.view(update.shape)


# ----------------------------------------------------------------------------
# per-kernel timing (measurement only)
# ----------------------------------------------------------------------------

def kernel_names():
    L = lib()
    return [L.dmr_kernel_name(i).decode() for i in range(L.dmr_kernel_count())]


def set_kernel_timing(enable: bool) -> None:
    rc = lib().dmr_set_kernel_timing(1 if enable else 0)
    if rc != 0:
        raise DmrError("dmr_set_kernel_timing", rc)


def set_kernel_timing_only(names) -> None:
    """Times only the named kernels (see kernel_names())."""
    ids = kernel_names()
    mask = 0
    for n in names:
        mask |= 1 << ids.index(n)
    rc = lib().dmr_set_kernel_timing_mask(mask)
    if rc != 0:
        raise DmrError("dmr_set_kernel_timing_mask", rc)


def reset_kernel_timing() -> None:
    rc = lib().dmr_reset_kernel_timing()
    if rc != 0:
        raise DmrError("dmr_reset_kernel_timing", rc)


def kernel_timing() -> dict:
    """{kernel name: (total ms, launches)} since the last reset."""
    L = lib()
    out = {}
    for i, name in enumerate(kernel_names()):
        ms, n = ctypes.c_double(), ctypes.c_int64()
        rc = L.dmr_kernel_timing(i, ctypes.byref(ms), ctypes.byref(n))
        if rc != 0:
            raise DmrError("dmr_kernel_timing", rc)
        out[name] = (ms.value, n.value)
    return out
