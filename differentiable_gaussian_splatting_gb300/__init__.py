"""Differentiable 3D Gaussian splatting rasterizer for NVIDIA GB300 (sm_103a).

Thin Python binding of the C ABI in ``include/gs.h`` (library ``libgs.so``).
The five calls of the hot path keep their C names:

    gs_project, gs_bin_sort, gs_rasterize_fwd, gs_rasterize_bwd, gs_project_bwd

Each takes torch CUDA tensors (or raw device addresses), checks shapes and
dtypes, and passes plain pointers to the library; every step of the path runs
in the library's CUDA kernels.  PyTorch only provides device memory and
streams.  There is no CPU fallback: if ``libgs.so`` is missing or no CUDA
device is present, the calls raise.

Next to the path stand the token operators of a network that predicts Gaussians
and is trained through it: ``gs_qk_norm_rope``, ``gs_attention_fwd``,
``gs_dropout_add``, ``gs_residual_norm`` and their gradients, and
``gs_clip_grad_norm``.  They take torch tensors of the current device, which a
small compiled module checks and passes on (``csrc/token_binding.cpp``).

``Rasterizer`` is a convenience that allocates the outputs and workspaces of
one view and runs the five calls in order.
"""

from __future__ import annotations

import ctypes as C
import os
import threading
from dataclasses import dataclass

from . import build as _build

__all__ = [
    "gs_project", "gs_bin_sort", "gs_rasterize_fwd", "gs_rasterize_bwd", "gs_project_bwd",
    "gs_project_sh16", "gs_project_bwd_sh16", "gs_project_bwd_adam", "AdamSettings",
    "gs_loss_l1_ssim", "gs_loss_workspace_bytes", "LossSettings",
    "gs_bin_sort_workspace_bytes", "gs_raster_workspace_bytes", "gs_bin_sort_noalloc",
    "gs_raster_stats", "gs_default_settings", "gs_status_string", "gs_num_tiles",
    "gs_qk_norm_rope", "gs_qk_norm_rope_bwd", "gs_qk_norm_rope_workspace_bytes",
    "gs_attention_fwd", "gs_attention_bwd", "gs_attention_workspace_bytes", "gs_attention_status",
    "gs_dropout_add", "gs_dropout_add_bwd",
    "gs_attention_window_fwd", "gs_attention_window_bwd", "gs_attention_window_workspace_bytes",
    "gs_residual_norm", "gs_residual_norm_bwd", "gs_residual_norm_workspace_bytes",
    "gs_clip_grad_norm", "gs_clip_grad_norm_workspace_bytes",
    "Camera", "Settings", "Rasterizer", "library",
    "GSError", "TILE", "GRAD2D", "SPLAT_FLOATS",
]

TILE = 16
GRAD2D = 9
SPLAT_FLOATS = 12
STATUS = {0: "ok", 1: "invalid argument", 2: "CUDA error", 3: "pair list capacity exceeded",
          4: "device wait timed out", 5: "workspace too small"}


class GSError(RuntimeError):
    def __init__(self, fn: str, status: int, extra: str = ""):
        self.status = status
        super().__init__(f"{fn}: {STATUS.get(status, status)} ({status}){extra}")


class Camera(C.Structure):
    """gs_camera: row-major 4x4 world->camera matrix, intrinsics, image size, near plane."""
    _fields_ = [("viewmat", C.c_float * 16), ("fx", C.c_float), ("fy", C.c_float),
                ("cx", C.c_float), ("cy", C.c_float), ("width", C.c_int32),
                ("height", C.c_int32), ("znear", C.c_float)]

    @classmethod
    def of(cls, cam) -> "Camera":
        """From any object with viewmat, fx, fy, cx, cy, width, height, znear."""
        if isinstance(cam, cls):
            return cam
        vm = [float(v) for v in _flat16(cam.viewmat)]
        return cls((C.c_float * 16)(*vm), float(cam.fx), float(cam.fy), float(cam.cx),
                   float(cam.cy), int(cam.width), int(cam.height), float(getattr(cam, "znear", 0.2)))


def _flat16(vm):
    try:
        import numpy as np
        return np.asarray(vm, dtype=np.float64).reshape(16).tolist()
    except ImportError:  # pragma: no cover
        return [x for row in vm for x in row]


class Settings(C.Structure):
    """gs_settings: scheduling of the blending kernels (never changes results)."""
    _fields_ = [("split_mode", C.c_int32), ("force_h", C.c_int32), ("force_k", C.c_int32),
                ("h_max", C.c_int32), ("policy_lambda", C.c_float), ("policy_beta", C.c_float),
                ("policy_eps", C.c_float)]


class AdamSettings(C.Structure):
    """gs_adam_settings: learning rates per parameter group, Adam's betas and eps, step t."""
    _fields_ = [("lr_means", C.c_float), ("lr_scales", C.c_float), ("lr_quats", C.c_float),
                ("lr_opacities", C.c_float), ("lr_sh0", C.c_float), ("lr_shN", C.c_float),
                ("beta1", C.c_float), ("beta2", C.c_float), ("eps", C.c_float),
                ("step", C.c_int32)]


class AdamMoments(C.Structure):
    """gs_adam_moments: device pointers of the first and second moments, one per
    parameter (means, log-scales, quaternions, opacity logits, SH)."""
    _fields_ = [("m", C.c_void_p * 5), ("v", C.c_void_p * 5)]


class LossSettings(C.Structure):
    """gs_loss_settings: weight of the SSIM term, the SSIM constants, the window's sigma."""
    _fields_ = [("lambda_", C.c_float), ("c1", C.c_float), ("c2", C.c_float),
                ("sigma", C.c_float)]

    @classmethod
    def default(cls) -> "LossSettings":
        return cls(0.2, 0.01 ** 2, 0.03 ** 2, 1.5)


class Heads(C.Structure):
    """gs_heads: a [tokens, heads, head_dim] array read by strides (in elements)."""
    _fields_ = [("data", C.c_void_p), ("token_stride", C.c_int64), ("head_stride", C.c_int64)]


class HeadNorm(C.Structure):
    """gs_head_norm: element type, rotated values, pairing, eps, rows of the angle table."""
    _fields_ = [("type", C.c_int32), ("rot", C.c_int32), ("interleaved", C.c_int32),
                ("eps", C.c_float), ("table_rows", C.c_int64)]


class AttentionShape(C.Structure):
    """gs_attention_shape: tokens, sequences, heads, mask and scale of an attention call."""
    _fields_ = [("tokens_q", C.c_int64), ("tokens_k", C.c_int64), ("batch", C.c_int32),
                ("heads_q", C.c_int32), ("heads_k", C.c_int32), ("head_dim", C.c_int32),
                ("causal", C.c_int32), ("scale", C.c_float)]


class Window(C.Structure):
    """gs_window: keys that a query sees before and behind its own, and first keys that all see."""
    _fields_ = [("left", C.c_int32), ("right", C.c_int32), ("sinks", C.c_int32)]


class Rows(C.Structure):
    """gs_rows: a [tokens, width] array by its row stride (in elements)."""
    _fields_ = [("data", C.c_void_p), ("row_stride", C.c_int64)]


class BlockNorm(C.Structure):
    """gs_block_norm: element type, kinds of the norms, rows of the gate, alpha, beta, eps."""
    _fields_ = [("type", C.c_int32), ("pre", C.c_int32), ("post", C.c_int32), ("batch", C.c_int32),
                ("alpha", C.c_float), ("beta", C.c_float), ("eps", C.c_float)]


class NormParams(C.Structure):
    """gs_norm_params and gs_norm_grads: weights and biases of both norms, gate."""
    _fields_ = [(n, C.c_void_p) for n in ("pre_weight", "pre_bias", "post_weight", "post_bias",
                                          "gate")]


class Array(C.Structure):
    """gs_array: a contiguous array of gradients."""
    _fields_ = [("data", C.c_void_p), ("elements", C.c_int64), ("type", C.c_int32)]


_lib = None
_lib_lock = threading.Lock()
_P = C.c_void_p
_I64 = C.c_int64


def library() -> C.CDLL:
    """Load libgs.so (building it first when the sources are newer)."""
    global _lib
    with _lib_lock:
        if _lib is None:
            path = _build.LIB
            if not _build.library_up_to_date():
                _build.build_library()
            if not os.path.exists(path):
                raise RuntimeError("libgs.so is not built; run differentiable_gaussian_splatting_gb300.build")
            lib = C.CDLL(path)
            _declare(lib)
            _lib = lib
        return _lib


def _declare(lib: C.CDLL) -> None:
    st = C.c_int
    lib.gs_default_settings.restype = Settings
    lib.gs_status_string.restype = C.c_char_p
    lib.gs_status_string.argtypes = [st]
    lib.gs_num_tiles.restype = _I64
    lib.gs_num_tiles.argtypes = [C.c_int32, C.c_int32]
    lib.gs_project.restype = st
    lib.gs_project.argtypes = [C.POINTER(Camera), _I64, C.c_int32] + [_P] * 9 + [_P]
    lib.gs_bin_sort_workspace_bytes.restype = C.c_size_t
    lib.gs_bin_sort_workspace_bytes.argtypes = [_I64, _I64, C.c_int32, C.c_int32]
    lib.gs_bin_sort.restype = st
    lib.gs_bin_sort.argtypes = [C.POINTER(Camera), _I64, _P, _P, _P, _P, C.c_size_t, _P, _I64,
                                _P, _P, _P, _P, _P]
    lib.gs_raster_workspace_bytes.restype = C.c_size_t
    lib.gs_raster_workspace_bytes.argtypes = [C.c_int32, C.c_int32, _I64, C.POINTER(Settings)]
    lib.gs_rasterize_fwd.restype = st
    lib.gs_rasterize_fwd.argtypes = [C.POINTER(Camera), C.POINTER(Settings), _I64, _P, _P, _I64,
                                     _P, _P, _P, C.c_size_t, _P, _P, _P, _P, _P]
    lib.gs_rasterize_bwd.restype = st
    lib.gs_rasterize_bwd.argtypes = [C.POINTER(Camera), C.POINTER(Settings), _I64, _P, _P, _I64,
                                     _P, _P, _P, C.c_size_t, _P, _P, _P, _P, _P, _P, _P]
    lib.gs_project_bwd.restype = st
    lib.gs_project_bwd.argtypes = [C.POINTER(Camera), _I64, C.c_int32] + [_P] * 13 + [_P]
    lib.gs_raster_stats.restype = st
    lib.gs_raster_stats.argtypes = [_P, C.c_size_t, _P, _P]
    lib.gs_project_sh16.restype = st
    lib.gs_project_sh16.argtypes = [C.POINTER(Camera), _I64, C.c_int32] + [_P] * 9 + [_P]
    lib.gs_project_bwd_sh16.restype = st
    lib.gs_project_bwd_sh16.argtypes = [C.POINTER(Camera), _I64, C.c_int32] + [_P] * 13 + [_P]
    lib.gs_project_bwd_adam.restype = st
    lib.gs_project_bwd_adam.argtypes = ([C.POINTER(Camera), _I64, C.c_int32] + [_P] * 8 +
                                        [C.POINTER(AdamMoments), C.POINTER(AdamSettings), _P,
                                         _P, _P])
    lib.gs_loss_workspace_bytes.restype = C.c_size_t
    lib.gs_loss_workspace_bytes.argtypes = [C.c_int32, C.c_int32]
    lib.gs_loss_l1_ssim.restype = st
    lib.gs_loss_l1_ssim.argtypes = [C.c_int32, C.c_int32, _P, _P, C.POINTER(LossSettings), _P, _P,
                                    _P, C.c_size_t, _P]
    H, N, A = C.POINTER(Heads), C.POINTER(HeadNorm), C.POINTER(AttentionShape)
    i32 = C.c_int32
    lib.gs_qk_norm_rope.restype = st
    lib.gs_qk_norm_rope.argtypes = [_I64, i32, i32, i32, N, H, H, _P, _P, _P, _P, H, H, _P]
    lib.gs_qk_norm_rope_workspace_bytes.restype = C.c_size_t
    lib.gs_qk_norm_rope_workspace_bytes.argtypes = [_I64, i32, i32, i32]
    lib.gs_qk_norm_rope_bwd.restype = st
    lib.gs_qk_norm_rope_bwd.argtypes = ([_I64, i32, i32, i32, N, H, H] + [_P] * 4 + [H] * 4 +
                                        [_P, _P, _P, C.c_size_t, _P])
    lib.gs_attention_workspace_bytes.restype = C.c_size_t
    lib.gs_attention_workspace_bytes.argtypes = [A]
    lib.gs_attention_fwd.restype = st
    lib.gs_attention_fwd.argtypes = [A, H, H, H, _P, _P, H, _P, _P, C.c_size_t, _P]
    lib.gs_attention_bwd.restype = st
    lib.gs_attention_bwd.argtypes = [A, H, H, H, _P, _P, H, _P, H, H, H, H, _P, C.c_size_t, _P]
    V = C.POINTER(Window)
    lib.gs_attention_window_workspace_bytes.restype = C.c_size_t
    lib.gs_attention_window_workspace_bytes.argtypes = [A, V]
    lib.gs_attention_window_fwd.restype = st
    lib.gs_attention_window_fwd.argtypes = [A, V, H, H, H, _P, _P, H, _P, _P, C.c_size_t, _P]
    lib.gs_attention_window_bwd.restype = st
    lib.gs_attention_window_bwd.argtypes = [A, V, H, H, H, _P, _P, H, _P, H, H, H, H, _P,
                                            C.c_size_t, _P]
    lib.gs_attention_status.restype = st
    lib.gs_attention_status.argtypes = [_P]
    lib.gs_dropout_add.restype = st
    lib.gs_dropout_add.argtypes = [_I64, i32, _P, _P, _P, _P, C.c_float, _P]
    lib.gs_dropout_add_bwd.restype = st
    lib.gs_dropout_add_bwd.argtypes = [_I64, i32, _P, _P, _P, C.c_float, _P]
    lib.gs_residual_norm.restype = st
    B, R, W = C.POINTER(BlockNorm), C.POINTER(Rows), C.POINTER(NormParams)
    lib.gs_residual_norm.argtypes = [_I64, i32, B, R, R, W, _P, R, R, _P]
    lib.gs_residual_norm_workspace_bytes.restype = C.c_size_t
    lib.gs_residual_norm_workspace_bytes.argtypes = [_I64, i32, i32]
    lib.gs_residual_norm_bwd.restype = st
    lib.gs_residual_norm_bwd.argtypes = [_I64, i32, B, R, R, W, _P, R, R, R, R, W, _P, C.c_size_t, _P]
    lib.gs_clip_grad_norm_workspace_bytes.restype = C.c_size_t
    lib.gs_clip_grad_norm_workspace_bytes.argtypes = [i32]
    lib.gs_clip_grad_norm.restype = st
    lib.gs_clip_grad_norm.argtypes = [i32, C.POINTER(Array), C.POINTER(Array), C.c_float, _P, _P, C.c_size_t, _P]
    lib.gs_bin_sort_noalloc.restype = st
    lib.gs_bin_sort_noalloc.argtypes = [C.POINTER(Camera), _I64, _P, _P, _P, _P, _I64, _P, _P, _P,
                                        _P, _P]


# ---------------------------------------------------------------------------
# argument marshalling
# ---------------------------------------------------------------------------
def _is_bf16(t) -> bool:
    import torch

    return isinstance(t, torch.Tensor) and t.dtype == torch.bfloat16


def _ptr(t, name, dtype=None, numel=None, optional=False):
    """Device address of a tensor (checked), an int address, or None."""
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if isinstance(t, int):
        return t
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch tensor or a device address")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name}: needs at least {numel} elements, has {t.numel()}")
    return t.data_ptr() if t.numel() > 0 else None


_torch = None  # the module, once a call has needed it


def _load_torch():
    global _torch
    if _torch is None:
        import torch

        _torch = torch
    return _torch


def _stream(stream):
    if stream is None:
        torch = _torch or _load_torch()
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is None:
            return torch.cuda.current_stream().cuda_stream
        # the same handle without building a Stream object (0.2 instead of 3 us)
        return raw(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, status: int, extra: str = "") -> None:
    if status != 0:
        raise GSError(fn, status, extra)


def _settings(settings) -> Settings:
    return settings if settings is not None else gs_default_settings()


def gs_default_settings() -> Settings:
    return library().gs_default_settings()


def gs_status_string(status: int) -> str:
    """The library's text for a gs_status code."""
    return library().gs_status_string(int(status)).decode()


def gs_num_tiles(width: int, height: int) -> int:
    """Number of 16 x 16 tiles covering a width x height image (0 for an empty image)."""
    return int(library().gs_num_tiles(int(width), int(height)))


def _f32():
    import torch

    return torch.float32


def _i32():
    import torch

    return torch.int32


def gs_project(cam, n, sh_degree, means, scales, quats, opacities, sh, splats, depths, radii,
               tiles_touched, stream=None):
    """Projection + SH colour + tile counts (see gs.h)."""
    K = (int(sh_degree) + 1) ** 2
    f, i = _f32(), _i32()
    st = library().gs_project(
        C.byref(Camera.of(cam)), int(n), int(sh_degree), _ptr(means, "means", f, 3 * n),
        _ptr(scales, "scales", f, 3 * n), _ptr(quats, "quats", f, 4 * n),
        _ptr(opacities, "opacities", f, n), _ptr(sh, "sh", f, 3 * K * n),
        _ptr(splats, "splats", f, SPLAT_FLOATS * n), _ptr(depths, "depths", f, n),
        _ptr(radii, "radii", i, 2 * n), _ptr(tiles_touched, "tiles_touched", i, n), _stream(stream))
    _check("gs_project", st)


def gs_project_sh16(cam, n, sh_degree, means, scales, quats, opacities, sh, splats, depths, radii,
                    tiles_touched, stream=None):
    """gs_project with the SH coefficients as a torch.bfloat16 tensor (see gs.h)."""
    import torch

    K = (int(sh_degree) + 1) ** 2
    f, i = _f32(), _i32()
    st = library().gs_project_sh16(
        C.byref(Camera.of(cam)), int(n), int(sh_degree), _ptr(means, "means", f, 3 * n),
        _ptr(scales, "scales", f, 3 * n), _ptr(quats, "quats", f, 4 * n),
        _ptr(opacities, "opacities", f, n), _ptr(sh, "sh", torch.bfloat16, 3 * K * n),
        _ptr(splats, "splats", f, SPLAT_FLOATS * n), _ptr(depths, "depths", f, n),
        _ptr(radii, "radii", i, 2 * n), _ptr(tiles_touched, "tiles_touched", i, n), _stream(stream))
    _check("gs_project_sh16", st)


def gs_bin_sort_workspace_bytes(n, capacity, width, height) -> int:
    return int(library().gs_bin_sort_workspace_bytes(int(n), int(capacity), int(width), int(height)))


def gs_bin_sort(cam, n, splats, depths, tiles_touched, workspace, sorted_ids, capacity,
                tile_ranges, lpt_order, counts_device=None, sync_pairs=True, stream=None):
    """Tile binning and sort into (tile, depth, id) order, with tile ranges and LPT order
    (per-tile buckets below 8 Mi pairs of capacity, a two-stage radix sort from there);
    returns the pair count I when sync_pairs (GSError status 3 names the count needed)."""
    import torch

    cam_c = Camera.of(cam)
    nt = library().gs_num_tiles(cam_c.width, cam_c.height)
    host = C.c_int64(-1)
    st = library().gs_bin_sort(
        C.byref(cam_c), int(n), _ptr(splats, "splats", _f32(), SPLAT_FLOATS * n, optional=n == 0),
        _ptr(depths, "depths", _f32(), n, optional=n == 0),
        _ptr(tiles_touched, "tiles_touched", _i32(), n, optional=n == 0),
        _ptr(workspace, "workspace", torch.uint8), workspace.numel(),
        _ptr(sorted_ids, "sorted_ids", _i32(), capacity), int(capacity),
        _ptr(tile_ranges, "tile_ranges", _i32(), 2 * nt), _ptr(lpt_order, "lpt_order", _i32(), nt),
        _ptr(counts_device, "counts_device", torch.int64, 2, optional=True),
        C.byref(host) if sync_pairs else None, _stream(stream))
    _check("gs_bin_sort", st, f"; pairs needed: {host.value}" if st == 3 else "")
    return int(host.value) if sync_pairs else None


def gs_bin_sort_noalloc(cam, n, splats, depths, tiles_touched, sorted_ids, capacity, tile_ranges,
                        lpt_order, counts_device=None, sync_pairs=True, stream=None):
    """gs_bin_sort on the library's fixed scratch (allocates nothing; see gs.h for its limits)."""
    import torch

    cam_c = Camera.of(cam)
    nt = library().gs_num_tiles(cam_c.width, cam_c.height)
    host = C.c_int64(-1)
    st = library().gs_bin_sort_noalloc(
        C.byref(cam_c), int(n), _ptr(splats, "splats", _f32(), SPLAT_FLOATS * n, optional=n == 0),
        _ptr(depths, "depths", _f32(), n, optional=n == 0),
        _ptr(tiles_touched, "tiles_touched", _i32(), n, optional=n == 0),
        _ptr(sorted_ids, "sorted_ids", _i32(), capacity), int(capacity),
        _ptr(tile_ranges, "tile_ranges", _i32(), 2 * nt), _ptr(lpt_order, "lpt_order", _i32(), nt),
        _ptr(counts_device, "counts_device", torch.int64, 2, optional=True),
        C.byref(host) if sync_pairs else None, _stream(stream))
    _check("gs_bin_sort_noalloc", st, f"; pairs needed: {host.value}" if st == 3 else "")
    return int(host.value) if sync_pairs else None


def gs_raster_workspace_bytes(width, height, capacity, settings=None) -> int:
    return int(library().gs_raster_workspace_bytes(int(width), int(height), int(capacity),
                                                   C.byref(_settings(settings))))


def gs_rasterize_fwd(cam, n, splats, sorted_ids, tile_ranges, lpt_order, workspace, image,
                     t_final, n_contrib, last_idx, settings=None, stream=None):
    """Forward blend (see gs.h); the pair capacity is sorted_ids' length."""
    import torch

    cam_c = Camera.of(cam)
    P = cam_c.width * cam_c.height
    st = library().gs_rasterize_fwd(
        C.byref(cam_c), C.byref(_settings(settings)), int(n),
        _ptr(splats, "splats", _f32(), SPLAT_FLOATS * n, optional=n == 0),
        _ptr(sorted_ids, "sorted_ids", _i32()), sorted_ids.numel(),
        _ptr(tile_ranges, "tile_ranges", _i32()),
        _ptr(lpt_order, "lpt_order", _i32()), _ptr(workspace, "workspace", torch.uint8),
        workspace.numel(), _ptr(image, "image", _f32(), 3 * P), _ptr(t_final, "t_final", _f32(), P),
        _ptr(n_contrib, "n_contrib", _i32(), P), _ptr(last_idx, "last_idx", _i32(), P),
        _stream(stream))
    _check("gs_rasterize_fwd", st)


def gs_rasterize_bwd(cam, n, splats, sorted_ids, tile_ranges, lpt_order, workspace, t_final,
                     last_idx, dL_dimage, dL_dt_final, grad2d, touched=None, settings=None,
                     stream=None):
    import torch

    cam_c = Camera.of(cam)
    P = cam_c.width * cam_c.height
    st = library().gs_rasterize_bwd(
        C.byref(cam_c), C.byref(_settings(settings)), int(n),
        _ptr(splats, "splats", _f32(), SPLAT_FLOATS * n, optional=n == 0),
        _ptr(sorted_ids, "sorted_ids", _i32()), sorted_ids.numel(),
        _ptr(tile_ranges, "tile_ranges", _i32()),
        _ptr(lpt_order, "lpt_order", _i32()), _ptr(workspace, "workspace", torch.uint8),
        workspace.numel(), _ptr(t_final, "t_final", _f32(), P),
        _ptr(last_idx, "last_idx", _i32(), P), _ptr(dL_dimage, "dL_dimage", _f32(), 3 * P),
        _ptr(dL_dt_final, "dL_dt_final", _f32(), P, optional=True),
        _ptr(grad2d, "grad2d", _f32(), GRAD2D * n, optional=n == 0),
        _ptr(touched, "touched", torch.uint8, n, optional=True), _stream(stream))
    _check("gs_rasterize_bwd", st)


def gs_project_bwd(cam, n, sh_degree, means, scales, quats, opacities, sh, tiles_touched, grad2d,
                   touched, dmeans, dscales, dquats, dopacities, dsh, stream=None):
    import torch

    K = (int(sh_degree) + 1) ** 2
    f, i = _f32(), _i32()
    st = library().gs_project_bwd(
        C.byref(Camera.of(cam)), int(n), int(sh_degree), _ptr(means, "means", f, 3 * n),
        _ptr(scales, "scales", f, 3 * n), _ptr(quats, "quats", f, 4 * n),
        _ptr(opacities, "opacities", f, n, optional=True), _ptr(sh, "sh", f, 3 * K * n),
        _ptr(tiles_touched, "tiles_touched", i, n), _ptr(grad2d, "grad2d", f, GRAD2D * n),
        _ptr(touched, "touched", torch.uint8, n, optional=True), _ptr(dmeans, "dmeans", f, 3 * n),
        _ptr(dscales, "dscales", f, 3 * n), _ptr(dquats, "dquats", f, 4 * n),
        _ptr(dopacities, "dopacities", f, n), _ptr(dsh, "dsh", f, 3 * K * n), _stream(stream))
    _check("gs_project_bwd", st)


def gs_project_bwd_sh16(cam, n, sh_degree, means, scales, quats, opacities, sh, tiles_touched,
                        grad2d, touched, dmeans, dscales, dquats, dopacities, dsh, stream=None):
    """gs_project_bwd with the SH coefficients as a torch.bfloat16 tensor; dsh is fp32."""
    import torch

    K = (int(sh_degree) + 1) ** 2
    f, i = _f32(), _i32()
    st = library().gs_project_bwd_sh16(
        C.byref(Camera.of(cam)), int(n), int(sh_degree), _ptr(means, "means", f, 3 * n),
        _ptr(scales, "scales", f, 3 * n), _ptr(quats, "quats", f, 4 * n),
        _ptr(opacities, "opacities", f, n, optional=True),
        _ptr(sh, "sh", torch.bfloat16, 3 * K * n),
        _ptr(tiles_touched, "tiles_touched", i, n), _ptr(grad2d, "grad2d", f, GRAD2D * n),
        _ptr(touched, "touched", torch.uint8, n, optional=True), _ptr(dmeans, "dmeans", f, 3 * n),
        _ptr(dscales, "dscales", f, 3 * n), _ptr(dquats, "dquats", f, 4 * n),
        _ptr(dopacities, "dopacities", f, n), _ptr(dsh, "dsh", f, 3 * K * n), _stream(stream))
    _check("gs_project_bwd_sh16", st)


def gs_project_bwd_adam(cam, n, sh_degree, means, log_scales, quats, opacity_logits, sh,
                        tiles_touched, grad2d, touched, m, v, settings: AdamSettings,
                        scales_out=None, opacities_out=None, stream=None):
    """gs_project_bwd fused with one Adam step on the raw parameters, in place (see gs.h).
    m and v: five tensors each, shaped like (means, log_scales, quats, opacity_logits, sh).
    scales_out / opacities_out (optional) receive exp(log_scales) and sigmoid(logits)
    after the step."""
    import torch

    K = (int(sh_degree) + 1) ** 2
    f, i = _f32(), _i32()
    sizes = (3 * n, 3 * n, 4 * n, n, 3 * K * n)
    names = ("means", "log_scales", "quats", "opacity_logits", "sh")
    if len(m) != 5 or len(v) != 5:
        raise ValueError("m and v need five tensors each")
    mom = AdamMoments()
    for k in range(5):
        mom.m[k] = _ptr(m[k], "m." + names[k], f, sizes[k])
        mom.v[k] = _ptr(v[k], "v." + names[k], f, sizes[k])
    params = (means, log_scales, quats, opacity_logits, sh)
    st = library().gs_project_bwd_adam(
        C.byref(Camera.of(cam)), int(n), int(sh_degree),
        *[_ptr(t, names[k], f, sizes[k]) for k, t in enumerate(params)],
        _ptr(tiles_touched, "tiles_touched", i, n), _ptr(grad2d, "grad2d", f, GRAD2D * n),
        _ptr(touched, "touched", torch.uint8, n, optional=True), C.byref(mom),
        C.byref(settings), _ptr(scales_out, "scales_out", f, 3 * n, optional=True),
        _ptr(opacities_out, "opacities_out", f, n, optional=True), _stream(stream))
    _check("gs_project_bwd_adam", st)


def gs_loss_workspace_bytes(width, height) -> int:
    return int(library().gs_loss_workspace_bytes(int(width), int(height)))


def gs_loss_l1_ssim(width, height, image, target, dL_dimage, loss_out, workspace,
                    settings: LossSettings | None = None, stream=None):
    """The L1 + SSIM loss of image against target and its gradient (see gs.h).
    loss_out: device float32[3] = (L, mean |x - y|, mean SSIM)."""
    import torch

    P = 3 * int(width) * int(height)
    f = _f32()
    ls = settings if settings is not None else LossSettings.default()
    st = library().gs_loss_l1_ssim(
        int(width), int(height), _ptr(image, "image", f, P), _ptr(target, "target", f, P),
        C.byref(ls), _ptr(dL_dimage, "dL_dimage", f, P), _ptr(loss_out, "loss_out", f, 3),
        _ptr(workspace, "workspace", torch.uint8), workspace.numel(), _stream(stream))
    _check("gs_loss_l1_ssim", st)


# ---------------------------------------------------------------------------
# token operators
# ---------------------------------------------------------------------------
_calls = None  # the compiled binding of these calls, once loaded


def _token_calls():
    """The compiled binding (csrc/token_binding.cpp): it checks the tensors (TypeError,
    ValueError), calls the library and returns the status.  Built when a call first needs it, if
    it is not there or was made for another torch or Python."""
    global _calls
    if _calls is None:
        import importlib.machinery
        import importlib.util

        _load_torch()
        library()
        with _lib_lock:
            if _calls is None:
                loader = importlib.machinery.ExtensionFileLoader("gs_token_binding",
                                                                 _build.build_binding())
                spec = importlib.util.spec_from_loader("gs_token_binding", loader)
                calls = importlib.util.module_from_spec(spec)
                loader.exec_module(calls)
                _calls = calls
    return _calls


def gs_qk_norm_rope(q, k, q_weight, k_weight, cos_sin, positions, q_out, k_out, eps=1e-6,
                    interleaved=False, stream=None):
    """RMS norm of every head of q and k and the position rotation, in one pass (see gs.h).
    q, k, q_out, k_out: [tokens, heads, head_dim] float32 or bfloat16, any strides with a
    contiguous last dimension; cos_sin [rows, rot] float32 (None: no rotation); weights and
    positions may be None."""
    st = (_calls or _token_calls()).qk_norm_rope(q, k, q_weight, k_weight, cos_sin, positions,
                                                 q_out, k_out, eps, interleaved, stream)
    if st:
        _check("gs_qk_norm_rope", st)


def gs_qk_norm_rope_workspace_bytes(tokens, heads_q, heads_k, head_dim) -> int:
    return int(library().gs_qk_norm_rope_workspace_bytes(int(tokens), int(heads_q), int(heads_k),
                                                         int(head_dim)))


def gs_qk_norm_rope_bwd(q, k, q_weight, k_weight, cos_sin, positions, dq_out, dk_out, dq, dk,
                        dq_weight, dk_weight, workspace, eps=1e-6, interleaved=False, stream=None):
    """Gradient of gs_qk_norm_rope (see gs.h); dq_weight and dk_weight (float32 [head_dim]) may
    be None."""
    st = (_calls or _token_calls()).qk_norm_rope_bwd(
        q, k, q_weight, k_weight, cos_sin, positions, dq_out, dk_out, dq, dk, dq_weight, dk_weight,
        workspace, eps, interleaved, stream)
    if st:
        _check("gs_qk_norm_rope_bwd", st)


def gs_attention_workspace_bytes(tokens_q, tokens_k, batch, heads_q, heads_k, head_dim) -> int:
    shape = AttentionShape(int(tokens_q), int(tokens_k), int(batch), int(heads_q), int(heads_k),
                           int(head_dim), 0, 1.0)
    return int(library().gs_attention_workspace_bytes(C.byref(shape)))


def gs_attention_fwd(q, k, v, out, lse, workspace, cu_q=None, cu_k=None, causal=False, scale=None,
                     stream=None):
    """Softmax attention over a ragged batch (see gs.h).  q, out [tokens_q, heads_q, head_dim],
    k, v [tokens_k, heads_k, head_dim] bfloat16, any strides with a contiguous last dimension;
    lse [heads_q, tokens_q] float32; cu_q, cu_k [batch + 1] int32 offsets (None: one sequence);
    scale defaults to head_dim ** -0.5."""
    st = (_calls or _token_calls()).attention_fwd(q, k, v, out, lse, workspace, cu_q, cu_k, causal,
                                                  scale, stream)
    if st:
        _check("gs_attention_fwd", st)


def gs_attention_bwd(q, k, v, out, lse, dout, dq, dk, dv, workspace, cu_q=None, cu_k=None,
                     causal=False, scale=None, stream=None):
    """Gradient of gs_attention_fwd from its out and lse (see gs.h)."""
    st = (_calls or _token_calls()).attention_bwd(q, k, v, out, lse, dout, dq, dk, dv, workspace,
                                                  cu_q, cu_k, causal, scale, stream)
    if st:
        _check("gs_attention_bwd", st)


def gs_attention_window_workspace_bytes(tokens_q, tokens_k, batch, heads_q, heads_k, head_dim, left,
                                        right=0, sinks=0) -> int:
    shape = AttentionShape(int(tokens_q), int(tokens_k), int(batch), int(heads_q), int(heads_k),
                           int(head_dim), 0, 1.0)
    window = Window(*[min(int(n), 2 ** 31 - 1) for n in (left, right, sinks)])
    return int(library().gs_attention_window_workspace_bytes(C.byref(shape), C.byref(window)))


def gs_attention_window_fwd(q, k, v, out, lse, workspace, left, right=0, sinks=0, cu_q=None,
                            cu_k=None, causal=False, scale=None, stream=None):
    """gs_attention_fwd over the `left` keys before a query's own, the `right` ones behind it and the
    first `sinks` of its sequence (see gs.h)."""
    st = (_calls or _token_calls()).attention_window_fwd(
        q, k, v, out, lse, workspace, left, right, sinks, cu_q, cu_k, causal, scale, stream)
    if st:
        _check("gs_attention_window_fwd", st)


def gs_attention_window_bwd(q, k, v, out, lse, dout, dq, dk, dv, workspace, left, right=0, sinks=0,
                            cu_q=None, cu_k=None, causal=False, scale=None, stream=None):
    """Gradient of gs_attention_window_fwd from its out and lse (see gs.h)."""
    st = (_calls or _token_calls()).attention_window_bwd(
        q, k, v, out, lse, dout, dq, dk, dv, workspace, left, right, sinks, cu_q, cu_k, causal,
        scale, stream)
    if st:
        _check("gs_attention_window_bwd", st)


def gs_attention_status(stream=None) -> None:
    """Waits for the stream; raises GSError status 4 if a bounded device wait of an attention
    call on this device has given up since this thread's last such check (or ever, at its
    first)."""
    _check("gs_attention_status", library().gs_attention_status(_stream(stream)))


def gs_dropout_add(x, residual, out, rng, p, stream=None):
    """out = residual + dropout(x) (see gs.h), all of one shape; residual may be None, out may be
    x or residual; rng: CUDA int64[2], seed and offset."""
    st = (_calls or _token_calls()).dropout_add(x, residual, out, rng, p, stream)
    if st:
        _check("gs_dropout_add", st)


def gs_dropout_add_bwd(dout, dx, rng, p, stream=None):
    """Gradient of gs_dropout_add by x, with the same rng (the residual's is dout itself)."""
    st = (_calls or _token_calls()).dropout_add_bwd(dout, dx, rng, p, stream)
    if st:
        _check("gs_dropout_add_bwd", st)


_NORMS = {"none": 0, "rms": 1, "layer": 2}


def _norm_kind(name, kind) -> int:
    if kind not in _NORMS:
        raise ValueError(f"{name}: expected 'none', 'rms' or 'layer', got {kind!r}")
    return _NORMS[kind]


def gs_residual_norm(x, y, r_out, h_out, pre_weight=None, pre_bias=None, post_weight=None,
                     post_bias=None, gate=None, cu=None, pre="rms", post="none", alpha=1.0, beta=1.0,
                     eps=1e-6, stream=None):
    """r = alpha x + beta gate post(y), h = pre(r) (see gs.h).  x, y, r_out, h_out: [tokens, width]
    float32 or bfloat16, any row stride; y and r_out may be None, h_out is None with pre "none".
    pre and post: "none", "rms" or "layer"; weights, biases and gate float32 or None; gate [width],
    or [batch, width] with cu, the int32 offsets [batch + 1] of its sequences."""
    st = (_calls or _token_calls()).residual_norm(
        x, y, r_out, h_out, pre_weight, pre_bias, post_weight, post_bias, gate, cu,
        _norm_kind("pre", pre), _norm_kind("post", post), alpha, beta, eps, stream)
    if st:
        _check("gs_residual_norm", st)


def gs_residual_norm_workspace_bytes(tokens, width, batch=1) -> int:
    return int(library().gs_residual_norm_workspace_bytes(int(tokens), int(width), int(batch)))


def gs_residual_norm_bwd(x, y, dr_out, dh_out, dx, dy, workspace, pre_weight=None, pre_bias=None,
                         post_weight=None, post_bias=None, gate=None, cu=None, pre="rms",
                         post="none", alpha=1.0, beta=1.0, eps=1e-6, dpre_weight=None,
                         dpre_bias=None, dpost_weight=None, dpost_bias=None, dgate=None,
                         stream=None):
    """Gradient of gs_residual_norm from its inputs x and y and the gradients of r_out (None = 0)
    and h_out (see gs.h); gradients of weights, biases and gate that are None are not wanted."""
    st = (_calls or _token_calls()).residual_norm_bwd(
        x, y, dr_out, dh_out, dx, dy, workspace, pre_weight, pre_bias, post_weight, post_bias, gate,
        cu, _norm_kind("pre", pre), _norm_kind("post", post), alpha, beta, eps, dpre_weight,
        dpre_bias, dpost_weight, dpost_bias, dgate, stream)
    if st:
        _check("gs_residual_norm_bwd", st)


def gs_clip_grad_norm_workspace_bytes(count) -> int:
    return int(library().gs_clip_grad_norm_workspace_bytes(int(count)))


def gs_clip_grad_norm(grads, max_norm, norm, workspace, outs=None, stream=None):
    """The norm over all of grads, a list of contiguous float32 or bfloat16 tensors, into norm
    (float32 [1]), and the gradients scaled to at most max_norm into outs, tensors of the same
    sizes and types (None: in place); see gs.h.  A finite max_norm beyond float32 counts as its
    largest number."""
    st = (_calls or _token_calls()).clip_grad_norm(grads, max_norm, norm, workspace, outs, stream)
    if st:
        _check("gs_clip_grad_norm", st)


def gs_raster_stats(workspace, stream=None) -> dict:
    out = (C.c_int64 * 16)()
    st = library().gs_raster_stats(_ptr(workspace, "workspace"), workspace.numel(), out,
                                   _stream(stream))
    _check("gs_raster_stats", st)
    return {"h": out[0], "k": out[1], "resident_ctas": out[2], "work_items": out[3],
            "device_error": out[4], "n_max": out[5], "n_min_nonempty": out[6],
            "n_total": out[7], "nonempty_tiles": out[8], "batches_tiles": out[9],
            "batches_chunks": out[10], "batches_skipped_on_flag": out[11],
            "batches_skipped_done": out[12], "batches_discarded": out[13]}


# ---------------------------------------------------------------------------
# convenience: one view, buffers allocated with torch
# ---------------------------------------------------------------------------
@dataclass
class Grads:
    means: "object"
    scales: "object"
    quats: "object"
    opacities: "object"
    sh: "object"


class Rasterizer:
    """Owns the device buffers of one view and runs the five calls in order.

    forward(means, scales, quats, opacities, sh) -> (image [H, W, 3], t_final [H, W])
    backward(dL_dimage, dL_dt_final=None) -> Grads
    Tensors are float32 CUDA tensors of the shapes documented in gs.h.
    """

    def __init__(self, cam, sh_degree: int, n: int, capacity: int | None = None,
                 settings: Settings | None = None, device="cuda"):
        import torch

        self.cam = Camera.of(cam)
        self.sh_degree = int(sh_degree)
        self.n = int(n)
        self.settings = settings if settings is not None else gs_default_settings()
        self.device = torch.device(device)
        W, H = self.cam.width, self.cam.height
        self.n_tiles = int(library().gs_num_tiles(W, H))
        dev, f, i = self.device, torch.float32, torch.int32
        self.splats = torch.empty((self.n, SPLAT_FLOATS), dtype=f, device=dev)
        self.depths = torch.empty(self.n, dtype=f, device=dev)
        self.radii = torch.empty((self.n, 2), dtype=i, device=dev)
        self.tiles_touched = torch.empty(self.n, dtype=i, device=dev)
        self.tile_ranges = torch.empty((self.n_tiles, 2), dtype=i, device=dev)
        self.lpt_order = torch.empty(self.n_tiles, dtype=i, device=dev)
        self.counts = torch.zeros(2, dtype=torch.int64, device=dev)
        self.image = torch.empty((H, W, 3), dtype=f, device=dev)
        self.t_final = torch.empty((H, W), dtype=f, device=dev)
        self.n_contrib = torch.empty((H, W), dtype=i, device=dev)
        self.last_idx = torch.empty((H, W), dtype=i, device=dev)
        self.grad2d = torch.empty((self.n, GRAD2D), dtype=f, device=dev)
        self.touched = torch.empty(self.n, dtype=torch.uint8, device=dev)
        self._alloc_pairs(capacity if capacity else max(4 * self.n, 1 << 16))
        self.n_pairs = None
        self._inputs = None

    def _alloc_pairs(self, capacity: int):
        import torch

        self.capacity = int(capacity)
        self.sorted_ids = torch.empty(self.capacity, dtype=torch.int32, device=self.device)
        self.bin_ws = torch.empty(gs_bin_sort_workspace_bytes(self.n, self.capacity, self.cam.width,
                                                              self.cam.height),
                                  dtype=torch.uint8, device=self.device)
        self.raster_ws = torch.empty(gs_raster_workspace_bytes(self.cam.width, self.cam.height,
                                                               self.capacity, self.settings),
                                     dtype=torch.uint8, device=self.device)

    def forward(self, means, scales, quats, opacities, sh, sync_pairs: bool = True):
        n = self.n
        # SH coefficients as torch.bfloat16 take the bfloat16-storage calls
        project = gs_project_sh16 if _is_bf16(sh) else gs_project
        project(self.cam, n, self.sh_degree, means, scales, quats, opacities, sh, self.splats,
                self.depths, self.radii, self.tiles_touched)
        while True:
            try:
                self.n_pairs = gs_bin_sort(self.cam, n, self.splats, self.depths,
                                           self.tiles_touched, self.bin_ws, self.sorted_ids,
                                           self.capacity, self.tile_ranges, self.lpt_order,
                                           self.counts, sync_pairs=sync_pairs)
                break
            except GSError as e:
                if e.status != 3:
                    raise
                self._alloc_pairs(int(self._needed(e) * 1.25) + 1)
        gs_rasterize_fwd(self.cam, n, self.splats, self.sorted_ids, self.tile_ranges,
                         self.lpt_order, self.raster_ws, self.image, self.t_final, self.n_contrib,
                         self.last_idx, self.settings)
        self._inputs = (means, scales, quats, opacities, sh)
        return self.image, self.t_final

    @staticmethod
    def _needed(e: GSError) -> int:
        return int(str(e).rsplit("pairs needed:", 1)[1].strip())

    def backward(self, dL_dimage, dL_dt_final=None) -> Grads:
        import torch

        n, K = self.n, (self.sh_degree + 1) ** 2
        means, scales, quats, opacities, sh = self._inputs
        gs_rasterize_bwd(self.cam, n, self.splats, self.sorted_ids, self.tile_ranges,
                         self.lpt_order, self.raster_ws, self.t_final, self.last_idx, dL_dimage,
                         dL_dt_final, self.grad2d, self.touched, self.settings)
        dev, f = self.device, torch.float32
        g = Grads(torch.empty((n, 3), dtype=f, device=dev), torch.empty((n, 3), dtype=f, device=dev),
                  torch.empty((n, 4), dtype=f, device=dev), torch.empty(n, dtype=f, device=dev),
                  torch.empty((n, K, 3), dtype=f, device=dev))
        project_bwd = gs_project_bwd_sh16 if _is_bf16(sh) else gs_project_bwd
        project_bwd(self.cam, n, self.sh_degree, means, scales, quats, opacities, sh,
                    self.tiles_touched, self.grad2d, self.touched, g.means, g.scales, g.quats,
                    g.opacities, g.sh)
        return g

    def stats(self) -> dict:
        return gs_raster_stats(self.raster_ws)
