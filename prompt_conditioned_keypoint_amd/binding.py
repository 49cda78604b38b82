"""ctypes binding of libgkdhead (the GKDT detection head on gfx950).

Argument marshalling only: shape/dtype/device checks, output allocation
with torch, and the call through the C ABI declared in include/gkdhead.h.
Every step of the computation runs in the library's HIP kernels. There is
no fallback: if libgkdhead.so is missing or a call fails, this module
raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgkdhead.so")

GKD_DTYPE_F32, GKD_DTYPE_BF16 = 0, 1
GKD_ABI_VERSION = 9          # include/gkdhead.h
GKD_KG_STATIC_WORKSPACE_BYTES = 64 << 20  # the no-allocation KG call's static workspace
GKD_HEATMAP_BF16 = 0x1       # gkd_kernel_heatmap flag: bfloat16 heatmaps
GKD_UPSAMPLE_CORNERS = 0x2   # gkd_kernel_heatmap flag: align_corners=True upsample
GKD_COORDS_CORNERS = 0x4     # decode flag: corner-aligned -1..1 coordinates
GKD_QUERY_TOKENS = 0x8       # query as [B, skip + H*W, C] tokens; skip in bits 8..15
GKD_TOKENS_VERSION = 1       # include/gkdtokens.h
GKD_ROPE_INTERLEAVED = 0x1   # gkd_qk_norm_rope flag: pairs (2i, 2i + 1)
GKD_ATTN_CAUSAL = 0x1        # gkd_prefix_attention flag: own keys up to the query's place
GKD_FP4_VERSION = 1          # include/gkdfp4.h
GKD_ACTS = {"none": 0, "relu": 1, "gelu": 2, "quick_gelu": 3, "silu": 4}
STATUS = {0: "GKD_OK", 1: "GKD_ERR_NULL", 2: "GKD_ERR_SHAPE", 3: "GKD_ERR_DTYPE",
          4: "GKD_ERR_VALUE", 5: "GKD_ERR_UNSUPPORTED", 6: "GKD_ERR_HIP",
          7: "GKD_ERR_ALIGN"}

_lib = None
_P, _I, _U32, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint32, ctypes.c_float


class GkdHeads(ctypes.Structure):
    """gkd_heads: data pointer and element strides of a [B,T,H,D] operand."""
    _fields_ = [("data", _P), ("batch", ctypes.c_int64), ("token", ctypes.c_int64),
                ("head", ctypes.c_int64)]


class GkdCache(ctypes.Structure):
    """gkd_cache: a cache's arrays and sizes."""
    _fields_ = [("codes", _P), ("scales", _P), ("pages", _I), ("page", _I), ("Hk", _I), ("D", _I)]


class GkdError(RuntimeError):
    """A gkd_* call returned a non-OK status."""

    def __init__(self, status: int, text: str):
        self.status = status
        super().__init__(f"{STATUS.get(status, status)}: {text}")


def load():
    """Load libgkdhead.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -c 'import "
            "__graft_entry__ as g; g.build()'` (hipcc, gfx950)")
    lib = ctypes.CDLL(LIB_PATH)
    lib.gkd_abi_version.restype = _I
    lib.gkd_status_string.restype = ctypes.c_char_p
    lib.gkd_status_string.argtypes = [_I]
    lib.gkd_last_error.restype = ctypes.c_char_p
    lib.gkd_vkp_pool.restype = _I
    lib.gkd_vkp_pool.argtypes = [_P, _P, _P, _I, _I, _I, _I, _I, _F, _F, _I, _U32,
                                 _P, _P]
    lib.gkd_kernel_heatmap.restype = _I
    lib.gkd_kernel_heatmap.argtypes = [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I,
                                       _U32, _P, _P, _P, _P, _P]
    lib.gkd_peak_decode.restype = _I
    lib.gkd_peak_decode.argtypes = [_P, _P, _I, _I, _I, _I, _U32, _P, _P, _P, _P]
    lib.gkd_roi_preprocess.restype = _I
    lib.gkd_roi_preprocess.argtypes = [_P, _I, _I, _P, _I, _I, _I, _U32, _P, _P]
    lib.gkd_roi_backproject.restype = _I
    lib.gkd_roi_backproject.argtypes = [_P, _P, _I, _I, _I, _I, _I, _U32, _P, _P]
    lib.gkd_kg_workspace_size.restype = ctypes.c_size_t
    lib.gkd_kg_workspace_size.argtypes = [_I, _I, _I, _I, _I, _I, _U32]
    lib.gkd_kg_transformer.restype = _I
    lib.gkd_kg_transformer.argtypes = [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _I, _I, _I,
                                       _U32, _P, _P, ctypes.c_size_t, _P]
    lib.gkd_kg_transformer_noalloc.restype = _I
    lib.gkd_kg_transformer_noalloc.argtypes = [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _I,
                                               _I, _I, _U32, _P, _P]
    _L, _Z, _H = ctypes.c_int64, ctypes.c_size_t, _P  # _H: gkd_heads * or gkd_cache *
    lib.gkd_tokens_version.restype = _I
    lib.gkd_linear_workspace_size.restype = _Z
    lib.gkd_linear_workspace_size.argtypes = [_I, _I, _I, _L, _L]
    lib.gkd_linear.restype = _I
    lib.gkd_linear.argtypes = [_P, _L, _P, _L, _P, _P, _L, _I, _I, _I, _I, _I, _I, _U32, _P, _L,
                               _P, _Z, _P]
    lib.gkd_qk_norm_rope.restype = _I
    lib.gkd_qk_norm_rope.argtypes = [_H, _I, _H, _I, _I, _I, _I, _P, _L, _I, _P, _I, _P, _P, _F,
                                     _I, _U32, _H, _H, _P]
    lib.gkd_prefix_attention_workspace_size.restype = _Z
    lib.gkd_prefix_attention_workspace_size.argtypes = [_I] * 7
    lib.gkd_prefix_attention.restype = _I
    lib.gkd_prefix_attention.argtypes = [_H, _H, _H, _I, _H, _H, _I, _P, _P, _P, _I, _I, _I, _I,
                                         _I, _F, _I, _U32, _H, _P, _Z, _P]
    lib.gkd_fp4_version.restype = _I
    lib.gkd_quantize_fp4.restype = _I
    lib.gkd_quantize_fp4.argtypes = [_P, _L, _I, _I, _I, _U32, _P, _P, _P]
    lib.gkd_linear_fp4_workspace_size.restype = _Z
    lib.gkd_linear_fp4_workspace_size.argtypes = [_I] * 3
    lib.gkd_linear_fp4.restype = _I
    lib.gkd_linear_fp4.argtypes = [_P, _L, _P, _P, _P, _P, _L, _I, _I, _I, _I, _I, _U32, _P, _L,
                                   _P, _Z, _P]
    lib.gkd_cache_append.restype = _I
    lib.gkd_cache_append.argtypes = [_H, _H, _I, _I, _P, _P, _H, _P, _I, _I, _U32, _P]
    lib.gkd_cache_read.restype = _I
    lib.gkd_cache_read.argtypes = [_H, _P, _I, _I, _I, _P, _P, _U32, _H, _H, _P]
    lib.gkd_cache_attention_workspace_size.restype = _Z
    lib.gkd_cache_attention_workspace_size.argtypes = [_I] * 7
    lib.gkd_cache_attention.restype = _I
    lib.gkd_cache_attention.argtypes = [_H, _H, _P, _I, _P, _P, _I, _I, _I, _F, _U32, _H, _P, _Z,
                                        _P]
    if lib.gkd_abi_version() != GKD_ABI_VERSION:
        raise ImportError("libgkdhead ABI version mismatch")
    if lib.gkd_tokens_version() != GKD_TOKENS_VERSION:
        raise ImportError("libgkdhead token operators' version mismatch")
    if lib.gkd_fp4_version() != GKD_FP4_VERSION:
        raise ImportError("libgkdhead four-bit operators' version mismatch")
    _lib = lib
    return lib


def _check(status: int):
    if status != 0:
        raise GkdError(status, load().gkd_last_error().decode())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(dev):
    return torch.cuda.current_stream(dev).cuda_stream


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return GKD_DTYPE_F32
    if t.dtype == torch.bfloat16:
        return GKD_DTYPE_BF16
    raise TypeError(f"features must be float32 or bfloat16, got {t.dtype}")


def _dev(t: torch.Tensor, name: str, dtype=None, ndim=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    return t


def vkp_pool(support: torch.Tensor, kpts: torch.Tensor, kpt_valid: torch.Tensor,
             stride: float = 16.0, sigma: float = 14.0,
             out: torch.Tensor | None = None, token_hw=None,
             token_skip: int = 0) -> torch.Tensor:
    """support [B,C,H,W] (f32|bf16), kpts [B,R,2] f32 px, kpt_valid [B,R] u8
    -> protos [B,R,C] in the support dtype (rows with kpt_valid == 0 are
    left as they are in `out`). token_hw=(H, W): the support map is the
    ViT's token sequence [B, token_skip + H*W, C] (GKD_QUERY_TOKENS)."""
    lib = load()
    if token_hw is None:
        _dev(support, "support", ndim=4)
        B, C, H, W = support.shape
        flags = 0
    else:
        _dev(support, "support", ndim=3)
        H, W = (int(v) for v in token_hw)
        B, T, C = support.shape
        if not 0 <= token_skip <= 255 or T != token_skip + H * W:
            raise ValueError("support must be [B, token_skip + H*W, C] with 0 <= token_skip <= 255")
        flags = GKD_QUERY_TOKENS | (token_skip << 8)
    _dev(kpts, "kpts", torch.float32, 3)
    _dev(kpt_valid, "kpt_valid", torch.uint8, 2)
    R = kpt_valid.shape[1]
    if kpts.shape != (B, R, 2) or kpt_valid.shape != (B, R):
        raise ValueError("kpts must be [B,R,2] and kpt_valid [B,R]")
    if out is None:
        out = torch.empty((B, R, C), dtype=support.dtype, device=support.device)
    _dev(out, "out", support.dtype)
    if out.shape != (B, R, C):
        raise ValueError("out must be [B,R,C]")
    _check(lib.gkd_vkp_pool(_ptr(support), _ptr(kpts), _ptr(kpt_valid), B, C, H, W, R,
                            float(stride), float(sigma), _dtype_code(support), flags,
                            _ptr(out), _stream(support.device)))
    return out


def kernel_heatmap(query: torch.Tensor, kern_vis=None, mask_vis=None, kern_txt=None,
                   mask_txt=None, decode: bool = True, out=None, out_decode=None,
                   heat_dtype=torch.float32, with_heatmaps: bool = True,
                   coords: str = "centres", align_corners: bool = False,
                   token_hw=None, token_skip: int = 0):
    """query [B,C,H,W] (f32|bf16); kern_* [B,R,C] in the query dtype with
    mask_* [B,R] u8 (None = modality absent).

    Returns heatmaps [B,R,4H,4W] in heat_dtype (float32, or bfloat16 via
    the GKD_HEATMAP_BF16 flag) and, if decode, (idx [B,R] i32, xy [B,R,2]
    f32, score [B,R] f32). Rows with no mask set are not written (they keep
    whatever `out` held). with_heatmaps=False computes the keypoints only
    (heatmaps NULL in the C call; decode must be True) and returns
    (idx, xy, score). coords: "centres" or "corners" (GKD_COORDS_CORNERS);
    align_corners: upsample on the align_corners=True grid
    (GKD_UPSAMPLE_CORNERS). token_hw=(H, W): the query is the ViT's token
    sequence [B, token_skip + H*W, C] (GKD_QUERY_TOKENS)."""
    lib = load()
    if token_hw is None:
        _dev(query, "query", ndim=4)
        B, C, H, W = query.shape
    else:
        _dev(query, "query", ndim=3)
        H, W = (int(v) for v in token_hw)
        B, T, C = query.shape
        if not 0 <= token_skip <= 255 or T != token_skip + H * W:
            raise ValueError("query must be [B, token_skip + H*W, C] with 0 <= token_skip <= 255")
    R = None
    for k, m, name in ((kern_vis, mask_vis, "vis"), (kern_txt, mask_txt, "txt")):
        if (k is None) != (m is None):
            raise ValueError(f"kern_{name} and mask_{name} go together")
        if k is not None:
            _dev(k, f"kern_{name}", query.dtype, 3)
            _dev(m, f"mask_{name}", torch.uint8, 2)
            if R is None:
                R = m.shape[1]
            if k.shape != (B, R, C) or m.shape != (B, R):
                raise ValueError(f"kern_{name} must be [B,R,C], mask_{name} [B,R]")
    if R is None:
        raise ValueError("at least one prompt modality is required")
    if heat_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"heat_dtype must be float32 or bfloat16, got {heat_dtype}")
    flags = ((GKD_HEATMAP_BF16 if heat_dtype == torch.bfloat16 else 0) | _coords_flag(coords) |
             (GKD_UPSAMPLE_CORNERS if align_corners else 0) |
             (GKD_QUERY_TOKENS | (token_skip << 8) if token_hw is not None else 0))
    if not with_heatmaps:
        if not decode:
            raise ValueError("with_heatmaps=False needs decode=True")
        if out is not None:
            raise ValueError("with_heatmaps=False takes no heatmap buffer")
    elif out is None:
        out = torch.empty((B, R, 4 * H, 4 * W), dtype=heat_dtype, device=query.device)
    if out is not None:
        _dev(out, "out", heat_dtype)
        if out.shape != (B, R, 4 * H, 4 * W):
            raise ValueError("out must be [B,R,4H,4W]")
    idx = xy = score = None
    if decode:
        if out_decode is None:
            idx = torch.empty((B, R), dtype=torch.int32, device=query.device)
            xy = torch.empty((B, R, 2), dtype=torch.float32, device=query.device)
            score = torch.empty((B, R), dtype=torch.float32, device=query.device)
        else:
            idx, xy, score = out_decode
    _check(lib.gkd_kernel_heatmap(_ptr(query), _ptr(kern_vis), _ptr(mask_vis),
                                  _ptr(kern_txt), _ptr(mask_txt), B, C, H, W, R,
                                  _dtype_code(query), flags, _ptr(out), _ptr(idx), _ptr(xy),
                                  _ptr(score), _stream(query.device)))
    if not with_heatmaps:
        return idx, xy, score
    if decode:
        return out, (idx, xy, score)
    return out


def _coords_flag(coords: str) -> int:
    if coords not in ("centres", "corners"):
        raise ValueError("coords must be 'centres' or 'corners'")
    return GKD_COORDS_CORNERS if coords == "corners" else 0


def peak_decode(heat: torch.Tensor, row_valid: torch.Tensor | None = None,
                coords: str = "centres"):
    """heat [B,R,Ho,Wo] f32, row_valid [B,R] u8 or None -> (idx [B,R] i32,
    xy [B,R,2] f32, score [B,R] f32); invalid rows get (-1, NaN, -inf).
    coords: "centres" ((2x + 1)/Wo - 1) or "corners" (2x/(Wo - 1) - 1)."""
    lib = load()
    _dev(heat, "heat", torch.float32, 4)
    B, R, Ho, Wo = heat.shape
    if row_valid is not None:
        _dev(row_valid, "row_valid", torch.uint8, 2)
        if row_valid.shape != (B, R):
            raise ValueError("row_valid must be [B,R]")
    idx = torch.empty((B, R), dtype=torch.int32, device=heat.device)
    xy = torch.empty((B, R, 2), dtype=torch.float32, device=heat.device)
    score = torch.empty((B, R), dtype=torch.float32, device=heat.device)
    _check(lib.gkd_peak_decode(_ptr(heat), _ptr(row_valid), B, R, Ho, Wo, _coords_flag(coords),
                               _ptr(idx), _ptr(xy), _ptr(score), _stream(heat.device)))
    return idx, xy, score


def roi_preprocess(image: torch.Tensor, boxes: torch.Tensor, size: int = 384,
                   dtype=torch.float32, out: torch.Tensor | None = None) -> torch.Tensor:
    """image [H,W,3] u8 RGB, boxes [B,4] i32 (x0, y0, x1, y1) -> the
    backbone input [B,3,size,size] in dtype (float32 or bfloat16): each box
    cropped, resized so its longer side is `size`, centre-padded with the
    mean colour and ImageNet-normalised."""
    lib = load()
    _dev(image, "image", torch.uint8, 3)
    _dev(boxes, "boxes", torch.int32, 2)
    if image.shape[2] != 3 or boxes.shape[1] != 4:
        raise ValueError("image must be [H,W,3] and boxes [B,4]")
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("dtype must be float32 or bfloat16")
    B = boxes.shape[0]
    if out is None:
        out = torch.empty((B, 3, size, size), dtype=dtype, device=image.device)
    else:
        _dev(out, "out", dtype, 4)
        if out.shape != (B, 3, size, size):
            raise ValueError("out must be [B,3,size,size]")
    _check(lib.gkd_roi_preprocess(_ptr(image), image.shape[0], image.shape[1], _ptr(boxes), B,
                                  size, 1 if dtype == torch.bfloat16 else 0, 0, _ptr(out),
                                  _stream(image.device)))
    return out


def roi_backproject(xy: torch.Tensor, boxes: torch.Tensor, image_hw, size: int = 384,
                    out: torch.Tensor | None = None) -> torch.Tensor:
    """xy [B,R,2] f32 in the ROI canvas's -1..1 frame -> image coordinates
    [B,R,2] f32 (continuous, pixel i covers [i, i + 1)); NaN stays NaN."""
    lib = load()
    _dev(xy, "xy", torch.float32, 3)
    _dev(boxes, "boxes", torch.int32, 2)
    B, R, two = xy.shape
    if two != 2 or boxes.shape != (B, 4):
        raise ValueError("xy must be [B,R,2] and boxes [B,4]")
    if out is None:
        out = torch.empty_like(xy)
    else:
        _dev(out, "out", torch.float32, 3)
        if out.shape != xy.shape:
            raise ValueError("out must be [B,R,2]")
    _check(lib.gkd_roi_backproject(_ptr(xy), _ptr(boxes), B, R, int(image_hw[0]),
                                   int(image_hw[1]), size, 0, _ptr(out), _stream(xy.device)))
    return out


def kg_workspace_size(B: int, C: int, H: int, W: int, R: int, d_ff: int = 1024,
                      tokens: bool = False) -> int:
    """Bytes of workspace gkd_kg_transformer needs for these sizes."""
    return int(load().gkd_kg_workspace_size(B, C, H, W, R, d_ff,
                                            GKD_QUERY_TOKENS if tokens else 0))


def kg_transformer(query: torch.Tensor, weights: torch.Tensor, kern_vis=None, mask_vis=None,
                   kern_txt=None, mask_txt=None, n_blocks: int = 2, d_ff: int = 1024,
                   token_hw=None, token_skip: int = 0, out=None,
                   workspace=None) -> torch.Tensor:
    """Kernel-generation transformer: prototypes [B,R,C] bf16 (with their
    [B,R] u8 masks) -> kernels [2,B,R,C] bf16: out[0] from the visual slots,
    out[1] from the text slots, ready as the heatmap call's kern_vis and
    kern_txt.
    query [B,C,H,W] bf16, or with token_hw=(H, W) the token sequence
    [B, token_skip + H*W, C]; weights: the flat bf16 array. workspace: a
    uint8 CUDA tensor of at least kg_workspace_size() bytes (allocated here
    when None), or "static" for gkd_kg_transformer_noalloc (the library's
    static workspace of GKD_KG_STATIC_WORKSPACE_BYTES per GPU; nothing is
    allocated by the call, `out` included when it is given)."""
    lib = load()
    if token_hw is None:
        _dev(query, "query", torch.bfloat16, 4)
        B, C, H, W = query.shape
        flags = 0
    else:
        _dev(query, "query", torch.bfloat16, 3)
        H, W = (int(v) for v in token_hw)
        B, T, C = query.shape
        if not 0 <= token_skip <= 255 or T != token_skip + H * W:
            raise ValueError("query must be [B, token_skip + H*W, C] with 0 <= token_skip <= 255")
        flags = GKD_QUERY_TOKENS | (token_skip << 8)
    _dev(weights, "weights", torch.bfloat16, 1)
    masks = [m for m in (mask_vis, mask_txt) if m is not None]
    if not masks:
        raise ValueError("give mask_vis, mask_txt or both")
    R = masks[0].shape[1]
    for k, m, name in ((kern_vis, mask_vis, "vis"), (kern_txt, mask_txt, "txt")):
        if m is None:
            continue
        _dev(m, "mask_" + name, torch.uint8, 2)
        _dev(k, "kern_" + name, torch.bfloat16, 3)
        if m.shape != (B, R) or k.shape != (B, R, C):
            raise ValueError(f"kern_{name} must be [B,R,C] and mask_{name} [B,R]")
    if out is None:
        out = torch.empty((2, B, R, C), dtype=torch.bfloat16, device=query.device)
    _dev(out, "out", torch.bfloat16, 4)
    if out.shape != (2, B, R, C):
        raise ValueError("out must be [2,B,R,C]")
    args = (_ptr(kern_vis) if mask_vis is not None else None, _ptr(mask_vis),
            _ptr(kern_txt) if mask_txt is not None else None, _ptr(mask_txt), _ptr(query),
            B, C, H, W, R, _ptr(weights), n_blocks, d_ff, 1, flags, _ptr(out))
    if workspace == "static":
        # no workspace argument: the library's own static device array
        _check(lib.gkd_kg_transformer_noalloc(*args, _stream(query.device)))
        return out
    need = int(lib.gkd_kg_workspace_size(B, C, H, W, R, d_ff, flags))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=query.device)
    _dev(workspace, "workspace", torch.uint8, 1)
    _check(lib.gkd_kg_transformer(*args, _ptr(workspace), workspace.numel(),
                                  _stream(query.device)))
    return out


# torch's own short cuts, where it has them (0.08 and 0.13 us; the public calls
# take 1.18 and 0.25)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _place(t, name):
    """Device index of a GPU tensor, which must be the current device (where
    kernels are launched)."""
    dev = t.get_device()  # -1 without a GPU's memory
    if dev < 0:
        raise ValueError(f"{name} must be a GPU tensor")
    if dev != _current_device():
        raise ValueError(f"{name} is on cuda:{dev}, the current device is "
                         f"cuda:{_current_device()}")
    return dev


def _beside(dev, t, name):
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")


def _dense(dev, t, name, dtype, shape):
    """The address of a contiguous tensor of this type and shape."""
    if t.get_device() != dev or t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        _dev(t, name, dtype, len(shape))
        _beside(dev, t, name)
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _heads(dev, t, name, dtype, ndim=4):
    """A [B,T,H,D] (ndim 3: [T,H,D]) operand with any strides but adjacent
    head elements, as the four fields of gkd_heads."""
    if t.get_device() != dev:
        _beside(dev, t, name)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    st = t.stride()
    if len(st) != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    if st[-1] != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}: the elements of a head must be adjacent")
    if ndim == 4:
        return t.data_ptr(), st[0], st[1], st[2]
    return t.data_ptr(), 0, st[0], st[1]


_NO_HEADS = (0, 0, 0, 0)
_HEADS_BYTES = ctypes.sizeof(GkdHeads)
_pack4, _pack6 = struct.Struct("16q").pack_into, struct.Struct("24q").pack_into  # gkd_heads
_pack_cached = struct.Struct("8q2q4i").pack_into  # two gkd_heads and a gkd_cache


class _Records(threading.local):
    """Each thread's place for a call's gkd_heads, which are read before the
    call returns."""

    def __init__(self):
        self.buf = ctypes.create_string_buffer(6 * _HEADS_BYTES)
        self.at = ctypes.addressof(self.buf)


_records = _Records()


def _int_sizes(fn, *sizes):
    """The C ABI takes sizes as ints, and ctypes would cut larger ones short."""
    if max(sizes) > 0x7fffffff:
        raise GkdError(2, f"{fn}: a size does not fit 32 bits: {sizes}")


def _workspace(workspace, need, dev):
    if need == 0:
        return None, 0
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev), need
    _dev(workspace, "workspace", torch.uint8, 1)
    _beside(dev, workspace, "workspace")
    return workspace, workspace.numel()


def _row_stride(t, name):
    """Row stride of a [..., n] tensor whose rows are evenly spaced."""
    shape = t.shape
    if t.is_contiguous():
        return shape[-1]
    st = t.stride()
    if shape[-1] > 1 and st[-1] != 1:
        raise ValueError(f"{name}: the elements of a row must be adjacent")
    if len(shape) == 2:
        return st[0] if shape[0] != 1 else shape[1]
    ld, span = None, 1
    for size, step in zip(reversed(shape[:-1]), reversed(st[:-1])):
        if size == 1:
            continue
        if ld is None:
            ld = step
        elif step != ld * span:
            raise ValueError(f"{name}: its rows must be evenly spaced")
        span *= size
    return shape[-1] if ld is None else ld


def linear_workspace_size(M: int, N: int, K: int, ldx: int | None = None,
                          ldw: int | None = None) -> int:
    """Bytes of workspace gkd_linear needs for these sizes and row strides."""
    _int_sizes("gkd_linear_workspace_size", M, N, K)
    return int(load().gkd_linear_workspace_size(M, N, K, K if ldx is None else ldx,
                                                K if ldw is None else ldw))


def linear(x: torch.Tensor, weight: torch.Tensor, bias=None, residual=None, act: str = "none",
           out_dtype=None, out=None, workspace=None) -> torch.Tensor:
    """act(x @ weight.T + bias) + residual: x [..., K] bf16, weight [N, K]
    bf16, bias [N] bf16, residual [..., N] in the output's dtype (bf16, or
    float32 by out_dtype, out or residual) -> [..., N]. Rows may be strided,
    evenly over all leading axes (of tokens [B, 5 + H*W, C] with B > 1, take
    them all, or each sequence's); x and weight start on 16-byte places.
    act: "none", "relu", "gelu", "quick_gelu" or "silu". `out` may be
    `residual` itself. workspace: a uint8 GPU tensor of at least
    linear_workspace_size() bytes (allocated here when None)."""
    lib = _lib or load()
    dev = _place(x, "x")
    if weight.get_device() != dev:
        _beside(dev, weight, "weight")
    bf16 = torch.bfloat16
    if x.dtype != bf16 or weight.dtype != bf16:
        raise TypeError(f"x and weight must be bfloat16, got {x.dtype} and {weight.dtype}")
    lead, wshape = x.shape, weight.shape
    if len(lead) < 1 or len(wshape) != 2 or lead[-1] != wshape[1]:
        raise ValueError(f"x must be [..., K] and weight [N, K], got {tuple(lead)} and "
                         f"{tuple(wshape)}")
    code = GKD_ACTS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {sorted(GKD_ACTS)}")
    N, K = wshape
    lead = lead[:-1]
    M = lead.numel()
    _int_sizes("gkd_linear", M, N, K)
    shape = lead + (N,)
    if out_dtype is None:
        out_dtype = (out.dtype if out is not None else
                     residual.dtype if residual is not None else bf16)
    if out_dtype != bf16 and out_dtype != torch.float32:
        raise TypeError(f"out_dtype must be bfloat16 or float32, got {out_dtype}")
    if out is None:
        out = x.new_empty(shape) if out_dtype == bf16 else x.new_empty(shape, dtype=out_dtype)
        ldo = N
    else:
        if out.get_device() != dev:
            _beside(dev, out, "out")
        if out.shape != shape or out.dtype != out_dtype:
            raise ValueError(f"out must be {tuple(shape)} of {out_dtype}")
        ldo = _row_stride(out, "out")
    rp = bp = None
    ldr = 0
    if residual is not None:
        if residual.get_device() != dev:
            _beside(dev, residual, "residual")
        if residual.shape != shape or residual.dtype != out_dtype:
            raise ValueError(f"residual must be {tuple(shape)} of {out_dtype}")
        rp, ldr = residual.data_ptr(), _row_stride(residual, "residual")
    if bias is not None:
        bp = _dense(dev, bias, "bias", bf16, (N,))
    ldx, ldw = _row_stride(x, "x"), _row_stride(weight, "weight")
    ws, ws_bytes = _workspace(workspace, lib.gkd_linear_workspace_size(M, N, K, ldx, ldw), dev)
    status = lib.gkd_linear(x.data_ptr(), ldx, weight.data_ptr(), ldw, bp, rp, ldr, M, N, K, code,
                            1, 1 if out_dtype == bf16 else 0, 0, out.data_ptr(), ldo,
                            None if ws is None else ws.data_ptr(), ws_bytes, _raw_stream(dev))
    if status:
        _check(status)
    return out


def qk_norm_rope(q: torch.Tensor, k, pos: torch.Tensor, freqs: torch.Tensor, q_weight=None,
                 k_weight=None, eps: float = 1e-6, interleaved: bool = False, q_out=None,
                 k_out=None):
    """Head norm and rotary positions in one pass: q [B,T,Hq,D] and k
    [B,T,Hk,D] (or None), float32 or bf16, strided views welcome; pos
    [T,n_axes] or [B,T,n_axes] float32; freqs [n_axes, rot/2] float32 (0
    where a frequency does not belong to an axis); q_weight, k_weight [D] or
    None (no norm). Returns (q_out, k_out), new and dense unless given; an
    output may be its input (in place)."""
    lib = _lib or load()
    dev, dtype = _place(q, "q"), q.dtype
    code = _dtype_code(q)
    hq = _heads(dev, q, "q", dtype)
    B, T, Hq, D = q.shape
    Hk, hk, hko = 0, _NO_HEADS, _NO_HEADS
    if k is not None:
        hk = _heads(dev, k, "k", dtype)
        Hk = k.shape[2]
        if k.shape != (B, T, Hk, D) or Hk < 1:
            raise ValueError(f"k must be [B,T,Hk,D], got {tuple(k.shape)}")
    elif k_out is not None:
        raise ValueError("k_out without k")
    if freqs.dim() != 2:
        raise ValueError(f"freqs must be [n_axes, rot/2], got {tuple(freqs.shape)}")
    A, half = freqs.shape
    _int_sizes("gkd_qk_norm_rope", B, T, Hq, Hk, D, A, 2 * half)
    pf = _dense(dev, freqs, "freqs", torch.float32, (A, half))
    own_pos = pos.dim() == 3
    pp = _dense(dev, pos, "pos", torch.float32, (B, T, A) if own_pos else (T, A))
    pwq = None if q_weight is None else _dense(dev, q_weight, "q_weight", dtype, (D,))
    pwk = None if k_weight is None else _dense(dev, k_weight, "k_weight", dtype, (D,))
    if q_out is None:
        q_out = q.new_empty((B, T, Hq, D))
        hqo = (q_out.data_ptr(), T * Hq * D, Hq * D, D)
    else:
        hqo = _heads(dev, q_out, "q_out", dtype)
        if q_out.shape != q.shape:
            raise ValueError("q_out must have q's shape")
    if k is not None:
        if k_out is None:
            k_out = q.new_empty((B, T, Hk, D))
            hko = (k_out.data_ptr(), T * Hk * D, Hk * D, D)
        else:
            hko = _heads(dev, k_out, "k_out", dtype)
            if k_out.shape != k.shape:
                raise ValueError("k_out must have k's shape")
    rec = _records
    at = rec.at
    _pack4(rec.buf, 0, *hq, *hk, *hqo, *hko)
    status = lib.gkd_qk_norm_rope(at, Hq, at + _HEADS_BYTES if Hk else None, Hk, B, T, D,
                                  pp, T * A if own_pos else 0, A, pf, 2 * half, pwq, pwk, eps,
                                  code, GKD_ROPE_INTERLEAVED if interleaved else 0,
                                  at + 2 * _HEADS_BYTES, at + 3 * _HEADS_BYTES if Hk else None,
                                  _raw_stream(dev))
    if status:
        _check(status)
    return q_out, k_out


def prefix_attention_workspace_size(B: int, Tq: int, Hq: int, Hk: int, D: int, P: int,
                                    S: int) -> int:
    """Bytes of workspace gkd_prefix_attention needs for these sizes."""
    _int_sizes("gkd_prefix_attention_workspace_size", B, Tq, Hq, Hk, D, P, S)
    return int(load().gkd_prefix_attention_workspace_size(B, Tq, Hq, Hk, D, P, S))


def prefix_attention(q: torch.Tensor, k_prefix=None, v_prefix=None, k_own=None, v_own=None,
                     own_len=None, q_len=None, own_mask=None, causal: bool = False, scale=None,
                     out=None, workspace=None) -> torch.Tensor:
    """Attention of q [B,Tq,Hq,D] bf16 over a prefix k_prefix, v_prefix
    [P,Hk,D] shared by the batch and each sequence's own keys k_own, v_own
    [B,S,Hk,D] (either pair may be None), of which the first own_len[b]
    (int32) with own_mask[b,j] (uint8) set count. causal: the q_len[b]
    (int32, default Tq) queries are the last of the own_len[b] own tokens and
    see own keys up to their place. Queries past q_len[b] are not computed:
    their rows of a given `out` stay as they are, those of a new one are zeros.
    scale: default D**-0.5. Returns out [B,Tq,Hq,D]; a query without keys gives
    zeros."""
    lib = _lib or load()
    bf16 = torch.bfloat16
    dev = _place(q, "q")
    hq = _heads(dev, q, "q", bf16)
    B, Tq, Hq, D = q.shape
    if (k_prefix is None) != (v_prefix is None) or (k_own is None) != (v_own is None):
        raise ValueError("keys and values go together")
    P = S = 0
    Hk = None
    kp = vp = ko = vo = _NO_HEADS
    if k_prefix is not None:
        kp = _heads(dev, k_prefix, "k_prefix", bf16, 3)
        vp = _heads(dev, v_prefix, "v_prefix", bf16, 3)
        P, Hk, d = k_prefix.shape
        if d != D or v_prefix.shape != k_prefix.shape:
            raise ValueError("k_prefix and v_prefix must be [P,Hk,D]")
    if k_own is not None:
        ko, vo = _heads(dev, k_own, "k_own", bf16), _heads(dev, v_own, "v_own", bf16)
        b, S, h, d = k_own.shape
        Hk = h if Hk is None else Hk
        if b != B or h != Hk or d != D or v_own.shape != k_own.shape:
            raise ValueError("k_own and v_own must be [B,S,Hk,D]")
    if Hk is None:
        raise ValueError("give prefix keys, own keys or both")
    _int_sizes("gkd_prefix_attention", B, Tq, Hq, Hk, D, P, S)
    pol = None if own_len is None else _dense(dev, own_len, "own_len", torch.int32, (B,))
    pql = None if q_len is None else _dense(dev, q_len, "q_len", torch.int32, (B,))
    pm = None if own_mask is None else _dense(dev, own_mask, "own_mask", torch.uint8, (B, S))
    if out is None:
        out = q.new_empty((B, Tq, Hq, D)) if q_len is None else q.new_zeros((B, Tq, Hq, D))
    ho = _heads(dev, out, "out", bf16)
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    ws, ws_bytes = _workspace(workspace, lib.gkd_prefix_attention_workspace_size(
        B, Tq, Hq, Hk, D, P, S), dev)
    rec = _records
    at = rec.at
    _pack6(rec.buf, 0, *hq, *kp, *vp, *ko, *vo, *ho)
    n = _HEADS_BYTES
    status = lib.gkd_prefix_attention(at, at + n, at + 2 * n, P, at + 3 * n, at + 4 * n, S,
                                      pol, pql, pm, B, Tq, Hq, Hk, D,
                                      D ** -0.5 if scale is None else scale, 1,
                                      GKD_ATTN_CAUSAL if causal else 0, at + 5 * n,
                                      None if ws is None else ws.data_ptr(), ws_bytes,
                                      _raw_stream(dev))
    if status:
        _check(status)
    return out


def _codes(dev, codes, scales, shape):
    """Addresses of the codes [..., n/2] and scale bytes [..., n/32] of values
    of this shape."""
    n = shape[-1]
    return (_dense(dev, codes, "codes", torch.uint8, shape[:-1] + (n // 2,)),
            _dense(dev, scales, "scales", torch.uint8, shape[:-1] + (n // 32,)))


def quantize_fp4(x: torch.Tensor, codes=None, scales=None):
    """Values x [..., K] (float32 or bf16, K a multiple of 32) as four-bit codes
    [..., K/2] and scale bytes [..., K/32], both uint8: value = code * 2^(scale -
    127), codes of 0, 0.5, 1, 1.5, 2, 3, 4 and 6 with a sign, a byte's low half
    the earlier one. Rows may be strided, evenly over all leading axes, and start
    on 16-byte places. A weight is laid out so once, for linear_fp4."""
    lib = _lib or load()
    dev = _place(x, "x")
    code = _dtype_code(x)
    if x.dim() < 1 or x.shape[-1] % 32 != 0 or x.shape[-1] == 0:
        raise ValueError(f"x must be [..., K] with K a multiple of 32, got {tuple(x.shape)}")
    lead, K = x.shape[:-1], x.shape[-1]
    N = lead.numel()
    _int_sizes("gkd_quantize_fp4", N, K)
    if codes is None:
        codes = x.new_empty(lead + (K // 2,), dtype=torch.uint8)
    if scales is None:
        scales = x.new_empty(lead + (K // 32,), dtype=torch.uint8)
    pc, ps = _codes(dev, codes, scales, x.shape)
    status = lib.gkd_quantize_fp4(x.data_ptr(), _row_stride(x, "x"), N, K, code, 0, pc, ps,
                                  _raw_stream(dev))
    if status:
        _check(status)
    return codes, scales


def linear_fp4_workspace_size(M: int, N: int, K: int) -> int:
    """Bytes of workspace gkd_linear_fp4 needs for these sizes."""
    _int_sizes("gkd_linear_fp4_workspace_size", M, N, K)
    return int(load().gkd_linear_fp4_workspace_size(M, N, K))


def linear_fp4(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, bias=None,
               residual=None, act: str = "none", out_dtype=None, out=None,
               workspace=None) -> torch.Tensor:
    """act(x @ weight.T + bias) + residual with the weight [N, K] as quantize_fp4
    leaves it: codes [N, K/2] and scales [N, K/32], uint8. x [..., K] bf16 (rows
    evenly spaced and on 16-byte places), bias [N] bf16, residual [..., N] in the
    output's dtype (bf16, or float32 by out_dtype, out or residual) -> [..., N].
    act, out and workspace as linear's (linear_fp4_workspace_size() bytes)."""
    lib = _lib or load()
    dev = _place(x, "x")
    bf16 = torch.bfloat16
    if x.dtype != bf16:
        raise TypeError(f"x must be bfloat16, got {x.dtype}")
    lead, cshape = x.shape, codes.shape
    if len(lead) < 1 or len(cshape) != 2 or lead[-1] != 2 * cshape[1]:
        raise ValueError(f"x must be [..., K] and codes [N, K/2], got {tuple(lead)} and "
                         f"{tuple(cshape)}")
    act_code = GKD_ACTS.get(act)
    if act_code is None:
        raise ValueError(f"act must be one of {sorted(GKD_ACTS)}")
    N, K = cshape[0], lead[-1]
    lead = lead[:-1]
    M = lead.numel()
    _int_sizes("gkd_linear_fp4", M, N, K)
    pc, ps = _codes(dev, codes, scales, (N, K))
    shape = lead + (N,)
    if out_dtype is None:
        out_dtype = (out.dtype if out is not None else
                     residual.dtype if residual is not None else bf16)
    if out_dtype != bf16 and out_dtype != torch.float32:
        raise TypeError(f"out_dtype must be bfloat16 or float32, got {out_dtype}")
    if out is None:
        out = x.new_empty(shape) if out_dtype == bf16 else x.new_empty(shape, dtype=out_dtype)
        ldo = N
    else:
        if out.get_device() != dev:
            _beside(dev, out, "out")
        if out.shape != shape or out.dtype != out_dtype:
            raise ValueError(f"out must be {tuple(shape)} of {out_dtype}")
        ldo = _row_stride(out, "out")
    rp = bp = None
    ldr = 0
    if residual is not None:
        if residual.get_device() != dev:
            _beside(dev, residual, "residual")
        if residual.shape != shape or residual.dtype != out_dtype:
            raise ValueError(f"residual must be {tuple(shape)} of {out_dtype}")
        rp, ldr = residual.data_ptr(), _row_stride(residual, "residual")
    if bias is not None:
        bp = _dense(dev, bias, "bias", bf16, (N,))
    ws, ws_bytes = _workspace(workspace, lib.gkd_linear_fp4_workspace_size(M, N, K), dev)
    status = lib.gkd_linear_fp4(x.data_ptr(), _row_stride(x, "x"), pc, ps, bp, rp, ldr, M, N, K,
                                act_code, 1 if out_dtype == bf16 else 0, 0, out.data_ptr(), ldo,
                                None if ws is None else ws.data_ptr(), ws_bytes, _raw_stream(dev))
    if status:
        _check(status)
    return out


def _cache(dev, codes, scales, table):
    """A cache's sizes (pages, page, Hk, D, L), its arrays' and its table's
    addresses, and the table's sequences."""
    shape = codes.shape
    if len(shape) != 5 or shape[1] != 2:
        raise ValueError(f"codes must be [pages, 2, Hk, page, D/2], got {tuple(shape)}")
    if table.dim() != 2:
        raise ValueError(f"table must be [B, L], got {tuple(table.shape)}")
    pages, _, Hk, page, half = shape
    B, L = table.shape
    pc, ps = _codes(dev, codes, scales, (pages, 2, Hk, page, 2 * half))
    return (pages, page, Hk, 2 * half, L), (pc, ps), _dense(dev, table, "table", torch.int32,
                                                           (B, L)), B


def cache_append(k: torch.Tensor, v: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                 table: torch.Tensor, start=None, count=None) -> None:
    """Quantises new tokens' k and v [B,T,Hk,D] (float32 or bf16, strided views
    welcome) into a cache's pages: codes [pages, 2, Hk, page, D/2] and scales
    [pages, 2, Hk, page, D/32], uint8, keys at [:, 0], values at [:, 1]; D 64 or
    128, page a multiple of 32. Token t < count[b] (int32, default T) of sequence
    b goes to place start[b] + t (int32, default 0), which is in row place % page
    of page table[b, place // page] (int32 [B, L]). Places past the table or
    without a page (an entry outside 0 .. pages - 1) are dropped; two tokens must
    not have the same place."""
    lib = _lib or load()
    dev = _place(k, "k")
    code = _dtype_code(k)
    hk, hv = _heads(dev, k, "k", k.dtype), _heads(dev, v, "v", k.dtype)
    sizes, arrays, pt, B = _cache(dev, codes, scales, table)
    pages, page, Hk, D, L = sizes
    T = k.shape[1]
    if k.shape != (B, T, Hk, D) or v.shape != k.shape:
        raise ValueError(f"k and v must be [{B}, T, {Hk}, {D}], got {tuple(k.shape)} and "
                         f"{tuple(v.shape)}")
    _int_sizes("gkd_cache_append", B, T, *sizes)
    pst = None if start is None else _dense(dev, start, "start", torch.int32, (B,))
    pct = None if count is None else _dense(dev, count, "count", torch.int32, (B,))
    rec = _records
    at = rec.at
    _pack_cached(rec.buf, 0, *hk, *hv, *arrays, pages, page, Hk, D)
    status = lib.gkd_cache_append(at, at + _HEADS_BYTES, B, T, pst, pct, at + 2 * _HEADS_BYTES, pt,
                                  L, code, 0, _raw_stream(dev))
    if status:
        _check(status)


def cache_read(codes: torch.Tensor, scales: torch.Tensor, table: torch.Tensor, T: int, start=None,
               count=None, k_out=None, v_out=None):
    """A cache's tokens in bfloat16: (k, v) [B,T,Hk,D] with the tokens at places
    start[b] + t, t < count[b]; zeros where there is no such place or page.
    Arguments as cache_append's. Tokens past count[b] of a given output stay as
    they are, those of a new one are zeros."""
    lib = _lib or load()
    dev = _place(codes, "codes")
    bf16 = torch.bfloat16
    sizes, arrays, pt, B = _cache(dev, codes, scales, table)
    pages, page, Hk, D, L = sizes
    _int_sizes("gkd_cache_read", B, T, *sizes)
    pst = None if start is None else _dense(dev, start, "start", torch.int32, (B,))
    pct = None if count is None else _dense(dev, count, "count", torch.int32, (B,))
    new = codes.new_empty if count is None else codes.new_zeros
    if k_out is None:
        k_out = new((B, T, Hk, D), dtype=bf16)
    if v_out is None:
        v_out = new((B, T, Hk, D), dtype=bf16)
    hk, hv = _heads(dev, k_out, "k_out", bf16), _heads(dev, v_out, "v_out", bf16)
    if k_out.shape != (B, T, Hk, D) or v_out.shape != (B, T, Hk, D):
        raise ValueError(f"k_out and v_out must be {(B, T, Hk, D)}")
    rec = _records
    at = rec.at
    _pack_cached(rec.buf, 0, *hk, *hv, *arrays, pages, page, Hk, D)
    status = lib.gkd_cache_read(at + 2 * _HEADS_BYTES, pt, L, B, T, pst, pct, 0, at,
                                at + _HEADS_BYTES, _raw_stream(dev))
    if status:
        _check(status)
    return k_out, v_out


def cache_attention_workspace_size(B: int, Tq: int, Hq: int, Hk: int, D: int, page: int,
                                   L: int) -> int:
    """Bytes of workspace gkd_cache_attention needs for these sizes."""
    _int_sizes("gkd_cache_attention_workspace_size", B, Tq, Hq, Hk, D, page, L)
    return int(load().gkd_cache_attention_workspace_size(B, Tq, Hq, Hk, D, page, L))


def cache_attention(q: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                    table: torch.Tensor, length=None, q_len=None, causal: bool = False, scale=None,
                    out=None, workspace=None) -> torch.Tensor:
    """Attention of q [B,Tq,Hq,D] bf16 over the first length[b] (int32, default
    all L * page) tokens of each sequence's pages in a cache (codes, scales and
    table as cache_append's). causal: the q_len[b] (int32, default Tq) queries are
    the last of the length[b] tokens and see those up to their place. Tokens
    without a page do not count. Queries past q_len[b] are not computed: their
    rows of a given `out` stay as they are, those of a new one are zeros. scale:
    default D**-0.5. Returns out [B,Tq,Hq,D]; a query without keys gives zeros."""
    lib = _lib or load()
    bf16 = torch.bfloat16
    dev = _place(q, "q")
    hq = _heads(dev, q, "q", bf16)
    sizes, arrays, pt, b = _cache(dev, codes, scales, table)
    pages, page, Hk, D, L = sizes
    B, Tq, Hq, d = q.shape
    if b != B or d != D:
        raise ValueError(f"q must be [{b}, Tq, Hq, {D}], got {tuple(q.shape)}")
    _int_sizes("gkd_cache_attention", B, Tq, Hq, *sizes)
    pl = None if length is None else _dense(dev, length, "length", torch.int32, (B,))
    pql = None if q_len is None else _dense(dev, q_len, "q_len", torch.int32, (B,))
    if out is None:
        out = q.new_empty((B, Tq, Hq, D)) if q_len is None else q.new_zeros((B, Tq, Hq, D))
    ho = _heads(dev, out, "out", bf16)
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    ws, ws_bytes = _workspace(workspace, lib.gkd_cache_attention_workspace_size(
        B, Tq, Hq, Hk, D, page, L), dev)
    rec = _records
    at = rec.at
    _pack_cached(rec.buf, 0, *hq, *ho, *arrays, pages, page, Hk, D)
    status = lib.gkd_cache_attention(at, at + 2 * _HEADS_BYTES, pt, L, pl, pql, B, Tq, Hq,
                                     D ** -0.5 if scale is None else scale,
                                     GKD_ATTN_CAUSAL if causal else 0, at + _HEADS_BYTES,
                                     None if ws is None else ws.data_ptr(), ws_bytes,
                                     _raw_stream(dev))
    if status:
        _check(status)
    return out
