"""GKDT parameter-free detection head on AMD MI355X (gfx950).

Calls over the C ABI of libgkdhead (include/gkdhead.h):
  vkp_pool         Gaussian-pooled visual keypoint prototypes
  kernel_heatmap   normalised 1x1 kernels x 4x-upsampled features, fused per
                   row over the prompt modalities, with the peak decode fused
  peak_decode      per-row argmax -> -1..1 keypoint + score
  roi_preprocess   detector boxes of an image -> the backbone's normalised
                   square input (crop, resize, centre pad, normalise)
  roi_backproject  -1..1 keypoints -> image coordinates
  kg_transformer   kernel-generation transformer: prototypes -> kernels
and the token operators (include/gkdtokens.h), the pieces of a transformer
block over image tokens and prompt rows:
  linear            matrix product with bias, activation and residual
  qk_norm_rope      head norm and rotary positions with several axes
  prefix_attention  attention of a batch that shares one prefix of keys
"""
from .binding import (GkdError, LIB_PATH, kernel_heatmap, kg_transformer, kg_workspace_size,
                      linear, linear_workspace_size, load, peak_decode, prefix_attention,
                      prefix_attention_workspace_size, qk_norm_rope, roi_backproject,
                      roi_preprocess, vkp_pool)

__all__ = ["GkdError", "LIB_PATH", "kernel_heatmap", "kg_transformer", "kg_workspace_size",
           "linear", "linear_workspace_size", "load", "peak_decode", "prefix_attention",
           "prefix_attention_workspace_size", "qk_norm_rope", "roi_backproject",
           "roi_preprocess", "vkp_pool"]
