"""GDLA (Grouped Differential Latent Attention) forward core for NVIDIA B200.

Python binding of the C-ABI library ``libgdla.so`` (hand-written sm_100a CUDA
kernels). PyTorch supplies device memory and streams; the computation happens
only in the library. See ``include/gdla.h`` for the ABI.
"""
from .ops import (DC, DL, DQK, DR, DV, GROUP, MAX_SINKS, PAGE_SIZES, GDLAError, attn_bwd,
                  attn_bwd_sinks_workspace_bytes, attn_bwd_workspace_bytes, attn_decode, attn_decode_latent,
                  attn_decode_paged, attn_fwd, cache_append, decode_latent_workspace_bytes, decode_paged_workspace_bytes,
                  decode_workspace_bytes, device_error, library, prologue, prologue_workspace_bytes)

__all__ = ["attn_fwd", "attn_bwd", "attn_bwd_workspace_bytes", "attn_bwd_sinks_workspace_bytes", "prologue",
           "prologue_workspace_bytes", "attn_decode", "attn_decode_latent", "cache_append", "attn_decode_paged",
           "decode_workspace_bytes", "decode_latent_workspace_bytes", "decode_paged_workspace_bytes", "device_error",
           "library", "GDLAError", "GROUP", "DQK", "DV", "DC", "DR", "DL", "MAX_SINKS", "PAGE_SIZES"]
