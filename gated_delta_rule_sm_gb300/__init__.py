"""GB300 (sm_103a) Kimi Delta Attention: chunkwise gated delta rule, forward and backward.

The computation lives in the CUDA library ``libkda_gb300.so`` behind the C
ABI in ``include/kda.h``; this package only marshals torch tensors to it
(``forward`` / ``backward``, the layer's short-convolution prologue
``short_conv`` / ``short_conv_backward`` and its gated output norm ``gated_norm`` /
``gated_norm_backward``, and for serving the single-token steps ``decode_step``, ``ssm_step`` and
``short_conv_step``, the prompts' ``ssm_scan`` and ``short_conv_prompt`` and the cache's
``pages_*``, attention over its pages among them; ``gated_scan``, ``gated_scan_backward`` and ``gated_step`` are
the gated linear recurrence) and draws seeded synthetic inputs
(``inputs``).  Importing the package does not load the library; the first
call does, and raises if it has not been built.
"""
from ._lib import (KdaError, backward, decode_step, device_status, forward, gated_norm,  # noqa: F401
                   gated_norm_backward, gated_scan, gated_scan_backward, gated_scan_saved_size, gated_step, load,
                   pages_append, pages_attention, pages_compact, pages_copy, pages_extend, pages_fork, pages_free,
                   saved_size, short_conv, short_conv_backward, short_conv_prompt, short_conv_step, ssm_scan, ssm_step)

__all__ = ["forward", "backward", "saved_size", "short_conv", "short_conv_backward", "gated_norm",
           "gated_norm_backward", "decode_step", "ssm_scan", "ssm_step", "short_conv_prompt", "short_conv_step",
           "gated_scan", "gated_scan_backward", "gated_scan_saved_size", "gated_step", "pages_append", "pages_attention",
           "pages_copy", "pages_fork", "pages_extend", "pages_free", "pages_compact", "load", "device_status",
           "KdaError"]
