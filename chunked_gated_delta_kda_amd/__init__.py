"""MI355X-native chunked gated delta-rule forward and backward passes (KDA and GDN),
linear attention with a decay for each head (LA), and the gated norm behind them.

The computation lives in libkda.so (HIP kernels for gfx950 behind the C ABI
of include/kda.h); this package is its thin Python binding.  Build the
library with ``python -m chunked_gated_delta_kda_amd.build``.
"""
from ._binding import (EXPORTS, LIB_PATH, LibKdaError, bwd_workspace_size, gated_norm_bwd,
                       gated_norm_fwd, gdn_bwd,
                       gdn_bwd_saved, gdn_decode, gdn_fwd, gdn_fwd_save, gdn_fwd_split, gdn_prep, kda_bwd,
                       kda_bwd_saved, kda_decode, kda_fwd, kda_fwd_noalloc, kda_fwd_save, kda_fwd_split,
                       kda_prep,
                       kda_recur, la_bwd, la_decode, la_fwd, la_workspace_size, load,
                       status_str, version, workspace_size)
from .autograd import chunk_gdn, chunk_kda, chunk_la, gated_norm

__all__ = ["chunk_la", "la_fwd", "la_bwd", "la_decode", "la_workspace_size", "gated_norm",
           "gated_norm_fwd", "gated_norm_bwd",
           "chunk_kda", "chunk_gdn", "kda_fwd", "gdn_fwd", "kda_fwd_split", "gdn_fwd_split",
           "kda_fwd_noalloc",
           "kda_prep", "gdn_prep", "kda_recur",
           "kda_decode", "gdn_decode", "kda_fwd_save", "gdn_fwd_save", "kda_bwd_saved",
           "gdn_bwd_saved", "kda_bwd", "gdn_bwd", "workspace_size", "bwd_workspace_size",
           "status_str", "version", "load", "LibKdaError", "EXPORTS", "LIB_PATH"]
