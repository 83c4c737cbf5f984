"""KDA on AMD Instinct MI355X (gfx950): chunked forward, backward and decode, the head-gated delta rule
beside it, and the norms around a block.

The compute path is libkda.so (hand-written HIP kernels behind a C ABI,
declared in include/kda.h); this package only marshals torch tensors into
that ABI.  The library is loaded on first use, and a missing library is an
error, never a fallback.
"""

from .api import chunk_bwd, chunk_fwd, chunk_fwd_noalloc, decode, decode_stats, gate_prefix, workspace_bytes  # noqa: E402,F401
from .gated import (gdr_chunk_bwd, gdr_chunk_fwd, gdr_decode, gdr_workspace_bytes, norm_gate_bwd,  # noqa: E402,F401
                    norm_gate_fwd)
from ._lib import KdaError, HipEvent  # noqa: E402,F401
