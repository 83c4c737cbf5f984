"""KDA on AMD Instinct MI355X (gfx950): chunked forward, backward and decode, the head-gated delta rule and linear
attention with a decay for each head beside it, the norms around a block, and the norms of queries and keys with their
rotation by position.

The compute path is libkda.so (hand-written HIP kernels behind a C ABI,
declared in include/kda.h); this package only marshals torch tensors into
that ABI.  The library is loaded on first use, and a missing library is an
error, never a fallback.
"""

from .api import chunk_bwd, chunk_fwd, chunk_fwd_noalloc, decode, decode_stats, gate_prefix, workspace_bytes  # noqa: E402,F401
from .gated import (gdr_chunk_bwd, gdr_chunk_fwd, gdr_decode, gdr_workspace_bytes, norm_gate_bwd,  # noqa: E402,F401
                    norm_gate_fwd)
from .linear import (lad_chunk_bwd, lad_chunk_fwd, lad_decode, lad_workspace_bytes, qk_norm_rope_bwd,  # noqa: E402,F401
                     qk_norm_rope_fwd)
from ._lib import KdaError, HipEvent  # noqa: E402,F401
