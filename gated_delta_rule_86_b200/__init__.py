"""B200-native (sm_100a) KDA operator: chunkwise prefill and recurrent decode, and the softmax
attention of the full-attention layers that hybrid models put beside it.

The computation lives in ``libkda_b200.so`` (C ABI in ``include/kda.h``);
``ops`` and ``attention`` are its thin Python binding.  Importing the package does not load the
library; the first call does, and fails loudly if it has not been built.
"""
from ._lib import EXPORTED, KdaError, load  # noqa: F401
from .attention import kda_attn, kda_attn_bwd, kda_attn_decode_step, kda_attn_fwd, kda_kv_append  # noqa: F401
from .ops import (device_error, gdn_chunk_fwd, gdn_decode_step, gdn_recurrent_fwd, kda_chunk,  # noqa: F401
                  kda_chunk_bwd, kda_chunk_fwd, kda_chunk_fwd_fused, kda_decode_step, kda_decode_step_fused,
                  kda_recurrent_fwd)

__all__ = ["kda_chunk_fwd", "kda_recurrent_fwd", "kda_decode_step", "kda_chunk_fwd_fused", "kda_decode_step_fused",
           "gdn_chunk_fwd", "gdn_recurrent_fwd", "gdn_decode_step", "kda_chunk", "kda_chunk_bwd", "kda_attn_fwd", "kda_attn_bwd", "kda_attn",
           "kda_kv_append", "kda_attn_decode_step", "device_error",
           "KdaError", "load"]
