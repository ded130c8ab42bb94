"""MSA (MiniMax Sparse Attention) hot path on B200: a C-ABI CUDA library
(``lib/libmsa.so``, built from ``csrc/`` for sm_100a) and a thin Python
binding.

  capi      -- calls with the C entry points' names (ctypes; the operators around
               the sparse path through ``lib/msa_calls.so``)
  pipeline  -- the five calls of one forward pass on one stream, and the calls
               around it: norms + rotation, the paged cache and its decode
               attention, window attention
  workloads -- seeded synthetic inputs (shared with tests and the benchmark)
"""
from . import capi, pipeline, workloads  # noqa: F401

__all__ = ["capi", "pipeline", "workloads"]
