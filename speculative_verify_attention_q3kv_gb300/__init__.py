"""q3kv: speculative-verify attention over a 3-bit, Hadamard-rotated, paged KV
cache, as hand-written CUDA for sm_103a behind a small C ABI (``include/q3kv.h``).

Python surface (argument marshalling only):
  api.make_desc, api.pool_bytes, api.workspace_bytes, api.Allocator,
  api.append, api.verify_attn (and the prefill, fp8_ and t5k_ forms)
  api.accept_greedy, api.accept_sample, api.accept_sample_nucleus, api.accept_draft
  api.make_rope_plan, api.rope: rotary positions with several axes
  api.verify_attn_lse, api.attn_mass, api.evict: eviction by attention mass
The CUDA library is built in-tree by ``build.build()``; nothing here falls back
to another implementation when it is missing.
"""
__all__ = ["api", "build"]
