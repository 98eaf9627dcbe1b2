"""Batched draft-token verification for speculative decoding on GB300 (sm_103a).

The work runs in libspecverify.so (hand-written CUDA behind the C ABI of
include/spec_verify.h); this package is the torch-facing binding:

    spec_verify_stochastic  acceptance u <= min(1, p/q), first rejection, residual or
                            bonus token by inverse CDF, with NKL and the greedy decision
    spec_verify_greedy      argmax-match verification
    spec_verify_tree        longest accepted root-to-leaf path of a draft tree
    spec_nkl                KL(q || p) / ln V per position

and, around the target's attention over the drafted tokens (include/spec_kv.h):

    KVCache                 a paged key/value cache in 8 bits
    spec_kv_append          quantises keys and values as it writes them
    spec_kv_read            reads cached tokens back
    spec_attention          scores a round's rows (chain or tree) over the cache, a prefix
                            that the batch shares computed once for all
    spec_attention_chunk    the same for chunks of a prompt

    Rope                    how heads rotate by positions (of one or several axes)
    spec_qk_rope            norm and rotation of queries and keys in one pass
    spec_qk_rope_append     the same with the cache's write

    spec_kv_weigh           the softmax weight that cached tokens gather
    spec_kv_evict           cuts sequences to a budget of tokens, the heaviest kept
"""
from .api import (KVCache, Rope, Workspace, spec_attention, spec_attention_chunk, spec_attention_chunk_workspace_bytes,
                  spec_attention_workspace_bytes, spec_kv_append, spec_kv_evict, spec_kv_read, spec_kv_weigh, spec_nkl,
                  spec_qk_rope, spec_qk_rope_append, spec_tree_depth, spec_verify_greedy, spec_verify_stochastic,
                  spec_verify_tree, spec_workspace_bytes)

__all__ = ["KVCache", "Rope", "Workspace", "spec_attention", "spec_attention_chunk", "spec_attention_chunk_workspace_bytes",
           "spec_attention_workspace_bytes", "spec_kv_append", "spec_kv_evict", "spec_kv_read", "spec_kv_weigh", "spec_nkl",
           "spec_qk_rope", "spec_qk_rope_append", "spec_tree_depth", "spec_verify_greedy", "spec_verify_stochastic",
           "spec_verify_tree", "spec_workspace_bytes"]
