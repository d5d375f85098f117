"""GB300 (sm_103a) hot path of the Medusa decode step.

The computation lives in libmedusa_gb300.so (hand-written CUDA kernels behind
the C ABI of include/medusa.h); this package is its thin Python binding:

  heads_topk          Medusa heads h + SiLU(W1 h + b1) -> W2, per-head top-k
  heads_topk_static   the same without a workspace (library-owned scratch)
  sparse_tree_paths   the most accurate rank tuples (host)
  tree_layout         node table, ancestor mask and paths of a tree (host)
  build_tree          candidate tokens of the tree nodes
  tree_attention      ancestor-masked attention of all candidates in one pass
  verify_accept_tree  greedy / typical acceptance, longest accepted branch
  verify_accept_tree_sample  typical acceptance, next token drawn from the
                      best node's softmax
  verify_accept_tree_draw  acceptance by tokens drawn from the target's
                      probabilities with given random numbers
  verify_project_tree the same as verify_accept_tree from the tree's hidden states: lm_head projection
                      on the tensor cores, reduced without writing the logits
  verify_accept_chain speculative-sampling acceptance with k + 1 tokens
  kv_compact          keep the accepted branch's KV rows and hidden state
  tree_attention_q8   tree attention over the 8-bit paged KV cache
  kv_append_q8        quantise prompt rows, decoded tokens or the accepted branch
                      into its pages
  kv_append_rope_q8   the same for rows that are not rotated yet, rotary positions
                      applied on the way, the rows' queries rotated beside them
  chunk_attention_q8  attention of a prompt, a piece of one or a decoded token over
                      the pages that hold its own keys
  rope_rows           rotary positions of a tree's or a chunk's queries and keys
  kv_pages_fork       fork, free and reserve: who holds which page
  kv_pages_compact    move the pages in use to the front of the pool
  device_status       raises if a bounded device wait gave up (MEDUSA_ERR_TIMEOUT)
  set_wait_limit      test hook: the tensor-core kernels' wait limit
"""
from ._native import MedusaError, lib  # noqa: F401
from .api import (build_tree, chunk_attention_q8, chunk_attention_q8_workspace, device_status, heads_topk, heads_topk_static, heads_topk_workspace,  # noqa: F401
                  kv_append_q8, kv_append_rope_q8, kv_compact, kv_pages_compact, kv_pages_compact_workspace, kv_pages_fork,
                  kv_pages_fork_workspace, rope_rows, set_wait_limit,
                  sparse_tree_paths, tree_attention, tree_attention_q8, tree_attention_q8_workspace,
                  tree_attention_workspace, tree_layout,
                  verify_accept_chain, verify_accept_tree, verify_accept_tree_draw, verify_draw_workspace, verify_accept_workspace,
                  verify_accept_tree_sample, verify_chain_workspace, verify_project_tree,
                  verify_project_workspace, verify_sample_workspace)
