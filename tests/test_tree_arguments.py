"""Refusals of the tree and eviction entry points that reach no GPU (CPU)."""
import ctypes as C

from head_latent_attention_qkv_gb300 import _lib

lib = _lib.lib
BAD = _lib.MLA_ERR_INVALID_ARG


def test_null_handles_are_refused():
    desc = _lib.mla_attn_desc_t(num_blocks=1, block_len=4, max_pages=1)
    d = C.byref(desc)
    assert lib.mla_tree_attention(None, None, None, None, 1, d, None, None, None, None, 0, None) == BAD
    assert b"tree attention" in lib.mla_last_error()
    assert lib.mla_draft_forward_tree(None, None, None, None, None, 1, d, None, None, None, 0, None) == BAD
    assert lib.mla_key_weights(None, None, None, None, 1, d, None, None, 1.0, None, None, 8, None, 0, None) == BAD
    assert lib.mla_cache_select(None, None, 8, None, 1, 4, 0, 0, None, None, None) == BAD
    assert lib.mla_cache_compact(None, None, 1, None, 1, None, 1, None, 4, None, None, None, 0, None, None,
                                 0, None, 0, None) == BAD
    assert lib.mla_tree_attention_workspace_bytes(None, d) == 0
    assert lib.mla_forward_tree_workspace_bytes(None, d) == 0
    assert lib.mla_key_weights_workspace_bytes(None, d, 8) == 0
    assert lib.mla_cache_compact_workspace_bytes(None, 1, 8) == 0
