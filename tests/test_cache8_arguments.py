"""Refusals of the 8-bit cache's and the verification's entry points that reach no GPU (CPU)."""
import ctypes as C

from head_latent_attention_qkv_gb300 import _lib

lib = _lib.lib
BAD = _lib.MLA_ERR_INVALID_ARG


def test_null_handles_are_refused():
    d = C.byref(_lib.mla_attn_desc_t(num_blocks=1, block_len=4, max_pages=1))
    c = C.byref(_lib.mla_cache8_t(latent=256, rope=256, scale=256))
    assert lib.mla_cache8_store(None, None, None, 1, c, 1, None) == BAD
    assert b"cache8 store" in lib.mla_last_error()
    assert lib.mla_cache8_load(None, c, 1, None, 1, None, None) == BAD
    assert lib.mla_latent_cache_append8(None, None, None, None, 1, c, 1, None, 0, None) == BAD
    assert lib.mla_latent_attention8(None, None, None, c, 1, d, None, None, None, None, 0, None) == BAD
    assert lib.mla_draft_forward8(None, None, None, None, c, 1, d, None, None, None, 0, None) == BAD
    assert lib.mla_cache8_compact(None, c, 1, None, 1, None, 1, None, 4, None, None, None, 0, None, None, 0, None, 0,
                                  None) == BAD
    assert lib.mla_verify_drafts(None, None, 4, None, 4, 1, None, None, None, None, 1, 1, 4, None, None, None, None) == BAD
    assert lib.mla_append8_workspace_bytes(None, 4) == 0
    assert lib.mla_latent_attention8_workspace_bytes(None, d) == 0
    assert lib.mla_forward8_workspace_bytes(None, d) == 0
    assert lib.mla_cache8_compact_workspace_bytes(None, 1, 8) == 0
