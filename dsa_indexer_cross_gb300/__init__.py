"""GB300-native DSA lightning indexer + causal top-k, IndexShare layer loop and sparse MLA
attention, the paged latent cache with the attention that reads it, and what a decode step needs around
it (shared prefixes, draft verification, key weights, eviction).  The compute runs in
libdsa.so (hand-written sm_103a kernels behind a C ABI, include/dsa.h); this package is its ctypes binding plus seeded input generators.
"""
from ._lib import (AttnDesc, DsaError, IndexCache, IndexerDesc, LayerIO, PagedCache, DSA_IDX_INDEPENDENT_ROWS,
                   DSA_IDX_ROPE_K, DSA_PAGE_ROWS, ProjDesc, dsa_indexer_projections, dsa_indexer_topk_paged,
                   dsa_sparse_attn_backward, dsa_sparse_attn_backward_workspace_size, dsa_indexer_backward,
                   dsa_indexer_backward_workspace_size,
                   dsa_sparse_attn_paged, paged_cache,
                   DSA_IDX_ROPE_Q, DSA_LAYER_FULL, DSA_LAYER_SHARED, attn_desc, dsa_donor_table,
                   dsa_indexer_topk, dsa_indexer_topk_static, dsa_indexer_workspace_size, dsa_layers_workspace_size, dsa_mtp_indexshare_step,
                   dsa_profile_enable,
                   dsa_profile_indexer_last, dsa_profile_read, dsa_indexer_static_status, dsa_debug_pipeline, dsa_rope_table,
                   dsa_sparse_attn, dsa_sparse_attn_workspace_size, dsa_workspace_status, indexer_desc,
                   indexshare_layers_forward, lib,
                   CacheWriteDesc, LatentCache, RopeDesc, RopeScaling, DSA_BF16, DSA_CACHE_BF16,
                   DSA_CACHE_FP8, DSA_CACHE_ROPE, DSA_F32, DSA_ROPE_INTERLEAVED, DSA_ROPE_INVERSE,
                   DSA_ROPE_SCALE_LINEAR, DSA_ROPE_SCALE_NONE, DSA_ROPE_SCALE_YARN,
                   cache_write_desc, dsa_latent_attn_paged, dsa_latent_attn_workspace_size,
                   dsa_latent_cache_read, dsa_latent_cache_write, dsa_rope_apply,
                   dsa_rope_table_scaled, latent_cache, rope_desc, rope_scaling_linear,
                   rope_scaling_yarn,
                   VerifyDesc, dsa_mtp_verify, verify_desc,
                   SharedRows, dsa_latent_attn_shared, dsa_latent_attn_shared_workspace_size, shared_rows,
                   dsa_latent_key_weights, dsa_latent_key_weights_workspace_size,
                   EvictDesc, dsa_latent_cache_evict, dsa_latent_cache_evict_workspace_size, evict_desc)

__all__ = ["AttnDesc", "DsaError", "IndexCache", "IndexerDesc", "LayerIO", "PagedCache", "DSA_PAGE_ROWS",
           "dsa_indexer_topk_paged", "dsa_sparse_attn_paged", "paged_cache", "ProjDesc", "dsa_indexer_projections", "dsa_sparse_attn_backward",
           "dsa_sparse_attn_backward_workspace_size", "dsa_indexer_backward", "dsa_indexer_backward_workspace_size", "DSA_IDX_INDEPENDENT_ROWS", "DSA_IDX_ROPE_K",
           "DSA_IDX_ROPE_Q", "DSA_LAYER_FULL", "DSA_LAYER_SHARED", "attn_desc", "dsa_donor_table", "dsa_indexer_topk", "dsa_indexer_topk_static",
           "dsa_indexer_workspace_size", "dsa_layers_workspace_size", "dsa_mtp_indexshare_step", "dsa_profile_enable",
           "dsa_profile_indexer_last", "dsa_profile_read", "dsa_indexer_static_status", "dsa_debug_pipeline", "dsa_rope_table", "dsa_sparse_attn",
           "dsa_sparse_attn_workspace_size", "dsa_workspace_status", "indexer_desc", "indexshare_layers_forward", "lib",
           "CacheWriteDesc", "LatentCache", "RopeDesc", "RopeScaling", "DSA_BF16", "DSA_CACHE_BF16",
           "DSA_CACHE_FP8", "DSA_CACHE_ROPE", "DSA_F32", "DSA_ROPE_INTERLEAVED", "DSA_ROPE_INVERSE",
           "DSA_ROPE_SCALE_LINEAR", "DSA_ROPE_SCALE_NONE", "DSA_ROPE_SCALE_YARN", "cache_write_desc",
           "dsa_latent_attn_paged", "dsa_latent_attn_workspace_size", "dsa_latent_cache_read",
           "dsa_latent_cache_write", "dsa_rope_apply", "dsa_rope_table_scaled", "latent_cache", "rope_desc",
           "rope_scaling_linear", "rope_scaling_yarn", "VerifyDesc", "dsa_mtp_verify", "verify_desc",
           "SharedRows", "dsa_latent_attn_shared", "dsa_latent_attn_shared_workspace_size", "shared_rows",
           "dsa_latent_key_weights", "dsa_latent_key_weights_workspace_size",
           "EvictDesc", "dsa_latent_cache_evict", "dsa_latent_cache_evict_workspace_size", "evict_desc"]
