"""The binding measures a workspace by what it holds: one with gaps is refused before anything is looked at (CPU)."""
import pytest
import torch

tq = pytest.importorskip("kv_cache_vector_fwht_b200")


def test_a_workspace_with_gaps_is_refused():
    q = tq.tq_build_codebook_host(128, 3, "prod", 0)
    cache = tq.KVCache(q, 1, 1, 64, value_bits=2, device="cpu")
    query, bounds = torch.zeros(1, 2, 3, 128), tq.alloc_block_bounds(cache, device="cpu")
    blocks = torch.zeros(1, 1, 1, dtype=torch.int32)
    for ws in (torch.zeros(1 << 20, dtype=torch.uint8)[::2], torch.zeros(1 << 10, 1 << 10, dtype=torch.uint8)[:, :512]):
        with pytest.raises(ValueError, match="workspace"):
            tq.tq_extend_attention(q, cache, query, query.clone(), ws)
        with pytest.raises(ValueError, match="workspace"):
            tq.tq_select_blocks(q, cache, bounds, query[:, :, 0].contiguous(), blocks, ws, n_sink=0)
        with pytest.raises(ValueError, match="workspace"):
            tq.tq_decode_attention_blocks(q, cache, query[:, :, 0].contiguous(), blocks, query[:, :, 0].contiguous(), ws)
