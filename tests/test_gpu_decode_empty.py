"""tq_decode_attention and its forms over a cache in which every sequence is empty: zeros, and empty records."""
import pytest
import torch

from gpu_util import require_cuda

pytestmark = pytest.mark.gpu

import kv_cache_vector_fwht_b200 as tq  # noqa: E402


@pytest.mark.parametrize("mode,bits,vbits", [("prod", 3, 2), ("prod", 4, 4), ("mse", 1, 4), ("mse", 4, 2), ("grouped", 2, 4)])
@pytest.mark.parametrize("heads", [(5, 1), (4, 2), (16, 2)])
def test_empty_sequences(mode, bits, vbits, heads):
    require_cuda()
    hq, hkv = heads
    q = tq.tq_build_codebook(128, bits, mode, 0, list(range(32)) if mode == "grouped" else None)
    cache = tq.KVCache(q, 3, hkv, 256, value_bits=vbits)
    query = torch.randn(3, hq, 128, device="cuda").bfloat16()
    ws = tq.alloc_decode_workspace(cache, hq)
    for _ in range(2):
        out = torch.full((3, hq, 128), float("nan"), device="cuda")
        tq.tq_decode_attention(q, cache, query, out, ws)
        tq.tq_sync_status()
        assert not out.any()
        out.fill_(float("nan"))
        tq.tq_decode_attention_noalloc(q, cache, query, out)
        part = torch.full((3, hq, tq.TQ_PART_FLOATS), float("nan"), device="cuda")
        tq.tq_decode_attention_partial(q, cache, query, part, ws)
        tq.tq_sync_status()
        assert not out.any() and part[..., 0].isneginf().all() and not part[..., 1:].any()
    tokens = torch.randn(3, hkv, 2, 128, device="cuda").bfloat16()
    tq.tq_append_decode(q, cache, tokens, tokens, query, out, ws)
    tq.tq_sync_status()
    assert out.isfinite().all() and out.any()
