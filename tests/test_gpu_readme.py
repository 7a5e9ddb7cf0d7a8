"""README's layer step runs as it is written, and gives what its parts promise."""
import os
import re

import pytest
import torch

from gpu_util import require_cuda

pytestmark = pytest.mark.gpu

import kv_cache_vector_fwht_b200 as tq  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16 = torch.bfloat16


def test_the_layer_of_the_readme_runs_as_written():
    require_cuda()
    text = open(os.path.join(ROOT, "README.md")).read()
    code = re.search(r"A layer's step[^`]*`rows`[^:]*:\n\n((?:    [^\n]*\n|\n)+)", text).group(1)
    code = "\n".join(line[4:] for line in code.splitlines())
    assert all(f in code for f in ("tq_norm_rope", "tq_append", "tq_block_bounds", "tq_extend_attention", "tq_select_blocks",
                                   "tq_decode_attention_blocks"))
    g = torch.Generator("cuda").manual_seed(1)
    for n in (5, 1):     # a chunk, a step
        hq, hk = 6, 2
        quantizer = tq.tq_build_codebook(128, 3, "prod", 0)
        cache = tq.KVCache(quantizer, 2, hk, 512, value_bits=2)
        old = torch.randn(2, hk, 300, 128, generator=g, device="cuda").to(BF16)
        tq.tq_append(quantizer, cache, old, old)
        space = dict(tq=tq, torch=torch, quantizer=quantizer, cache=cache, n_tokens=n, batch=2, n_q_heads=hq, n_kv_heads=hk,
                     rows=torch.randn(2, n, (hq + 2 * hk) * 128, generator=g, device="cuda").to(BF16),
                     positions=(300 + torch.arange(n, device="cuda", dtype=torch.int32)).expand(2, n).contiguous(),
                     inv_freq=(1e4 ** (-torch.arange(64, device="cuda") / 64)).float(),
                     wq=torch.ones(128, device="cuda", dtype=BF16), wk=torch.ones(128, device="cuda", dtype=BF16),
                     bounds=tq.alloc_block_bounds(cache))
        tq.tq_block_bounds(quantizer, cache, space["bounds"], 300)
        exec(code, space)
        tq.tq_sync_status()
        assert cache.lengths == [300 + n] * 2
        assert space["out"].shape == (2, hq, n, 128) and space["out"].isfinite().all()
        # six blocks a sequence and room for eight: the step over selected blocks is the one over the whole context
        whole = torch.empty((2, hq, n, 128), device="cuda", dtype=BF16)
        tq.tq_extend_attention(quantizer, cache, space["q_out"], whole, tq.alloc_extend_workspace(cache, hq, n))
        tq.tq_sync_status()
        assert space["out"].any() and (space["out"].float() - whole.float()).abs().max() <= 2.0 ** -7 * whole.abs().max()
