"""tq_append and tq_append_decode refuse values that are not laid out as the keys are."""
import pytest
import torch

from gpu_util import require_cuda

pytestmark = pytest.mark.gpu

import kv_cache_vector_fwht_b200 as tq  # noqa: E402

BF16 = torch.bfloat16


def test_values_are_contiguous_and_like_the_keys():
    """A view of a projection's rows was read as if it were contiguous: other heads' and tokens' values."""
    require_cuda()
    q = tq.tq_build_codebook(128, 3, "prod", 0)
    cache = tq.KVCache(q, 2, 2, 64, value_bits=2)
    rows = torch.randn(2, 3, 2, 128, device="cuda").to(BF16)
    k, view = rows.transpose(1, 2).contiguous(), rows.transpose(1, 2)
    query, out = torch.zeros(2, 4, 128, device="cuda", dtype=BF16), torch.zeros(2, 4, 128, device="cuda")
    ws = tq.alloc_decode_workspace(cache, 4)
    for v in (view, k.float(), k[:, :, :2].contiguous(), k[:, :1].contiguous()):
        with pytest.raises(AssertionError):
            tq.tq_append(q, cache, k, v)
        with pytest.raises(AssertionError):
            tq.tq_append_decode(q, cache, k, v, query, out, ws)
    assert cache.lengths == [0, 0]
    tq.tq_append(q, cache, k, k)
    tq.tq_append_decode(q, cache, k, k, query, out, ws)
    torch.cuda.synchronize()
    assert cache.lengths == [6, 6]
