"""tq_extend_attention over contexts that come from memory at uneven pace: the same bits in every run, and the right ones."""
import pytest
import torch

from around import attention64, check, quantizers
from gpu_util import download_pair, require_cuda

pytestmark = pytest.mark.gpu

import kv_cache_vector_fwht_b200 as tq  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("mode,bits,vbits", [("prod", 4, 4), ("prod", 3, 4), ("prod", 2, 4), ("prod", 4, 2), ("mse", 4, 4), ("mse", 3, 4),
                                             ("mse", 1, 2), ("grouped", 2, 4), ("grouped", 3, 4)])
@pytest.mark.parametrize("heads,n", [(5, 1), (6, 5), (6, 8), (6, 10), (6, 16), (6, 20)])
def test_the_same_bits_in_every_run(mode, bits, vbits, heads, n):
    """Every tile of query rows (16 to 128) and stage count of the raw tiles; 40 (sequence, KV head) pairs, from cold and
    from warm caches. A tile that is read before it has arrived shows as a difference between the runs, or from the definition."""
    require_cuda()
    B, length = 20, 20000
    qo, qg = quantizers(mode, bits)
    cache = tq.KVCache(qg, B, 2, length + 16 - length % 16, value_bits=vbits, device="cuda:0")
    g = torch.Generator("cuda").manual_seed(n)
    for at in range(0, length, 4000):
        k, v = (torch.randn(B, 2, 4000, 128, generator=g, device="cuda").to(BF16) for _ in range(2))
        tq.tq_append(qg, cache, k, v)
    q = torch.randn(B, 2 * heads, n, 128, generator=g, device="cuda").to(BF16)
    ws, flush = tq.alloc_extend_workspace(cache, 2 * heads, n), torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    outs = []
    for i in range(12):
        if i % 3 == 0:
            flush.fill_(i)
        outs.append(torch.empty(q.shape, dtype=F32, device="cuda"))
        tq.tq_extend_attention(qg, cache, q, outs[-1], ws)
    tq.tq_sync_status()
    assert all(torch.equal(outs[0], o) for o in outs[1:])
    for b, h in ((0, 0), (B - 1, 1)):
        oc = download_pair(cache, b, h, length)
        some = q[b:b + 1, h * heads:h * heads + 1, -1:]
        ref, tol = attention64(qo, oc, some.float().cpu().numpy(), [[length]], vbits)
        check(outs[0][b:b + 1, h * heads:h * heads + 1, -1:], ref, tol, F32)


@pytest.mark.parametrize("mode,bits,vbits", [("prod", 3, 4), ("mse", 2, 2), ("grouped", 2, 4)])
@pytest.mark.parametrize("heads,n", [(5, 1), (3, 20), (8, 12)])
@pytest.mark.parametrize("length", [3, 71, 143])
def test_rows_behind_the_end_change_no_bit(mode, bits, vbits, heads, n, length):
    """Zeros, the largest norms, NaN or another sequence's rows behind the end: the outputs are the same, to the bit."""
    require_cuda()
    qo, qg = quantizers(mode, bits)
    cache = tq.KVCache(qg, 1, 1, 160, value_bits=vbits, device="cuda:0")
    g = torch.Generator("cuda").manual_seed(length)
    k, v = (torch.randn(1, 1, length, 128, generator=g, device="cuda").to(BF16) for _ in range(2))
    tq.tq_append(qg, cache, k, v)
    q = 3 * torch.randn(1, heads, n, 128, generator=g, device="cuda")
    ws, outs = tq.alloc_extend_workspace(cache, heads, n), []
    for junk in (0, 0x7bff, 0x7bff - (1 << 11), -1, 0x3c00):
        cache.k_norms[length:] = junk
        cache.v_params[length:] = junk
        cache.k_idx[length:] = junk & 255
        outs.append(torch.empty(q.shape, dtype=F32, device="cuda"))
        tq.tq_extend_attention(qg, cache, q, outs[-1], ws)
    tq.tq_sync_status()
    assert outs[0].isfinite().all() and all(torch.equal(outs[0], o) for o in outs[1:])
