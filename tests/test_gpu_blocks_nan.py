"""tq_block_bounds and tq_select_blocks with norms that are not finite."""
import pytest
import torch

import workloads as W
from around import make_case
from gpu_util import require_cuda

pytestmark = pytest.mark.gpu

import kv_cache_vector_fwht_b200 as tq  # noqa: E402


@pytest.mark.parametrize("mode,bits", [("mse", 1), ("mse", 2), ("mse", 3), ("mse", 4), ("prod", 2), ("prod", 3), ("prod", 4),
                                       ("grouped", 1), ("grouped", 2), ("grouped", 3)])
def test_a_nan_norm_reaches_its_blocks_bounds(mode, bits):
    """A NaN among a block's keys makes the bounds of its channels NaN (grouped: of the group's channels), those of
    other blocks stay as they are; an infinite one makes the bound on its side infinite. The selection takes such a block first."""
    require_cuda()
    qo, qg, oc, cache, g = make_case(41, mode, bits, 0, [400, 130], 2, 400)
    clean, bounds = tq.alloc_block_bounds(cache), tq.alloc_block_bounds(cache)
    tq.tq_block_bounds(qg, cache, clean, 400)
    norms = cache.k_norms.view(2, 2, 400, -1)
    for row in (0, 1, 31, 32, 63):    # of block 2, sequence 0, head 1
        kept = norms[0, 1, 128 + row].clone()
        norms[0, 1, 128 + row, 0] = 0x7e00
        bounds.fill_(5.0)
        tq.tq_block_bounds(qg, cache, bounds, 400)
        tq.tq_sync_status()
        c = 32 if mode == "grouped" else 128
        assert bounds[0, 1, 2, :, :c].isnan().all()
        back = bounds.clone()
        back[0, 1, 2, :, :c] = clean[0, 1, 2, :, :c]
        back[1, :, 3:] = clean[1, :, 3:]       # no tokens: left as they were
        assert torch.equal(back, clean)
        norms[0, 1, 128 + row] = kept
    if mode == "grouped":
        norms[0, 1, 399, 1] = 0x7e00
        tq.tq_block_bounds(qg, cache, bounds, 1)
        assert bounds[0, 1, 6, :, 32:].isnan().all() and torch.equal(bounds[0, 1, 6, :, :32], clean[0, 1, 6, :, :32])
        norms[0, 1, 399, 1] = 0
    norms[0, 1, 130, 0] = 0x7c00
    tq.tq_block_bounds(qg, cache, bounds, 400)
    assert bounds[0, 1, 2, :, :32].isinf().any(0).all()   # one key's coordinate is the least or the largest
    norms[0, 1, 130, 0] = 0x7e00
    tq.tq_block_bounds(qg, cache, bounds, 400)
    ids = torch.empty((2, 2, 1), dtype=torch.int32, device="cuda:0")
    q = torch.from_numpy(W.gaussian(g, (2, 4, 128))).cuda()
    tq.tq_select_blocks(qg, cache, bounds, q, ids, tq.alloc_blocks_workspace(cache, 4, 1), n_sink=0, n_recent=0)
    tq.tq_sync_status()
    assert ids[0, 1, 0] == 2
