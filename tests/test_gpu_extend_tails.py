"""tq_extend_attention where most of a row's weights lie far below its largest, and where scores keep rising."""
import math

import numpy as np
import pytest
import torch

import oracle as O
from around import quantizers
from gpu_util import require_cuda

pytestmark = pytest.mark.gpu

import kv_cache_vector_fwht_b200 as tq  # noqa: E402

F32 = torch.float32


def extend(qg, cache, q, **kw):
    out = torch.full(q.shape, float("nan"), device="cuda:0", dtype=F32)
    tq.tq_extend_attention(qg, cache, q.cuda(), out, tq.alloc_extend_workspace(cache, q.shape[1], q.shape[2]), **kw)
    tq.tq_sync_status()
    return out


def flat_tail(length, gap, sink, rows_of_heads, n):
    """One token `gap` above all others (base 2), whose keys are zero; its value is 0 and theirs are 1. Returns the
    call's output and the exact one: the others' share of the weights."""
    qo, qg = quantizers("mse", 4)
    cache = tq.KVCache(qg, 1, 1, length, value_bits=4, device="cuda:0")
    g = torch.Generator("cuda").manual_seed(length)
    cache.k_idx.copy_(torch.randint(0, 256, cache.k_idx.shape, generator=g, device="cuda", dtype=torch.uint8))
    cache.k_norms.zero_()
    cache.k_norms.view(torch.float16)[sink] = 11.0
    cache.v_q.zero_()
    cache.v_params.zero_()
    cache.v_params.view(torch.float16)[:, :, 0] = 1.0
    cache.v_params.view(torch.float16)[sink] = 0.0
    cache.set_lengths([length])
    khat = O.reconstruct_keys(qo, dict(idx=cache.k_idx[sink:sink + 1].cpu().numpy(),
                                       norms=cache.k_norms[sink:sink + 1].cpu().numpy().view(np.uint16)))[0]
    q = torch.from_numpy(khat * gap * math.log(2) * math.sqrt(128) / (khat @ khat)).to(F32)
    z = (q.double().numpy() @ khat) / math.sqrt(128)
    tail = (length - 1) * math.exp(-z)
    out = extend(qg, cache, q.expand(1, rows_of_heads, n, 128), causal=False)
    return out, tail / (1 + tail), z


@pytest.mark.parametrize("rows_of_heads,n,length", [(1, 128 * 148, 1 << 14), (1, 128 * 148, 1 << 17), (1, 128 * 148, 1 << 20), (1, 1, 1 << 20),
                                                    (16, 1, 1 << 17), (40, 1, 1 << 17)])
@pytest.mark.parametrize("gap", [15.0, 20.0, 25.3, 27.0, 30.0])
@pytest.mark.parametrize("first", [True, False])
def test_a_long_flat_tail_under_one_large_weight(rows_of_heads, n, length, gap, first):
    """Weights down to 2^-30 of the largest, up to a million of them: their sum counts in the numerator as it does
    below. The share is off by the score's error, |z| (2^-11 + 2^-12) (rotated query, levels: fp16), by 2^-11 twice (value
    and weight, half a step each), by what all weights together lose as subnormal numbers, 2^-11 of the sum, and by
    the tensor cores' sums: a product is cut off at the last of the 24 bits of the sum that it is added to, so
    `length` products of one sign lose less than length 2^-23 of their sum."""
    require_cuda()
    out, want, z = flat_tail(length, gap, 0 if first else length - 1, rows_of_heads, n)
    bound = want * (math.expm1(z * 1.5 * 2.0 ** -11) * 1.01 + 2 * 2.0 ** -11 + length * 2.0 ** -23) + 2.0 ** -11
    off = (out.double() - want).abs().max().item()
    assert off <= bound, f"off by {off:.2e} of a share of {want:.2e}, bound {bound:.2e}"


@pytest.mark.parametrize("heads,n", [(2, 1), (40, 1), (5, 20)])
@pytest.mark.parametrize("step", [3.0, 7.5, 14.9, 15.1, 40.0])
def test_scores_that_rise_tile_by_tile(heads, n, step):
    """Every tile's scores lie `step` (base 2) above the tile's before: below, next to and beyond what raises a reference."""
    require_cuda()
    tiles, qo, qg = 12, *quantizers("mse", 4)
    cache = tq.KVCache(qg, 1, 1, 128 * tiles, value_bits=4, device="cuda:0")
    g = torch.Generator("cuda").manual_seed(5)
    cache.k_idx.copy_(torch.randint(0, 256, (1, 64), generator=g, device="cuda", dtype=torch.uint8).expand(128 * tiles, 64))
    norms = (1.0 + torch.arange(128 * tiles, device="cuda") // 128).half()
    cache.k_norms.view(torch.float16)[:, 0] = norms
    cache.v_q.zero_()
    values = torch.randn(128 * tiles, 4, generator=g, device="cuda").half()
    cache.v_params.zero_()
    cache.v_params.view(torch.float16)[:, :, 0] = values
    cache.set_lengths([128 * tiles])
    one = O.reconstruct_keys(qo, dict(idx=cache.k_idx[:1].cpu().numpy(), norms=cache.k_norms[:1].cpu().numpy().view(np.uint16)))[0]
    q = torch.from_numpy(one * step * math.log(2) * math.sqrt(128) / (one @ one)).to(F32)
    z = (q.double().numpy() @ one) / math.sqrt(128) * norms.double().cpu().numpy()
    w = np.exp(z - z.max())
    w /= w.sum()
    v = values.double().cpu().numpy().repeat(32, 1)
    want = w @ v
    e = np.expm1(np.abs(z) * 1.5 * 2.0 ** -11) * 1.01 + 2.0 ** -11
    bound = (w * e) @ np.abs(v) + np.abs(want) * (w @ e) + 2.0 ** -11 * np.abs(v).max() + 2.0 ** -11 * (w @ np.abs(v))
    out = extend(qg, cache, q.expand(1, heads, n, 128), causal=False).double().cpu().numpy()
    assert (np.abs(out - want) <= bound).all()
