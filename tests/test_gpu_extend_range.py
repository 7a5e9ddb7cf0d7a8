"""tq_extend_attention and tq_decode_attention_blocks with query rows of very unlike lengths side by side."""
import numpy as np
import pytest
import torch

import oracle as O
import workloads as W
from around import attention64, causal_limits, check, make_case
from gpu_util import require_cuda

pytestmark = pytest.mark.gpu

import kv_cache_vector_fwht_b200 as tq  # noqa: E402

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
# sizes of the plain rows, and of those beside them: the squares of 1e25 pass fp32's range
PLAIN = {BF16: 1.0, F32: 1.0, F16: 2.0 ** -7}
LONG = {BF16: (1e6, 1e12, 1e25), F32: (1e6, 1e12, 1e25), F16: (1e-3, 500.0, 1e4)}


def extend(qg, cache, q, **kw):
    out = torch.full(q.shape, float("nan"), device="cuda:0", dtype=F32)
    tq.tq_extend_attention(qg, cache, q.cuda(), out, tq.alloc_extend_workspace(cache, q.shape[1], q.shape[2]), **kw)
    tq.tq_sync_status()
    return out


def of_length(g, shape, dtype, which):
    """Gaussian rows; row (h, t) is LONG[dtype][(h + t) % 4] large, i = (h + t + 2) % 4, or plain where i is 3."""
    q = torch.from_numpy(W.gaussian(g, shape))
    f = torch.tensor(list(LONG[dtype]) + [PLAIN[dtype]])
    at = (torch.arange(shape[1])[:, None] + torch.arange(shape[2]) + 2) % 4
    if which is not None:   # only one row is long
        at = torch.where((torch.arange(shape[1])[:, None] * shape[2] + torch.arange(shape[2])) == which[0], which[1], 3)
    return (q * f[at][None, :, :, None]).to(dtype), (at == 3)


def check_rows(out, ref, tol, plain, lo, hi):
    """The plain rows within their bounds; the others finite and between the values they mix."""
    pick = plain[None].expand(out.shape[:3])
    check(out[pick.cuda()], ref[pick.numpy()], tol[pick.numpy()], F32)
    assert out.isfinite().all()
    got = out.double().cpu().numpy()
    assert (got <= hi + 2e-3 * np.abs(hi) + 1e-6).all() and (got >= lo - 2e-3 * np.abs(lo) - 1e-6).all()


def hull(oc, vbits, n):
    v = O.dequantize_values(oc["v_q"][0, 0, :n], oc["v_params"][0, 0, :n], vbits, 128)
    return v.min(0), v.max(0)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("mode,bits", [("prod", 3), ("grouped", 2), ("mse", 4)])
@pytest.mark.parametrize("group,n", [(2, 2), (5, 5), (4, 10), (12, 5), (30, 3), (13, 10)])
@pytest.mark.parametrize("which", [None, (0, 1), (3, 2)])
def test_rows_of_unlike_lengths_in_a_tile(dtype, mode, bits, group, n, which):
    """4, 25, 40, 60, 90 and 130 rows, every fourth a plain one or all but one: a row's outputs depend on it alone."""
    require_cuda()
    lengths = [190]
    qo, qg, oc, cache, g = make_case(31, mode, bits, 4, lengths, 1, 192, lo=0.5 / PLAIN[dtype], hi=2 / PLAIN[dtype])
    q, plain = of_length(g, (1, group, n, 128), dtype, which)
    with np.errstate(over="ignore", invalid="ignore"):   # the bounds of rows 1e12 long are infinite
        ref, tol = attention64(qo, oc, q.double().numpy(), causal_limits(lengths, n), 4)
    check_rows(extend(qg, cache, q), ref, tol, plain, *hull(oc, 4, 190))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("group,n", [(2, 2), (4, 12), (8, 12)])
def test_one_key_gives_its_value_whatever_the_score(dtype, group, n):
    """The softmax of one score is 1: scores from -1e33 to 1e33."""
    require_cuda()
    qo, qg, oc, cache, g = make_case(32, "mse", 4, 4, [1], 1, 16, lo=1.0, hi=1.0)
    khat = O.reconstruct_keys(qo, dict(idx=oc["k_idx"][0, 0, :1], norms=oc["k_norms"][0, 0, :1]))[0]
    size = torch.tensor([1e32, -1e32, 1.0, -1e20, 1e-20, -3.0])[torch.arange(group * n) % 6].view(1, group, n, 1)
    q = (size * torch.from_numpy(khat).float() / np.linalg.norm(khat)).to(dtype)
    v = O.dequantize_values(oc["v_q"][0, 0, :1], oc["v_params"][0, 0, :1], 4, 128)[0]
    ref = np.broadcast_to(v, q.shape)
    check(extend(qg, cache, q, causal=False), ref, 2.0 ** -11 * np.abs(ref), F32)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [5, 40, 100])
def test_rows_that_see_nothing_change_no_other(dtype, n):
    """A sequence of three tokens asked for n: its first rows see nothing, and hold anything."""
    require_cuda()
    lengths = [3, 120]
    qo, qg, oc, cache, g = make_case(33, "prod", 4, 2, lengths, 1, 128)
    q = torch.from_numpy(W.gaussian(g, (2, 2, n, 128))).to(dtype)
    ref, tol = attention64(qo, oc, q.double().numpy(), causal_limits(lengths, n), 2)
    for junk in (1e30, 3e38, float("inf"), float("nan")):
        q[0, :, :n - 3] = junk
        out = extend(qg, cache, q)
        check(out, ref, tol, F32)
        assert not out[0, :, :n - 3].any()


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_heads_of_unlike_lengths_over_listed_blocks(dtype):
    require_cuda()
    qo, qg, oc, cache, g = make_case(34, "prod", 4, 4, [500], 1, 512, lo=0.5 / PLAIN[dtype], hi=2 / PLAIN[dtype])
    q, plain = of_length(g, (1, 12, 1, 128), dtype, None)
    blocks = torch.tensor([[[0, 3, 7]]], dtype=torch.int32, device="cuda:0")
    out = torch.full((1, 12, 128), float("nan"), device="cuda:0", dtype=F32)
    tq.tq_decode_attention_blocks(qg, cache, q[:, :, 0].contiguous().cuda(), blocks, out, tq.alloc_blocks_workspace(cache, 12, 3))
    tq.tq_sync_status()
    keys = [[[t for i in (0, 3, 7) for t in range(64 * i, min(500, 64 * i + 64))]]]
    with np.errstate(over="ignore", invalid="ignore"):
        ref, tol = attention64(qo, oc, q.double().numpy(), [[500]], 4, keys=keys)
    check_rows(out[:, :, None], ref, tol, plain, *hull(oc, 4, 500))
