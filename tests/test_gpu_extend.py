"""tq_extend_attention: several query tokens over the packed cache, against its definition in 64 bits."""
import numpy as np
import pytest
import torch

import oracle as O
import workloads as W
from around import attention64, causal_limits, check, full_limits, make_case
from gpu_util import require_cuda, to_device

pytestmark = pytest.mark.gpu

import kv_cache_vector_fwht_b200 as tq  # noqa: E402

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def query_rows(g, shape, dtype):
    return torch.from_numpy(W.gaussian(g, shape)).to(dtype)


def extend(qg, cache, q, out_dtype, **kw):
    """Runs the call with outputs filled with NaN; the device's status must stay clean."""
    out = torch.full(q.shape, float("nan"), device="cuda:0", dtype=out_dtype)
    ws = tq.alloc_extend_workspace(cache, q.shape[1], q.shape[2])
    tq.tq_extend_attention(qg, cache, q.cuda(), out, ws, **kw)
    tq.tq_sync_status()
    return out


@pytest.mark.parametrize("mode,bits", [("mse", 1), ("mse", 2), ("mse", 3), ("mse", 4), ("prod", 2), ("prod", 3), ("prod", 4),
                                       ("grouped", 1), ("grouped", 2), ("grouped", 3)])
@pytest.mark.parametrize("vbits", [2, 4])
def test_every_cache_kind(mode, bits, vbits):
    require_cuda()
    lengths = [300, 77]
    qo, qg, oc, cache, g = make_case(1, mode, bits, vbits, lengths, 2, 304)
    q = query_rows(g, (2, 6, 3, 128), BF16)
    ref, tol = attention64(qo, oc, q.float().numpy(), causal_limits(lengths, 3), vbits)
    check(extend(qg, cache, q, F32), ref, tol, F32)


@pytest.mark.parametrize("group,n", [(1, 1), (5, 3), (16, 1), (3, 7), (8, 4), (7, 5), (1, 48), (4, 13), (8, 8), (5, 14),
                                     (12, 8), (1, 97), (8, 16), (3, 50), (5, 27)])
@pytest.mark.parametrize("causal", [True, False])
def test_numbers_of_query_rows(group, n, causal):
    """1 to 150 rows of a KV head: every tile of the kernel, full and not, one tile and two; lengths that
    end inside a tile, at its end, and before the first query token."""
    require_cuda()
    lengths = [384, 129, 40]
    qo, qg, oc, cache, g = make_case(2, "prod", 3, 4, lengths, 1, 384)
    q = query_rows(g, (3, group, n, 128), BF16)
    limits = causal_limits(lengths, n) if causal else full_limits(lengths, n)
    ref, tol = attention64(qo, oc, q.float().numpy(), limits, 4)
    check(extend(qg, cache, q, F32, causal=causal), ref, tol, F32)


@pytest.mark.parametrize("length", [0, 1, 2, 15, 16, 63, 64, 65, 127, 128, 129, 257])
def test_short_lengths(length):
    require_cuda()
    lengths = [length, 1]
    qo, qg, oc, cache, g = make_case(3, "mse", 4, 2, lengths, 2, 272)
    q = query_rows(g, (2, 4, 2, 128), BF16)
    ref, tol = attention64(qo, oc, q.float().numpy(), causal_limits(lengths, 2), 2)
    out = extend(qg, cache, q, F32)
    check(out, ref, tol, F32)
    # rows that see nothing are exact zeros
    for b, L in enumerate(lengths):
        for t in range(2):
            if L - 2 + t + 1 <= 0:
                assert not out[b, :, t].any()


@pytest.mark.parametrize("q_dtype", [BF16, F16, F32])
@pytest.mark.parametrize("out_dtype", [BF16, F16, F32])
@pytest.mark.parametrize("size", [1e-3, 1.0, 300.0])
def test_types_and_query_sizes(q_dtype, out_dtype, size):
    """Queries are brought to one size before they are rounded: small and large ones lose nothing."""
    require_cuda()
    lengths = [200]
    qo, qg, oc, cache, g = make_case(4, "prod", 4, 4, lengths, 1, 208, lo=0.5 / size, hi=2 / size)
    q = (size * torch.from_numpy(W.gaussian(g, (1, 4, 2, 128)))).to(q_dtype)
    ref, tol = attention64(qo, oc, q.double().numpy(), causal_limits(lengths, 2), 4)
    check(extend(qg, cache, q, out_dtype), ref, tol, out_dtype)


@pytest.mark.parametrize("q_dtype", [BF16, F16, F32])
@pytest.mark.parametrize("mode,bits", [("prod", 3), ("grouped", 1), ("mse", 2)])
@pytest.mark.parametrize("group,n", [(5, 5), (4, 11), (12, 5), (30, 3), (13, 10)])
def test_types_at_many_rows(q_dtype, mode, bits, group, n):
    """25, 44, 60, 90 and 130 rows of each query type: rows of 16 bits and of 32 are rotated in different ways."""
    require_cuda()
    lengths = [190]
    qo, qg, oc, cache, g = make_case(17, mode, bits, 4, lengths, 1, 192)
    q = query_rows(g, (1, group, n, 128), q_dtype)
    ref, tol = attention64(qo, oc, q.double().numpy(), causal_limits(lengths, n), 4)
    check(extend(qg, cache, q, F32), ref, tol, F32)


def test_strided_queries_and_outputs():
    """A projection's (batch, tokens, heads, d) rows as a view, and an output inside a larger one whose
    other elements stay as they are."""
    require_cuda()
    lengths, n = [150, 99], 4
    qo, qg, oc, cache, g = make_case(5, "grouped", 2, 4, lengths, 2, 160)
    rows = query_rows(g, (2, n, 10 * 128), BF16).cuda()
    q = rows[..., 2 * 128:8 * 128].view(2, n, 6, 128).transpose(1, 2)
    big = torch.full((2, n, 9 * 128), 7.0, device="cuda:0", dtype=F32)
    out = big[..., 128:7 * 128].view(2, n, 6, 128).transpose(1, 2)
    tq.tq_extend_attention(qg, cache, q, out, tq.alloc_extend_workspace(cache, 6, n))
    tq.tq_sync_status()
    ref, tol = attention64(qo, oc, q.float().cpu().numpy(), causal_limits(lengths, n), 4)
    check(out, ref, tol, F32)
    assert (big[..., :128] == 7).all() and (big[..., 7 * 128:] == 7).all()


def test_head_maps_and_scale():
    require_cuda()
    lengths = [210]
    qo, qg, oc, cache, g = make_case(6, "mse", 3, 4, lengths, 4, 224)
    q = query_rows(g, (1, 9, 2, 128), BF16)
    head_map = [3, 0, 3, 3, 0, 3, 3, 3, 1]     # uneven, out of order, KV head 2 unused
    ref, tol = attention64(qo, oc, q.float().numpy(), causal_limits(lengths, 2), 4, head_map=head_map, scale=0.05)
    check(extend(qg, cache, q, F32, head_map=head_map, sm_scale=0.05), ref, tol, F32)


@pytest.mark.parametrize("mode,bits,vbits,group,n", [("prod", 4, 4, 8, 1), ("prod", 3, 2, 7, 5), ("mse", 4, 4, 4, 32)])
def test_long_context_in_many_splits(mode, bits, vbits, group, n):
    """Contexts shared by many blocks of threads, of unequal lengths; peaked weights (keys up to 8 times as long)."""
    require_cuda()
    lengths = [9000, 3333]
    qo, qg, oc, cache, g = make_case(7, mode, bits, vbits, lengths, 1, 9008, lo=1.0, hi=8.0)
    q = query_rows(g, (2, group, n, 128), BF16)
    some = list(range(n)) if n < 8 else [0, n // 2, n - 1]
    ref, tol = attention64(qo, oc, q[:, :, some].float().numpy(), [[lim[t] for t in some] for lim in causal_limits(lengths, n)], vbits)
    a = extend(qg, cache, q, F32)
    check(a[:, :, some], ref, tol, F32)
    assert torch.equal(a, extend(qg, cache, q, F32))   # the same bits every time


def test_growing_maximum():
    """Keys whose scores rise along the context raise the reference maxima again and again."""
    require_cuda()
    qo, qg, oc, cache, g = make_case(8, "mse", 4, 4, [1], 1, 1040)
    q = query_rows(g, (1, 2, 1, 128), F32)
    up = np.linspace(0.05, 12, 1024)[:, None]
    K = up[None, None] * q[0, 0, 0].numpy()[None, None, None] + 0.05 * W.gaussian(g, (1, 1, 1024, 128))
    V = W.gaussian(g, (1, 1, 1024, 128))
    from gpu_util import oracle_cache, upload_cache
    oc = oracle_cache(qo, K.astype(np.float32), V, 4, [1024])
    upload_cache(cache, oc)
    ref, tol = attention64(qo, oc, q.numpy(), [[1024]], 4)
    check(extend(qg, cache, q, F32), ref, tol, F32)


def test_stale_rows_and_later_tokens_do_not_reach_a_row():
    """Rows behind the end of a sequence hold anything (here: all bits set, which are NaN norms and
    parameters); a later token with infinite value parameters or an infinite norm reaches
    only the query rows that see it, and there only the channels it spoils."""
    require_cuda()
    lengths, n = [70, 33], 3
    qo, qg, oc, cache, g = make_case(9, "prod", 3, 4, lengths, 1, 144)
    q = query_rows(g, (2, 2, n, 128), BF16)
    for plane in (cache.k_idx, cache.k_signs, cache.k_norms, cache.v_q, cache.v_params):
        rows = plane.view(2, 144, -1)
        for b, L in enumerate(lengths):
            rows[b, L:] = -1 if plane.dtype == torch.int16 else 255
    ref, tol = attention64(qo, oc, q.float().numpy(), causal_limits(lengths, n), 4)
    check(extend(qg, cache, q, F32), ref, tol, F32)
    # token 68 of sequence 0: seen by rows 1 and 2 alone; the scale of its second group is infinite
    params = cache.v_params.view(2, 144, 4, 2)
    finite = params[0, 68, 1, 1].item()
    params[0, 68, 1, 1] = 0x7c00
    out = extend(qg, cache, q, F32)
    assert out[0, :, 1:, 32:64].isnan().all()
    out[0, :, 1:, 32:64] = torch.from_numpy(ref[0, :, 1:, 32:64]).float()
    check(out, ref, tol, F32)
    params[0, 68, 1, 1] = finite
    # and an infinite norm at token 69, which row 2 alone sees: a score of +inf makes the softmax NaN, one of -inf a
    # weight of zero (the sign is that of the codebook part: the sketch's weight is r16 / inf = 0)
    cache.k_norms.view(2, 144, 2)[0, 69, 0] = 0x7c00
    out = extend(qg, cache, q, F32)
    without, wtol = attention64(qo, oc, q.float().numpy(), [[68, 69, 69], causal_limits(lengths, n)[1]], 4)
    codes = O.unpack_bits(oc["k_idx"][0, 0, 69:70], 2, 128)
    for h in range(2):
        if qo.cent[codes[0]] @ (qo.Pi @ q[0, h, 2].double().numpy()) > 0:
            assert out[0, h, 2].isnan().all()
            out[0, h, 2] = torch.from_numpy(without[0, h, 2]).float()
    check(out, without, wtol, F32)


@pytest.mark.parametrize("group,n", [(2, 2), (6, 9)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_query_row_that_is_not_finite_spoils_no_other(group, n, dtype):
    require_cuda()
    lengths = [140]
    qo, qg, oc, cache, g = make_case(18, "prod", 4, 2, lengths, 1, 144)
    q = query_rows(g, (1, group, n, 128), dtype)
    ref, tol = attention64(qo, oc, q.double().numpy(), causal_limits(lengths, n), 2)
    q[0, 0, 0, 3], q[0, 1, 1, 7] = float("inf"), float("nan")
    out = extend(qg, cache, q, F32)
    for h, t in ((0, 0), (1, 1)):
        assert out[0, h, t].isnan().all()
        out[0, h, t] = torch.from_numpy(ref[0, h, t]).float()
    check(out, ref, tol, F32)


def test_many_items_with_a_split_last_round():
    """More tiles of query rows than SMs: whole rounds, and the last few tiles shared by all SMs."""
    require_cuda()
    n = 128 * 150
    qo, qg, oc, cache, g = make_case(19, "mse", 2, 2, [n], 1, n)
    q = query_rows(g, (1, 1, n, 128), BF16)
    some = [0, 1, 127, 128, 255, 256, 9600, 12345, n - 2, n - 1]
    ref, tol = attention64(qo, oc, q[:, :, some].float().numpy(), [[t + 1 for t in some]], 2)
    out = extend(qg, cache, q, F32)
    check(out[:, :, some], ref, tol, F32)
    assert out.isfinite().all()


def test_many_long_sequences():
    """Over 64 sequences, each in several splits."""
    require_cuda()
    lengths = [1500 - 20 * i for i in range(66)]
    qo, qg, oc, cache, g = make_case(20, "mse", 2, 2, lengths, 1, 1504)
    q = query_rows(g, (66, 1, 2, 128), BF16)
    ref, tol = attention64(qo, oc, q.float().numpy(), causal_limits(lengths, 2), 2)
    check(extend(qg, cache, q, F32), ref, tol, F32)


def test_many_sequences():
    require_cuda()
    lengths = [1 + 7 * i % 90 for i in range(70)]
    qo, qg, oc, cache, g = make_case(10, "mse", 2, 2, lengths, 1, 96)
    q = query_rows(g, (70, 2, 2, 128), BF16)
    ref, tol = attention64(qo, oc, q.float().numpy(), causal_limits(lengths, 2), 2)
    check(extend(qg, cache, q, F32), ref, tol, F32)


def test_a_captured_call_follows_the_lengths_on_the_device():
    """A captured call, replayed for the lengths that the device holds then: longer and shorter than at the capture."""
    require_cuda()
    qo, qg, oc, cache, g = make_case(11, "prod", 3, 2, [4000, 4000], 1, 4000)
    q = query_rows(g, (2, 4, 2, 128), BF16).cuda()
    out = torch.empty(q.shape, device="cuda:0", dtype=F32)
    ws = tq.alloc_extend_workspace(cache, 4, 2)
    cache.set_lengths([100, 900])
    tq.tq_extend_attention(qg, cache, q, out, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tq.tq_extend_attention(qg, cache, q, out, ws)
    for lengths in ([100, 900], [4000, 0], [1, 3999], [2500, 17]):
        cache.len_dev.copy_(torch.tensor(lengths, dtype=torch.int32))
        graph.replay()
        tq.tq_sync_status()
        short = dict(oc, len=np.array(lengths))
        ref, tol = attention64(qo, short, q.float().cpu().numpy(), causal_limits(lengths, 2), 2)
        check(out, ref, tol, F32)


def test_two_streams_with_a_workspace_each():
    require_cuda()
    qo, qg, oc, cache, g = make_case(12, "prod", 4, 4, [6000], 1, 6000)
    qs = [query_rows(g, (1, 8, 1, 128), BF16).cuda() for _ in range(2)]
    want = [extend(qg, cache, q.cpu(), F32) for q in qs]
    streams, outs = [torch.cuda.Stream() for _ in qs], [torch.empty_like(w) for w in want]
    spaces = [tq.alloc_extend_workspace(cache, 8, 1) for _ in qs]
    torch.cuda.synchronize()
    for _ in range(10):
        for q, o, ws, s in zip(qs, outs, spaces, streams):
            tq.tq_extend_attention(qg, cache, q, o, ws, stream=s)
    torch.cuda.synchronize()
    tq.tq_sync_status()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_one_workspace_for_calls_of_any_size():
    """Large, small and listed-block calls in turn on one workspace leave it as the next one needs it."""
    require_cuda()
    qo, qg, oc, cache, g = make_case(13, "mse", 4, 4, [5000, 70], 2, 5008)
    cases = [(8, 1), (4, 40), (2, 3), (8, 1), (4, 40)]
    size = max(max(tq.tq_extend_workspace_bytes(cache, h, n) for h, n in cases), tq.tq_blocks_workspace_bytes(cache, 8, 20))
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda:0")
    bounds = tq.alloc_block_bounds(cache)
    tq.tq_block_bounds(qg, cache, bounds, cache.capacity)
    ids = torch.empty((2, 2, 20), dtype=torch.int32, device="cuda:0")
    seen = {}
    for h, n in cases:
        q = query_rows(W.rng(h + n), (2, h, n, 128), BF16).cuda()
        out = torch.empty(q.shape, device="cuda:0", dtype=F32)
        tq.tq_extend_attention(qg, cache, q, out, ws)
        step = torch.empty((2, h, 128), device="cuda:0", dtype=F32)
        tq.tq_select_blocks(qg, cache, bounds, q[:, :, 0].contiguous(), ids, ws)
        tq.tq_decode_attention_blocks(qg, cache, q[:, :, 0].contiguous(), ids, step, ws)
        torch.cuda.synchronize()
        assert not ws[:64 << 10].any()
        if (h, n) in seen:
            assert all(torch.equal(a, b) for a, b in zip(seen[h, n], (out, ids, step)))
        seen[h, n] = out.clone(), ids.clone(), step.clone()
    tq.tq_sync_status()


def test_rows_beyond_32_bit_offsets():
    """The last KV head's rows lie more than 2^31 bytes into the index and value planes."""
    require_cuda()
    cap, hkv = 1 << 23, 8
    qo, qg, oc, small, g = make_case(14, "mse", 4, 4, [200], 1, 208)
    cache = tq.KVCache(qg, 1, hkv, cap, value_bits=4, device="cuda:0")
    cache.set_lengths([200])
    for name in ("k_idx", "k_norms", "v_q", "v_params"):
        plane, src = getattr(cache, name).view(hkv, cap, -1), getattr(small, name)
        plane[:, :200] = 0
        plane[hkv - 1, :208] = src.view(208, -1)
    q = query_rows(g, (1, hkv, 2, 128), BF16)
    ref, tol = attention64(qo, oc, q[:, hkv - 1:].float().numpy(), causal_limits([200], 2), 4)
    check(extend(qg, cache, q, F32)[:, hkv - 1:], ref, tol, F32)


def test_single_tokens_agree_with_the_decode():
    """n_tokens = 1 is tq_decode_attention's operator; the two differ by the extension's 16-bit operands."""
    require_cuda()
    lengths = [2000, 1777]
    qo, qg, oc, cache, g = make_case(15, "prod", 4, 4, lengths, 2, 2000)
    q = query_rows(g, (2, 16, 128), BF16).cuda()
    out = torch.empty((2, 16, 128), device="cuda:0", dtype=F32)
    tq.tq_decode_attention(qg, cache, q, out, tq.alloc_decode_workspace(cache, 16))
    ref, tol = attention64(qo, oc, q[:, :, None].float().cpu().numpy(), full_limits(lengths, 1), 4)
    got = extend(qg, cache, q[:, :, None].cpu(), F32)
    check(got, ref, tol, F32)
    check(got[:, :, 0], out.double().cpu().numpy(), tol[:, :, 0] + 1e-4, F32)
    assert to_device(np.zeros(1), F32).is_cuda


def test_refusals_on_the_device():
    dev = require_cuda()
    qo, qg, oc, cache, g = make_case(16, "mse", 2, 2, [20], 1, 32)
    q = torch.zeros((1, 2, 3, 128), device=dev, dtype=BF16)
    ws = tq.alloc_extend_workspace(cache, 2, 3)
    with pytest.raises(ValueError, match="query"):
        tq.tq_extend_attention(qg, cache, q[0], q[0], ws)
    with pytest.raises(ValueError, match="shape"):
        tq.tq_extend_attention(qg, cache, q, q[:, :1], ws)
    with pytest.raises(ValueError, match="current CUDA device"):
        tq.tq_extend_attention(qg, cache, q.cpu(), q, ws)
    with pytest.raises(ValueError, match="head_map"):
        tq.tq_extend_attention(qg, cache, q, q.clone(), ws, head_map=[0])
    with pytest.raises(tq.TQError) as e:
        tq.tq_extend_attention(qg, cache, q, q.clone(), ws[:1000])
    assert e.value.status == tq.TQ_EINVAL
    tq.tq_extend_attention(qg, cache, q[:, :, :0], q[:, :, :0], ws)   # no tokens: nothing to do
    tq.tq_sync_status()
