"""Block bounds, block selection and decode over listed blocks, and the operators around the cache in one
run, against their definitions in 64 bits."""
import numpy as np
import pytest
import torch

import oracle as O
import workloads as W
from around import attention64, check, make_case, pair_planes, quantizers
from gpu_util import download_pair, require_cuda

pytestmark = pytest.mark.gpu

import kv_cache_vector_fwht_b200 as tq  # noqa: E402

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
BLOCK = tq.TQ_BLOCK


def rotated_levels(qo, planes):
    """The codebook part of the keys in rotated coordinates, the groups' channels side by side."""
    norms = O.fp16_from_bits(planes["norms"])
    if qo.mode != "grouped":
        bits = qo.bits - 1 if qo.mode == "prod" else qo.bits
        return norms[:, :1] * qo.cent[O.unpack_bits(planes["idx"], O.storage_width(bits), 128)]
    parts, at = [], 0
    for i, g in enumerate(qo.groups):
        w = O.storage_width(g.bits)
        nb = g.channels.size * w // 8
        parts.append(norms[:, i:i + 1] * g.cent[O.unpack_bits(planes["idx"][:, at:at + nb], w, g.channels.size)])
        at += nb
    return np.concatenate(parts, 1)


def rotated_query(qo, q):
    if qo.mode != "grouped":
        return qo.Pi @ q
    return np.concatenate([g.Pi @ q[g.channels] for g in qo.groups])


@pytest.mark.parametrize("mode,bits", [("mse", 1), ("mse", 2), ("mse", 3), ("mse", 4), ("prod", 2), ("prod", 3), ("prod", 4),
                                       ("grouped", 1), ("grouped", 2), ("grouped", 3)])
@pytest.mark.parametrize("n_tokens", [1, 70, 100000])
def test_bounds(mode, bits, n_tokens):
    """Every cache kind; sequences of no, one, whole and partial blocks; only the last tokens' blocks change."""
    require_cuda()
    lengths = [0, 1, 63, 64, 65, 200, 640]
    qo, qg, oc, cache, g = make_case(21, mode, bits, 0, lengths, 2, 656)
    bounds = tq.alloc_block_bounds(cache)
    bounds.fill_(77.0)
    tq.tq_block_bounds(qg, cache, bounds, n_tokens)
    tq.tq_sync_status()
    got = bounds.double().cpu().numpy()
    for b, L in enumerate(lengths):
        first, used = max(0, L - n_tokens) // BLOCK, -(-L // BLOCK)
        for h in range(2):
            assert (got[b, h, :first] == 77).all() and (got[b, h, used:] == 77).all()
            if L:
                y = rotated_levels(qo, pair_planes(qo, oc, b, h, L))
                for i in range(first, used):
                    part = y[i * BLOCK:(i + 1) * BLOCK]
                    for which, want in enumerate((part.min(0), part.max(0))):
                        # the level's 2^-12, the result's half step 2^-11, and 32-bit products
                        assert np.all(np.abs(got[b, h, i, which] - want) <= np.abs(want) * (2.0 ** -11 + 2.0 ** -12 + 2.0 ** -20) + 2.0 ** -25)


def choice(qo, bounds, query, lengths, select, sink, recent, head_map):
    """The chosen blocks by a plain sort (numpy, 64 bits)."""
    B, hkv = bounds.shape[:2]
    ids = np.full((B, hkv, select), -1, np.int64)
    for b in range(B):
        used = -(-lengths[b] // BLOCK)
        for kv in range(hkv):
            heads = [h for h in range(query.shape[1]) if head_map[h] == kv]
            lo, hi = bounds[b, kv, :used, 0], bounds[b, kv, :used, 1]
            score = np.zeros(used)
            if heads:
                q = np.array([rotated_query(qo, query[b, h].astype(np.float64)) for h in heads])
                score = np.max([np.maximum(x * lo, x * hi).sum(1) for x in q], 0)   # np.max keeps NaN
            score = np.where(np.isnan(score), np.finfo(float).max, score)
            score[:sink] = np.inf
            score[max(0, used - recent):] = np.inf
            order = np.argsort(-score, kind="stable")[:select]
            ids[b, kv, :len(order)] = np.sort(order)
    return ids


def make_bounds(g, B, hkv, nb, same=0):
    mid = 0.5 * g.standard_normal((B, hkv, nb, 1, 128))
    wide = 1 + g.random((B, hkv, nb, 2, 128))
    out = (mid + wide * np.array([[-1.0], [1.0]])).astype(np.float16)
    if same:   # equal blocks: equal scores
        out[:, :, same:] = out[:, :, np.arange(same, nb) % same]
    return out


@pytest.mark.parametrize("mode,bits", [("prod", 3), ("mse", 4), ("grouped", 2)])
@pytest.mark.parametrize("group,dtype", [(1, BF16), (8, F16), (5, F32), (21, BF16)])
@pytest.mark.parametrize("select,sink,recent,same", [(1, 0, 0, 0), (6, 1, 2, 0), (20, 2, 0, 7), (3, 1, 2, 0), (64, 1, 1, 0), (100, 0, 3, 3)])
def test_selection(mode, bits, group, dtype, select, sink, recent, same):
    require_cuda()
    lengths = [4000, 0, 1, 64 * 21 + 5, 64 * 20]
    qo, qg = quantizers(mode, bits)
    g = np.random.default_rng(select + group)
    cache = tq.KVCache(qg, 5, 2, 4000, value_bits=0, device="cuda:0")
    cache.set_lengths(lengths)
    nb = -(-4000 // BLOCK)
    bounds = make_bounds(g, 5, 2, nb, same)
    if same == 7:
        bounds[0, 0, 11, 1, 5] = np.nan
    query = torch.from_numpy(g.standard_normal((5, 2 * group, 128)).astype(np.float32)).to(dtype)
    ids = torch.full((5, 2, select), -5, dtype=torch.int32, device="cuda:0")
    ws = tq.alloc_blocks_workspace(cache, 2 * group, select)
    for _ in range(2):
        tq.tq_select_blocks(qg, cache, torch.from_numpy(bounds).cuda(), query.cuda(), ids, ws, n_sink=sink, n_recent=recent)
        tq.tq_sync_status()
        want = choice(qo, bounds.astype(np.float64), query.double().numpy(), lengths, select, sink, recent,
                      O.default_head_map(2 * group, 2))
        assert np.array_equal(ids.cpu().numpy(), want)
    assert not ws[:64 << 10].any()


def test_selection_of_many_blocks_and_uneven_heads():
    """More blocks than fit the keys' shared memory; a KV head that no query head reads takes the lowest."""
    require_cuda()
    cap = 64 * 5000
    qo, qg = quantizers("mse", 2)
    g = np.random.default_rng(5)
    cache = tq.KVCache(qg, 1, 3, cap, value_bits=0, device="cuda:0")
    cache.set_lengths([cap - 100])
    bounds = make_bounds(g, 1, 3, 5000)
    query = torch.from_numpy(g.standard_normal((1, 4, 128)).astype(np.float32))
    head_map = [2, 0, 2, 2]
    ids = torch.empty((1, 3, 300), dtype=torch.int32, device="cuda:0")
    ws = tq.alloc_blocks_workspace(cache, 4, 300)
    tq.tq_select_blocks(qg, cache, torch.from_numpy(bounds).cuda(), query.cuda(), ids, ws, n_sink=1, n_recent=2, head_map=head_map)
    tq.tq_sync_status()
    want = choice(qo, bounds.astype(np.float64), query.numpy(), [cap - 100], 300, 1, 2, head_map)
    assert np.array_equal(ids.cpu().numpy(), want)


@pytest.mark.parametrize("kind", ["nan few", "nan many", "nan all", "close", "close and far", "equal", "low and nan"])
@pytest.mark.parametrize("select,blocks", [(3, 700), (40, 700), (300, 700), (40, 2100), (700, 2100), (9, 41)])
def test_selection_of_crowded_scores(kind, select, blocks):
    """Scores of which many are NaN, equal or apart by the last bits: the threshold among its like."""
    require_cuda()
    qo, qg = quantizers("mse", 3)
    g = np.random.default_rng(select)
    lengths = [64 * blocks - 9, 64 * (blocks - 30)]
    cache = tq.KVCache(qg, 2, 2, 64 * blocks, value_bits=0, device="cuda:0")
    cache.set_lengths(lengths)
    bounds = make_bounds(g, 2, 2, blocks)
    if kind.startswith("nan"):
        share = {"nan few": 0.01, "nan many": 0.5, "nan all": 1.0}[kind]
        bounds[g.random((2, 2, blocks)) < share, 1, 77] = np.nan
    elif kind == "low and nan":
        bounds = (-40000 * np.ones(bounds.shape)).astype(np.float16)
        bounds[:, :, ::3, 0, 5] = np.nan
    else:
        bounds[:] = bounds[:, :, :1]
        if kind != "equal":   # 60 scores, a multiple of 2^-10 |q_3| apart
            bounds[:, :, :, 0, 3] = -1 - 2.0 ** -10 * (np.arange(blocks) % 60)
            bounds[:, :, :, 1, 3] = 1 + 2.0 ** -10 * (np.arange(blocks) % 60)
        if kind == "close and far":
            bounds[:, :, 17, 1] = 60000.0
            bounds[:, :, 17, 0] = -60000.0
    query = torch.from_numpy(g.standard_normal((2, 6, 128)).astype(np.float32))
    ids = torch.empty((2, 2, select), dtype=torch.int32, device="cuda:0")
    ws = tq.alloc_blocks_workspace(cache, 6, select)
    tq.tq_select_blocks(qg, cache, torch.from_numpy(bounds).cuda(), query.cuda(), ids, ws, n_sink=1, n_recent=1)
    tq.tq_sync_status()
    want = choice(qo, bounds.astype(np.float64), query.double().numpy(), lengths, select, 1, 1, O.default_head_map(6, 2))
    assert np.array_equal(ids.cpu().numpy(), want)


@pytest.mark.parametrize("mode,bits,vbits", [("prod", 4, 4), ("mse", 2, 2), ("grouped", 3, 4)])
@pytest.mark.parametrize("group,out_dtype", [(1, F32), (7, BF16), (24, F32)])
def test_listed_blocks(mode, bits, vbits, group, out_dtype):
    """Lists in and out of order, with holes, blocks behind the end, outside the cache and listed twice."""
    require_cuda()
    lengths = [1000, 130, 0, 64]
    qo, qg, oc, cache, g = make_case(22, mode, bits, vbits, lengths, 2, 1008)
    nb = -(-1008 // BLOCK)
    lists = np.array([[[0, 3, 7, 15, -1], [15, 2, 2, 9, 0]], [[0, 1, 2, -1, -1], [2, 14, -1, 99, nb]],
                      [[0, 1, -1, -1, -1], [-1] * 5], [[0, 0, 0, 0, 0], [-7, 2**30, 0, 5, -1]]], np.int32)
    q = torch.from_numpy(W.gaussian(g, (4, 2 * group, 128))).to(BF16)
    keys = [[[i * BLOCK + t for i in lists[b, h] if 0 <= i < nb for t in range(BLOCK)] for h in range(2)] for b in range(4)]
    keys = [[[t for t in keys[b][h] if t < lengths[b]] for h in range(2)] for b in range(4)]
    ref, tol = attention64(qo, oc, q[:, :, None].float().numpy(), [[L] for L in lengths], vbits, keys=keys)
    out = torch.full(q.shape, float("nan"), device="cuda:0", dtype=out_dtype)
    ws = tq.alloc_blocks_workspace(cache, 2 * group, 5)
    tq.tq_decode_attention_blocks(qg, cache, q.cuda(), torch.from_numpy(lists).cuda(), out, ws)
    tq.tq_sync_status()
    check(out, ref[:, :, 0], tol[:, :, 0], out_dtype)


def test_many_listed_blocks_in_splits():
    require_cuda()
    qo, qg, oc, cache, g = make_case(23, "prod", 3, 2, [9000], 1, 9008)
    lists = np.sort(g.choice(140, 101, replace=False)).astype(np.int32)[None, None]
    keys = [[[i * BLOCK + t for i in lists[0, 0] for t in range(BLOCK) if i * BLOCK + t < 9000]]]
    q = torch.from_numpy(W.gaussian(g, (1, 8, 128))).to(BF16)
    ref, tol = attention64(qo, oc, q[:, :, None].float().numpy(), [[9000]], 2, keys=keys)
    outs = []
    for _ in range(2):
        out = torch.empty(q.shape, device="cuda:0", dtype=F32)
        tq.tq_decode_attention_blocks(qg, cache, q.cuda(), torch.from_numpy(lists).cuda(), out,
                                      tq.alloc_blocks_workspace(cache, 8, 101))
        tq.tq_sync_status()
        outs.append(out)
    check(outs[0], ref[:, :, 0], tol[:, :, 0], F32)
    assert torch.equal(*outs)


def test_captured_selection_and_attention():
    require_cuda()
    qo, qg, oc, cache, g = make_case(24, "mse", 4, 4, [3000], 2, 3008)
    bounds = tq.alloc_block_bounds(cache)
    q = torch.from_numpy(W.gaussian(g, (1, 4, 128))).to(BF16).cuda()
    ids, out = torch.empty((1, 2, 12), dtype=torch.int32, device="cuda:0"), torch.empty(q.shape, device="cuda:0", dtype=F32)
    ws = tq.alloc_blocks_workspace(cache, 4, 12)

    def step():
        tq.tq_block_bounds(qg, cache, bounds, 3000)
        tq.tq_select_blocks(qg, cache, bounds, q, ids, ws, n_sink=1, n_recent=2)
        tq.tq_decode_attention_blocks(qg, cache, q, ids, out, ws)

    step()
    torch.cuda.synchronize()
    want = ids.clone(), out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(5):
        ids.zero_()
        out.zero_()
        graph.replay()
    tq.tq_sync_status()
    assert torch.equal(ids, want[0]) and torch.equal(out, want[1])


@pytest.mark.parametrize("captured", [False, True])
def test_calls_between_copies_fills_and_two_streams(captured):
    """The operators directly behind copies, fills, other kernels, each other and another stream's work, all
    of which write what they read: every pass equals one that waits after each step."""
    require_cuda()
    qo, qg, oc, cache, g = make_case(25, "prod", 3, 2, [6000, 2500], 2, 6016)
    dev = "cuda:0"
    inputs = [torch.from_numpy(W.gaussian(g, (2, 6, 1, 128))).to(BF16).to(dev) for _ in range(3)]
    src, q, turned, half = (torch.empty_like(inputs[0]) for _ in range(4))
    pos, pos_src = torch.zeros((2, 1), dtype=torch.int32, device=dev), torch.tensor([[5999], [2499]], dtype=torch.int32, device=dev)
    freq = torch.from_numpy((1e4 ** -(np.arange(64) / 64)).astype(np.float32)).to(dev)
    bounds = tq.alloc_block_bounds(cache)
    ids = torch.empty((2, 2, 9), dtype=torch.int32, device=dev)
    outs = [torch.empty((2, 6, 1, 128), dtype=F32, device=dev), torch.empty((2, 6, 128), dtype=F32, device=dev),
            torch.empty((2, 6, 1, 128), dtype=F32, device=dev)]
    ws, ws_side = (tq.alloc_extend_workspace(cache, 6, 1) for _ in range(2))
    ws_blocks = tq.alloc_blocks_workspace(cache, 6, 9)
    side = torch.cuda.Stream()

    def run(wait=lambda: None):
        now = torch.cuda.current_stream()
        pos.zero_()
        side.wait_stream(now)
        with torch.cuda.stream(side):
            pos.copy_(pos_src)
        q.copy_(src)
        now.wait_stream(side)
        wait()
        tq.tq_norm_rope(q, None, turned, None, pos, freq, norm=True)
        wait()
        bounds.zero_()
        wait()
        tq.tq_block_bounds(qg, cache, bounds, 6000)
        wait()
        tq.tq_select_blocks(qg, cache, bounds, turned[:, :, 0], ids, ws_blocks, n_sink=1, n_recent=1)
        wait()
        side.wait_stream(now)
        with torch.cuda.stream(side):
            tq.tq_extend_attention(qg, cache, turned, outs[2], ws_side)
        wait()
        tq.tq_decode_attention_blocks(qg, cache, turned[:, :, 0], ids, outs[1], ws_blocks)
        wait()
        torch.mul(turned, 0.5, out=half)
        wait()
        tq.tq_extend_attention(qg, cache, half, outs[0], ws)
        wait()
        now.wait_stream(side)

    want = []
    for x in inputs:
        src.copy_(x)
        run(torch.cuda.synchronize)
        want.append([t.clone() for t in (turned, bounds, ids, *outs)])
    assert not torch.equal(want[0][3], want[1][3])
    again = run
    if captured:
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            run()
        again = graph.replay
    for i in range(30):
        src.copy_(inputs[i % 3])
        again()
        for got, w in zip((turned, bounds, ids, *outs), want[i % 3]):
            assert torch.equal(got, w)
    tq.tq_sync_status()


@pytest.mark.parametrize("mode,bits,vbits", [("prod", 4, 4), ("mse", 3, 2), ("grouped", 2, 4)])
def test_a_prompt_and_steps_with_all_of_them(mode, bits, vbits):
    """As a model's layer uses them: the projection's rows are normed and rotated, keys and values appended, their blocks'
    bounds taken; a prompt in two chunks through tq_extend_attention, then steps that attend to selected
    blocks. Each attention is held to its definition on the rows that the cache holds then."""
    require_cuda()
    B, hq, hkv, cap = 2, 8, 2, 512
    qo, qg = quantizers(mode, bits)
    cache = tq.KVCache(qg, B, hkv, cap, value_bits=vbits, device="cuda:0")
    bounds = tq.alloc_block_bounds(cache)
    g = torch.Generator("cuda").manual_seed(3)
    wq, wk = ((1 + 0.1 * torch.randn(128, generator=g, device="cuda")).to(BF16) for _ in range(2))
    freq = 1e4 ** (-torch.arange(64, device="cuda") / 64)
    at = 0
    for n in (130, 201, 1, 1, 3):
        x = torch.randn(B, n, (hq + 2 * hkv) * 128, generator=g, device="cuda").to(BF16)
        q, k, v = (t.view(B, n, -1, 128).transpose(1, 2) for t in x.split([hq * 128, hkv * 128, hkv * 128], -1))
        pos = (at + torch.arange(n, device="cuda", dtype=torch.int32)).repeat(B, 1)
        kn = torch.empty((B, hkv, n, 128), dtype=BF16, device="cuda")
        tq.tq_norm_rope(q, k, q, kn, pos, freq, q_weight=wq, k_weight=wk)
        tq.tq_append(qg, cache, kn, v.contiguous())
        tq.tq_block_bounds(qg, cache, bounds, n)
        at += n
        out = torch.empty((B, n, hq, 128), dtype=BF16, device="cuda").transpose(1, 2)
        tq.tq_extend_attention(qg, cache, q, out, tq.alloc_extend_workspace(cache, hq, n))
        ids, step = None, None
        if n == 1:
            ids = torch.empty((B, hkv, 4), dtype=torch.int32, device="cuda")
            step = torch.empty((B, hq, 128), dtype=BF16, device="cuda")
            ws = tq.alloc_blocks_workspace(cache, hq, 4)
            last = q[:, :, 0].contiguous()
            tq.tq_select_blocks(qg, cache, bounds, last, ids, ws, n_sink=1, n_recent=1)
            tq.tq_decode_attention_blocks(qg, cache, last, ids, step, ws)
        tq.tq_sync_status()
        parts = [[download_pair(cache, b, h, at) for h in range(hkv)] for b in range(B)]
        oc = {name: np.concatenate([np.concatenate([p[name] for p in row], 1) for row in parts], 0)
              for name in ("k_idx", "k_norms", "k_signs", "v_q", "v_params") if parts[0][0][name] is not None}
        oc["len"] = np.array([at] * B)
        some = sorted({0, n // 2, n - 1})
        ref, tol = attention64(qo, oc, q[:, :, some].float().cpu().numpy(), [[at - n + t + 1 for t in some]] * B, vbits)
        check(out[:, :, some], ref, tol, BF16)
        if n == 1:
            want = choice(qo, bounds.double().cpu().numpy(), last.double().cpu().numpy(), [at] * B, 4, 1, 1, O.default_head_map(hq, hkv))
            assert np.array_equal(ids.cpu().numpy(), want)
            keys = [[[i * BLOCK + t for i in want[b, h] for t in range(BLOCK) if i >= 0 and i * BLOCK + t < at] for h in range(hkv)] for b in range(B)]
            ref, tol = attention64(qo, oc, last[:, :, None].float().cpu().numpy(), [[at]] * B, vbits, keys=keys)
            check(step, ref[:, :, 0], tol[:, :, 0], BF16)
