"""tq_norm_rope against its definition in 64 bits."""
import numpy as np
import pytest
import torch

from gpu_util import require_cuda

pytestmark = pytest.mark.gpu

import kv_cache_vector_fwht_b200 as tq  # noqa: E402

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def reference(x, w, norm, eps, pos, freq, axes, interleaved):
    """(values, the sum of magnitudes that a rounding in 32 bits is relative to)."""
    y = x.double()
    if norm:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt()
        y = y * w.double() if w is not None else y
    pairs = freq.numel()
    pos = pos if pos.dim() == 3 else pos[None]
    angle = pos.double()[list(axes) if axes is not None else [0] * pairs].permute(1, 2, 0) * freq.double()
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    z, size = y.clone(), y.abs()
    a, b = (slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)) if interleaved else (slice(0, pairs), slice(pairs, 2 * pairs))
    z[..., a], z[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
    size[..., a] = size[..., b] = y[..., a].abs() + y[..., b].abs()
    return z, size


def check(got, want, size, dtype):
    """Half a step of the output's type, and 2^-20 of the pair for the 32-bit arithmetic: the norm (a sum of 128
    squares, the root, two products: under 8 roundings of 2^-24 in y), the turn (cos and sin off by 2^-22 from
    the angle's 2^-25 turns and the functions' 2 ulp; two products and a sum)."""
    bound = torch.finfo(dtype).eps / 2 * want.abs() + 2.0 ** -20 * size + torch.finfo(dtype).smallest_normal * 2.0 ** -9
    worst = ((got.double() - want).abs() / bound).max().item() if got.numel() else 0.0
    assert worst <= 1, f"{worst:.2f} times the bound"


def inputs(seed, batch, n, hq, hk, dtype, axes, far, pairs):
    g = torch.Generator("cuda").manual_seed(seed)
    q = (3 * torch.randn(batch, hq, n, 128, generator=g, device="cuda")).to(dtype)
    k = (0.01 * torch.randn(batch, hk, n, 128, generator=g, device="cuda")).to(dtype)
    pos = torch.randint(-far // 10, far, (axes, batch, n), generator=g, device="cuda", dtype=torch.int32)
    freq = (5e5 ** (-torch.arange(pairs, device="cuda", dtype=torch.float64) / max(1, pairs))).float()
    wq, wk = ((1 + 0.3 * torch.randn(128, generator=g, device="cuda")).to(dtype) for _ in range(2))
    return q, k, pos, freq, wq, wk


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [16, 64, 96, 128])
@pytest.mark.parametrize("axes", [1, 3])
def test_types_pairs_and_axes(dtype, interleaved, rot, axes):
    require_cuda()
    pairs = rot // 2
    q, k, pos, freq, wq, wk = inputs(rot + axes, 2, 5, 6, 2, dtype, axes, 1_000_000, pairs)
    axis = [i * axes // pairs for i in range(pairs)] if axes > 1 else None
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    tq.tq_norm_rope(q, k, qo, ko, pos, freq, q_weight=wq, k_weight=wk, eps=1e-5, axis_of_freq=axis, interleaved=interleaved)
    for x, o, w in ((q, qo, wq), (k, ko, wk)):
        want, size = reference(x, w, True, 1e-5, pos, freq, axis, interleaved)
        check(o, want, size, dtype)


@pytest.mark.parametrize("batch,n,hq,hk", [(1, 1, 1, 0), (1, 1, 1, 1), (3, 1, 28, 4), (1, 3, 64, 8), (1, 700, 12, 2), (2, 333, 5, 1),
                                           (1, 2, 200, 56), (5, 7, 17, 1), (1, 1, 0, 4)])
@pytest.mark.parametrize("norm", [False, True])
def test_shapes(batch, n, hq, hk, norm):
    """One token and one head up to hundreds; queries or keys alone; a norm without weights and none."""
    require_cuda()
    q, k, pos, freq, _, _ = inputs(batch + n, batch, n, max(hq, 1), max(hk, 1), BF16, 1, 4096, 64)
    q, k = (q if hq else None), (k if hk else None)
    qo, ko = (torch.empty_like(x) if x is not None else None for x in (q, k))
    tq.tq_norm_rope(q, k, qo, ko, pos[0].contiguous(), freq, norm=norm)
    for x, o in ((q, qo), (k, ko)):
        if x is not None:
            want, size = reference(x, None, norm, 1e-6, pos, freq, None, False)
            check(o, want, size, BF16)


def test_projection_views_appended_layout_and_in_place():
    """Queries and keys as views of one projection's rows; keys straight into the layout that tq_append takes;
    in place; the projection's other elements stay."""
    require_cuda()
    B, n, hq, hk = 2, 9, 6, 2
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(B, n, (hq + 2 * hk) * 128, generator=g, device="cuda").to(F16)
    keep = x.clone()
    q = x[..., :hq * 128].view(B, n, hq, 128).transpose(1, 2)
    k = x[..., hq * 128:(hq + hk) * 128].view(B, n, hk, 128).transpose(1, 2)
    _, _, pos, freq, wq, wk = inputs(2, B, n, 1, 1, F16, 1, 100, 64)
    wants = [reference(t, w, True, 1e-6, pos, freq, None, True) for t, w in ((q, wq), (k, wk))]
    ko = torch.empty((B, hk, n, 128), dtype=F16, device="cuda")
    tq.tq_norm_rope(q, k, q, ko, pos, freq, q_weight=wq, k_weight=wk, interleaved=True)
    check(q, *wants[0], F16)
    check(ko, *wants[1], F16)
    assert torch.equal(x[..., hq * 128:], keep[..., hq * 128:])


def test_rows_of_zeros_and_large_values():
    require_cuda()
    q = torch.zeros(1, 3, 2, 128, device="cuda")
    q[0, 1] = 1e18
    q[0, 2, 0, 5] = float("inf")
    out = torch.empty_like(q)
    pos, freq = torch.tensor([[3, 70000]], dtype=torch.int32, device="cuda"), torch.ones(64, device="cuda")
    tq.tq_norm_rope(q, None, out, None, pos, freq, norm=True)
    assert not out[0, 0].any()
    want, size = reference(q, None, True, 1e-6, pos, freq, None, False)
    check(out[0, 1:2], want[0, 1:2], size[0, 1:2], F32)
    check(out[0, 2, 1], want[0, 2, 1], size[0, 2, 1], F32)   # a spoilt row spoils no other


def test_channels_that_do_not_turn_are_only_scaled():
    require_cuda()
    q, _, pos, freq, _, _ = inputs(3, 1, 4, 2, 1, BF16, 1, 4096, 8)
    out = torch.empty_like(q)
    tq.tq_norm_rope(q, None, out, None, pos, freq, norm=False)
    assert torch.equal(out[..., 16:], q[..., 16:]) and not torch.equal(out[..., :16], q[..., :16])
    nothing = torch.empty(0, device="cuda")
    tq.tq_norm_rope(q, None, out, None, pos, nothing, norm=False)
    assert torch.equal(out, q)


def test_capture_and_another_stream():
    require_cuda()
    q, k, pos, freq, wq, wk = inputs(4, 2, 6, 8, 2, BF16, 1, 4096, 64)
    want, got = (torch.empty_like(q), torch.empty_like(k)), (torch.zeros_like(q), torch.zeros_like(k))
    tq.tq_norm_rope(q, k, *want, pos, freq, q_weight=wq, k_weight=wk)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tq.tq_norm_rope(q, k, *got, pos, freq, q_weight=wq, k_weight=wk)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    s = torch.cuda.Stream()
    for t in got:
        t.zero_()
    torch.cuda.synchronize()
    tq.tq_norm_rope(q, k, *got, pos, freq, q_weight=wq, k_weight=wk, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert np.isfinite(got[0].float().cpu().numpy()).all()
