"""tq_norm_rope with the axes of its frequencies given as lists, arrays and tensors."""
import array

import numpy as np
import pytest
import torch

from gpu_util import require_cuda

pytestmark = pytest.mark.gpu

import kv_cache_vector_fwht_b200 as tq  # noqa: E402

BF16 = torch.bfloat16


@pytest.mark.parametrize("make", [np.array, lambda a: np.array(a, dtype=np.uint8), torch.tensor, tuple, bytes, lambda a: array.array("l", a), lambda a: np.repeat(a, 2)[::2]],
                         ids=["int64", "uint8", "tensor", "tuple", "bytes", "array", "strided"])
def test_axes_given_as_any_sequence(make):
    require_cuda()
    g = torch.Generator("cuda").manual_seed(3)
    q = torch.randn(2, 3, 5, 128, generator=g, device="cuda").to(BF16)
    pos = torch.randint(0, 5000, (3, 2, 5), generator=g, device="cuda", dtype=torch.int32)
    freq = (1e4 ** (-torch.arange(64, device="cuda") / 64)).float()
    axes = [i % 3 for i in range(64)]
    want, got = torch.empty_like(q), torch.empty_like(q)
    tq.tq_norm_rope(q, None, want, None, pos, freq, axis_of_freq=axes)
    tq.tq_norm_rope(q, None, got, None, pos, freq, axis_of_freq=make(axes))
    assert torch.equal(want, got)


def test_axes_out_of_range_are_refused():
    require_cuda()
    q = torch.zeros(1, 1, 1, 128, device="cuda")
    pos, freq = torch.zeros(3, 1, 1, device="cuda", dtype=torch.int32), torch.ones(64, device="cuda")
    for axes in ([256] * 64, [-1] * 64, np.full(64, 256), np.full(64, -1)):
        with pytest.raises(ValueError):
            tq.tq_norm_rope(q, None, q, None, pos, freq, axis_of_freq=axes)
    for axes in ([0.0] * 64, np.zeros(64)):
        with pytest.raises(TypeError):
            tq.tq_norm_rope(q, None, q, None, pos, freq, axis_of_freq=axes)
    for axes in ([3] * 64, np.full(64, 3)):
        with pytest.raises(tq.TQError):
            tq.tq_norm_rope(q, None, q, None, pos, freq, axis_of_freq=axes)
