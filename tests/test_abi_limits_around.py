"""Sizes at which the operators around the cache would count beyond 32 bits, and outputs whose rows lie on one
another: refused, on CPU (fake device pointers, a quantizer without tables: a valid call ends in TQ_ECUDA)."""
import ctypes

import pytest

tq = pytest.importorskip("kv_cache_vector_fwht_b200")

from test_abi_errors_around import dev, heads, make_cache  # noqa: E402

lib = tq._lib
EINVAL, EUNSUP, ECUDA, OK = tq.TQ_EINVAL, tq.TQ_EUNSUPPORTED, tq.TQ_ECUDA, tq.TQ_OK
BF16 = tq.TQ_BF16


@pytest.fixture(scope="module")
def q():
    return tq.tq_build_codebook_host(128, 3, "prod", 0)


@pytest.mark.parametrize("capacity,status", [(1 << 30, ECUDA), ((1 << 30) + 16, EUNSUP), ((1 << 31) - 16, EUNSUP)])
def test_capacity(q, capacity, status):
    """Position 2^30 stands for a token that does not exist, and 2^31 - 16 rows and a tile more pass 32 bits."""
    c = make_cache(batch=1, n_kv=1, cap=capacity, lens=(10,))
    p, size = ctypes.byref(c), 1 << 40
    assert lib.tq_extend_attention(q.handle, p, heads(), BF16, 4, 3, 1, None, 0.0, heads(dev(11)), BF16, dev(30), size, None) == status
    assert lib.tq_block_bounds(q.handle, p, dev(9), 5, None) == status
    assert lib.tq_select_blocks(q.handle, p, dev(9), dev(10), BF16, 4, None, 3, 1, 1, dev(12), dev(13), size, None) == status
    assert lib.tq_decode_attention_blocks(q.handle, p, dev(10), BF16, 4, None, 0.0, dev(12), 3, dev(11), BF16, dev(13), size, None) == status
    n = ctypes.c_size_t()
    want = OK if status == ECUDA else EUNSUP
    assert lib.tq_extend_workspace_bytes(p, 4, 3, ctypes.byref(n)) == want
    assert lib.tq_blocks_workspace_bytes(p, 4, 3, ctypes.byref(n)) == want


@pytest.mark.parametrize("select,status", [(1 << 30, ECUDA), ((1 << 30) + 1, EUNSUP), ((1 << 31) - 1, EUNSUP)])
def test_blocks_listed(q, select, status):
    c = make_cache(batch=1, n_kv=1, lens=(10,))
    p, size = ctypes.byref(c), 1 << 40
    assert lib.tq_select_blocks(q.handle, p, dev(9), dev(10), BF16, 4, None, select, 1, 1, dev(12), dev(13), size, None) == status
    assert lib.tq_decode_attention_blocks(q.handle, p, dev(10), BF16, 4, None, 0.0, dev(12), select, dev(11), BF16, dev(13), size, None) == status
    n = ctypes.c_size_t()
    assert lib.tq_blocks_workspace_bytes(p, 4, select, ctypes.byref(n)) == (OK if status == ECUDA else EUNSUP)
    assert status != ECUDA or n.value < 1 << 31   # room for 1024 partial records at most


def test_rows_of_a_workspace(q):
    c, n = make_cache(), ctypes.c_size_t()
    assert lib.tq_extend_workspace_bytes(ctypes.byref(c), 4, 1 << 28, ctypes.byref(n)) == OK
    assert lib.tq_extend_workspace_bytes(ctypes.byref(c), 4, (1 << 28) + 1, ctypes.byref(n)) == EUNSUP


@pytest.mark.parametrize("stride", [0, 64, -64, 120])
@pytest.mark.parametrize("name", ["sb", "sh", "st"])
def test_outputs_whose_rows_overlap(q, stride, name):
    """Two rows on one place: which of them stays is a race. An input may repeat its rows."""
    c = make_cache()
    out = heads(dev(11), **{name: stride})
    assert lib.tq_extend_attention(q.handle, ctypes.byref(c), heads(), BF16, 4, 3, 1, None, 0.0, out, BF16, dev(30), 1 << 30, None) == EINVAL
    assert lib.tq_extend_attention(q.handle, ctypes.byref(c), heads(**{name: 0}), BF16, 4, 3, 1, None, 0.0, heads(dev(11)), BF16, dev(30),
                                   1 << 30, None) == ECUDA
    rope = tq.Rope(dev(1), dev(2), None, 1, 128, 0)
    none = tq.Heads(None, 0, 0, 0)
    assert lib.tq_norm_rope(ctypes.byref(rope), BF16, 2, 4, 128, 2, heads(), out, None, 0, none, none, None, 1, 1e-6, None) == EINVAL
    assert lib.tq_norm_rope(ctypes.byref(rope), BF16, 2, 4, 128, 0, none, none, None, 2, heads(), out, None, 1, 1e-6, None) == EINVAL
    assert lib.tq_norm_rope(ctypes.byref(rope), BF16, 2, 4, 128, 2, heads(**{name: 0}), heads(dev(11)), None, 0, none, none, None, 1, 1e-6,
                            None) == ECUDA


def test_strides_that_no_step_takes_are_free(q):
    """One sequence, one head or one token: their stride is not used."""
    c = make_cache(batch=1, lens=(10,))
    out = heads(dev(11), sb=0, st=0)
    assert lib.tq_extend_attention(q.handle, ctypes.byref(c), heads(), BF16, 4, 1, 1, None, 0.0, out, BF16, dev(30), 1 << 30, None) == ECUDA
    assert lib.tq_extend_attention(q.handle, ctypes.byref(c), heads(), BF16, 4, 3, 1, None, 0.0, heads(dev(11), st=-512), BF16, dev(30),
                                   1 << 30, None) == ECUDA
