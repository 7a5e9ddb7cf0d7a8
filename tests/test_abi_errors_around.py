"""Host argument checks of the operators around the cache (tq_norm_rope, tq_extend_attention,
tq_block_bounds, tq_select_blocks, tq_decode_attention_blocks), on CPU: fake device pointers, a
quantizer without device tables, so that a call whose arguments are all valid ends in TQ_ECUDA
and any other status shows the check that fired. Nothing is launched."""
import ctypes

import pytest

tq = pytest.importorskip("kv_cache_vector_fwht_b200")

lib = tq._lib
EINVAL, EUNSUP, ECUDA, OK = tq.TQ_EINVAL, tq.TQ_EUNSUPPORTED, tq.TQ_ECUDA, tq.TQ_OK
F32, BF16, F16 = tq.TQ_F32, tq.TQ_BF16, tq.TQ_F16


def dev(i):
    """Distinct fake device buffers, 1 MiB apart (16-byte aligned)."""
    return (1 << 32) + i * (1 << 20)


@pytest.fixture(scope="module")
def q():
    return tq.tq_build_codebook_host(128, 3, "prod", 0)


def make_cache(batch=2, n_kv=2, cap=64, vbits=2, lens=(10, 20), d=128, signs=dev(2)):
    host = (ctypes.c_int32 * batch)(*lens)
    desc = tq.KVCacheDesc(batch, n_kv, cap, d, vbits, 32, tq.KeyPlanes(dev(1), signs, dev(3)),
                          tq.ValuePlanes(dev(4) if vbits else None, dev(5) if vbits else None), dev(6), host)
    desc.keep = host
    return desc


def heads(data=dev(10), sb=1024, sh=128, st=128):
    return tq.Heads(data, sb, sh, st)


# ------------------------------------------------------------------ tq_norm_rope
@pytest.mark.parametrize("change,status", [
    ({}, ECUDA),
    (dict(rope=False), EINVAL),
    (dict(d=64), EUNSUP),
    (dict(dtype=7), EUNSUP),
    (dict(batch=-1), EINVAL),
    (dict(n=-1), EINVAL),
    (dict(batch=0), OK),
    (dict(n=0), OK),
    (dict(hq=-1), EINVAL),
    (dict(hq=0, hk=0), OK),
    (dict(rot=24), EINVAL),
    (dict(rot=-16), EINVAL),
    (dict(rot=144), EINVAL),
    (dict(pos=None), EINVAL),
    (dict(pos=dev(1) + 2), EINVAL),
    (dict(freq=None), EINVAL),
    (dict(axes=0), EINVAL),
    (dict(axes=256), EINVAL),
    (dict(axis=b"\x01" * 64), EINVAL),            # one axis: only 0
    (dict(eps=-1.0), EINVAL),
    (dict(eps=float("nan")), EINVAL),
    (dict(q=heads(None)), EINVAL),
    (dict(q=heads(dev(10) + 8)), EINVAL),
    (dict(qo=heads(dev(11), st=132)), EINVAL),    # rows off 16 bytes (bf16)
    (dict(k=heads(dev(12), sb=1028)), EINVAL),
    (dict(ko=heads(None)), EINVAL),
    (dict(wq=dev(20) + 4), EINVAL),
])
def test_norm_rope_checks(change, status):
    a = dict(rope=True, dtype=BF16, batch=2, n=4, d=128, hq=2, hk=2, rot=128, pos=dev(1), freq=dev(2), axes=1, axis=None,
             q=heads(dev(10)), qo=heads(dev(11)), wq=dev(20), k=heads(dev(12)), ko=heads(dev(13)), wk=None, eps=1e-6)
    a.update(change)
    rope = tq.Rope(a["pos"], a["freq"], a["axis"], a["axes"], a["rot"], 0)
    got = lib.tq_norm_rope(ctypes.byref(rope) if a["rope"] else None, a["dtype"], a["batch"], a["n"], a["d"], a["hq"], a["q"],
                           a["qo"], a["wq"], a["hk"], a["k"], a["ko"], a["wk"], 1, a["eps"], None)
    assert got == status


def test_norm_rope_unused_side_and_unturned_rows_need_no_pointers():
    rope = tq.Rope(None, None, None, 0, 0, 0)      # rot_dim 0: no positions, no frequencies
    none = tq.Heads(None, 0, 0, 0)
    assert lib.tq_norm_rope(ctypes.byref(rope), F32, 1, 1, 128, 1, heads(dev(1)), heads(dev(2)), None, 0, none, none, None,
                            0, -1.0, None) == ECUDA


# ------------------------------------------------------------------ tq_extend_attention
@pytest.mark.parametrize("change,status", [
    ({}, ECUDA),
    (dict(q=None), EINVAL),
    (dict(cache=None), EINVAL),
    (dict(cache=make_cache(d=64)), EUNSUP),
    (dict(cache=make_cache(vbits=0)), EINVAL),      # attention needs values
    (dict(cache=make_cache(signs=None)), EINVAL),
    (dict(cache=make_cache(lens=(10, 65))), EINVAL),
    (dict(cache=make_cache(lens=(-1, 5))), EINVAL),
    (dict(hq=0), EINVAL),
    (dict(hq=3), EINVAL),
    (dict(hq=514), EINVAL),
    (dict(map=[0, 1, 2, 0]), EINVAL),
    (dict(map=[0, -1, 1, 0]), EINVAL),
    (dict(map=[0, 1, 1, 1]), ECUDA),
    (dict(n=-1), EINVAL),
    (dict(n=0), OK),
    (dict(n=1 << 29), EUNSUP),
    (dict(qdt=5), EUNSUP),
    (dict(odt=5), EUNSUP),
    (dict(qdt=F16, odt=F32), ECUDA),
    (dict(query=heads(None)), EINVAL),
    (dict(query=heads(dev(10) + 2)), EINVAL),
    (dict(query=heads(dev(10), sh=129)), EINVAL),
    (dict(out=heads(None)), EINVAL),
    (dict(out=heads(dev(11), st=4)), EINVAL),
    (dict(ws=None), EINVAL),
    (dict(ws=dev(30) + 8), EINVAL),
    (dict(short=1), EINVAL),
])
def test_extend_checks(q, change, status):
    a = dict(q=q.handle, cache=make_cache(), query=heads(dev(10)), qdt=BF16, hq=4, n=3, map=None, out=heads(dev(11)), odt=BF16,
             ws=dev(30), short=0)
    a.update(change)
    n = ctypes.c_size_t()
    need = 1 << 30
    if a["cache"] is not None and lib.tq_extend_workspace_bytes(ctypes.byref(a["cache"]), a["hq"], max(0, a["n"]), ctypes.byref(n)) == OK:
        need = n.value
    m = (ctypes.c_int32 * a["hq"])(*a["map"]) if a["map"] else None
    got = lib.tq_extend_attention(a["q"], ctypes.byref(a["cache"]) if a["cache"] is not None else None, a["query"], a["qdt"], a["hq"], a["n"], 1, m, 0.0, a["out"], a["odt"],
                                  a["ws"], need - a["short"], None)
    assert got == status


def test_workspace_sizes():
    n = ctypes.c_size_t()
    c = make_cache()
    assert lib.tq_extend_workspace_bytes(ctypes.byref(c), 4, 3, ctypes.byref(n)) == OK and n.value >= 64 << 10
    small = n.value
    assert lib.tq_extend_workspace_bytes(ctypes.byref(c), 4, 500, ctypes.byref(n)) == OK and n.value > small
    assert lib.tq_extend_workspace_bytes(ctypes.byref(c), 0, 3, ctypes.byref(n)) == EINVAL
    assert lib.tq_extend_workspace_bytes(ctypes.byref(c), 4, -1, ctypes.byref(n)) == EINVAL
    assert lib.tq_extend_workspace_bytes(None, 4, 3, ctypes.byref(n)) == EINVAL
    assert lib.tq_blocks_workspace_bytes(ctypes.byref(c), 4, 2, ctypes.byref(n)) == OK and n.value > 64 << 10
    assert lib.tq_blocks_workspace_bytes(ctypes.byref(c), 4, 0, ctypes.byref(n)) == EINVAL
    assert lib.tq_blocks_workspace_bytes(ctypes.byref(c), 4, 2, None) == EINVAL


# ------------------------------------------------------------------ bounds, selection, listed blocks
@pytest.mark.parametrize("change,status", [
    ({}, ECUDA), (dict(n=0), OK), (dict(n=-1), EINVAL), (dict(bounds=None), EINVAL), (dict(bounds=dev(9) + 4), EINVAL),
    (dict(cache=make_cache(vbits=0)), ECUDA),      # keys are enough
    (dict(q=None), EINVAL), (dict(cache=None), EINVAL),
])
def test_bounds_checks(q, change, status):
    a = dict(q=q.handle, cache=make_cache(), bounds=dev(9), n=5)
    a.update(change)
    assert lib.tq_block_bounds(a["q"], ctypes.byref(a["cache"]) if a["cache"] is not None else None, a["bounds"], a["n"], None) == status


@pytest.mark.parametrize("change,status", [
    ({}, ECUDA),
    (dict(sel=0), EINVAL),
    (dict(sink=-1), EINVAL),
    (dict(recent=-1), EINVAL),
    (dict(sink=2, recent=1, sel=2), EINVAL),
    (dict(sink=2, recent=0, sel=2), ECUDA),
    (dict(bounds=None), EINVAL),
    (dict(query=None), EINVAL),
    (dict(query=dev(10) + 4), EINVAL),
    (dict(qdt=9), EUNSUP),
    (dict(ids=None), EINVAL),
    (dict(ids=dev(12) + 2), EINVAL),
    (dict(ws=None), EINVAL),
    (dict(size=1000), EINVAL),
    (dict(cache=make_cache(batch=1, lens=(5,), n_kv=600), hq=4, map=[0, 1, 2, 3]), EUNSUP),
])
def test_select_checks(q, change, status):
    a = dict(cache=make_cache(), bounds=dev(9), query=dev(10), qdt=BF16, hq=4, map=None, sel=3, sink=1, recent=1, ids=dev(12),
             ws=dev(13), size=1 << 20)
    a.update(change)
    m = (ctypes.c_int32 * a["hq"])(*a["map"]) if a["map"] else None
    assert lib.tq_select_blocks(q.handle, ctypes.byref(a["cache"]), a["bounds"], a["query"], a["qdt"], a["hq"], m, a["sel"],
                                a["sink"], a["recent"], a["ids"], a["ws"], a["size"], None) == status


@pytest.mark.parametrize("change,status", [
    ({}, ECUDA), (dict(sel=0), EINVAL), (dict(ids=None), EINVAL), (dict(query=None), EINVAL), (dict(out=None), EINVAL),
    (dict(out=dev(11) + 8), EINVAL), (dict(odt=4), EUNSUP), (dict(cache=make_cache(vbits=0)), EINVAL), (dict(size=1 << 15), EINVAL),
    (dict(hq=5), EINVAL),
])
def test_decode_blocks_checks(q, change, status):
    a = dict(cache=make_cache(), query=dev(10), qdt=BF16, hq=4, ids=dev(12), sel=3, out=dev(11), odt=BF16, ws=dev(13), size=1 << 24)
    a.update(change)
    assert lib.tq_decode_attention_blocks(q.handle, ctypes.byref(a["cache"]), a["query"], a["qdt"], a["hq"], None, 0.0, a["ids"],
                                          a["sel"], a["out"], a["odt"], a["ws"], a["size"], None) == status


# ------------------------------------------------------------------ the binding's own checks
def test_binding_refuses_tensors_of_another_kind():
    import torch
    x = torch.zeros(1, 2, 3, 128)
    pos, freq = torch.zeros(1, 3, dtype=torch.int32), torch.ones(64)
    with pytest.raises(ValueError, match="needed"):
        tq.tq_norm_rope(None, None, None, None, pos, freq)
    with pytest.raises(ValueError, match="outputs as their inputs"):
        tq.tq_norm_rope(x, None, x[:, :1], None, pos, freq)
    with pytest.raises(ValueError, match="output without"):
        tq.tq_norm_rope(x, None, x, x, pos, freq)
    with pytest.raises(ValueError, match="one type"):
        tq.tq_norm_rope(x, x.half(), x, x.half(), pos, freq)
    with pytest.raises(ValueError, match="adjacent"):
        tq.tq_norm_rope(x.transpose(2, 3)[:, :, :, :3].new_zeros(1, 2, 3, 256)[..., ::2], None, x, None, pos, freq)
    with pytest.raises(ValueError, match="weights"):
        tq.tq_norm_rope(x, None, x, None, pos, freq, q_weight=torch.ones(64))
    with pytest.raises(ValueError, match="positions"):
        tq.tq_norm_rope(x, None, x, None, pos.long(), freq)
    with pytest.raises(ValueError, match="positions"):
        tq.tq_norm_rope(x, None, x, None, torch.zeros(2, 2, dtype=torch.int32), freq)
    with pytest.raises(ValueError, match="inv_freq"):
        tq.tq_norm_rope(x, None, x, None, pos, freq.double())
