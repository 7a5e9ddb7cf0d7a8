"""A decode over a cache in which every sequence is empty is planned like any other (CPU: in a process of its own, because
an integer division by zero would end it)."""
import os
import subprocess
import sys

import pytest

pytest.importorskip("kv_cache_vector_fwht_b200")

HERE = os.path.dirname(os.path.abspath(__file__))
CALL = """
import ctypes, sys
sys.path[:0] = [{here!r}, {root!r}]
import kv_cache_vector_fwht_b200 as tq
from test_abi_errors_around import dev, make_cache
q = tq.tq_build_codebook_host(128, 3, "prod", 0)
c = make_cache(lens=(0, 0))
got = tq._lib.tq_append_decode(q.handle, ctypes.byref(c), dev(20), dev(21), tq.TQ_BF16, 0, dev(22), tq.TQ_BF16, 4, None, 0.0,
                               dev(23), tq.TQ_F32, None, 0, dev(24), 1 << 30, None)
assert got in (tq.TQ_OK, tq.TQ_ECUDA), got
got = tq._lib.tq_decode_attention_noalloc(q.handle, ctypes.byref(c), dev(22), tq.TQ_BF16, 4, None, 0.0, dev(23), tq.TQ_F32,
                                          None, 0, None)
assert got == tq.TQ_ECUDA, got
"""


def test_a_cache_of_empty_sequences():
    r = subprocess.run([sys.executable, "-c", CALL.format(here=HERE, root=os.path.dirname(HERE))], capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stderr[-1000:])
