"""Kernels that may start before the stream's previous kernel has ended: what their sources must and must not hold."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kv_cache_vector_fwht_b200", "csrc")


def code(name):
    """A source file without its comments."""
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))


def early():
    return [n for n in sorted(os.listdir(CSRC)) if re.search(r"__global__", code(n)) and "wait_for_grid();" in code(n)]


def test_there_are_such_kernels():
    assert {"blocks.cu", "extend_kernel.cuh", "rope.cu"} <= set(early())


@pytest.mark.parametrize("name", early())
def test_no_load_that_takes_memory_for_constant(name):
    """The previous kernel may still be writing what these read: ld.global.nc (__ldg, and load4 and load8, which use
    it) may be served from a cache that does not see it, and may be moved before the wait."""
    found = re.findall(r"__ldg\s*\(|ld\.global\.nc|\bload[48]\s*<", code(name))
    assert not found


@pytest.mark.parametrize("name", early())
def test_every_kernel_waits(name):
    kernels = re.findall(r"__global__[^;{]*?\b(k_\w+)\s*\(", code(name))
    assert kernels and len(re.findall(r"wait_for_grid\(\);", code(name))) == len(kernels)


def test_the_decode_reads_no_cache_row_as_constant():
    """tq_append_decode launches the decode over the append: what it reads behind its wait was written meanwhile."""
    text = code("decode_kernel.cuh")
    after = text[text.index("grid_dependency_wait();"):]
    assert "load_keys" in after and not re.search(r"__ldg\s*\(|\bload[48]\s*<", after)
