"""Kernels that may start before the stream's previous kernel ends (programmatic
serialization) must not read global memory by the read-only path: it promises
data that does not change while the grid runs, and the previous kernel may still
write it. Read from the sources, on the CPU."""
import os
import re

import pytest

from fp8_fine_grained_gb300 import build as libbuild

READ_ONLY = re.compile(r"__ldg\s*\(|ld\.global\.nc|const\s+\w+\s*\*\s*__restrict__|\w+\s+const\s*\*\s*__restrict__")


def code(path):
    """A source file without its comments."""
    with open(path) as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


SOURCES = sorted(f for f in os.listdir(libbuild.CSRC) if f.endswith((".cu", ".cuh")))
EARLY = [f for f in SOURCES if f.endswith(".cu") and "griddep_wait" in code(os.path.join(libbuild.CSRC, f))]


def test_the_early_starters_are_found():
    assert {"norm.cu", "clip.cu", "gated_bwd.cu", "gemm_gated.cu", "gemm.cu", "gemm_mx.cu"} <= set(EARLY)


@pytest.mark.parametrize("name", EARLY + [f for f in SOURCES if f.endswith(".cuh")])
def test_no_read_only_loads(name):
    found = READ_ONLY.search(code(os.path.join(libbuild.CSRC, name)))
    assert found is None, "%s: %s" % (name, found.group(0))


def test_the_search_finds_each_form():
    for text in ("v = __ldg(p + 1);", 'asm("ld.global.nc.v4.u32");', "const float *__restrict__ x",
                 "const uint16_t * __restrict__ x", "float const *__restrict__ x"):
        assert READ_ONLY.search(text)
    assert not READ_ONLY.search("uint8_t *__restrict__ q; const float *x;")
