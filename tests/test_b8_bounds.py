"""Paged 8-bit cache at its limits: what the kernels rely on between threads, the largest work lists, and
the precision that include/tq.h states."""
import os
import re

import numpy as np
import pytest

import b8_reference as ref
from test_b8 import Pair, lib, m  # noqa: F401  (the two modules of entry points are fixtures)

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kv_cache_vector_03_b200", "csrc")


def source(name):
    """The code of a source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


# ----------------------------------------------------------------------------- CPU
def test_the_page_ring_is_ready_before_any_warp_uses_it():
    """All warps of a CTA issue copies into the ring whose barriers the first warp initialises: a barrier of the
    block stands between, on every path (the plan has none where every warp makes it for itself)."""
    code = source("k_b8_attn.cu")
    assert code.count("tq_fence_mbar_init();") == 1
    after = code[code.index("tq_fence_mbar_init();"):]
    assert "__syncthreads();" in after[:after.index("tq_pdl_wait();")]
