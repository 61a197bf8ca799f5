"""Paged 8-bit cache at its limits: what the kernels rely on between threads, the largest work lists, and
the precision that include/tq.h states."""
import os
import re

import numpy as np
import pytest

import b8_reference as ref
from test_b8 import Pair, close, lib, m  # noqa: F401  (lib and m are fixtures)

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


def test_shuffles_name_their_threads():
    """A mask taken from whoever is together after a branch need not hold a shuffle's partner."""
    for name in os.listdir(CSRC):
        assert "__activemask" not in source(name), name


# ----------------------------------------------------------------------------- GPU
@pytest.mark.gpu
@pytest.mark.parametrize("d,g,n_q", [(64, 4, 1), (40, 3, 1), (64, 4, 2), (64, 16, 1)])
def test_attention_where_some_warps_have_nothing(m, d, g, n_q):
    """One to nine units a segment: the sums of warps without a unit, and of warps whose factor is 0 (their tokens
    lie far below the largest logit), stand beside those of the others. At D = 64 two threads share an item."""
    lens = [32 * k + (k % 3) * 7 for k in range(1, 9)]
    p = Pair(m, d, 2, len(lens), 11, 70 + d + g)
    p.append(lens)
    q, q64 = p.queries(n_q, g, "bf16")
    ws = p.workspace(n_q, g)
    for scale in (d ** -0.5, 5.0):
        out = p.torch.full(q.shape, float("nan"), device="cuda")
        m.tq_b8_attention(p.cache, q, scale, out, ws)
        got = out.double().cpu().numpy().reshape(q64.shape)
        for s, sq in enumerate(p.seqs):
            want, _, size, reach = ref.attention(sq, q64[s], scale)
            close(got[s], want, size, reach, d)
    assert p.ok(ws)
