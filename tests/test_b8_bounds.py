"""Paged 8-bit cache at its limits: what the kernels rely on between threads, the largest work lists, and
the precision that include/tq.h states."""
import ctypes
import os
import re
import subprocess

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


SHARES = r"""
#include <cstdio>
#include "b8_shares.h"
// units, segments and CTAs on each line of input: shares have to be in order, cover the price and know their own units
int main() {
    long long units, segments, ctas;
    while (scanf("%lld %lld %lld", &units, &segments, &ctas) == 3) {
        B8Shares s;
        s.make((int)units, (int)segments, (int)ctas);
        const long long price = units + (long long)s.per * segments;
        bool good = s.per >= 0 && price < (1ll << 31) && s.price((int)units, (int)segments) == price && s.share(0) == 0 &&
                    s.share((int)ctas) == price && s.base > 0;
        for (int c = 0; good && c < ctas; ++c) {
            const int lo = s.share(c), hi = s.share(c + 1);
            good = lo < hi && s.owner(lo) == c && s.owner(hi - 1) == c;
        }
        printf("%d %d\n", (int)good, s.per);
    }
}
"""


def test_equal_shares_over_the_largest_lists(tmp_path):
    """The host accepts (blocks + 1) x segments up to 2^30; a segment has at most two units more than blocks: up to 2^29
    segments of one to three units. Their shares are worked out in 32 bits."""
    (tmp_path / "shares.cpp").write_text(SHARES)
    subprocess.check_call(["g++", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", CSRC, "-o",
                           str(tmp_path / "shares"), str(tmp_path / "shares.cpp")])
    cases = []
    for segments in (1, 2, 295, 296, 297, 5000, 10 ** 6, 195225786, 195225787, 214954800, 196608000, 2 ** 28, 390451573, 2 ** 29 - 1, 2 ** 29):
        for each in (1, 2, 3, 31, 33, 2 ** 10, 2 ** 23):
            units = segments * each
            if segments * max(2, each - 1) <= 2 ** 30:
                cases += [(units, segments, c) for c in {1, 2, min(units, 7), min(units, 296), min(units, 384)} if c <= units]
    r = subprocess.run([str(tmp_path / "shares")], input="\n".join("%d %d %d" % c for c in cases), text=True,
                       capture_output=True, check=True)
    out = [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
    assert len(out) == len(cases) > 200
    for case, (good, per) in zip(cases, out):
        assert good, case
        assert (per == 0) == (case[0] + 10 * case[1] >= 2 ** 31), case       # priced beside its units wherever that fits


@pytest.mark.parametrize("n_q,g,n_sel,weights", [(16384, 1, 1, 0), (1, 16384, 0, 1), (16384, 1, 1 << 23, 1), (16384, 1, 0, 1),
                                                 (8192, 2, 3, 0)])
def test_workspaces_beyond_64_bits_are_unsupported(lib, n_q, g, n_sel, weights):
    """Sizes that do not fit a size_t are no sizes, and the calls that would need them are refused."""
    c = lib.tq_b8_cache(64, 1024, 65535, 64, 1 << 23, 0x10000, 0x20000, 0x30000, 0x40000)
    r = ctypes.byref(c)
    assert lib.lib.tq_b8_workspace_bytes(r, n_q, g, n_sel, weights) == 0
    ws, most = 0x100000, 2 ** 64 - 1
    if n_sel:
        assert lib.lib.tq_b8_select(r, 0x1000, 1, n_q, g, 0, 0, n_sel, 0x2000, ws, most, None) == lib.TQ_ERR_UNSUPPORTED
    if weights and not n_sel:
        st = lib.lib.tq_b8_attention(r, 0x1000, 1, n_q, g, 0.1, None, 0, None, 0x5000, 1.0, 0x2000, ws, most, None)
        assert st == lib.TQ_ERR_UNSUPPORTED


def test_an_empty_selection_is_refused(lib):
    """A tensor without entries has no address, which would ask for all blocks."""
    import torch
    d, n_kv, n_seq, nb = 64, 2, 3, 4
    c = lib.Cache8(d, torch.zeros(12, lib.tq_b8_page_bytes(d, n_kv), dtype=torch.uint8),
                   torch.zeros(n_seq, nb, dtype=torch.int32), torch.zeros(n_seq, dtype=torch.int32),
                   torch.zeros(n_seq, n_kv, 2, 32, d, dtype=torch.bfloat16))
    q, sel = torch.zeros(n_seq, 1, 4, d), torch.zeros(n_seq, 1, n_kv, 0, dtype=torch.int32)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="sel"):
        lib.tq_b8_attention(c, q, 1.0, torch.zeros_like(q), ws, sel=sel)
    with pytest.raises(ValueError, match="sel"):
        lib.tq_b8_select(c, q, sel, ws, n_first=0, n_last=0)


def test_no_sequences_with_a_selection_is_a_no_op(lib):
    """As without one: tensors of no sequences have no addresses."""
    r = ctypes.byref(lib.tq_b8_cache(128, 8, 0, 64, 16, 0x10000, None, None, None))
    for n_sel in (0, 4):
        st = lib.lib.tq_b8_attention(r, None, 1, 1, 4, 0.1, None, n_sel, None, None, 1.0, None, 0x100000, 1 << 20, None)
        assert st == lib.TQ_OK


def within(got, sq, q, scale, lost=0.0, n_sum=64):
    """Output rows against 64 bits, where a logit of whole pages is off by 2^-23 of itself (its whole-number sum and its
    distance to the block's largest in fp32), by 2^-24 max |q| max |k| (the small pieces' share of that sum) and by
    `lost`, what q itself loses. Weights move by twice that; their pieces, exponentials, matrix products and up to n_sum
    additions in a row are off by 2^-24 of sum w |v| each (n_sum + 64 of them in all)."""
    want, weight, size, _ = ref.attention(sq, q, scale)
    k = np.abs(sq.values()[:, :, 0])                                             # [n, n_kv, d]
    logit = np.abs(scale * np.einsum("ihgd,nhd->ihgn", q, sq.values()[:, :, 0])).max(axis=-1)
    dl = 2.0 ** -23 * logit + abs(scale) * 2.0 ** -24 * np.abs(q).max(axis=-1) * k.max() + lost
    bound = (np.expm1(2 * dl) + (n_sum + 64) * 2.0 ** -24) * size
    err = np.abs(got - want).max(axis=-1)
    assert np.isfinite(got).all()
    assert (err <= bound + 1e-30).all(), (float((err / np.maximum(bound, 1e-30)).max()), (err / np.maximum(size, 1e-300)).max(axis=(0, 1, 2)))
    return dl


@pytest.mark.parametrize("d,n", [(128, 64), (128, 1024), (64, 320), (256, 96)])
def test_the_bounds_see_what_a_kernel_could_lose(d, n):
    """Planted in the reference: weights in one fp16 piece, weights cut off 2^-20 below a heavy token without a value, and a
    query in 14 bits are outside the bounds; fp32 weights and a query in 22 bits are inside."""
    rng = np.random.default_rng(d + n)
    n_kv, g, scale = 2, 4, d ** -0.5
    sq = ref.Seq(n_kv, d)
    k, v = rng.standard_normal((n, n_kv, d)), rng.standard_normal((n, n_kv, d))
    k[..., 0], k[5], v[5] = 0.0, 0.0, 0.0
    k[5, :, 0] = 16.0 / (4.0 * scale)
    sq.append(k, v)
    q = np.ldexp(np.rint(np.ldexp(rng.standard_normal((1, n_kv, g, d)).clip(-3.9, 3.9), 18)), -18)   # 20 bits below 4
    q[..., 0] = 4.0
    x = sq.values()

    def answer(q, weights):
        l = scale * np.einsum("ihgd,nhd->ihgn", q, x[:, :, 0])
        e = np.exp(l - l.max(axis=-1, keepdims=True))
        return np.einsum("ihgn,nhd->ihgd", weights(e), x[:, :, 1]) / e.sum(axis=-1, keepdims=True)

    within(answer(q, lambda e: e.astype(np.float32).astype(np.float64)), sq, q, scale)
    step = 4.0 * 2.0 ** -21
    within(answer(np.rint(q / step) * step, lambda e: e), sq, q, scale)
    for planted in (lambda: answer(q, lambda e: (e * 2.0 ** 15).astype(np.float16) / 2.0 ** 15),
                    lambda: answer(q, lambda e: np.where(e < 2.0 ** -20, 0.0, e)),
                    lambda: answer(np.rint(q / (step * 256)) * (step * 256), lambda e: e)):
        with pytest.raises(AssertionError):
            within(planted(), sq, q, scale)


def test_attention_refuses_to_write_over_its_queries_and_scales_beyond_fp32(lib):
    """A query row is read again by every part of its segment; scale log2(e) is held in fp32."""
    r = ctypes.byref(lib.tq_b8_cache(128, 8, 2, 64, 16, 0x10000, 0x20000, 0x30000, 0x40000))

    def call(q=0x1000, out=0x2000, scale=0.1):
        return lib.lib.tq_b8_attention(r, q, 0, 1, 4, scale, None, 0, None, None, 1.0, out, 0x100000, 256, None)
    assert call(out=0x1000) == lib.TQ_ERR_ARG
    for scale in (3e38, -2.5e38):
        assert call(scale=scale) == lib.TQ_ERR_ARG
    assert call() == call(scale=2e38) == lib.TQ_ERR_WORKSPACE


# ----------------------------------------------------------------------------- GPU
@pytest.mark.gpu
def test_selections_of_196_million_segments(m):
    """An accepted call whose segments' prices together pass 31 bits: 4096 sequences x 6000 query tokens x 8 kv heads, one
    block of 32 tokens each. Every row is written; those of every 64th sequence are compared."""
    import torch
    d, n_kv, n_seq, n_q, nb = 8, 8, 4096, 6000, 188
    gen = torch.Generator(device="cuda").manual_seed(5)
    pages = torch.zeros(nb, m.tq_b8_page_bytes(d, n_kv), dtype=torch.uint8, device="cuda")
    table = torch.arange(nb, dtype=torch.int32, device="cuda").repeat(n_seq, 1)
    length = torch.full((n_seq,), 32 * nb, dtype=torch.int32, device="cuda")
    open_ = torch.zeros(n_seq, n_kv, 2, 32, d, dtype=torch.bfloat16, device="cuda")
    ws = m.workspace(256)
    one = m.Cache8(d, pages, table[:1], length[:1], open_[:1])                   # the pages that all sequences share
    k, v = (torch.randn(1, 32 * nb, n_kv, d, generator=gen, device="cuda") for _ in range(2))
    m.tq_b8_append(one, k, v, ws)
    m.tq_b8_read(one, k, v, ws)                                                  # as the cache holds them
    cache = m.Cache8(d, pages, table, length, open_)
    q = torch.randn(n_seq, n_q, n_kv, d, generator=gen, device="cuda", dtype=torch.bfloat16)
    sel = torch.randint(0, nb, (n_seq, n_q, n_kv, 1), generator=gen, device="cuda", dtype=torch.int32)
    out = torch.full(q.shape, float("nan"), device="cuda")
    ws = m.workspace(m.tq_b8_workspace_bytes(cache, n_q, 1, 1, weights=False))
    m.tq_b8_attention(cache, q, d ** -0.5, out, ws, sel=sel)
    assert m.tq_get_status(ws) == m.TQ_OK
    assert not any(torch.isnan(out[s:s + 256]).any() for s in range(0, n_seq, 256))
    kb, vb = (x[0].view(nb, 32, n_kv, d).permute(2, 0, 1, 3).double() for x in (k, v))  # [n_kv, nb, 32, d]
    heads, t = torch.arange(n_kv, device="cuda"), torch.arange(32, device="cuda")
    last = 32 * nb - n_q + torch.arange(n_q, device="cuda")
    for s in list(range(0, n_seq, 64)) + [n_seq - 1]:
        b = sel[s, :, :, 0].long()                                               # [n_q, n_kv]
        kk, vv = kb[heads, b], vb[heads, b]                                      # [n_q, n_kv, 32, d]
        seen = 32 * b[..., None] + t <= last[:, None, None]
        l = torch.einsum("qhd,qhtd->qht", q[s].double(), kk) * d ** -0.5
        top = torch.where(seen, l, -torch.inf).amax(-1, keepdim=True)
        w = torch.where(seen, torch.exp(l - torch.where(top > -torch.inf, top, 0.0)), 0.0)
        w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
        want, size = torch.einsum("qht,qhtd->qhd", w, vv), torch.einsum("qht,qhtd->qhd", w, vv.abs())
        # with |q| <= 6 and sum |k| <= 48 a logit is off by 8 ** -0.5 * 2^-22 * 6 * 48 for q's fixed point and as much for
        # the fp32 factors, 5e-5 in all; weights move by twice that, their sums and the quotient by a few 2^-22: 2^-13
        assert ((out[s].double() - want).abs() <= 2.0 ** -13 * size.amax(-1, keepdim=True)).all(), s


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


def fill(p, k, v):
    """k, v [n_seq, n, n_kv, d] (numpy) into an empty Pair."""
    p.length += k.shape[1]
    m, cuda = p.m, lambda x: p.torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda()
    m.tq_b8_append(p.cache, cuda(k), cuda(v), p.ws)
    for s, sq in enumerate(p.seqs):
        sq.append(k[s], v[s])


@pytest.mark.gpu
@pytest.mark.parametrize("d,g,n,where,heavy", [
    (128, 4, 64, 0, 0.0), (128, 4, 2048, 5, 0.0), (64, 3, 64, 31, 2e-3), (64, 3, 2048, 1000, 0.0), (256, 2, 1024, 3, 0.0),
    (128, 16, 2048, 0, 2e-3), (64, 16, 64, 7, 0.0), (128, 4, 64, 0, 0.02), (80, 4, 96, 40, 0.0), (8, 2, 64, 9, 0.0),
    (128, 4, 64, 0, 1.0)])
def test_attention_sinks(m, d, g, n, where, heavy):
    """One token lies 8 to 60 nats above the rest, and its value is zero, rounds to zero, is small or as large as the others':
    what the light tokens add keeps its precision, in the heavy token's block and in others."""
    gaps = [8.0, 12.0, 16.0, 20.0, 22.0, 27.0, 35.0, 60.0]
    n_kv, scale = 2, d ** -0.5
    p = Pair(m, d, n_kv, len(gaps), n // 32 + 1, 90 + d + g + n, width=32768 // n_kv if g > 8 else None)
    k = p.rng.standard_normal((len(gaps), n, n_kv, d))
    v = p.rng.standard_normal((len(gaps), n, n_kv, d))
    k[..., 0] = 0.0
    k[:, where], v[:, where] = 0.0, v[:, where] * heavy
    k[:, where, :, 0] = (np.array(gaps) / (4.0 * scale))[:, None]
    fill(p, k, v)
    q = np.rint(64 * p.rng.standard_normal((len(gaps), 1, n_kv, g, d)).clip(-3.9, 3.9)) / 64    # exact in 22 bits
    q[..., 0] = 4.0
    qt = p.torch.from_numpy(q.astype(np.float32).reshape(len(gaps), 1, n_kv * g, d)).cuda()
    ws = p.workspace(1, g)
    out = p.torch.full(qt.shape, float("nan"), device="cuda")
    m.tq_b8_attention(p.cache, qt, scale, out, ws)
    acc = p.torch.zeros(len(gaps), n_kv, 32 * p.nb, device="cuda")
    again = p.torch.full(qt.shape, float("nan"), device="cuda")
    m.tq_b8_attention(p.cache, qt, scale, again, ws, acc_out=acc)
    assert p.torch.equal(out, again) and p.ok(ws)
    got = out.double().cpu().numpy().reshape(q.shape)
    for s, sq in enumerate(p.seqs):
        within(got[s], sq, q[s], scale)


@pytest.mark.gpu
@pytest.mark.parametrize("d,g,n_q", [(128, 4, 1), (64, 2, 3), (40, 9, 1)])
def test_attention_over_values_of_zeros(m, d, g, n_q):
    """Blocks and tokens whose values are all zeros, or zeros in the first channels alone, count in the weights."""
    n, n_kv, scale = 192, 2, d ** -0.5
    p = Pair(m, d, n_kv, 2, 7, 95 + d)
    k, v = p.rng.standard_normal((2, n, n_kv, d)), p.rng.standard_normal((2, n, n_kv, d))
    v[:, :32] = 0.0
    v[:, 32:64, 0] = 0.0
    v[:, 40:70] = 0.0
    v[:, 96:120, :, :8] = 0.0
    v[1, 128:191] = 0.0                                                          # all but the last token of two blocks
    fill(p, k, v)
    q = np.rint(64 * p.rng.standard_normal((2, n_q, n_kv, g, d))) / 64
    qt = p.torch.from_numpy(q.astype(np.float32).reshape(2, n_q, n_kv * g, d)).cuda()
    ws = p.workspace(n_q, g)
    out = p.torch.full(qt.shape, float("nan"), device="cuda")
    m.tq_b8_attention(p.cache, qt, scale, out, ws)
    got = out.double().cpu().numpy().reshape(q.shape)
    for s, sq in enumerate(p.seqs):
        within(got[s], sq, q[s], scale)
    assert p.ok(ws)


@pytest.mark.gpu
@pytest.mark.parametrize("n,selected", [(60, False), (64, False), (47, True), (33, True)])
def test_accumulated_weights_of_large_logits(m, n, selected):
    """A row's accumulated weights are those of its value sum and add up to 1, however large the logits are. Keys and
    queries are whole numbers, keys with an element of 127 (scale 1) and each there several times, values the unit vectors:
    equal logits are equal in every path, the output is the weights themselves."""
    import torch
    d, n_kv, g = 64, 2, 3
    for scale in (1e-5, 1e-4, 1e-3, 0.01, 0.1, 1.0, 10.0, 1e2, 1e4, -1e-3, -1.0, -1e4):
        p = Pair(m, d, n_kv, 1, 3, 110)
        kinds = np.rint(60 * p.rng.standard_normal((8, n_kv, d))).clip(-126, 126)
        kinds[..., 0] = 127
        k, v = kinds[np.arange(n) % 8][None], np.zeros((1, n, n_kv, d))
        v[0, np.arange(n), :, np.arange(n)] = 1.0
        fill(p, k, v)
        q = np.rint(50 * p.rng.standard_normal((1, 1, n_kv, g, d)))
        qt = torch.from_numpy(q.astype(np.float32).reshape(1, 1, n_kv * g, d)).cuda()
        want, weight, _, _ = ref.attention(p.seqs[0], q[0], scale)
        sel = torch.tensor([0, 1, -1], dtype=torch.int32, device="cuda").expand(1, 1, n_kv, 3).contiguous() if selected else None
        ws = p.workspace(1, g, 3 if selected else 0)
        out, acc = torch.zeros(qt.shape, device="cuda"), torch.zeros(1, n_kv, 32 * p.nb, device="cuda")
        m.tq_b8_attention(p.cache, qt, scale, out, ws, sel=sel, acc_out=acc)
        assert p.ok(ws)
        w = out.double().cpu().numpy().reshape(n_kv, g, d)[..., :n]                   # a weight per token
        a = acc[0].double().cpu().numpy()[:, :n]
        # two ways to the same weights: pieces of 22 bits (off by 2^-34 at least) and fp32 sums against fp32 sums
        assert (np.abs(a - w.sum(axis=1)) <= 2.0 ** -18 * a + g * 2.0 ** -33).all(), scale
        assert (np.abs(a.sum(axis=1) - g) <= g * 2.0 ** -18).all(), (scale, a.sum(axis=1))
        # against 64 bits: a logit is off by 2^-22 of itself (ties stay ties); where rows are ties of whole numbers apart, by nothing
        logits = np.abs(scale) * np.abs(np.einsum("hgd,nhd->hgn", q[0, 0], p.seqs[0].values()[:, :, 0])).max(axis=(1, 2))
        rel = np.expm1(2 * np.minimum(logits * 2.0 ** -22, 1.0)) + 2.0 ** -18
        if (logits * 2.0 ** -22 < 2.0 ** -6).all():
            assert (np.abs(a - weight) <= rel[:, None] * weight + 2.0 ** -40).all(), scale


@pytest.mark.gpu
@pytest.mark.parametrize("n_q,g,selected", [(1, 5, False), (3, 2, False), (1, 4, True)])
def test_accumulated_weights_at_any_alignment(m, n_q, g, selected):
    """acc_in and acc_out need be aligned to an element alone: the same bits as from 16-byte aligned ones."""
    import torch
    d, n_kv, lens = 64, 2, [0, 1, 30, 97, 160]
    p = Pair(m, d, n_kv, len(lens), 6, 120)
    p.append(lens)
    q, _ = p.queries(n_q, g, "bf16")
    sel = torch.tensor([0, 2, 3, -1], dtype=torch.int32, device="cuda").expand(len(lens), n_q, n_kv, 4).contiguous() if selected else None
    ws = p.workspace(n_q, g, 4 if selected else 0)
    shape, got = (len(lens), n_kv, 32 * p.nb), []
    size = shape[0] * shape[1] * shape[2]
    base = torch.rand(size, device="cuda")
    for at_in, at_out in ((0, 0), (1, 0), (0, 3), (2, 1)):
        room_in, room_out = torch.zeros(size + 4, device="cuda"), torch.full((size + 4,), 7.0, device="cuda")
        a, b = room_in[at_in:at_in + size].view(shape), room_out[at_out:at_out + size].view(shape)
        a.copy_(base.view(shape))
        m.tq_b8_attention(p.cache, q, 0.1, torch.zeros(q.shape, device="cuda"), ws, sel=sel, acc_in=a, acc_out=b, decay=0.5)
        got.append(b.clone())
        assert (room_out[:at_out] == 7.0).all() and (room_out[at_out + size:] == 7.0).all()
        for s, n in enumerate(lens):
            assert (b[s, :, n:] == 7.0).all() and (b[s, :, :n] != 7.0).all()
    assert all(torch.equal(got[0], x) for x in got[1:]) and p.ok(ws)


@pytest.mark.gpu
@pytest.mark.parametrize("d,g,dtype", [(128, 4, "f32"), (128, 8, "bf16"), (64, 3, "f32"), (256, 2, "bf16"), (40, 5, "f32")])
def test_attention_queries_of_a_wide_range(m, d, g, dtype):
    """Elements of a row from 2^-24 to 1 of the largest, which meets keys of zero in half of the rows: a logit is off by at
    most what q's fixed point loses, scale 2^-22 max |q| sum |k|. Rows whose elements fixed point holds are not off at all."""
    import torch
    n_kv, n, scale = 2, 160, d ** -0.5
    p = Pair(m, d, n_kv, 2, 6, 130 + d + g)
    k, v = p.rng.standard_normal((2, n, n_kv, d)), p.rng.standard_normal((2, n, n_kv, d))
    k[0, ..., 0] = 0.0
    fill(p, k, v)
    q = np.exp2(p.rng.uniform(-20, 4, (2, 1, n_kv, g, d))) * p.rng.choice([-1.0, 1.0], (2, 1, n_kv, g, d))
    q[..., 0] = 16 * (1 + 2.0 ** -7)
    q[:, :, :, 0] = np.ldexp(np.rint(q[:, :, :, 0] * 2 ** 16), -16)              # 21 bits below 16: held
    qt = torch.from_numpy(q.astype(np.float32).reshape(2, 1, n_kv * g, d)).cuda()
    qt = qt if dtype == "f32" else qt.to(torch.bfloat16)
    q = qt.double().cpu().numpy().reshape(q.shape)
    ws = p.workspace(1, g)
    out = torch.zeros(qt.shape, device="cuda")
    m.tq_b8_attention(p.cache, qt, scale, out, ws)
    got = out.double().cpu().numpy().reshape(q.shape)
    for s, sq in enumerate(p.seqs):
        reach = np.abs(sq.values()[:, :, 0]).sum(axis=2).max(axis=0)             # [n_kv]
        lost = scale * 2.0 ** -22 * np.abs(q[s]).max(axis=-1) * reach[None, :, None]
        within(got[s], sq, q[s], scale, lost=lost)
        within(got[s][:, :, :1], sq, q[s][:, :, :1], scale)
    assert p.ok(ws)


@pytest.mark.gpu
@pytest.mark.parametrize("d,g,n,where", [(128, 4, 70, 66), (64, 3, 327, 320), (128, 16, 70, 69), (256, 2, 60, 33), (80, 4, 85, 84)])
def test_attention_sinks_in_the_open_block(m, d, g, n, where):
    """The same where the heavy token without a value has not left the open block yet. A segment's open block comes last
    and its weights keep 24 bits however light they are, so the full blocks' tokens keep their precision beside it."""
    gaps = [8.0, 16.0, 20.0, 24.0, 35.0, 50.0]
    n_kv, scale = 1, d ** -0.5
    p = Pair(m, d, n_kv, len(gaps), n // 32 + 1, 140 + d + g, width=32768 // n_kv if g > 8 else None)
    k = p.rng.standard_normal((len(gaps), n, n_kv, d))
    v = p.rng.standard_normal((len(gaps), n, n_kv, d))
    k[..., 0] = 0.0
    k[:, n // 32 * 32:], v[:, n // 32 * 32:] = 0.0, 0.0                          # open tokens: logits of 0, no values
    k[:, where, :, 0] = (np.array(gaps) / (4.0 * scale))[:, None]
    fill(p, k, v)
    q = np.rint(64 * p.rng.standard_normal((len(gaps), 1, n_kv, g, d)).clip(-3.9, 3.9)) / 64
    q[..., 0] = 4.0
    qt = p.torch.from_numpy(q.astype(np.float32).reshape(len(gaps), 1, n_kv * g, d)).cuda()
    ws = p.workspace(1, g)
    out = p.torch.full(qt.shape, float("nan"), device="cuda")
    acc = p.torch.zeros(len(gaps), n_kv, 32 * p.nb, device="cuda")
    m.tq_b8_attention(p.cache, qt, scale, out, ws, acc_out=acc)
    got = out.double().cpu().numpy().reshape(q.shape)
    for s, sq in enumerate(p.seqs):
        within(got[s], sq, q[s], scale)
    assert ((acc.sum(dim=-1) - g).abs() <= g * 2.0 ** -18).all() and p.ok(ws)


@pytest.mark.gpu
@pytest.mark.parametrize("log2_logit", [60000.0, 70000.0, 1e6, 2.0 ** 29, 1.5 * 2.0 ** 30, 1.5 * 2.0 ** 33])
def test_weights_of_a_sink_with_a_huge_logit(m, log2_logit):
    """A token without a value takes all of the attention, by a logit whose neighbours in fp32 lie apart: its weight is 1 a
    row, every other one 0, and the output 0."""
    import torch
    d, n_kv, g, n = 64, 2, 3, 96
    p = Pair(m, d, n_kv, 1, 4, 150)
    k, v = p.rng.standard_normal((1, n, n_kv, d)), p.rng.standard_normal((1, n, n_kv, d))
    k[..., 0] = 0.0
    k[:, 40], v[:, 40] = 0.0, 0.0
    k[:, 40, :, 0] = 64.0
    fill(p, k, v)
    q = torch.zeros(1, 1, n_kv * g, d, device="cuda")
    q[..., 0], q[..., 1] = 4.0, 2.0 ** -18
    scale = log2_logit / 256 / 1.4426950408889634
    ws = p.workspace(1, g)
    out, acc = torch.full(q.shape, 5.0, device="cuda"), torch.zeros(1, n_kv, 32 * p.nb, device="cuda")
    m.tq_b8_attention(p.cache, q, scale, out, ws, acc_out=acc)
    want = torch.zeros_like(acc)
    want[:, :, 40] = g
    assert ((acc - want).abs() <= g * 2.0 ** -18).all(), acc[0, :, 32:48]
    assert torch.isfinite(out).all() and (out.abs() <= 2.0 ** -30).all() and p.ok(ws)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.1, 1e5, -1e9])
def test_a_seen_key_that_is_not_a_number(m, scale):
    """A NaN in the open block's keys is every answer's that sees it, and no other's, however large the logits are."""
    import torch
    d, n_kv, g, n = 64, 2, 3, 70
    p = Pair(m, d, n_kv, 2, 3, 160)
    k, v = p.rng.standard_normal((2, n, n_kv, d)), p.rng.standard_normal((2, n, n_kv, d))
    k[0, 67, 0, 9] = np.nan
    fill(p, k, v)
    q, _ = p.queries(1, g, "f32")
    ws = p.workspace(1, g)
    out, acc = torch.zeros(q.shape, device="cuda"), torch.zeros(2, n_kv, 32 * p.nb, device="cuda")
    m.tq_b8_attention(p.cache, q, scale, out, ws, acc_out=acc)
    assert torch.isnan(out[0, :, :g]).all() and torch.isnan(acc[0, 0, :n]).all()
    assert torch.isfinite(out[0, :, g:]).all() and torch.isfinite(out[1]).all() and torch.isfinite(acc[0, 1]).all()
    assert ((acc[1].sum(dim=-1) - g).abs() <= g * 2.0 ** -18).all() and p.ok(ws)
