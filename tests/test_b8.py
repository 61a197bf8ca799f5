"""Paged 8-bit cache: the reference's own checks and the library's refusals (CPU), then parity of
append, read, attention, selection and eviction with the plain 64-bit reference (GPU)."""
import ctypes
import math

import numpy as np
import pytest

import b8_reference as ref


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    import kv_cache_vector_03_b200 as m
    return m


# ----------------------------------------------------------------------------- CPU
def test_reference_page_round_trip():
    rng = np.random.default_rng(1)
    for d, n_kv in ((8, 1), (64, 3), (80, 2), (200, 1)):
        s = ref.Seq(n_kv, d)
        s.append(rng.standard_normal((70, n_kv, d)), rng.standard_normal((70, n_kv, d)))
        for j, (codes, scales) in enumerate(s.blocks):
            c, sc, lo, hi = ref.unpack(s.page(j), d, n_kv)
            assert np.array_equal(c, codes) and np.array_equal(sc, scales)
            assert np.array_equal(lo, codes[:, 0].min(axis=1)) and np.array_equal(hi, codes[:, 0].max(axis=1))
            assert np.abs(codes).max(axis=(2, 3)).min() == 127       # the largest value has code 127


def test_reference_error_bound_and_repeatability():
    """A code is off by at most half a step; the splitting of a prompt over calls changes nothing;
    moving a whole block changes nothing."""
    rng = np.random.default_rng(2)
    k, v = rng.standard_normal((96, 2, 40)) * 3, rng.standard_normal((96, 2, 40))
    one, many = ref.Seq(2, 40), ref.Seq(2, 40)
    one.append(k, v)
    for a, b in ((0, 1), (1, 33), (33, 34), (34, 96)):
        many.append(k[a:b], v[a:b])
    for (c, s), (c2, s2) in zip(one.blocks, many.blocks):
        assert np.array_equal(c, c2) and np.array_equal(s, s2)
    x = np.stack([ref.to_bf16(k), ref.to_bf16(v)], axis=2)
    step = np.repeat(np.stack([s for _, s in one.blocks]), 32, axis=0)[..., None].astype(np.float64)
    # inv and the scale are each rounded twice, by 2^-24 of themselves: values up to 127 steps move by 127 * 2^-22
    assert np.all(np.abs(one.values() - x) <= step * (0.5 + 127 * 2 ** -22))
    acc = np.zeros((2, 96), np.float32)
    new, kept, _ = ref.evict(one, acc, 2, 0, 0)                       # all tie: the first 64 stay
    assert np.array_equal(kept, np.tile(np.arange(64), (2, 1)))
    for j in range(2):
        assert np.array_equal(new.page(j), one.page(j))


def test_page_sizes(lib):
    for d, n_kv in ((8, 1), (64, 8), (80, 5), (128, 8), (136, 3), (256, 1)):
        assert lib.tq_b8_page_bytes(d, n_kv) == ref.page_bytes(d, n_kv)
    for d, n_kv in ((0, 1), (12, 1), (264, 1), (128, 0), (128, 1025)):
        assert lib.tq_b8_page_bytes(d, n_kv) == 0


def host_cache(lib, d=128, n_kv=8, n_seq=2, n_pages=64, max_blocks=16, pages=0x10000, table=0x20000, length=0x30000,
               open_=0x40000):
    return lib.tq_b8_cache(d, n_kv, n_seq, n_pages, max_blocks, pages, table, length, open_)


BAD_CACHES = [dict(d=12), dict(d=264), dict(d=0), dict(n_kv=0), dict(n_kv=1025), dict(n_seq=-1), dict(n_seq=65536),
              dict(n_pages=-1), dict(n_pages=1 << 31), dict(max_blocks=0), dict(max_blocks=(1 << 23) + 1),
              dict(pages=None), dict(pages=0x10040), dict(table=None), dict(table=0x20002), dict(length=None),
              dict(open_=None), dict(open_=0x40008)]


def calls(lib, c):
    """Every entry point with arguments that are fine but for the cache."""
    r, ws, n = ctypes.byref(c), 0x100000, 1 << 40
    return [lib.lib.tq_b8_append(r, 0x1000, 0x2000, 1, 3, 4096, 1024, None, ws, n, None),
            lib.lib.tq_b8_read(r, 5, 0x1000, 0x2000, 1, ws, n, None),
            lib.lib.tq_b8_attention(r, 0x1000, 1, 1, 4, 0.1, None, 0, None, None, 1.0, 0x2000, ws, n, None),
            lib.lib.tq_b8_select(r, 0x1000, 1, 1, 4, 1, 1, 4, 0x2000, ws, n, None),
            lib.lib.tq_b8_evict(r, 0x1000, 4, 1, 1, 0x2000, 0x3000, 0x4000, 0x5000, ws, n, None)]


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_bad_caches_are_refused(lib, bad):
    for st in calls(lib, host_cache(lib, **bad)):
        assert st in (lib.TQ_ERR_ARG, lib.TQ_ERR_UNSUPPORTED)
    for st in (lib.lib.tq_b8_append(None, 0x1000, 0x2000, 1, 3, 4096, 1024, None, 0x100000, 1 << 40, None),
               lib.lib.tq_b8_read(None, 5, 0x1000, 0x2000, 1, 0x100000, 1 << 40, None)):
        assert st == lib.TQ_ERR_ARG


def test_empty_work_is_a_no_op(lib):
    assert calls(lib, host_cache(lib, n_seq=0)) == [lib.TQ_OK] * 5
    r = ctypes.byref(host_cache(lib))
    assert lib.lib.tq_b8_append(r, 0x1000, 0x2000, 1, 0, 4096, 1024, None, 0x100000, 1 << 40, None) == lib.TQ_OK
    assert lib.lib.tq_b8_read(r, 0, 0x1000, 0x2000, 1, 0x100000, 1 << 40, None) == lib.TQ_OK


def test_append_and_read_refusals(lib):
    r = ctypes.byref(host_cache(lib))

    def append(k=0x1000, v=0x2000, dt=1, n=3, ss=4096, ts=1024, add=None, ws=0x100000, wb=256):
        return lib.lib.tq_b8_append(r, k, v, dt, n, ss, ts, add, ws, wb, None)
    for bad in (dict(k=None), dict(v=None), dict(k=0x1008), dict(v=0x2004), dict(dt=2), dict(n=-1), dict(ss=-8),
                dict(ss=4), dict(ts=1020), dict(add=0x3002), dict(ws=None), dict(ws=0x100010)):
        assert append(**bad) == lib.TQ_ERR_ARG, bad
    assert append(wb=255) == lib.TQ_ERR_WORKSPACE
    assert append(n=(1 << 28) + 1) == lib.TQ_ERR_UNSUPPORTED

    def read(n=5, k=0x1000, v=0x2000, dt=1, ws=0x100000, wb=256):
        return lib.lib.tq_b8_read(r, n, k, v, dt, ws, wb, None)
    for bad in (dict(n=-1), dict(k=None), dict(k=0x1008), dict(v=None), dict(dt=7), dict(ws=None)):
        assert read(**bad) == lib.TQ_ERR_ARG, bad
    assert read(wb=0) == lib.TQ_ERR_WORKSPACE
    assert read(n=(1 << 28) + 1) == lib.TQ_ERR_UNSUPPORTED


def test_attention_refusals(lib):
    c = host_cache(lib)
    r = ctypes.byref(c)

    def call(q=0x1000, dt=1, n_q=1, g=4, scale=0.1, sel=None, n_sel=0, ai=None, ao=None, decay=1.0, out=0x2000,
             ws=0x100000, wb=1 << 40):
        return lib.lib.tq_b8_attention(r, q, dt, n_q, g, scale, sel, n_sel, ai, ao, decay, out, ws, wb, None)
    for bad in (dict(q=None), dict(q=0x1001), dict(dt=3), dict(n_q=0), dict(g=0), dict(scale=math.inf),
                dict(scale=math.nan), dict(sel=0x3000), dict(n_sel=4), dict(sel=0x3002, n_sel=4), dict(n_sel=-1),
                dict(sel=0x3000, n_sel=(1 << 23) + 1), dict(ai=0x4000), dict(ao=0x4001), dict(decay=math.inf), dict(out=None),
                dict(out=0x2008), dict(ws=None), dict(ws=0x100080)):
        assert call(**bad) == lib.TQ_ERR_ARG, bad
    assert call(n_q=128, g=129) == lib.TQ_ERR_UNSUPPORTED
    assert call(sel=0x3000, n_sel=4, ao=0x5000, n_q=2) == lib.TQ_ERR_UNSUPPORTED
    for n_q, n_sel, weights in ((1, 0, 0), (1, 0, 1), (3, 0, 1), (1, 4, 1)):
        need = lib.lib.tq_b8_workspace_bytes(r, n_q, 4, n_sel, weights)
        assert need >= 256 and need % 256 == 0
        assert call(n_q=n_q, sel=0x3000 if n_sel else None, n_sel=n_sel, ao=0x5000 if weights else None,
                    wb=need - 1) == lib.TQ_ERR_WORKSPACE
    assert lib.lib.tq_b8_workspace_bytes(ctypes.byref(host_cache(lib, d=12)), 1, 4, 0, 0) == 0
    assert lib.lib.tq_b8_workspace_bytes(r, 128, 129, 0, 0) == 0
    assert lib.lib.tq_b8_workspace_bytes(r, 0, 0, 0, 0) >= 256


def test_select_and_evict_refusals(lib):
    c = host_cache(lib)
    r = ctypes.byref(c)

    def select(q=0x1000, dt=1, n_q=1, g=4, nf=1, nl=1, n_sel=4, sel=0x2000, ws=0x100000, wb=1 << 40):
        return lib.lib.tq_b8_select(r, q, dt, n_q, g, nf, nl, n_sel, sel, ws, wb, None)
    for bad in (dict(q=None), dict(dt=9), dict(n_q=0), dict(g=-1), dict(nf=-1), dict(nl=-1), dict(nf=3, nl=2),
                dict(n_sel=0), dict(n_sel=(1 << 23) + 1), dict(nf=2 ** 31 - 1, nl=2 ** 31 - 1), dict(sel=None), dict(ws=None)):
        assert select(**bad) == lib.TQ_ERR_ARG, bad
    assert select(wb=lib.lib.tq_b8_workspace_bytes(r, 1, 4, 4, 0) - 1) == lib.TQ_ERR_WORKSPACE

    def evict(acc=0x1000, keep=4, nf=4, nl=32, dst=0x2000, kept=0x3000, lo=0x4000, ao=0x5000, ws=0x100000, wb=256):
        return lib.lib.tq_b8_evict(r, acc, keep, nf, nl, dst, kept, lo, ao, ws, wb, None)
    for bad in (dict(acc=None), dict(keep=0), dict(keep=(1 << 23) + 1), dict(nf=-1), dict(nl=-1), dict(nf=100, nl=29),
                dict(nf=2 ** 62, nl=2 ** 62), dict(dst=None), dict(kept=None), dict(lo=None), dict(ao=None),
                dict(lo=0x30000), dict(ao=0x1000), dict(kept=0x3001), dict(ws=None)):
        assert evict(**bad) == lib.TQ_ERR_ARG, bad
    assert evict(wb=8) == lib.TQ_ERR_WORKSPACE


def test_binding_refuses_wrong_tensors(lib):
    """The binding's checks run before anything touches a GPU."""
    import torch
    d, n_kv, n_seq, nb = 64, 2, 3, 4
    pages = torch.zeros(12, lib.tq_b8_page_bytes(d, n_kv), dtype=torch.uint8)
    table = torch.zeros(n_seq, nb, dtype=torch.int32)
    length = torch.zeros(n_seq, dtype=torch.int32)
    open_ = torch.zeros(n_seq, n_kv, 2, 32, d, dtype=torch.bfloat16)
    c = lib.Cache8(d, pages, table, length, open_)
    for bad in ((pages[:, 1:], table, length, open_), (pages, table.long(), length, open_),
                (pages, table[:2], length, open_), (pages, table.t().contiguous().t(), length, open_),
                (pages, table, length[:2], open_), (pages, table, length, open_[..., :32]),
                (pages, table, length, open_.float())):
        with pytest.raises((ValueError, TypeError)):
            lib.Cache8(d, *bad)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    q, out = torch.zeros(n_seq, 1, 4, d), torch.zeros(n_seq, 1, 4, d)
    for kw in (dict(q=q[:2]), dict(q=q[..., :32]), dict(q=torch.zeros(n_seq, 1, 3, d)), dict(q=q.half()),
               dict(out=out.bfloat16()), dict(out=out[:, :, :2]), dict(sel=torch.zeros(n_seq, 1, 2, 3)),
               dict(sel=torch.zeros(n_seq, 2, 2, 3, dtype=torch.int32)), dict(acc_out=torch.zeros(n_seq, n_kv, 5))):
        a = dict(q=q, out=out)
        a.update(kw)
        with pytest.raises((ValueError, TypeError)):
            lib.tq_b8_attention(c, a.pop("q"), 1.0, a.pop("out"), ws, **a)
    k = torch.zeros(n_seq, 5, n_kv, d)
    for a, b in ((k[:2], k[:2]), (k, k[:, :4]), (k, k.bfloat16()), (k.transpose(1, 2).contiguous().transpose(1, 2), k),
                 (k[0], k[0]), (k.expand(n_seq, 5, n_kv, d)[:, ::2], k[:, :3])):
        with pytest.raises((ValueError, TypeError)):
            lib.tq_b8_append(c, a, b, ws)


# ----------------------------------------------------------------------------- GPU
class Pair:
    """The same cache in the library and in the reference."""

    def __init__(self, m, d, n_kv, n_seq, max_blocks, seed, spare=0, width=None):
        import torch
        self.m, self.torch, self.rng = m, torch, np.random.default_rng(seed)
        self.d, self.n_kv, self.n_seq, self.nb = d, n_kv, n_seq, max_blocks
        n_pages = n_seq * max_blocks + spare
        self.names = self.rng.permutation(n_pages).astype(np.int32)
        # pages nobody has written and the open block hold what would show: NaN scales, NaN tokens
        self.pages = torch.full((n_pages, m.tq_b8_page_bytes(d, n_kv)), 255, dtype=torch.uint8, device="cuda")
        table = self.names[:n_seq * max_blocks].reshape(n_seq, max_blocks)
        if width is not None:                        # a longer table, whose further entries name no page
            self.nb = width
            table = np.concatenate([table, np.full((n_seq, width - max_blocks), -1, np.int32)], axis=1)
        self.table = torch.from_numpy(table.copy()).cuda()
        self.length = torch.zeros(n_seq, dtype=torch.int32, device="cuda")
        self.open_ = torch.full((n_seq, n_kv, 2, 32, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.cache = m.Cache8(d, self.pages, self.table, self.length, self.open_)
        self.seqs = [ref.Seq(n_kv, d) for _ in range(n_seq)]
        self.ws = m.workspace(256)

    def tokens(self, n, outliers=True):
        k = self.rng.standard_normal((n, self.n_kv, self.d)).astype(np.float32)
        if outliers and self.d >= 16:
            k[..., 3] *= 20
        return k, self.rng.standard_normal((n, self.n_kv, self.d)).astype(np.float32)

    def append(self, counts, dtype="f32", n_new=None, garbage=float("nan")):
        torch = self.torch
        n_new = max(counts) if n_new is None else n_new
        k = np.full((self.n_seq, n_new, self.n_kv, self.d), garbage, np.float32)
        v = k.copy()
        for s, n in enumerate(counts):
            k[s, :n], v[s, :n] = self.tokens(n)
            self.seqs[s].append(k[s, :n], v[s, :n])
        self.length += torch.tensor(counts, dtype=torch.int32, device="cuda")
        kt, vt = (torch.from_numpy(x).cuda().to(torch.float32 if dtype == "f32" else torch.bfloat16) for x in (k, v))
        self.m.tq_b8_append(self.cache, kt, vt, self.ws, add=torch.tensor(counts, dtype=torch.int32, device="cuda"))

    def check_bytes(self):
        pages, table, open_ = self.pages.cpu().numpy(), self.table.cpu().numpy(), self.open_.float().cpu().numpy()
        D = ref.padded(self.d)
        used = set()
        for s, q in enumerate(self.seqs):
            for j in range(len(q.blocks)):
                used.add(int(table[s, j]))
                got, want = pages[table[s, j]].copy(), q.page(j)
                for h in range(self.n_kv):                      # unused bytes of an entry
                    got[h * (32 + 2 * D) + 8:h * (32 + 2 * D) + 32] = 0
                    for o in (32, 32 + D):
                        got[h * (32 + 2 * D) + o + self.d:h * (32 + 2 * D) + o + D] = 0
                end = self.n_kv * (32 + 2 * D)
                got[end:ref.header_bytes(self.d, self.n_kv)] = 0
                assert np.array_equal(got, want), f"sequence {s} block {j}"
            r = len(q.open)
            assert np.array_equal(open_[s, :, :, :r], q.open.transpose(1, 2, 0, 3), equal_nan=True)
        for name in set(range(len(pages))) - used:
            assert (pages[name] == 255).all(), f"page {name} was written"

    def queries(self, n_q, g, dtype):
        torch = self.torch
        q = self.rng.standard_normal((self.n_seq, n_q, self.n_kv * g, self.d)).astype(np.float32)
        t = torch.from_numpy(q).cuda().to(torch.float32 if dtype == "f32" else torch.bfloat16)
        return t, t.double().cpu().numpy().reshape(self.n_seq, n_q, self.n_kv, g, self.d)

    def workspace(self, n_q, g, n_sel=0):
        return self.m.workspace(max(self.m.tq_b8_workspace_bytes(self.cache, n_q, g, n) for n in {0, n_sel}))

    def ok(self, ws=None):
        return self.m.tq_get_status(self.ws if ws is None else ws) == self.m.TQ_OK


def close(got, want, size, reach, d):
    """|got - want| per row against the fp32 bound. A logit is a sum of at most 2 d products (two
    pieces of q), each addition of which is off by at most 2^-23 of the sum of magnitudes `reach`, plus
    2^-22 of it for q's own pieces and 2^-22 for the scale factors: dl <= reach (2 d + 4) 2^-23.
    Weights then move by a factor exp(+-2 dl); their two pieces, the exponential and the fp32 sums
    over up to 2^12 partial terms add 2^-12 (each addition 2^-24 of the running sum): all of it
    relative to sum_t w_t |v_t|."""
    dl = reach * (2 * d + 4) * 2.0 ** -23
    bound = (np.expm1(2 * dl) + 2.0 ** -12) * size
    err = np.abs(got - want).max(axis=-1)
    assert np.isfinite(got).all()
    assert np.all(err <= bound + 1e-30), f"worst {np.max(err / np.maximum(bound, 1e-30))} of the bound"


@pytest.fixture(scope="module")
def m():
    import kv_cache_vector_03_b200 as mod
    return mod


@pytest.mark.gpu
@pytest.mark.parametrize("d,n_kv,dtype", [(128, 8, "bf16"), (128, 3, "f32"), (64, 2, "bf16"), (40, 1, "f32"),
                                          (8, 5, "bf16"), (200, 2, "f32"), (256, 1, "bf16")])
def test_append_bytes(m, d, n_kv, dtype):
    """Tokens in pieces of every kind give the reference's bytes: none, one, a block's end in the
    middle of a piece, whole blocks, several blocks."""
    p = Pair(m, d, n_kv, 4, 12, 10 + d)
    for counts in ([1, 0, 31, 32], [1, 33, 1, 0], [30, 1, 0, 64], [33, 0, 95, 1], [0, 127, 1, 2], [1, 1, 1, 1]):
        p.append(counts, dtype, n_new=max(counts) + 3)
    p.append([2, 0, 1, 0], dtype, n_new=32 * p.nb + 50)       # more rows than any sequence holds, few of them tokens
    assert p.ok()
    p.check_bytes()


@pytest.mark.gpu
def test_append_strided_views(m):
    """k and v as views into one fused projection, without counts."""
    import torch
    d, n_kv, n_seq, n = 96, 3, 2, 45
    p = Pair(m, d, n_kv, n_seq, 4, 5)
    fused = torch.randn(n_seq, n + 2, 4 * n_kv * d, device="cuda").to(torch.bfloat16)
    k = fused[:, 1:n + 1, n_kv * d:2 * n_kv * d].unflatten(2, (n_kv, d))
    v = fused[:, 1:n + 1, 3 * n_kv * d:].unflatten(2, (n_kv, d))
    p.length += n
    m.tq_b8_append(p.cache, k, v, p.ws)
    for s in range(n_seq):
        p.seqs[s].append(k[s].float().cpu().numpy(), v[s].float().cpu().numpy())
    assert p.ok()
    p.check_bytes()


@pytest.mark.gpu
def test_append_values_that_are_not_finite_or_tiny(m):
    """They count as 0 and are reported when their block is quantized; an all-zero and a tiny block are zeros."""
    import torch
    d, n_kv = 64, 2
    p = Pair(m, d, n_kv, 3, 4, 6)
    k, v = (np.random.default_rng(7).standard_normal((3, 32, n_kv, d)).astype(np.float32) for _ in range(2))
    k[0, 3, 0, 5], k[0, 4, 1, 6], v[0, 31, 1, 63], v[0, 0, 0, 0] = np.inf, np.nan, -np.inf, 3.4e38
    k[1], v[1] = 0.0, 1e-33
    for part in ((0, 20), (20, 32)):
        p.length += part[1] - part[0]
        m.tq_b8_append(p.cache, torch.from_numpy(k[:, part[0]:part[1]].copy()).cuda(),
                       torch.from_numpy(v[:, part[0]:part[1]].copy()).cuda(), p.ws)
        assert m.tq_get_status(p.ws) == (m.TQ_OK if part[0] == 0 else m.TQ_ERR_RANGE)
    for s in range(3):
        p.seqs[s].append(k[s], v[s])
    p.check_bytes()


@pytest.mark.gpu
def test_append_out_of_range(m):
    """Lengths, counts and pages that cannot be are reported, and nothing is written for them."""
    import torch
    d, n_kv = 64, 1
    k = torch.randn(1, 40, n_kv, d, device="cuda")
    for length, add, page in ((-1, 1, None), (129, 1, None), (2 ** 31 - 1, 40, None), (10, 11, None), (10, -1, None),
                              (50, 41, None), (40, 40, 4), (40, 40, -1), (40, 40, 2 ** 31 - 1)):
        p = Pair(m, d, n_kv, 1, 4, 8)
        if page is not None:
            p.table[0, 0] = page
        p.length.fill_(length)
        m.tq_b8_append(p.cache, k, k, p.ws, add=torch.tensor([add], dtype=torch.int32, device="cuda"))
        assert m.tq_get_status(p.ws) == m.TQ_ERR_RANGE, (length, add, page)
        assert (p.pages == 255).all()
        if page is None:
            assert torch.isnan(p.open_).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d,n_kv,dtype", [(128, 8, "bf16"), (80, 3, "f32"), (256, 2, "bf16"), (8, 1, "f32")])
def test_read(m, d, n_kv, dtype):
    import torch
    p = Pair(m, d, n_kv, 4, 5, 20 + d)
    p.append([0, 31, 64, 133])
    td = torch.float32 if dtype == "f32" else torch.bfloat16
    for n_tok in (1, 33, 160, 333):
        k, v = (torch.full((4, n_tok, n_kv, d), 768.0, dtype=td, device="cuda") for _ in range(2))
        m.tq_b8_read(p.cache, k, v, p.ws)
        for s, q in enumerate(p.seqs):
            n = min(len(q), n_tok)
            x = q.values()[len(q) - n:]
            for side, got in enumerate((k, v)):
                g = got[s].double().cpu().numpy()
                assert (g[:n_tok - n] == 768.0).all()
                half = 2.0 ** -24 if dtype == "f32" else 2.0 ** -8 + 2.0 ** -24     # code * scale is rounded to fp32 first
                assert np.all(np.abs(g[n_tok - n:] - x[:, :, side]) <= half * np.abs(x[:, :, side]) + 1e-40)
    assert p.ok()


CASES = [  # d, n_kv, g, n_q, lengths, dtype
    (128, 8, 4, 1, [500], "bf16"), (128, 2, 1, 1, [1, 0, 31, 32, 33], "bf16"), (128, 2, 8, 1, [257, 64, 1000], "f32"),
    (64, 3, 3, 2, [0, 1, 2, 33, 96], "f32"), (64, 1, 7, 5, [3, 64, 66, 290], "bf16"), (40, 2, 5, 3, [70, 5], "bf16"),
    (8, 1, 2, 1, [40], "f32"), (200, 2, 4, 1, [100, 45], "bf16"), (256, 1, 8, 2, [129, 31], "f32"),
    (64, 4, 6, 4, [160 + (977 + 40503 * s) % 1140 for s in range(24)], "f32"),
    (128, 1, 16, 3, [320], "bf16"), (96, 1, 33, 1, [77], "f32"), (128, 1, 2, 40, [37, 64, 200], "bf16")]


@pytest.mark.gpu
@pytest.mark.parametrize("d,n_kv,g,n_q,lens,dtype", CASES)
def test_attention(m, d, n_kv, g, n_q, lens, dtype, width=None):
    import torch
    p = Pair(m, d, n_kv, len(lens), -(-max(lens) // 32) + 1, 30 + d + g, width=width)
    p.append(lens)
    q, q64 = p.queries(n_q, g, dtype)
    ws = p.workspace(n_q, g)
    outs = []
    for weights in (False, True):
        out = torch.full(q.shape, float("nan"), device="cuda")
        if not weights:
            m.tq_b8_attention(p.cache, q, d ** -0.5, out, ws)
        else:
            acc = torch.rand(len(lens), n_kv, 32 * p.nb, device="cuda")
            acc_out = torch.full_like(acc, 99.0)
            m.tq_b8_attention(p.cache, q, d ** -0.5, out, ws, acc_in=acc, acc_out=acc_out, decay=0.75)
            plain = torch.full_like(acc, 99.0)
            out2 = torch.empty_like(out)
            m.tq_b8_attention(p.cache, q, d ** -0.5, out2, ws, acc_out=plain)
            assert torch.equal(out, out2)
        outs.append(out)
    assert p.ok(ws)
    assert torch.equal(outs[0], outs[1])
    got = outs[0].double().cpu().numpy().reshape(q64.shape)
    for s, sq in enumerate(p.seqs):
        want, weight, size, reach = ref.attention(sq, q64[s], d ** -0.5)
        close(got[s], want, size, reach, d)
        n, old = len(sq), max(0, len(sq) - n_q)
        # a weight is off by its logit's error twice over (dl as in close) and fp32 sums over the rows
        rel = np.expm1(2 * reach.max(initial=0) * (2 * d + 4) * 2.0 ** -23) + 2.0 ** -12
        w = plain[s].double().cpu().numpy()
        assert np.all(np.abs(w[:, :n] - weight) <= rel * weight + 1e-30) and (w[:, n:] == 99.0).all()
        w, a = acc_out[s].double().cpu().numpy(), acc[s].double().cpu().numpy()
        sums = weight.copy()
        sums[:, :old] += 0.75 * a[:, :old]
        assert np.all(np.abs(w[:, :n] - sums) <= rel * sums + 1e-30) and (w[:, n:] == 99.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d,n_kv,g,n_q,lens,dtype", [
    (128, 2, 4, 4, [0, 70, 1200, 33], "bf16"), (64, 2, 8, 2, [900, 31, 64, 1], "f32"), (96, 1, 5, 6, [500, 45], "f32"),
    (40, 1, 1, 32, [129, 2000], "bf16"), (200, 1, 16, 1, [300], "bf16")])
def test_attention_of_many_rows_over_wide_tables(m, d, n_kv, g, n_q, lens, dtype):
    """16 query rows and more where the cache has room for much: two tiles of rows at a time."""
    test_attention(m, d, n_kv, g, n_q, lens, dtype, width=32768 // n_kv)


@pytest.mark.gpu
@pytest.mark.parametrize("d,n_seq,long", [(256, 200, 1100), (64, 300, 1100), (64, 300, 40), (128, 40, 1500), (128, 3, 6000),
                                           (128, 1, 9000), (256, 2, 20000), (64, 1, 80000)])
def test_attention_many_ragged_sequences(m, d, n_seq, long):
    """Batches of more sequences than a warp, a block or the grid has members, with few long ones among short
    and empty ones, so that work is cut within and between sequences; the same bits every time."""
    import torch
    lens = [(7 * s) % 45 for s in range(n_seq)]
    for s in (0, n_seq // 2, n_seq - 1):
        lens[s] = long - s % 7
    p = Pair(m, d, 1, n_seq, -(-long // 32) + 1, 40 + d)
    p.append(lens)
    q, q64 = p.queries(1, 3, "bf16")
    ws = p.workspace(1, 3)
    out, again = torch.full(q.shape, float("nan"), device="cuda"), torch.empty(q.shape, device="cuda")
    m.tq_b8_attention(p.cache, q, 0.1, out, ws)
    for _ in range(3):
        m.tq_b8_attention(p.cache, q, 0.1, again, ws)
        assert torch.equal(out, again)
    assert p.ok(ws)
    got = out.double().cpu().numpy().reshape(q64.shape)
    for s, sq in enumerate(p.seqs):
        want, _, size, reach = ref.attention(sq, q64[s], 0.1)
        close(got[s], want, size, reach, d)


@pytest.mark.gpu
@pytest.mark.parametrize("d,n_kv,g,lens", [
    (64, 8, 2, [250 + (977 + 40503 * s) % 1751 for s in range(30)]),
    (64, 6, 1, [0, 31] + [600 + (977 + 40503 * s) % 4301 for s in range(16)]),
    (128, 2, 4, [100, 9000, 4000, 1700, 33])])
def test_attention_parts_of_ragged_sequences(m, d, n_kv, g, lens):
    """Fewer segments than the grid has CTAs, of lengths far apart, so that parts are evened out."""
    import torch
    p = Pair(m, d, n_kv, len(lens), -(-max(lens) // 32) + 1, 47)
    p.append(lens)
    q, q64 = p.queries(1, g, "bf16")
    ws = p.workspace(1, g)
    out = torch.full(q.shape, float("nan"), device="cuda")
    m.tq_b8_attention(p.cache, q, 0.1, out, ws)
    assert p.ok(ws)
    got = out.double().cpu().numpy().reshape(q64.shape)
    for s, sq in enumerate(p.seqs):
        want, _, size, reach = ref.attention(sq, q64[s], 0.1)
        close(got[s], want, size, reach, d)


@pytest.mark.gpu
def test_attention_extremes(m):
    """Large logits of both signs, a negative scale, a zero query, a query that is not finite (its own
    row only), a tiny and a huge query."""
    import torch
    d, n_kv, g = 128, 1, 6
    p = Pair(m, d, n_kv, 1, 4, 50)
    p.append([100])
    q, _ = p.queries(1, g, "f32")
    q[0, 0, 0] *= 300.0
    q[0, 0, 1] = 0.0
    q[0, 0, 2] *= 1e-30
    q[0, 0, 3, 7] = float("inf")
    q[0, 0, 4, 9] = float("nan")
    q[0, 0, 5] *= 1e30
    ws = p.workspace(1, g)
    for scale in (0.1, -0.1):
        out = torch.zeros(q.shape, device="cuda")
        m.tq_b8_attention(p.cache, q, scale, out, ws)
        got = out.double().cpu().numpy().reshape(1, 1, g, d)
        q64 = q.double().cpu().numpy().reshape(1, 1, g, d)
        for j in (0, 1, 2):
            want, _, size, reach = ref.attention(p.seqs[0], q64[:, :, j:j + 1], scale)
            close(got[:, :, j:j + 1], want, size, reach, d)
        assert np.isnan(got[0, 0, 3]).all() and np.isnan(got[0, 0, 4]).all()
        x = p.seqs[0].values()
        top = np.argmax(scale * (x[:, 0, 0] @ q64[0, 0, 5]))     # one token takes everything
        assert np.allclose(got[0, 0, 5], x[top, 0, 1], rtol=0, atol=2.0 ** -20 * np.abs(x[top, 0, 1]).max())


@pytest.mark.gpu
def test_attention_bad_pages_and_lengths(m):
    """A page outside the pool is left out and reported; a length that cannot be counts as none."""
    import torch
    p = Pair(m, 64, 2, 3, 6, 51)
    p.append([130, 40, 90])
    for bad in (-1, p.pages.shape[0], 2 ** 31 - 1, -2 ** 31):
        table = p.table.clone()
        table[0, 1] = bad
        c = m.Cache8(64, p.pages, table, p.length, p.open_)
        q, q64 = p.queries(1, 2, "bf16")
        ws = p.workspace(1, 2)
        out, acc = torch.zeros(q.shape, device="cuda"), torch.zeros(3, 2, 192, device="cuda")
        m.tq_b8_attention(c, q, 0.125, out, ws, acc_out=acc)
        assert m.tq_get_status(ws) == m.TQ_ERR_RANGE
        part = ref.Seq(2, 64)
        part.blocks, part.open = [p.seqs[0].blocks[j] for j in (0, 2, 3)], p.seqs[0].open
        got = out.double().cpu().numpy().reshape(q64.shape)
        for s, sq in ((0, part), (1, p.seqs[1]), (2, p.seqs[2])):
            want, _, size, reach = ref.attention(sq, q64[s], 0.125)
            close(got[s], want, size, reach, 64)
        assert (acc[0, :, 32:64] == 0).all()
    for n in (-5, 193, 2 ** 31 - 1):
        length = p.length.clone()
        length[1] = n
        c = m.Cache8(64, p.pages, p.table, length, p.open_)
        out = torch.full(q.shape, 5.0, device="cuda")
        m.tq_b8_attention(c, q, 0.125, out, ws)
        assert m.tq_get_status(ws) == m.TQ_ERR_RANGE
        assert (out[1] == 0).all() and torch.isfinite(out).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d,n_kv,g,n_q,lens,n_sel,nf,nl,dtype", [
    (128, 2, 4, 1, [700, 90, 31], 5, 1, 1, "bf16"), (64, 3, 1, 1, [1500], 7, 0, 0, "f32"),
    (40, 1, 9, 3, [400, 66, 2], 4, 1, 2, "f32"), (256, 1, 8, 1, [640], 6, 2, 1, "bf16"),
    (128, 1, 12, 2, [320, 321], 10, 0, 1, "bf16"), (64, 2, 4, 1, [100, 31], 40, 1, 1, "bf16"), (8, 2, 2, 1, [999], 3, 1, 2, "f32")])
def test_select_and_sparse_attention(m, d, n_kv, g, n_q, lens, n_sel, nf, nl, dtype):
    import torch
    p = Pair(m, d, n_kv, len(lens), -(-max(lens) // 32) + 2, 60 + d)
    p.append(lens)
    q, q64 = p.queries(n_q, g, dtype)
    ws = p.workspace(n_q, g, n_sel)
    sel = torch.full((len(lens), n_q, n_kv, n_sel), 77, dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, float("nan"), device="cuda")
    acc = torch.full((len(lens), n_kv, 32 * p.nb), 99.0, device="cuda")
    m.tq_b8_select(p.cache, q, sel, ws, n_first=nf, n_last=nl)
    m.tq_b8_attention(p.cache, q, d ** -0.5, out, ws, sel=sel)
    if n_q == 1:
        old = torch.rand_like(acc)
        out2 = torch.empty_like(out)
        m.tq_b8_attention(p.cache, q, d ** -0.5, out2, ws, sel=sel, acc_in=old, acc_out=acc, decay=0.5)
        assert torch.equal(out, out2)
    assert p.ok(ws)
    got, picked = out.double().cpu().numpy().reshape(q64.shape), sel.cpu().numpy()
    for s, sq in enumerate(p.seqs):
        want_sel = ref.select(sq, q64[s], n_sel, nf, nl)
        assert np.array_equal(picked[s], want_sel)
        want, weight, size, reach = ref.attention(sq, q64[s], d ** -0.5, sel=want_sel)
        close(got[s], want, size, reach, d)
        if n_q == 1:
            n = len(sq)
            rel = np.expm1(2 * reach.max(initial=0) * (2 * d + 4) * 2.0 ** -23) + 2.0 ** -12
            sums = weight.copy()
            sums[:, :max(0, n - 1)] += 0.5 * old[s, :, :max(0, n - 1)].double().cpu().numpy()
            a = acc[s].double().cpu().numpy()
            assert np.all(np.abs(a[:, :n] - sums) <= rel * sums + 1e-30) and (a[:, n:] == 99.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d,n_kv,g,n_q,lens,width,n_sel", [
    (64, 2, 3, 1, [700, 2100, 64, 0], 300, 9), (128, 1, 9, 2, [4200], 300, 20), (256, 2, 4, 1, [1500, 900], 600, 3),
    (40, 1, 1, 1, [9000], 300, 40), (64, 5, 2, 3, [330 + 97 * s for s in range(10)], 300, 8),
    (128, 3, 1, 1, [40 + 31 * s for s in range(50)], 400, 12), (64, 1, 17, 1, [3300, 64], 104, 2)])
def test_select_over_tables_of_several_widths(m, d, n_kv, g, n_q, lens, width, n_sel):
    """Rows of few and of many blocks, few and many rows, and rows with no more blocks than are chosen."""
    import torch
    p = Pair(m, d, n_kv, len(lens), width, 76)
    p.append(lens)
    q, q64 = p.queries(n_q, g, "f32")
    ws = p.workspace(n_q, g, n_sel)
    sel = torch.full((len(lens), n_q, n_kv, n_sel), 77, dtype=torch.int32, device="cuda")
    m.tq_b8_select(p.cache, q, sel, ws, n_first=1, n_last=1)
    assert p.ok(ws)
    for s, sq in enumerate(p.seqs):
        assert np.array_equal(sel[s].cpu().numpy(), ref.select(sq, q64[s], n_sel, 1, 1)), s


@pytest.mark.gpu
def test_select_ties_and_odd_queries(m):
    """Equal blocks score the same: the lowest numbers win. A query of zeros, NaN or infinities scores 0."""
    import torch
    d = 64
    p = Pair(m, d, 1, 1, 20, 70)
    k, v = p.tokens(32)
    for _ in range(19):
        p.length += 32
        m.tq_b8_append(p.cache, torch.from_numpy(k[None]).cuda(), torch.from_numpy(v[None]).cuda(), p.ws)
        p.seqs[0].append(k, v)
    ws = p.workspace(1, 1, 6)
    for fill in (None, 0.0, float("nan"), float("inf")):
        q, q64 = p.queries(1, 1, "f32")
        if fill is not None:
            q[0, 0, 0, 5 if fill else slice(None)] = fill
            q64 = q.double().cpu().numpy().reshape(1, 1, 1, 1, d)
        sel = torch.zeros(1, 1, 1, 6, dtype=torch.int32, device="cuda")
        m.tq_b8_select(p.cache, q, sel, ws, n_first=0, n_last=2)
        assert sel.flatten().tolist() == [0, 1, 2, 3, 17, 18]
        assert np.array_equal(sel[0].cpu().numpy(), ref.select(p.seqs[0], q64[0], 6, 0, 2))


@pytest.mark.gpu
def test_select_scores_that_underflow_are_ties(m):
    """Block 0's score is negative and below the smallest fp32 number, the others' are 0: the lowest number wins."""
    import torch
    d = 64
    p = Pair(m, d, 1, 1, 4, 73)
    for x in (-(2.0 ** -99), 0.0, 0.0, 0.0):
        k = np.full((32, 1, d), x, np.float32)
        p.length += 32
        m.tq_b8_append(p.cache, torch.from_numpy(k[None]).cuda(), torch.from_numpy(k[None]).cuda(), p.ws)
        p.seqs[0].append(k, k)
    ws = p.workspace(1, 1, 1)
    q = torch.full((1, 1, 1, d), 2.0 ** -99, device="cuda")
    sel = torch.full((1, 1, 1, 1), 77, dtype=torch.int32, device="cuda")
    m.tq_b8_select(p.cache, q, sel, ws, n_first=0, n_last=0)
    assert p.ok(ws) and sel.flatten().tolist() == [0]
    assert ref.select(p.seqs[0], q.double().cpu().numpy().reshape(1, 1, 1, d), 1, 0, 0).flatten().tolist() == [0]


@pytest.mark.gpu
def test_sparse_attention_with_a_hand_made_selection(m):
    """Entries outside the full blocks are passed over; the order does not matter to the result's meaning."""
    import torch
    d, n_kv, g = 128, 2, 4
    p = Pair(m, d, n_kv, 2, 12, 71)
    p.append([333, 20])
    q, q64 = p.queries(1, g, "bf16")
    sel = torch.tensor([[7, -1, 2, 99, 10, 0, -2 ** 31], [5, 4, 3, 2, 1, 0, -1]], dtype=torch.int32, device="cuda")
    sel = sel[None, None].expand(2, 1, 2, 7).contiguous()
    ws = p.workspace(1, g, 7)
    out = torch.zeros(q.shape, device="cuda")
    m.tq_b8_attention(p.cache, q, 0.1, out, ws, sel=sel)
    assert p.ok(ws)
    for s, sq in enumerate(p.seqs):
        want, _, size, reach = ref.attention(sq, q64[s], 0.1, sel=sel[s].cpu().numpy())
        close(out[s].double().cpu().numpy().reshape(want.shape), want, size, reach, d)


@pytest.mark.gpu
@pytest.mark.parametrize("d,n_kv,lens,keep,nf,nl", [
    (128, 3, [700, 64, 31, 0], 4, 4, 32), (64, 2, [1111], 9, 0, 0), (40, 1, [300, 333], 5, 160, 0),
    (256, 2, [400], 7, 3, 50), (128, 1, [2000, 64], 1, 0, 32), (8, 2, [500], 15, 1, 1), (64, 1, [100, 70], 9, 4, 128)])
def test_evict(m, d, n_kv, lens, keep, nf, nl):
    import torch
    nb = -(-max(lens) // 32) + 1
    p = Pair(m, d, n_kv, len(lens), nb, 80 + d, spare=len(lens) * nb)
    p.append(lens)
    n_seq = len(lens)
    acc = torch.from_numpy(np.exp(2 * p.rng.standard_normal((n_seq, n_kv, 32 * p.nb))).astype(np.float32)).cuda()
    acc[:, :, ::7] = 0.5                                             # ties
    acc[:, 0, 1::11] = -3.0
    acc[:, -1, 2::13] = float("nan")
    dst = torch.from_numpy(p.names[n_seq * p.nb:].reshape(n_seq, p.nb).copy()).cuda()
    kept = torch.full((n_seq, n_kv, 32 * keep), 7, dtype=torch.int32, device="cuda")
    length, acc_out = torch.zeros_like(p.length), torch.full_like(acc, 99.0)
    before = p.pages.clone()
    m.tq_b8_evict(p.cache, acc, keep, dst, kept, length, acc_out, p.ws, n_first=nf, n_last=nl)
    assert p.ok()
    a = acc.cpu().numpy()
    for s, sq in enumerate(p.seqs):
        new, want_kept, moved = ref.evict(sq, np.nan_to_num(a[s], nan=0.0), keep, nf, nl)
        assert np.array_equal(kept[s].cpu().numpy(), want_kept)
        assert int(length[s]) == len(new)
        got = acc_out[s].cpu().numpy()
        assert np.array_equal(np.nan_to_num(got[:, :len(new)], nan=0.0), moved) and (got[:, len(new):] == 99.0).all()
        p.seqs[s] = new
    old = p.table.flatten().long()
    assert torch.equal(p.pages[old], before[old])
    p.pages[old] = 255
    p.table.copy_(dst)
    p.length.copy_(length)
    p.check_bytes()


@pytest.mark.gpu
def test_evict_into_its_own_pages_within_budget(m):
    """A sequence within its budget may keep its pages: the bytes stay."""
    import torch
    p = Pair(m, 128, 2, 2, 8, 90, spare=8)
    p.append([250, 100])
    acc = torch.rand(2, 2, 256, device="cuda")
    dst = p.table.clone()
    dst[0] = torch.from_numpy(p.names[16:]).cuda()
    kept = torch.zeros(2, 2, 160, dtype=torch.int32, device="cuda")
    length, acc_out = torch.zeros_like(p.length), torch.zeros_like(acc)
    own = p.pages[p.table[1].long()].clone()
    m.tq_b8_evict(p.cache, acc, 5, dst, kept, length, acc_out, p.ws)
    assert p.ok() and length.tolist() == [160 + 250 % 32, 100]
    assert torch.equal(p.pages[p.table[1].long()], own)
    assert kept[1, 0, :97].tolist() == list(range(96)) + [-1]
    assert torch.equal(acc_out[1, :, :100], acc[1, :, :100])


@pytest.mark.gpu
def test_a_session_and_its_replayed_step(m):
    """Prompt, decode steps that accumulate weights, eviction, more steps with selected blocks; the step
    is captured once and replayed while lengths and tables change, on a stream of its own."""
    import torch
    d, n_kv, g, n_seq, nb = 64, 2, 4, 3, 16
    p = Pair(m, d, n_kv, n_seq, nb, 95, spare=n_seq * nb)
    p.append([300, 95, 1])
    ws = p.workspace(1, g, 4)
    acc = torch.zeros(n_seq, n_kv, 32 * nb, device="cuda")
    k = torch.zeros(n_seq, 1, n_kv, d, device="cuda")
    v = torch.zeros_like(k)
    q = torch.zeros(n_seq, 1, n_kv * g, d, device="cuda")
    out, sparse = torch.zeros_like(q), torch.zeros_like(q)
    sel = torch.zeros(n_seq, 1, n_kv, 4, dtype=torch.int32, device="cuda")

    def step():
        p.length.add_(1)
        m.tq_b8_append(p.cache, k, v, ws)
        m.tq_b8_attention(p.cache, q, 0.125, out, ws, acc_in=acc, acc_out=acc, decay=0.9)
        m.tq_b8_select(p.cache, q, sel, ws)
        m.tq_b8_attention(p.cache, q, 0.125, sparse, ws, sel=sel)

    want_acc = [np.zeros((n_kv, 32 * nb)) for _ in range(n_seq)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    saved = [t.clone() for t in (p.length, p.open_, p.pages, acc)]
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    for t, o in zip((p.length, p.open_, p.pages, acc), saved):
        t.copy_(o)
    with torch.cuda.graph(graph, stream=side):
        step()

    def replay(count):
        for _ in range(count):
            kn, vn = zip(*(p.tokens(1) for _ in range(n_seq)))
            qn = p.rng.standard_normal((n_seq, 1, n_kv * g, d)).astype(np.float32)
            for t, x in ((k, np.stack(kn)), (v, np.stack(vn)), (q, qn)):
                t.copy_(torch.from_numpy(x.astype(np.float32)))
            graph.replay()
            torch.cuda.synchronize()
            for s, sq in enumerate(p.seqs):
                sq.append(kn[s], vn[s])
                q64 = qn[s].astype(np.float64).reshape(1, n_kv, g, d)
                want, weight, size, reach = ref.attention(sq, q64, 0.125)
                close(out[s].double().cpu().numpy().reshape(want.shape), want, size, reach, d)
                n = len(sq)
                want_acc[s][:, :n] = 0.9 * want_acc[s][:, :n] + weight
                got = acc[s].double().cpu().numpy()
                rel = np.expm1(2 * reach.max() * (2 * d + 4) * 2.0 ** -23) + 2.0 ** -12
                assert np.all(np.abs(got - want_acc[s]) <= rel * want_acc[s] + 1e-30)
                want_sel = ref.select(sq, q64, 4, 1, 1)
                assert np.array_equal(sel[s].cpu().numpy(), want_sel)
                want, _, size, reach = ref.attention(sq, q64, 0.125, sel=want_sel)
                close(sparse[s].double().cpu().numpy().reshape(want.shape), want, size, reach, d)

    replay(3)
    dst = torch.from_numpy(p.names[n_seq * nb:].reshape(n_seq, nb).copy()).cuda()
    kept = torch.zeros(n_seq, n_kv, 32 * 5, dtype=torch.int32, device="cuda")
    length, acc_out = torch.zeros_like(p.length), torch.zeros_like(acc)
    a = acc.cpu().numpy()
    m.tq_b8_evict(p.cache, acc, 5, dst, kept, length, acc_out, ws, n_first=2, n_last=16)
    for s in range(n_seq):
        p.seqs[s], want_kept, moved = ref.evict(p.seqs[s], a[s], 5, 2, 16)
        assert np.array_equal(kept[s].cpu().numpy(), want_kept)
        want_acc[s][:] = 0
        want_acc[s][:, :moved.shape[1]] = moved
    p.pages[p.table.flatten().long()] = 255
    p.table.copy_(dst)
    p.length.copy_(length)
    acc.copy_(acc_out)
    replay(34)
    assert p.ok(ws)
    p.check_bytes()


@pytest.mark.gpu
def test_pool_beyond_4_gib(m):
    """Pages whose byte offsets pass 32 bits."""
    import torch
    d, n_kv = 128, 8
    p = Pair(m, d, n_kv, 1, 3, 97)
    n_pages = (5 << 30) // m.tq_b8_page_bytes(d, n_kv)
    pages = torch.empty(n_pages, m.tq_b8_page_bytes(d, n_kv), dtype=torch.uint8, device="cuda")
    p.pages = pages
    p.table.copy_(torch.tensor([[n_pages - 1, n_pages - 2, n_pages - 3]], dtype=torch.int32))
    p.cache = m.Cache8(d, pages, p.table, p.length, p.open_)
    p.append([90])
    q, q64 = p.queries(1, 4, "bf16")
    ws = p.workspace(1, 4)
    out = torch.zeros(q.shape, device="cuda")
    m.tq_b8_attention(p.cache, q, 0.1, out, ws)
    assert p.ok(ws) and p.ok()
    want, _, size, reach = ref.attention(p.seqs[0], q64[0], 0.1)
    close(out[0].double().cpu().numpy().reshape(want.shape), want, size, reach, d)


@pytest.mark.gpu
def test_values_that_a_query_does_not_see(m):
    """Several new tokens, the last of which are not finite in keys and values: queries before them answer as
    if they were not there, those that see them do not."""
    import torch
    for d, n_old in ((64, 37), (128, 64), (200, 13)):
        p = Pair(m, d, 2, 1, 4, 98)
        p.append([n_old])
        k, v = p.tokens(3)
        kb, vb = k.copy(), v.copy()
        kb[1, 0, 3], vb[1, 0, 5], vb[2, 1, 0], kb[2, 1, 1] = np.nan, np.inf, np.nan, -np.inf
        p.length += 3
        p.seqs[0].append(k, v)
        m.tq_b8_append(p.cache, torch.from_numpy(kb[None]).cuda(), torch.from_numpy(vb[None]).cuda(), p.ws)
        q, q64 = p.queries(3, 2, "bf16")
        ws = p.workspace(3, 2)
        out = torch.zeros(q.shape, device="cuda")
        m.tq_b8_attention(p.cache, q, 0.1, out, ws)
        assert p.ok(ws)
        got = out.double().cpu().numpy().reshape(q64.shape)[0]
        want, _, size, reach = ref.attention(p.seqs[0], q64[0], 0.1)
        close(got[0], want[0], size[0], reach[0], d)
        close(got[1, 1], want[1, 1], size[1, 1], reach[1, 1], d)      # head 1 is hurt by the last token only
        assert not np.isfinite(got[1, 0]).all() and not np.isfinite(got[2]).all()


@pytest.mark.gpu
def test_read_and_evict_bad_pages(m):
    """A source page outside the pool counts as zeros and is left out of reads; a target page outside it is
    not written; both are reported."""
    import torch
    p = Pair(m, 64, 1, 1, 6, 99, spare=6)
    p.append([192])
    table = p.table.clone()
    table[0, 2] = p.pages.shape[0]
    c = m.Cache8(64, p.pages, table, p.length, p.open_)
    k, v = (torch.full((1, 192, 1, 64), 768.0, device="cuda") for _ in range(2))
    m.tq_b8_read(c, k, v, p.ws)
    assert m.tq_get_status(p.ws) == m.TQ_ERR_RANGE
    x = p.seqs[0].values()
    for side, got in enumerate((k, v)):
        g = got[0, :, 0].double().cpu().numpy()
        assert (g[64:96] == 768.0).all()
        keep = np.r_[0:64, 96:192]
        assert np.all(np.abs(g[keep] - x[keep, 0, side]) <= 2.0 ** -24 * np.abs(x[keep, 0, side]) + 1e-40)
    acc = torch.arange(192, dtype=torch.float32, device="cuda").reshape(1, 1, 192)
    dst = torch.from_numpy(p.names[6:].reshape(1, 6).copy()).cuda()
    dst[0, 1] = -7
    kept, length = torch.zeros(1, 1, 96, dtype=torch.int32, device="cuda"), torch.zeros_like(p.length)
    acc_out, before = torch.zeros_like(acc), p.pages.clone()
    m.tq_b8_evict(c, acc, 3, dst, kept, length, acc_out, p.ws, n_first=64)
    assert m.tq_get_status(p.ws) == m.TQ_ERR_RANGE
    assert kept[0, 0].tolist() == list(range(64)) + list(range(160, 192)) and length.tolist() == [96]
    assert acc_out[0, 0, :96].tolist() == [float(t) for t in kept[0, 0].tolist()]
    written = (p.pages != before).any(dim=1).nonzero().flatten().tolist()
    assert set(written) <= {int(dst[0, 0]), int(dst[0, 2])}


@pytest.mark.gpu
def test_evict_and_select_of_long_rows(m):
    """Rows longer than the choosing kernel keeps in registers: 20011 tokens, 17000 blocks."""
    import torch
    p = Pair(m, 8, 1, 1, 626, 101, spare=626)
    p.append([20011])
    acc = torch.rand(1, 1, 626 * 32, device="cuda")
    acc[0, 0, 5000:9000] = 0.5                                        # a tie across the border
    dst = torch.from_numpy(p.names[626:].reshape(1, 626).copy()).cuda()
    for keep in (10, 313, 600):
        kept, length = torch.zeros(1, 1, 32 * keep, dtype=torch.int32, device="cuda"), torch.zeros_like(p.length)
        m.tq_b8_evict(p.cache, acc, keep, dst, kept, length, torch.zeros_like(acc), p.ws, n_first=5, n_last=100)
        want = ref.choose(acc[0, 0].cpu().numpy(), 625 * 32, 32 * keep, 5, 100)
        assert np.array_equal(kept[0, 0].cpu().numpy(), want)
    # block selection: only lengths, tables and summaries matter
    nb = 17000
    d, n_pages = 8, 64
    pages = torch.zeros(n_pages, m.tq_b8_page_bytes(d, 1), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(3)
    lo = rng.integers(-127, 1, (n_pages, d)).astype(np.int8)
    hi = rng.integers(0, 128, (n_pages, d)).astype(np.int8)
    scale = rng.uniform(0.01, 0.02, n_pages).astype(np.float32)
    host = np.zeros((n_pages, 32 + 128), np.uint8)
    host[:, :4] = scale.view(np.uint8).reshape(-1, 4)
    host[:, 32:32 + d], host[:, 96:96 + d] = lo.view(np.uint8), hi.view(np.uint8)
    pages[:, :160] = torch.from_numpy(host).cuda()
    table = torch.from_numpy(rng.integers(0, n_pages, (1, nb)).astype(np.int32)).cuda()      # pages many times over: ties
    length = torch.full((1,), nb * 32, dtype=torch.int32, device="cuda")
    c = m.Cache8(d, pages, table, length, torch.zeros(1, 1, 2, 32, d, dtype=torch.bfloat16, device="cuda"))
    q = torch.randn(1, 1, 2, d, device="cuda")
    for n_sel in (3, 500, 16500):
        ws = m.workspace(m.tq_b8_workspace_bytes(c, 1, 2, n_sel))
        sel = torch.zeros(1, 1, 1, n_sel, dtype=torch.int32, device="cuda")
        m.tq_b8_select(c, q, sel, ws)
        assert m.tq_get_status(ws) == m.TQ_OK
        best = np.full(n_pages, -np.inf, np.float32)
        for x in q[0, 0].double().cpu().numpy():
            a = np.float32(np.abs(x).max())
            qi = np.rint(x * np.float64(np.float32(1) / a * np.float32(127)))
            whole = np.maximum(qi * lo, qi * hi).sum(axis=1).astype(np.float32)
            best = np.maximum(best, whole * scale * (a * ref.INV127))
        want = ref.choose(best[table[0].cpu().numpy()], nb, n_sel, 1, 1)
        assert np.array_equal(sel[0, 0, 0].cpu().numpy(), want)


@pytest.mark.gpu
def test_streams_graphs_and_workspaces(m):
    """Calls at once on two streams with workspaces of their own; two captured graphs that share one
    workspace, replayed in turn; a workspace that other calls have used; a reset workspace."""
    import torch
    d, n_kv, g = 128, 4, 4
    p = Pair(m, d, n_kv, 3, 70, 102)
    p.append([2200, 700, 33])
    qs, outs, want = [], [], []
    for _ in range(2):
        q, q64 = p.queries(1, g, "bf16")
        qs.append(q)
        outs.append(torch.zeros(q.shape, device="cuda"))
        want.append([ref.attention(sq, q64[s], 0.1) for s, sq in enumerate(p.seqs)])

    def check():
        for out, w in zip(outs, want):
            got = out.double().cpu().numpy().reshape(3, 1, n_kv, g, d)
            for s in range(3):
                close(got[s], w[s][0], w[s][2], w[s][3], d)
            out.zero_()

    need = m.tq_b8_workspace_bytes(p.cache, 1, g)
    dirty = torch.randint(1, 255, (need,), dtype=torch.uint8, device="cuda")
    m.tq_reset_status(dirty)
    assert (dirty[:256] == 0).all() and (dirty[256:] != 0).any()
    spaces = [dirty, m.workspace(need)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for q, out, ws, st in zip(qs, outs, spaces, streams):
            m.tq_b8_attention(p.cache, q, 0.1, out, ws, stream=st)
    torch.cuda.synchronize()
    check()
    graphs = []
    for q, out in zip(qs, outs):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            m.tq_b8_attention(p.cache, q, 0.1, out, dirty)
        graphs.append(gr)
    for _ in range(3):
        for gr in graphs:
            gr.replay()
    torch.cuda.synchronize()
    check()
    x = torch.randn(2, 64, d, device="cuda")
    packed = torch.zeros(m.tq_q8_packed_bytes(d, 2, 64), dtype=torch.uint8, device="cuda")
    for q, out in zip(qs, outs):
        m.tq_q8_quantize(x, d, 2, 64, 64 * d, packed, dirty)
        m.tq_b8_attention(p.cache, q, 0.1, out, dirty)
    check()
    assert m.tq_get_status(dirty) == m.TQ_OK and (dirty[:256] == 0).all()
