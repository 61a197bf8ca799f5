"""Plain 64-bit reference of the paged 8-bit cache, written from the format description in
include/tq.h (numpy, one block or one token at a time). Test infrastructure: shares no code
with the library."""
from __future__ import annotations

import numpy as np

BLOCK = 32
INV127 = np.float32(1) / np.float32(127)


def padded(d):
    return 64 if d <= 64 else 128 if d <= 128 else 256


def header_bytes(d, n_kv):
    return -(-n_kv * (32 + 2 * padded(d)) // 128) * 128


def page_bytes(d, n_kv):
    return header_bytes(d, n_kv) + n_kv * 64 * padded(d)


def to_bf16(x):
    """fp32 -> the bf16 value it rounds to (fp64); infinities and NaN stay."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7fff + ((u >> 16) & 1)) >> 16 << 16).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(x), np.nan, r).astype(np.float64)


def swz(t, D):
    s = 0
    if t & 2:
        s |= 2
    if (t ^ (t >> 2)) & 1:
        s |= 4
    return s & (D // 16 - 1)


def quantize(x):
    """x [32, d] -> codes (int), scale (fp32), whether every value was finite."""
    fin = np.isfinite(x)
    x = np.where(fin, x, 0.0)
    a = np.float32(np.max(np.abs(x)))
    if a < np.float32(2.0 ** -100):
        return np.zeros(x.shape, int), np.float32(0), bool(fin.all())
    inv = np.float32(1) / a * np.float32(127)
    return np.rint(x * np.float64(inv)).astype(int), a * INV127, bool(fin.all())


def page_of(kc, ks, vc, vs):
    """Codes [n_kv, 32, d], scales [n_kv] -> the page's bytes (unused bytes 0)."""
    n_kv, _, d = kc.shape
    D = padded(d)
    out = np.zeros(page_bytes(d, n_kv), np.uint8)
    for h in range(n_kv):
        e = h * (32 + 2 * D)
        out[e:e + 4] = np.frombuffer(np.float32(ks[h]).tobytes(), np.uint8)
        out[e + 4:e + 8] = np.frombuffer(np.float32(vs[h]).tobytes(), np.uint8)
        out[e + 32:e + 32 + d] = kc[h].min(axis=0).astype(np.int8).view(np.uint8)
        out[e + 32 + D:e + 32 + D + d] = kc[h].max(axis=0).astype(np.int8).view(np.uint8)
        for side, codes in enumerate((kc[h], vc[h])):
            base = header_bytes(d, n_kv) + (2 * h + side) * BLOCK * D
            for t in range(BLOCK):
                row = np.full(D, 128, np.uint8)
                row[:d] = (codes[t] + 128).astype(np.uint8)
                for ch in range(D // 16):
                    at = base + t * D + (ch ^ swz(t, D)) * 16
                    out[at:at + 16] = row[ch * 16:ch * 16 + 16]
    return out


def unpack(page, d, n_kv):
    """A page's bytes -> codes [n_kv, 2, 32, d] (int), scales [n_kv, 2] (fp32), lo, hi [n_kv, d]."""
    D = padded(d)
    codes = np.zeros((n_kv, 2, BLOCK, d), int)
    scales = np.zeros((n_kv, 2), np.float32)
    lo, hi = np.zeros((n_kv, d), int), np.zeros((n_kv, d), int)
    for h in range(n_kv):
        e = h * (32 + 2 * D)
        scales[h] = page[e:e + 8].copy().view(np.float32)
        lo[h] = page[e + 32:e + 32 + d].view(np.int8)
        hi[h] = page[e + 32 + D:e + 32 + D + d].view(np.int8)
        for side in range(2):
            base = header_bytes(d, n_kv) + (2 * h + side) * BLOCK * D
            for t in range(BLOCK):
                row = np.concatenate([page[base + t * D + (ch ^ swz(t, D)) * 16:][:16] for ch in range(D // 16)])
                codes[h, side, t] = row[:d].astype(int) - 128
    return codes, scales, lo, hi


class Seq:
    """One sequence: full blocks as codes and scales, open tokens as bf16 values."""

    def __init__(self, n_kv, d):
        self.n_kv, self.d = n_kv, d
        self.blocks = []                 # (codes [n_kv, 2, 32, d], scales [n_kv, 2])
        self.open = np.zeros((0, n_kv, 2, d))
        self.finite = True

    def __len__(self):
        return BLOCK * len(self.blocks) + len(self.open)

    def append(self, k, v):
        """k, v [n, n_kv, d] fp32"""
        x = np.stack([to_bf16(k), to_bf16(v)], axis=2)
        self.open = np.concatenate([self.open, x])
        while len(self.open) >= BLOCK:
            blk, self.open = self.open[:BLOCK], self.open[BLOCK:]
            codes = np.zeros((self.n_kv, 2, BLOCK, self.d), int)
            scales = np.zeros((self.n_kv, 2), np.float32)
            for h in range(self.n_kv):
                for side in range(2):
                    codes[h, side], scales[h, side], fin = quantize(blk[:, h, side])
                    self.finite = self.finite and fin
            self.blocks.append((codes, scales))

    def page(self, j):
        codes, scales = self.blocks[j]
        return page_of(codes[:, 0], scales[:, 0], codes[:, 1], scales[:, 1])

    def values(self):
        """[len, n_kv, 2, d] in 64 bits"""
        parts = [(c * s.astype(np.float64)[:, :, None, None]).transpose(2, 0, 1, 3) for c, s in self.blocks]
        return np.concatenate(parts + [self.open]) if parts else self.open


def attention(seq, q, scale, sel=None, n_full=None):
    """q [n_q, n_kv, g, d] -> out [n_q, n_kv, g, d], weights [n_kv, len], size [n_q, n_kv, g] (sum of w |v|,
    for tolerances) and reach [n_q, n_kv, g] (largest scale * sum |q_i k_i|). sel: blocks [n_q, n_kv, n_sel]."""
    n_q, n_kv, g, d = q.shape
    x, n = seq.values(), len(seq)
    out, size, reach = np.zeros(q.shape), np.zeros(q.shape[:3]), np.zeros(q.shape[:3])
    weight = np.zeros((n_kv, n))
    for i in range(n_q):
        last = n - n_q + i
        for h in range(n_kv):
            pos = np.arange(max(0, last + 1))
            if sel is not None:
                full = len(seq.blocks)
                pos = np.concatenate([np.arange(BLOCK * b, BLOCK * b + BLOCK) for b in sel[i, h] if 0 <= b < full] +
                                     [np.arange(BLOCK * full, n)]).astype(int)
                pos = pos[pos <= last]
            if last < 0 or len(pos) == 0:
                continue
            k, v = x[pos, h, 0], x[pos, h, 1]
            l = scale * (q[i, h] @ k.T)
            w = np.exp(l - l.max(axis=1, keepdims=True))
            w /= w.sum(axis=1, keepdims=True)
            out[i, h] = w @ v
            size[i, h] = (w @ np.abs(v)).max(axis=1)
            reach[i, h] = (abs(scale) * (np.abs(q[i, h]) @ np.abs(k).T)).max(axis=1)
            np.add.at(weight[h], pos, w.sum(axis=0))
    return out, weight, size, reach


def choose(key, n, k, nf, nl):
    """Ascending indices of the chosen, filled up with -1."""
    if n <= k:
        got = list(range(n))
    else:
        must = set(range(nf)) | set(range(n - nl, n))
        rest = sorted((t for t in range(n) if t not in must), key=lambda t: (-key[t], t))
        got = sorted(must | set(rest[:k - len(must)]))
    return np.array(got + [-1] * (k - len(got)), np.int32)


def select(seq, q, n_sel, nf, nl):
    """q [n_q, n_kv, g, d] -> sel [n_q, n_kv, n_sel], by the definition's whole numbers and fp32 products."""
    n_q, n_kv, g, d = q.shape
    out = np.zeros((n_q, n_kv, n_sel), np.int32)
    n = len(seq)
    for i in range(n_q):
        last = n - n_q + i
        nb = 0 if last < 0 else min(n // BLOCK, last // BLOCK + 1)
        for h in range(n_kv):
            score = np.full(nb, -np.inf, np.float32)
            for j in range(g):
                x = q[i, h, j]
                a = np.float32(np.max(np.abs(x))) if np.isfinite(x).all() else np.float32(0)
                live = a >= np.float32(2.0 ** -100)
                qi = np.rint(x * np.float64(np.float32(1) / a * np.float32(127))) if live else np.zeros(d)
                step = a * INV127 if live else np.float32(0)
                for b in range(nb):
                    kc = seq.blocks[b][0][h, 0]
                    whole = np.maximum(qi * kc.min(axis=0), qi * kc.max(axis=0)).sum()
                    score[b] = max(score[b], np.float32(np.float32(whole) * seq.blocks[b][1][h, 0]) * step)
            out[i, h] = choose(score, nb, n_sel, nf, nl)
    return out


def evict(seq, acc, keep, nf, nl):
    """acc [n_kv, >= len] fp32 -> new Seq, kept [n_kv, 32 keep], acc of the tokens that stay [n_kv, new len]"""
    full, n_kv, d = len(seq.blocks), seq.n_kv, seq.d
    new = Seq(n_kv, d)
    new.open = seq.open
    left = min(full, keep)
    new.blocks = [(np.zeros((n_kv, 2, BLOCK, d), int), np.zeros((n_kv, 2), np.float32)) for _ in range(left)]
    kept = np.zeros((n_kv, BLOCK * keep), np.int32)
    moved = np.zeros((n_kv, len(new)), np.float32)
    for h in range(n_kv):
        key = np.where(acc[h] > 0, acc[h], 0)
        kept[h] = choose(key, BLOCK * full, BLOCK * keep, nf, nl)
        moved[h] = np.concatenate([acc[h][kept[h][:BLOCK * left]], acc[h][BLOCK * full:len(seq)]])
        for j in range(left):
            src = kept[h][BLOCK * j:BLOCK * j + BLOCK]
            for side in range(2):
                code = np.stack([seq.blocks[t // BLOCK][0][h, side, t % BLOCK] for t in src])
                sc = np.array([seq.blocks[t // BLOCK][1][h, side] for t in src], np.float32)
                top = np.abs(code).max(axis=1).astype(np.float32) * INV127 * sc
                s = top.max()
                ratio = sc / s if s > 0 else np.zeros(BLOCK, np.float32)
                new.blocks[j][0][h, side] = np.rint(code * ratio.astype(np.float64)[:, None]).astype(int)
                new.blocks[j][1][h, side] = s
    return new, kept, moved
