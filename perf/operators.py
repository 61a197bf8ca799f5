"""Workloads of the paged 8-bit KV cache: appending tokens, decode attention over the cache,
attention over selected blocks, and eviction of the tokens that were attended to least.

``run`` computes each of them twice over: as elementary torch operations on the cache's bytes,
or, with ``own`` set, by the library's entry points.

The cache. A page holds 32 tokens of all kv heads. With D = 64, 128 or 256 (the head size d
rounded up) and n_kv heads, a page is
  header, n_kv entries of 32 + 2 D bytes: the key scale and the value scale (fp32), 24 unused
    bytes, then lo[D] and hi[D] (int8): the smallest and the largest key code of each channel;
    the header is padded to a multiple of 128 bytes;
  codes, n_kv entries of 64 D bytes: keys [32][D], then values [32][D], each code an unsigned
    byte (code + 128). The 16-byte chunk c of token t lies at chunk c ^ swz(t) of its row,
    swz(t) = ((t & 2) | (((t ^ (t >> 2)) & 1) << 2)) mod (D / 16).
A block (32 tokens of one head) has one scale for its keys and one for its values: with
a = max |x|, scale = a / 127 and code = rint(x * (127 / a)). The last len mod 32 tokens of a
sequence wait in bf16 in the open block until it is full.
"""
import math

import torch

own = False

BLOCK = 32
F32 = torch.float32


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of a serving batch: every sequence gets one token, some blocks fill up
        dict(name="append step b64", op="append", n_seq=64, tokens=2000, ragged=True, n_kv=8, d=128, n_new=1,
             dtype="bf16"),
        # the prefill append of the batched serving workload
        dict(name="append prompt 64x512", op="append", n_seq=64, tokens=1024, ragged=False, n_kv=8, d=128,
             n_new=512, dtype="bf16"),
        # odd prompt pieces of several lengths, fp32 rows, a head size that is not a power of two
        dict(name="append pieces fp32 d80", op="append", n_seq=9, tokens=2777, ragged=True, n_kv=5, d=80,
             n_new=777, dtype="f32"),
        # the smallest decode step: one short conversation, latency
        dict(name="decode 1x500", op="attention", n_seq=1, tokens=500, ragged=False, n_kv=8, g=4, d=128, n_q=1,
             dtype="bf16", weights=False),
        # single-sequence decode at 32K
        dict(name="decode 1x32768", op="attention", n_seq=1, tokens=32768, ragged=False, n_kv=8, g=4, d=128, n_q=1,
             dtype="bf16", weights=False),
        # batched decode serving, the largest call
        dict(name="decode 64x8192", op="attention", n_seq=64, tokens=8192, ragged=False, n_kv=8, g=4, d=128, n_q=1,
             dtype="bf16", weights=False),
        # ragged batch, four new tokens each (draft tokens to verify), small heads, fp32 queries
        dict(name="decode 24x5001 q4 fp32 d64", op="attention", n_seq=24, tokens=5001, ragged=True, n_kv=4, g=6,
             d=64, n_q=4, dtype="f32", weights=False),
        # a decode step that also accumulates the attention weights that eviction goes by
        dict(name="decode weights 16x8100", op="attention", n_seq=16, tokens=8100, ragged=True, n_kv=8, g=4, d=128,
             n_q=1, dtype="bf16", weights=True),
        # long context: 64 of 4096 blocks
        dict(name="sparse 1x131072", op="sparse", n_seq=1, tokens=131072, ragged=False, n_kv=8, g=4, d=128, n_q=1,
             dtype="bf16", n_sel=64),
        # a batch of long ragged sequences
        dict(name="sparse 32x16384", op="sparse", n_seq=32, tokens=16384, ragged=True, n_kv=8, g=4, d=128, n_q=1,
             dtype="bf16", n_sel=48),
        # one sequence over its budget
        dict(name="evict 1x4096", op="evict", n_seq=1, tokens=4111, ragged=False, n_kv=8, d=128, keep=64),
        # a whole batch back to half its length
        dict(name="evict 32x8192", op="evict", n_seq=32, tokens=8192, ragged=True, n_kv=8, d=128, keep=128),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["append", "attention", "attention", "sparse", "evict"])
    n_kv = rng.choice([1, 2, 3, 4, 5, 8, 8])
    d = rng.choice([40, 64, 80, 96, 128, 128, 128, 192, 256])
    room = 64 * 8192 * 8 * 128 // (2 * n_kv * (64 if d <= 64 else 128 if d <= 128 else 256))  # tokens in all
    c = dict(op=op, n_kv=n_kv, d=d, ragged=rng.random() < 0.6)
    if op == "append":
        c["n_seq"] = log(1, 64)
        c["n_new"] = min(log(1, 1024), max(1, room // (4 * c["n_seq"])))
        c["tokens"] = c["n_new"] + rng.randrange(0, 1000)
        c["dtype"] = rng.choice(["bf16", "bf16", "f32"])
    elif op == "attention":
        c["tokens"] = log(40, 65536)
        c["n_seq"] = log(1, max(1, min(64, room // c["tokens"])))
        c["g"] = rng.choice([1, 2, 3, 4, 5, 7, 8])
        c["n_q"] = rng.choice([1, 1, 1, 2, 3, 5])
        c["dtype"] = rng.choice(["bf16", "bf16", "f32"])
        c["weights"] = rng.random() < 0.4
    elif op == "sparse":
        c["tokens"] = log(2000, 131072)
        c["n_seq"] = log(1, max(1, min(32, room // c["tokens"])))
        c["g"] = rng.choice([1, 2, 4, 4, 8])
        c["n_q"] = 1
        c["dtype"] = rng.choice(["bf16", "bf16", "f32"])
        c["n_sel"] = rng.randrange(4, 129)
    else:
        c["tokens"] = log(300, 32768)
        c["n_seq"] = log(1, max(1, min(32, room // c["tokens"])))
        c["keep"] = max(5, int(c["tokens"] // BLOCK * rng.uniform(0.2, 0.9)))
    return c


def lengths(case):
    """Tokens of each sequence, those appended in this pass included."""
    n, most = case["n_seq"], case["tokens"]
    if not case["ragged"]:
        return [most] * n
    least = max(1, most // 8)
    return [least + (977 + 40503 * s) % (most - least + 1) for s in range(n)]


def added(case):
    return [min(case["n_new"], v) for v in lengths(case)]


def padded(d):
    return 64 if d <= 64 else 128 if d <= 128 else 256


def header_bytes(d, n_kv):
    return -(-n_kv * (32 + 2 * padded(d)) // 128) * 128


def page_bytes(d, n_kv):
    return header_bytes(d, n_kv) + n_kv * 64 * padded(d)


def work(case):
    """Each input read once, each output written once; the products of scores and values."""
    d, n_kv, n_seq = case["d"], case["n_kv"], case["n_seq"]
    lens = lengths(case)
    code = 2 * d * n_kv                                   # key and value codes of one token
    if case["op"] == "append":
        width = 2 if case["dtype"] == "bf16" else 4
        new = sum(added(case))
        sealed = sum(v // BLOCK - (v - a) // BLOCK for v, a in zip(lens, added(case)))
        back = sum(min(v, window(case)) for v in lens)
        return {"bytes": new * code * width + sealed * n_kv * (BLOCK + 1) * 2 * d + back * code * 2, "flops": 0}
    if case["op"] == "evict":
        full = [v // BLOCK for v in lens]
        kept = sum(min(f, case["keep"]) * BLOCK for f in full)
        left = sum(min(f, case["keep"]) * BLOCK + v % BLOCK for f, v in zip(full, lens))
        return {"bytes": sum(lens) * n_kv * 4 + left * n_kv * 4 + kept * (2 * code + 4 * n_kv) + left * code * 2,
                "flops": 0}
    rows = case["g"] * case["n_q"] * n_kv
    io = n_seq * rows * d * ((2 if case["dtype"] == "bf16" else 4) + 4)
    if case["op"] == "sparse":
        full = [v // BLOCK for v in lens]
        seen = [min(f, case["n_sel"]) * BLOCK + v % BLOCK for f, v in zip(full, lens)]
        return {"bytes": io + sum(full) * n_kv * (2 * d + 4) + sum(seen) * code + n_seq * n_kv * case["n_sel"] * 4,
                "flops": 4 * rows * d * sum(seen) + 4 * rows * d * sum(full)}
    more = sum(lens) * n_kv * 8 if case["weights"] else 0
    return {"bytes": io + sum(lens) * code + more, "flops": 4 * rows * d * sum(lens)}


# ----------------------------------------------------------------------------- the cache's bytes, in torch
def swizzle(D, device):
    """Where byte i of token t's row lies: [32, D]."""
    t = torch.arange(BLOCK, device=device)[:, None]
    i = torch.arange(D, device=device)[None, :]
    s = ((t & 2) | (((t ^ (t >> 2)) & 1) << 2)) & (D // 16 - 1)
    return (((i // 16) ^ s) * 16 + i % 16)


def quantize_blocks(x):
    """x [..., 32, d] as fp32 -> codes (fp32 whole numbers) and scales [...]."""
    a = x.abs().amax(dim=(-1, -2))
    live = a >= 2.0 ** -100
    inv = torch.where(live, 127.0 / torch.where(live, a, 1.0), 0.0)
    code = (x.double() * inv.double()[..., None, None]).round().float()   # a product next to a border: exact in 64 bits
    return code, torch.where(live, a / 127.0, 0.0)


def to_bytes(kc, vc, ks, vs, D):
    """Codes [n, n_kv, 32, d] and scales [n, n_kv] -> pages [n, page bytes]."""
    n, n_kv, _, d = kc.shape
    dev = kc.device
    head = torch.zeros(n, n_kv, 32 + 2 * D, dtype=torch.uint8, device=dev)
    head[..., 0:4] = ks.reshape(-1).view(torch.uint8).view(n, n_kv, 4)
    head[..., 4:8] = vs.reshape(-1).view(torch.uint8).view(n, n_kv, 4)
    head[..., 32:32 + d] = kc.amin(dim=2).to(torch.int8).view(torch.uint8)
    head[..., 32 + D:32 + D + d] = kc.amax(dim=2).to(torch.int8).view(torch.uint8)
    rows = torch.full((n, n_kv, 2, BLOCK, D), 128, dtype=torch.uint8, device=dev)
    rows[:, :, 0, :, :d] = (kc + 128).to(torch.uint8)
    rows[:, :, 1, :, :d] = (vc + 128).to(torch.uint8)
    where = swizzle(D, dev).expand_as(rows)
    rows = torch.empty_like(rows).scatter_(-1, where, rows)
    out = torch.zeros(n, page_bytes(d, n_kv), dtype=torch.uint8, device=dev)
    out[:, :n_kv * (32 + 2 * D)] = head.view(n, -1)
    out[:, header_bytes(d, n_kv):] = rows.view(n, -1)
    return out


def from_bytes(pages, d, n_kv):
    """pages [n, page bytes] -> codes [n, n_kv, 2, 32, d] (fp32) and scales [n, n_kv, 2]."""
    D, n = padded(d), pages.shape[0]
    scales = pages[:, :n_kv * (32 + 2 * D)].reshape(n, n_kv, -1)[..., :8].contiguous().view(F32)
    rows = pages[:, header_bytes(d, n_kv):].reshape(n, n_kv, 2, BLOCK, D)
    codes = rows.gather(-1, swizzle(D, pages.device).expand_as(rows))[..., :d].to(F32) - 128.0
    return codes, scales


def summaries(pages, d, n_kv):
    """pages [n, page bytes] -> lo and hi codes [n, n_kv, d] (fp32) and key scales [n, n_kv]."""
    D, n = padded(d), pages.shape[0]
    head = pages[:, :n_kv * (32 + 2 * D)].reshape(n, n_kv, 32 + 2 * D)
    lohi = head[..., 32:].contiguous().view(torch.int8).view(n, n_kv, 2, D)[..., :d].to(F32)
    return lohi[:, :, 0], lohi[:, :, 1], head[..., :4].contiguous().view(F32)[..., 0]


def read_back(pages, table, length, open_, n_tok, k_out, v_out):
    """The last n_tok tokens of every sequence as values; rows before a sequence's first token stay."""
    n_seq, n_kv, _, _, d = open_.shape
    D, dev = padded(d), pages.device
    pos = length[:, None].long() - n_tok + torch.arange(n_tok, device=dev)
    blk, t = torch.div(pos, BLOCK, rounding_mode="floor"), pos % BLOCK
    name = table.gather(1, blk.clamp(0, table.shape[1] - 1)).long()
    body = pages[:, header_bytes(d, n_kv):].unflatten(1, (n_kv, 2, BLOCK, D))
    head = pages[:, :n_kv * (32 + 2 * D)].unflatten(1, (n_kv, 32 + 2 * D))
    scales = head[name][..., :8].contiguous().view(F32)                     # [n_seq, n_tok, n_kv, 2]
    row = swizzle(D, dev)[t][:, :, None, :].expand(-1, -1, n_kv, -1)
    s = torch.arange(n_seq, device=dev)[:, None]
    paged = (blk < (length // BLOCK)[:, None])[..., None, None]
    for side, out in enumerate((k_out, v_out)):
        code = body[name, :, side, t].gather(-1, row)[..., :d].to(F32) - 128.0
        x = torch.where(paged, code * scales[..., side, None], open_[s, :, side, t].to(F32))
        out.copy_(torch.where((pos >= 0)[..., None, None], x.to(out.dtype), out))


# ----------------------------------------------------------------------------- inputs
def window(case):
    """Tokens read back after an append: those that came, and all of a block that they filled."""
    return case["n_new"] + BLOCK - 1


def keys_and_values(gen, shape, dev):
    """Keys N(0, 1) with four outlier channels per head scaled by 20, values N(0, 1) (bf16)."""
    k = torch.randn(shape, generator=gen, device=dev)
    v = torch.randn(shape, generator=gen, device=dev)
    n_kv, d = shape[-2], shape[-1]
    chan = torch.rand(n_kv, d, generator=gen, device=dev).argsort(dim=1)[:, :4]
    boost = torch.ones(n_kv, d, device=dev).scatter_(1, chan, 20.0)
    return (k * boost).to(torch.bfloat16), v.to(torch.bfloat16)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 17)
    n_seq, n_kv, d = case["n_seq"], case["n_kv"], case["d"]
    lens = lengths(case)
    most = -(-max(lens) // BLOCK)
    spare = n_seq * most if case["op"] == "evict" else 0
    names = torch.randperm(n_seq * most + spare, generator=gen, device=dev).to(torch.int32)
    st = {"case": case, "lens": lens}
    st["length"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    st["table"] = names[:n_seq * most].view(n_seq, most).contiguous()
    pages = torch.zeros(names.numel() + 1, page_bytes(d, n_kv), dtype=torch.uint8, device=dev)
    open_ = torch.zeros(n_seq, n_kv, 2, BLOCK, d, dtype=torch.bfloat16, device=dev)
    for s in range(n_seq):                                  # a sequence's past, one sequence at a time
        k, v = keys_and_values(gen, (most * BLOCK, n_kv, d), dev)
        k, v = (x.view(most, BLOCK, n_kv, d).transpose(1, 2) for x in (k, v))
        (kc, ks), (vc, vs) = quantize_blocks(k.float()), quantize_blocks(v.float())
        pages[st["table"][s].long()] = to_bytes(kc, vc, ks, vs, padded(d))
        blk = (lens[s] - (added(case)[s] if case["op"] == "append" else 0)) // BLOCK
        if blk < most:
            open_[s, :, 0], open_[s, :, 1] = k[blk], v[blk]
    st["pages"], st["open"], st["open_before"] = pages, open_, open_.clone()
    if case["op"] == "append":
        k, v = keys_and_values(gen, (n_seq, case["n_new"], n_kv, d), dev)
        st["k"], st["v"] = (k, v) if case["dtype"] == "bf16" else (k.float(), v.float())
        st["add"] = torch.tensor(added(case), dtype=torch.int32, device=dev)
        back = (n_seq, window(case), n_kv, d)
    elif case["op"] == "evict":
        st["dst"] = names[n_seq * most:].view(n_seq, most).contiguous()
        st["acc"] = torch.randn(n_seq, n_kv, most * BLOCK, generator=gen, device=dev).mul_(2.5).exp_()
        st["acc_out"] = torch.zeros_like(st["acc"])
        st["kept"] = torch.zeros(n_seq, n_kv, case["keep"] * BLOCK, dtype=torch.int32, device=dev)
        st["length_out"] = torch.zeros_like(st["length"])
        back = (n_seq, max(min(v // BLOCK, case["keep"]) * BLOCK + v % BLOCK for v in lens), n_kv, d)
    else:
        q = torch.randn(n_seq, case["n_q"], n_kv * case["g"], d, generator=gen, device=dev)
        st["q"] = q.to(torch.bfloat16) if case["dtype"] == "bf16" else q
        st["out"] = torch.zeros(n_seq, case["n_q"], n_kv * case["g"], d, device=dev)
        if case["op"] == "sparse":
            st["sel"] = torch.zeros(n_seq, case["n_q"], n_kv, case["n_sel"], dtype=torch.int32, device=dev)
        elif case["weights"]:
            st["acc"] = torch.rand(n_seq, n_kv, most * BLOCK, generator=gen, device=dev)
            st["acc_out"] = torch.zeros_like(st["acc"])
        return st
    st["k_back"] = torch.zeros(back, dtype=torch.bfloat16, device=dev)
    st["v_back"] = torch.zeros(back, dtype=torch.bfloat16, device=dev)
    return st


# ----------------------------------------------------------------------------- the plain forms
def plain_append(st):
    k, v, open_, table, length, add = (st[n] for n in ("k", "v", "open", "table", "length", "add"))
    n_seq, n_kv, _, _, d = open_.shape
    n_new = k.shape[1]
    first = (length - add).long()
    b0 = first // BLOCK
    nb = (n_new + 2 * BLOCK - 2) // BLOCK
    pos = b0[:, None] * BLOCK + torch.arange(nb * BLOCK, device=k.device)       # positions of the blocks touched
    came = (pos >= first[:, None]) & (pos < length[:, None])
    s = torch.arange(n_seq, device=k.device)[:, None]
    src = (pos - first[:, None]).clamp(0, n_new - 1)
    x = []
    for side, new in enumerate((k, v)):
        old = open_[s, :, side, pos % BLOCK]
        x.append(torch.where(came[..., None, None], new.to(torch.bfloat16)[s, src], old)
                 .view(n_seq, nb, BLOCK, n_kv, d).transpose(2, 3))
    blk = b0[:, None] + torch.arange(nb, device=k.device)
    (kc, ks), (vc, vs) = quantize_blocks(x[0].float()), quantize_blocks(x[1].float())
    done = (blk + 1) * BLOCK <= length[:, None]
    page = table.gather(1, blk.clamp(max=table.shape[1] - 1)).long()
    rows = to_bytes(kc.flatten(0, 1), vc.flatten(0, 1), ks.flatten(0, 1), vs.flatten(0, 1), padded(d))
    spare = st["pages"].shape[0] - 1                         # blocks that are not full go to the page nobody has
    st["pages"][torch.where(done, page, spare).reshape(-1)] = rows
    now = (length // BLOCK).long() - b0                      # the block that is open afterwards
    fresh = torch.arange(BLOCK, device=k.device)[None, :] < (length % BLOCK)[:, None]
    after = torch.stack([y[s[:, 0], now.clamp(max=nb - 1)] for y in x], dim=2)
    open_.copy_(torch.where(fresh[:, None, None, :, None], after, open_))
    read_back(st["pages"], table, length, open_, st["k_back"].shape[1], st["k_back"], st["v_back"])
    return st["k_back"], st["v_back"]


def attend(q, k, v, seen, scale):
    """q [..., r, d], k and v [..., t, d], seen [..., r, t] -> outputs and weights, rows that see nothing zero."""
    score = (q @ k.transpose(-1, -2)) * scale
    score = torch.where(seen, score, -math.inf)
    top = score.amax(dim=-1, keepdim=True)
    e = torch.where(seen, (score - torch.where(top > -math.inf, top, 0.0)).exp(), 0.0)
    total = e.sum(dim=-1, keepdim=True)
    w = e / torch.where(total > 0, total, 1.0)
    return w @ v, w


def tokens_of(st, blocks):
    """The named blocks (by number, [n_seq, n_kv or 1, n]) of each sequence, then its open block:
    keys, values [n_seq, n_kv, 32 (n + 1), d] and their positions, -1 where there is no token."""
    open_, table, length, pages = (st[n] for n in ("open", "table", "length", "pages"))
    n_seq, n_kv, _, _, d = open_.shape
    full = (length // BLOCK).long()[:, None, None]
    there = (blocks >= 0) & (blocks < full)
    page = table[torch.arange(n_seq, device=pages.device)[:, None, None], blocks.clamp(0, table.shape[1] - 1)].long()
    n = blocks.shape[-1]
    if blocks.shape[1] == 1:
        codes, scales = from_bytes(pages[page.reshape(-1)], d, n_kv)
        codes = codes.view(n_seq, n, n_kv, 2, BLOCK, d).transpose(1, 2)
        scales = scales.view(n_seq, n, n_kv, 2).transpose(1, 2)
    else:
        D = padded(d)
        h = torch.arange(n_kv, device=pages.device)[None, :, None]
        body = pages[:, header_bytes(d, n_kv):].unflatten(1, (n_kv, 2, BLOCK, D))[page, h]
        codes = body.gather(-1, swizzle(D, pages.device).expand_as(body))[..., :d].to(F32) - 128.0
        head = pages[:, :n_kv * (32 + 2 * D)].unflatten(1, (n_kv, 32 + 2 * D))[..., :8][page, h]
        scales = head.contiguous().view(F32)
    x = codes * scales[..., None, None]
    pos = blocks[..., None] * BLOCK + torch.arange(BLOCK, device=pages.device)
    pos = torch.where(there[..., None], pos, -1).flatten(2).expand(n_seq, n_kv, -1)
    t = torch.arange(BLOCK, device=pages.device)
    tail = torch.where(t < (length % BLOCK)[:, None], full[:, 0] * BLOCK + t, -1)[:, None].expand(n_seq, n_kv, BLOCK)
    pos = torch.cat([pos, tail], dim=-1)
    k = torch.cat([x[:, :, :, 0].flatten(2, 3), open_[:, :, 0].to(F32)], dim=2)
    v = torch.cat([x[:, :, :, 1].flatten(2, 3), open_[:, :, 1].to(F32)], dim=2)
    v = torch.where((pos >= 0)[..., None], v, 0.0)
    return k, v, pos


def heads_of(q, n_kv):
    """q [n_seq, n_q, n_kv g, d] -> [n_seq, n_kv, n_q g, d] in fp32"""
    n_seq, n_q, n_h, d = q.shape
    return q.to(F32).view(n_seq, n_q, n_kv, n_h // n_kv, d).transpose(1, 2).flatten(2, 3)


def plain_attention(st):
    case, q, length = st["case"], st["q"], st["length"]
    n_seq, n_q, n_h, d = q.shape
    n_kv, g = case["n_kv"], case["g"]
    blocks = torch.arange(st["table"].shape[1], device=q.device).expand(n_seq, 1, -1)
    k, v, pos = tokens_of(st, blocks)
    mine = (length[:, None] - n_q + torch.arange(n_q, device=q.device)).repeat_interleave(g, dim=1)
    seen = (pos[:, :, None, :] >= 0) & (pos[:, :, None, :] <= mine[:, None, :, None])
    o, w = attend(heads_of(q, n_kv), k, v, seen, d ** -0.5)
    st["out"].copy_(o.view(n_seq, n_kv, n_q, g, d).transpose(1, 2).flatten(2, 3))
    if not case["weights"]:
        return st["out"]
    t = torch.arange(st["acc"].shape[-1], device=q.device)
    new = w.sum(dim=2)
    n_all = new.shape[-1] - BLOCK                            # open tokens come last: put them at their positions
    total = new[..., :n_all].clone()
    at = pos[..., n_all:]
    total.scatter_add_(2, at.clamp(min=0), torch.where(at >= 0, new[..., n_all:], 0.0))
    old = torch.where(t < (length - n_q)[:, None, None], st["acc"], 0.0)
    st["acc_out"].copy_(torch.where(t < length[:, None, None], old * 0.9 + total, st["acc_out"]))
    return st["out"], st["acc_out"]


def plain_select(st):
    q, length, table = st["q"], st["length"], st["table"]
    n_seq, n_q, n_h, d = q.shape
    n_kv, n_sel = st["case"]["n_kv"], st["sel"].shape[-1]
    lo, hi, ks = summaries(st["pages"][table.reshape(-1).long()], d, n_kv)
    nb = table.shape[1]
    lo, hi = (x.view(n_seq, nb, n_kv, d).transpose(1, 2) for x in (lo, hi))
    ks = ks.view(n_seq, nb, n_kv).transpose(1, 2)
    x = q[:, 0].to(F32).view(n_seq, n_kv, -1, d)
    a = x.abs().amax(dim=-1, keepdim=True)
    qi = (x.double() * (127.0 / a).double()).round().float()
    whole = qi.clamp(min=0) @ hi.transpose(-1, -2) + qi.clamp(max=0) @ lo.transpose(-1, -2)  # whole numbers below 2^24
    score = ((whole * ks[:, :, None, :]) * (a / 127.0)).amax(dim=2)
    b = torch.arange(nb, device=q.device)
    full = (length // BLOCK)[:, None, None]
    score = torch.where((b < 1) | (b >= full - 1), math.inf, score)
    score = torch.where(b < full, score, -math.inf)
    order = score.argsort(dim=-1, descending=True, stable=True)[..., :n_sel]
    order = torch.where(order < full, order, 1 << 30).sort(dim=-1).values
    order = torch.where(order < full, order, -1)
    st["sel"].fill_(-1)
    st["sel"][:, 0, :, :order.shape[-1]] = order.to(torch.int32)
    return st["sel"]


def plain_sparse(st):
    q = st["q"]
    n_seq, _, n_h, d = q.shape
    n_kv = st["case"]["n_kv"]
    sel = plain_select(st)
    k, v, pos = tokens_of(st, sel[:, 0].long())
    o, _ = attend(heads_of(q, n_kv), k, v, (pos >= 0)[:, :, None, :].expand(-1, -1, n_h // n_kv, -1), d ** -0.5)
    st["out"].copy_(o.reshape(n_seq, 1, n_h, d))
    return sel, st["out"]


def plain_evict(st):
    pages, table, length, open_, acc, dst = (st[n] for n in ("pages", "table", "length", "open", "acc", "dst"))
    n_seq, n_kv, _, _, d = open_.shape
    keep = st["case"]["keep"]
    most = min(keep, table.shape[1])
    full = (length // BLOCK).long()[:, None, None]
    t = torch.arange(acc.shape[-1], device=acc.device)
    key = torch.where((t < FIRST) | (t >= full * BLOCK - LAST), math.inf, acc.clamp(min=0))
    key = torch.where(t < full * BLOCK, key, -1.0)
    order = key.argsort(dim=-1, descending=True, stable=True)[..., :most * BLOCK]
    order = torch.where(order < full * BLOCK, order, 1 << 30).sort(dim=-1).values
    there = order < full * BLOCK
    st["kept"].fill_(-1)
    st["kept"][..., :most * BLOCK] = torch.where(there, order, -1).to(torch.int32)
    src = torch.where(there, order, 0)
    s = torch.arange(n_seq, device=acc.device)[:, None, None]
    h = torch.arange(n_kv, device=acc.device)[None, :, None]
    blk, row = src // BLOCK, src % BLOCK
    codes, scales = from_bytes(pages[table.reshape(-1).long()], d, n_kv)
    at = s * table.shape[1] + blk
    out = []
    for side in range(2):
        c = codes[at, h, side, row].view(n_seq, n_kv, most, BLOCK, d)
        sc = scales[at, h, side].view(n_seq, n_kv, most, BLOCK)
        live = there.view(n_seq, n_kv, most, BLOCK)
        top = (c.abs().amax(dim=-1) / 127.0) * sc
        new = torch.where(live, top, 0.0).amax(dim=-1)
        ratio = torch.where(new[..., None] > 0, sc / torch.where(new > 0, new, 1.0)[..., None], 0.0)
        out += [(c.double() * ratio.double()[..., None]).round().float(), new]
    rows = to_bytes(out[0].transpose(1, 2).flatten(0, 1), out[2].transpose(1, 2).flatten(0, 1),
                    out[1].transpose(1, 2).flatten(0, 1), out[3].transpose(1, 2).flatten(0, 1), padded(d))
    live = torch.arange(most, device=acc.device) < full[:, 0]
    pages[torch.where(live, dst[:, :most].long(), pages.shape[0] - 1).reshape(-1)] = rows
    left = full.clamp(max=keep) * BLOCK
    st["length_out"].copy_((left[:, 0, 0] + length % BLOCK).to(torch.int32))
    gone = full * BLOCK - left
    moved = torch.where(t < left, torch.cat([src, src.new_zeros(n_seq, n_kv, acc.shape[-1] - src.shape[-1])], -1),
                        (t + gone).clamp(max=acc.shape[-1] - 1))
    st["acc_out"].copy_(torch.where(t < st["length_out"][:, None, None], acc.gather(2, moved), st["acc_out"]))
    read_back(pages, dst, st["length_out"], open_, st["k_back"].shape[1], st["k_back"], st["v_back"])
    return st["kept"], st["length_out"], st["acc_out"], st["k_back"], st["v_back"]


FIRST, LAST = 4, 128    # tokens that eviction never takes: the first ones, the most recent ones


# ----------------------------------------------------------------------------- one pass
def handles(st):
    """The cache and a workspace, as a program keeps them for its session."""
    import kv_cache_vector_03_b200 as tq
    if "cache" not in st:
        case = st["case"]
        st["tq"] = tq
        st["cache"] = tq.Cache8(case["d"], st["pages"], st["table"], st["length"], st["open"])
        need = 0
        if case["op"] == "evict":
            st["after"] = tq.Cache8(case["d"], st["pages"], st["dst"], st["length_out"], st["open"])
        if case["op"] in ("attention", "sparse"):
            need = tq.tq_b8_workspace_bytes(st["cache"], case["n_q"], case["g"], case.get("n_sel", 0))
        st["ws"] = tq.workspace(max(need, tq.tq_b8_workspace_bytes(st["cache"])))
    return tq


def run(state):
    st, op = state, state["case"]["op"]
    if op == "append" and st["case"]["n_new"] > 1:
        st["open"].copy_(st["open_before"])     # tokens of a block that filled up give way to later ones
    if own:
        tq = handles(st)
        if op == "append":
            tq.tq_b8_append(st["cache"], st["k"], st["v"], st["ws"], add=st["add"])
            tq.tq_b8_read(st["cache"], st["k_back"], st["v_back"], st["ws"])
            return st["k_back"], st["v_back"]
        if op == "evict":
            tq.tq_b8_evict(st["cache"], st["acc"], st["case"]["keep"], st["dst"], st["kept"], st["length_out"],
                           st["acc_out"], st["ws"], n_first=FIRST, n_last=LAST)
            tq.tq_b8_read(st["after"], st["k_back"], st["v_back"], st["ws"])
            return st["kept"], st["length_out"], st["acc_out"], st["k_back"], st["v_back"]
        scale = st["case"]["d"] ** -0.5
        if op == "sparse":
            tq.tq_b8_select(st["cache"], st["q"], st["sel"], st["ws"], n_first=1, n_last=1)
            tq.tq_b8_attention(st["cache"], st["q"], scale, st["out"], st["ws"], sel=st["sel"])
            return st["sel"], st["out"]
        if st["case"]["weights"]:
            tq.tq_b8_attention(st["cache"], st["q"], scale, st["out"], st["ws"], acc_in=st["acc"],
                               acc_out=st["acc_out"], decay=0.9)
            return st["out"], st["acc_out"]
        tq.tq_b8_attention(st["cache"], st["q"], scale, st["out"], st["ws"])
        return st["out"]
    return {"append": plain_append, "attention": plain_attention, "sparse": plain_sparse,
            "evict": plain_evict}[op](st)


# ----------------------------------------------------------------------------- the definitions in 64 bits
def byte_at(pages, name, h, side, t, i, d, n_kv):
    """Address of a code in the pool: page `name`, kv head h, keys (0) or values (1), token t, channel i."""
    D = padded(d)
    turn = (t % 4) // 2 * 2 + (t + t // 4) % 2 * 4
    turn = turn % (D // 16)
    chunk = torch.bitwise_xor(i // 16, turn)
    return name * pages.shape[1] + header_bytes(d, n_kv) + ((h * 2 + side) * BLOCK + t) * D + chunk * 16 + i % 16


def scale_at(pages, name, h, side, d):
    at = name * pages.shape[1] + h * (32 + 2 * padded(d)) + 4 * side
    b = torch.stack([pages.view(-1)[at + j].to(torch.int64) << (8 * j) for j in range(4)]).sum(0)
    return b.to(torch.int32).view(F32).double()


def sequence(st, s, table=None, blocks=None):
    """Keys and values of sequence s in 64 bits, [n_kv, tokens, d], of its full blocks (or those named)."""
    pages, d, n_kv = st["pages"], st["case"]["d"], st["case"]["n_kv"]
    dev = pages.device
    table = st["table"] if table is None else table
    nb = st["lens"][s] // BLOCK if blocks is None else blocks
    h = torch.arange(n_kv, device=dev)[:, None, None, None]
    name = table[s, :nb].long()[None, :, None, None]
    t = torch.arange(BLOCK, device=dev)[None, None, :, None]
    i = torch.arange(d, device=dev)[None, None, None, :]
    out = []
    for side in range(2):
        code = pages.view(-1)[byte_at(pages, name, h, side, t, i, d, n_kv)].double() - 128
        out.append((code * scale_at(pages, name, h, side, d)).reshape(n_kv, nb * BLOCK, d))
    return out


def with_open(st, s, k, v):
    r = st["lens"][s] % BLOCK
    return (torch.cat([k, st["open"][s, :, 0, :r].double()], 1), torch.cat([v, st["open"][s, :, 1, :r].double()], 1))


def exact_attention(case, st):
    n_q, g, n_kv, d = case["n_q"], case["g"], case["n_kv"], case["d"]
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    acc = st["acc_out"].double().clone() if case["weights"] else None
    for s, n in enumerate(st["lens"]):
        k, v = with_open(st, s, *sequence(st, s))
        weight = torch.zeros(n_kv, n, dtype=torch.float64, device="cuda")
        for j in range(n_q):
            last = n - n_q + j
            if last < 0:
                continue
            for h in range(n_kv):
                q = st["q"][s, j, h * g:(h + 1) * g].double()
                w = torch.softmax(q @ k[h, :last + 1].T / math.sqrt(d), dim=-1)
                out[s, j, h * g:(h + 1) * g] = w @ v[h, :last + 1]
                weight[h, :last + 1] += w.sum(0)
        if acc is not None:
            old = max(0, n - n_q)
            weight[:, :old] += 0.9 * st["acc"][s, :, :old].double()
            acc[s, :, :n] = weight
    return out if acc is None else (out, acc)


def exact_sparse(case, st):
    g, n_kv, d = case["g"], case["n_kv"], case["d"]
    D = padded(d)
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    pages = st["pages"]
    entry = 32 + 2 * D
    i = torch.arange(d, device="cuda")
    for s, n in enumerate(st["lens"]):
        nb = n // BLOCK
        name = st["table"][s, :nb].long()
        k, v = sequence(st, s)
        r = n % BLOCK
        for h in range(n_kv):
            base = (name * pages.shape[1] + h * entry + 32)[:, None] + i
            lo = pages.view(-1)[base].view(torch.int8).double()
            hi = pages.view(-1)[base + D].view(torch.int8).double()
            ks = scale_at(pages, name, torch.tensor(h, device="cuda"), 0, d)
            q = st["q"][s, 0, h * g:(h + 1) * g].double()
            # the score is whole numbers and three fp32 roundings by definition: the choice is discrete
            top = q.abs().amax(dim=1, keepdim=True).float()
            qi = (q * (127 / top).double()).round()
            best = torch.full((nb,), -math.inf, device="cuda")
            for m in range(g):
                whole = torch.maximum(qi[m] * lo, qi[m] * hi).sum(1).float()
                best = torch.maximum(best, whole * ks.float() * (top[m] / 127))
            if nb:
                best[0] = best[-1] = math.inf
            take = torch.sort(best, descending=True, stable=True).indices[:case["n_sel"]].sort().values
            at = (take[:, None] * BLOCK + torch.arange(BLOCK, device="cuda")).reshape(-1)
            kk = torch.cat([k[h, at], st["open"][s, h, 0, :r].double()])
            vv = torch.cat([v[h, at], st["open"][s, h, 1, :r].double()])
            if kk.shape[0]:
                out[s, 0, h * g:(h + 1) * g] = torch.softmax(q @ kk.T / math.sqrt(d), dim=-1) @ vv
    return None, out


def block64(x):
    """[n_kv, 32 n, d] as the cache gives it back: one scale for 32 tokens of a head."""
    n_kv, n, d = x.shape
    x = x.reshape(n_kv, n // BLOCK, BLOCK * d)
    a = x.abs().amax(dim=-1, keepdim=True)
    a = torch.where(a > 0, a, 1.0)
    return ((x * 127 / a).round() * a / 127).reshape(n_kv, n, d)


def exact_append(case, st):
    wide = window(case)
    backs = [torch.zeros(st["k_back"].shape, dtype=torch.float64, device="cuda") for _ in range(2)]
    for s, n in enumerate(st["lens"]):
        a = added(case)[s]
        b0 = (n - a) // BLOCK
        past = sequence(st, s, blocks=b0)
        for side, new in enumerate((st["k"], st["v"])):
            held = st["open"][s, :, side, :(n - a) % BLOCK].double()
            x = torch.cat([held, new[s, :a].to(torch.bfloat16).double().transpose(0, 1)], dim=1)
            m = x.shape[1] // BLOCK * BLOCK
            if m:
                x = torch.cat([block64(x[:, :m]), x[:, m:]], dim=1)
            x = torch.cat([past[side], x], dim=1)
            w = min(n, wide)
            backs[side][s, wide - w:] = x[:, n - w:].transpose(0, 1)
    return tuple(backs)


def moved64(code, scale):
    """Codes [32 n, d] with a scale for each token as the new blocks give them back. The scales and
    their ratios are fp32 by the format's definition; half of all ties would else fall by chance."""
    top = code.abs().amax(dim=1).float() / 127 * scale.float()
    new = top.reshape(-1, BLOCK).amax(dim=1, keepdim=True).expand(-1, BLOCK).reshape(-1)
    ratio = torch.where(new > 0, scale.float() / new, 0.0)
    return (code * ratio.double()[:, None]).round() * new.double()[:, None]


def exact_evict(case, st):
    keep, n_kv, d = case["keep"], case["n_kv"], case["d"]
    backs = [torch.zeros(st["k_back"].shape, dtype=torch.float64, device="cuda") for _ in range(2)]
    acc = torch.zeros(st["acc"].shape, dtype=torch.float64, device="cuda")
    wide, pages = st["k_back"].shape[1], st["pages"]
    i = torch.arange(d, device="cuda")[None, :]
    for s, n in enumerate(st["lens"]):
        nb, r = n // BLOCK, n % BLOCK
        left = min(nb, keep) * BLOCK
        for h in range(n_kv):
            rank = st["acc"][s, h, :nb * BLOCK].double().clone()
            rank[:FIRST] = math.inf
            rank[max(0, nb * BLOCK - LAST):] = math.inf
            take = torch.sort(rank, descending=True, stable=True).indices[:left].sort().values
            acc[s, h, :left] = st["acc"][s, h, take].double()
            name = st["table"][s, take // BLOCK].long()
            head = torch.tensor(h, device="cuda")
            for side in range(2):
                at = byte_at(pages, name[:, None], head, side, (take % BLOCK)[:, None], i, d, n_kv)
                x = moved64(pages.view(-1)[at].double() - 128, scale_at(pages, name, head, side, d))
                backs[side][s, wide - left - r:, h] = torch.cat([x, st["open"][s, h, side, :r].double()])
        acc[s, :, left:left + r] = st["acc"][s, :, nb * BLOCK:n].double()
    return None, None, acc, backs[0], backs[1]


def exact(case, seed):
    st = prepare(case, seed)
    return {"append": exact_append, "attention": exact_attention, "sparse": exact_sparse,
            "evict": exact_evict}[case["op"]](case, st)
