"""Python binding of libtq, the TurboQuant KV-vector hot path for B200 (sm_100a).

Argument marshalling only: every function forwards torch device pointers and sizes to the
C ABI in include/tq.h; all arithmetic runs in the CUDA library. PyTorch provides device
memory and streams. Importing this package fails loudly if libtq.so has not been built
(run ``python kv_cache_vector_03_b200/build.py`` or ``__graft_entry__.build()``).
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtq.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"libtq.so is missing at {LIB_PATH}: build it with python kv_cache_vector_03_b200/build.py")

lib = ctypes.CDLL(LIB_PATH)

TQ_OK, TQ_ERR_ARG, TQ_ERR_UNSUPPORTED, TQ_ERR_CUDA = 0, -1, -2, -3
TQ_ERR_RANGE, TQ_ERR_TIMEOUT, TQ_ERR_NOCONV, TQ_ERR_WORKSPACE = -4, -5, -6, -7
TQ_F32, TQ_BF16 = 0, 1
TQ_OP_QUANTIZE, TQ_OP_LOGITS, TQ_OP_PV, TQ_OP_TOPK, TQ_OP_DEQUANTIZE = 0, 1, 2, 3, 4
TQ_EST_QJL, TQ_EST_MSE = 0, 1
TQ_TEST_STALL = 0x100   # test hook: see include/tq.h
EXPORTED = ["tq_make_codebook", "tq_block_bytes", "tq_record_bytes", "tq_packed_bytes", "tq_prep_bytes",
            "tq_prepare", "tq_workspace_bytes", "tq_quantize", "tq_logits", "tq_pv", "tq_topk",
            "tq_dequantize", "tq_reset_status", "tq_get_status", "tq_status_string", "tq_abi_version",
            "tq_logits_noalloc", "tq_attention", "tq_attention_workspace_bytes", "tq_logits_est", "tq_topk_est",
            "tq_q8_packed_bytes", "tq_q8_quantize", "tq_q8_logits", "tq_attention_q8",
            "tq_attention_q8_workspace_bytes", "tq_b8_page_bytes", "tq_b8_workspace_bytes", "tq_b8_append",
            "tq_b8_read", "tq_b8_attention", "tq_b8_select", "tq_b8_evict"]
TQ_B8_BLOCK = 32


class tq_codec(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int), ("m", ctypes.c_int), ("mse_bits", ctypes.c_int), ("qjl", ctypes.c_int),
                ("pi", ctypes.c_void_p), ("s", ctypes.c_void_p), ("centroids", ctypes.c_void_p),
                ("prep", ctypes.c_void_p), ("prep_bytes", ctypes.c_size_t)]


class tq_b8_cache(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int), ("n_kv", ctypes.c_int), ("n_seq", ctypes.c_int64), ("n_pages", ctypes.c_int64),
                ("max_blocks", ctypes.c_int64), ("pages", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("len", ctypes.c_void_p), ("open", ctypes.c_void_p)]


_P, _I, _I64, _SZ, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
_CP = ctypes.POINTER(tq_codec)
_BP = ctypes.POINTER(tq_b8_cache)
_sig = {
    "tq_make_codebook": (_I, [_I, _I, _P, _P, _P]),
    "tq_block_bytes": (_SZ, [_CP]),
    "tq_record_bytes": (_SZ, [_CP]),
    "tq_packed_bytes": (_SZ, [_CP, _I64, _I64]),
    "tq_prep_bytes": (_SZ, [_CP]),
    "tq_prepare": (_I, [_CP, _P]),
    "tq_workspace_bytes": (_SZ, [_CP, _I, _I64, _I64, _I64]),
    "tq_quantize": (_I, [_CP, _P, _I, _I64, _I64, _I64, _P, _P, _SZ, _P]),
    "tq_logits": (_I, [_CP, _P, _I64, _I, _I64, _P, _I, _I, _P, _I, _F, _P, _P, _SZ, _P]),
    "tq_logits_noalloc": (_I, [_CP, _P, _I64, _I, _I64, _P, _I, _I, _P, _I, _F, _P, _P]),
    "tq_pv": (_I, [_CP, _P, _I64, _I, _I64, _P, _I, _P, _P, _SZ, _P]),
    "tq_attention_workspace_bytes": (_SZ, [_CP, _CP, _I64, _I, _I64, _I, _I]),
    "tq_attention": (_I, [_CP, _CP, _P, _P, _I64, _I, _I64, _P, _I, _I, _P, _P, _I, _F, _F, _P, _P, _SZ, _P]),
    "tq_attention_q8_workspace_bytes": (_SZ, [_CP, _I64, _I, _I64, _I, _I]),
    "tq_attention_q8": (_I, [_CP, _P, _P, _I64, _I, _I64, _P, _I, _I, _P, _P, _I, _F, _F, _P, _P, _SZ, _P]),
    "tq_topk": (_I, [_CP, _P, _I64, _P, _I64, _I, _P, _P, _P, _SZ, _P]),
    "tq_logits_est": (_I, [_CP, _P, _I64, _I, _I64, _P, _I, _I, _P, _I, _F, _P, _P, _SZ, _I, _P]),
    "tq_q8_packed_bytes": (_SZ, [_I, _I64, _I64]),
    "tq_q8_quantize": (_I, [_P, _I, _I, _I64, _I64, _I64, _P, _P, _SZ, _P]),
    "tq_q8_logits": (_I, [_P, _I, _I64, _I, _I64, _P, _I, _I, _P, _I, _F, _P, _P]),
    "tq_topk_est": (_I, [_CP, _P, _I64, _P, _I64, _I, _P, _P, _P, _SZ, _I, _P]),
    "tq_dequantize": (_I, [_CP, _P, _I64, _I64, _P, _P, _SZ, _P]),
    "tq_b8_page_bytes": (_SZ, [_I, _I]),
    "tq_b8_workspace_bytes": (_SZ, [_BP, _I, _I, _I, _I]),
    "tq_b8_append": (_I, [_BP, _P, _P, _I, _I64, _I64, _I64, _P, _P, _SZ, _P]),
    "tq_b8_read": (_I, [_BP, _I64, _P, _P, _I, _P, _SZ, _P]),
    "tq_b8_attention": (_I, [_BP, _P, _I, _I, _I, _F, _P, _I, _P, _P, _F, _P, _P, _SZ, _P]),
    "tq_b8_select": (_I, [_BP, _P, _I, _I, _I, _I, _I, _I, _P, _P, _SZ, _P]),
    "tq_b8_evict": (_I, [_BP, _P, _I64, _I64, _I64, _P, _P, _P, _P, _P, _SZ, _P]),
    "tq_reset_status": (_I, [_P, _P]),
    "tq_get_status": (_I, [_P, _P]),
    "tq_status_string": (ctypes.c_char_p, [_I]),
    "tq_abi_version": (_I, []),
}
for _name, (_res, _args) in _sig.items():
    _fn = getattr(lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


class TQError(RuntimeError):
    def __init__(self, fn, status):
        super().__init__(f"{fn} -> {status} ({lib.tq_status_string(status).decode()})")
        self.status = status


def _check(fn, st):
    if st != TQ_OK:
        raise TQError(fn, st)
    return st


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype(t):
    import torch
    if t.dtype == torch.float32:
        return TQ_F32
    if t.dtype == torch.bfloat16:
        return TQ_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


# ----------------------------------------------------------------------------- API
def tq_make_codebook(d: int, mse_bits: int):
    """Host Lloyd-Max codebook: (centroids, bounds, normalised mse) as fp64 numpy arrays."""
    nl = 1 << mse_bits
    c = np.zeros(nl)
    t = np.zeros(nl - 1)
    mse = ctypes.c_double()
    _check("tq_make_codebook", lib.tq_make_codebook(d, mse_bits, c.ctypes.data, t.ctypes.data, ctypes.byref(mse)))
    return c, t, mse.value


class Codec:
    """A tq_codec with its device matrices and prepared operands (kept alive here)."""

    def __init__(self, d, m, mse_bits, qjl, pi, s, centroids=None, stream=None):
        import torch
        self.pi = pi.to(device="cuda", dtype=torch.float32).contiguous()
        self.s = s.to(device="cuda", dtype=torch.float32).contiguous() if qjl else None
        if centroids is None:
            centroids = tq_make_codebook(d, mse_bits)[0]
        self.centroids = np.ascontiguousarray(centroids, dtype=np.float64)
        self.c = tq_codec(d, m if qjl else 0, mse_bits, int(qjl), self.pi.data_ptr(),
                          self.s.data_ptr() if qjl else None, self.centroids.ctypes.data, None, 0)
        nprep = lib.tq_prep_bytes(ctypes.byref(self.c))
        if nprep == 0:
            raise TQError("tq_prep_bytes", TQ_ERR_UNSUPPORTED)
        self.prep = torch.empty(nprep, dtype=torch.uint8, device="cuda")
        self.c.prep = self.prep.data_ptr()
        self.c.prep_bytes = nprep
        _check("tq_prepare", lib.tq_prepare(ctypes.byref(self.c), _stream(stream)))

    @property
    def ref(self):
        return ctypes.byref(self.c)

    def block_bytes(self):
        return lib.tq_block_bytes(self.ref)

    def record_bytes(self):
        return lib.tq_record_bytes(self.ref)

    def packed_bytes(self, n_streams, n_tok):
        return lib.tq_packed_bytes(self.ref, n_streams, n_tok)

    def workspace_bytes(self, op, a=0, b=0, c=0):
        return lib.tq_workspace_bytes(self.ref, op, a, b, c)


def workspace(nbytes):
    import torch
    ws = torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device="cuda")
    return ws


def tq_quantize(codec: Codec, x, n_streams, n_tok, x_stream_stride, packed, ws, stream=None):
    return _check("tq_quantize", lib.tq_quantize(codec.ref, _ptr(x), _dtype(x), n_streams, n_tok, x_stream_stride,
                                                 _ptr(packed), _ptr(ws), ws.numel(), _stream(stream)))


def tq_logits(codec: Codec, packed, n_seq, n_kv, n_tok, q, g, tail, n_tail, scale, out, ws, stream=None,
              estimator=None):
    if estimator is None:
        return _check("tq_logits", lib.tq_logits(codec.ref, _ptr(packed), n_seq, n_kv, n_tok, _ptr(q), _dtype(q), g,
                                                 _ptr(tail), n_tail, scale, _ptr(out), _ptr(ws), ws.numel(),
                                                 _stream(stream)))
    return _check("tq_logits_est", lib.tq_logits_est(codec.ref, _ptr(packed), n_seq, n_kv, n_tok, _ptr(q), _dtype(q),
                                                     g, _ptr(tail), n_tail, scale, _ptr(out), _ptr(ws), ws.numel(),
                                                     estimator, _stream(stream)))


def tq_logits_noalloc(codec: Codec, packed, n_seq, n_kv, n_tok, q, g, tail, n_tail, scale, out, stream=None):
    """tq_logits with the library's fixed device scratch instead of a caller workspace."""
    return _check("tq_logits_noalloc", lib.tq_logits_noalloc(codec.ref, _ptr(packed), n_seq, n_kv, n_tok, _ptr(q),
                                                             _dtype(q), g, _ptr(tail), n_tail, scale, _ptr(out),
                                                             _stream(stream)))


def tq_pv(codec: Codec, packed_v, n_seq, n_kv, n_tok, P, g, out, ws, stream=None):
    return _check("tq_pv", lib.tq_pv(codec.ref, _ptr(packed_v), n_seq, n_kv, n_tok, _ptr(P), g, _ptr(out), _ptr(ws),
                                     ws.numel(), _stream(stream)))


def tq_attention_workspace_bytes(kcodec: Codec, vcodec: Codec, n_seq, n_kv, n_tok, g, n_tail):
    return lib.tq_attention_workspace_bytes(kcodec.ref, vcodec.ref, n_seq, n_kv, n_tok, g, n_tail)


def tq_attention(kcodec: Codec, vcodec: Codec, packed_k, packed_v, n_seq, n_kv, n_tok, q, g, tail_k, tail_v, n_tail,
                 scale, out, ws, v_skip=0.0, stream=None):
    return _check("tq_attention", lib.tq_attention(kcodec.ref, vcodec.ref, _ptr(packed_k), _ptr(packed_v), n_seq, n_kv,
                                                   n_tok, _ptr(q), _dtype(q), g, _ptr(tail_k), _ptr(tail_v), n_tail,
                                                   scale, v_skip, _ptr(out), _ptr(ws), ws.numel(), _stream(stream)))


def tq_attention_q8_workspace_bytes(vcodec: Codec, n_seq, n_kv, n_tok, g, n_tail):
    return lib.tq_attention_q8_workspace_bytes(vcodec.ref, n_seq, n_kv, n_tok, g, n_tail)


def tq_attention_q8(vcodec: Codec, packed_k8, packed_v, n_seq, n_kv, n_tok, q, g, tail_k, tail_v, n_tail, scale, out,
                    ws, v_skip=0.0, stream=None):
    return _check("tq_attention_q8", lib.tq_attention_q8(vcodec.ref, _ptr(packed_k8), _ptr(packed_v), n_seq, n_kv,
                                                         n_tok, _ptr(q), _dtype(q), g, _ptr(tail_k), _ptr(tail_v),
                                                         n_tail, scale, v_skip, _ptr(out), _ptr(ws), ws.numel(),
                                                         _stream(stream)))


def tq_topk(codec: Codec, packed_db, n_db, q, n_q, k, idx, score, ws, stream=None, estimator=None):
    if estimator is None:
        return _check("tq_topk", lib.tq_topk(codec.ref, _ptr(packed_db), n_db, _ptr(q), n_q, k, _ptr(idx),
                                             _ptr(score), _ptr(ws), ws.numel(), _stream(stream)))
    return _check("tq_topk_est", lib.tq_topk_est(codec.ref, _ptr(packed_db), n_db, _ptr(q), n_q, k, _ptr(idx),
                                                 _ptr(score), _ptr(ws), ws.numel(), estimator, _stream(stream)))


def tq_q8_packed_bytes(d, n_streams, n_tok):
    return lib.tq_q8_packed_bytes(d, n_streams, n_tok)


def tq_q8_quantize(x, d, n_streams, n_tok, x_stream_stride, packed, ws, stream=None):
    return _check("tq_q8_quantize", lib.tq_q8_quantize(_ptr(x), _dtype(x), d, n_streams, n_tok, x_stream_stride,
                                                       _ptr(packed), _ptr(ws), ws.numel(), _stream(stream)))


def tq_q8_logits(packed, d, n_seq, n_kv, n_tok, q, g, tail, n_tail, scale, out, stream=None):
    return _check("tq_q8_logits", lib.tq_q8_logits(_ptr(packed), d, n_seq, n_kv, n_tok, _ptr(q), _dtype(q), g,
                                                   _ptr(tail), n_tail, scale, _ptr(out), _stream(stream)))


def tq_b8_page_bytes(d, n_kv):
    return lib.tq_b8_page_bytes(d, n_kv)


class Cache8:
    """A tq_b8_cache over the caller's tensors (kept alive here, all on one GPU).

    pages uint8 [n_pages, tq_b8_page_bytes(d, n_kv)], table int32 [n_seq, max_blocks], length int32
    [n_seq], open_ bf16 [n_seq, n_kv, 2, 32, d]. Their contents may change between calls."""

    def __init__(self, d, pages, table, length, open_):
        import torch
        self.f32, self.i32, self.u8 = torch.float32, torch.int32, torch.uint8
        self.dtypes = {torch.float32: TQ_F32, torch.bfloat16: TQ_BF16}
        self.getters = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
        if open_.dim() != 5 or open_.shape[2:] != (2, TQ_B8_BLOCK, d):
            raise ValueError(f"open_ is [n_seq, n_kv, 2, {TQ_B8_BLOCK}, {d}]: got {tuple(open_.shape)}")
        n_seq, n_kv = open_.shape[:2]
        nbytes = lib.tq_b8_page_bytes(d, n_kv)
        if nbytes == 0:
            raise TQError("tq_b8_page_bytes", TQ_ERR_UNSUPPORTED)
        if pages.dim() != 2 or table.dim() != 2:
            raise ValueError("pages is [n_pages, page bytes], table is [n_seq, max_blocks]")
        self.d, self.n_kv, self.n_seq, self.max_blocks = d, n_kv, n_seq, table.shape[1]
        self.index = pages.get_device()           # -1 on the CPU, where no call is made
        self.row = (n_seq, n_kv, TQ_B8_BLOCK * self.max_blocks)
        self.c = tq_b8_cache(d, n_kv, n_seq, pages.shape[0], self.max_blocks,
                             _tensor(self, "pages", pages, torch.uint8, (pages.shape[0], nbytes)),
                             _tensor(self, "table", table, torch.int32, (n_seq, self.max_blocks)),
                             _tensor(self, "length", length, torch.int32, (n_seq,)),
                             _tensor(self, "open_", open_, torch.bfloat16, open_.shape))
        self.pages, self.table, self.length, self.open_ = pages, table, length, open_
        self.ref = ctypes.byref(self.c)


def _tensor(cache, name, t, dtype, shape):
    """t's address, after the checks that a wrong tensor would fail silently."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == cache.index and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{name}: {dtype} wanted, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(shape)} wanted, got {tuple(t.shape)}")
    if t.get_device() != cache.index:
        raise ValueError(f"{name} is on device {t.get_device()}, the cache on {cache.index}")
    raise ValueError(f"{name}: a contiguous tensor is wanted")


def _b8_dtype(cache, t):
    dt = cache.dtypes.get(t.dtype)
    if dt is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return dt


def _b8_call(name, fn, cache, ws, stream, *args):
    """Enqueues fn(cache, *args, ws, stream) on the cache's GPU."""
    dev = cache.index
    if dev < 0 or ws.get_device() != dev or ws.dtype is not cache.u8 or not ws.is_contiguous():
        raise ValueError(f"ws is a contiguous uint8 tensor on the cache's GPU ({dev}): got {ws.dtype} on {ws.device}")
    raw, here = cache.getters
    if stream is None:
        stream = raw(dev)
    else:
        if stream.device.index != dev:
            raise ValueError(f"the stream is on {stream.device}, the cache on GPU {dev}")
        stream = stream.cuda_stream
    if here() == dev:
        st = fn(cache.ref, *args, ws.data_ptr(), ws.numel(), stream)
    else:
        import torch
        with torch.cuda.device(dev):
            st = fn(cache.ref, *args, ws.data_ptr(), ws.numel(), stream)
    if st != TQ_OK:
        raise TQError(name, st)
    return st


def _queries(cache, q):
    shape = q.shape
    if len(shape) != 4 or shape[2] % cache.n_kv:
        raise ValueError(f"q is [n_seq, n_q, n_kv * g, d] with n_kv = {cache.n_kv}: got {tuple(shape)}")
    n_q, n_h = shape[1], shape[2]
    return (_tensor(cache, "q", q, q.dtype, (cache.n_seq, n_q, n_h, cache.d)), _b8_dtype(cache, q), n_q,
            n_h // cache.n_kv)


def _selection(cache, sel, n_q):
    n_sel = sel.shape[-1] if sel.dim() else 0
    if n_sel == 0:
        raise ValueError(f"sel is [n_seq, n_q, n_kv, n_sel] with n_sel >= 1: got {tuple(sel.shape)}")
    return _tensor(cache, "sel", sel, cache.i32, (cache.n_seq, n_q, cache.n_kv, n_sel)), n_sel


def tq_b8_workspace_bytes(cache, n_q=0, g=0, n_sel=0, weights=True):
    n = lib.tq_b8_workspace_bytes(cache.ref, n_q, g, n_sel, int(weights))
    if n == 0:
        raise TQError("tq_b8_workspace_bytes", TQ_ERR_UNSUPPORTED)
    return n


def tq_b8_append(cache, k, v, ws, add=None, stream=None):
    """k, v [n_seq, n_new, n_kv, d] (views with other sequence and token strides too); cache.length counts them."""
    n_seq, n_kv, d, dev = cache.n_seq, cache.n_kv, cache.d, cache.index
    n_new = k.shape[1] if k.dim() == 4 else -1
    shape = (n_seq, n_new, n_kv, d)
    if not (k.shape == shape and v.shape == shape and k.dtype is v.dtype):
        raise ValueError(f"k, v: shape {shape} and one type wanted, got {tuple(k.shape)} and {tuple(v.shape)}, "
                         f"{k.dtype} and {v.dtype}")
    if k.get_device() != dev or v.get_device() != dev:
        raise ValueError(f"k and v are on devices {k.get_device()} and {v.get_device()}, the cache on {dev}")
    ks, vs = k.stride(), v.stride()
    if n_new and n_seq and (ks[3] != 1 or vs[3] != 1 or (n_kv > 1 and (ks[2] != d or vs[2] != d))):
        raise ValueError(f"k, v: heads and channels lie next to each other, got strides {ks} and {vs}")
    seq, tok = (ks[0] if n_seq > 1 else 0), (ks[1] if n_new > 1 else 0)
    if ks != vs and ((n_seq > 1 and vs[0] != seq) or (n_new > 1 and vs[1] != tok)):
        raise ValueError(f"k and v have other strides: {ks}, {vs}")
    counts = None if add is None else _tensor(cache, "add", add, cache.i32, (cache.n_seq,))
    return _b8_call("tq_b8_append", lib.tq_b8_append, cache, ws, stream, k.data_ptr(), v.data_ptr(),
                    _b8_dtype(cache, k), n_new, seq, tok, counts)


def tq_b8_read(cache, k, v, ws, stream=None):
    """The last n_tok tokens of every sequence into k, v [n_seq, n_tok, n_kv, d] (fp32 or bf16)."""
    shape = (cache.n_seq, k.shape[1] if k.dim() == 4 else -1, cache.n_kv, cache.d)
    return _b8_call("tq_b8_read", lib.tq_b8_read, cache, ws, stream, shape[1], _tensor(cache, "k", k, k.dtype, shape),
                    _tensor(cache, "v", v, k.dtype, shape), _b8_dtype(cache, k))


def tq_b8_attention(cache, q, scale, out, ws, sel=None, acc_in=None, acc_out=None, decay=1.0, stream=None):
    """q [n_seq, n_q, n_kv * g, d] fp32 or bf16 -> out (fp32, the same shape); sel from tq_b8_select; acc_in and
    acc_out fp32 [n_seq, n_kv, 32 * max_blocks]: the accumulated attention weights that tq_b8_evict goes by."""
    qp, dt, n_q, g = _queries(cache, q)
    op = _tensor(cache, "out", out, cache.f32, q.shape)
    sp, n_sel, ip, ap = None, 0, None, None
    if sel is not None:
        sp, n_sel = _selection(cache, sel, n_q)
    if acc_in is not None:
        ip = _tensor(cache, "acc_in", acc_in, cache.f32, cache.row)
    if acc_out is not None:
        ap = _tensor(cache, "acc_out", acc_out, cache.f32, cache.row)
    return _b8_call("tq_b8_attention", lib.tq_b8_attention, cache, ws, stream, qp, dt, n_q, g, scale, sp, n_sel, ip, ap,
                    decay, op)


def tq_b8_select(cache, q, sel, ws, n_first=1, n_last=1, stream=None):
    """Fills sel int32 [n_seq, n_q, n_kv, n_sel] with the blocks tq_b8_attention is to look at."""
    qp, dt, n_q, g = _queries(cache, q)
    sp, n_sel = _selection(cache, sel, n_q)
    return _b8_call("tq_b8_select", lib.tq_b8_select, cache, ws, stream, qp, dt, n_q, g, n_first, n_last, n_sel, sp)


def tq_b8_evict(cache, acc, keep_blocks, dst_table, kept, length_out, acc_out, ws, n_first=0, n_last=0, stream=None):
    """Keeps 32 * keep_blocks of each sequence's paged tokens; dst_table and length_out are the cache afterwards."""
    ap, op = _tensor(cache, "acc", acc, cache.f32, cache.row), _tensor(cache, "acc_out", acc_out, cache.f32, cache.row)
    dp = _tensor(cache, "dst_table", dst_table, cache.i32, (cache.n_seq, cache.max_blocks))
    kp = _tensor(cache, "kept", kept, cache.i32, (cache.n_seq, cache.n_kv, TQ_B8_BLOCK * keep_blocks))
    lp = _tensor(cache, "length_out", length_out, cache.i32, (cache.n_seq,))
    return _b8_call("tq_b8_evict", lib.tq_b8_evict, cache, ws, stream, ap, keep_blocks, n_first, n_last, dp, kp, lp, op)


def tq_dequantize(codec: Codec, packed, n_streams, n_tok, out, ws=None, stream=None):
    return _check("tq_dequantize", lib.tq_dequantize(codec.ref, _ptr(packed), n_streams, n_tok, _ptr(out), _ptr(ws),
                                                     0 if ws is None else ws.numel(), _stream(stream)))


def tq_reset_status(ws, stream=None):
    return _check("tq_reset_status", lib.tq_reset_status(_ptr(ws), _stream(stream)))


def tq_get_status(ws, stream=None) -> int:
    """TQ_OK or TQ_ERR_RANGE (data-dependent faults since the last read); clears the word."""
    return lib.tq_get_status(_ptr(ws), _stream(stream))
