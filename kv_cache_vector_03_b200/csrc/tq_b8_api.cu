// C-ABI entry points of the paged 8-bit cache (declared and documented in include/tq.h):
// argument checks, workspace layout and kernel launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "k_b8.cuh"
#include "tq.h"

namespace {

static_assert(64 + kB8Counters <= TQ_STATUS_BYTES, "the arrival counts share the status word's bytes");
constexpr int64_t kMaxBlocks = (int64_t)1 << 23, kMaxRows = (int64_t)1 << 28;

size_t align_up(size_t v) { return (v + TQ_ALIGN - 1) / TQ_ALIGN * TQ_ALIGN; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
int cuda_status(cudaError_t e) {
    return e == cudaSuccess ? TQ_OK : e == cudaErrorInvalidValue ? TQ_ERR_UNSUPPORTED : TQ_ERR_CUDA;
}

int check_shape(const tq_b8_cache* c) {
    if (!c) return TQ_ERR_ARG;
    if (c->d < 8 || c->d > 256 || c->d % 8) return TQ_ERR_UNSUPPORTED;
    if (c->n_kv < 1 || c->n_seq < 0 || c->n_pages < 0 || c->max_blocks < 1) return TQ_ERR_ARG;
    if (c->n_kv > 1024 || c->n_seq > 65535 || c->n_pages > 0x7fffffffLL || c->max_blocks > kMaxBlocks)
        return TQ_ERR_UNSUPPORTED;
    return TQ_OK;
}

int check_cache(const tq_b8_cache* c) {
    const int st = check_shape(c);
    if (st != TQ_OK || c->n_seq == 0) return st;
    if ((c->n_pages > 0 && !c->pages) || !c->table || !c->len || !c->open) return TQ_ERR_ARG;
    if (!aligned(c->pages, 128) || !aligned(c->table, 4) || !aligned(c->len, 4) || !aligned(c->open, 16))
        return TQ_ERR_ARG;
    return TQ_OK;
}

int check_queries(int q_dtype, int n_q, int g) {
    if (q_dtype != TQ_F32 && q_dtype != TQ_BF16) return TQ_ERR_ARG;
    if (n_q < 1 || g < 1) return TQ_ERR_ARG;
    if ((int64_t)n_q * g > 16384) return TQ_ERR_UNSUPPORTED;
    return TQ_OK;
}

B8Cache view(const tq_b8_cache* c, void* ws) {
    B8Cache v;
    v.pages = static_cast<uint8_t*>(c->pages);
    v.table = c->table;
    v.len = c->len;
    v.open = static_cast<uint16_t*>(c->open);
    v.status = static_cast<uint32_t*>(ws);
    v.d = c->d; v.D = b8_padded(c->d); v.n_kv = c->n_kv;
    v.n_seq = c->n_seq; v.n_pages = c->n_pages; v.max_blocks = c->max_blocks;
    v.header_bytes = (int64_t)b8_header_bytes(v.D, v.n_kv);
    v.page_bytes = (int64_t)tq_b8_page_bytes(v.d, v.n_kv);
    return v;
}

// regions after the status word; a call uses those of its own kind, so they share the space. total is 0 where the two that
// grow with rows x blocks pass kMaxWs (the products of all limits pass 64 bits)
constexpr size_t kMaxWs = (size_t)1 << 62;
struct B8Ws { size_t key, part, ml, norm, logits, total; int64_t logit_row, ref_at; int rows, row_tile; };
B8Ws b8_ws(const tq_b8_cache* c, int n_q, int g, int n_sel, bool weights) {
    B8Ws w = {};
    const size_t rows = (size_t)c->n_seq * c->n_kv * (size_t)n_q;
    size_t off = TQ_STATUS_BYTES;
    w.key = off;
    if (n_sel && rows > kMaxWs / 4 / (size_t)c->max_blocks) return w;
    const size_t select_end = align_up(off + (n_sel ? rows * (size_t)c->max_blocks * 4 : 0));
    w.ref_at = n_sel ? (int64_t)(n_sel + 1) * kB8Block : c->max_blocks * kB8Block;   // then a reference per unit: the halves of an
    w.logit_row = w.ref_at + (w.ref_at / kB8Block + 1 + 31) / 32 * 32;              // open block are two
    // rows and blocks of one virtual sequence (k_b8_attn.cu): of a sequence, with a selection of a query token
    w.rows = n_sel ? g : n_q * g;
    const int64_t blocks = c->n_seq * c->n_kv * (n_sel ? (int64_t)n_q * n_sel : c->max_blocks);
    const int tile = w.row_tile = b8_attn_row_tile(b8_padded(c->d), w.rows, blocks);
    const size_t slots = rows && g ? 2 * (size_t)b8_attn_grid() * tile : 0;
    w.part = off; off = align_up(off + slots * b8_padded(c->d) * 4);
    w.ml = off; off = align_up(off + slots * 8);
    w.norm = off; off = align_up(off + (weights ? rows * g * 8 : 0));
    if (weights && rows * g > kMaxWs / 4 / (size_t)w.logit_row) return w;
    w.logits = off; off = align_up(off + (weights ? rows * g * (size_t)w.logit_row * 4 : 0));
    w.total = std::max(select_end, off);
    return w;
}

int check_ws(const void* ws, size_t bytes, size_t need) {
    if (need == 0) return TQ_ERR_UNSUPPORTED;
    if (!ws || !aligned(ws, 256)) return TQ_ERR_ARG;
    return bytes < need ? TQ_ERR_WORKSPACE : TQ_OK;
}

}  // namespace

extern "C" {

size_t tq_b8_page_bytes(int d, int n_kv) {
    if (d < 8 || d > 256 || d % 8 || n_kv < 1 || n_kv > 1024) return 0;
    const int D = b8_padded(d);
    return b8_header_bytes(D, n_kv) + (size_t)n_kv * 64 * D;
}

size_t tq_b8_workspace_bytes(const tq_b8_cache* c, int n_q, int g, int n_sel, int weights) {
    if (check_shape(c) != TQ_OK || n_q < 0 || g < 0 || n_sel < 0 || n_sel > kMaxBlocks || (int64_t)n_q * g > 16384) return 0;
    return b8_ws(c, n_q, g, n_sel, weights != 0).total;
}

int tq_b8_append(const tq_b8_cache* c, const void* k, const void* v, tq_dtype dtype, int64_t n_new, int64_t seq_stride,
                 int64_t tok_stride, const int32_t* add, void* ws, size_t ws_bytes, void* stream) {
    int st = check_cache(c);
    if (st != TQ_OK) return st;
    if (dtype != TQ_F32 && dtype != TQ_BF16) return TQ_ERR_ARG;
    if (n_new < 0 || seq_stride < 0 || tok_stride < 0 || seq_stride % 8 || tok_stride % 8) return TQ_ERR_ARG;
    if (n_new > kMaxRows) return TQ_ERR_UNSUPPORTED;
    if (c->n_seq == 0 || n_new == 0) return TQ_OK;
    if (!k || !v || !aligned(k, 16) || !aligned(v, 16) || (add && !aligned(add, 4))) return TQ_ERR_ARG;
    if ((st = check_ws(ws, ws_bytes, TQ_STATUS_BYTES)) != TQ_OK) return st;
    B8AppendParams p;
    p.c = view(c, ws);
    p.k = k; p.v = v; p.dtype = dtype;
    p.n_new = n_new; p.seq_stride = seq_stride; p.tok_stride = tok_stride; p.add = add;
    return cuda_status(b8_launch_append(p, static_cast<cudaStream_t>(stream)));
}

int tq_b8_read(const tq_b8_cache* c, int64_t n_tok, void* k, void* v, tq_dtype dtype, void* ws, size_t ws_bytes,
               void* stream) {
    int st = check_cache(c);
    if (st != TQ_OK) return st;
    if (dtype != TQ_F32 && dtype != TQ_BF16) return TQ_ERR_ARG;
    if (n_tok < 0) return TQ_ERR_ARG;
    if (c->n_seq == 0 || n_tok == 0) return TQ_OK;
    if (!k || !v || !aligned(k, 16) || !aligned(v, 16)) return TQ_ERR_ARG;
    if ((st = check_ws(ws, ws_bytes, TQ_STATUS_BYTES)) != TQ_OK) return st;
    if (n_tok > kMaxRows) return TQ_ERR_UNSUPPORTED;
    B8ReadParams p;
    p.c = view(c, ws);
    p.n_tok = n_tok; p.k = k; p.v = v; p.dtype = dtype;
    return cuda_status(b8_launch_read(p, static_cast<cudaStream_t>(stream)));
}

int tq_b8_attention(const tq_b8_cache* c, const void* q, tq_dtype q_dtype, int n_q, int g, float scale,
                    const int32_t* sel, int n_sel, const float* acc_in, float* acc_out, float decay, float* out,
                    void* ws, size_t ws_bytes, void* stream) {
    int st = check_cache(c);
    if (st != TQ_OK) return st;
    if ((st = check_queries(q_dtype, n_q, g)) != TQ_OK) return st;
    const double scale2 = (double)scale * 1.4426950408889634074;   // log2(e)
    if (!std::isfinite((float)scale2) || !std::isfinite(decay)) return TQ_ERR_ARG;
    if (n_sel < 0 || n_sel > kMaxBlocks || (c->n_seq > 0 && (n_sel > 0) != (sel != nullptr))) return TQ_ERR_ARG;
    if (acc_in && !acc_out) return TQ_ERR_ARG;
    if (n_sel && acc_out && n_q != 1) return TQ_ERR_UNSUPPORTED;
    if (c->n_seq == 0) return TQ_OK;
    if (!q || !out || q == out || !aligned(q, 16) || !aligned(out, 16) || !aligned(sel, 4) ||
        !aligned(acc_in, 4) || !aligned(acc_out, 4))
        return TQ_ERR_ARG;
    const B8Ws W = b8_ws(c, n_q, g, n_sel, acc_out != nullptr);
    if ((st = check_ws(ws, ws_bytes, W.total)) != TQ_OK) return st;
    uint8_t* wsb = static_cast<uint8_t*>(ws);
    B8AttnParams p;
    std::memset(&p, 0, sizeof(p));
    p.c = view(c, ws);
    p.q = q; p.q_dtype = q_dtype; p.n_q = n_q; p.g = g;
    p.scale_hi = (float)scale2;
    p.scale_lo = (float)(scale2 - (double)p.scale_hi);
    p.sel = sel; p.n_sel = n_sel;
    p.acc_in = acc_in; p.acc_out = acc_out; p.decay = decay;
    p.out = out;
    p.norm = reinterpret_cast<float2*>(wsb + W.norm);
    p.logits = reinterpret_cast<float*>(wsb + W.logits);
    p.logit_row = W.logit_row; p.ref_at = W.ref_at;
    p.part = reinterpret_cast<float*>(wsb + W.part);
    p.part_ml = reinterpret_cast<float*>(wsb + W.ml);
    p.count = reinterpret_cast<uint32_t*>(wsb) + 16;
    p.grid = b8_attn_grid();
    p.row_tile = W.row_tile;
    p.row_tiles = (W.rows + p.row_tile - 1) / p.row_tile;
    return cuda_status(b8_launch_attention(p, static_cast<cudaStream_t>(stream)));
}

int tq_b8_select(const tq_b8_cache* c, const void* q, tq_dtype q_dtype, int n_q, int g, int n_first, int n_last,
                 int n_sel, int32_t* sel, void* ws, size_t ws_bytes, void* stream) {
    int st = check_cache(c);
    if (st != TQ_OK) return st;
    if ((st = check_queries(q_dtype, n_q, g)) != TQ_OK) return st;
    if (n_first < 0 || n_last < 0 || n_sel < 1 || (int64_t)n_first + n_last > n_sel || n_sel > kMaxBlocks)
        return TQ_ERR_ARG;
    if (c->n_seq == 0) return TQ_OK;
    if (!q || !sel || !aligned(q, q_dtype == TQ_F32 ? 4 : 2) || !aligned(sel, 4)) return TQ_ERR_ARG;
    const B8Ws W = b8_ws(c, n_q, g, n_sel, false);
    if ((st = check_ws(ws, ws_bytes, W.total)) != TQ_OK) return st;
    B8SelectParams p;
    p.c = view(c, ws);
    p.q = q; p.q_dtype = q_dtype; p.n_q = n_q; p.g = g;
    p.n_first = n_first; p.n_last = n_last; p.n_sel = n_sel; p.sel = sel;
    p.key = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(ws) + W.key);
    return cuda_status(b8_launch_select(p, static_cast<cudaStream_t>(stream)));
}

int tq_b8_evict(const tq_b8_cache* c, const float* acc, int64_t keep_blocks, int64_t n_first, int64_t n_last,
                const int32_t* dst_table, int32_t* kept, int32_t* len_out, float* acc_out, void* ws, size_t ws_bytes,
                void* stream) {
    int st = check_cache(c);
    if (st != TQ_OK) return st;
    if (keep_blocks < 1 || keep_blocks > kMaxBlocks || n_first < 0 || n_last < 0 ||
        n_first > keep_blocks * kB8Block || n_last > keep_blocks * kB8Block - n_first)
        return TQ_ERR_ARG;
    if (c->n_seq == 0) return TQ_OK;
    if (!acc || !dst_table || !kept || !len_out || !acc_out) return TQ_ERR_ARG;
    if (!aligned(acc, 4) || !aligned(dst_table, 4) || !aligned(kept, 4) || !aligned(len_out, 4) || !aligned(acc_out, 4))
        return TQ_ERR_ARG;
    if (len_out == c->len || acc_out == acc) return TQ_ERR_ARG;
    if ((st = check_ws(ws, ws_bytes, b8_ws(c, 0, 0, 0, false).total)) != TQ_OK) return st;
    B8EvictParams p;
    p.c = view(c, ws);
    p.acc = acc; p.keep_blocks = keep_blocks; p.n_first = n_first; p.n_last = n_last;
    p.dst_table = dst_table; p.kept = kept; p.len_out = len_out; p.acc_out = acc_out;
    return cuda_status(b8_launch_evict(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
