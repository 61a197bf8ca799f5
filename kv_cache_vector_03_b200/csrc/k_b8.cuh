// Paged 8-bit cache: the page layout and the parameter blocks of its kernels (the layout is
// documented in include/tq.h).
#pragma once
#include "tq_device.cuh"

constexpr int kB8Block = 32;
constexpr int kB8Counters = 192;   // bytes of arrival counts (4 bits a CTA) behind the status word, in its 256 bytes
constexpr float kB8Inv127 = 1.f / 127.f;               // rounded to fp32; 127 times it rounds to 1
constexpr float kB8MinMax = 7.8886090522101181e-31f;   // 2^-100: a block whose largest |x| is below it is stored as zeros

static inline int b8_padded(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }
static inline size_t b8_header_bytes(int D, int n_kv) { return ((size_t)n_kv * (32 + 2 * D) + 127) / 128 * 128; }

// the caller's cache, as the kernels see it
struct B8Cache {
    uint8_t* pages;
    const int32_t* table;
    const int32_t* len;
    uint16_t* open;          // bf16 bits [n_seq][n_kv][2][32][d]
    uint32_t* status;
    int64_t page_bytes, header_bytes, max_blocks;
    int64_t n_seq, n_pages;
    int n_kv, d, D;
};

// two fp32 operations in one instruction, each rounded as by itself
TQ_DEVICE uint64_t f2_bits(float2 a) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
    return r;
}
TQ_DEVICE float2 f2_of(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
TQ_DEVICE float2 f2_fma(float2 a, float2 b, float2 c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)), "l"(f2_bits(c)));
    return f2_of(r);
}
TQ_DEVICE float2 f2_add(float2 a, float2 b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)));
    return f2_of(r);
}
TQ_DEVICE float2 f2_mul(float2 a, float2 b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_bits(a)), "l"(f2_bits(b)));
    return f2_of(r);
}
TQ_DEVICE float2 f2(float a) { return make_float2(a, a); }

TQ_DEVICE int b8_swz(int t, int chunks) { return ((t & 2) | (((t ^ (t >> 2)) & 1) << 2)) & (chunks - 1); }

// a sequence's length, 0 (and the status flag) where it cannot be
TQ_DEVICE int b8_len(const B8Cache& c, int64_t s) {
    const int n = c.len[s];
    if (n < 0 || (int64_t)n > c.max_blocks * kB8Block) {
        tq_raise(c.status, TQ_FLAG_RANGE);
        return 0;
    }
    return n;
}

// the page that a table entry names, or null (and the status flag) outside the pool
TQ_DEVICE uint8_t* b8_page(const B8Cache& c, int name) {
    if (name < 0 || (int64_t)name >= c.n_pages) {
        tq_raise(c.status, TQ_FLAG_RANGE);
        return nullptr;
    }
    return c.pages + (size_t)name * c.page_bytes;
}
TQ_DEVICE uint8_t* b8_entry(const B8Cache& c, uint8_t* page, int h) { return page + (size_t)h * (32 + 2 * c.D); }
TQ_DEVICE uint8_t* b8_codes(const B8Cache& c, uint8_t* page, int h, int side) {
    return page + c.header_bytes + (size_t)(2 * h + side) * (kB8Block * c.D);
}
TQ_DEVICE uint16_t* b8_open(const B8Cache& c, int64_t s, int h, int side) {
    return c.open + (size_t)((s * c.n_kv + h) * 2 + side) * kB8Block * c.d;
}

struct B8AppendParams {
    B8Cache c;
    const void* k;
    const void* v;
    int dtype;
    int64_t n_new, seq_stride, tok_stride;
    const int32_t* add;
};
struct B8ReadParams {
    B8Cache c;
    int64_t n_tok;
    void* k;
    void* v;
    int dtype;
};
struct B8AttnParams {
    B8Cache c;
    const void* q;
    int q_dtype, n_q, g;
    float scale_hi, scale_lo;   // scale * log2(e) as two floats
    const int32_t* sel;
    int n_sel;
    const float* acc_in;
    float* acc_out;
    float decay;
    float* out;
    float* logits;           // [n_seq * n_kv][n_q * g][logit_row], when acc_out is asked for: a row's tokens, their logits in the
                             // log2 domain next to the reference of their unit (k_b8_attn.cu), and from ref_at on these references
    float2* norm;            // [n_seq * n_kv][n_q * g] a row's reference and what its weights are multiplied with
    int64_t logit_row, ref_at;
    float* part;             // [2 grid][row_tile][D] partial value sums, [2 grid][row_tile][2] their maximum and sum
    float* part_ml;
    uint32_t* count;         // kB8Counters bytes, zero between calls: how many parts of a segment have arrived
    int grid, row_tile, row_tiles;
};
struct B8SelectParams {
    B8Cache c;
    const void* q;
    int q_dtype, n_q, g, n_first, n_last, n_sel;
    int32_t* sel;
    uint32_t* key;           // [n_seq * n_q * n_kv][max_blocks] order-preserving bits of the scores
};
struct B8EvictParams {
    B8Cache c;
    const float* acc;
    int64_t keep_blocks, n_first, n_last;
    const int32_t* dst_table;
    int32_t* kept;
    int32_t* len_out;
    float* acc_out;
};

int b8_attn_row_tile(int D, int rows, int64_t blocks);   // query rows a unit is computed for at once
int b8_attn_grid();                      // CTAs of one wave
cudaError_t b8_launch_append(const B8AppendParams& p, cudaStream_t st);
cudaError_t b8_launch_read(const B8ReadParams& p, cudaStream_t st);
cudaError_t b8_launch_attention(const B8AttnParams& p, cudaStream_t st);
cudaError_t b8_launch_select(const B8SelectParams& p, cudaStream_t st);
cudaError_t b8_launch_evict(const B8EvictParams& p, cudaStream_t st);
