// Choosing: blocks by a bound on their logits (tq_b8_select), tokens by accumulated attention
// weight, and the move of the tokens that stay (tq_b8_evict).
//
// Score. For codes between lo_i and hi_i, sum_i qi_i code_i <= sum_i max(qi_i lo_i, qi_i hi_i) =
// <min(qi, 0), lo> + <max(qi, 0), hi>: one int8 product of length 2 D with the block's summary,
// exact in int32, on the int8 tensor cores (16 blocks x 8 heads per warp). A block costs 2 D + 4
// bytes here where attention reads 64 D. Bound by the chain table -> summary: 16 x 512 blocks of 8 heads in 12.9 us
// (80 registers, nothing spilled; held to 64, four CTAs an SM: 1 to 4 us more).
//
// Choice of the k largest of n. Keys are order-preserving 32-bit patterns. The k-th largest is
// found digit by digit (11 + 11 + 10 bits, fewer once all keys with the digits so far are taken) from histograms in
// shared memory; a last pass in index order writes what lies above it and the first of what equals it, by prefix sums,
// so the result is ascending and ties go to the lowest index. A row is one CTA's, its keys in registers: a chain of
// barriers: 8 rows of 4096 blocks 7.3 us, 32 of up to 8192 tokens 12.6 (cold; both kernels of a selection over 8 x 4096
// blocks, overlapped: 10).
#include <algorithm>
#include <cfloat>

#include "k_b8.cuh"

namespace {

constexpr int kScoreWarps = 8;
constexpr int kMoveWarps = 4;
constexpr float kRound = 12583040.f;     // 1.5 * 2^23 + 128: a sum's low byte is code + 128

TQ_DEVICE uint32_t order_bits(float f) {
    const uint32_t u = __float_as_uint(f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// full blocks that begin at or before the position of query token i
TQ_DEVICE int candidates(int n, int n_q, int i) {
    const int last = n - n_q + i;
    return last < 0 ? 0 : min(n >> 5, (last >> 5) + 1);
}

struct ScoreRow {
    int s, h, nb;                                    // sequence, kv head, candidates
    TQ_DEVICE ScoreRow(const B8SelectParams& p, int row) {
        const int si = row / p.c.n_kv;
        h = row - si * p.c.n_kv;
        s = p.n_q == 1 ? si : si / p.n_q;
        nb = candidates(b8_len(p.c, s), p.n_q, si - s * p.n_q);
    }
};

// Scores of blocks from .. to - 1 of a row (sequence, query token, kv head) as ordered bits in key: a CTA's warps take 16
// blocks each in turn, the first summaries on their way while the query heads become int8, with AHEAD (more registers) the
// next ones while these are multiplied.
template <int D, bool AHEAD>
TQ_DEVICE void score(const B8SelectParams& p, int row, const ScoreRow& x, int from, int to, uint32_t* key) {
    constexpr int CH = D / 32;       // 16-byte chunks a lane takes of a summary's 2 D bytes
    constexpr int STEP = kScoreWarps * 16;
    const B8Cache& c = p.c;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
    __shared__ uint32_t s_q[8][2 * D / 4 + 4];   // + 4 words: the 8 rows of a load fall on distinct banks
    __shared__ float s_step[8];
    const int32_t* table = c.table + x.s * c.max_blocks;
    struct Part {                    // summaries and key scales of rows gq and gq + 8 of 16 blocks
        uint4 a[2][CH];
        float ks[2];
    };
    auto load = [&](Part& z, int b0) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const uint8_t* e = nullptr;
            if (b0 + gq + 8 * r < to) {
                uint8_t* page = b8_page(c, table[b0 + gq + 8 * r]);
                if (page) e = b8_entry(c, page, x.h);
            }
            z.ks[r] = e ? *reinterpret_cast<const float*>(e) : 0.f;
#pragma unroll
            for (int k = 0; k < CH; ++k)
                z.a[r][k] = e ? *reinterpret_cast<const uint4*>(e + 32 + 16 * (tq + 4 * k)) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    for (int g0 = 0; g0 < p.g; g0 += 8) {        // 8 query heads at a time
        Part z;
        load(z, from + 16 * w);
        if (g0) __syncthreads();
        {   // warp w holds query head g0 + w as int8: negative parts against lo, positive ones against hi
            const int j = g0 + w;
            const int64_t at = ((int64_t)row * p.g + j) * c.d;
            float v[D / 32], am = 0.f;
            bool fin = true;
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
                const int e = lane * (D / 32) + k;
                v[k] = j < p.g && e < c.d ? tq_load_elem(p.q, p.q_dtype, at + e) : 0.f;
                fin = fin && isfinite(v[k]);
                am = fmaxf(am, fabsf(v[k]));
            }
            am = tq_warp_max(am);
            const bool live = __all_sync(0xffffffffu, fin) && am >= kB8MinMax;
            const float inv = live ? (1.f / am) * 127.f : 0.f;
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
                const int e = lane * (D / 32) + k;
                const int qi = live ? (int)(__float_as_uint(fmaf(v[k], inv, kRound)) & 0xffu) - 128 : 0;
                reinterpret_cast<int8_t*>(s_q[w])[e] = (int8_t)min(qi, 0);
                reinterpret_cast<int8_t*>(s_q[w])[D + e] = (int8_t)max(qi, 0);
            }
            if (lane == 0) s_step[w] = live ? am * kB8Inv127 : 0.f;
        }
        __syncthreads();
        for (int b0 = from + 16 * w; b0 < to; b0 += STEP) {
            Part next;
            if (AHEAD && b0 + STEP < to) load(next, b0 + STEP);
            int acc[4] = {0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < CH; ++k) {
                const uint32_t* b = &s_q[gq][4 * (tq + 4 * k)];
                tq_imma(acc, z.a[0][k].x, z.a[1][k].x, z.a[0][k].y, z.a[1][k].y, b[0], b[1]);
                tq_imma(acc, z.a[0][k].z, z.a[1][k].z, z.a[0][k].w, z.a[1][k].w, b[2], b[3]);
            }
            float best[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int k = 0; k < 4; ++k) {        // blocks gq, gq, gq + 8, gq + 8; heads 2 tq, 2 tq + 1
                const int j = 2 * tq + (k & 1);
                if (g0 + j < p.g)
                    best[k >> 1] = fmaxf(best[k >> 1], __fmul_rn(__fmul_rn((float)acc[k], z.ks[k >> 1]), s_step[j]));
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 1));
                best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 2));
                const int b = b0 + gq + 8 * r;
                if (tq == 0 && b < to) {         // (a block's key is this lane's alone, in every round of heads)
                    const uint32_t u = order_bits(best[r] + 0.f);   // a score that underflows from below is 0 too
                    key[b] = g0 ? max(key[b], u) : u;
                }
            }
            if (AHEAD) z = next;
            else if (b0 + STEP < to) load(z, b0 + STEP);
        }
    }
}

// One CTA per row and range of blocks. A row with no more candidates than places needs no scores.
template <int D>
__global__ void __launch_bounds__(kScoreWarps * 32) k_b8_score(const __grid_constant__ B8SelectParams p, int ranges, int range) {
    tq_pdl_launch_dependents();
    tq_pdl_wait();
    const int row = blockIdx.x / ranges, from = (blockIdx.x - row * ranges) * range;
    const ScoreRow x(p, row);
    const int to = min(x.nb, from + range);
    if (from < to && x.nb > p.n_sel) score<D, false>(p, row, x, from, to, p.key + row * p.c.max_blocks);
}

// Ascending indices of the chosen of n: all of them if n <= k, else the first nf, the last nl and the
// k - nf - nl largest keys between, ties to the lowest; the rest of out[0 .. k) is -1. A thread holds KEYS keys in
// registers; up to KEYS * THREADS keys are read once, more once for each digit.
template <int THREADS, int KEYS, typename Key>
TQ_DEVICE void pick(int n, int64_t k64, int nf, int nl, Key key, int32_t* out) {
    constexpr int NW = THREADS / 32, BINS = 2048 / THREADS, CHUNK = KEYS * THREADS;
    __shared__ uint32_t s_hist[2048], s_cnt[KEYS][NW], s_tot[KEYS], s_warp[NW], s_digit, s_left, s_here;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    if (n <= k64) {
        for (int64_t j = tid; j < k64; j += THREADS) out[j] = j < n ? (int32_t)j : -1;
        return;
    }
    const int k = (int)k64, m0 = nf, m1 = n - nl;
    uint32_t left = (uint32_t)(k - nf - nl);      // how many the middle gives
    uint32_t prefix = 0, mask = 0, u[KEYS];
    const bool any = left > 0;
    auto load = [&](int c0) {
#pragma unroll
        for (int i = 0; i < KEYS; ++i) {
            const int t = c0 + i * THREADS + tid;
            u[i] = t >= m0 && t < m1 ? key(t) : 0u;
        }
    };
    if (any) {
        load(0);
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int sh = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const uint32_t digit = pass == 2 ? 1023u : 2047u;
#pragma unroll
            for (int b = 0; b < BINS; ++b) s_hist[b * THREADS + tid] = 0;
            __syncthreads();
#pragma unroll 1
            for (int c0 = 0; c0 < n; c0 += CHUNK) {
                if (n > CHUNK) load(c0);
#pragma unroll
                for (int i = 0; i < KEYS; ++i) {
                    const int t = c0 + i * THREADS + tid;
                    if (t >= m0 && t < m1 && (u[i] & mask) == prefix) atomicAdd(&s_hist[(u[i] >> sh) & digit], 1u);
                }
            }
            __syncthreads();
            // the largest digit with at least `left` keys at or above it; thread t has BINS bins, from the top
            uint32_t h[BINS], sum = 0;
#pragma unroll
            for (int b = 0; b < BINS; ++b) {
                h[b] = s_hist[2047 - BINS * tid - b];
                sum += h[b];
            }
            uint32_t incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += x;
            }
            if (lane == 31) s_warp[w] = incl;
            __syncthreads();
            uint32_t above = incl - sum + __reduce_add_sync(0xffffffffu, lane < w && lane < NW ? s_warp[lane] : 0u);
            if (above < left && above + sum >= left) {
#pragma unroll
                for (int b = 0; b < BINS; ++b) {
                    if (above < left && above + h[b] >= left) {
                        s_digit = 2047 - BINS * tid - b;
                        s_left = left - above;
                        s_here = h[b];
                    }
                    above += h[b];
                }
            }
            __syncthreads();
            prefix |= s_digit << sh;
            mask |= digit << sh;
            left = s_left;
            if (s_here == left) break;               // every key with these digits is taken: the others do not matter
        }
    }
    // What lies above prefix in the digits looked at is taken, and the first `left` of what equals it: an index's place is
    // the number taken for sure before it plus the number of ties before it, up to `left`.
    const uint32_t below = (1u << lane) - 1;
    uint32_t sure0 = 0, ties0 = 0;
#pragma unroll 1
    for (int c0 = 0; c0 < n; c0 += CHUNK) {
        if (any && n > CHUNK) load(c0);
        uint32_t is_sure = 0, is_tie = 0;            // a bit per key
#pragma unroll
        for (int i = 0; i < KEYS; ++i) {
            const int t = c0 + i * THREADS + tid;
            const bool mid = any && t >= m0 && t < m1;
            const uint32_t v = u[i] & mask;
            const bool sure = t < n && (t < m0 || t >= m1 || (mid && v > prefix)), tie = mid && v == prefix;
            const uint32_t bs = __ballot_sync(0xffffffffu, sure), bt = __ballot_sync(0xffffffffu, tie);
            if (lane == 0) s_cnt[i][w] = __popc(bs) | __popc(bt) << 16;
            is_sure |= (uint32_t)sure << i;
            is_tie |= (uint32_t)tie << i;
        }
        __syncthreads();
        for (int i = w; i < KEYS; i += NW) {
            const uint32_t v = lane < NW ? s_cnt[i][lane] : 0u;
            uint32_t incl = v;
#pragma unroll
            for (int o = 1; o < NW; o <<= 1) {
                const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += x;
            }
            if (lane < NW) s_cnt[i][lane] = incl - v;
            if (lane == NW - 1) s_tot[i] = incl;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < KEYS; ++i) {
            const bool sure = is_sure >> i & 1u, tie = is_tie >> i & 1u;
            const uint32_t bs = __ballot_sync(0xffffffffu, sure), bt = __ballot_sync(0xffffffffu, tie);
            const uint32_t c = s_cnt[i][w], ties = ties0 + (c >> 16) + __popc(bt & below);
            if (sure || (tie && ties < left))
                out[sure0 + (c & 0xffffu) + __popc(bs & below) + min(ties, left)] = c0 + i * THREADS + tid;
            sure0 += s_tot[i] & 0xffffu;
            ties0 += s_tot[i] >> 16;
        }
        __syncthreads();
    }
}

struct ScoreKey {
    const uint32_t* key;
    TQ_DEVICE uint32_t operator()(int t) const { return key[t]; }
};
struct WeightKey {
    const float* acc;
    TQ_DEVICE uint32_t operator()(int t) const { return __float_as_uint(fmaxf(acc[t], 0.f) + 0.f); }
};

template <int THREADS, int KEYS>
__global__ void __launch_bounds__(THREADS) k_b8_pick_blocks(const __grid_constant__ B8SelectParams p) {
    tq_pdl_launch_dependents();
    tq_pdl_wait();
    const int row = blockIdx.x, si = row / p.c.n_kv, s = p.n_q == 1 ? si : si / p.n_q;
    const int nb = candidates(b8_len(p.c, s), p.n_q, si - s * p.n_q);
    pick<THREADS, KEYS>(nb, p.n_sel, p.n_first, p.n_last, ScoreKey{p.key + row * p.c.max_blocks},
                        p.sel + (int64_t)row * p.n_sel);
}

// Scores and choice of a whole row in one CTA: 160 rows of 512 blocks in 17 us cold, 256 of up to 512 in 14.8 warm.
constexpr int kFusedBlocks = 512;
template <int D>
__global__ void __launch_bounds__(kScoreWarps * 32) k_b8_score_pick(const __grid_constant__ B8SelectParams p) {
    __shared__ uint32_t s_key[kFusedBlocks];
    tq_pdl_launch_dependents();
    tq_pdl_wait();
    const int row = blockIdx.x;
    const ScoreRow x(p, row);
    if (x.nb > p.n_sel) score<D, true>(p, row, x, 0, x.nb, s_key);
    __syncthreads();
    pick<kScoreWarps * 32, kFusedBlocks / (kScoreWarps * 32)>(x.nb, p.n_sel, p.n_first, p.n_last, ScoreKey{s_key},
                                                             p.sel + (int64_t)row * p.n_sel);
}

template <int THREADS, int KEYS>
__global__ void __launch_bounds__(THREADS) k_b8_pick_tokens(const __grid_constant__ B8EvictParams p) {
    tq_pdl_launch_dependents();
    tq_pdl_wait();
    const int row = blockIdx.x, s = row / p.c.n_kv, n = b8_len(p.c, s) & ~31;
    // (n_first and n_last are at most the tokens kept, and matter where there are more than those)
    pick<THREADS, KEYS>(n, 32 * p.keep_blocks, (int)p.n_first, (int)p.n_last,
                        WeightKey{p.acc + row * p.c.max_blocks * 32}, p.kept + row * 32 * p.keep_blocks);
}

// the range of bytes c + 128, word by word
struct ByteRange {
    uint32_t lo = 0x00ff00ffu, hi = 0u;              // 16-bit minima and maxima of the even and odd bytes
    TQ_DEVICE void take(uint32_t w) {
        const uint32_t e = w & 0x00ff00ffu, o = __byte_perm(w, 0, 0x4341);
        lo = __vimin3_u16x2(lo, e, o);
        hi = __vimax3_u16x2(hi, e, o);
    }
    TQ_DEVICE int top() const {                      // the largest |c|
        const int l = (int)min(lo & 0xffffu, lo >> 16), h = (int)max(hi & 0xffffu, hi >> 16);
        return max(h - 128, 128 - l);
    }
};

// One warp per (sequence, new block, head), keys and values together where the registers hold both (D <= 128): gathers
// 32 kept tokens, finds the new scales, requantizes by one multiply-add per code and writes the block, its scales and
// summary. The warps of new block keep_blocks move what belongs to the open block: its acc, the length.
// Bound by the chain kept -> table -> rows (all rows of a warp under way at once) and by instructions: 500 MB in 104 us
// (32 sequences of up to 8192 tokens to half), 0.73 of the measured copy rate. Registers are held to four CTAs an SM: with
// three 117 us, with five (spilled) 104. A lane holds 16 channels
// of D / 16 tokens; codes stay packed but for the multiply-add, maxima and the summary's ranges are taken on 16-bit pairs.
template <int D>
struct MoveSides { static constexpr int n = D == 256 ? 1 : 2; };
template <int D>
__global__ void __launch_bounds__(kMoveWarps * 32, 4) k_b8_move(const __grid_constant__ B8EvictParams p) {
    constexpr int CH = D / 16, TPI = 32 / CH, IT = CH;   // 16-byte chunks of a row; tokens per step; steps
    constexpr int NS = MoveSides<D>::n;
    const B8Cache& c = p.c;
    tq_pdl_launch_dependents();
    tq_pdl_wait();
    const int lane = threadIdx.x & 31;
    int64_t id = (int64_t)blockIdx.x * kMoveWarps + (threadIdx.x >> 5);
    const int h = (int)(id % c.n_kv);
    id /= c.n_kv;
    const int side0 = NS == 1 ? (int)(id & 1) : 0;
    if (NS == 1) id >>= 1;
    const int64_t j = id % (p.keep_blocks + 1), s = id / (p.keep_blocks + 1);
    if (s >= c.n_seq) return;
    const int n = b8_len(c, s), nfull = n >> 5, r = n & 31;
    const int left = (int)min((int64_t)nfull, p.keep_blocks);
    const int64_t arow = (s * c.n_kv + h) * c.max_blocks * 32;
    if (j == p.keep_blocks) {
        if (side0 == 0 && lane < r) p.acc_out[arow + 32 * left + lane] = p.acc[arow + 32 * nfull + lane];
        if (side0 == 0 && h == 0 && lane == 0) p.len_out[s] = 32 * left + r;
        return;
    }
    if (j >= left) return;
    const int tok = p.kept[((s * c.n_kv + h) * p.keep_blocks + j) * 32 + lane];
    uint8_t* page = b8_page(c, c.table[s * c.max_blocks + (tok >> 5)]);
    uint8_t* dst = b8_page(c, p.dst_table[s * c.max_blocks + j]);
    float2 sc = make_float2(0.f, 0.f);                   // key and value scale of token `lane`
    if (page) sc = *reinterpret_cast<const float2*>(b8_entry(c, page, h));
    const uint8_t* row = page ? b8_codes(c, page, h, side0) + (tok & 31) * D : nullptr;
    const int ch = lane % CH, t0 = lane / CH;
    uint4 x[NS][IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int t = t0 + i * TPI;
        const uint8_t* rp = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, (unsigned long long)row, t));
        const int tk = __shfl_sync(0xffffffffu, tok, t) & 31;
#pragma unroll
        for (int y = 0; y < NS; ++y)
            x[y][i] = rp ? tq_ldg_stream(rp + y * 32 * D + ((ch ^ b8_swz(tk, CH)) << 4))
                         : make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u);
    }
    if (side0 == 0) p.acc_out[arow + 32 * j + lane] = p.acc[arow + tok];
    float top[NS];
#pragma unroll
    for (int y = 0; y < NS; ++y) {
        const float mine = (NS == 1 ? side0 : y) ? sc.y : sc.x;
        top[y] = 0.f;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            ByteRange br;
            br.take(x[y][i].x);
            br.take(x[y][i].y);
            br.take(x[y][i].z);
            br.take(x[y][i].w);
            int m = br.top();
#pragma unroll
            for (int o = 1; o < CH; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            top[y] = fmaxf(top[y], __fmul_rn(__fmul_rn((float)m, kB8Inv127), __shfl_sync(0xffffffffu, mine, t0 + i * TPI)));
        }
        top[y] = tq_warp_max(top[y]);
    }
    if (!dst) return;
    uint8_t* e = b8_entry(c, dst, h);
#pragma unroll
    for (int y = 0; y < NS; ++y) {
        const int side = NS == 1 ? side0 : y;
        const float ratio = top[y] > 0.f ? (side ? sc.y : sc.x) / top[y] : 0.f;
        uint8_t* drow = b8_codes(c, dst, h, side);
        uint32_t lo[8], hi[8];                           // 16-bit ranges of this lane's 16 channels
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            lo[k] = 0x00ff00ffu;
            hi[k] = 0u;
        }
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int t = t0 + i * TPI;
            const float rt = __shfl_sync(0xffffffffu, ratio, t);
            const uint32_t u[4] = {x[y][i].x, x[y][i].y, x[y][i].z, x[y][i].w};
            uint32_t o[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float2 f[2];
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    f[k] = f2_fma(f2_add(make_float2(__uint_as_float(__byte_perm(u[q], 0x4b000000u, 0x7440 + 2 * k)),
                                                     __uint_as_float(__byte_perm(u[q], 0x4b000000u, 0x7441 + 2 * k))),
                                         f2(-8388736.f)),
                                  f2(rt), f2(kRound));
                o[q] = __byte_perm(__byte_perm(__float_as_uint(f[0].x), __float_as_uint(f[0].y), 0x0040),
                                   __byte_perm(__float_as_uint(f[1].x), __float_as_uint(f[1].y), 0x0040), 0x5410);
                if (side == 0) {
                    const uint32_t ev = o[q] & 0x00ff00ffu, od = __byte_perm(o[q], 0, 0x4341);
                    lo[2 * q] = __vminu2(lo[2 * q], ev);
                    hi[2 * q] = __vmaxu2(hi[2 * q], ev);
                    lo[2 * q + 1] = __vminu2(lo[2 * q + 1], od);
                    hi[2 * q + 1] = __vmaxu2(hi[2 * q + 1], od);
                }
            }
            *reinterpret_cast<uint4*>(drow + t * D + ((ch ^ b8_swz(t, CH)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        if (lane == 0) *reinterpret_cast<float*>(e + 4 * side) = top[y];
        if (side) continue;
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
            for (int o = CH; o < 32; o <<= 1) {
                lo[k] = __vminu2(lo[k], __shfl_xor_sync(0xffffffffu, lo[k], o));
                hi[k] = __vmaxu2(hi[k], __shfl_xor_sync(0xffffffffu, hi[k], o));
            }
        if (lane < CH) {
            uint32_t l[4], g[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {                // even bytes from one pair, odd bytes from the other
                l[q] = (lo[2 * q] | lo[2 * q + 1] << 8) ^ 0x80808080u;
                g[q] = (hi[2 * q] | hi[2 * q + 1] << 8) ^ 0x80808080u;
            }
            *reinterpret_cast<uint4*>(e + 32 + 16 * ch) = make_uint4(l[0], l[1], l[2], l[3]);
            *reinterpret_cast<uint4*>(e + 32 + D + 16 * ch) = make_uint4(g[0], g[1], g[2], g[3]);
        }
    }
}

}  // namespace

cudaError_t b8_launch_select(const B8SelectParams& p, cudaStream_t st) {
    const int64_t rows = p.c.n_seq * p.n_q * p.c.n_kv;
    // One kernel for both where a row is a step or two of one CTA, or four and the rows alone fill the GPU: selection and
    // attention of 16 sequences of 8000 tokens, 8 heads, 27 us instead of 30, 32 of 16384 45 and 48; but 8 of 16000
    // 28.8 and 28.2, 16 of 32000 49 and 42.
    if (p.c.max_blocks <= (rows >= tq_device_sms() ? kFusedBlocks : kFusedBlocks / 2)) {
        if (rows > 0x7fffffffLL) return cudaErrorInvalidValue;
        return tq_launch_pdl(p.c.D == 64    ? k_b8_score_pick<64>
                             : p.c.D == 128 ? k_b8_score_pick<128>
                                            : k_b8_score_pick<256>,
                             dim3((unsigned)rows), dim3(kScoreWarps * 32), 0, st, p);
    }
    // Ranges of blocks: a step of 128 each, longer where that gives more than four waves of CTAs
    const int64_t steps = (p.c.max_blocks + kScoreWarps * 16 - 1) / (kScoreWarps * 16), slots = 16 * (int64_t)tq_device_sms();
    const int64_t per = std::max<int64_t>(1, (rows * steps + slots - 1) / slots), ranges = (steps + per - 1) / per;
    if (rows * ranges > 0x7fffffffLL) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)(rows * ranges)), block(kScoreWarps * 32);
    const cudaError_t e = tq_launch_pdl(p.c.D == 64    ? k_b8_score<64>
                                        : p.c.D == 128 ? k_b8_score<128>
                                                       : k_b8_score<256>,
                                        grid, block, 0, st, p, (int)ranges, (int)(per * kScoreWarps * 16));
    if (e != cudaSuccess) return e;
    // as few keys a thread as hold a whole row: little code runs
    const dim3 r((unsigned)rows);
    if (p.c.max_blocks <= 1024) return tq_launch_pdl(k_b8_pick_blocks<256, 4>, r, dim3(256), 0, st, p);
    if (p.c.max_blocks <= 4096) return tq_launch_pdl(k_b8_pick_blocks<1024, 4>, r, dim3(1024), 0, st, p);
    return tq_launch_pdl(k_b8_pick_blocks<1024, 16>, r, dim3(1024), 0, st, p);
}

cudaError_t b8_launch_evict(const B8EvictParams& p, cudaStream_t st) {
    const int64_t rows = p.c.n_seq * p.c.n_kv;
    const int64_t grid = (rows * (p.c.D == 256 ? 2 : 1) * (p.keep_blocks + 1) + kMoveWarps - 1) / kMoveWarps;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    const dim3 r((unsigned)rows);
    const int64_t most = p.c.max_blocks * 32;
    const cudaError_t e = most <= 1024   ? tq_launch_pdl(k_b8_pick_tokens<256, 4>, r, dim3(256), 0, st, p)
                          : most <= 4096 ? tq_launch_pdl(k_b8_pick_tokens<1024, 4>, r, dim3(1024), 0, st, p)
                          : most <= 8192 ? tq_launch_pdl(k_b8_pick_tokens<1024, 8>, r, dim3(1024), 0, st, p)
                                         : tq_launch_pdl(k_b8_pick_tokens<1024, 16>, r, dim3(1024), 0, st, p);
    if (e != cudaSuccess) return e;
    return tq_launch_pdl(p.c.D == 64 ? k_b8_move<64> : p.c.D == 128 ? k_b8_move<128> : k_b8_move<256>,
                         dim3((unsigned)grid), dim3(kMoveWarps * 32), 0, st, p);
}
