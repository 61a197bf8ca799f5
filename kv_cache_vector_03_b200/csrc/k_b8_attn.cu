// Decode attention over the paged 8-bit cache (tq_b8_attention).
#include <cfloat>

#include "k_b8.cuh"

namespace {

constexpr int kWarps = 8;
constexpr float kLog2e = 1.4426950408889634f;

// One CTA per (sequence, query token, query head); its warps take the blocks in turn, lane t
// scoring token t, then every lane summing D / 32 channels.
template <int D>
__global__ void __launch_bounds__(kWarps * 32) k_b8_attn(const __grid_constant__ B8AttnParams p) {
    constexpr int CPL = D / 32;
    const B8Cache& c = p.c;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t id = blockIdx.x;
    const int n_h = c.n_kv * p.g, jh = (int)(id % n_h);
    id /= n_h;
    const int i = (int)(id % p.n_q);
    const int64_t s = id / p.n_q;
    const int h = jh / p.g, row = i * p.g + jh % p.g;
    const int n = b8_len(c, s), last = n - p.n_q + i, nfull = n >> 5, r = n & 31;
    const int64_t qrow = ((s * p.n_q + i) * n_h + jh) * c.d;
    __shared__ float s_q[D], s_o[kWarps][D], s_m[kWarps], s_l[kWarps];
    for (int k = threadIdx.x; k < D; k += kWarps * 32)
        s_q[k] = k < c.d ? tq_load_elem(p.q, p.q_dtype, qrow + k) * (p.scale * kLog2e) : 0.f;
    __syncthreads();
    float m = -INFINITY, l = 0.f, o[CPL];
#pragma unroll
    for (int k = 0; k < CPL; ++k) o[k] = 0.f;
    const int32_t* sel = p.sel ? p.sel + ((s * p.n_q + i) * c.n_kv + h) * p.n_sel : nullptr;
    const int units = last < 0 ? 0 : (sel ? p.n_sel : nfull) + (r ? 1 : 0);
    float* lg = p.acc_out ? p.logits + ((s * c.n_kv + h) * (int64_t)(p.n_q * p.g) + row) * p.logit_row : nullptr;
    for (int u = w; u < units; u += kWarps) {
        const bool open = u == (sel ? p.n_sel : nfull);
        const int b = open ? nfull : sel ? sel[u] : u;
        const uint8_t* page = nullptr;
        if (!open && b >= 0 && b < nfull) page = b8_page(c, c.table[s * c.max_blocks + b]);
        float x = -INFINITY;
        if (open && lane < r && 32 * nfull + lane <= last) {
            const uint16_t* k = b8_open(c, s, h, 0) + lane * c.d;
            x = 0.f;
            for (int e = 0; e < c.d; ++e) x = fmaf(s_q[e], __uint_as_float((uint32_t)k[e] << 16), x);
        } else if (page && 32 * b + lane <= last) {
            const uint8_t* k = b8_codes(c, const_cast<uint8_t*>(page), h, 0) + lane * D;
            x = 0.f;
            for (int e = 0; e < D; ++e)
                x = fmaf(s_q[e], (float)((int)k[(((e >> 4) ^ b8_swz(lane, D / 16)) << 4) + (e & 15)] - 128), x);
            x *= *reinterpret_cast<const float*>(b8_entry(c, const_cast<uint8_t*>(page), h));
        }
        if (lg) lg[(sel ? u : b) * 32 + lane] = x;
        const float mn = fmaxf(m, tq_warp_max(x)), ref = mn == -INFINITY ? 0.f : mn;
        const float f = tq_exp2(m - ref), pr = tq_exp2(x - ref);
        m = mn;
        l = l * f + tq_warp_sum(pr);
#pragma unroll
        for (int k = 0; k < CPL; ++k) o[k] *= f;
        if (!open && !page) continue;
        const float vs = open ? 1.f : *reinterpret_cast<const float*>(b8_entry(c, const_cast<uint8_t*>(page), h) + 4);
        const int cnt = open ? r : 32;
        for (int t = 0; t < cnt; ++t) {
            const float wt = __shfl_sync(0xffffffffu, pr, t) * vs;
            if (32 * b + t > last) break;
#pragma unroll
            for (int k = 0; k < CPL; ++k) {
                const int e = lane + 32 * k;
                float v = 0.f;
                if (open) {
                    if (e < c.d) v = __uint_as_float((uint32_t)b8_open(c, s, h, 1)[t * c.d + e] << 16);
                } else {
                    v = (float)((int)b8_codes(c, const_cast<uint8_t*>(page), h, 1)[t * D + (((e >> 4) ^ b8_swz(t, D / 16)) << 4) +
                                                                                (e & 15)] - 128);
                }
                o[k] = fmaf(wt, v, o[k]);
            }
        }
    }
    if (lane == 0) { s_m[w] = m; s_l[w] = l; }
#pragma unroll
    for (int k = 0; k < CPL; ++k) s_o[w][lane + 32 * k] = o[k];
    __syncthreads();
    float M = -INFINITY, L = 0.f;
    for (int k = 0; k < kWarps; ++k) M = fmaxf(M, s_m[k]);
    const float ref = M == -INFINITY ? 0.f : M;
    for (int k = 0; k < kWarps; ++k) L += s_l[k] * tq_exp2(s_m[k] - ref);
    for (int e = threadIdx.x; e < c.d; e += kWarps * 32) {
        float a = 0.f;
        for (int k = 0; k < kWarps; ++k) a += s_o[k][e] * tq_exp2(s_m[k] - ref);
        p.out[qrow + e] = L == 0.f ? 0.f : a / L;
    }
    if (p.acc_out && threadIdx.x == 0)
        p.lse[(s * c.n_kv + h) * (int64_t)(p.n_q * p.g) + row] = L == 0.f ? INFINITY : ref + log2f(L);
}

// acc_out[t] = decay * acc_in[t] + sum over rows of 2^(logit - lse), rows in order: one thread per
// token, so nothing is added atomically. With a selection a table in shared memory says which of
// its entries holds a block.
constexpr int kAccTok = 256;
__global__ void __launch_bounds__(kAccTok) k_b8_acc(const __grid_constant__ B8AttnParams p, int64_t tiles) {
    const B8Cache& c = p.c;
    const int64_t sh = blockIdx.x / tiles, s = sh / c.n_kv;
    const int n = b8_len(c, s), nfull = n >> 5, rows = p.n_q * p.g;
    const int64_t t0 = (blockIdx.x - sh * tiles) * kAccTok, t = t0 + threadIdx.x;
    if (t0 >= n) return;
    __shared__ int s_at[kAccTok / 32];
    if (p.sel) {
        if (threadIdx.x < kAccTok / 32) s_at[threadIdx.x] = t0 / 32 + threadIdx.x == nfull ? p.n_sel : -1;
        __syncthreads();
        for (int u = threadIdx.x; u < p.n_sel; u += kAccTok) {
            const int b = p.sel[sh * p.n_sel + u] - (int)(t0 / 32);
            if (b >= 0 && b < kAccTok / 32 && b + t0 / 32 < nfull) s_at[b] = u;
        }
        __syncthreads();
    }
    if (t >= n) return;
    const int64_t at = sh * c.max_blocks * 32 + t;
    float a = p.acc_in && t < n - p.n_q ? p.decay * p.acc_in[at] : 0.f;
    const int u = p.sel ? s_at[threadIdx.x >> 5] : (int)(t >> 5);
    if (u >= 0) {
        const float* lg = p.logits + sh * rows * p.logit_row + (int64_t)u * 32 + (t & 31);
        float w = 0.f;
        for (int r = 0; r < rows; ++r) {
            const float e = p.lse[sh * rows + r];
            if (e != INFINITY) w += tq_exp2(lg[r * p.logit_row] - e);
        }
        a += w;
    }
    p.acc_out[at] = a;
}

}  // namespace

cudaError_t b8_launch_attention(const B8AttnParams& p, cudaStream_t st) {
    const int64_t grid = p.c.n_seq * p.n_q * p.c.n_kv * p.g;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (p.c.D == 64) k_b8_attn<64><<<(unsigned)grid, kWarps * 32, 0, st>>>(p);
    else if (p.c.D == 128) k_b8_attn<128><<<(unsigned)grid, kWarps * 32, 0, st>>>(p);
    else k_b8_attn<256><<<(unsigned)grid, kWarps * 32, 0, st>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !p.acc_out) return e;
    const int64_t tiles = (p.c.max_blocks * 32 + kAccTok - 1) / kAccTok;
    if (tiles * p.c.n_seq * p.c.n_kv > 0x7fffffffLL) return cudaErrorInvalidValue;
    k_b8_acc<<<(unsigned)(tiles * p.c.n_seq * p.c.n_kv), kAccTok, 0, st>>>(p, tiles);
    return cudaGetLastError();
}
