// Decode attention over the paged 8-bit cache (tq_b8_attention).
//
// Work is a list of units: a unit is one 32-token block of one (sequence, kv head, tile of query
// rows), and a sequence's open block is its last unit. Query rows (query token, head of the
// group) that share a kv head share its units, so codes are read once for up to 8 NT rows. The
// list is laid out in memory by nobody: every CTA of one persistent wave sums the lengths, takes an
// equal contiguous share and walks it, so batches of any mixture of lengths are balanced. A
// segment (the units of one sequence, head and tile) that lies in one CTA is finished there; parts of
// a segment go to the workspace and k_b8_merge joins them in order.
//
// A warp takes every kWarps-th unit of its CTA's share and streams pages through a ring of its own
// in shared memory with bulk copies (64 D + 16 bytes a unit), the page numbers of 32 units ahead
// in its lanes' registers. Products run on the fp16 tensor cores with tokens as the M dimension,
// so 8 query rows cost one n-tile: S^T = K Q^T and O^T += V^T P^T. Codes become exact fp16 values by
// a byte permute into 1024 + (code + 128) and one subtraction of 1152. q is scaled by a power of two per
// row and split into fp16 pieces: one holds a bf16 q exactly, two hold 22 bits of an fp32 q. Weights
// are split into two fp16 pieces too: one piece alone is off by 2^-12, which an fp32 output shows.
// Scales multiply after the products: the key scale on the logits (as a product kept in two
// floats, so that large logits lose nothing), the value scale on each block's partial sum.
#include <cfloat>

#include "k_b8.cuh"

namespace {

constexpr uint32_t kWaitLimit = 1u << 22;
constexpr float kBias = 7.f;         // weights are kept as 2^(7 + logit - m): their small pieces stay normal in fp16
constexpr float kSlack = 8.f;        // m follows the maximum once it is passed by 2^8: 2^(7 + 8) < 65504
constexpr int kMinUnits = 8;         // units a CTA takes at least
constexpr int kAccTok = 256;

template <int D>
struct Ring {
    static constexpr int warps = D == 256 ? 4 : 8;
    static constexpr int stages = D == 64 ? 4 : 2;
    static constexpr int stage_bytes = 64 * D + 128;   // keys, values, scales
};
template <int D, int NT>
constexpr size_t smem_bytes() {
    return (size_t)Ring<D>::warps * (Ring<D>::stages * Ring<D>::stage_bytes + 8 * NT * D * 4);
}

TQ_DEVICE uint32_t h2sub(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// bytes SEL of w, each code + 128, as two exact fp16 codes
template <int SEL>
TQ_DEVICE uint32_t codes_h2(uint32_t w) { return h2sub(__byte_perm(w, 0x64646464u, SEL), 0x64806480u); }

TQ_DEVICE uint32_t pack_h2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
TQ_DEVICE uint32_t pack_bf2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
TQ_DEVICE float2 unpack_h2(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }
TQ_DEVICE float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
TQ_DEVICE float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
TQ_DEVICE uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
TQ_DEVICE void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ------------------------------------------------------------------------ the list of units
// "virtual sequences": a sequence, or with a selection one query token of it
struct Plan {
    int64_t total, u0, u1, n_virt;
    int ctas;
};
TQ_DEVICE int virt_units(const B8AttnParams& p, int64_t v, int& n) {
    if (!p.sel) {
        n = b8_len(p.c, v);
        return (n >> 5) + ((n & 31) ? 1 : 0);
    }
    n = b8_len(p.c, v / p.n_q);
    return n - p.n_q + (int)(v % p.n_q) < 0 ? 0 : p.n_sel + ((n & 31) ? 1 : 0);
}
template <int THREADS>
TQ_DEVICE int64_t block_scan(int64_t x, int64_t* s, int64_t& total) {   // inclusive; s: THREADS / 32 words
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) s[w] = x;
    __syncthreads();
    total = 0;
    int64_t before = 0;
#pragma unroll
    for (int k = 0; k < THREADS / 32; ++k) {
        if (k < w) before += s[k];
        total += s[k];
    }
    return x + before;
}
TQ_DEVICE int64_t share(const Plan& pl, int c) { return pl.total * c / pl.ctas; }
TQ_DEVICE int owner(const Plan& pl, int64_t u) { return (int)(((u + 1) * pl.ctas - 1) / pl.total); }

template <int THREADS>
TQ_DEVICE void plan_total(const B8AttnParams& p, Plan& pl, int64_t* s) {
    pl.n_virt = p.sel ? p.c.n_seq * p.n_q : p.c.n_seq;
    pl.total = 0;
    for (int64_t v0 = 0; v0 < pl.n_virt; v0 += THREADS) {
        const int64_t v = v0 + threadIdx.x;
        int n;
        int64_t sum;
        block_scan<THREADS>(v < pl.n_virt ? (int64_t)virt_units(p, v, n) * p.c.n_kv * p.row_tiles : 0, s, sum);
        pl.total += sum;
    }
    const int64_t most = (pl.total + kMinUnits - 1) / kMinUnits;
    pl.ctas = (int)(most < p.grid ? (most > 1 ? most : 1) : p.grid);
}

template <int D, int NT, int QP>
__global__ void __launch_bounds__(Ring<D>::warps * 32, 1) k_b8_attn(const __grid_constant__ B8AttnParams p) {
    constexpr int NW = Ring<D>::warps, ST = Ring<D>::stages, SB = Ring<D>::stage_bytes;
    constexpr int KC = D / 64;           // 16-byte key chunks of a lane per token
    constexpr int MT = D / 16;           // m-tiles of O^T
    constexpr int VW = D / 32;           // value words (4 channels) of a lane per token
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t s_full[NW * ST];
    __shared__ int64_t s_scan[NW], s_start[2];
    __shared__ float s_m[NW][8 * NT], s_l[NW][8 * NT];
    const B8Cache& c = p.c;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
    uint8_t* ring = smem + (size_t)w * ST * SB;
    float* s_o = reinterpret_cast<float*>(smem + (size_t)NW * ST * SB);
    if (lane < ST) tq_mbar_init(&s_full[w * ST + lane], 2);
    tq_fence_mbar_init();
    tq_pdl_launch_dependents();

    Plan pl;
    plan_total<NW * 32>(p, pl, s_scan);
    if ((int)blockIdx.x >= pl.ctas || pl.total == 0) return;
    pl.u0 = share(pl, blockIdx.x);
    pl.u1 = share(pl, blockIdx.x + 1);
    const int segs = c.n_kv * p.row_tiles;
    {
        int64_t base = 0;
        for (int64_t v0 = 0; v0 < pl.n_virt; v0 += NW * 32) {
            const int64_t v = v0 + threadIdx.x;
            int n;
            int64_t sum;
            const int64_t x = v < pl.n_virt ? (int64_t)virt_units(p, v, n) * segs : 0;
            const int64_t before = base + block_scan<NW * 32>(x, s_scan, sum) - x;
            if (before <= pl.u0 && pl.u0 < before + x) {
                s_start[0] = v;
                s_start[1] = pl.u0 - before;
            }
            base += sum;
            if (base > pl.u0) break;
        }
        __syncthreads();
    }

    // this warp's units, NW apart: lane l of a batch holds where unit 32 batch + l lies
    int64_t fv = s_start[0], fx = s_start[1] + w + NW * lane, fu = pl.u0 + w + NW * lane;
    int name = -1, blk = -1, head = 0, next_name = -1, next_blk = -1, next_head = 0;
    auto fetch = [&](int& rname, int& rblk, int& rhead) {
        rname = rblk = -1;
        rhead = 0;
        if (fu < pl.u1) {
            int n, units = virt_units(p, fv, n);
            while (fx >= (int64_t)units * segs) {
                fx -= (int64_t)units * segs;
                units = virt_units(p, ++fv, n);
            }
            const int seg = (int)(fx / units), off = (int)(fx - (int64_t)seg * units);
            const int64_t s = p.sel ? fv / p.n_q : fv;
            rhead = seg / p.row_tiles;
            if ((n & 31) && off == units - 1) {
                rname = -2;
                rblk = n >> 5;
            } else {
                rblk = p.sel ? p.sel[(fv * c.n_kv + rhead) * p.n_sel + off] : off;
                if (rblk >= 0 && rblk < (n >> 5)) {
                    rname = c.table[s * c.max_blocks + rblk];
                    if (rname < 0 || rname >= c.n_pages) {
                        tq_raise(c.status, TQ_FLAG_RANGE);
                        rname = -1;
                    }
                }
            }
        }
        fu += 32 * NW;
        fx += 32 * NW;
    };
    const int mine = (int)((pl.u1 - pl.u0 - w + NW - 1) / NW);   // this warp's units (none: <= 0)
    uint32_t in_flight = 0, phase = 0;                           // a bit per stage
    auto issue = [&](int i) {                                    // i counts up from 0, once each
        if ((i & 31) == 0) {
            if (i == 0) fetch(name, blk, head);
            else { name = next_name; blk = next_blk; head = next_head; }
            fetch(next_name, next_blk, next_head);
        }
        const int nm = __shfl_sync(0xffffffffu, name, i & 31), h = __shfl_sync(0xffffffffu, head, i & 31);
        if (nm < 0) return;
        const int st = i % ST;
        in_flight |= 1u << st;
        if (lane == 0) {
            const uint8_t* page = c.pages + (size_t)nm * c.page_bytes;
            uint8_t* dst = ring + st * SB;
            tq_bulk_load(dst, page + c.header_bytes + (size_t)h * (64 * D), 64 * D, &s_full[w * ST + st]);
            tq_bulk_load(dst + 64 * D, page + (size_t)h * (32 + 2 * D), 16, &s_full[w * ST + st]);
        }
    };
    __syncwarp();
    bool ok = true;                                              // no wait of this warp has run out
    // a batch changes while units of the last one are in flight, so what a unit is stays with its stage
    int kind[ST], where[ST];
    auto stage_in = [&](int i) {
        const int st = i % ST;
        if (ok && i < mine) issue(i);
        const int k = __shfl_sync(0xffffffffu, name, i & 31), b = __shfl_sync(0xffffffffu, blk, i & 31);
#pragma unroll
        for (int x = 0; x < ST; ++x)
            if (x == st) {
                kind[x] = k;
                where[x] = b;
            }
    };
#pragma unroll
    for (int i = 0; i < ST; ++i) stage_in(i);

    int i = 0;
    int64_t v = s_start[0], x0 = s_start[1];
    for (int64_t u = pl.u0; u < pl.u1;) {
        int n, units = virt_units(p, v, n);
        while (x0 >= (int64_t)units * segs) {
            x0 -= (int64_t)units * segs;
            units = virt_units(p, ++v, n);
        }
        const int seg = (int)(x0 / units), off = (int)(x0 - (int64_t)seg * units);
        const int part = (int)min((int64_t)(units - off), pl.u1 - u);
        const int h = seg / p.row_tiles, row0 = (seg - h * p.row_tiles) * 8 * NT;
        const int64_t s = p.sel ? v / p.n_q : v;
        const int first_q = p.sel ? (int)(v - s * p.n_q) : 0;
        const int rows = p.sel ? p.g : p.n_q * p.g;
        const int64_t qbase = (s * p.n_q + first_q) * c.n_kv * p.g + (int64_t)h * p.g;   // row of query row 0
        auto q_row = [&](int r) { return qbase + (int64_t)(r / p.g) * c.n_kv * p.g + r % p.g; };

        // q as B fragments: row gq of each n-tile, channels 16 (tq + 4 c) + 4 k .. + 3
        uint32_t qf[NT][QP][KC * 4][2];
        float fh[NT][2], fl[NT][2];      // logits factor (key scale aside) of rows 2 tq, 2 tq + 1
        int last[NT][2];                 // the last position that these rows see
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = row0 + 8 * nt + gq;
            float q[KC * 16];
            uint32_t top = 0;
            const int64_t at = r < rows ? q_row(r) * c.d : 0;
#pragma unroll
            for (int k = 0; k < KC * 2; ++k) {
                const int e = 16 * (tq + 4 * (k >> 1)) + 8 * (k & 1);
                if (r < rows && e < c.d) {
                    if (QP == 1) {
                        const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + at + e);
                        const uint32_t u4[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            q[8 * k + 2 * j] = bf_lo(u4[j]);
                            q[8 * k + 2 * j + 1] = bf_hi(u4[j]);
                        }
                    } else {
                        const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + at + e);
                        const float4 a = f[0], b = f[1];
                        q[8 * k] = a.x; q[8 * k + 1] = a.y; q[8 * k + 2] = a.z; q[8 * k + 3] = a.w;
                        q[8 * k + 4] = b.x; q[8 * k + 5] = b.y; q[8 * k + 6] = b.z; q[8 * k + 7] = b.w;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) q[8 * k + j] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(q[8 * k + j]) & 0x7fffffffu);
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int eb = max((int)(top >> 23), 27);
            const float up = __uint_as_float((uint32_t)(267 - min(eb, 254)) << 23);      // 2^(140 - eb)
            const float down = __uint_as_float((uint32_t)(min(eb, 254) - 13) << 23);     // 2^(eb - 140)
#pragma unroll
            for (int k = 0; k < KC * 4; ++k)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float a = q[4 * k + 2 * e] * up, b = q[4 * k + 2 * e + 1] * up;
                    qf[nt][0][k][e] = pack_h2(a, b);
                    if (QP == 2) {
                        const float2 t = unpack_h2(qf[nt][0][k][e]);
                        qf[nt][QP - 1][k][e] = pack_h2(a - t.x, b - t.y);
                    }
                }
            const float f0 = eb >= 255 ? NAN : down;     // a row that is not finite answers NaN
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float f = __shfl_sync(0xffffffffu, f0, (2 * tq + e) * 4);
                fh[nt][e] = f * p.scale_hi;
                fl[nt][e] = f * p.scale_lo;
                const int rr = row0 + 8 * nt + 2 * tq + e;
                last[nt][e] = rr < rows ? n - p.n_q + first_q + rr / p.g : -1;
            }
        }
        const int all_see = n - p.n_q + first_q;         // every row sees the positions up to here

        float m[NT][2], l[NT][2], o[MT][NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[nt][e] = -INFINITY;
                l[nt][e] = 0.f;
            }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.f;

        for (int k = (int)((w - (u - pl.u0) % NW + NW) % NW); k < part; k += NW, ++i) {
            const int st = i % ST;
            int what = 0, b = 0;
#pragma unroll
            for (int x = 0; x < ST; ++x)
                if (x == st) {
                    what = kind[x];
                    b = where[x];
                }
            if (what >= 0) {
                ok = ok && __all_sync(0xffffffffu, tq_mbar_wait(&s_full[w * ST + st], phase >> st & 1u, kWaitLimit));
                if (ok) {
                    phase ^= 1u << st;
                    in_flight &= ~(1u << st);
                } else {
                    what = -1;
                }
            }
            float* lg = nullptr;                          // this unit's logits, [row][logit_row], if they are wanted
            if (p.acc_out)
                lg = p.logits + ((s * c.n_kv + h) * (int64_t)(p.n_q * p.g) + row0) * p.logit_row +
                     (int64_t)(p.sel ? off + k : b) * 32;
            float sc[2][NT][4];                           // S^T: tokens 16 mt + gq (+ 8), rows 2 tq, 2 tq + 1
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[mt][nt][e] = 0.f;
            const uint8_t* kp = ring + st * SB;
            const uint8_t* vp = kp + 32 * D;
            float ks = 1.f, vs = 1.f;
            const int r = n & 31;
            if (what >= 0) {
                const float2 kv = *reinterpret_cast<const float2*>(kp + 64 * D);
                ks = kv.x;
                vs = kv.y;
#pragma unroll
                for (int cc = 0; cc < KC; ++cc) {
                    uint4 kw[4];
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        kw[t] = *reinterpret_cast<const uint4*>(
                            kp + (gq + 8 * t) * D + (((tq + 4 * cc) ^ b8_swz(gq + 8 * t, D / 16)) << 4));
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        uint32_t lo[4], hi[4];
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            const uint32_t word = x == 0 ? kw[t].x : x == 1 ? kw[t].y : x == 2 ? kw[t].z : kw[t].w;
                            lo[t] = codes_h2<0x4140>(word);
                            hi[t] = codes_h2<0x4342>(word);
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int qp = 0; qp < QP; ++qp) {
                                const uint32_t* q = qf[nt][qp][cc * 4 + x];
                                tq_hmma(sc[0][nt], lo[0], lo[1], hi[0], hi[1], q[0], q[1]);
                                tq_hmma(sc[1][nt], lo[2], lo[3], hi[2], hi[3], q[0], q[1]);
                            }
                    }
                }
            } else if (what == -2) {
                // open block: bf16 keys; q again in bf16 pieces (1 holds a bf16 q, 3 hold 22 bits)
                const uint16_t* kg = b8_open(c, s, h, 0);
#pragma unroll
                for (int cc = 0; cc < KC; ++cc) {
                    const int e0 = 16 * (tq + 4 * cc);
                    uint32_t kw[4][8];
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            uint4 a = make_uint4(0u, 0u, 0u, 0u);
                            if (gq + 8 * t < r && e0 + 8 * y < c.d)
                                a = *reinterpret_cast<const uint4*>(kg + (gq + 8 * t) * c.d + e0 + 8 * y);
                            kw[t][4 * y] = a.x; kw[t][4 * y + 1] = a.y; kw[t][4 * y + 2] = a.z; kw[t][4 * y + 3] = a.w;
                        }
#pragma unroll
                    for (int x = 0; x < 4; ++x)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float a[4];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float2 t = unpack_h2(qf[nt][0][cc * 4 + x][e]);
                                a[2 * e] = t.x;
                                a[2 * e + 1] = t.y;
                                if (QP == 2) {
                                    const float2 z = unpack_h2(qf[nt][QP - 1][cc * 4 + x][e]);
                                    a[2 * e] += z.x;
                                    a[2 * e + 1] += z.y;
                                }
                            }
#pragma unroll
                            for (int pc = 0; pc < 2 * QP - 1; ++pc) {
                                const uint32_t b0 = pack_bf2(a[0], a[1]), b1 = pack_bf2(a[2], a[3]);
                                a[0] -= bf_lo(b0); a[1] -= bf_hi(b0); a[2] -= bf_lo(b1); a[3] -= bf_hi(b1);
                                mma_bf16(sc[0][nt], kw[0][2 * x], kw[1][2 * x], kw[0][2 * x + 1], kw[1][2 * x + 1], b0, b1);
                                mma_bf16(sc[1][nt], kw[2][2 * x], kw[3][2 * x], kw[2][2 * x + 1], kw[3][2 * x + 1], b0, b1);
                            }
                        }
                }
            }
            // logits, running maximum, weights
            const int left = what == -1 ? 0 : what == -2 ? r : 32;          // tokens of this unit
            const bool masked = left < 32 || 32 * b + 31 > all_see;
            float ga[NT][2], gb[NT][2];
            bool grown = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    ga[nt][e] = fh[nt][e] * ks;
                    gb[nt][e] = fmaf(fh[nt][e], ks, -ga[nt][e]) + fl[nt][e] * ks;
                    float top = -INFINITY;
#pragma unroll
                    for (int t = 0; t < 4; ++t) {                            // token gq + 8 t
                        const float raw = sc[t >> 1][nt][2 * (t & 1) + e];
                        float y = fmaf(raw, ga[nt][e], raw * gb[nt][e]);
                        if (masked && (gq + 8 * t >= left || 32 * b + gq + 8 * t > last[nt][e])) y = -INFINITY;
                        top = fmaxf(top, y);
                        if (lg && row0 + 8 * nt + 2 * tq + e < rows)
                            lg[(8 * nt + 2 * tq + e) * p.logit_row + gq + 8 * t] = y;
                    }
                    grown = grown || top > m[nt][e] + kSlack;
                }
            if (what == -1) {
                stage_in(i + ST);
                continue;
            }
            if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top = m[nt][e];
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            const float raw = sc[t >> 1][nt][2 * (t & 1) + e];
                            float y = fmaf(raw, ga[nt][e], raw * gb[nt][e]);
                            if (masked && (gq + 8 * t >= left || 32 * b + gq + 8 * t > last[nt][e])) y = -INFINITY;
                            top = fmaxf(top, y);
                        }
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                        const float f = m[nt][e] == -INFINITY ? 0.f : tq_exp2(m[nt][e] - top);
                        m[nt][e] = top;
                        l[nt][e] *= f;
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            o[mt][nt][e] *= f;
                            o[mt][nt][2 + e] *= f;
                        }
                    }
            }
            // Beyond 2^16 m itself is rounded by more than a weight could show: subtract the rounded logits
            // there, of which the largest is m exactly.
            bool big = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) big = big || fabsf(m[nt][0]) >= 65536.f || fabsf(m[nt][1]) >= 65536.f;
            big = __any_sync(0xffffffffu, big);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float mm = m[nt][e] == -INFINITY ? 0.f : m[nt][e];
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        float& x = sc[t >> 1][nt][2 * (t & 1) + e];
                        const float small = x * gb[nt][e];
                        float pr = tq_exp2(big ? __fadd_rn(__fsub_rn(fmaf(x, ga[nt][e], small), mm), kBias)
                                               : fmaf(x, ga[nt][e], small + (kBias - mm)));
                        if (masked && (gq + 8 * t >= left || 32 * b + gq + 8 * t > last[nt][e])) pr = 0.f;
                        x = pr;
                        l[nt][e] += pr;
                    }
                }
            if (what >= 0) {
                uint32_t pf[2][NT][2][2];                 // P^T as B fragments: [token half][n-tile][piece][register]
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float a = sc[y][nt][2 * e], b2 = sc[y][nt][2 * e + 1];
                            const uint32_t hi = pack_h2(a, b2);
                            const float2 t = unpack_h2(hi);
                            pf[y][nt][0][e] = transpose8(hi);
                            pf[y][nt][1][e] = transpose8(pack_h2(a - t.x, b2 - t.y));
                        }
                uint32_t vw[8][VW];                       // tokens 16 y + 2 tq, + 1, + 8, + 9
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    const int tok = 16 * (t >> 2) + 2 * tq + (t & 1) + 8 * (t >> 1 & 1);
                    const uint8_t* row = vp + tok * D;
                    if (D == 64) {
                        const uint2 a = *reinterpret_cast<const uint2*>(row + (((gq >> 1) ^ b8_swz(tok, D / 16)) << 4) + (gq & 1) * 8);
                        vw[t][0] = a.x; vw[t][1] = a.y;
                    } else {
#pragma unroll
                        for (int y = 0; y < VW / 4; ++y) {
                            const uint4 a = *reinterpret_cast<const uint4*>(row + (((gq + 8 * y) ^ b8_swz(tok, D / 16)) << 4));
                            vw[t][4 * y] = a.x; vw[t][4 * y + 1] = a.y; vw[t][4 * y + 2] = a.z; vw[t][4 * y + 3] = a.w;
                        }
                    }
                }
#pragma unroll
                for (int x = 0; x < VW; ++x) {
                    float acc[2][NT][4];
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) acc[j][nt][e] = 0.f;
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint32_t v0 = vw[4 * y][x], v1 = vw[4 * y + 1][x], v8 = vw[4 * y + 2][x], v9 = vw[4 * y + 3][x];
                        const uint32_t l0 = __byte_perm(v0, v1, 0x5140), h0 = __byte_perm(v0, v1, 0x7362);
                        const uint32_t l8 = __byte_perm(v8, v9, 0x5140), h8 = __byte_perm(v8, v9, 0x7362);
                        const uint32_t a0 = codes_h2<0x4140>(l0), a1 = codes_h2<0x4342>(l0), a2 = codes_h2<0x4140>(l8),
                                       a3 = codes_h2<0x4342>(l8);
                        const uint32_t b0 = codes_h2<0x4140>(h0), b1 = codes_h2<0x4342>(h0), b2 = codes_h2<0x4140>(h8),
                                       b3 = codes_h2<0x4342>(h8);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int pc = 0; pc < 2; ++pc) {
                                tq_hmma(acc[0][nt], a0, a1, a2, a3, pf[y][nt][pc][0], pf[y][nt][pc][1]);
                                tq_hmma(acc[1][nt], b0, b1, b2, b3, pf[y][nt][pc][0], pf[y][nt][pc][1]);
                            }
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[2 * x + j][nt][e] = fmaf(vs, acc[j][nt][e], o[2 * x + j][nt][e]);
                }
            } else {
                // open block: bf16 values, three bf16 pieces of the weights. A value that is not finite must
                // not meet the zero weight of a row that does not see its token: then token by token.
                const uint16_t* vg = b8_open(c, s, h, 1);
                bool wild = false;
                for (int t = lane; t < r * c.d / 8; t += 32) {
                    const uint4 a = reinterpret_cast<const uint4*>(vg)[t];
                    const uint32_t u4[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        wild = wild || (u4[y] & 0x7f80u) == 0x7f80u || (u4[y] & 0x7f800000u) == 0x7f800000u;
                }
                if (!__any_sync(0xffffffffu, wild)) {
                    uint32_t pf[2][NT][3][2];
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float a = sc[y][nt][2 * e], b2 = sc[y][nt][2 * e + 1];
#pragma unroll
                                for (int pc = 0; pc < 3; ++pc) {
                                    const uint32_t t = pack_bf2(a, b2);
                                    a -= bf_lo(t);
                                    b2 -= bf_hi(t);
                                    pf[y][nt][pc][e] = transpose8(t);
                                }
                            }
#pragma unroll
                    for (int x = 0; x < D / 64; ++x) {            // 8 channels D / 8 gq + 8 x
                        uint32_t vw[8][4];
                        const int e0 = gq * (D / 8) + 8 * x;
#pragma unroll
                        for (int t = 0; t < 8; ++t) {
                            const int tok = 16 * (t >> 2) + 2 * tq + (t & 1) + 8 * (t >> 1 & 1);
                            uint4 a = make_uint4(0u, 0u, 0u, 0u);
                            const int ch = D == 256 ? 16 * (gq + 8 * (x >> 1)) + 8 * (x & 1) : e0;
                            if (tok < r && ch < c.d) a = *reinterpret_cast<const uint4*>(vg + tok * c.d + ch);
                            vw[t][0] = a.x; vw[t][1] = a.y; vw[t][2] = a.z; vw[t][3] = a.w;
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j)               // m-tile 4 x + j: channels + 2 j, + 2 j + 1
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const uint32_t v0 = vw[4 * y][j], v1 = vw[4 * y + 1][j], v8 = vw[4 * y + 2][j],
                                               v9 = vw[4 * y + 3][j];
                                const uint32_t a0 = __byte_perm(v0, v1, 0x5410), a1 = __byte_perm(v0, v1, 0x7632);
                                const uint32_t a2 = __byte_perm(v8, v9, 0x5410), a3 = __byte_perm(v8, v9, 0x7632);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                    for (int pc = 0; pc < 3; ++pc)
                                        mma_bf16(o[4 * x + j][nt], a0, a1, a2, a3, pf[y][nt][pc][0], pf[y][nt][pc][1]);
                            }
                    }
                } else {
                    for (int t = 0; t < r; ++t)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int src = (t & 7) * 4 + tq;
                                const float x0 = __shfl_sync(0xffffffffu, sc[0][nt][e], src);
                                const float x1 = __shfl_sync(0xffffffffu, sc[0][nt][2 + e], src);
                                const float x2 = __shfl_sync(0xffffffffu, sc[1][nt][e], src);
                                const float x3 = __shfl_sync(0xffffffffu, sc[1][nt][2 + e], src);
                                const float pr = t < 8 ? x0 : t < 16 ? x1 : t < 24 ? x2 : x3;
                                if (pr == 0.f) continue;
#pragma unroll
                                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                                    for (int y = 0; y < 2; ++y) {
                                        const int ch = D == 256 ? 16 * (gq + 8 * (mt >> 3)) + 2 * (mt & 7) + y
                                                                : gq * (D / 8) + 2 * mt + y;
                                        if (ch < c.d)
                                            o[mt][nt][2 * y + e] =
                                                fmaf(pr, __uint_as_float((uint32_t)vg[t * c.d + ch] << 16), o[mt][nt][2 * y + e]);
                                    }
                            }
                }
            }
            __syncwarp();                                 // every lane has read the stage
            stage_in(i + ST);
        }

        // the warps' sums meet: one maximum per row, then a sum over the warps in order
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], d);
                if (gq == 0) {
                    s_m[w][8 * nt + 2 * tq + e] = m[nt][e];
                    s_l[w][8 * nt + 2 * tq + e] = l[nt][e];
                }
            }
        __syncthreads();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * nt + 2 * tq + e;
                float top = -INFINITY;
#pragma unroll
                for (int x = 0; x < NW; ++x) top = fmaxf(top, s_m[x][r]);
                const float f = m[nt][e] == -INFINITY ? (l[nt][e] == 0.f ? 0.f : NAN) : tq_exp2(m[nt][e] - top);
                float* dst = s_o + (size_t)(w * 8 * NT + r) * D;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int ch = D == 256 ? 16 * (gq + 8 * (mt >> 3)) + 2 * (mt & 7) + y : gq * (D / 8) + 2 * mt + y;
                        dst[ch] = f == 0.f ? 0.f : o[mt][nt][2 * y + e] * f;
                    }
            }
        __syncthreads();
        const bool whole = part == units;
        const int slot = 2 * blockIdx.x + (off == 0 ? 1 : 0);
        for (int t = threadIdx.x; t < 8 * NT * (D / 4); t += NW * 32) {
            const int r = t / (D / 4), e = t % (D / 4) * 4;
            if (row0 + r >= rows) continue;
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int x = 0; x < NW; ++x) top = fmaxf(top, s_m[x][r]);
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int x = 0; x < NW; ++x) {
                const float4 y = *reinterpret_cast<const float4*>(s_o + (size_t)(x * 8 * NT + r) * D + e);
                a.x += y.x; a.y += y.y; a.z += y.z; a.w += y.w;
                const float mx = s_m[x][r];
                sum += mx == -INFINITY ? s_l[x][r] : s_l[x][r] * tq_exp2(mx - top);
            }
            if (whole) {
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                if (e < c.d)
                    *reinterpret_cast<float4*>(p.out + q_row(row0 + r) * c.d + e) =
                        make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
                if (e == 0 && p.acc_out)
                    p.lse[(s * c.n_kv + h) * (int64_t)(p.n_q * p.g) + row0 + r] =
                        sum == 0.f ? INFINITY : (top == -INFINITY ? 0.f : top) + log2f(sum) - kBias;
            } else {
                *reinterpret_cast<float4*>(p.part + ((size_t)slot * 8 * NT + r) * D + e) = a;
                if (e == 0) {
                    p.part_ml[((size_t)slot * 8 * NT + r) * 2] = top;
                    p.part_ml[((size_t)slot * 8 * NT + r) * 2 + 1] = sum;
                }
            }
        }
        __syncthreads();                                  // s_m and s_o are free again
        u += part;
        x0 += part;
    }
    if (!ok) {
        // a copy did not land in time: record it and give those in flight a bounded time
        if (lane == 0) {
            tq_raise(c.status, TQ_FLAG_TIMEOUT);
            for (int st = 0; st < ST; ++st)
                if (in_flight >> st & 1u) tq_mbar_wait(&s_full[w * ST + st], phase >> st & 1u, kWaitLimit);
        }
    }
}

// Joins the parts of a segment that several CTAs shared, in their order; rows of sequences without
// any token are zeros. One CTA per segment.
constexpr int kMergeThreads = 256;
template <int D, int NT>
__global__ void __launch_bounds__(kMergeThreads) k_b8_merge(const __grid_constant__ B8AttnParams p) {
    __shared__ int64_t s_scan[kMergeThreads / 32];
    const B8Cache& c = p.c;
    const int segs = c.n_kv * p.row_tiles;
    const int64_t v = blockIdx.x / segs;
    const int seg = (int)(blockIdx.x - v * segs), h = seg / p.row_tiles, row0 = (seg - h * p.row_tiles) * 8 * NT;
    Plan pl;
    plan_total<kMergeThreads>(p, pl, s_scan);
    int64_t before = 0;
    for (int64_t v0 = 0; v0 <= v; v0 += kMergeThreads) {
        const int64_t x = v0 + threadIdx.x;
        int n;
        int64_t sum;
        block_scan<kMergeThreads>(x < v ? (int64_t)virt_units(p, x, n) * segs : 0, s_scan, sum);
        before += sum;
    }
    int n;
    const int units = virt_units(p, v, n);
    const int64_t s = p.sel ? v / p.n_q : v;
    const int first_q = p.sel ? (int)(v - s * p.n_q) : 0;
    const int rows = p.sel ? p.g : p.n_q * p.g;
    const int64_t qbase = (s * p.n_q + first_q) * c.n_kv * p.g + (int64_t)h * p.g;
    const int64_t a0 = before + (int64_t)seg * units, a1 = a0 + units;
    const int c0 = units ? owner(pl, a0) : 0, c1 = units ? owner(pl, a1 - 1) : 0;
    tq_pdl_wait();
    if (units && c0 == c1) return;                        // finished where it was computed
    for (int t = threadIdx.x; t < 8 * NT * (D / 4); t += kMergeThreads) {
        const int r = t / (D / 4), e = t % (D / 4) * 4;
        if (row0 + r >= rows) continue;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        float top = -INFINITY, sum = 0.f;
        if (units) {
            for (int x = c0; x <= c1; ++x) {
                const int slot = 2 * x + (share(pl, x) <= a0 ? 1 : 0);
                top = fmaxf(top, p.part_ml[((size_t)slot * 8 * NT + r) * 2]);
            }
            for (int x = c0; x <= c1; ++x) {
                const int slot = 2 * x + (share(pl, x) <= a0 ? 1 : 0);
                const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + ((size_t)slot * 8 * NT + r) * 2);
                const float f = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : NAN) : tq_exp2(ml.x - top);
                if (f == 0.f) continue;
                const float4 y = *reinterpret_cast<const float4*>(p.part + ((size_t)slot * 8 * NT + r) * D + e);
                a.x = fmaf(y.x, f, a.x); a.y = fmaf(y.y, f, a.y); a.z = fmaf(y.z, f, a.z); a.w = fmaf(y.w, f, a.w);
                sum = fmaf(ml.y, f, sum);
            }
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int64_t row = qbase + (int64_t)((row0 + r) / p.g) * c.n_kv * p.g + (row0 + r) % p.g;
        if (e < c.d)
            *reinterpret_cast<float4*>(p.out + row * c.d + e) = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
        if (e == 0 && p.acc_out)
            p.lse[(s * c.n_kv + h) * (int64_t)(p.n_q * p.g) + row0 + r] =
                sum == 0.f ? INFINITY : (top == -INFINITY ? 0.f : top) + log2f(sum) - kBias;
    }
}

// acc_out[t] = decay * acc_in[t] + sum over rows of 2^(logit - lse), rows in order: one thread per
// token, so nothing is added atomically. With a selection a table in shared memory says which of
// its entries holds a block.
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

template <int D, int NT, int QP>
cudaError_t launch(const B8AttnParams& p, cudaStream_t st) {
    static TqLaunchCache cache;
    cudaError_t e = tq_kernel_setup(k_b8_attn<D, NT, QP>, Ring<D>::warps * 32, smem_bytes<D, NT>(), cache, nullptr, nullptr);
    if (e != cudaSuccess) return e;
    k_b8_attn<D, NT, QP><<<(unsigned)p.grid, Ring<D>::warps * 32, smem_bytes<D, NT>(), st>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const int64_t segs = (p.sel ? p.c.n_seq * p.n_q : p.c.n_seq) * p.c.n_kv * p.row_tiles;
    if (segs > 0x7fffffffLL) return cudaErrorInvalidValue;
    return tq_launch_pdl(k_b8_merge<D, NT>, dim3((unsigned)segs), dim3(kMergeThreads), 0, st, p);
}

}  // namespace

int b8_attn_row_tile(int D, int rows) { return rows <= 8 || D == 256 ? 8 : 16; }
int b8_attn_grid() { return tq_device_sms(); }

cudaError_t b8_launch_attention(const B8AttnParams& p, cudaStream_t st) {
    const int64_t virt = p.sel ? p.c.n_seq * p.n_q : p.c.n_seq;
    const int64_t tiles = (p.c.max_blocks * 32 + kAccTok - 1) / kAccTok;
    if (virt * p.c.n_kv * p.row_tiles > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (p.acc_out && tiles * p.c.n_seq * p.c.n_kv > 0x7fffffffLL) return cudaErrorInvalidValue;
    const bool wide = p.row_tile == 16, f32 = p.q_dtype == 0;
    cudaError_t e;
    if (p.c.D == 64) e = wide ? (f32 ? launch<64, 2, 2>(p, st) : launch<64, 2, 1>(p, st)) : (f32 ? launch<64, 1, 2>(p, st) : launch<64, 1, 1>(p, st));
    else if (p.c.D == 128) e = wide ? (f32 ? launch<128, 2, 2>(p, st) : launch<128, 2, 1>(p, st)) : (f32 ? launch<128, 1, 2>(p, st) : launch<128, 1, 1>(p, st));
    else e = f32 ? launch<256, 1, 2>(p, st) : launch<256, 1, 1>(p, st);
    if (e != cudaSuccess || !p.acc_out) return e;
    k_b8_acc<<<(unsigned)(tiles * p.c.n_seq * p.c.n_kv), kAccTok, 0, st>>>(p, tiles);
    return cudaGetLastError();
}
