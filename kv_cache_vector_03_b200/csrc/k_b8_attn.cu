// Decode attention over the paged 8-bit cache (tq_b8_attention).
//
// Mathematics. With key codes c_t (scale s), value codes v_t (scale u), l_t = s <q, c_t> scale log2(e) and a reference m,
//   o = sum_t 2^(l_t - m) u v_t / sum_t 2^(l_t - m)
// over 32-token blocks, m following the largest logit (online softmax; only when it is passed by 2^6, which changes
// nothing but the exponents' range).
//
// Work is a list of units: a 32-token block, or 16 tokens of an open block, for one (sequence, kv head, tile of 8 or 16
// query rows). Query rows (query token, head of the group) share their kv head's units, so codes are read once for a
// tile. The list is written down nowhere: the CTAs of one wave each sum the lengths, take their share and walk it, so
// lengths stay on the device (a captured graph follows them) and ragged batches are balanced. A segment is the units of
// one sequence, head and tile; parts of a segment that lie in several CTAs are joined by the CTA that brings the last.
//
// Streams. Pages come by bulk copies (64 D + 16 bytes) into a ring of a CTA's stages, the warps taking units in turn;
// every wait has a limit.
//
// Products, tokens as the M dimension so that 8 query rows cost one n-tile:
//   S^T = K Q^T in int8: the stored bytes are unsigned, code + 128; q is scaled by a power of two per row to 22 bits and
//     split into three int8 pieces; sums are exact in int32, start at -128 sum(q piece), and become floats through the
//     bits of 1.5 * 2^23. No key is converted. (fp16 products of converted keys cost 170 instructions a unit where
//     this costs 90.) 22 bits below a row's largest element hold bf16 exactly down to 2^-14 of it; what is cut off moves a
//     logit by up to scale 2^-22 max |q| sum |k|.
//   O^T += V^T P^T in fp16: a byte permute into 1024 + (code + 128) and a subtraction of 1152 make exact fp16 codes. The
//     weights are two fp16 pieces: one alone is off by 2^-12, which an fp32 result shows. Each block's sum is scaled by
//     u into fp32 registers. The pieces hold 22 bits of a weight down to 2^-12 of the one at m; below, they are off by
//     2^-34 of that. So m goes by tokens that have a value: one whose value codes are all zeros (an attention sink) may pass it
//     by 2^80 and counts in the denominator alone. (With m at a sink 20 nats above 8192 tokens, what these add up to was
//     off by 7e-4 of itself, and lost from 23 nats on.)
// Key scale and softmax scale are one product kept in two floats and applied next to m, so a logit is off by little more
// than the rounding of its whole-number sum to fp32, 2^-24 of it.
//
// fp32 work goes two at a time (f2_*, rounded the same): 64 x 8192 181 -> 174 us.
//
// What bounds it: HBM for large calls (64 sequences x 8192 tokens, 8 kv heads, 4 heads a group, D = 128: 1.08 GB in 177 to
// 187 us in short runs, 0.93 to 0.88 of the measured copy rate, and 197, 0.83, in a long run at the power limit); for small
// ones the fixed chain launch, lengths, page table, page, unit, meeting of the warps (one sequence of 500 tokens: 13 us; of
// 32768: 25 us, 10 of them HBM); instructions where 16 query rows share little data. A unit takes 647 warp instructions at 8
// rows. The tensor pipes are busy 16 % (fp16) and 12 % (int8) of the time, so the warp-level matrix instructions do not
// bind. (tcgen05 could take four pages as its 128 rows and q's pieces as 24 columns: nothing gained where HBM binds, untried for
// many query rows, where the instructions do.)
#include <algorithm>
#include <cfloat>

#include "b8_shares.h"
#include "k_b8.cuh"

namespace {

constexpr uint32_t kWaitLimit = 1u << 22;
constexpr float kBias = 9.f;         // weights are kept as 2^(9 + logit - m),
constexpr float kSlack = 6.f;        // m follows the maximum once it is passed by 2^6: 2^(9 + 6) < 65504
constexpr float kSink = 80.f;        // tokens whose values are all zeros may pass m by 2^80
constexpr float kMost = kBias + kSlack + kSink;
// units a CTA takes at least, where segments are shared (one sequence of 8192 tokens: with 4 21.2 us, 8 18.6; 16 ragged ones
// of 1500: with 8 20.5 us, 16 28.7)
constexpr int kMinUnits = 8;
// segments up to here are not shared (one sequence of 1024 tokens: with 32 16.4 us, 16 14.4; of 500: 14.3 and 15.6; 16 ragged
// ones of 600: 16.4 and 18.5)
constexpr int kWholeUnits = 32;
constexpr int kStraddle = 24;        // price of a cut inside a CTA's share, in units (10000 cycles)
constexpr int kGroup = 16;           // parts that are joined at a time, where there are many
constexpr int kAccTok = 128;        // threads of a CTA that adds up weights

// Two CTAs share an SM, so that one computes while the other starts or joins a segment (one CTA of 16 warps: 205 us for
// 64 x 8192; two of 8: 199). Warps and ring stages of one of them, and in how many rounds its warps' sums meet in shared
// memory. Warps: as many as spill next to nothing (64 x 8192 at D = 128, 8 rows: 6 warps 180 us, 7 with more spilled 199, 8
// 193, and 4 or 5 no better than 6; at D = 64 8 warps 115 us, 6 125).
constexpr int kCtasPerSm = 2;
template <int D, int NT>
struct Shape {
    static constexpr int warps = D == 256 || NT * D == 256 ? 4 : D == 128 ? 6 : 8;
    static constexpr int stages = D == 64 ? 20 : D == 128 ? 10 : 5;
    static constexpr int stage_bytes = 64 * D + 128;   // keys, values, scales
    static constexpr int rounds = NT * D == 64 ? 1 : NT * D == 128 ? 2 : D == 256 ? 2 : 4;
    static constexpr size_t smem = (size_t)stages * stage_bytes + (size_t)warps * 8 * NT * (D / rounds + 4) * 4;
};

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
// The accumulator comes in and goes out separately, so that a chain starts from any register (or zero); not
// volatile, so that chains interleave.
#define B8_MMA(NAME, KIND, T, R)                                                                                        \
    TQ_DEVICE void NAME(T (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1, T c0,  \
                        T c1, T c2, T c3) {                                                                             \
        asm("mma.sync.aligned." KIND " {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"                        \
            : "=" R(d[0]), "=" R(d[1]), "=" R(d[2]), "=" R(d[3])                                                        \
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), R(c0), R(c1), R(c2), R(c3));                        \
    }                                                                                                                   \
    TQ_DEVICE void NAME(T (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {      \
        NAME(d, a0, a1, a2, a3, b0, b1, d[0], d[1], d[2], d[3]);                                                        \
    }
B8_MMA(mma_f16, "m16n8k16.row.col.f32.f16.f16.f32", float, "f")
B8_MMA(mma_bf16, "m16n8k16.row.col.f32.bf16.bf16.f32", float, "f")
B8_MMA(mma_u8s8, "m16n8k32.row.col.s32.u8.s8.s32", int, "r")
#undef B8_MMA
TQ_DEVICE uint32_t atomic_add_acq_rel(uint32_t* at, uint32_t v) {
    uint32_t old;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(old) : "l"(at), "r"(v) : "memory");
    return old;
}

// ------------------------------------------------------------------------ the list of units
// "virtual sequences": a sequence, or with a selection one query token of it. The host has checked that (blocks + 1) x
// segments is at most 2^30; a segment has at most two units more than blocks, so there are at most 3 * 2^29 units.
template <bool SP>
TQ_DEVICE int virt_units(const B8AttnParams& p, int v, int& n) {
    const int s = SP && p.n_q > 1 ? v / p.n_q : v;
    n = b8_len(p.c, s);
    const int open = ((n & 31) + 15) / 16;
    if (!SP) return (n >> 5) + open;
    return n - p.n_q + (v - s * p.n_q) < 0 ? 0 : p.n_sel + open;
}
struct Plan {
    int mine;                    // how many units this CTA has,
    int virt, x;                 // from unit x of virtual sequence virt on
    int c0, c1;                  // the CTAs that share this CTA's only segment, or c0 = -1: ask owner()
    int before;                  // (then) the price of all virtual sequences before virt
    B8Shares shares;             // (and) the equal shares
};
// Sums the units of all virtual sequences and finds this CTA's share of them, one of three ways:
//   short segments (up to kWholeUnits units), or so many that whole ones come out even: shares begin and end
//     between segments, nothing is joined;
//   no more segments than CTAs: each segment is cut into parts, a CTA each, in proportion to its length or evened out. A CTA
//     with parts of two segments would pay for a second start and end (about 5 us, kStraddle units), and
//     everyone would wait for it;
//   else equal shares of a price (b8_shares.h), cut where they fall. A begun segment costs its queries and the meeting
//     of the warps beside its units.
// Up to 32 virtual sequences: every warp for itself, a lane each; more: the block, a thread each, tile by tile.
template <int THREADS, bool SP>
TQ_DEVICE void make_plan(const B8AttnParams& p, int n_virt, int segs, Plan& pl) {
    constexpr int NW = THREADS / 32;
    __shared__ int s_sum[NW], s_max[NW], s_at[2][4];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const bool small = n_virt <= 32;
    const int me = small ? lane : (int)threadIdx.x;
    int all;                                         // the sum over the tile
    auto scan = [&](int x) {                         // inclusive sum up to this thread
        int incl = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (small) {
            all = __shfl_sync(0xffffffffu, incl, 31);
            return incl;
        }
        __syncthreads();
        if (lane == 31) s_sum[w] = incl;
        __syncthreads();
        const int sw = lane < NW ? s_sum[lane] : 0;
        all = (int)__reduce_add_sync(0xffffffffu, sw);
        return incl + (int)__reduce_add_sync(0xffffffffu, lane < w ? sw : 0);
    };
    auto units_of = [&](int v) {
        int n;
        return v < n_virt ? virt_units<SP>(p, v, n) : 0;
    };
    // the thread for which `mine` holds hands its values to all of its warp or block
    auto hand = [&](bool mine, int k, int x, int y, int z, int t) {
        if (small) {
            const uint32_t who = __ballot_sync(0xffffffffu, mine);
            if (who) {
                const int src = __ffs(who) - 1;
                x = __shfl_sync(0xffffffffu, x, src);
                y = __shfl_sync(0xffffffffu, y, src);
                z = __shfl_sync(0xffffffffu, z, src);
                t = __shfl_sync(0xffffffffu, t, src);
            }
            return make_int4(x, y, z, t);
        }
        if (mine) {
            s_at[k][0] = x;
            s_at[k][1] = y;
            s_at[k][2] = z;
            s_at[k][3] = t;
        }
        __syncthreads();
        return make_int4(s_at[k][0], s_at[k][1], s_at[k][2], s_at[k][3]);
    };
    int total = 0, longest = 0, units = 0, incl = 0, filled = 0;   // filled: virtual sequences that have units
#pragma unroll 1
    for (int v0 = 0; v0 < n_virt; v0 += small ? 32 : THREADS) {
        units = units_of(v0 + me);
        longest = max(longest, units);
        incl = scan(units * segs);
        total += all;
        filled += small ? __popc(__ballot_sync(0xffffffffu, units > 0)) : __syncthreads_count(units > 0);
    }
    longest = (int)__reduce_max_sync(0xffffffffu, longest);
    pl.mine = 0;
    pl.c0 = -1;
    if (total == 0) return;
    if (!small) {
        if (lane == 0) s_max[w] = longest;
        __syncthreads();
        longest = (int)__reduce_max_sync(0xffffffffu, lane < NW ? s_max[lane] : 0);
    }
    const bool one = n_virt <= THREADS;              // units and incl are this thread's virtual sequence's
    const int n_segs = n_virt * segs;
    const bool whole = longest <= kWholeUnits ||
                       (n_segs > p.grid && (n_segs + p.grid - 1) / p.grid * longest <= total / p.grid + kStraddle);
    if (!whole && n_segs <= p.grid && one) {
        // 1 + floor(units spare / total) parts each are never more than the grid together. Where that leaves parts well
        // above the average and there are CTAs to spare: the smallest cap on a part's units that they can keep, to 1/64
        // (30 ragged sequences of 2000: 33 us by the first rule, 29.7; the search itself costs 1 us).
        const int spare = max(0, min(p.grid, total / kMinUnits) - n_segs), most = n_segs + spare;
        int parts = units ? 1 + (int)((uint32_t)units * (uint32_t)spare / (uint32_t)total) : 0;
        if (small && 8 * spare >= n_segs) {
            int cap = (int)__reduce_max_sync(0xffffffffu, units ? (units + parts - 1) / parts : 0), low = total / most;
            if (cap - low > kB8Segment) {
#pragma unroll 1
                while (cap - low > 1 + (cap >> 6)) {             // cap can be kept, low cannot
                    const int mid = (low + cap) >> 1;
                    if ((int)__reduce_add_sync(0xffffffffu, (units + mid - 1) / mid * segs) <= most) cap = mid;
                    else low = mid;
                }
                parts = (units + cap - 1) / cap;
            }
        }
        const int upto = scan(parts * segs), b = blockIdx.x;
        const bool far = units > parts * (total / p.grid + kStraddle);
        if (!(small ? __any_sync(0xffffffffu, far) : __syncthreads_or(far))) {
            if (b >= all) return;
            const bool mine = upto - parts * segs <= b && b < upto;
            const int pp = max(parts, 1), j = b - (upto - parts * segs), seg = j / pp, part = j - seg * pp;
            const int wide = units / pp, extra = units - wide * pp;
            const int4 x = hand(mine, 0, me, seg * units + part * wide + min(part, extra), wide + (part < extra ? 1 : 0), 0);
            const int4 y = hand(mine, 1, b - part, b - part + parts - 1, 0, 0);
            pl.virt = x.x;
            pl.x = x.y;
            pl.mine = x.z;
            pl.c0 = y.x;
            pl.c1 = y.y;
            return;
        }
    }
    const int ctas = min(p.grid, whole ? min(total, n_segs) : max(1, total / kMinUnits));
    pl.shares.make(total, segs * filled, ctas);
    const int per = pl.shares.per, price = pl.shares.price(total, segs * filled);
    if ((int)blockIdx.x >= ctas) return;
    const int lo = pl.shares.share(blockIdx.x), hi = pl.shares.share(blockIdx.x + 1);
    int4 start = make_int4(0, 0, 0, 0), end = make_int4(0, 0, total, 0);   // virtual sequence, its unit, units before, price before
#pragma unroll 1
    for (int v0 = 0, base = 0, base_price = 0;; v0 += THREADS) {
        if (!one) {
            units = units_of(v0 + me);
            incl = scan(units * segs);
        }
        const int here = one ? total : all, mine = units ? units + per : 0, upto = scan(mine * segs);
        const int first = upto - mine * segs;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int u = (k ? hi : lo) - base_price;
            if (u < 0 || u >= all) continue;             // not in this tile
            const bool is = first <= u && u < upto;
            const int seg = is ? (u - first) / mine : 0, off = is ? max(0, u - first - seg * mine - per) : 0;
            const int x = seg * units + (whole ? 0 : off);
            (k ? end : start) = hand(is, k, v0 + me, x, base + incl - units * segs + x, base_price + first);
        }
        base += here;
        base_price += all;
        if (base_price > hi || base_price >= price) break;
    }
    pl.virt = start.x;
    pl.x = start.y;
    pl.mine = end.z - start.z;
    pl.before = start.w;
}

template <int D>
TQ_DEVICE int channel(int gq, int mt, int y) {   // the channel of row gq + 8 y of O^T's m-tile mt
    return D == 256 ? 16 * (gq + 8 * (mt >> 3)) + 2 * (mt & 7) + y : gq * (D / 8) + 2 * mt + y;
}

// a unit's page: where its codes and its scales are; or half of an open block: where its keys and values are
struct __align__(8) Record {
    const uint8_t* a;
    const uint8_t* b;
    int what;                                        // 0 a page, -1 nothing, -2, -3 a half of the open block
    int block;
};

template <int D, int NT, bool WT, bool SP>
__global__ void __launch_bounds__(Shape<D, NT>::warps * 32, kCtasPerSm) k_b8_attn(const __grid_constant__ B8AttnParams p) {
    using Sh = Shape<D, NT>;
    constexpr int NW = Sh::warps, ST = Sh::stages, SB = Sh::stage_bytes, RD = Sh::rounds;
    constexpr int MT = D / 16;           // m-tiles of O^T
    constexpr int VW = D / 32;           // value words (4 channels) of a lane per token
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t s_full[ST];
    __shared__ int2 s_meta[ST];                      // what a stage holds, and its block
    __shared__ int s_unit[ST];                       // and of which unit
    __shared__ Record s_rec[NW][32];
    __shared__ float2 s_ml[8 * NT][NW];              // the warps' maxima and sums
    __shared__ float s_fac[8 * NT][NW], s_top[8 * NT], s_sum[8 * NT], s_f[8 * NT];
    __shared__ int s_last;
    __shared__ uint2 s_q[NT * 3 * (D / 32) * 32];     // q as B fragments, three int8 pieces
    __shared__ int s_qsum[3][8 * NT];                // -128 times the sum of a row's piece, + the bits of 1.5 * 2^23
    float* s_o = reinterpret_cast<float*>(smem + (size_t)ST * SB);
    const B8Cache& c = p.c;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
    if (threadIdx.x < ST) {
        tq_mbar_init(&s_full[threadIdx.x], 1);
        s_unit[threadIdx.x] = -1;
    }
    tq_fence_mbar_init();
    __syncthreads();                                 // every warp issues copies into the ring: it is set up by now
    tq_pdl_launch_dependents();
    tq_pdl_wait();                                   // nothing is read before the kernel in front is done

    const int segs = c.n_kv * p.row_tiles;
    const int n_virt = (int)(SP ? c.n_seq * p.n_q : c.n_seq);
    const int rows = SP ? p.g : p.n_q * p.g;      // query rows of a virtual sequence and kv head
    auto q_row = [&](int v, int h, int r) {
        const int t = SP ? 0 : r / p.g;           // query token within the virtual sequence
        return ((int64_t)v * (SP ? 1 : p.n_q) + t) * c.n_kv * p.g + h * p.g + r - t * p.g;
    };
    Plan pl;
    make_plan<NW * 32, SP>(p, n_virt, segs, pl);
    // rows of sequences without a token are zeros
#pragma unroll 1
    for (int v = blockIdx.x; v < n_virt; v += gridDim.x) {
        int n;
        if (virt_units<SP>(p, v, n) == 0) {
#pragma unroll 1
            for (int hr = w; hr < c.n_kv * rows; hr += NW) {
                float* out = p.out + q_row(v, hr / rows, hr % rows) * c.d;
                for (int e = lane; e < c.d; e += 32) out[e] = 0.f;
                if (WT && lane == 0) p.norm[(int64_t)v * c.n_kv * rows + hr] = make_float2(0.f, 0.f);
            }
        }
    }
    const int mine = pl.mine;
    if (mine <= 0) return;
    // (what is not needed before a segment's end waits in shared memory)
    __shared__ Plan s_plan;
    __shared__ int s_before;
    if (threadIdx.x == 0) {
        s_plan = pl;
        s_before = pl.before;
    }

    // Unit i of the share goes to warp i mod NW and stage i mod ST; who has consumed a stage refills it with
    // unit i + ST. The k-th unit that this warp issues is a(k) = w + NW k for the first `early` ones, which it
    // issues before it has consumed any, then w + ST + NW (k - early). Lane l looks up a(l), a(l + 32), ..., whose
    // records stand in rec[k mod 32]; 16 at a time are looked up when the 16 before them have been used.
    const int early = (ST - w + NW - 1) / NW;
    int fi = lane < early ? w + NW * lane : w + ST + NW * (lane - early), fv = pl.virt, fx = pl.x + fi;
    Record* rec = s_rec[w];
    auto fetch = [&](int to) {
        Record r = {nullptr, nullptr, -1, 0};
        if (fi < mine) {
            int n, units;
#pragma unroll 1
            while (fx >= (units = virt_units<SP>(p, fv, n)) * segs && fv + 1 < n_virt) {
                fx -= units * segs;
                ++fv;
            }
            const int seg = fx / units, off = fx - seg * units, pages = SP ? p.n_sel : n >> 5;
            const int h = p.row_tiles == 1 ? seg : seg / p.row_tiles, s = SP && p.n_q > 1 ? fv / p.n_q : fv;
            if (off >= pages) {
                const uint16_t* k = b8_open(c, s, h, 0) + 16 * (off - pages) * c.d;
                r = {reinterpret_cast<const uint8_t*>(k), reinterpret_cast<const uint8_t*>(k + 32 * c.d), -2 - (off - pages),
                     n >> 5};
            } else {
                r.block = SP ? p.sel[((int64_t)fv * c.n_kv + h) * p.n_sel + off] : off;
                if (r.block >= 0 && r.block < (n >> 5)) {
                    const uint8_t* page = b8_page(c, c.table[(int64_t)s * c.max_blocks + r.block]);
                    if (page) r = {page + c.header_bytes + (size_t)h * (64 * D), page + (size_t)h * (32 + 2 * D), 0, r.block};
                }
            }
        }
        rec[lane] = r;
        fx += to - fi;
        fi = to;
    };
    bool ok = true;                                  // no wait of this warp has run out
    int issued = 0;
    auto issue = [&](int i, int st) {                // i = a(issued), st = i mod ST
        if (!ok || i >= mine) return;
        if ((issued & 15) == 0) {
            const bool all = issued == 0;
            __syncwarp();
            if (all || (lane >> 4) == ((issued >> 4) - 1 & 1)) fetch(all ? w + ST + NW * (32 + lane - early) : fi + 32 * NW);
            __syncwarp();
        }
        if (lane == 0) {
            const Record r = rec[issued & 31];
            s_meta[st] = make_int2(r.what, r.block);
            *const_cast<volatile int*>(&s_unit[st]) = i;
            uint8_t* dst = smem + (size_t)st * SB;
            if (r.what == -1)
                tq_mbar_arrive(&s_full[st]);
            else if (r.what == 0)
                tq_bulk_load2(dst, r.a, 64 * D, dst + 64 * D, r.b, 16, &s_full[st]);
            else
                tq_bulk_load2(dst, r.a, 32 * c.d, dst + 32 * D, r.b, 32 * c.d, &s_full[st]);
        }
        ++issued;
    };

    int i = w, v = pl.virt, x0 = pl.x;               // i: this warp's next unit, in stage st
    int st = w % ST;
    uint32_t phase = 0;
    // where a lane's values (tokens 2 tq, 2 tq + 1) lie in a page; 8 tokens on is 8 D on
    const uint32_t sv0 = b8_swz(2 * tq, D / 16), sv1 = b8_swz(2 * tq + 1, D / 16);
    const uint32_t vch = D == 64 ? gq >> 1 : gq, vhalf = D == 64 ? (gq & 1) * 8 : 0;
    // ldmatrix: lane l gives the row address of token l mod 16, chunk l / 16 (of a pair; pair x is 32 x bytes on, an
    // exclusive or since the swizzle is one)
    const uint32_t at_k = (lane & 15) * D + (((lane >> 4) ^ b8_swz(lane & 15, D / 16)) << 4);
    const uint32_t at_v0 = 32 * D + 2 * tq * D + ((vch ^ sv0) << 4) + vhalf;
    const uint32_t at_v1 = 32 * D + (2 * tq + 1) * D + ((vch ^ sv1) << 4) + vhalf;
    for (int u = 0; u < mine;) {
        int n, units;
#pragma unroll 1
        while (x0 >= (units = virt_units<SP>(p, v, n)) * segs && v + 1 < n_virt) {
            x0 -= units * segs;
            if (threadIdx.x == 0 && units) s_before += (units + s_plan.shares.per) * segs;
            ++v;
        }
        const int seg = x0 / units, off = x0 - seg * units;
        const int part = min(units - off, mine - u);
        const int h = p.row_tiles == 1 ? seg : seg / p.row_tiles, row0 = (seg - h * p.row_tiles) * 8 * NT;
        const int s = SP && p.n_q > 1 ? v / p.n_q : v;
        const int all_see = n - p.n_q + (SP ? v - s * p.n_q : 0);          // every row sees the positions up to here

        if (u == 0) {
#pragma unroll 1
            for (int k = 0; k < early; ++k) issue(w + NW * k, w + NW * k);
        }
        // q, while the first pages are on their way: a warp per row, a lane per 4 channels. A row is scaled by a
        // power of two to between 2^21 and 2^22 and rounded to whole numbers, which three int8 pieces hold.
#pragma unroll 1
        for (int r = w; r < 8 * NT; r += NW) {
            constexpr int Q4 = D == 256 ? 2 : 1;
            float4 q[Q4];
            uint32_t top = 0;
            const int64_t at = row0 + r < rows ? q_row(v, h, row0 + r) * c.d : 0;
#pragma unroll
            for (int k = 0; k < Q4; ++k) {
                const int e = 4 * (lane + 32 * k);
                q[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (row0 + r < rows && e < c.d) {
                    if (p.q_dtype) {
                        const uint2 x = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.q) + at + e);
                        q[k] = make_float4(bf_lo(x.x), bf_hi(x.x), bf_lo(x.y), bf_hi(x.y));
                    } else {
                        q[k] = *reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + at + e);
                    }
                }
                top = max(max(top, max(__float_as_uint(q[k].x) & 0x7fffffffu, __float_as_uint(q[k].y) & 0x7fffffffu)),
                          max(__float_as_uint(q[k].z) & 0x7fffffffu, __float_as_uint(q[k].w) & 0x7fffffffu));
            }
            top = __reduce_max_sync(0xffffffffu, top);
            const int eb = min(max((int)(top >> 23), 27), 254);
            // 2^(148 - eb), or 0 for a row that is not finite, which answers NaN
            const float up = top >= 0x7f800000u ? 0.f : __uint_as_float((uint32_t)(275 - eb) << 23);
            int sum[3] = {0, 0, 0};
#pragma unroll
            for (int k = 0; k < Q4; ++k) {
                const float f[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
                uint32_t word[3] = {0u, 0u, 0u};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int x = __float2int_rn(f[j] * up), hi = (x + 32896) >> 16, y = x - (hi << 16);
                    const int piece[3] = {hi, (y + 128) >> 8, y - (((y + 128) >> 8) << 8)};
#pragma unroll
                    for (int z = 0; z < 3; ++z) {
                        word[z] |= (uint32_t)(piece[z] & 0xff) << (8 * j);
                        sum[z] += piece[z];
                    }
                }
                // channels 4 id .. + 3: k-step id / 8, register id / 4 mod 2, lane id mod 4
                const int id = lane + 32 * k;
                if (id < D / 4)
#pragma unroll
                    for (int z = 0; z < 3; ++z)
                        reinterpret_cast<uint32_t*>(s_q)[((((r >> 3) * 3 + z) * (D / 32) + (id >> 3)) * 32 + (r & 7) * 4 + (id & 3)) *
                                                             2 + (id >> 2 & 1)] = word[z];
            }
#pragma unroll
            for (int z = 0; z < 3; ++z) sum[z] = (int)__reduce_add_sync(0xffffffffu, sum[z]);
            if (lane < 3) s_qsum[lane][r] = 0x4b400000 - 128 * (lane == 0 ? sum[0] : lane == 1 ? sum[1] : sum[2]);
            if (lane == 0) s_f[r] = up == 0.f ? NAN : __uint_as_float((uint32_t)(eb - 21) << 23);
        }
        __syncthreads();
        float fh[NT][2], fl[NT][2];      // logits factor (key scale aside) of rows 2 tq, 2 tq + 1
        float m[NT][2], l[NT][2], o[MT][NT][4];
        bool big = false;                // some |m| is beyond 2^16
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float f = s_f[8 * nt + 2 * tq + e];
                fh[nt][e] = f * p.scale_hi;
                fl[nt][e] = f * p.scale_lo;
                m[nt][e] = -INFINITY;
                l[nt][e] = 0.f;
            }
        int sees[NT][2];                   // the last position that these rows see
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) sees[nt][e] = SP ? all_see : all_see + (row0 + 8 * nt + 2 * tq + e) / p.g;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.f;

        // this lane's first logit of a row's first token, if logits are wanted
        float* lg = WT ? p.logits + (((int64_t)s * c.n_kv + h) * (p.n_q * p.g) + row0 + 2 * tq) * p.logit_row + gq : nullptr;
        for (; i < u + part; i += NW) {
            // The barrier's parity tells one phase from the next, not from the one after: unit i has to be the
            // stage's before its phase is waited for, since the warp that refills it may be far behind.
            for (uint32_t it = 0; ok && *const_cast<volatile int*>(&s_unit[st]) != i; ++it) ok = it < kWaitLimit;
            ok = __all_sync(0xffffffffu, ok && tq_mbar_wait(&s_full[st], phase, kWaitLimit));
            const int what = ok ? s_meta[st].x : -1, b = ok ? s_meta[st].y : 0;
            // where in a row of logits this unit's are
            const int at = off + i - u, pages = SP ? p.n_sel : n >> 5, col = at < pages ? 32 * at : 32 * pages + 16 * (at - pages);
            // (an open half is 16 tokens, and nothing only where a wait has run out)
            if (WT && what == -1)
                for (int r = 0; r < 8 * NT && row0 + r < rows; ++r) {
                    float* to = p.logits + (((int64_t)s * c.n_kv + h) * (p.n_q * p.g) + row0 + r) * p.logit_row;
                    if (at < pages || lane < 16) to[col + lane] = -INFINITY;
                    if (lane == 0) to[p.ref_at + at] = 0.f;
                }
            if (what != -1) {
                float sc[2][NT][4];                           // S^T: tokens 16 mt + gq (+ 8), rows 2 tq, 2 tq + 1
                const uint8_t* kp = smem + (size_t)st * SB;
                const uint8_t* vp = kp + 32 * D;
                float ks = 1.f, vs = 1.f;
                const int half = -2 - what;                   // of the open block
                const int left = what >= 0 ? 32 : min(16, (n & 31) - 16 * half), pos0 = what >= 0 ? 32 * b : 32 * b + 16 * half;
                if (what >= 0) {
                    const float2 kv = *reinterpret_cast<const float2*>(kp + 64 * D);
                    ks = kv.x;
                    vs = kv.y;
                    int acc[3][2][NT][4];                     // [piece][token half]: the codes are unsigned, code + 128
#pragma unroll
                    for (int x = 0; x < D / 32; ++x) {        // 32 channels: chunks 2 x, 2 x + 1
                        uint32_t k[2][4];
                        const uint32_t ka = tq_smem_addr(kp) + (at_k ^ (32 * x));
                        tq_ldsm_x4(ka, k[0][0], k[0][1], k[0][2], k[0][3]);
                        tq_ldsm_x4(ka + 16 * D, k[1][0], k[1][1], k[1][2], k[1][3]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int z = 0; z < 3; ++z) {
                                const uint2 q = s_q[((nt * 3 + z) * (D / 32) + x) * 32 + lane];
#pragma unroll
                                for (int mt = 0; mt < 2; ++mt) {
                                    if (x == 0) {
                                        const int2 y = *reinterpret_cast<const int2*>(&s_qsum[z][8 * nt + 2 * tq]);
                                        mma_u8s8(acc[z][mt][nt], k[mt][0], k[mt][1], k[mt][2], k[mt][3], q.x, q.y, y.x, y.y, y.x,
                                                 y.y);
                                    } else {
                                        mma_u8s8(acc[z][mt][nt], k[mt][0], k[mt][1], k[mt][2], k[mt][3], q.x, q.y);
                                    }
                                }
                            }
                    }
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; e += 2) {  // sums below 2^22: the low bits of 1.5 * 2^23 + sum
                                float2 x[3];
#pragma unroll
                                for (int z = 0; z < 3; ++z)
                                    x[z] = f2_add(make_float2(__int_as_float(acc[z][mt][nt][e]), __int_as_float(acc[z][mt][nt][e + 1])),
                                                  f2(-12582912.f));
                                const float2 y = f2_fma(x[0], f2(65536.f), f2_fma(x[1], f2(256.f), x[2]));
                                sc[mt][nt][e] = y.x;
                                sc[mt][nt][e + 1] = y.y;
                            }
                } else {
                    // 16 tokens of the open block in bf16; q put together again and split into bf16 pieces, which
                    // three hold. Rows behind the last token hold anything and count as zeros.
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) sc[mt][nt][e] = 0.f;
#pragma unroll 1
                    for (int y = 0; y < D / 16; ++y) {        // 4 channels e0 .. + 3
                        const int e0 = 16 * y + 4 * tq;
                        uint2 k0 = make_uint2(0u, 0u), k1 = k0;
                        if (gq < left && e0 < c.d) k0 = *reinterpret_cast<const uint2*>(kp + (gq * c.d + e0) * 2);
                        if (gq + 8 < left && e0 < c.d) k1 = *reinterpret_cast<const uint2*>(kp + ((gq + 8) * c.d + e0) * 2);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                            for (int z = 0; z < 3; ++z) {
                                const uint32_t word =
                                    reinterpret_cast<const uint32_t*>(s_q)[(((nt * 3 + z) * (D / 32) + (y >> 1)) * 32 + lane) * 2 + (y & 1)];
#pragma unroll
                                for (int j = 0; j < 4; ++j) a[j] = fmaf(a[j], 256.f, (float)(int8_t)(word >> (8 * j)));
                            }
#pragma unroll
                            for (int pc = 0; pc < 3; ++pc) {
                                const uint32_t b0 = pack_bf2(a[0], a[1]), b1 = pack_bf2(a[2], a[3]);
                                a[0] -= bf_lo(b0); a[1] -= bf_hi(b0); a[2] -= bf_lo(b1); a[3] -= bf_hi(b1);
                                mma_bf16(sc[0][nt], k0.x, k1.x, k0.y, k1.y, b0, b1);
                            }
                        }
                    }
                }
                // logits, running maximum, weights
                const bool masked = left < 32 || pos0 + 31 > all_see;
                auto gone = [&](int nt, int e, int t) { return gq + 8 * t >= left || pos0 + gq + 8 * t > sees[nt][e]; };
                float2 ga[NT], gb[NT];                        // of rows 2 tq, 2 tq + 1
                float top[NT][2];
                bool grown = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float2 f = make_float2(fh[nt][0], fh[nt][1]);
                    ga[nt] = f2_mul(f, f2(ks));
                    gb[nt] = f2_fma(make_float2(fl[nt][0], fl[nt][1]), f2(ks), f2_fma(f, f2(ks), make_float2(-ga[nt].x, -ga[nt].y)));
                    float2 y[4];                                                 // of token gq + 8 t
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        y[t] = f2_mul(make_float2(sc[t >> 1][nt][2 * (t & 1)], sc[t >> 1][nt][2 * (t & 1) + 1]), ga[nt]);
                    if (masked) {
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            if (gone(nt, 0, t)) y[t].x = -INFINITY;
                            if (gone(nt, 1, t)) y[t].y = -INFINITY;
                        }
                    }
                    top[nt][0] = fmaxf(fmaxf(y[0].x, y[1].x), fmaxf(y[2].x, y[3].x));
                    top[nt][1] = fmaxf(fmaxf(y[0].y, y[1].y), fmaxf(y[2].y, y[3].y));
                    grown = grown || top[nt][0] > m[nt][0] + kSlack || top[nt][1] > m[nt][1] + kSlack;
                }
                uint32_t zeros = 0;                           // which tokens' values are all zeros, where it matters
                if (__any_sync(0xffffffffu, grown)) {
                    if (what >= 0) {
                        // token `lane`: channels 0 .. 3, which seldom are zeros all, before the rest
                        const uint8_t* row = vp + lane * D;
                        const uint32_t four = *reinterpret_cast<const uint32_t*>(row + (b8_swz(lane, D / 16) << 4));
                        zeros = __ballot_sync(0xffffffffu, four == 0x80808080u);
                        if (zeros) {
                            bool none = four == 0x80808080u;
#pragma unroll 1
                            for (int k = 0; none && k < D / 16; ++k) {
                                const uint4 a = *reinterpret_cast<const uint4*>(row + ((k ^ (lane & (D / 16 - 1))) << 4));
                                none = (a.x & a.y & a.z & a.w) == 0x80808080u && (a.x | a.y | a.z | a.w) == 0x80808080u;
                            }
                            zeros = __ballot_sync(0xffffffffu, none);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    top[nt][e] = -INFINITY;
#pragma unroll
                                    for (int t = 0; t < 4; ++t) {
                                        const float y = __fmul_rn(sc[t >> 1][nt][2 * (t & 1) + e], e ? ga[nt].y : ga[nt].x);
                                        if (!(masked && gone(nt, e, t))) top[nt][e] = fmaxf(top[nt][e], zeros >> (gq + 8 * t) & 1u ? y - kSink : y);
                                    }
                                }
                        }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float t = top[nt][e];
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, d));
                            t = fmaxf(m[nt][e], ceilf(t));        // whole numbers: no difference of two of them is rounded
                            const float f = m[nt][e] == -INFINITY ? 0.f : tq_exp2(m[nt][e] - t);
                            m[nt][e] = t;
                            big = big || (fabsf(t) >= 65536.f && t != -INFINITY);
                            l[nt][e] *= f;
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt) {
                                o[mt][nt][e] *= f;
                                o[mt][nt][2 + e] *= f;
                            }
                        }
                    big = __any_sync(0xffffffffu, big);
                }
                if (big) {
                    // Beyond 2^16 exact logits pass the rounded ones, from which m comes, by more than a weight could show: take
                    // the rounded ones.
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
#pragma unroll
                            for (int t = 0; t < 4; ++t) {
                                float& x = sc[t >> 1][nt][2 * (t & 1) + e];
                                const float mm = m[nt][e] == -INFINITY ? 0.f : m[nt][e];
                                x = __fadd_rn(__fsub_rn(__fmul_rn(x, e ? ga[nt].y : ga[nt].x), mm), kBias);
                                if (x > kMost) x = kMost;       // (y - kSink may have been rounded to y - 128; NaN stays)
                            }
                } else {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float2 ref = make_float2(kBias - (m[nt][0] == -INFINITY ? 0.f : m[nt][0]),
                                                       kBias - (m[nt][1] == -INFINITY ? 0.f : m[nt][1]));
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            float* x = &sc[t >> 1][nt][2 * (t & 1)];
                            const float2 v2 = make_float2(x[0], x[1]), y = f2_fma(v2, gb[nt], f2_fma(v2, ga[nt], ref));
                            x[0] = y.x;
                            x[1] = y.y;
                        }
                    }
                }
                if (masked) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
#pragma unroll
                            for (int t = 0; t < 4; ++t)
                                if (gone(nt, e, t)) sc[t >> 1][nt][2 * (t & 1) + e] = -INFINITY;
                }
                if (WT) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float* to = lg + col + 8 * nt * p.logit_row;
#pragma unroll
                        for (int t = 0; t < 4; ++t)
                            if (what >= 0 || t < 2) {                            // (an open half is 16 tokens)
                                if (row0 + 8 * nt + 2 * tq < rows) to[8 * t] = sc[t >> 1][nt][2 * (t & 1)];
                                if (row0 + 8 * nt + 2 * tq + 1 < rows) to[p.logit_row + 8 * t] = sc[t >> 1][nt][2 * (t & 1) + 1];
                            }
                        to += p.ref_at + at - col;
                        if (gq == 0 && row0 + 8 * nt + 2 * tq < rows) to[0] = m[nt][0] == -INFINITY ? 0.f : m[nt][0];
                        if (gq == 0 && row0 + 8 * nt + 2 * tq + 1 < rows) to[p.logit_row] = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        float* x = &sc[t >> 1][nt][2 * (t & 1)];
                        x[0] = tq_exp2(x[0]);
                        x[1] = tq_exp2(x[1]);
                        const float2 y = f2_add(make_float2(l[nt][0], l[nt][1]), make_float2(x[0], x[1]));
                        l[nt][0] = y.x;
                        l[nt][1] = y.y;
                    }
                if (zeros) {                                  // their weights may pass fp16, and have nothing to weigh
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int t = 0; t < 4; ++t)
                            if (zeros >> (gq + 8 * t) & 1u) sc[t >> 1][nt][2 * (t & 1)] = sc[t >> 1][nt][2 * (t & 1) + 1] = 0.f;
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
                                const float2 t = unpack_h2(hi), rest = f2_add(make_float2(a, b2), make_float2(-t.x, -t.y));
                                pf[y][nt][0][e] = transpose8(hi);
                                pf[y][nt][1][e] = transpose8(pack_h2(rest.x, rest.y));
                            }
#pragma unroll
                    for (int z = 0; z < VW / 2; ++z) {        // 8 channels of a lane at a time
                        uint32_t vw[8][2];                    // tokens 16 y + 2 tq, + 1, + 8, + 9
#pragma unroll
                        for (int t = 0; t < 8; ++t) {
                            const uint2 a = *reinterpret_cast<const uint2*>(
                                kp + (t & 1 ? at_v1 : at_v0) + (16 * (t >> 2) + 8 * (t >> 1 & 1)) * D + (z & 1) * 8 +
                                (z >> 1) * 128);
                            vw[t][0] = a.x; vw[t][1] = a.y;
                        }
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            float acc[2][NT][4];
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const uint32_t v0 = vw[4 * y][x], v1 = vw[4 * y + 1][x];
                                const uint32_t v8 = vw[4 * y + 2][x], v9 = vw[4 * y + 3][x];
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
                                        const uint32_t p0 = pf[y][nt][pc][0], p1 = pf[y][nt][pc][1];
                                        if (y == 0 && pc == 0) {
                                            mma_f16(acc[0][nt], a0, a1, a2, a3, p0, p1, 0.f, 0.f, 0.f, 0.f);
                                            mma_f16(acc[1][nt], b0, b1, b2, b3, p0, p1, 0.f, 0.f, 0.f, 0.f);
                                        } else {
                                            mma_f16(acc[0][nt], a0, a1, a2, a3, p0, p1);
                                            mma_f16(acc[1][nt], b0, b1, b2, b3, p0, p1);
                                        }
                                    }
                            }
#pragma unroll
                            for (int j = 0; j < 2; ++j)
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                    for (int e = 0; e < 4; e += 2) {
                                        float* y = &o[2 * (2 * z + x) + j][nt][e];
                                        const float2 v2 = f2_fma(f2(vs), make_float2(acc[j][nt][e], acc[j][nt][e + 1]),
                                                                 make_float2(y[0], y[1]));
                                        y[0] = v2.x;
                                        y[1] = v2.y;
                                    }
                        }
                    }
                } else {
                    // open block: bf16 values, three bf16 pieces of the weights. A value that is not finite must
                    // not meet the zero weight of a row that does not see its token: then token by token.
                    bool wild = false;
                    for (int t = lane; t < left * c.d / 8; t += 32) {
                        const uint4 a = reinterpret_cast<const uint4*>(vp)[t];
                        const uint32_t u4[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            wild = wild || (u4[y] & 0x7f80u) == 0x7f80u || (u4[y] & 0x7f800000u) == 0x7f800000u;
                    }
                    if (!__any_sync(0xffffffffu, wild)) {
                        uint32_t pf[NT][3][2];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float a = sc[0][nt][2 * e], b2 = sc[0][nt][2 * e + 1];
#pragma unroll
                                for (int pc = 0; pc < 3; ++pc) {
                                    const uint32_t t = pack_bf2(a, b2);
                                    a -= bf_lo(t);
                                    b2 -= bf_hi(t);
                                    pf[nt][pc][e] = transpose8(t);
                                }
                            }
#pragma unroll
                        for (int x = 0; x < D / 64; ++x) {            // 8 channels of a lane: m-tiles 4 x .. 4 x + 3
                            uint32_t vw[4][4];
#pragma unroll
                            for (int t = 0; t < 4; ++t) {
                                const int tok = 2 * tq + (t & 1) + 8 * (t >> 1), ch = channel<D>(gq, 4 * x, 0);
                                uint4 a = make_uint4(0u, 0u, 0u, 0u);
                                if (tok < left && ch < c.d) a = *reinterpret_cast<const uint4*>(vp + (tok * c.d + ch) * 2);
                                vw[t][0] = a.x; vw[t][1] = a.y; vw[t][2] = a.z; vw[t][3] = a.w;
                            }
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint32_t a0 = __byte_perm(vw[0][j], vw[1][j], 0x5410);
                                const uint32_t a1 = __byte_perm(vw[0][j], vw[1][j], 0x7632);
                                const uint32_t a2 = __byte_perm(vw[2][j], vw[3][j], 0x5410);
                                const uint32_t a3 = __byte_perm(vw[2][j], vw[3][j], 0x7632);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                    for (int pc = 0; pc < 3; ++pc)
                                        mma_bf16(o[4 * x + j][nt], a0, a1, a2, a3, pf[nt][pc][0], pf[nt][pc][1]);
                            }
                        }
                    } else {
#pragma unroll 1
                        for (int t = 0; t < left; ++t)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const float y0 = __shfl_sync(0xffffffffu, sc[0][nt][e], (t & 7) * 4 + tq);
                                    const float y1 = __shfl_sync(0xffffffffu, sc[0][nt][2 + e], (t & 7) * 4 + tq);
                                    const float pr = t < 8 ? y0 : y1;
                                    if (pr == 0.f) continue;
#pragma unroll
                                    for (int mt = 0; mt < MT; ++mt) {
                                        const int ch = channel<D>(gq, mt, 0);
                                        if (ch < c.d) {
                                            const uint32_t v2 = *reinterpret_cast<const uint32_t*>(vp + (t * c.d + ch) * 2);
                                            o[mt][nt][e] = fmaf(pr, bf_lo(v2), o[mt][nt][e]);
                                            o[mt][nt][2 + e] = fmaf(pr, bf_hi(v2), o[mt][nt][2 + e]);
                                        }
                                    }
                                }
                    }
                }
            }
            __syncwarp();                                 // every lane has read the stage
            issue(i + ST, st);
            st += NW;
            if (st >= ST) {
                st -= ST;
                phase ^= 1u;
            }
        }

        // the warps' sums meet: one maximum per row, then a sum over the warps in a fixed order
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], d);
                if (gq == 0) s_ml[8 * nt + 2 * tq + e][w] = make_float2(m[nt][e], l[nt][e]);
            }
        __syncthreads();
        for (int r = w; r < 8 * NT; r += NW) {
            const float2 ml = lane < NW ? s_ml[r][lane] : make_float2(-INFINITY, 0.f);
            const float top = tq_warp_max(ml.x), sum = tq_warp_sum(ml.x == -INFINITY ? ml.y : ml.y * tq_exp2(ml.x - top));
            if (lane < NW) s_fac[r][lane] = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : NAN) : tq_exp2(ml.x - top);
            if (lane == 0) {
                s_top[r] = top;
                s_sum[r] = sum;
            }
        }
        const bool whole = part == units;
        const size_t slot = 2 * (size_t)blockIdx.x + (off == 0 ? 1 : 0);
        constexpr int LC = 2 * MT / RD, RS = 8 * LC + 4;  // channels of a lane per round; a row's pitch
        constexpr int G = NW == 8 ? 2 : 1, items = 8 * NT * 2 * LC;   // G threads share an item
#pragma unroll
        for (int rd = 0; rd < RD; ++rd) {
            if (rd) __syncthreads();
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (row0 + 8 * nt + 2 * tq + e >= rows) continue;
                    float* dst = s_o + (size_t)(w * 8 * NT + 8 * nt + 2 * tq + e) * RS + gq * LC;
#pragma unroll
                    for (int k = 0; k < LC / 4; ++k) {
                        const int mt = rd * (MT / RD) + 2 * k;
                        *reinterpret_cast<float4*>(dst + 4 * k) =
                            make_float4(o[mt][nt][e], o[mt][nt][2 + e], o[mt + 1][nt][e], o[mt + 1][nt][2 + e]);
                    }
                }
            __syncthreads();
            const int xg = threadIdx.x % G;
            for (int t = threadIdx.x / G; t < items; t += NW * 32 / G) {
                const int r = t / (2 * LC), cg = t % (2 * LC) / (LC / 4), c4 = t % (LC / 4) * 4;
                if (row0 + r >= rows) continue;           // (the G threads of an item are neighbours in a warp)
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int y = 0; y < NW / G; ++y) {
                    const int x = xg * (NW / G) + y;
                    const float f = s_fac[r][x];
                    const float4 z = *reinterpret_cast<const float4*>(s_o + (size_t)(x * 8 * NT + r) * RS + cg * LC + c4);
                    if (f != 0.f) {
                        a.x = fmaf(z.x, f, a.x); a.y = fmaf(z.y, f, a.y); a.z = fmaf(z.z, f, a.z); a.w = fmaf(z.w, f, a.w);
                    }
                }
                const uint32_t team = ((1u << G) - 1u) << (lane & ~(G - 1));   // they share r, so all of them come here
#pragma unroll
                for (int d = 1; d < G; d <<= 1) {
                    a.x += __shfl_xor_sync(team, a.x, d); a.y += __shfl_xor_sync(team, a.y, d);
                    a.z += __shfl_xor_sync(team, a.z, d); a.w += __shfl_xor_sync(team, a.w, d);
                }
                const int ch = channel<D>(cg, rd * (MT / RD) + c4 / 2, 0);
                if (xg == 0) {
                    if (whole) {
                        const float sum = s_sum[r], inv = sum == 0.f ? 0.f : 1.f / sum;
                        if (ch < c.d)
                            *reinterpret_cast<float4*>(p.out + q_row(v, h, row0 + r) * c.d + ch) =
                                make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
                    } else {
                        *reinterpret_cast<float4*>(p.part + (slot * 8 * NT + r) * D + ch) = a;
                    }
                }
            }
        }
        float2* norm = p.norm + ((int64_t)s * c.n_kv + h) * (p.n_q * p.g) + row0;
        // (logits below m hold kBias too, and so does the sum)
        auto norm_of = [](float top, float sum) {
            return sum == 0.f ? make_float2(0.f, 0.f) : make_float2(top == -INFINITY ? 0.f : top, 1.f / sum);
        };
        if (threadIdx.x < 8 * NT && row0 + threadIdx.x < rows) {
            const float top = s_top[threadIdx.x], sum = s_sum[threadIdx.x];
            if (!whole)
                *reinterpret_cast<float2*>(p.part_ml + (slot * 8 * NT + threadIdx.x) * 2) = make_float2(top, sum);
            else if (WT)
                norm[threadIdx.x] = norm_of(top, sum);
        }
        __syncthreads();                                  // s_o and the row sums are free again
        if (!whole) {
            // Joining the parts of CTAs c0 .. c1, in their order: the CTA that brings the last one does it. More than
            // 3 kGroup parts are joined in groups of kGroup first, each by the last of its own, into the group's first
            // part, and then the groups; so no CTA adds up more than 3 kGroup. (In one go, 296 parts of 8 rows at D = 256
            // took 90 us.)
            const int per = s_plan.shares.per, start = s_before + seg * (units + per) + per;
            const int c0 = s_plan.c0 >= 0 ? s_plan.c0 : s_plan.shares.owner(start);
            const int c1 = s_plan.c0 >= 0 ? s_plan.c1 : s_plan.shares.owner(start + units - 1);
            const int parts = c1 - c0 + 1;
            const bool two = parts > 3 * kGroup;
#pragma unroll 1
            for (int level = two ? 0 : 1; level < 2; ++level) {
                const bool done = level == 1;
                const int first = done ? c0 : c0 + ((int)blockIdx.x - c0) / kGroup * kGroup, step = done && two ? kGroup : 1;
                const int count = !two ? parts : done ? (parts + kGroup - 1) / kGroup : min(kGroup, c1 - first + 1);
                if (count == 1) continue;                 // (a group of one is its own sum)
                if (threadIdx.x == 0) {
                    // Arrival counts, back at 0 afterwards. The 4-bit fields of CTAs c0 .. c1 - 1 are this segment's alone:
                    // one counts up to 15 parts; where there are more, the group's 15 or 16 fields hold two aligned
                    // 16-bit ones, the first for the group (or all parts), the second for the groups.
                    int bit = 4 * first;
                    uint32_t field = 15u;
                    if (count > 15 || (two && done)) {
                        bit = ((bit + 15) & ~15) + (two && done ? 16 : 0);
                        field = 65535u;
                    }
                    const int sh = bit & 31;
                    const uint32_t got = (atomic_add_acq_rel(p.count + (bit >> 5), 1u << sh) >> sh & field) + 1;
                    s_last = (int)got == count;
                    if (s_last) atomicSub(p.count + (bit >> 5), got << sh);
                }
                __syncthreads();
                if (!s_last) break;
                __threadfence();
                auto slot_of = [&](int k) {                     // of part (or group) k
                    const int x = first + k * step;
                    return 2 * (size_t)x + (x == c0);
                };
                auto ml_at = [&](int k, int r) {                // its maximum and sum; then the factor instead
                    return reinterpret_cast<float2*>(p.part_ml + (slot_of(k) * 8 * NT + r) * 2);
                };
                const int valid = min(8 * NT, rows - row0);
                for (int r = w; r < valid; r += NW) {
                    float2 ml[2];                               // of the first 64 parts; more are read twice
                    float top = -INFINITY, sum = 0.f;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int x = lane + 32 * k;
                        ml[k] = x < count ? __ldcg(ml_at(x, r)) : make_float2(-INFINITY, 0.f);
                        top = fmaxf(top, ml[k].x);
                    }
#pragma unroll 1
                    for (int x = lane + 64; x < count; x += 32) top = fmaxf(top, __ldcg(ml_at(x, r)).x);
                    top = tq_warp_max(top);
                    auto factor = [&](int x, float2 v) {
                        const float y = v.x == -INFINITY ? (v.y == 0.f ? 0.f : NAN) : tq_exp2(v.x - top);
                        __stcg(&ml_at(x, r)->x, y);
                        sum = y == 0.f ? sum : fmaf(v.y, y, sum);
                    };
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if (lane + 32 * k < count) factor(lane + 32 * k, ml[k]);
#pragma unroll 1
                    for (int x = lane + 64; x < count; x += 32) factor(x, __ldcg(ml_at(x, r)));
                    sum = tq_warp_sum(sum);
                    if (lane == 0) {
                        s_top[r] = top;
                        s_sum[r] = sum;
                        if (WT && done) norm[r] = norm_of(top, sum);
                    }
                }
                __syncthreads();
                // 4 rows at a time: thread (part group, 4 channels) adds up every PG-th part, then the groups meet
                constexpr int PG = NW * 32 / (D / 4);
                static_assert(PG * 4 * D * 4 <= NW * 8 * NT * RS * 4, "the groups' sums fit where the warps' did");
                const int pg = threadIdx.x / (D / 4), ch = threadIdx.x % (D / 4) * 4;
#pragma unroll 1
                for (int r0 = 0; r0 < valid; r0 += 4) {
                    float4 a[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) a[r] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
                    for (int x = pg; x < count; x += PG) {
                        float y[4];
                        float4 z[4];
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const bool there = r0 + r < valid;
                            y[r] = there ? __ldcg(&ml_at(x, r0 + r)->x) : 0.f;
                            z[r] = there ? __ldcg(reinterpret_cast<const float4*>(p.part + (slot_of(x) * 8 * NT + r0 + r) * D + ch))
                                         : make_float4(0.f, 0.f, 0.f, 0.f);
                        }
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (y[r] != 0.f) {
                                a[r].x = fmaf(z[r].x, y[r], a[r].x); a[r].y = fmaf(z[r].y, y[r], a[r].y);
                                a[r].z = fmaf(z[r].z, y[r], a[r].z); a[r].w = fmaf(z[r].w, y[r], a[r].w);
                            }
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r) *reinterpret_cast<float4*>(s_o + ((size_t)pg * 4 + r) * D + ch) = a[r];
                    __syncthreads();
                    for (int t = threadIdx.x; t < D; t += NW * 32) {           // (row, 4 channels)
                        const int r = t / (D / 4), e = t % (D / 4) * 4;
                        if (r0 + r >= valid) continue;
                        float4 b = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int x = 0; x < PG; ++x) {
                            const float4 z = *reinterpret_cast<const float4*>(s_o + ((size_t)x * 4 + r) * D + e);
                            b.x += z.x; b.y += z.y; b.z += z.z; b.w += z.w;
                        }
                        const float inv = s_sum[r0 + r] == 0.f ? 0.f : 1.f / s_sum[r0 + r];
                        if (!done)
                            *reinterpret_cast<float4*>(p.part + (slot_of(0) * 8 * NT + r0 + r) * D + e) = b;
                        else if (e < c.d)
                            *reinterpret_cast<float4*>(p.out + q_row(v, h, row0 + r0 + r) * c.d + e) =
                                make_float4(b.x * inv, b.y * inv, b.z * inv, b.w * inv);
                    }
                    __syncthreads();
                }
                if (!done && threadIdx.x < valid)
                    __stcg(ml_at(0, threadIdx.x), make_float2(s_top[threadIdx.x], s_sum[threadIdx.x]));
                __syncthreads();
            }
            __syncthreads();
        }
        u += part;
        x0 += part;
    }
    if (!ok && lane == 0) {
        // a copy did not land in time: record it and give those that may be in flight a bounded time
        tq_raise(c.status, TQ_FLAG_TIMEOUT);
        for (int k = max(w, i - NW * (early + 1)); k < min(i, mine); k += NW)
            tq_mbar_wait(&s_full[k % ST], (uint32_t)(k / ST) & 1u, kWaitLimit);
    }
}

// acc_out[t] = decay * acc_in[t] + sum over rows of 2^(x + (ref - top)) / sum, rows in order, with a token's logit x next to
// its unit's reference ref and the row's reference top: whole numbers, so a weight is as precise as in the value sum,
// however large the logits are. One thread adds up a token, so nothing is added atomically. A thread has kAccPer tokens next
// to each other, which share a reference, and takes four rows at a time, to have that many loads under way (registers for
// them at 8 CTAs an SM; left to itself the compiler takes 32 and waits: one sequence of 4000 tokens 19.9 us instead of 18.0).
// With a selection a table in shared memory says which of its entries holds a block.
constexpr int kAccPer = 4, kAccTile = kAccTok * kAccPer;
__global__ void __launch_bounds__(kAccTok, 8) k_b8_acc(const __grid_constant__ B8AttnParams p, int splits) {
    const B8Cache& c = p.c;
    tq_pdl_launch_dependents();
    tq_pdl_wait();
    const int sh = blockIdx.x / splits, s = sh / c.n_kv;
    const int n = b8_len(c, s), nfull = n >> 5, rows = p.n_q * p.g;
    const float2* norm = p.norm + (int64_t)sh * rows;
    const int64_t at = (int64_t)sh * c.max_blocks * 32;
    const bool wide = (((uintptr_t)p.acc_in | (uintptr_t)p.acc_out) & 15) == 0;   // (rows are multiples of 128 bytes)
    __shared__ int s_at[kAccTile / 32];
    for (int t0 = (blockIdx.x - sh * splits) * kAccTile; t0 < n; t0 += splits * kAccTile) {
        if (p.sel) {
            __syncthreads();
            if (threadIdx.x < kAccTile / 32) s_at[threadIdx.x] = t0 / 32 + threadIdx.x == nfull ? p.n_sel : -1;
            __syncthreads();
            for (int u = threadIdx.x; u < p.n_sel; u += kAccTok) {
                const int b = p.sel[(int64_t)sh * p.n_sel + u] - t0 / 32;
                if (b >= 0 && b < kAccTile / 32 && b + t0 / 32 < nfull) s_at[b] = u;
            }
            __syncthreads();
        }
        const int i = kAccPer * threadIdx.x, t = t0 + i;
        if (t >= n) continue;
        const bool all = wide && t + kAccPer <= n - p.n_q;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p.acc_in && all) {
            a = *reinterpret_cast<const float4*>(p.acc_in + at + t);
            a = make_float4(p.decay * a.x, p.decay * a.y, p.decay * a.z, p.decay * a.w);
        } else if (p.acc_in) {
            float* to = &a.x;
#pragma unroll
            for (int k = 0; k < kAccPer; ++k)
                if (t + k < n - p.n_q) to[k] = p.decay * p.acc_in[at + t + k];
        }
        const int u = p.sel ? s_at[i >> 5] : t >> 5;         // where the tokens are in a row of logits
        float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
        if (u >= 0) {
            const bool half = u == (p.sel ? p.n_sel : nfull) && (t & 16);            // the open block's second
            const float* lg = p.logits + (int64_t)sh * rows * p.logit_row;
            const int64_t col = (int64_t)u * 32 + (t & 31), ref = p.ref_at + u + (half ? 1 : 0);
            for (int r0 = 0; r0 < rows; r0 += 4) {
                float2 e[4];
                float4 y[4];
                float d[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int rr = min(r0 + r, rows - 1);            // (a row behind the last counts 0)
                    const float* row = lg + rr * p.logit_row;
                    e[r] = norm[rr];
                    y[r] = *reinterpret_cast<const float4*>(row + col);
                    d[r] = row[ref];
                    if (r0 + r >= rows) e[r].y = 0.f;
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float down = d[r] - e[r].x;
                    w.x = fmaf(tq_exp2(y[r].x + down), e[r].y, w.x);
                    w.y = fmaf(tq_exp2(y[r].y + down), e[r].y, w.y);
                    w.z = fmaf(tq_exp2(y[r].z + down), e[r].y, w.z);
                    w.w = fmaf(tq_exp2(y[r].w + down), e[r].y, w.w);
                }
            }
        }
        w = make_float4(a.x + w.x, a.y + w.y, a.z + w.z, a.w + w.w);
        if (wide && t + kAccPer <= n) {
            *reinterpret_cast<float4*>(p.acc_out + at + t) = w;
        } else {
            const float v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < kAccPer; ++k)
                if (t + k < n) p.acc_out[at + t + k] = v[k];
        }
    }
}

template <int D, int NT, bool WT, bool SP>
cudaError_t launch_one(const B8AttnParams& p, cudaStream_t st) {
    using Sh = Shape<D, NT>;
    static TqLaunchCache cache;
    const cudaError_t e = tq_kernel_setup(k_b8_attn<D, NT, WT, SP>, Sh::warps * 32, Sh::smem, cache, nullptr, nullptr);
    if (e != cudaSuccess) return e;
    return tq_launch_pdl(k_b8_attn<D, NT, WT, SP>, dim3((unsigned)p.grid), dim3(Sh::warps * 32), Sh::smem, st, p);
}
template <int D, int NT>
cudaError_t launch(const B8AttnParams& p, cudaStream_t st) {
    if (p.sel) return p.acc_out ? launch_one<D, NT, true, true>(p, st) : launch_one<D, NT, false, true>(p, st);
    return p.acc_out ? launch_one<D, NT, true, false>(p, st) : launch_one<D, NT, false, false>(p, st);
}

}  // namespace

// Two n-tiles a unit where both are full and there is much to read: they share the conversion of the values and the
// traffic of the pages, at the price of fewer warps (registers). 16 query rows over 64 x 8192 tokens: 284 us, in two
// tiles of 8 346 us; over 16 x 8192 99 and 99; over 4 x 4000 41 and 28. 24 rows at D = 64 with two tiles, the second
// half empty: 44 us, in three of 8 39. `blocks`: what the cache can hold (or a selection names), over all kv heads.
int b8_attn_row_tile(int D, int rows, int64_t blocks) {
    return D <= 128 && rows > 8 && (rows + 7) / 8 % 2 == 0 && blocks >= 32768 ? 16 : 8;
}
int b8_attn_grid() { return std::min(kCtasPerSm * tq_device_sms(), 2 * kB8Counters); }

cudaError_t b8_launch_attention(const B8AttnParams& p, cudaStream_t st) {
    const int64_t virt = p.sel ? p.c.n_seq * p.n_q : p.c.n_seq;
    // the kernel counts units in 31 bits (and their price, b8_shares.h)
    const int64_t most = (p.sel ? p.n_sel : p.c.max_blocks) + 1;
    if (virt * p.c.n_kv * p.row_tiles > 0x3fffffffLL || most * (virt * p.c.n_kv * p.row_tiles) > 0x3fffffffLL)
        return cudaErrorInvalidValue;
    const bool wide = p.row_tile == 16;
    cudaError_t e;
    if (p.c.D == 64) e = wide ? launch<64, 2>(p, st) : launch<64, 1>(p, st);
    else if (p.c.D == 128) e = wide ? launch<128, 2>(p, st) : launch<128, 1>(p, st);
    else e = launch<256, 1>(p, st);
    if (e != cudaSuccess || !p.acc_out) return e;
    // one CTA per tile of tokens; fewer, which go on, where the capacity gives many more than 32 an SM
    const int64_t rows = p.c.n_seq * p.c.n_kv, tiles = (p.c.max_blocks * 32 + kAccTile - 1) / kAccTile;
    const int64_t splits = std::max<int64_t>(1, std::min(tiles, 32 * (int64_t)tq_device_sms() / rows));
    return tq_launch_pdl(k_b8_acc, dim3((unsigned)(rows * splits)), dim3(kAccTok), 0, st, p, (int)splits);
}
