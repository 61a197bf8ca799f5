// Paged 8-bit cache: tokens in (tq_b8_append), tokens back out (tq_b8_read).
//
// Append. One warp per (sequence, head, keys or values, block that the call touches). A lane holds
// 8 channels of D/8 tokens in registers, so a block is read once: its largest |x| (an integer
// maximum over the bf16 bits, which also shows values that are not finite) gives the scale, then
// every value becomes a code by one fused multiply-add with 1.5 * 2^23 + 128: the sum's rounding is
// the rounding of the exact product to a whole number, halves to even, and its low byte is
// code + 128. The smallest and largest code of a channel are the codes of its smallest and largest
// value, since the map is monotone. The warp of a call's first block reads the open block's
// tokens and then, in program order, writes the tokens that stay open, so no other warp
// touches the open block. Bound by HBM: 64 x 512 tokens of 8 heads (d = 128, bf16), 203 MB in 40 us, 0.78 of the
// measured copy rate.
//
// Read. Codes times scale, in the caller's layout. Bound by HBM: 727 MB (32 sequences of up to 4127 tokens as bf16) in 109 us,
// the measured copy rate; 64 x 543 tokens in 36 us.
#include "k_b8.cuh"

namespace {

constexpr float kRound = 12583040.f;     // 1.5 * 2^23 + 128
constexpr int kAppendWarps = 4;
constexpr int kReadWarps = 8;
constexpr int kReadTok = 8;

// past L1, of memory that this kernel may write later
TQ_DEVICE uint4 load_once(const uint4* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}
// 8 fp32 channels as bf16 pairs
TQ_DEVICE uint4 round8(uint4 a, uint4 b) {
    const __nv_bfloat162 r[4] = {__floats2bfloat162_rn(__uint_as_float(a.x), __uint_as_float(a.y)),
                                 __floats2bfloat162_rn(__uint_as_float(a.z), __uint_as_float(a.w)),
                                 __floats2bfloat162_rn(__uint_as_float(b.x), __uint_as_float(b.y)),
                                 __floats2bfloat162_rn(__uint_as_float(b.z), __uint_as_float(b.w))};
    return *reinterpret_cast<const uint4*>(r);
}
template <bool F32>
TQ_DEVICE uint4 load8(const void* base, int64_t elem) {
    if (!F32) return tq_ldg_stream(static_cast<const uint16_t*>(base) + elem);
    return round8(tq_ldg_stream(static_cast<const float*>(base) + elem), tq_ldg_stream(static_cast<const float*>(base) + elem + 4));
}

TQ_DEVICE uint32_t code2(uint32_t w, float inv) {   // two codes + 128 in the low two bytes
    const float2 c = f2_fma(make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)), f2(inv), f2(kRound));
    return __byte_perm(__float_as_uint(c.x), __float_as_uint(c.y), 0x0040);
}
TQ_DEVICE uint2 code8(uint4 x, float inv) {
    return make_uint2(__byte_perm(code2(x.x, inv), code2(x.y, inv), 0x5410),
                      __byte_perm(code2(x.z, inv), code2(x.w, inv), 0x5410));
}
TQ_DEVICE uint32_t drop_nonfinite(uint32_t w) {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
    return w;
}
TQ_DEVICE uint32_t bf2_min(uint32_t a, uint32_t b) {
    __nv_bfloat162 r = __hmin2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<uint32_t*>(&r);
}
TQ_DEVICE uint32_t bf2_max(uint32_t a, uint32_t b) {
    __nv_bfloat162 r = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<uint32_t*>(&r);
}

template <int D, bool F32>
__global__ void __launch_bounds__(kAppendWarps * 32) k_b8_append(const __grid_constant__ B8AppendParams p, int nbt) {
    constexpr int CH = D / 8;        // 8-channel chunks of a row; also token steps of a lane
    constexpr int TPI = 32 / CH;     // tokens of one step
    const B8Cache& c = p.c;
    tq_pdl_launch_dependents();
    tq_pdl_wait();
    const int lane = threadIdx.x & 31;
    int64_t id = (int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
    const int h = (int)(id % c.n_kv);
    id /= c.n_kv;
    const int side = (int)(id & 1);
    id >>= 1;
    const int j = (int)(id % nbt);
    const int64_t s = id / nbt;
    if (s >= c.n_seq) return;
    const int n = b8_len(c, s);
    const int64_t add = p.add ? p.add[s] : p.n_new;
    if (add < 0 || add > p.n_new || add > n) {
        if (lane == 0) tq_raise(c.status, TQ_FLAG_RANGE);
        return;
    }
    if (add == 0) return;
    const int first = n - (int)add, b0 = first >> 5, b1 = n >> 5, b = b0 + j;
    const void* src = side ? p.v : p.k;
    uint16_t* open = b8_open(c, s, h, side);
    const int64_t row0 = s * p.seq_stride + (int64_t)h * c.d;
    const int ch = lane % CH, t0 = lane / CH;
    const bool in = ch * 8 < c.d;
    if (b < b1) {
        uint8_t* page = b8_page(c, c.table[s * c.max_blocks + b]);
        // fp32 rows eight at a time, all their loads before the first is rounded (9 x 777 tokens, d = 80: 9.5 us instead
        // of 14.3)
        uint4 x[CH];
        constexpr int STEP = F32 && CH > 8 ? 8 : CH;
#pragma unroll
        for (int i0 = 0; i0 < CH; i0 += STEP) {
            uint4 more[STEP];
#pragma unroll
            for (int i = 0; i < STEP; ++i) {
                const int t = t0 + (i0 + i) * TPI, pos = 32 * b + t;
                x[i0 + i] = more[i] = make_uint4(0u, 0u, 0u, 0u);
                if (in) {
                    const bool old = pos < first;
                    const int64_t at = row0 + (pos - first) * p.tok_stride + ch * 8;
                    const uint4* from = reinterpret_cast<const uint4*>(
                        old ? open + t * c.d + ch * 8 : static_cast<const uint16_t*>(src) + (F32 ? 2 * at : at));
                    x[i0 + i] = load_once(from);
                    if (F32 && !old) more[i] = load_once(from + 1);
                }
            }
#pragma unroll
            for (int i = 0; i < STEP; ++i)
                if (F32 && 32 * b + t0 + (i0 + i) * TPI >= first) x[i0 + i] = round8(x[i0 + i], more[i]);
        }
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < CH; ++i)
            m = __vmaxu2(__vmaxu2(m, __vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu)),
                         __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu));
        m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
        if (m >= 0x7f80u) {
            if (lane == 0) tq_raise(c.status, TQ_FLAG_RANGE);
            m = 0u;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                x[i] = make_uint4(drop_nonfinite(x[i].x), drop_nonfinite(x[i].y), drop_nonfinite(x[i].z),
                                  drop_nonfinite(x[i].w));
                m = __vmaxu2(__vmaxu2(m, __vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu)),
                             __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu));
            }
            m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
        }
        const float a = __uint_as_float(m << 16);
        const bool live = a >= kB8MinMax;
        const float inv = live ? (1.f / a) * 127.f : 0.f, scale = live ? a * kB8Inv127 : 0.f;
        if (page) {
            uint8_t* rows = b8_codes(c, page, h, side);
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int t = t0 + i * TPI;
                *reinterpret_cast<uint2*>(rows + t * D + (((ch >> 1) ^ b8_swz(t, D / 16)) << 4) + (ch & 1) * 8) =
                    code8(x[i], inv);
            }
            uint8_t* e = b8_entry(c, page, h);
            if (lane == 0) *reinterpret_cast<float*>(e + 4 * side) = scale;
            if (side == 0) {
                uint4 lo = x[0], hi = x[0];
#pragma unroll
                for (int i = 1; i < CH; ++i) {
                    lo = make_uint4(bf2_min(lo.x, x[i].x), bf2_min(lo.y, x[i].y), bf2_min(lo.z, x[i].z),
                                    bf2_min(lo.w, x[i].w));
                    hi = make_uint4(bf2_max(hi.x, x[i].x), bf2_max(hi.y, x[i].y), bf2_max(hi.z, x[i].z),
                                    bf2_max(hi.w, x[i].w));
                }
#pragma unroll
                for (int o = CH; o < 32; o <<= 1) {
                    lo = make_uint4(bf2_min(lo.x, __shfl_xor_sync(0xffffffffu, lo.x, o)),
                                    bf2_min(lo.y, __shfl_xor_sync(0xffffffffu, lo.y, o)),
                                    bf2_min(lo.z, __shfl_xor_sync(0xffffffffu, lo.z, o)),
                                    bf2_min(lo.w, __shfl_xor_sync(0xffffffffu, lo.w, o)));
                    hi = make_uint4(bf2_max(hi.x, __shfl_xor_sync(0xffffffffu, hi.x, o)),
                                    bf2_max(hi.y, __shfl_xor_sync(0xffffffffu, hi.y, o)),
                                    bf2_max(hi.z, __shfl_xor_sync(0xffffffffu, hi.z, o)),
                                    bf2_max(hi.w, __shfl_xor_sync(0xffffffffu, hi.w, o)));
                }
                if (lane < CH) {
                    uint2 l8 = code8(lo, inv), h8 = code8(hi, inv);
                    *reinterpret_cast<uint2*>(e + 32 + ch * 8) = make_uint2(l8.x ^ 0x80808080u, l8.y ^ 0x80808080u);
                    *reinterpret_cast<uint2*>(e + 32 + D + ch * 8) = make_uint2(h8.x ^ 0x80808080u, h8.y ^ 0x80808080u);
                }
            }
        }
    }
    if (j == 0 && (n & 31)) {
        __syncwarp();   // every lane has read what the open block held
        if (in)
            for (int pos = max(first, 32 * b1) + t0; pos < n; pos += TPI)
                *reinterpret_cast<uint4*>(open + (pos & 31) * c.d + ch * 8) =
                    load8<F32>(src, row0 + (pos - first) * p.tok_stride + ch * 8);
    }
}

// One warp per (sequence, kReadTok tokens of one block, keys or values, 32 pieces of the heads): a lane takes a piece of
// one head, 16 bytes of the result, for all these tokens, so that that many loads are under way and a warp's stores are
// contiguous. (A lane with 16 channels of 4 tokens, whose stores leave gaps for the next, and a warp for all heads in turn:
// 124 us instead of 109 for 727 MB, 6.7 instead of 4.9 for 64 x 32 tokens.)
template <int D, bool F32>
__global__ void __launch_bounds__(kReadWarps * 32) k_b8_read(const __grid_constant__ B8ReadParams p, int groups, int parts) {
    constexpr int E = F32 ? 4 : 8;                       // channels of a piece
    const B8Cache& c = p.c;
    tq_pdl_launch_dependents();
    tq_pdl_wait();
    const int lane = threadIdx.x & 31;
    const uint32_t warp = blockIdx.x * kReadWarps + (threadIdx.x >> 5), id = warp / (uint32_t)parts;
    const uint32_t i = (warp - id * parts) * 32 + lane, pieces = c.d / E;
    const int side = (int)(id & 1), group = (int)(id >> 1);
    if (group >= groups) return;
    const int64_t s = blockIdx.y;
    const int n = b8_len(c, s);
    const int64_t from = max((int64_t)0, n - p.n_tok);
    const int64_t pos = (from & ~(int64_t)(kReadTok - 1)) + kReadTok * (int64_t)group;   // up to n, its tokens pos, pos + 1, ...
    if (pos >= n) return;
    const int b = (int)(pos >> 5), t0 = (int)(pos & 31);
    const bool paged = b < (n >> 5);
    uint8_t* page = nullptr;
    if (paged && !(page = b8_page(c, c.table[s * c.max_blocks + b]))) return;
    if (i >= c.n_kv * pieces) return;
    const int h = (int)(i / pieces), ch = (int)(i - h * pieces) * E;
    const int64_t tok = (int64_t)c.n_kv * c.d;           // a token's values
    const int64_t at = (s * p.n_tok + pos - (n - p.n_tok)) * tok + (int64_t)i * E;
    void* out = side ? p.v : p.k;
    const int lo = (int)max((int64_t)0, from - pos), hi = (int)min((int64_t)kReadTok, n - pos);   // which of the tokens
    if (paged) {
        const float sc = *reinterpret_cast<const float*>(b8_entry(c, page, h) + 4 * side);
        const uint8_t* codes = b8_codes(c, page, h, side) + (ch & 15);
        uint32_t w[kReadTok][E / 4];
#pragma unroll
        for (int t = 0; t < kReadTok; ++t) {
            const uint8_t* at_c = codes + (t0 + t) * D + (((ch >> 4) ^ b8_swz(t0 + t, D / 16)) << 4);
            if (F32) {
                w[t][0] = __ldcs(reinterpret_cast<const uint32_t*>(at_c));
            } else {
                const uint2 x = __ldcs(reinterpret_cast<const uint2*>(at_c));
                w[t][0] = x.x;
                w[t][E / 4 - 1] = x.y;
            }
        }
#pragma unroll
        for (int t = 0; t < kReadTok; ++t) {
            if (t < lo || t >= hi) continue;
            float f[E];
#pragma unroll
            for (int k = 0; k < E; ++k)
                f[k] = sc * (__uint_as_float(__byte_perm(w[t][k >> 2], 0x4b000000u, 0x7440 + (k & 3))) - 8388736.f);
            uint4 r;
            if (F32) {
                r = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
            } else {
                __nv_bfloat162 y[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) y[k] = __floats2bfloat162_rn(f[2 * k % E], f[(2 * k + 1) % E]);
                r = *reinterpret_cast<uint4*>(y);
            }
            reinterpret_cast<uint4*>(out)[(at + t * tok) / E] = r;
        }
    } else {
        const uint16_t* src = b8_open(c, s, h, side) + t0 * c.d + ch;
#pragma unroll
        for (int t = 0; t < kReadTok; ++t) {
            if (t < lo || t >= hi) continue;
            uint4 r;
            if (F32) {
                const uint2 x = *reinterpret_cast<const uint2*>(src + t * c.d);
                r = make_uint4(x.x << 16, x.x & 0xffff0000u, x.y << 16, x.y & 0xffff0000u);
            } else {
                r = *reinterpret_cast<const uint4*>(src + t * c.d);
            }
            reinterpret_cast<uint4*>(out)[(at + t * tok) / E] = r;
        }
    }
}

}  // namespace

// kern<D, input or output in fp32>(p, more...) as a programmatic dependent of the kernel in front
#define B8_LAUNCH(KERN, GRID, WARPS, ...)                                                                              \
    (p.c.D == 64    ? tq_launch_pdl(p.dtype ? KERN<64, false> : KERN<64, true>, dim3(GRID), dim3(WARPS * 32), 0, st,   \
                                    __VA_ARGS__)                                                                       \
     : p.c.D == 128 ? tq_launch_pdl(p.dtype ? KERN<128, false> : KERN<128, true>, dim3(GRID), dim3(WARPS * 32), 0, st, \
                                    __VA_ARGS__)                                                                       \
                    : tq_launch_pdl(p.dtype ? KERN<256, false> : KERN<256, true>, dim3(GRID), dim3(WARPS * 32), 0, st, \
                                    __VA_ARGS__))

cudaError_t b8_launch_append(const B8AppendParams& p, cudaStream_t st) {
    const int64_t nbt = (p.n_new + 62) / 32;   // a call touches at most this many blocks of a sequence
    const int64_t grid = (p.c.n_seq * nbt * 2 * p.c.n_kv + kAppendWarps - 1) / kAppendWarps;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    return B8_LAUNCH(k_b8_append, (unsigned)grid, kAppendWarps, p, (int)nbt);
}

cudaError_t b8_launch_read(const B8ReadParams& p, cudaStream_t st) {
    const int64_t groups = (p.n_tok + kReadTok - 1) / kReadTok + 1;   // the first and the last may be cut
    const int parts = (p.c.n_kv * (p.c.d / (p.dtype ? 8 : 4)) + 31) / 32;
    const int64_t warps = groups * 2 * parts;
    if (warps > 0x7fffffffLL) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)((warps + kReadWarps - 1) / kReadWarps), (unsigned)p.c.n_seq);
    return B8_LAUNCH(k_b8_read, grid, kReadWarps, p, (int)groups, parts);
}
