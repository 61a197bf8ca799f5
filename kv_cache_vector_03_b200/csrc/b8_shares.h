// Equal shares of the attention's list of units (k_b8_attn.cu), as plain 32-bit arithmetic that holds over every
// list that the host accepts: up to 2^29 segments of up to three units, 3 * 2^29 units in all.
#pragma once

#ifdef __CUDACC__
#define B8_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define B8_HOST_DEVICE inline
#endif

constexpr int kB8Segment = 10;       // what a segment costs beside its units, in units (8000 cycles)

// A segment is priced at its units and `per` more, for what each begun segment costs, so that CTAs with many segments
// get fewer units. Where those prices do not fit 31 bits (195 M segments of one unit and more) segments are priced at
// their units alone: there they are short and nearly alike, so shares of the units are shares of the segments too.
struct B8Shares {
    int per;                         // price of a segment beside its units
    int base, extra;                 // a share's price: base, one more for the first `extra` CTAs
    B8_HOST_DEVICE void make(int units, int segments, int ctas) {
        per = units + (long long)kB8Segment * segments <= 0x7fffffffLL ? kB8Segment : 0;
        base = price(units, segments) / ctas;
        extra = price(units, segments) - base * ctas;
    }
    B8_HOST_DEVICE int price(int units, int segments) const { return units + per * segments; }
    B8_HOST_DEVICE int share(int c) const { return c * base + (c < extra ? c : extra); }   // where CTA c's share begins
    B8_HOST_DEVICE int owner(int u) const {                                                // the CTA whose share holds u
        const int wide = extra * (base + 1);
        return u < wide ? u / (base + 1) : extra + (u - wide) / base;
    }
};
