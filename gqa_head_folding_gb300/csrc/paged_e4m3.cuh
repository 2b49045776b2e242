// paged_e4m3.cuh -- the format of an 8-bit page: E4M3 codes, and for each
// (page, KV head) of keys and of values an exponent e; value = value(code) 2^e.
//
// A power of two, because a code has an exponent of its own: a factor of any
// other value would gain nothing (the relative step of a code stays 2^-3), and
// a page can move to a larger exponent without a rounding, but for the codes
// that fall under the smallest normal one. The exponent never meets a code in
// 16 bits: attention multiplies the score of a key by 2^e, and takes a value's
// into the argument of the exponential.
#pragma once

#include "paged_sched.cuh"

namespace gqaq {

// Exponents of a page. Attention weighs a token by 2^(score + e - reference) and
// adds 2^-e times that to the row's sum: of two tokens with equal scores, whose
// pages' exponents are as far apart as can be, the lesser weighs 2^-96, 30 binary
// places above where 32-bit floats end. 448 * 2^48 is 1.3e17.
constexpr int kLeastPageExp = -48, kMostPageExp = 48;

// A weight is rounded to fp16 relative to 2^-kHeadroom of the row's largest
// 2^(score + e) so far. Of a token whose page lies at most kHeadroom exponents
// under the largest so far it keeps what 16-bit pages' weights keep: fp16's 11
// bits down to 2^-14 of the row's largest softmax weight, and 2^-25 of that where
// it is less. A page farther down would lose its tokens' bits to a page that may
// hold nothing in their channels, so its weights are taken in two bfloat16 numbers
// (off by 2^-17, with the range of 32-bit floats), against its codes in bfloat16,
// which are exact too.
constexpr float kHeadroom = 6.f;

__device__ __forceinline__ uint32_t f16x2_to_bf16x2(uint32_t x) {
    const float2 f = half2_bits_to_float2(x);
    return pack2<true>(f.x, f.y);
}

__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

// A score's factor past the range of 32 bits stays a number, so that a score of zero stays zero.
__device__ __forceinline__ float finite32(float x) {
    float r;
    asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(__int_as_float(0x7f7fffff)));
    return r;
}

// The least exponent whose largest value, 448 * 2^e, reaches `amax` (its bits;
// finite, not negative), within the range.
__device__ __forceinline__ int page_exp_of(uint32_t amax) {
    const int x = (int)(amax >> 23) - 127;  // amax = m 2^x, 1 <= m < 2; 448 = 1.75 * 2^8
    const int e = x - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
    return min(max(e, kLeastPageExp), kMostPageExp);
}

// Four fp32 values -> four codes, the first in the lowest byte.
__device__ __forceinline__ uint32_t f32x4_to_e4m3x4(f32x2 lo, f32x2 hi) {
    const float2 a = unpair32(lo), b = unpair32(hi);
    uint32_t r;
    asm("{\n\t.reg .b16 s, t;\n\tcvt.rn.satfinite.e4m3x2.f32 s, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 t, %4, %3;\n\tmov.b32 %0, {s, t};\n\t}"
        : "=r"(r)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

// Four codes times 2^-d, rounded to codes again.
__device__ __forceinline__ uint32_t e4m3x4_shift(uint32_t w, float by) {
    uint32_t lo, hi;
    e4m3x4_to_f16x2x2(w, lo, hi);
    const float2 a = half2_bits_to_float2(lo), b = half2_bits_to_float2(hi);
    return f32x4_to_e4m3x4(pair32(a.x * by, a.y * by), pair32(b.x * by, b.y * by));
}

// What attention takes of a page's exponents: the factor of its keys' scores,
// what its values add to the argument of the exponential, and the inverse of
// that, which turns a weight back into its share of the row's sum.
__device__ __forceinline__ float4 page_factors(int ke, int ve) { return make_float4(pow2i(ke), (float)ve, pow2i(-ve), 0.f); }
// The first two; the factor negative in a far tile.
__device__ __forceinline__ float2 page_factors2(int ke, int ve, bool far) { return make_float2(far ? -pow2i(ke) : pow2i(ke), (float)ve); }

// A loader warp's way along an item's pages: 32 table entries at a time, a lane
// each, with the entries two batches ahead and their pages' exponents one (an
// exponent's load waits for its entry's). P: the kernel's parameters, which have
// the work (w), k_exp, v_exp, zero_row and status.
template <typename P>
struct PageFeed {
    const int *next;          // this lane's entry that is loaded next
    int left;                 // entries from there on
    int kv;
    int raw;                  // two batches ahead: the entry, if left > -32
    int row1, k1, v1;         // one ahead
    bool here1;
    int row, ke, ve;          // the batch in use: first row in the pool, exponents
    int top;                  // largest exponent of values in the item so far
    bool far;                 // the batch has a page more than kHeadroom under it

    __device__ __forceinline__ void entry() {
        if (left > 0) raw = *next;
        next += 32;
        left -= 32;
    }
    __device__ __forceinline__ void step(const P &p) {
        row = row1;
        ke = min(max(k1, kLeastPageExp), kMostPageExp);
        ve = min(max(v1, kLeastPageExp), kMostPageExp);
        top = max(top, __reduce_max_sync(0xffffffffu, here1 ? ve : kLeastPageExp));
        far = top - __reduce_min_sync(0xffffffffu, here1 ? ve : kMostPageExp) > (int)kHeadroom;
        const bool here = left > -32, good = (uint32_t)raw < (uint32_t)p.w.num_pages;
        if (ke != k1 || ve != v1 || (here && !good)) raise_flag(p.status, GQAQ_DEV_BAD_PAGE);
        row1 = p.zero_row;
        k1 = v1 = 0;
        here1 = here;
        if (here && good) {
            const int unit = raw * p.w.Hkv + kv;
            row1 = unit << p.w.shift;
            k1 = p.k_exp[unit];
            v1 = p.v_exp[unit];
        }
        entry();
    }
    // The item that the walk is in, from its tile w.local on.
    __device__ __forceinline__ void start(const P &p, const PagedWalk &w, int lane) {
        const int held = (int)(((int64_t)w.s.len + (1 << p.w.shift) - 1) >> p.w.shift);
        const int at = (w.local << (kPagedTileLog - p.w.shift)) + lane;
        next = p.w.table + (int64_t)w.b * p.w.max_pages + at;
        left = held - at;
        kv = w.kv;
        raw = 0;
        row1 = p.zero_row;
        k1 = v1 = 0;
        here1 = false;
        top = kLeastPageExp;
        entry();
        step(p);
        step(p);
    }
};

}  // namespace gqaq
