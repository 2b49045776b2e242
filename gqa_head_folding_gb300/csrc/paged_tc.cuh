// paged_tc.cuh -- what the two paged attention kernels on the 5th-generation
// tensor cores (16-bit and 8-bit pages) share: the item's shape, its place in
// tensor memory, the warps' instructions, and the end of an item.
#pragma once

#include <math.h>

#include "paged_sched.cuh"
#include "umma.cuh"

namespace gqaq {

// An item: 256 rows in two row tiles of 128, context tiles of 128 tokens.
template <int D>
struct PtcShape {
    static constexpr int RB = 256;                   // rows per item
    static constexpr int KH = D / 64;                // 64-channel blocks
    static constexpr int BLK = 128 * 128;            // one block of 128 rows of 16 bits
    static constexpr int TILE = KH * BLK;            // a Q, K or V tile of 16 bits
    static constexpr int O_COL = 0, S_COL = 256;     // O of group g at 128 g, S at 256 + 128 g
    static constexpr int ML = 2 * RB;                // floats of a partial's (m, l)
    static constexpr int PART = ML + RB * D;         // floats of a partial
};

constexpr int kMinUnits = 2;        // units per CTA below which a small step uses fewer CTAs (two at least: see PagedParts)
constexpr int kItemTiles = 5;       // what an item costs beside its tiles: its start, epilogue and merge, in tiles (without it a mixed batch took 95 us for 74)
constexpr float kSumLimit = 32768.f;  // of 64 P: above it some P passes 2^9
constexpr float kRefMove = 9.f;       // log2 of the P that moves a row's reference
constexpr float kRefDrop = 6.f;       // the new reference's distance under the row's maximum

struct PtcParams {
    PagedWorkParams w;
    uint16_t *out;
    float *part;       // [grid][2] partials: a CTA's first and last segment
    unsigned *count;   // [grid]: arrivals at the split item that begins in a CTA's range; zero between calls
    int *status;
    int G, gshift, Hq, S;
    int zero_row;      // rows of the pools: a box from here on reads zeros
    float scale_log2;
    uint64_t timeout_ns;
    int test_stall;
    int wide_out;      // out is 32-byte aligned
};

inline void fill_ptc(const PagedAttnArgs &a, const LaunchCtx &ctx, PtcParams &p) {
    const gqaq_paged_dims &d = *a.dims;
    p.G = d.num_q_heads / d.num_kv_heads;
    p.gshift = p.G == 1 ? 0 : p.G == 2 ? 1 : p.G == 4 ? 2 : 3;
    fill_paged_work(a, 8 - p.gshift, 128 >> p.gshift, kItemTiles, p.w);  // blocks of 256 rows; above 128 a tile runs twice
    p.out = static_cast<uint16_t *>(a.out);
    p.count = reinterpret_cast<unsigned *>(a.workspace);
    p.part = reinterpret_cast<float *>(static_cast<uint8_t *>(a.workspace) + kPagedCountBytes);
    p.status = ctx.status;
    p.Hq = d.num_q_heads;
    p.S = d.page_size;
    p.zero_row = d.num_pages * d.num_kv_heads * d.page_size;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    if (p.scale_log2 == 0.f) p.scale_log2 = 1e-30f;  // 2^(s - max) is 1 all the same, and a masked score's product stays -inf
    p.timeout_ns = ctx.timeout_ns;
    p.test_stall = ctx.test_stall;
    p.wide_out = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
}

__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
// Waits for this thread's loads; names the registers, so that no use of them moves above it.
__device__ __forceinline__ void tmem_ld32_wait(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                   "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                   "+r"(r[30]), "+r"(r[31])::"memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
                 "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}

// True on the 64 threads of barrier `id` when any of them passed true.
__device__ __forceinline__ bool pair_any(int id, bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\tbar.red.or.pred p, %2, 64, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)pred), "r"(id)
        : "memory");
    return r != 0;
}

// One product of a converged warp: its elected lane issues four K-steps (always
// the same lane, so that its commits cover them). With the operands in
// warp-uniform control flow the descriptors stay in uniform registers; issued
// from a one-lane branch each MMA took about 100 cycles, twice its work.
// Both operands from shared memory, 32 bytes (two descriptor units) per step.
__device__ __forceinline__ void warp_mma_ss4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred q, p, t;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
        "elect.sync _|q, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
        "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// A from tensor memory (8 columns per step), B 16 rows of 128 bytes per step.
__device__ __forceinline__ void warp_mma_ts4(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred q, p, t;\n\t.reg .b32 a1, a2, a3;\n\t.reg .b64 b1, b2, b3;\n\t"
        "elect.sync _|q, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "add.s32 a1, %1, 8;\n\tadd.s32 a2, %1, 16;\n\tadd.s32 a3, %1, 24;\n\t"
        "add.s64 b1, %2, 128;\n\tadd.s64 b2, %2, 256;\n\tadd.s64 b3, %2, 384;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, t;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, t;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void warp_commit(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}

// The end of a segment, for the 512 softmax threads: the sums of a row's two
// threads, then of the two groups where they share the rows; the output of a
// whole item, or a part of one that several CTAs share, which the last of them
// to arrive merges. Thread (g, h, row) holds the reference and its sum of row
// `row` of group g; nx: the group's tiles, n: the segment's, dual: two row tiles.
template <int D, bool BF16, typename Wait>
__device__ __forceinline__ void ptc_finish(const PtcParams &p, const PagedWalk &w, PagedSched *sched, float *xchg, uint32_t o_done,
                                           uint32_t o_free, uint32_t tlane, int g, int h, int row, int n, int nx, bool dual, bool live,
                                           bool warp_live, int rho, float ref, float l, uint32_t &oph, bool &ok, Wait &&wait) {
    using C = PtcShape<D>;
    const int lane = threadIdx.x & 31, tid = threadIdx.x;
    const int TB = C::RB >> p.gshift;
    // ---- epilogue: sums of the two halves, then of the two groups if they share the rows ----
    if (nx > 0) {
        ok = ok && wait(o_done + 8 * g, oph);
        oph ^= 1u;
    }
    tc_fence_before();
    const bool whole = w.whole();
    float w0 = 1.f, w1 = 0.f;  // weights of O0 and O1 (one row tile), or w0 of this group's O
    float M = ref, L = l;
    if (h == 1) xchg[128 * g + row] = l;
    named_bar_sync(1, 512);
    if (h == 0) L = l + xchg[128 * g + row];
    float2 *both = reinterpret_cast<float2 *>(xchg);
    if (!dual) {
        named_bar_sync(1, 512);
        if (g == 1 && h == 0) both[row] = make_float2(ref, L);
        named_bar_sync(1, 512);
        if (g == 0 && h == 0) {
            const float2 o = both[row];
            M = fmaxf(ref, o.x);
            w0 = ref == -INFINITY ? 0.f : fast_exp2(ref - M);
            w1 = o.x == -INFINITY ? 0.f : fast_exp2(o.x - M);
            L = w0 * L + w1 * o.y;
            if (whole) {
                const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
                w0 *= inv;
                w1 *= inv;
            }
            both[row] = make_float2(w0, w1);
        }
        named_bar_sync(1, 512);
        const float2 o = both[row];
        w0 = o.x;
        w1 = o.y;
    } else {
        if (h == 0) {
            if (whole) w0 = L > 0.f || L != L ? 1.f / L : 0.f;
            xchg[128 * g + row] = w0;
        }
        named_bar_sync(1, 512);
        w0 = xchg[128 * g + row];
    }
    tc_fence_after();
    // this thread's share of its row's D channels: half of them, or a quarter where four threads share it
    const int nc = dual ? D / 2 : D / 4, c0 = dual ? h * nc : (2 * g + h) * nc;
    const uint32_t o0 = tlane + C::O_COL + (dual ? 128u * (uint32_t)g : 0u), o1 = tlane + C::O_COL + 128u;
    const bool second = !dual && n > 1;
    const int q_row = w.s.q0 + w.rb * TB + (rho >> p.gshift);
    uint16_t *dst = p.out + ((int64_t)q_row * p.Hq + w.kv * p.G + (rho & (p.G - 1))) * D;
    const int slot = w.slot();
    float *part = p.part + ((int64_t)blockIdx.x * 2 + slot) * C::PART;
    if (warp_live) {
        if (!whole && live && h == 0 && (dual || g == 0)) reinterpret_cast<float2 *>(part)[rho] = make_float2(M, L);
#pragma unroll 1
        for (int c = c0; c < c0 + nc; c += 16) {
            uint32_t a[16], b[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) a[e] = b[e] = 0u;
            if (ok) {
                tmem_ld16(o0 + (uint32_t)c, a);
                if (second) tmem_ld16(o1 + (uint32_t)c, b);
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                // a weight of zero: no keys, and nothing of that O may count
                float y = w0 == 0.f ? 0.f : __uint_as_float(a[e]) * w0;
                if (second && w1 != 0.f) y = fmaf(__uint_as_float(b[e]), w1, y);
                a[e] = __float_as_uint(y);
            }
            if (!live) continue;
            if (whole) {
                uint32_t x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = pack2<BF16>(__uint_as_float(a[2 * e]), __uint_as_float(a[2 * e + 1]));
                if (p.wide_out) {  // a lane's 32 bytes are one sector: half the stores of scattered rows
                    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(__cvta_generic_to_global(dst + c)),
                                 "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                                 : "memory");
                } else {
                    *reinterpret_cast<uint4 *>(dst + c) = make_uint4(x[0], x[1], x[2], x[3]);
                    *reinterpret_cast<uint4 *>(dst + c + 8) = make_uint4(x[4], x[5], x[6], x[7]);
                }
            } else {
                float4 *acc = reinterpret_cast<float4 *>(part + C::ML) + (int64_t)(c / 4) * C::RB + rho;
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                    acc[(e / 4) * C::RB] = make_float4(__uint_as_float(a[e]), __uint_as_float(a[e + 1]),
                                                       __uint_as_float(a[e + 2]), __uint_as_float(a[e + 3]));
            }
        }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(o_free);
    named_bar_sync(1, 512);  // xchg is free again; partial stores are done

    if (!whole) {
        // ---- arrive at the split item; the last arrival merges it ----
        const PagedParts parts(*sched, w.off, w.tiles, w.us);
        const int np = parts.n;
        if (tid == 0) {
            // the barrier orders every thread's partial stores before this
            // release; the last arrival acquires all of them
            const unsigned old = atomic_add_acq_rel_gpu(&p.count[parts.lo], 1u);
            const int last = old + 1u == (unsigned)np;
            if (last) p.count[parts.lo] = 0u;
            sched->last = last;
        }
        named_bar_sync(1, 512);
        if (sched->last && live) {
            const float *base = p.part + parts.lo * 2 * C::PART;
            auto part_of = [&](int i) { return base + (int64_t)(2 * i + (i == 0 ? 1 : 0)) * C::PART; };
            float mx = -INFINITY, sum = 0.f;
            for (int i = 0; i < np; ++i) mx = fmaxf(mx, __ldcg(part_of(i) + 2 * rho));
            for (int i = 0; i < np; ++i) {
                const float2 ml = __ldcg(reinterpret_cast<const float2 *>(part_of(i)) + rho);
                // without a reference the sum is 0, or NaN where every score that the row sees in the part is
                sum += ml.x == -INFINITY ? ml.y : fast_exp2(ml.x - mx) * ml.y;
            }
            const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
#pragma unroll 1
            for (int c = c0; c < c0 + nc; c += 16) {
                float4 a[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) a[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
                for (int i = 0; i < np; ++i) {
                    const float *pi = part_of(i);
                    const float m = __ldcg(pi + 2 * rho);
                    const float f = (m == -INFINITY ? 0.f : fast_exp2(m - mx)) * inv;  // NaN where inv is
                    const float4 *acc = reinterpret_cast<const float4 *>(pi + C::ML) + (int64_t)(c / 4) * C::RB + rho;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float4 x = __ldcg(acc + e * C::RB);
                        a[e].x = fmaf(f, x.x, a[e].x);
                        a[e].y = fmaf(f, x.y, a[e].y);
                        a[e].z = fmaf(f, x.z, a[e].z);
                        a[e].w = fmaf(f, x.w, a[e].w);
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    uint4 x;
                    x.x = pack2<BF16>(a[e].x, a[e].y);
                    x.y = pack2<BF16>(a[e].z, a[e].w);
                    x.z = pack2<BF16>(a[e + 1].x, a[e + 1].y);
                    x.w = pack2<BF16>(a[e + 1].z, a[e + 1].w);
                    *reinterpret_cast<uint4 *>(dst + c + 4 * e) = x;
                }
            }
        }
    }
}

}  // namespace gqaq
