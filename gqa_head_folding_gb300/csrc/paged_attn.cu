// paged_attn.cu -- paged attention for single tokens and short drafts (at most
// eight rows per KV head; over 8-bit pages up to 32), and the choice between it
// and the tensor-memory kernels.
//
// A request's q_len tokens and the G query heads of a KV head form at most
// eight rows, which are the N = 8 side of mma.sync m16n8k16; the tokens of the
// cache are the M side, so a K or V row is read from HBM once for all of them
// and no row of the tensor core's tile is padding of a 128-row block:
//   S^T [16 tokens x 8] = K Q^T,   O^T [D x 8] += V^T P^T
// with an online softmax in the log2 domain on the S^T fragments: the row
// maxima are gathered across lanes, and the sums and outputs rescaled, only
// when a tile holds a score 2^8 above the reference (P <= 2^8 keeps fp16
// exact enough). Sums and outputs are fp32; each P is rounded once (over 8-bit
// pages: see PagedWarp8).
//
// Kernel shape (persistent CTAs, one launch): the tiles of 128 tokens of all
// (request, KV head) items are split evenly (paged_sched.cuh); warp 8 gathers
// a tile from its pages with TMA, one box per page and operand, into a ring of
// stages (three over 16-bit pages, three to ten over 8-bit ones); warps 0-7 own 16
// tokens of each tile. At the end of an item's
// segment the eight warps' states merge in shared memory; an item cut by a
// range boundary leaves an fp32 partial and the CTA that arrives last merges
// them.
//
// What bounds it: HBM (batch 8 at up to 64K, 8 KV heads of 128 channels: 224 us,
// 6.6 TB/s, 97% of the copy rate); with little data the chain of schedule (2
// us), first tile (1.3), tiles, state merge (0.6), arrival (1.1) and merge of
// the parts (one request at 4K, 8 KV heads of 64 channels: 10.3 us).
//
// Over 8-bit pages the codes are widened to fp16 between shared memory and the
// product, by the lane that needs them, once for all blocks of eight rows. Half
// the bytes: the batch of 8 at up to 64K takes 132 us (5.7 TB/s, 85% of the
// copy rate, 49% of the issue slots), with two CTAs per SM (one with five stages
// 139), one request at 4K 10.1. Two 16s of tokens per warp and tile, whose products
// are independent, were no faster at 64 channels (one request 10.7 us, 32 of 1K to 4K 29.7
// for 28.9) and spill at 128.
#include <math.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "attn_mma.cuh"
#include "paged_e4m3.cuh"

namespace gqaq {
namespace {

constexpr int kRows = kFewRows;   // rows of an item: q_len * G at most
constexpr int kMinUnits = 2;      // tiles per CTA below which a small step uses fewer CTAs (8 KV heads of 64 channels over 4K tokens: two 10.4 us, four 11.7)

template <int D, bool KV8, int NB>
struct PdCfg {
    // Eight warps that compute and one that loads get 168 registers a thread at most. Where that is too little, three idle
    // warps fill the loader's warpgroup, which hands the others some of its registers: 8 * 224 + 4 * 56 = 12 * 168.
    static constexpr bool SHIFT_REGS = D == 128 && NB == 3;
    static constexpr int THREADS = SHIFT_REGS ? 384 : 288;
    static constexpr int KBYTES = 128 * D * (KV8 ? 1 : 2);
    static constexpr int STAGE = 2 * KBYTES;
    static constexpr int MIN_BLOCKS = NB > 1 || (D == 128 && !KV8) ? 1 : 2;
    static constexpr int NSTAGE = KV8 ? (MIN_BLOCKS == 1 ? 5 : 3) * (128 / D) : 3;
    static constexpr int MROWS = NB > 1 ? (MIN_BLOCKS == 1 ? 8 : 4) : KV8 && D == 128 ? 2 : 4;  // rows merged at a time
    static constexpr int MERGE = 8 * MROWS * (D + 2) * 4;
    static constexpr int FACTORS = KV8 ? NSTAGE * 16 * 8 : 0;  // of a tile's pages, beside each stage
    static constexpr bool SHARED_Q = KV8 && NB > (D == 128 ? 1 : 3);  // Q in shared memory, as the products take it: it has no room beside O
    static constexpr int QBYTES = SHARED_Q ? NB * D * 16 : 0;
    static constexpr int MISC = 512;
    static constexpr int SMEM = 1024 + NSTAGE * STAGE + MERGE + FACTORS + QBYTES + MISC;
    // What an item costs beside its tiles, in tiles: more, where it has more rows to bring and to merge (128 channels, 32
    // requests of 500 to 4K, 8 and 16 rows: one 49 and 63 us, two 47 and 57, five 45 and 53; 64 channels, 8 and 24 rows: one 28.5
    // and 52 us, two 27.9 and 47, five 29.4 and 45).
    static constexpr int ITEM_TILES = !KV8 ? 1 : D == 128 ? 2 * NB : NB + 1;
    static constexpr int PART = kRows * NB * (D + 2);     // floats of a partial: (m, l, acc) per row
    static_assert(MIN_BLOCKS * (SMEM + 1024) <= 228 * 1024, "shared memory");
};

struct PdParams {
    PagedWorkParams w;
    const uint16_t *q;
    uint16_t *out;
    float *part;
    unsigned *count;
    int *status;
    int gshift, Hq, S, zero_row;
    float scale_log2;
    uint64_t timeout_ns;
    int test_stall;
    const int8_t *k_exp, *v_exp;  // 8-bit pages
    unsigned *begun, *read;       // not null: the launch before is of the same call, and this one may run beside it
};

template <bool BF16>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        mma_16816(d, a, b0, b1);
}

template <bool BF16>
__device__ __forceinline__ uint16_t round16(float x) {
    return (uint16_t)(pack2<BF16>(x, 0.f) & 0xffffu);
}

// One warp's share: 16 tokens of a tile against the item's rows. Lane r * 4 + c
// holds columns 2c, 2c + 1 of tokens r and r + 8 in S^T, and channels 16 i + r,
// + 8 of the same columns in O^T.
template <int D, bool BF16>
struct PagedWarp {
    static constexpr int KS = D / 16, KH = D / 64;
    int lane, r, c;
    uint32_t qb[KS][2];
    int lim[2];           // last position of columns 2c, 2c + 1
    float m[2], l[2], o[KS][4];

    // 16-byte chunk ch8 of a row: rows lie one behind the other, 128-byte swizzled lines
    __device__ __forceinline__ static uint32_t chunk(uint32_t base, int row, int ch8) {
        const int line = row * KH + (ch8 >> 3);
        return base + (uint32_t)(line * 128 + (((ch8 & 7) ^ (line & 7)) << 4));
    }
    __device__ __forceinline__ void begin(const PdParams &p, const PagedWalk &w, int warp) {
        const int G = 1 << p.gshift, rows = w.s.m << p.gshift;
        const bool live = r < rows;
        const uint16_t *qr = p.q + ((int64_t)(w.s.q0 + (live ? r >> p.gshift : 0)) * p.Hq + w.kv * G + (live ? r & (G - 1) : 0)) * D;
#pragma unroll
        for (int j = 0; j < KS; ++j) {
            qb[j][0] = live ? *reinterpret_cast<const uint32_t *>(qr + 16 * j + 2 * c) : 0u;
            qb[j][1] = live ? *reinterpret_cast<const uint32_t *>(qr + 16 * j + 8 + 2 * c) : 0u;
        }
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) lim[i] = w.s.start + min((2 * c + i) >> p.gshift, w.s.m - 1);
#pragma unroll
        for (int i = 0; i < KS; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    }
    // Stage rows row0 .. row0 + 15, tokens tok0 ..; n of them (a prefix) exist.
    // Columns may see fewer: `mask` when some limit falls inside.
    __device__ __forceinline__ void tile(uint32_t kb, uint32_t vb, int row0, int tok0, int n, bool mask, float scale_log2) {
        const int mi = lane >> 3, rr = lane & 7;
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < KS; ++j) {
            uint32_t a[4];
            ldsm_x4(chunk(kb, row0 + (mi & 1) * 8 + rr, 2 * j + (mi >> 1)), a);
            mma16<BF16>(s, a, qb[j][0], qb[j][1]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] *= scale_log2;
        if (mask) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] = tok0 + r + 8 * (e >> 1) <= lim[e & 1] ? s[e] : -INFINITY;
        }
        float t0 = fmaxf(s[0], s[2]), t1 = fmaxf(s[1], s[3]);
        if (__any_sync(0xffffffffu, t0 > m[0] + 8.f || t1 > m[1] + 8.f)) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) {
                t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, x));
                t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, x));
            }
            const float n0 = fmaxf(m[0], t0), n1 = fmaxf(m[1], t1);
            // a column that has seen no token keeps the reference -inf and all zeros
            const float a0 = m[0] == -INFINITY ? 0.f : fast_exp2(m[0] - n0), a1 = m[1] == -INFINITY ? 0.f : fast_exp2(m[1] - n1);
            m[0] = n0;
            m[1] = n1;
            l[0] *= a0;
            l[1] *= a1;
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                o[i][0] *= a0;
                o[i][1] *= a1;
                o[i][2] *= a0;
                o[i][3] *= a1;
            }
        }
        const float r0 = m[0] == -INFINITY ? 0.f : m[0], r1 = m[1] == -INFINITY ? 0.f : m[1];
        s[0] = fast_exp2(s[0] - r0);
        s[1] = fast_exp2(s[1] - r1);
        s[2] = fast_exp2(s[2] - r0);
        s[3] = fast_exp2(s[3] - r1);
        l[0] += s[0] + s[2];
        l[1] += s[1] + s[3];
        const uint32_t pb0 = movmatrix_trans(pack2<BF16>(s[0], s[1])), pb1 = movmatrix_trans(pack2<BF16>(s[2], s[3]));
        const bool cut = n < 16;  // rows behind the request may hold anything: 0 * NaN would reach O
        const uint32_t mk0 = (2 * c < n ? 0x0000ffffu : 0u) | (2 * c + 1 < n ? 0xffff0000u : 0u);
        const uint32_t mk1 = (2 * c + 8 < n ? 0x0000ffffu : 0u) | (2 * c + 9 < n ? 0xffff0000u : 0u);
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            uint32_t a[4];
            ldsm_x4_trans(chunk(vb, row0 + (mi >> 1) * 8 + rr, 2 * i + (mi & 1)), a);
            if (cut) {
                a[0] &= mk0;
                a[1] &= mk0;
                a[2] &= mk1;
                a[3] &= mk1;
            }
            mma16<BF16>(o[i], a, pb0, pb1);
        }
    }
    // (m, l, acc) of rows first .. first + MROWS - 1 to this warp's slot of the merge buffer.
    __device__ __forceinline__ void store(float *slot, int, int first) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float ls = l[i];
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, x);
            const int n = 2 * c + i - first;
            if (n < 0 || n >= PdCfg<D, false, 1>::MROWS) continue;
            float *w = slot + n * (D + 2);
            if (r == 0) {
                w[0] = m[i];
                w[1] = ls;
            }
#pragma unroll
            for (int j = 0; j < KS; ++j) {
                w[2 + 16 * j + r] = o[j][i];
                w[2 + 16 * j + r + 8] = o[j][2 + i];
            }
        }
    }
};

// The same over 8-bit pages (paged_e4m3.cuh). With code_k and code_v the values
// of the codes, ke and ve their pages' exponents and s = scale log2(e) 2^ke q . code_k:
//   w = 2^(s + ve - ref),  O += w code_v,  l += w 2^-ve,  out = O / l
// so neither exponent meets a number of 16 bits, and the codes reach the tensor
// core as they decode, exactly, to fp16. The largest w is at least 2^kHeadroom;
// a tile with a page more than kHeadroom exponents under the item's largest so
// far takes its w in two bfloat16 numbers (the loader marks it: the factors of its
// keys are negative): the batch of 8 at 64K takes 149 us for 132 where every
// context begins with such a large page. A tile's whole work in two copies costs
// nothing where there is none; one copy with a branch before V took 147. Queries
// are fp16 there too: a bfloat16 row is taken times a power of two that brings its
// largest channel into [2^14, 2^15): channels down to 2^-31 of it keep all their
// bits, smaller ones are off by at most 2^-39 of it.
// Lane r * 4 + c reads bytes D/4 c .. of K rows r and r + 8, and bytes D/8 r ..
// of V rows 2c, 2c + 1, 2c + 8 and 2c + 9: channel (D/4) c + 4 j + e of q meets
// its like in step j, and channel (D/8) r + 2 i + h of O lies in o[i][2 h], o[i][2 h + 1].
template <int D, bool BF16, int NB>
struct PagedWarp8 {
    static constexpr int KS = D / 16;
    static constexpr bool SHARED_Q = PdCfg<D, true, NB>::SHARED_Q;
    int lane, r, c;
    uint32_t qb[SHARED_Q ? 1 : NB][KS][2];
    uint32_t qs;              // SHARED_Q: this lane's words of Q, step (b, j) at + 256 (b KS + j)
    int start, last, gshift;  // position of the item's first token, its last token, log2 of G
    float mul[NB][2];         // factor of the scores of columns 2c, 2c + 1
    float m[NB][2], l[NB][2], o[NB][KS][4];

    // 8 bytes from `byte` on of a row of D codes: lines of 128 bytes swizzled by 128, rows of 64 by 64
    __device__ __forceinline__ static uint32_t at(uint32_t base, int row, int byte) {
        if (D == 128) return base + (uint32_t)(row * 128 + (((byte >> 4) ^ (row & 7)) << 4) + (byte & 15));
        return base + (uint32_t)(row * 64 + (((byte >> 4) ^ ((row >> 1) & 3)) << 4) + (byte & 15));
    }
    __device__ __forceinline__ void begin(const PdParams &p, const PagedWalk &w, int warp) {
        const int G = 1 << p.gshift, rows = w.s.m << p.gshift;
        start = w.s.start;
        last = w.s.m - 1;
        gshift = p.gshift;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            auto &x = qb[SHARED_Q ? 0 : b];
            const int row = 8 * b + r;
            const bool live = row < rows;
            const uint16_t *qr =
                p.q + ((int64_t)(w.s.q0 + (live ? row >> p.gshift : 0)) * p.Hq + w.kv * G + (live ? row & (G - 1) : 0)) * D + (D / 4) * c;
#pragma unroll
            for (int j = 0; j < KS; ++j) {
                const uint2 y = live ? *reinterpret_cast<const uint2 *>(qr + 4 * j) : make_uint2(0u, 0u);
                x[j][0] = y.x;
                x[j][1] = y.y;
            }
            mul[b][0] = mul[b][1] = p.scale_log2;
            if (BF16) {
                uint32_t top = 0u;  // bits of the row's largest finite magnitude
#pragma unroll
                for (int j = 0; j < KS; ++j)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t lo = x[j][i] & 0x7fffu, hi = (x[j][i] >> 16) & 0x7fffu;
                        top = max(top, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
                    }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int e = max((int)(top >> 7) - 127 - 14, -100);
                const float by = pow2i(-e), back = pow2i(e);
#pragma unroll
                for (int j = 0; j < KS; ++j)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        x[j][i] = pack2<false>(__uint_as_float(x[j][i] << 16) * by, __uint_as_float(x[j][i] & 0xffff0000u) * by);
#pragma unroll
                for (int i = 0; i < 2; ++i) mul[b][i] = finite32(mul[b][i] * __shfl_sync(0xffffffffu, back, 4 * (2 * c + i)));
            }
            if constexpr (SHARED_Q) {  // each of the eight warps leaves one step for all
#pragma unroll
                for (int j = 0; j < KS; ++j)
                    if (j == warp) asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(qs + 256u * (uint32_t)(b * KS + j)), "r"(x[j][0]), "r"(x[j][1]) : "memory");
            }
            m[b][0] = m[b][1] = -INFINITY;
            l[b][0] = l[b][1] = 0.f;
#pragma unroll
            for (int i = 0; i < KS; ++i) o[b][i][0] = o[b][i][1] = o[b][i][2] = o[b][i][3] = 0.f;
        }
    }
    // As PagedWarp::tile; f0, f1: factors of the pages of this lane's tokens r and r + 8. A code is decoded once for
    // all NB blocks of eight rows.
    __device__ __forceinline__ void tile(uint32_t kb, uint32_t vb, int row0, int tok0, int n, bool mask, const float2 &f0, const float2 &f1) {
        if (__builtin_expect(__any_sync(0xffffffffu, f0.x < 0.f), 0)) tile_of<true>(kb, vb, row0, tok0, n, mask, f0, f1);
        else tile_of<false>(kb, vb, row0, tok0, n, mask, f0, f1);
    }
    template <bool FAR>
    __device__ __forceinline__ void tile_of(uint32_t kb, uint32_t vb, int row0, int tok0, int n, bool mask, const float2 &f0, const float2 &f1) {
        constexpr int KB = D / 4, VB = D / 8;  // bytes of a row that a lane reads
        float s[NB][4];
        {
            uint32_t a0[KB / 4], a1[KB / 4];
#pragma unroll
            for (int h = 0; h < KB / 16; ++h) {
                const uint4 x = lds128(at(kb, row0 + r, KB * c + 16 * h)), y = lds128(at(kb, row0 + r + 8, KB * c + 16 * h));
                a0[4 * h] = x.x; a0[4 * h + 1] = x.y; a0[4 * h + 2] = x.z; a0[4 * h + 3] = x.w;
                a1[4 * h] = y.x; a1[4 * h + 1] = y.y; a1[4 * h + 2] = y.z; a1[4 * h + 3] = y.w;
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) s[b][0] = s[b][1] = s[b][2] = s[b][3] = 0.f;
#pragma unroll
            for (int j = 0; j < KS; ++j) {
                uint32_t a[4];
                e4m3x4_to_f16x2x2(a0[j], a[0], a[2]);
                e4m3x4_to_f16x2x2(a1[j], a[1], a[3]);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    if constexpr (SHARED_Q) {
                        const uint2 q = lds64(qs + 256u * (uint32_t)(b * KS + j));
                        mma_16816(s[b], a, q.x, q.y);
                    } else {
                        mma_16816(s[b], a, qb[b][j][0], qb[b][j][1]);
                    }
                }
            }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 &f = e < 2 ? f0 : f1;
                s[b][e] = fmaf(s[b][e] * (FAR ? fabsf(f.x) : f.x), mul[b][e & 1], f.y);
            }
        if (mask) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int lim = start + min((8 * b + 2 * c + (e & 1)) >> gshift, last);
                    s[b][e] = tok0 + r + 8 * (e >> 1) <= lim ? s[b][e] : -INFINITY;
                }
        }
        bool above = false;
#pragma unroll
        for (int b = 0; b < NB; ++b)
            above = above || fmaxf(s[b][0], s[b][2]) > m[b][0] + 8.f || fmaxf(s[b][1], s[b][3]) > m[b][1] + 8.f;
        if (__any_sync(0xffffffffu, above)) {
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float t0 = fmaxf(s[b][0], s[b][2]), t1 = fmaxf(s[b][1], s[b][3]);
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) {
                    t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, x));
                    t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, x));
                }
                const float n0 = fmaxf(m[b][0], t0), n1 = fmaxf(m[b][1], t1);
                // a column that has seen no token keeps the reference -inf and all zeros
                const float a0 = m[b][0] == -INFINITY ? 0.f : fast_exp2(m[b][0] - n0), a1 = m[b][1] == -INFINITY ? 0.f : fast_exp2(m[b][1] - n1);
                m[b][0] = n0;
                m[b][1] = n1;
                l[b][0] *= a0;
                l[b][1] *= a1;
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    o[b][i][0] *= a0;
                    o[b][i][1] *= a1;
                    o[b][i][2] *= a0;
                    o[b][i][3] *= a1;
                }
            }
        }
        const float u0 = fast_exp2(-f0.y), u1 = fast_exp2(-f1.y);
        uint32_t pb[NB][2];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const float r0 = m[b][0] == -INFINITY ? 0.f : m[b][0] - kHeadroom, r1 = m[b][1] == -INFINITY ? 0.f : m[b][1] - kHeadroom;
            s[b][0] = fast_exp2(s[b][0] - r0);
            s[b][1] = fast_exp2(s[b][1] - r1);
            s[b][2] = fast_exp2(s[b][2] - r0);
            s[b][3] = fast_exp2(s[b][3] - r1);
            l[b][0] = fmaf(s[b][0], u0, fmaf(s[b][2], u1, l[b][0]));
            l[b][1] = fmaf(s[b][1], u0, fmaf(s[b][3], u1, l[b][1]));
        }
        const bool cut = n < 16;  // rows behind the request may hold anything: 0 * NaN would reach O
        const uint32_t mk0 = (2 * c < n ? 0x0000ffffu : 0u) | (2 * c + 1 < n ? 0xffff0000u : 0u);
        const uint32_t mk1 = (2 * c + 8 < n ? 0x0000ffffu : 0u) | (2 * c + 9 < n ? 0xffff0000u : 0u);
        uint32_t v[4][VB / 4];  // tokens 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const uint32_t from = at(vb, row0 + 2 * c + (t & 1) + (t >> 1) * 8, VB * r);
            if constexpr (VB == 16) {
                const uint4 x = lds128(from);
                v[t][0] = x.x; v[t][1] = x.y; v[t][2] = x.z; v[t][3] = x.w;
            } else {
                const uint2 x = lds64(from);
                v[t][0] = x.x; v[t][1] = x.y;
            }
        }
        if constexpr (FAR) {
            far_values(s, vb, row0, cut, mk0, mk1);
            return;
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            pb[b][0] = movmatrix_trans(pack2<false>(s[b][0], s[b][1]));
            pb[b][1] = movmatrix_trans(pack2<false>(s[b][2], s[b][3]));
        }
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;  // channels 2i, 2i + 1 of two tokens, token inner
            uint32_t a[4];
            e4m3x4_to_f16x2x2(byte_perm(v[0][i >> 1], v[1][i >> 1], sel), a[0], a[1]);
            e4m3x4_to_f16x2x2(byte_perm(v[2][i >> 1], v[3][i >> 1], sel), a[2], a[3]);
            if (cut) {
                a[0] &= mk0;
                a[1] &= mk0;
                a[2] &= mk1;
                a[3] &= mk1;
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) mma_16816(o[b][i], a, pb[b][0], pb[b][1]);
        }
    }
    // O += w code_v of 16 tokens whose page lies far under another: w in two bfloat16 numbers, which have 32-bit floats' range.
    // One block of rows after the other, so that the two need no registers that the common way does not have.
    __device__ __forceinline__ void far_values(const float (&s)[NB][4], uint32_t vb, int row0, bool cut, uint32_t mk0, uint32_t mk1) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t x = pack2<true>(s[b][2 * h], s[b][2 * h + 1]);
                hi[h] = movmatrix_trans(x);
                lo[h] = movmatrix_trans(pack2<true>(s[b][2 * h] - __uint_as_float(x << 16), s[b][2 * h + 1] - __uint_as_float(x & 0xffff0000u)));
            }
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;
                uint32_t a[4], y[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) y[t] = lds32(at(vb, row0 + 2 * c + (t & 1) + (t >> 1) * 8, (D / 8) * r + 4 * (i >> 1)));
                e4m3x4_to_f16x2x2(byte_perm(y[0], y[1], sel), a[0], a[1]);
                e4m3x4_to_f16x2x2(byte_perm(y[2], y[3], sel), a[2], a[3]);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    a[x] = f16x2_to_bf16x2(a[x]);
                    if (cut) a[x] &= x < 2 ? mk0 : mk1;
                }
                mma16<true>(o[b][i], a, hi[0], hi[1]);
                mma16<true>(o[b][i], a, lo[0], lo[1]);
            }
        }
    }
    // (m, l, acc) of rows first .. first + MROWS - 1, which are of block b, to this warp's slot of the merge buffer.
    __device__ __forceinline__ void store(float *slot, int b, int first) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float ls = l[b][i];
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, x);
            const int n = 8 * b + 2 * c + i - first;
            if (n < 0 || n >= PdCfg<D, true, NB>::MROWS) continue;
            float *w = slot + n * (D + 2);
            if (r == 0) {
                w[0] = m[b][i];
                w[1] = ls;
            }
#pragma unroll
            for (int j = 0; j < KS; ++j) *reinterpret_cast<float2 *>(w + 2 + (D / 8) * r + 2 * j) = make_float2(o[b][j][i], o[b][j][2 + i]);
        }
    }
};

// An item this CTA arrived at last, to be merged at the end of its range.
struct PdSplit {
    int64_t off, out;  // tile offset of the item; first element of its output
    int tiles, rows, last;
};

template <int D, bool BF16, bool KV8, int NB>
__device__ __forceinline__ void paged_decode(const CUtensorMap &kmap, const CUtensorMap &vmap, const PdParams &p) {
    using C = PdCfg<D, KV8, NB>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *stages = smem;
    float *merge = reinterpret_cast<float *>(stages + C::NSTAGE * C::STAGE);
    float2 *factors = reinterpret_cast<float2 *>(reinterpret_cast<uint8_t *>(merge) + C::MERGE);  // [stage][16]
    uint64_t *full = reinterpret_cast<uint64_t *>(reinterpret_cast<uint8_t *>(factors) + C::FACTORS + C::QBYTES);
    uint64_t *empty = full + C::NSTAGE;
    int64_t *scratch = reinterpret_cast<int64_t *>(empty + C::NSTAGE);
    PagedSched *sched = reinterpret_cast<PagedSched *>(scratch + 12);
    PdSplit *split = reinterpret_cast<PdSplit *>(sched + 1);
    static_assert((2 * C::NSTAGE + 12) * 8 + sizeof(PagedSched) + 2 * sizeof(PdSplit) <= C::MISC, "misc region");
    volatile int *abort_flag = &sched->abort;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
    if (warp == 8 && lane == 0) {
        for (int s = 0; s < C::NSTAGE; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 8);
        }
        fence_mbar_init();
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
    }
    if (p.begun != nullptr) {
        pdl_release();
        // A loader's thread. It was set before this launch was released; no launch waits for it: where it is not seen, the
        // whole of the launch before is waited for. (Always waiting so: mixed batches of 32 with two chunks of 500 tokens 83 us
        // for 81, of 4 with one of 40 tokens 36 for 27; reading the call's inputs without it 80 and 27.)
        if (tid == 256 && load_acquire_gpu(p.begun) == 0u) pdl_wait();
        __syncthreads();
        // the last CTA to have read it takes it back, beside the schedule
        if (tid == 256 && atomic_add_acq_rel_gpu(p.read, 1u) + 1u == gridDim.x) *p.begun = *p.read = 0u;
    } else {
        pdl_wait_and_release();
    }
    paged_schedule(p.w, sched, scratch, kMinUnits, 0);
    if (warp < 8) paged_zero_rows(p.w, reinterpret_cast<uint4 *>(p.out), p.Hq * D / 8, p.status, 256);
    if (sched->t_begin >= sched->t_end) return;
    PagedWalk w;
    if (!w.init(p.w, *sched)) return;

    if (warp >= 8) {
        // ---- loader: a lane per page ----
        if constexpr (C::SHIFT_REGS) {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
            if (warp > 8) return;
        }
        if (p.test_stall) return;
        const uint64_t pol = l2_policy_evict_first();
        const int ppt = kPagedTile >> p.w.shift;
        const uint32_t box = (uint32_t)(p.S * D * (KV8 ? 1 : 2));
        int i = 0;
        bool ok = true;
        do {
            const int n = w.seg_len();
            if constexpr (KV8) {
                const int per = 32 / ppt;  // tiles of a batch of entries
                PageFeed<PdParams> feed;
                feed.start(p, w, lane);
                for (int t = 0, x = 0; t < n; ++t, ++i, ++x) {
                    if (x == per) {
                        feed.step(p);
                        x = 0;
                    }
                    const int s = i % C::NSTAGE;
                    if (i >= C::NSTAGE) {
                        if (lane == 0) ok = mbar_wait(smem_u32(&empty[s]), ((uint32_t)(i / C::NSTAGE) & 1u) ^ 1u, p.timeout_ns, abort_flag);
                        ok = __shfl_sync(0xffffffffu, ok, 0);
                        if (!ok) break;
                    }
                    const int from = x * ppt + lane;
                    const int row = __shfl_sync(0xffffffffu, feed.row, from), ke = __shfl_sync(0xffffffffu, feed.ke, from),
                              ve = __shfl_sync(0xffffffffu, feed.ve, from);
                    const uint32_t fb = smem_u32(&full[s]);
                    if (lane == 0) mbar_expect_tx(fb, (uint32_t)C::STAGE);
                    __syncwarp();
                    if (lane < ppt) {
                        const uint32_t dst = smem_u32(stages + s * C::STAGE) + (uint32_t)lane * box;
                        tma_load_2d(dst, &kmap, 0, row, fb, pol);
                        tma_load_2d(dst + C::KBYTES, &vmap, 0, row, fb, pol);
                        factors[s * 16 + lane] = page_factors2(ke, ve, feed.far);
                    }
                    __syncwarp();  // the factors are written before the phase can end
                    if (lane == 0) mbar_arrive(fb);
                }
            } else {
                const int held = (int)(((int64_t)w.s.len + p.S - 1) >> p.w.shift);
                const int *table = p.w.table + (int64_t)w.b * p.w.max_pages;
                auto row_of = [&](int tile) {
                    const int e = tile * ppt + lane;
                    if (lane >= ppt || e >= held) return p.zero_row;
                    const int page = table[e];
                    if (page < 0 || page >= p.w.num_pages) {
                        raise_flag(p.status, GQAQ_DEV_BAD_PAGE);
                        return p.zero_row;
                    }
                    return (page * p.w.Hkv + w.kv) << p.w.shift;
                };
                int row = row_of(w.local);
                for (int t = 0; t < n; ++t, ++i) {
                    const int s = i % C::NSTAGE;
                    if (i >= C::NSTAGE) {
                        if (lane == 0) ok = mbar_wait(smem_u32(&empty[s]), ((uint32_t)(i / C::NSTAGE) & 1u) ^ 1u, p.timeout_ns, abort_flag);
                        ok = __shfl_sync(0xffffffffu, ok, 0);
                        if (!ok) break;
                    }
                    const uint32_t fb = smem_u32(&full[s]);
                    if (lane == 0) mbar_arrive_expect_tx(fb, (uint32_t)C::STAGE);
                    __syncwarp();
                    if (lane < ppt) {
                        const uint32_t dst = smem_u32(stages + s * C::STAGE) + (uint32_t)lane * box;
                        tma_load_3d(dst, &kmap, 0, 0, row, fb, pol);
                        tma_load_3d(dst + C::KBYTES, &vmap, 0, 0, row, fb, pol);
                    }
                    if (t + 1 < n) row = row_of(w.local + t + 1);
                }
            }
            if (!ok) break;
        } while (w.advance(p.w));
        if (lane == 0) {
            if (!ok) {
                raise_flag(p.status, GQAQ_DEV_TIMEOUT);
                *abort_flag = 1;
            }
            // every copy issued lands before this CTA may retire, also where a consumer has given up on it
            for (int it = i > C::NSTAGE ? i - C::NSTAGE : 0; it < i; ++it)
                mbar_wait(smem_u32(&full[it % C::NSTAGE]), (uint32_t)(it / C::NSTAGE) & 1u, kLandNs, nullptr);
        }
        return;
    }

    // ---- consumers; after a timeout they still walk and arrive, so the counters stay in step ----
    if constexpr (C::SHIFT_REGS) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    std::conditional_t<KV8, PagedWarp8<D, BF16, NB>, PagedWarp<D, BF16>> wa;
    wa.lane = lane;
    wa.r = lane >> 2;
    wa.c = lane & 3;
    if constexpr (KV8) wa.qs = smem_u32(reinterpret_cast<uint8_t *>(factors) + C::FACTORS) + 8 * lane;
    int i = 0, nsplit = 0;
    do {
        const int n = w.seg_len();
        const bool whole = w.whole();
        const int rows = w.s.m << p.gshift;
        wa.begin(p, w, warp);
        if constexpr (C::SHARED_Q) named_bar_sync(1, 256);  // the item before has been merged behind one
        for (int t = 0; t < n; ++t, ++i) {
            const int s = i % C::NSTAGE;
            bool ok = *abort_flag == 0;
            if (ok) {
                if (lane == 0) ok = mbar_wait(smem_u32(&full[s]), (uint32_t)(i / C::NSTAGE) & 1u, p.timeout_ns, abort_flag);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok && lane == 0) {
                    raise_flag(p.status, GQAQ_DEV_TIMEOUT);
                    *abort_flag = 1;
                }
            }
            const int tok0 = (w.local + t) * kPagedTile + 16 * warp;
            const int rem = min(w.s.len, w.s.start + w.s.m) - tok0;  // tokens some row sees
            if (ok && rem > 0) {
                const uint32_t kb = smem_u32(stages + s * C::STAGE);
                const int n16 = rem < 16 ? rem : 16;
                if constexpr (KV8) {
                    const float2 *f = factors + s * 16;
                    wa.tile(kb, kb + C::KBYTES, 16 * warp, tok0, n16, tok0 + 15 > w.s.start, f[(16 * warp + wa.r) >> p.w.shift],
                            f[(16 * warp + wa.r + 8) >> p.w.shift]);
                } else {
                    wa.tile(kb, kb + C::KBYTES, 16 * warp, tok0, n16, tok0 + 15 > w.s.start, p.scale_log2);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&empty[s]));
        }

        // ---- merge the eight warps' states, MROWS rows at a time ----
        const int64_t out0 = ((int64_t)w.s.q0 * p.Hq + (w.kv << p.gshift)) * D;
        float *part = p.part + ((int64_t)blockIdx.x * 2 + w.slot()) * C::PART;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            for (int first = 8 * b; first < min(rows, 8 * b + 8); first += C::MROWS) {
                wa.store(merge + warp * C::MROWS * (D + 2), b, first);
                named_bar_sync(1, 256);
                const int nr = min(rows - first, (int)C::MROWS);
                for (int x = tid; x < nr * D; x += 256) {
                    const int row = x / D, d = x - row * D;
                    const float *src = merge + row * (D + 2);
                    float mx = -INFINITY;
#pragma unroll
                    for (int j = 0; j < 8; ++j) mx = fmaxf(mx, src[j * C::MROWS * (D + 2)]);
                    float L = 0.f, acc = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float *sj = src + j * C::MROWS * (D + 2);
                        const float f = sj[0] == -INFINITY ? 0.f : fast_exp2(sj[0] - mx);
                        L = fmaf(f, sj[1], L);
                        acc = fmaf(f, sj[2 + d], acc);
                    }
                    const int rho = first + row;
                    if (whole) {
                        p.out[out0 + ((int64_t)(rho >> p.gshift) * p.Hq + (rho & ((1 << p.gshift) - 1))) * D + d] =
                            round16<BF16>(L > 0.f || L != L ? acc / L : 0.f);
                    } else {
                        float *ps = part + rho * (D + 2);
                        ps[2 + d] = acc;
                        if (d == 0) {
                            ps[0] = mx;
                            ps[1] = L;
                        }
                    }
                }
                named_bar_sync(1, 256);
            }
        }
        if (!whole) {
            if (tid == 0) {
                // the barrier above orders every thread's partial stores before this
                // release; the last arrival acquires all of them
                const PagedParts parts(*sched, w.off, w.tiles, 0);
                const unsigned old = atomic_add_acq_rel_gpu(&p.count[parts.lo], 1u);
                PdSplit &sp = split[nsplit];
                sp.off = w.off;
                sp.out = out0;
                sp.tiles = w.tiles;
                sp.rows = rows;
                sp.last = old + 1u == (unsigned)parts.n;
                if (sp.last) p.count[parts.lo] = 0u;
            }
            ++nsplit;  // at most the first and the last segment of a range
        }
    } while (w.advance(p.w));

    if (nsplit == 0) return;
    named_bar_sync(1, 256);  // thread 0's arrivals are recorded
    for (int k = 0; k < nsplit; ++k) {
        const PdSplit sp = split[k];
        if (!sp.last) continue;
        const PagedParts parts(*sched, sp.off, sp.tiles, 0);
        const int np = parts.n;
        // partials: slot 0, but the first CTA's (1)
        const float *base = p.part + parts.lo * 2 * C::PART;
        const float *p0 = base + C::PART;
        for (int x = tid; x < sp.rows * D; x += 256) {
            const int rho = x / D, d = x - rho * D;
            const int at = rho * (D + 2);
            // eight parts at a time, all their loads in flight together
            float mx = -INFINITY, L = 0.f, acc = 0.f;
            for (int j0 = 0; j0 < np; j0 += 8) {
                float2 ml[8];
                float a[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    ml[i] = make_float2(-INFINITY, 0.f);
                    a[i] = 0.f;
                    if (j0 + i < np) {
                        const float *pj = (j0 + i == 0 ? p0 : base + (int64_t)2 * (j0 + i) * C::PART) + at;
                        ml[i] = __ldcg(reinterpret_cast<const float2 *>(pj));
                        a[i] = __ldcg(pj + 2 + d);
                    }
                }
                float top = mx;
#pragma unroll
                for (int i = 0; i < 8; ++i) top = fmaxf(top, ml[i].x);
                const float f0 = mx == -INFINITY ? 0.f : fast_exp2(mx - top);
                L *= f0;
                acc *= f0;
                mx = top;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float f = ml[i].x == -INFINITY ? 0.f : fast_exp2(ml[i].x - top);
                    L = fmaf(f, ml[i].y, L);
                    acc = fmaf(f, a[i], acc);
                }
            }
            p.out[sp.out + ((int64_t)(rho >> p.gshift) * p.Hq + (rho & ((1 << p.gshift) - 1))) * D + d] =
                round16<BF16>(L > 0.f || L != L ? acc / L : 0.f);
        }
    }
}

template <int D, bool BF16, bool KV8, int NB>
__global__ void __launch_bounds__(PdCfg<D, KV8, NB>::THREADS, PdCfg<D, KV8, NB>::MIN_BLOCKS)
    paged_decode_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                        const __grid_constant__ PdParams p) {
    paged_decode<D, BF16, KV8, NB>(kmap, vmap, p);
    if (p.begun != nullptr && threadIdx.x == 0) pdl_wait();
}

template <int D, bool BF16, bool KV8, int NB>
int decode_grid(const LaunchCtx &ctx) {
    using C = PdCfg<D, KV8, NB>;
    // CTAs per SM, asked for once per device
    static std::atomic<int> occ[64] = {};
    if (ctx.device < 0 || ctx.device >= 64) return -1;
    int per_sm = occ[ctx.device].load(std::memory_order_acquire);
    if (per_sm == 0) {
        auto kern = paged_decode_kernel<D, BF16, KV8, NB>;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, C::THREADS, C::SMEM) != cudaSuccess || per_sm < 1)
            return -1;
        if (C::SHIFT_REGS) {  // the warps that ask for more would wait for ever for registers that the launch did not bring
            cudaFuncAttributes attr;
            if (cudaFuncGetAttributes(&attr, kern) != cudaSuccess || attr.numRegs * C::THREADS < 224 * 256 + 56 * 128) return -1;
        }
        if (per_sm > C::MIN_BLOCKS) per_sm = C::MIN_BLOCKS;
        occ[ctx.device].store(per_sm, std::memory_order_release);
    }
    const int grid = per_sm * ctx.num_sms;
    return ctx.max_ctas > 0 && ctx.max_ctas < grid ? ctx.max_ctas : grid;
}

template <int D, bool BF16, bool KV8, int NB>
int launch_decode(const PagedAttnArgs &a, const LaunchCtx &ctx) {
    using C = PdCfg<D, KV8, NB>;
    const gqaq_paged_dims &d = *a.dims;
    const bool beside = a.share == 1;
    const int grid = std::min(decode_grid<D, BF16, KV8, NB>(ctx), (int)(kPagedCountBytes / 8 - (beside ? 2 : 0)));  // a counter each
    if (grid < 1) return GQAQ_ERR_CUDA;
    const uint64_t rows = (uint64_t)d.num_pages * d.num_kv_heads * d.page_size;
    CUtensorMap kmap, vmap;
    if (KV8) {
        if (!encode_tensor_map_u8(&kmap, a.k_pages, rows, D, d.page_size, D)) return GQAQ_ERR_CUDA;
        if (!encode_tensor_map_u8(&vmap, a.v_pages, rows, D, d.page_size, D)) return GQAQ_ERR_CUDA;
    } else {
        if (!encode_tensor_map_kpage(&kmap, a.k_pages, rows, D, d.page_size)) return GQAQ_ERR_CUDA;
        if (!encode_tensor_map_kpage(&vmap, a.v_pages, rows, D, d.page_size)) return GQAQ_ERR_CUDA;
    }
    const int G = d.num_q_heads / d.num_kv_heads;
    PdParams p;
    fill_paged_work(a, 23, 1 << 23, C::ITEM_TILES, p.w);  // one block: every token of a request
    p.q = static_cast<const uint16_t *>(a.q);
    p.out = static_cast<uint16_t *>(a.out);
    // beside another launch's: the second half of the counters, and what lies behind its partials
    unsigned *counters = reinterpret_cast<unsigned *>(a.workspace);
    p.begun = beside ? counters + kPagedBegunWord : nullptr;
    p.read = beside ? counters + kPagedReadWord : nullptr;
    p.count = counters + (beside ? kPagedCountBytes / 8 : 0);
    p.part = reinterpret_cast<float *>(static_cast<uint8_t *>(a.workspace) + (beside ? paged_tc_workspace_bytes(&d, ctx) : kPagedCountBytes));
    p.status = ctx.status;
    p.gshift = G == 1 ? 0 : G == 2 ? 1 : G == 4 ? 2 : 3;
    p.Hq = d.num_q_heads;
    p.S = d.page_size;
    p.zero_row = (int)rows;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.timeout_ns = ctx.timeout_ns;
    p.test_stall = ctx.test_stall;
    p.k_exp = a.k_exp;
    p.v_exp = a.v_exp;
    const cudaError_t e = launch_kernel(paged_decode_kernel<D, BF16, KV8, NB>, dim3((unsigned)grid), dim3(C::THREADS), C::SMEM, ctx, 0,
                                        kmap, vmap, p);
    return e == cudaSuccess ? GQAQ_OK : GQAQ_ERR_CUDA;
}

// Blocks of eight rows that the decode kernel takes over 8-bit pages, both sides measured against the tensor-memory
// kernel (four query heads per KV head, bf16). 32 requests of 500 to 4K, 8 KV heads: 64 channels, 1 to 4 blocks 28, 39, 45
// and 57 us against 59; 128 channels, 1 to 3 blocks 47, 53 and 64 against 72. More do not fit the registers. Few requests
// at 4K, whose parts one CTA merges: 64 channels, 3 blocks 16 to 19 against 19 to 26; 4 blocks, one request 21 to 24 against 19
// to 20, two requests or eight on one KV head 23 and 24 against 23, four on eight 23 against 26; 128 channels, 2 blocks 19 to
// 22 against 25 to 32, 3 blocks of one request 25 to 26 on either side, of more 26 to 27 against 28 to 33. So only
// the fourth block of a single request goes to the other kernel. One number serves the whole batch, from max_q_len, so
// requests of fewer rows compute with the blocks of the longest (of 500 to 4K, 64 and 128 channels: 32 single tokens 27 and
// 41 us, 31 and one of five tokens 47 and 63, 32 of five 47 and 64).
constexpr int kMostBlocks64 = 4, kMostBlocks128 = 3;
int most_blocks(const gqaq_paged_dims &d) { return d.head_dim == 128 ? kMostBlocks128 : d.batch == 1 ? kMostBlocks64 - 1 : kMostBlocks64; }

// Floats of the partials of an SM's CTAs, in the widest of the kernel's forms.
template <int D, int NB>
constexpr size_t part_floats() {
    const size_t mine = 2 * PdCfg<D, true, NB>::MIN_BLOCKS * PdCfg<D, true, NB>::PART;
    if constexpr (NB == 1) return mine;
    else return std::max(mine, part_floats<D, NB - 1>());
}
size_t decode_part_bytes(const gqaq_paged_dims *d, const LaunchCtx &ctx) {
    return ctx.num_sms * (d->head_dim == 128 ? part_floats<128, kMostBlocks128>() : part_floats<64, kMostBlocks64>()) * sizeof(float);
}

template <int D, bool KV8, int NB>
int launch_blocks(const PagedAttnArgs &a, const LaunchCtx &ctx) {
    return a.dims->dtype == GQAQ_BF16 ? launch_decode<D, true, KV8, NB>(a, ctx) : launch_decode<D, false, KV8, NB>(a, ctx);
}
int launch_rows16(const PagedAttnArgs &a, const LaunchCtx &ctx) {  // 16-bit pages: eight rows
    return a.dims->head_dim == 128 ? launch_blocks<128, false, 1>(a, ctx) : launch_blocks<64, false, 1>(a, ctx);
}
int launch_rows8(const PagedAttnArgs &a, int blocks, const LaunchCtx &ctx) {  // 8-bit pages
    if (a.dims->head_dim == 128) {
        switch (blocks) {
            case 1: return launch_blocks<128, true, 1>(a, ctx);
            case 2: return launch_blocks<128, true, 2>(a, ctx);
            default: return launch_blocks<128, true, 3>(a, ctx);
        }
    }
    switch (blocks) {
        case 1: return launch_blocks<64, true, 1>(a, ctx);
        case 2: return launch_blocks<64, true, 2>(a, ctx);
        case 3: return launch_blocks<64, true, 3>(a, ctx);
        default: return launch_blocks<64, true, 4>(a, ctx);
    }
}

}  // namespace

// Both kernels' partials, since they may run beside each other. Each has half of the counters, one for each of its CTAs.
size_t paged_attn_workspace_bytes(const gqaq_paged_dims *d, const LaunchCtx &ctx) {
    return paged_tc_workspace_bytes(d, ctx) + decode_part_bytes(d, ctx);
}

int launch_paged_attn(const PagedAttnArgs &a, const LaunchCtx &ctx) {
    if (a.workspace_bytes < paged_attn_workspace_bytes(a.dims, ctx)) return GQAQ_ERR_WORKSPACE;
    // Up to eight rows per KV head, over 8-bit pages up to most_blocks times that: the decode kernel (32 query and 8 KV heads of
    // 64 channels: one request at 4K 10.4 us against 18.4, 32 requests of 1K to 4K 31.4 against 43.8; over 8-bit pages 10.0
    // against 19.0 and, of 500 to 4K, 25 against 60). Above, the tensor-memory kernel (16-bit pages, 16 requests of up to 9K
    // with 3 to 6 drafted tokens, 12 to 24 rows: 44 to 65 us, where two and three N blocks of mma.sync took 52 to 196).
    const int64_t rows = (int64_t)a.max_q_len * (a.dims->num_q_heads / a.dims->num_kv_heads);
    if (a.k_exp == nullptr) return rows > kRows ? launch_paged_tc(a, ctx) : launch_rows16(a, ctx);
    if (rows <= most_blocks(*a.dims) * kRows) return launch_rows8(a, (int)(rows + kRows - 1) / kRows, ctx);
    if (a.dims->batch == 1) return launch_paged_tc_e4m3(a, ctx);
    // Over 8-bit pages a batch whose longest request goes there may hold short ones too: those of up to eight rows go to the
    // decode kernel, by their own rows, in a launch beside it (a mixed batch 107 -> 81 us; the two alone 60 and 23). One of nine
    // rows and more shares the tensor-memory kernel, where it costs a row tile.
    PagedAttnArgs part = a;
    part.share = 2;
    const int rc = launch_paged_tc_e4m3(part, ctx);
    part.share = 1;
    return rc != GQAQ_OK ? rc : launch_rows8(part, 1, ctx);
}

}  // namespace gqaq
