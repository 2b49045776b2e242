// paged_attn_tc.cu -- paged attention on the 5th-generation tensor cores, for
// chunks of new tokens and for batches that mix chunks with single tokens.
//
// Mathematics: per row, softmax(scale q . k) v over the row's keys in one
// pass. P = 2^(s - ref) against a reference that follows the row's maximum
// only when it has to: while the sum of a tile's P stays under 2^15 nothing is
// rescaled (P fits fp16, and the reference sits 2^6 under the maximum that set
// it, so small P keep their bits); otherwise the row's sum and output move to
// the new reference. Sums and outputs are held in 32 bits; each P is rounded
// once to the dtype, as the tensor core takes it.
//
// Kernel shape (one persistent CTA per SM, one launch):
//  - an item is 256 rows (two tiles of 128) of one (request, KV head), see
//    paged_sched.cuh; a CTA walks the tiles of its range.
//  - warp 16 loads Q and the K tiles, warp 18 the V tiles: one 64-channel box
//    of S rows per page and column block, so a tile of 128 tokens is gathered
//    from its pages in the order of the table; each tile lands in a ring of
//    its own. Boxes of pages past the request read out of bounds: zeros.
//  - warp 17 issues the MMAs: S = Q K^T (M 128, N 128) and O += P V (A = P from
//    tensor memory, B = V, N = D).
//  - warps 0-7 and 8-15 are two softmax groups, two threads per row (64 tokens
//    each: twice the warps halve the time from S to P, which the tensor core
//    waits for), each group with its own S and O in tensor memory (S0, S1, O0,
//    O1: 512 columns at D = 128).
//    An item of two row tiles gives each group one of them; every K / V tile
//    then serves 256 rows. An item of one row tile gives both groups the same
//    rows and every other K / V tile, and they merge at its end. Either way
//    the tensor core works for one group while the other takes its softmax.
//  - an item cut by the end of a range leaves fp32 partials (m, l, acc), laid
//    out [channel / 4][row] so that a warp's stores are contiguous; the CTA
//    that arrives last merges them and resets the counter.
//  - warp 19 watches the S barriers for the softmax warps. These clear the rows
//    of a last page's V that lie past its request.
//
// What bounds it. Where a chunk is long (1024 tokens at the end of 32K, 32 heads
// of 128 channels): in bursts at 2,070 MHz the chain from S over the softmax to
// PV (420 us, 1,290 TFLOP/s, 68% of the measured GEMM rate; at 8K the tensor
// pipe is busy 48% of the cycles, the one of the exponentials 24%), in a running
// stream the power cap (1,370 W, 1,570 MHz: 475 us, 67% of the sustained rate).
// HBM where rows are few (five drafted tokens of 16 requests, contexts up to 9K,
// 8 KV heads of 128 channels: 34 tiles of 64 KB in 43.5 of 64 us on each SM),
// and the start and end of items where contexts are short (3 to 4 us each).
#include <math.h>

#include "paged_sched.cuh"
#include "umma.cuh"

namespace gqaq {
namespace {

template <int D>
struct PtcCfg {
    static constexpr int THREADS = 640;              // 16 softmax warps, K, MMA, V, notifier
    static constexpr int RB = 256;                   // rows per item
    static constexpr int KH = D / 64;                // 64-channel blocks
    static constexpr int BLK = 128 * 128;            // one block of 128 rows
    static constexpr int TILE = KH * BLK;            // a Q, K or V tile
    static constexpr int NK = D == 128 ? 2 : 4;      // K ring
    static constexpr int NV = D == 128 ? 3 : 6;      // V ring
    static constexpr int MISC = 2048;                // 1 KB of (m, l), barriers, schedule
    static constexpr int SMEM = 1024 + (2 + NK + NV) * TILE + MISC;
    static constexpr int O_COL = 0, S_COL = 256;     // O of group g at 128 g, S at 256 + 128 g
    static constexpr int ML = 2 * RB;                // floats of a partial's (m, l)
    static constexpr int PART = ML + RB * D;         // floats of a partial
    static_assert(SMEM <= 227 * 1024, "shared memory");
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

// The softmax warps' place in the CTA's range. One thread moves it on and all
// read it from shared memory: held by each thread it spilled registers of the
// loop over tiles, whose reloads missed the small L1 that is left beside the
// tiles (2 of 3.5 thousand cycles per tile).
struct PtcSegment {
    PagedWorkParams p;  // the launch's, for the calls below (through a reference to the kernel's parameter each field was a slow load)
    PagedWalk w;
    int v_before;  // V tiles before this segment
    int more;
};

// One thread's work on it, as calls of their own: in registers, away from the
// loop's (on the copy in shared memory the first took 2.9 us).
__device__ __noinline__ bool segment_begin(PtcSegment &at, const PagedSched &sched) {
    const PagedWorkParams p = at.p;
    const PagedSched s = sched;
    PagedWalk w;
    const bool more = w.init(p, s);
    at.w = w;
    return more;
}
__device__ __noinline__ bool segment_next(PtcSegment &at) {
    const PagedWorkParams p = at.p;
    PagedWalk w = at.w;
    const bool more = w.advance(p);
    at.w = w;
    return more;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(PtcCfg<D>::THREADS, 1)
    paged_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap vmap, const __grid_constant__ PtcParams p) {
    using C = PtcCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *sq = smem;                        // two Q tiles
    uint8_t *sk = sq + 2 * C::TILE;
    uint8_t *sv = sk + C::NK * C::TILE;
    float *xchg = reinterpret_cast<float *>(sv + C::NV * C::TILE);  // [256]
    uint64_t *kfull = reinterpret_cast<uint64_t *>(xchg + 256);
    uint64_t *kempty = kfull + C::NK;
    uint64_t *vfull = kempty + C::NK;
    uint64_t *vempty = vfull + C::NV;
    uint64_t *qfull = vempty + C::NV;
    uint64_t *qempty = qfull + 1;
    uint64_t *s_ready = qempty + 1;   // [2]
    uint64_t *p_ready = s_ready + 2;  // [2]
    uint64_t *o_done = p_ready + 2;   // [2]: a group's last PV of a segment
    uint64_t *o_free = o_done + 2;    // the epilogue has read O
    uint64_t *drain = o_free + 1;
    int64_t *scratch = reinterpret_cast<int64_t *>(drain + 1);  // [12]
    PagedSched *sched = reinterpret_cast<PagedSched *>(scratch + 12);
    PtcSegment *seg_s = reinterpret_cast<PtcSegment *>(sched + 1);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(seg_s + 1);
    static_assert(256 * 4 + (2 * C::NK + 2 * C::NV + 10 + 12) * 8 + sizeof(PagedSched) + sizeof(PtcSegment) + 8 <= C::MISC, "misc region");
    volatile int *abort_flag = &sched->abort;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) seg_s->p = p.w;
    if (warp == 16 && lane == 0) {
        for (int s = 0; s < C::NK; ++s) {
            mbar_init(smem_u32(&kfull[s]), 1);
            mbar_init(smem_u32(&kempty[s]), 1);
        }
        for (int s = 0; s < C::NV; ++s) {
            mbar_init(smem_u32(&vfull[s]), 1);
            mbar_init(smem_u32(&vempty[s]), 1);
        }
        mbar_init(smem_u32(qfull), 1);
        mbar_init(smem_u32(qempty), 1);
        for (int g = 0; g < 2; ++g) {
            mbar_init(smem_u32(&s_ready[g]), 1);
            mbar_init(smem_u32(&p_ready[g]), 8);  // the group's warps
            mbar_init(smem_u32(&o_done[g]), 1);
        }
        mbar_init(smem_u32(o_free), 16);
        mbar_init(smem_u32(drain), 1);
        fence_mbar_init();
        prefetch_tensormap(&qmap);
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
    }
    if (warp == 17) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)), "n"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    pdl_wait_and_release();
    tc_fence_before();
    paged_schedule(p.w, sched, scratch, kMinUnits, D / 64);  // a part of 256 rows is 66 KB per 64 channels: two units' time
    tc_fence_after();
    const uint32_t tbase = *tslot;
    if (warp < 16) paged_zero_rows(p.w, reinterpret_cast<uint4 *>(p.out), p.Hq * D / 8, p.status, 512);
    const bool work = sched->t_begin < sched->t_end;

    if (work) {
        const int TB = C::RB >> p.gshift;  // tokens of an item
        if ((warp == 16 || warp == 18) && !p.test_stall) {
            // --------------------------------------------------------------
            // Loaders: K (and Q) in warp 16, V in warp 18. A lane per page.
            // --------------------------------------------------------------
            PagedWalk w;
            bool more = w.init(p.w, *sched);
            const bool is_k = warp == 16;
            const int NS = is_k ? C::NK : C::NV;
            uint64_t *full = is_k ? kfull : vfull, *empty = is_k ? kempty : vempty;
            const CUtensorMap *map = is_k ? &kmap : &vmap;
            uint8_t *ring = is_k ? sk : sv;
            const uint64_t pol = l2_policy_evict_first();
            const int ppt = kPagedTile >> p.w.shift;
            int seg = 0, i = 0, n_q = 0;  // segments, tiles and Q tiles asked for
            bool ok = true;
            while (more) {
                const int n = w.seg_len();
                const int rows = min(TB, w.s.m - w.rb * TB) * p.G;
                if (is_k) {
                    if (seg > 0) {
                        ok = warp_mbar_wait_slow(smem_u32(qempty), (uint32_t)(seg - 1) & 1u, p.timeout_ns, abort_flag);
                        if (!ok) break;
                    }
                    ++n_q;
                    if (lane == 0) {
                        const int nq = rows > 128 ? 2 : 1;
                        mbar_arrive_expect_tx(smem_u32(qfull), (uint32_t)(nq * C::TILE));
                        for (int x = 0; x < nq; ++x)
                            for (int kh = 0; kh < C::KH; ++kh)
                                tma_load_3d(smem_u32(sq) + x * C::TILE + kh * C::BLK, &qmap, 64 * kh, w.kv * p.G,
                                            w.s.q0 + w.rb * TB + x * (TB / 2), smem_u32(qfull), pol);
                    }
                }
                const int held = (int)(((int64_t)w.s.len + p.S - 1) >> p.w.shift);
                const int *table = p.w.table + (int64_t)w.b * p.w.max_pages;
                auto row_of = [&](int tile) {  // this lane's page of the tile, as a row of the pool
                    const int e = tile * ppt + lane;
                    if (lane >= ppt || e >= held) return p.zero_row;
                    const int page = table[e];
                    if (page < 0 || page >= p.w.num_pages) {
                        if (is_k) raise_flag(p.status, GQAQ_DEV_BAD_PAGE);
                        return p.zero_row;
                    }
                    return (page * p.w.Hkv + w.kv) << p.w.shift;
                };
                int row = row_of(w.local);
                for (int t = 0; t < n; ++t, ++i) {
                    const int s = i % NS;
                    if (i >= NS) {
                        ok = warp_mbar_wait_slow(smem_u32(&empty[s]), ((uint32_t)(i / NS) & 1u) ^ 1u, p.timeout_ns, abort_flag);
                        if (!ok) break;
                    }
                    const uint32_t fb = smem_u32(&full[s]);
                    if (lane == 0) mbar_arrive_expect_tx(fb, (uint32_t)C::TILE);
                    __syncwarp();
                    if (lane < ppt) {
                        const uint32_t dst = smem_u32(ring) + (uint32_t)(s * C::TILE) + ((uint32_t)lane << (p.w.shift + 7));
#pragma unroll
                        for (int kh = 0; kh < C::KH; ++kh) tma_load_2d(dst + kh * C::BLK, map, 64 * kh, row, fb, pol);
                    }
                    if (t + 1 < n) row = row_of(w.local + t + 1);
                }
                if (!ok) break;
                ++seg;
                more = w.advance(p.w);
            }
            if (lane == 0) {
                if (!ok) {
                    raise_flag(p.status, GQAQ_DEV_TIMEOUT);
                    *abort_flag = 1;
                }
                // every copy issued lands before this CTA may retire, also where another warp has given up on it
                for (int it = i > NS ? i - NS : 0; it < i; ++it)
                    mbar_wait(smem_u32(&full[it % NS]), (uint32_t)(it / NS) & 1u, kLandNs, nullptr);
                if (n_q > 0) mbar_wait(smem_u32(qfull), (uint32_t)(n_q - 1) & 1u, kLandNs, nullptr);
            }
        } else if (warp == 17) {
            // --------------------------------------------------------------
            // MMA issuer (the whole warp walks, one elected lane issues).
            // Products alternate between the groups: event e is tile e / 2 of
            // group e % 2 (two row tiles), or tile e for group e % 2 (one).
            // S(e + 2) follows PV(e), which frees its tensor memory: the core
            // runs one thread's MMAs in order.
            // --------------------------------------------------------------
            PagedWalk w;
            bool more = w.init(p.w, *sched);
            constexpr uint32_t IDESC_S = umma_idesc(128, 128, 0, BF16);
            constexpr uint32_t IDESC_O = umma_idesc(128, D, 1, BF16);
            const uint64_t qdesc0 = umma_desc(smem_u32(sq), 16);
            const uint64_t kdesc0 = umma_desc(smem_u32(sk), 16);
            const uint64_t vdesc0 = umma_desc(smem_u32(sv), C::BLK);
            int ks = 0, vs = 0;             // ring slots and their phases
            uint32_t kp = 0, vp = 0;
            uint32_t pp = 0;                // phases of p_ready (bits 0, 1)
            uint32_t sp = 0;                // phase of the segment's barriers
            bool first_seg = true, ok = true;
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                return warp_mbar_wait(smem_u32(bar), parity, p.timeout_ns, abort_flag);
            };
            auto segment = [&](auto dual_c, int ne) {
                constexpr bool DUAL = decltype(dual_c)::value;
                auto issue_s = [&](int e) {
                    const int x = e & 1;
                    if (!DUAL || x == 0) ok = wait(&kfull[ks], kp);
                    if (!ok) return;
                    tc_fence_after();
                    const uint64_t qd = qdesc0 + (uint64_t)(DUAL && x ? C::TILE >> 4 : 0);
                    const uint64_t kd = kdesc0 + (uint64_t)(ks * (C::TILE >> 4));
                    const uint32_t sd = tbase + C::S_COL + 128u * (uint32_t)x;
#pragma unroll
                    for (int kh = 0; kh < C::KH; ++kh)
                        warp_mma_ss4(sd, qd + (uint64_t)(kh * (C::BLK >> 4)), kd + (uint64_t)(kh * (C::BLK >> 4)), IDESC_S, kh > 0);
                    warp_commit(smem_u32(&s_ready[x]));
                    if (!DUAL || x == 1) {
                        warp_commit(smem_u32(&kempty[ks]));
                        if (++ks == C::NK) {
                            ks = 0;
                            kp ^= 1u;
                        }
                    }
                    if (e == ne - 1) warp_commit(smem_u32(qempty));
                };
                issue_s(0);
                if (ok && ne > 1) issue_s(1);
#pragma unroll 1
                for (int e = 0; e < ne && ok; ++e) {
                    const int x = e & 1;
                    if (!DUAL || x == 0) ok = wait(&vfull[vs], vp);
                    if (e == 0 && !first_seg) ok = ok && wait(o_free, sp ^ 1u);  // the last segment's O has been read
                    ok = ok && wait(&p_ready[x], (pp >> x) & 1u);
                    if (!ok) break;
                    pp ^= 1u << x;
                    tc_fence_after();
                    const uint64_t vd = vdesc0 + (uint64_t)(vs * (C::TILE >> 4));
                    const uint32_t od = tbase + C::O_COL + 128u * (uint32_t)x, pd = tbase + C::S_COL + 128u * (uint32_t)x;
                    warp_mma_ts4(od, pd, vd, IDESC_O, e > 1);              // P of tokens 0-63: columns 0-31
                    warp_mma_ts4(od, pd + 64u, vd + 512u, IDESC_O, 1);     // of tokens 64-127: columns 64-95
                    if (!DUAL || x == 1) {
                        warp_commit(smem_u32(&vempty[vs]));
                        if (++vs == C::NV) {
                            vs = 0;
                            vp ^= 1u;
                        }
                    }
                    if (e + 2 >= ne) warp_commit(smem_u32(&o_done[x]));
                    if (e + 2 < ne) issue_s(e + 2);
                }
            };
            while (more) {
                const int n = w.seg_len();
                const int rows = min(TB, w.s.m - w.rb * TB) * p.G;
                ok = wait(qfull, sp);
                if (ok) {
                    if (rows > 128) segment(std::true_type(), 2 * n);
                    else segment(std::false_type(), n);
                }
                sp ^= 1u;
                first_seg = false;
                more = ok && w.advance(p.w);
            }
            if (!ok && lane == 0) {
                raise_flag(p.status, GQAQ_DEV_TIMEOUT);
                *abort_flag = 1;
            }
            __syncwarp();
            warp_commit(smem_u32(drain));  // every issued MMA completes before TMEM is released
            mbar_wait(smem_u32(drain), 0u, kLandNs, nullptr);
            __syncwarp();
        } else if (warp == 19) {
            // --------------------------------------------------------------
            // Notifier: watches the S barriers for the softmax warps, which wait
            // at a hardware barrier per group instead. Sixteen warps that probe
            // a shared-memory barrier fill the queue that every arrival and
            // every other barrier goes through.
            // --------------------------------------------------------------
            PagedWalk w;
            bool more = w.init(p.w, *sched);
            uint32_t sph = 0;
            bool ok = true;
            while (more) {
                const int n = w.seg_len();
                const int ne = min(TB, w.s.m - w.rb * TB) * p.G > 128 ? 2 * n : n;
                for (int e = 0; e < ne; ++e) {
                    const int x = e & 1;
                    if (ok) {
                        ok = warp_mbar_wait(smem_u32(&s_ready[x]), (sph >> x) & 1u, p.timeout_ns, abort_flag);
                        if (!ok && lane == 0) {
                            raise_flag(p.status, GQAQ_DEV_TIMEOUT);
                            *abort_flag = 1;
                        }
                    }
                    sph ^= 1u << x;
                    tc_fence_after();
                    tc_fence_before();
                    named_bar_sync(10 + x, 288);  // also after a timeout: the groups pass once per tile
                }
                more = w.advance(p.w);
            }
        } else if (warp < 16) {
            // --------------------------------------------------------------
            // Softmax groups: two threads per row, tokens 64 h .. 64 h + 63 of
            // a tile each. They share the row's reference and agree on moving
            // it (a predicate over the pair of warps); each keeps its sum.
            // --------------------------------------------------------------
            const int g = warp >> 3, h = (warp >> 2) & 1, row = (warp & 3) * 32 + lane, tid = threadIdx.x;
            const int pair_bar = 2 + g * 4 + (warp & 3);
            const uint32_t tlane = tbase + ((uint32_t)((warp & 3) * 32) << 16);
            const uint32_t scol = tlane + C::S_COL + 128u * (uint32_t)g + 64u * (uint32_t)h;
            const uint32_t ocol = tlane + C::O_COL + 128u * (uint32_t)g + (uint32_t)(h * (D / 2));  // the half it rescales
            const float mul = p.scale_log2;              // any sign, not zero
            const float hide = mul > 0.f ? -INFINITY : INFINITY;  // a masked score: its product is -inf
            uint32_t oph = 0;  // phase of o_done
            bool ok = true;
            if (tid == 0) {
                seg_s->more = segment_begin(*seg_s, *sched);
                seg_s->v_before = 0;
            }
            named_bar_sync(1, 512);
            const PagedWalk &w = seg_s->w;
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                const bool r = warp_mbar_wait(smem_u32(bar), parity, p.timeout_ns, abort_flag);
                if (!r && lane == 0) {
                    raise_flag(p.status, GQAQ_DEV_TIMEOUT);
                    *abort_flag = 1;
                }
                return r;
            };
            while (seg_s->more) {
                const int n = w.seg_len();
                const int rows = min(TB, w.s.m - w.rb * TB) * p.G;
                const bool dual = rows > 128;
                const int nx = dual ? n : (n + 1 - g) / 2;          // this group's tiles
                const int r0 = dual ? 128 * g : 0;                  // its first row
                const int rho = r0 + row;                           // this thread's
                const bool live = rho < rows, warp_live = r0 + (warp & 3) * 32 < rows;
                const int pos0 = w.s.start + w.rb * TB;             // the block's first position
                const int first0 = w.local * kPagedTile, len = w.s.len;
                const int lim = pos0 + (rho >> p.gshift);           // this row's
                const int lim_lo = pos0 + ((r0 + (warp & 3) * 32) >> p.gshift);  // the warp's least
                // a row behind the item's weighs nothing and never has its reference moved, so that no other depends on it
                float ref = live ? -INFINITY : INFINITY, l = 0.f;
                for (int k = 0; k < nx; ++k) {
                    const int jj = dual ? k : 2 * k + g;             // tile within the segment
                    const int tile0 = first0 + jj * kPagedTile;      // its first token
                    const int tok0 = tile0 + 64 * h;                 // this thread's
                    named_bar_sync(10 + g, 288);  // S is complete (after a timeout it holds anything)
                    tc_fence_after();
                    if (warp_live) {
                        const bool mask = tok0 + 63 > lim_lo;  // warp-uniform
                        uint32_t pk[32];
                        // P of these tokens against reference r; returns their sum
                        auto exps = [&](float r) {
                            const float nref = r == -INFINITY ? 0.f : -r;
                            const uint64_t mul2 = pair32(mul, mul), nref2 = pair32(nref, nref);
                            uint64_t sum0 = 0, sum1 = 0;  // two pairs of partial sums
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                uint32_t x[32];
                                tmem_ld32_async(scol + 32u * c, x);
                                tmem_ld32_wait(x);
                                if (__builtin_expect(mask, 0)) {
#pragma unroll
                                    for (int e = 0; e < 32; ++e)
                                        if (tok0 + 32 * c + e > lim) x[e] = __float_as_uint(hide);
                                }
#pragma unroll
                                for (int e = 0; e < 32; e += 2) {
                                    const float2 y = unpair32(fma2(pair32(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), mul2, nref2));
                                    const float e0 = fast_exp2(y.x), e1 = fast_exp2(y.y);
                                    uint64_t &sum = (e & 2) ? sum1 : sum0;
                                    sum = add2(sum, pair32(e0, e1));
                                    pk[16 * c + (e >> 1)] = pack2<BF16>(e0, e1);
                                }
                            }
                            const float2 t = unpair32(add2(sum0, sum1));
                            return t.x + t.y;
                        };
                        float cs = 0.f;
                        const bool fresh = __all_sync(0xffffffffu, fabsf(ref) == INFINITY);  // of both warps: they share ref
                        // one copy of the exponentials serves both passes: the second, after a
                        // row's reference has moved, is rare, and code that is jumped over costs fetches
#pragma unroll 1
                        for (int pass = fresh ? 0 : 1;; ++pass) {
                            if (pass > 0) cs = exps(ref);
                            if (pass > 1) break;
                            const bool redo = (ref == -INFINITY && lim >= tile0) || cs > kSumLimit;  // the row's first keys, or far above
                            if (__builtin_expect(!pair_any(pair_bar, redo), 1)) {
                                if (pass == 0) {
#pragma unroll
                                    for (int e = 0; e < 32; ++e) pk[e] = 0u;  // every row of the pair is masked in this tile
                                }
                                break;
                            }
                            // the row's maximum over both halves becomes the reference
                            float r4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                            for (int c = 0; c < 2; ++c) {
                                uint32_t x[32];
                                tmem_ld32(scol + 32u * c, x);
#pragma unroll
                                for (int e = 0; e < 32; ++e) {
                                    const float y = tok0 + 32 * c + e > lim ? -INFINITY : __uint_as_float(x[e]) * mul;
                                    r4[e & 3] = fmaxf(r4[e & 3], y);
                                }
                            }
                            float top = fmaxf(fmaxf(r4[0], r4[1]), fmaxf(r4[2], r4[3]));
                            float *slot = xchg + 128 * g + row;
                            if (h == 1) *slot = top;
                            named_bar_sync(pair_bar, 64);
                            if (h == 0) *slot = top = fmaxf(top, *slot);
                            named_bar_sync(pair_bar, 64);
                            if (h == 1) top = *slot;
                            float alpha = 1.f;
                            if (top > ref + kRefMove) {  // any maximum, where there is no reference yet
                                alpha = fast_exp2(ref - (top - kRefDrop));
                                ref = top - kRefDrop;
                                l *= alpha;
                            }
                            if (k > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                                // S of this tile is complete, hence every earlier PV of the group
#pragma unroll 1
                                for (int c = 0; c < D / 2; c += 32) {
                                    uint32_t o[32];
                                    tmem_ld32(ocol + (uint32_t)c, o);
#pragma unroll
                                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                                    tmem_st32(ocol + (uint32_t)c, o);
                                }
                            }
                            pass = 1;  // the next pass is the last
                        }
                        l += cs;
                        tmem_st32(scol, pk);  // over the first half of the scores it read
                        tmem_wait_st();
                    }
                    // rows of the last page past the request may hold anything: zero
                    // them, so that 0 * NaN cannot reach O (pages past it read zeros)
                    if (__builtin_expect(ok && (g == 0 || !dual) && len < tile0 + kPagedTile && (len & (p.S - 1)) != 0, 0)) {
                        const int v = seg_s->v_before + jj, s = v % C::NV;
                        ok = wait(&vfull[s], (uint32_t)(v / C::NV) & 1u);
                        if (ok && tile0 + row >= len && h < C::KH) {
#pragma unroll
                            for (int q = 0; q < 8; ++q)
                                *reinterpret_cast<uint4 *>(sv + s * C::TILE + h * C::BLK + row * 128 + q * 16) = make_uint4(0u, 0u, 0u, 0u);
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&p_ready[g]));
                }

                // ---- epilogue: sums of the two halves, then of the two groups if they share the rows ----
                if (nx > 0) {
                    ok = ok && wait(&o_done[g], oph);
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
                if (lane == 0) mbar_arrive(smem_u32(o_free));
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
                named_bar_sync(1, 512);  // the segment has been read
                if (tid == 0) {
                    seg_s->v_before += n;
                    seg_s->more = segment_next(*seg_s);
                }
                named_bar_sync(1, 512);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 17) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tbase), "n"(512));
}

template <int D, bool BF16>
int launch_t(const PagedAttnArgs &a, const LaunchCtx &ctx) {
    using C = PtcCfg<D>;
    static std::atomic<uint64_t> ready{0};
    const int rc = allow_smem(reinterpret_cast<const void *>(paged_tc_kernel<D, BF16>), C::SMEM, ready, ctx);
    if (rc != GQAQ_OK) return rc;
    const gqaq_paged_dims &d = *a.dims;
    const int grid = paged_tc_grid(ctx);
    const uint64_t rows = (uint64_t)d.num_pages * d.num_kv_heads * d.page_size;
    PtcParams p;
    p.G = d.num_q_heads / d.num_kv_heads;
    p.gshift = p.G == 1 ? 0 : p.G == 2 ? 1 : p.G == 4 ? 2 : 3;
    fill_paged_work(a, 8 - p.gshift, 128 >> p.gshift, kItemTiles, p.w);  // blocks of 256 rows; above 128 a tile runs twice
    CUtensorMap qmap, kmap, vmap;
    if (!encode_tensor_map_heads(&qmap, a.q, d.max_tokens, d.num_q_heads, D, p.G, 128 / p.G)) return GQAQ_ERR_CUDA;
    if (!encode_tensor_map_2d(&kmap, a.k_pages, rows, D, 64, d.page_size, true)) return GQAQ_ERR_CUDA;
    if (!encode_tensor_map_2d(&vmap, a.v_pages, rows, D, 64, d.page_size, true)) return GQAQ_ERR_CUDA;
    p.out = static_cast<uint16_t *>(a.out);
    p.count = reinterpret_cast<unsigned *>(a.workspace);
    p.part = reinterpret_cast<float *>(static_cast<uint8_t *>(a.workspace) + kPagedCountBytes);
    p.status = ctx.status;
    p.Hq = d.num_q_heads;
    p.S = d.page_size;
    p.zero_row = (int)rows;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    if (p.scale_log2 == 0.f) p.scale_log2 = 1e-30f;  // 2^(s - max) is 1 all the same, and a masked score's product stays -inf
    p.timeout_ns = ctx.timeout_ns;
    p.test_stall = ctx.test_stall;
    p.wide_out = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
    const cudaError_t e = launch_kernel(paged_tc_kernel<D, BF16>, dim3((unsigned)grid), dim3(C::THREADS), C::SMEM, ctx, 0, qmap,
                                        kmap, vmap, p);
    return e == cudaSuccess ? GQAQ_OK : GQAQ_ERR_CUDA;
}

}  // namespace

int paged_tc_grid(const LaunchCtx &ctx) {
    return ctx.max_ctas > 0 && ctx.max_ctas < ctx.num_sms ? ctx.max_ctas : ctx.num_sms;
}

size_t paged_tc_workspace_bytes(const gqaq_paged_dims *d, const LaunchCtx &ctx) {
    const size_t part = d->head_dim == 128 ? PtcCfg<128>::PART : PtcCfg<64>::PART;
    return kPagedCountBytes + (size_t)ctx.num_sms * 2 * part * sizeof(float);
}

int launch_paged_tc(const PagedAttnArgs &a, const LaunchCtx &ctx) {
    if (a.dims->dtype == GQAQ_BF16) return a.dims->head_dim == 128 ? launch_t<128, true>(a, ctx) : launch_t<64, true>(a, ctx);
    return a.dims->head_dim == 128 ? launch_t<128, false>(a, ctx) : launch_t<64, false>(a, ctx);
}

}  // namespace gqaq
