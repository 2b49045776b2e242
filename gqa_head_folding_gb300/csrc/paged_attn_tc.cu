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
//  - warp 8 loads Q and the K tiles, warp 10 the V tiles: one 64-channel box
//    of S rows per page and column block, so a tile of 128 tokens is gathered
//    from its pages in the order of the table; each tile lands in a ring of
//    its own. Boxes of pages past the request read out of bounds: zeros.
//  - warp 9 issues the MMAs: S = Q K^T (M 128, N 128) and O += P V (A = P from
//    tensor memory, B = V, N = D).
//  - warps 0-3 and 4-7 are two softmax groups, a thread per row, each with its
//    own S and O in tensor memory (S0, S1, O0, O1: 512 columns at D = 128).
//    An item of two row tiles gives each group one of them; every K / V tile
//    then serves 256 rows. An item of one row tile gives both groups the same
//    rows and every other K / V tile, and they merge at its end. Either way
//    the tensor core works for one group while the other takes its softmax.
//  - an item cut by the end of a range leaves fp32 partials (m, l, acc), laid
//    out [channel / 4][row] so that a warp's stores are contiguous; the CTA
//    that arrives last merges them and resets the counter.
#include <math.h>

#include "paged_sched.cuh"
#include "umma.cuh"

namespace gqaq {
namespace {

template <int D>
struct PtcCfg {
    static constexpr int THREADS = 352;              // 8 softmax warps, K, MMA, V
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

constexpr int kMinTiles = 2;        // tiles per CTA below which a small step uses fewer CTAs
constexpr float kSumLimit = 32768.f;
constexpr float kRefDrop = 6.f;     // the reference's distance under the maximum that sets it (log2)

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

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    if (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
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
    float2 *xchg = reinterpret_cast<float2 *>(sv + C::NV * C::TILE);  // [128]
    uint64_t *kfull = reinterpret_cast<uint64_t *>(xchg + 128);
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
    int64_t *scratch = reinterpret_cast<int64_t *>(drain + 1);  // [8]
    PagedSched *sched = reinterpret_cast<PagedSched *>(scratch + 8);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sched + 1);
    static_assert(128 * 8 + (2 * C::NK + 2 * C::NV + 10 + 8) * 8 + sizeof(PagedSched) + 8 <= C::MISC, "misc region");
    volatile int *abort_flag = &sched->abort;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 8 && lane == 0) {
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
            mbar_init(smem_u32(&p_ready[g]), 4);  // the group's four warps
            mbar_init(smem_u32(&o_done[g]), 1);
        }
        mbar_init(smem_u32(o_free), 8);
        mbar_init(smem_u32(drain), 1);
        fence_mbar_init();
        prefetch_tensormap(&qmap);
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)), "n"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    pdl_wait_and_release();
    tc_fence_before();
    paged_schedule(p.w, sched, scratch, kMinTiles);
    tc_fence_after();
    const uint32_t tbase = *tslot;
    if (warp < 8) paged_zero_rows(p.w, reinterpret_cast<uint4 *>(p.out), p.Hq * D / 8, p.status, 256);
    const bool work = sched->t_begin < sched->t_end;

    if (work) {
        const int TB = C::RB >> p.gshift;  // tokens of an item
        PagedWalk w;
        w.init(p.w, *sched);
        if ((warp == 8 || warp == 10) && !p.test_stall) {
            // --------------------------------------------------------------
            // Loaders: K (and Q) in warp 8, V in warp 10. A lane per page.
            // --------------------------------------------------------------
            const bool is_k = warp == 8;
            const int NS = is_k ? C::NK : C::NV;
            uint64_t *full = is_k ? kfull : vfull, *empty = is_k ? kempty : vempty;
            const CUtensorMap *map = is_k ? &kmap : &vmap;
            uint8_t *ring = is_k ? sk : sv;
            const uint64_t pol = l2_policy_evict_first();
            const int ppt = kPagedTile >> p.w.shift;
            int seg = 0, i = 0;
            bool ok = true;
            do {
                const int n = w.seg_len();
                const int rows = min(TB, w.s.m - w.rb * TB) * p.G;
                if (is_k) {
                    if (seg > 0) {
                        if (lane == 0) ok = mbar_wait(smem_u32(qempty), (uint32_t)(seg - 1) & 1u, p.timeout_ns, abort_flag);
                        ok = __shfl_sync(0xffffffffu, ok, 0);
                        if (!ok) break;
                    }
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
                        if (lane == 0) ok = mbar_wait(smem_u32(&empty[s]), ((uint32_t)(i / NS) & 1u) ^ 1u, p.timeout_ns, abort_flag);
                        ok = __shfl_sync(0xffffffffu, ok, 0);
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
            } while (w.next(w.seg_len(), p.w));
            if (!ok && lane == 0) {
                raise_flag(p.status, GQAQ_DEV_TIMEOUT);
                *abort_flag = 1;
                // let every copy already issued land before this CTA may retire
                for (int it = i > NS ? i - NS : 0; it < i; ++it)
                    mbar_wait(smem_u32(&full[it % NS]), (uint32_t)(it / NS) & 1u, p.timeout_ns, nullptr);
                if (is_k)
                    for (int it = seg > 1 ? seg - 1 : 0; it <= seg; ++it)  // Q of this segment, if it was asked for
                        mbar_wait(smem_u32(qfull), (uint32_t)it & 1u, p.timeout_ns / 8, nullptr);
            }
        } else if (warp == 9 && lane == 0) {
            // --------------------------------------------------------------
            // MMA issuer (one thread). Products alternate between the groups:
            // event e is tile e / 2 of group e % 2 (two row tiles), or tile e
            // for group e % 2 (one). S(e + 2) follows PV(e), which frees its
            // tensor memory: the core runs one thread's MMAs in order.
            // --------------------------------------------------------------
            constexpr uint32_t IDESC_S = umma_idesc(128, 128, 0, BF16);
            constexpr uint32_t IDESC_O = umma_idesc(128, D, 1, BF16);
            const uint64_t qdesc0 = umma_desc(smem_u32(sq), 16);
            const uint64_t kdesc0 = umma_desc(smem_u32(sk), 16);
            const uint64_t vdesc0 = umma_desc(smem_u32(sv), C::BLK);
            int kc = 0;             // K / V tiles before this segment
            int seg = 0;
            uint32_t pc = 0;        // parity of the next P of each group (bits 0, 1)
            bool ok = true;
            do {
                const int n = w.seg_len();
                const int rows = min(TB, w.s.m - w.rb * TB) * p.G;
                const bool dual = rows > 128;
                const int ne = dual ? 2 * n : n;
                ok = mbar_wait(smem_u32(qfull), (uint32_t)seg & 1u, p.timeout_ns, abort_flag);
                auto issue_s = [&](int e) {
                    const int x = e & 1, j = kc + (dual ? e >> 1 : e), s = j % C::NK;
                    if (!dual || x == 0) ok = ok && mbar_wait(smem_u32(&kfull[s]), (uint32_t)(j / C::NK) & 1u, p.timeout_ns, abort_flag);
                    if (!ok) return;
                    tc_fence_after();
                    const uint64_t qd = qdesc0 + (uint64_t)(dual && x ? C::TILE >> 4 : 0);
                    const uint64_t kd = kdesc0 + (uint64_t)((s * C::TILE) >> 4);
                    const uint32_t sd = tbase + C::S_COL + 128u * (uint32_t)x;
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const uint64_t o = (uint64_t)(((ks >> 2) * C::BLK + (ks & 3) * 32) >> 4);
                        umma_ss(sd, qd + o, kd + o, IDESC_S, ks > 0);
                    }
                    umma_commit(smem_u32(&s_ready[x]));
                    if (!dual || x == 1) umma_commit(smem_u32(&kempty[s]));
                    if (e == ne - 1) umma_commit(smem_u32(qempty));
                };
                issue_s(0);
                if (ne > 1) issue_s(1);
                for (int e = 0; e < ne && ok; ++e) {
                    const int x = e & 1, j = kc + (dual ? e >> 1 : e), s = j % C::NV;
                    ok = mbar_wait(smem_u32(&p_ready[x]), (pc >> x) & 1u, p.timeout_ns, abort_flag);
                    pc ^= 1u << x;
                    if (e == 0 && seg > 0)  // the last segment's O has been read
                        ok = ok && mbar_wait(smem_u32(o_free), (uint32_t)(seg - 1) & 1u, p.timeout_ns, abort_flag);
                    if (!dual || x == 0) ok = ok && mbar_wait(smem_u32(&vfull[s]), (uint32_t)(j / C::NV) & 1u, p.timeout_ns, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t vd = vdesc0 + (uint64_t)((s * C::TILE) >> 4);
                    const uint32_t od = tbase + C::O_COL + 128u * (uint32_t)x, pd = tbase + C::S_COL + 128u * (uint32_t)x;
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        umma_ts(od, pd + 8u * kk, vd + (uint64_t)((kk * 16 * 128) >> 4), IDESC_O, (e > 1 || kk > 0) ? 1 : 0);
                    if (!dual || x == 1) umma_commit(smem_u32(&vempty[s]));
                    if (e + 2 >= ne) umma_commit(smem_u32(&o_done[x]));
                    if (e + 2 < ne) issue_s(e + 2);
                }
                kc += n;
                ++seg;
            } while (ok && w.next(w.seg_len(), p.w));
            if (!ok) {
                raise_flag(p.status, GQAQ_DEV_TIMEOUT);
                *abort_flag = 1;
            }
            umma_commit(smem_u32(drain));  // every issued MMA completes before TMEM is released
            mbar_wait(smem_u32(drain), 0u, p.timeout_ns, nullptr);
        } else if (warp < 8) {
            // --------------------------------------------------------------
            // Softmax groups: thread = row
            // --------------------------------------------------------------
            const int g = warp >> 2, row = threadIdx.x & 127, tid = threadIdx.x;
            const uint32_t tlane = tbase + ((uint32_t)((warp & 3) * 32) << 16);
            const uint32_t scol = tlane + C::S_COL + 128u * (uint32_t)g;
            const uint32_t ocol = tlane + C::O_COL + 128u * (uint32_t)g;
            const bool neg = !(p.scale_log2 > 0.f);  // a positive scale folds into the exponent
            const float mul = neg ? 1.f : p.scale_log2;
            int sc = 0, oc = 0;  // S tiles and finished segments of this group
            int vc = 0;          // V tiles before this segment
            bool ok = true;
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                bool r = true;
                if (lane == 0) r = mbar_wait(smem_u32(bar), parity, p.timeout_ns, abort_flag);
                r = __shfl_sync(0xffffffffu, r, 0);
                if (!r && lane == 0) {
                    raise_flag(p.status, GQAQ_DEV_TIMEOUT);
                    *abort_flag = 1;
                }
                return r;
            };
            do {
                const int n = w.seg_len();
                const int rows = min(TB, w.s.m - w.rb * TB) * p.G;
                const bool dual = rows > 128;
                const int nx = dual ? n : (n + 1 - g) / 2;          // this group's tiles
                const int r0 = dual ? 128 * g : 0;                  // its first row
                const int rho = r0 + row;                           // this thread's
                const bool live = rho < rows, warp_live = r0 + (warp & 3) * 32 < rows;
                const int pos0 = w.s.start + w.rb * TB;             // the block's first position
                const int lim = pos0 + (rho >> p.gshift);           // this row's
                const int lim_lo = pos0 + ((r0 + (warp & 3) * 32) >> p.gshift);  // the warp's least
                float ref = -INFINITY, l = 0.f;
                for (int k = 0; k < nx; ++k) {
                    const int jj = dual ? k : 2 * k + g;  // tile within the segment
                    const int tok0 = (w.local + jj) * kPagedTile;
                    ok = ok && wait(&s_ready[g], (uint32_t)sc & 1u);
                    ++sc;
                    tc_fence_after();
                    if (ok && warp_live) {
                        const bool mask = tok0 + kPagedTile - 1 > lim_lo;  // warp-uniform
                        uint32_t pk[64];
                        // P of the tile against reference r; returns its sum
                        auto exps = [&](float r) {
                            const float nref = r == -INFINITY ? 0.f : -r;
                            float s4[4] = {0.f, 0.f, 0.f, 0.f};
                            uint32_t v[2][32];
                            tmem_ld32_async(scol, v[0]);
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                tmem_ld32_wait(v[c & 1]);
                                if (c < 3) tmem_ld32_async(scol + 32u * (c + 1), v[(c + 1) & 1]);
                                uint32_t (&x)[32] = v[c & 1];
                                if (neg) {
#pragma unroll
                                    for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * p.scale_log2);
                                }
                                if (mask) {
#pragma unroll
                                    for (int e = 0; e < 32; ++e)
                                        if (tok0 + 32 * c + e > lim) x[e] = __float_as_uint(-INFINITY);
                                }
#pragma unroll
                                for (int e = 0; e < 32; e += 2) {
                                    const float e0 = fast_exp2(fmaf(__uint_as_float(x[e]), mul, nref));
                                    const float e1 = fast_exp2(fmaf(__uint_as_float(x[e + 1]), mul, nref));
                                    s4[(e >> 1) & 3] += e0 + e1;
                                    pk[16 * c + (e >> 1)] = pack2<BF16>(e0, e1);
                                }
                            }
                            return (s4[0] + s4[1]) + (s4[2] + s4[3]);
                        };
                        float cs = 0.f;
                        bool redo = ref == -INFINITY && lim >= tok0;  // the row's first keys
                        const bool fresh = __all_sync(0xffffffffu, ref == -INFINITY);
                        if (!fresh) {
                            cs = exps(ref);
                            redo = redo || cs > kSumLimit;
                        }
                        if (fresh || __any_sync(0xffffffffu, redo)) {
                            float r4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                            for (int c = 0; c < 4; ++c) {
                                uint32_t x[32];
                                tmem_ld32(scol + 32u * c, x);
#pragma unroll
                                for (int e = 0; e < 32; ++e) {
                                    float y = __uint_as_float(x[e]);
                                    if (neg) y *= p.scale_log2;
                                    if (tok0 + 32 * c + e > lim) y = -INFINITY;
                                    r4[e & 3] = fmaxf(r4[e & 3], y);
                                }
                            }
                            const float top = fmaxf(fmaxf(r4[0], r4[1]), fmaxf(r4[2], r4[3])) * mul - kRefDrop;
                            float alpha = 1.f;
                            if (redo && top > ref) {
                                alpha = fast_exp2(ref - top);  // 0 from no reference
                                ref = top;
                                l *= alpha;
                            }
                            if (k > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                                // S of this tile is complete, hence every earlier PV of the group
#pragma unroll 1
                                for (int c = 0; c < D / 32; ++c) {
                                    uint32_t o[32];
                                    tmem_ld32(ocol + 32u * c, o);
#pragma unroll
                                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                                    tmem_st32(ocol + 32u * c, o);
                                }
                            }
                            cs = exps(ref);
                        }
                        l += cs;
                        tmem_st32(scol, *reinterpret_cast<uint32_t (*)[32]>(&pk[0]));
                        tmem_st32(scol + 32u, *reinterpret_cast<uint32_t (*)[32]>(&pk[32]));
                        tmem_wait_st();
                    }
                    // rows of the last page past the request may hold anything: zero
                    // them, so that 0 * NaN cannot reach O (pages past it read zeros)
                    if (ok && (g == 0 || !dual) && w.s.len < tok0 + kPagedTile && (w.s.len & (p.S - 1)) != 0) {
                        const int v = vc + jj, s = v % C::NV;
                        ok = wait(&vfull[s], (uint32_t)(v / C::NV) & 1u);
                        if (ok && tok0 + row >= w.s.len) {
#pragma unroll
                            for (int q = 0; q < 8 * C::KH; ++q)
                                *reinterpret_cast<uint4 *>(sv + s * C::TILE + (q >> 3) * C::BLK + row * 128 + (q & 7) * 16) =
                                    make_uint4(0u, 0u, 0u, 0u);
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&p_ready[g]));
                }
                vc += n;

                // ---- epilogue ----
                if (nx > 0) {
                    ok = ok && wait(&o_done[g], (uint32_t)oc & 1u);
                    ++oc;
                }
                tc_fence_after();
                const bool whole = w.whole();
                float w0 = 1.f, w1 = 0.f;  // weights of O0 and O1 (one row tile), or w0 of this group's O
                float M = ref, L = l;
                if (!dual) {
                    if (g == 1) xchg[row] = make_float2(ref, l);
                    tc_fence_before();
                    named_bar_sync(1, 256);
                    if (g == 0) {
                        const float2 o = xchg[row];
                        M = fmaxf(ref, o.x);
                        w0 = ref == -INFINITY ? 0.f : fast_exp2(ref - M);
                        w1 = o.x == -INFINITY ? 0.f : fast_exp2(o.x - M);
                        L = w0 * l + w1 * o.y;
                        if (whole) {
                            const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
                            w0 *= inv;
                            w1 *= inv;
                        }
                        xchg[row] = make_float2(w0, w1);
                    }
                    named_bar_sync(1, 256);
                    tc_fence_after();
                    if (g == 1) {
                        const float2 o = xchg[row];
                        w0 = o.x;
                        w1 = o.y;
                    }
                } else if (whole) {
                    w0 = L > 0.f || L != L ? 1.f / L : 0.f;
                }
                // this thread's share: its row's D channels (two row tiles), or half of them
                const int c0 = dual ? 0 : g * (D / 2), nc = dual ? D : D / 2;
                const uint32_t o0 = tlane + C::O_COL + (dual ? 128u * (uint32_t)g : 0u), o1 = tlane + C::O_COL + 128u;
                const bool second = !dual && n > 1;
                const int q_row = w.s.q0 + w.rb * TB + (rho >> p.gshift);
                uint16_t *dst = p.out + ((int64_t)q_row * p.Hq + w.kv * p.G + (rho & (p.G - 1))) * D;
                const int slot = w.first ? 0 : 1;
                float *part = p.part + ((int64_t)blockIdx.x * 2 + slot) * C::PART;
                if (warp_live) {
                    if (!whole && live && (dual || g == 0)) reinterpret_cast<float2 *>(part)[rho] = make_float2(M, L);
#pragma unroll 1
                    for (int c = c0; c < c0 + nc; c += 32) {
                        uint32_t a[32];
                        if (ok) {
                            tmem_ld32(o0 + (uint32_t)c, a);
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; ++e) a[e] = 0u;
                        }
#pragma unroll
                        for (int e = 0; e < 32; ++e) a[e] = w0 == 0.f ? 0u : __float_as_uint(__uint_as_float(a[e]) * w0);
                        if (second) {
                            uint32_t b[32];
                            if (ok) {
                                tmem_ld32(o1 + (uint32_t)c, b);
                            } else {
#pragma unroll
                                for (int e = 0; e < 32; ++e) b[e] = 0u;
                            }
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (w1 != 0.f) a[e] = __float_as_uint(fmaf(__uint_as_float(b[e]), w1, __uint_as_float(a[e])));
                        }
                        if (!live) continue;
                        if (whole) {
#pragma unroll
                            for (int e = 0; e < 32; e += 8) {
                                uint4 h;
                                h.x = pack2<BF16>(__uint_as_float(a[e]), __uint_as_float(a[e + 1]));
                                h.y = pack2<BF16>(__uint_as_float(a[e + 2]), __uint_as_float(a[e + 3]));
                                h.z = pack2<BF16>(__uint_as_float(a[e + 4]), __uint_as_float(a[e + 5]));
                                h.w = pack2<BF16>(__uint_as_float(a[e + 6]), __uint_as_float(a[e + 7]));
                                *reinterpret_cast<uint4 *>(dst + c + e) = h;
                            }
                        } else {
                            float4 *acc = reinterpret_cast<float4 *>(part + C::ML) + (int64_t)(c / 4) * C::RB + rho;
#pragma unroll
                            for (int e = 0; e < 32; e += 4)
                                acc[(e / 4) * C::RB] = make_float4(__uint_as_float(a[e]), __uint_as_float(a[e + 1]),
                                                                   __uint_as_float(a[e + 2]), __uint_as_float(a[e + 3]));
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(o_free));

                if (!whole) {
                    // ---- arrive at the split item; the last arrival merges it ----
                    const int64_t T = sched->T;
                    const int gp = sched->grid;
                    const int64_t c_lo = tile_owner(w.off, T, gp);
                    const int np = (int)(tile_owner(w.off + w.tiles - 1, T, gp) - c_lo) + 1;
                    named_bar_sync(1, 256);
                    if (tid == 0) {
                        // the barrier orders every thread's partial stores before this
                        // release; the last arrival acquires all of them
                        const unsigned old = atomic_add_acq_rel_gpu(&p.count[c_lo], 1u);
                        const int last = old + 1u == (unsigned)np;
                        if (last) p.count[c_lo] = 0u;
                        sched->last = last;
                    }
                    named_bar_sync(1, 256);
                    if (sched->last && live) {
                        // partials: slot 0 (a range's first segment), but the first CTA's,
                        // which is its last unless the item begins its range
                        const int slot_lo = tile_begin(c_lo, T, gp) == w.off ? 0 : 1;
                        const float *base = p.part + c_lo * 2 * C::PART;
                        auto part_of = [&](int i) { return base + (int64_t)(2 * i + (i == 0 ? slot_lo : 0)) * C::PART; };
                        float mx = -INFINITY, sum = 0.f;
                        for (int i = 0; i < np; ++i) mx = fmaxf(mx, __ldcg(part_of(i) + 2 * rho));
                        for (int i = 0; i < np; ++i) {
                            const float2 ml = __ldcg(reinterpret_cast<const float2 *>(part_of(i)) + rho);
                            if (ml.x != -INFINITY) sum += fast_exp2(ml.x - mx) * ml.y;
                        }
                        const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
#pragma unroll 1
                        for (int c = c0; c < c0 + nc; c += 32) {
                            float4 a[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) a[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
                            for (int i = 0; i < np; ++i) {
                                const float *pi = part_of(i);
                                const float m = __ldcg(pi + 2 * rho);
                                const float f = m == -INFINITY ? 0.f : fast_exp2(m - mx) * inv;
                                const float4 *acc = reinterpret_cast<const float4 *>(pi + C::ML) + (int64_t)(c / 4) * C::RB + rho;
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    const float4 x = __ldcg(acc + e * C::RB);
                                    a[e].x = fmaf(f, x.x, a[e].x);
                                    a[e].y = fmaf(f, x.y, a[e].y);
                                    a[e].z = fmaf(f, x.z, a[e].z);
                                    a[e].w = fmaf(f, x.w, a[e].w);
                                }
                            }
#pragma unroll
                            for (int e = 0; e < 8; e += 2) {
                                uint4 h;
                                h.x = pack2<BF16>(a[e].x, a[e].y);
                                h.y = pack2<BF16>(a[e].z, a[e].w);
                                h.z = pack2<BF16>(a[e + 1].x, a[e + 1].y);
                                h.w = pack2<BF16>(a[e + 1].z, a[e + 1].w);
                                *reinterpret_cast<uint4 *>(dst + c + 4 * e) = h;
                            }
                        }
                    }
                }
            } while (w.next(w.seg_len(), p.w));
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tbase), "n"(512));
}

template <int D, bool BF16>
int launch_t(const PagedAttnArgs &a, const LaunchCtx &ctx) {
    using C = PtcCfg<D>;
    static bool ready[64] = {};
    if (ctx.device < 0 || ctx.device >= 64) return GQAQ_ERR_UNSUPPORTED;
    if (!ready[ctx.device]) {
        if (cudaFuncSetAttribute(paged_tc_kernel<D, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
            return GQAQ_ERR_CUDA;
        ready[ctx.device] = true;
    }
    const gqaq_paged_dims &d = *a.dims;
    const int grid = paged_tc_grid(ctx);
    const uint64_t rows = (uint64_t)d.num_pages * d.num_kv_heads * d.page_size;
    PtcParams p;
    
    p.G = d.num_q_heads / d.num_kv_heads;
    p.gshift = p.G == 1 ? 0 : p.G == 2 ? 1 : p.G == 4 ? 2 : 3;
    fill_paged_work(a, 8 - p.gshift, p.w);  // 256 rows
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
    p.timeout_ns = ctx.timeout_ns;
    p.test_stall = ctx.test_stall;
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
