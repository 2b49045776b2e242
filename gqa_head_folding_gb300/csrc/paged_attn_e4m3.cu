// paged_attn_e4m3.cu -- paged attention over 8-bit pages on the 5th-generation
// tensor cores, for chunks of new tokens and for batches that mix chunks with
// single tokens.
//
// Mathematics (paged_e4m3.cuh has the pages' format): with the codes' values
// code_k and code_v, their pages' exponents ke and ve, and one row q,
//   s = scale log2(e) 2^ke (q . code_k) + ve,   w = 2^(s - ref)
//   O += w code_v,   l += w 2^-ve,   out = O / l
// Neither exponent meets a number of 16 bits: the codes become fp16 exactly as
// they are, and w is rounded once to fp16, or taken in two bfloat16 numbers, and
// the codes in bfloat16, where a segment's pages of V lie more than kHeadroom
// exponents apart. The walker looks through their exponents while the segment's
// first tiles are on their way. P of 16 tokens is then eight columns of the first
// numbers and eight of the second, in place of the 16 scores: the 1024-token chunk
// below takes 944 us for 441 where every segment has such pages. Each role's loop in
// two copies costs 3 us there; a flag per tile, read in one loop, took 502 to 532.
// The products of scores are fp16 whatever the dtype: a bfloat16 row of q is taken
// times a power of two that brings its largest channel into [2^14, 2^15) (channels
// down to 2^-31 of it keep all their bits, smaller ones are off by at most 2^-39 of
// it), since both operands of a product have one type and a code costs a
// conversion more to bfloat16. The reference moves as in paged_attn_tc.cu.
//
// Kernel shape: that of paged_attn_tc.cu (items of 256 rows, two softmax groups
// with S and O in tensor memory, the notifier, the same end of an item), with
// the cache brought as codes and widened on the way:
//  - warp 16 loads Q and, a lane per page, the tiles of codes of K and V in turn
//    into a ring of raw tiles, and leaves the pages' factors beside them.
//  - warps 20-23 turn a raw tile into the fp16 tile, 128-byte swizzled, that the
//    products read (E4M3 has no wider partner in one tcgen05.mma), and clear the
//    rows of a last page's V that lie past its request.
//  - warp 18 walks the CTA's range and hands its segments to the other warps
//    through a ring: each of them walking for itself would take registers that
//    the softmax warps have no room to give (they hold 96, the others 48).
//
// What bounds it. A 1024-token chunk of a 32K context (32 heads of 128 channels):
// 441 us, 1,230 TFLOP/s, 63% of a large library product's rate; the tensor pipe is busy 52% of
// the cycles and the exponentials 26%, and the rest is the chain S, softmax, PV of
// the two row tiles. Sixteen requests of up to 9K tokens with seven drafted tokens
// (28 live rows of 128; 8 KV heads of 128 channels): 69 us for 25 us of bytes.
// There a tile takes 2,400 cycles: 660 to widen each 16 KB of K and V, 190 for
// the fence between these writes and the product that reads them, 1,040 to issue the
// products, and waits between them. Loads and widening ran one tile after the
// other until two loads of codes were kept in flight (78 -> 70 us). Four row tiles
// of a quarter of the rows, and S of the next tile before PV of this one, were no faster.
#include "paged_e4m3.cuh"
#include "paged_tc.cuh"

namespace gqaq {
namespace {

template <int D>
struct P8Cfg : PtcShape<D> {
    static constexpr int THREADS = 768;                // 16 softmax warps; loader, MMA, walker, notifier; 4 that widen
    static constexpr int RAW = 128 * D;                // a tile of codes
    static constexpr int NR = D == 128 ? 2 : 6;        // raw ring (K and V in turn)
    static constexpr int NR1 = D == 128 ? 4 : 6;       // where no item has two row tiles: the second one's place serves too
    static constexpr int NK = D == 128 ? 2 : 4;        // K ring
    static constexpr int NV = D == 128 ? 2 : 4;        // V ring
    // Factors of tile t lie in slot t % NF. They are written when K of tile t is asked for, which waits until a raw
    // tile NR1 before it is free, so that V of tile t - NR1 / 2 - 1 has been widened, for which PV of tile
    // t - NR1 / 2 - 1 - NV, and with it that tile's softmax, had ended.
    static constexpr int NF = NR1 / 2 + 1 + NV;
    static constexpr int NSEG = 3;
    static constexpr int SEG = 8 * ((int)(sizeof(PagedWalk) + 7) / 8 + 1);
    static constexpr int BARS = 2 * NK + 2 * NV + 2 * NR1 + NF + 3 * NSEG + 11;
    // bytes from the start of shared memory: two Q tiles, the raw ring, the K and V rings, the exchange of 256 numbers, the
    // factors, the barriers, and what the schedule and the walker leave
    static constexpr int AT_R = 2 * PtcShape<D>::TILE, AT_K = AT_R + NR * RAW, AT_V = AT_K + NK * PtcShape<D>::TILE;
    static constexpr int AT_X = AT_V + NV * PtcShape<D>::TILE, AT_F = AT_X + 1024, AT_BAR = AT_F + NF * 256;
    static constexpr int AT_SCRATCH = AT_BAR + BARS * 8, AT_SCHED = AT_SCRATCH + 12 * 8;
    static constexpr int AT_SEG = AT_SCHED + (int)sizeof(PagedSched), AT_SLOT = AT_SEG + NSEG * SEG, AT_MORE = AT_SLOT + 4;
    static constexpr int SMEM = AT_MORE + 4;
    // the barriers
    static constexpr int KFULL = AT_BAR, KEMPTY = KFULL + 8 * NK, VFULL = KEMPTY + 8 * NK, VEMPTY = VFULL + 8 * NV;
    static constexpr int RFULL = VEMPTY + 8 * NV, REMPTY = RFULL + 8 * NR1, FFULL = REMPTY + 8 * NR1, SEG_FULL = FFULL + 8 * NF;
    static constexpr int SEG_EMPTY = SEG_FULL + 8 * NSEG, FAR_FULL = SEG_EMPTY + 8 * NSEG, QFULL = FAR_FULL + 8 * NSEG, QEMPTY = QFULL + 8;
    static constexpr int QREADY = QEMPTY + 8;    // Q has been turned into fp16 (bfloat16 only)
    static constexpr int S_READY = QREADY + 8, P_READY = S_READY + 16;
    static constexpr int O_DONE = P_READY + 16;  // a group's last PV of a segment
    static constexpr int O_FREE = O_DONE + 16;   // the epilogue has read O
    static constexpr int DRAIN = O_FREE + 8;
    static_assert((NR1 - NR) * RAW <= PtcShape<D>::TILE, "the second row tile's place");
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

static_assert(kRefDrop >= kHeadroom, "the largest weight of a row");

struct P8Params : PtcParams {
    const int8_t *k_exp, *v_exp;
    int one_tile;  // no item has more than 128 rows
    unsigned *begun;  // not null: another launch of this call runs beside this one
};

template <int D>
struct P8Segment {
    PagedWalk w;
    int more;  // 0: the range is done
    int far;   // known later (FAR_FULL): its weights are bfloat16 numbers
};

// 128 rows of D codes, brought by TMA (D = 128: 128-byte swizzled, D = 64: as
// they are), to 64-channel blocks of fp16 rows, 128-byte swizzled; 128 threads,
// 16 codes each at a time. rows: those from here on become zeros. Which lanes
// share a quarter of a warp's access is chosen so that neither the loads nor the
// stores meet in a bank: with D = 128 rows r and r ^ 5 (their chunks of 16 codes
// lie in unlike halves of a raw line, their chunks of 8 channels at unlike
// places of an fp16 line), with D = 64 neighbouring rows.
template <int D>
__device__ __forceinline__ void widen_tile(uint32_t raw, uint32_t dst, int warp, int lane, int rows) {
    constexpr int BLK = PtcShape<D>::BLK;
    constexpr int N = D / 16;  // steps of 8 rows by 64 channels for each warp
    const int c = lane & 3, r8 = D == 128 ? (lane >> 3) ^ (lane & 4 ? 5 : 0) : lane >> 2;
    const int row0 = warp * 32 + r8;
    const uint32_t from = D == 128 ? raw + (uint32_t)(row0 * 128 + ((c ^ r8) << 4)) : raw + (uint32_t)(row0 * 64 + c * 16);
    const uint32_t to = dst + (uint32_t)(row0 * 128 + (((2 * c) ^ r8) << 4));
    auto st = [](uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
    };
#pragma unroll
    for (int k0 = 0; k0 < N; k0 += 2) {
        uint4 x[2];  // two steps' loads together
#pragma unroll
        for (int k = k0; k < k0 + 2; ++k) {
            const int kh = D == 128 ? k & 1 : 0, g = D == 128 ? k >> 1 : k;
            x[k - k0] = lds128((from ^ (uint32_t)(kh * 64)) + (uint32_t)(g * 8 * D));
        }
#pragma unroll
        for (int k = k0; k < k0 + 2; ++k) {
            const int kh = D == 128 ? k & 1 : 0, g = D == 128 ? k >> 1 : k;
            uint32_t y[8];
            e4m3x4_to_f16x2x2(x[k - k0].x, y[0], y[1]);
            e4m3x4_to_f16x2x2(x[k - k0].y, y[2], y[3]);
            e4m3x4_to_f16x2x2(x[k - k0].z, y[4], y[5]);
            e4m3x4_to_f16x2x2(x[k - k0].w, y[6], y[7]);
            st(to + (uint32_t)(kh * BLK + g * 1024), y[0], y[1], y[2], y[3]);
            st((to ^ 16u) + (uint32_t)(kh * BLK + g * 1024), y[4], y[5], y[6], y[7]);
        }
    }
    if (__builtin_expect(rows < row0 - r8 + 32, 0)) {
#pragma unroll 1
        for (int k = 0; k < N; ++k) {
            const int kh = D == 128 ? k & 1 : 0, g = D == 128 ? k >> 1 : k;
            if (row0 + 8 * g < rows) continue;
            st(to + (uint32_t)(kh * BLK + g * 1024), 0u, 0u, 0u, 0u);
            st((to ^ 16u) + (uint32_t)(kh * BLK + g * 1024), 0u, 0u, 0u, 0u);
        }
    }
}

// What this thread has just widened (its zeros too), fp16 to bfloat16 in place.
template <int D>
__device__ __forceinline__ void rewiden_tile(uint32_t dst, int warp, int lane) {
    const int c = lane & 3, r8 = D == 128 ? (lane >> 3) ^ (lane & 4 ? 5 : 0) : lane >> 2;
    const uint32_t to = dst + (uint32_t)((warp * 32 + r8) * 128 + (((2 * c) ^ r8) << 4));
#pragma unroll 1
    for (int k = 0; k < 2 * (D / 16); ++k) {
        const int step = k >> 1, kh = D == 128 ? step & 1 : 0, g = D == 128 ? step >> 1 : step;
        const uint32_t at = (to ^ (uint32_t)((k & 1) << 4)) + (uint32_t)(kh * PtcShape<D>::BLK + g * 1024);
        const uint4 x = lds128(at);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(f16x2_to_bf16x2(x.x)), "r"(f16x2_to_bf16x2(x.y)),
                     "r"(f16x2_to_bf16x2(x.z)), "r"(f16x2_to_bf16x2(x.w))
                     : "memory");
    }
}

// The product of 32 tokens' weights in two bfloat16 numbers: of each 16 tokens A has eight columns of the first and eight of the
// second; B as warp_mma_ts4.
__device__ __forceinline__ void warp_mma_far(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred q, p, t;\n\t.reg .b32 a1, a2, a3;\n\t.reg .b64 b1;\n\t"
        "elect.sync _|q, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "add.s32 a1, %1, 8;\n\tadd.s32 a2, %1, 16;\n\tadd.s32 a3, %1, 24;\n\tadd.s64 b1, %2, 128;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], %2, %3, t;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b1, %3, t;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b1, %3, t;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Whether a segment's weights have to be bfloat16 numbers: it has pages of V more than kHeadroom exponents apart. For a
// warp: 256 pages at a time, whose exponents are on their way while the next ones' table entries are (8 K tokens in pages of 16
// take about 1.5 us, beside the segment's first loads).
__device__ __forceinline__ bool segment_far(const P8Params &p, const PagedWalk &w, int lane) {
    const int log = kPagedTileLog - p.w.shift, held = (int)(((int64_t)w.s.len + (1 << p.w.shift) - 1) >> p.w.shift);
    const int *table = p.w.table + (int64_t)w.b * p.w.max_pages;
    const int last = min((w.local + w.seg_len()) << log, held);
    int lo = kMostPageExp, hi = kLeastPageExp, page[8];
    auto entries = [&](int e0) {
#pragma unroll
        for (int u = 0; u < 8; ++u) page[u] = e0 + 32 * u < last ? table[e0 + 32 * u] : -1;
    };
    entries((w.local << log) + lane);
    for (int e0 = (w.local << log) + lane; e0 - lane < last; e0 += 256) {
        int e[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) e[u] = (uint32_t)page[u] < (uint32_t)p.w.num_pages ? p.v_exp[page[u] * p.w.Hkv + w.kv] : 0;  // a bad page: zeros
        entries(e0 + 256);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int x = min(max(e[u], kLeastPageExp), kMostPageExp);
            lo = e0 + 32 * u < last ? min(lo, x) : lo;
            hi = e0 + 32 * u < last ? max(hi, x) : hi;
        }
    }
    return __reduce_max_sync(0xffffffffu, hi) - __reduce_min_sync(0xffffffffu, lo) > (int)kHeadroom;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(P8Cfg<D>::THREADS, 1)
    paged_tc8_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const __grid_constant__ P8Params p) {
    using C = P8Cfg<D>;
    extern __shared__ __align__(1024) uint8_t smem8[];
    int64_t *scratch = reinterpret_cast<int64_t *>(smem8 + C::AT_SCRATCH);  // [12]
    PagedSched *sched = reinterpret_cast<PagedSched *>(smem8 + C::AT_SCHED);
    static_assert(sizeof(P8Segment<D>) <= C::SEG && C::DRAIN + 8 == C::AT_SCRATCH, "segment ring, barriers");
    volatile int *abort_flag = &sched->abort;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 16 && lane == 0) {
        const uint32_t at = smem_u32(smem8);
        auto init = [&](int first, int n, uint32_t count) {
            for (int x = 0; x < n; ++x) mbar_init(at + (uint32_t)(first + 8 * x), count);
        };
        init(C::KFULL, C::NK, 4);  // the widening warps
        init(C::KEMPTY, C::NK, 1);
        init(C::VFULL, C::NV, 4);
        init(C::VEMPTY, C::NV, 1);
        init(C::RFULL, C::NR1, 1);
        init(C::REMPTY, C::NR1, 4);
        init(C::FFULL, C::NF, 1);
        init(C::SEG_FULL, C::NSEG, 1);
        init(C::FAR_FULL, C::NSEG, 1);
        init(C::SEG_EMPTY, C::NSEG, 8);  // loader, MMA, notifier, four widening warps, softmax
        init(C::QFULL, 3, 1);            // and QEMPTY, QREADY
        init(C::S_READY, 2, 1);
        init(C::P_READY, 2, 8);          // the group's warps
        init(C::O_DONE, 2, 1);
        init(C::O_FREE, 1, 16);
        init(C::DRAIN, 1, 1);
        fence_mbar_init();
        prefetch_tensormap(&qmap);
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
    }
    if (warp == 17) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem8 + C::AT_SLOT)), "n"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    pdl_wait();
    if (threadIdx.x == 0) {  // the launch beside this one may begin when every CTA has waited, and reads what they waited for
        if (p.begun != nullptr && blockIdx.x == 0) store_release_gpu(p.begun, 1u);
        pdl_release();
    }
    tc_fence_before();
    paged_schedule(p.w, sched, scratch, kMinUnits, D / 64);
    tc_fence_after();
    const uint32_t tbase = *reinterpret_cast<uint32_t *>(smem8 + C::AT_SLOT);
    if (warp < 16) paged_zero_rows(p.w, reinterpret_cast<uint4 *>(p.out), p.Hq * D / 8, p.status, 512);

    if (sched->t_begin < sched->t_end) {
        const int TB = C::RB >> p.gshift;  // tokens of an item
        const uint32_t at = smem_u32(smem8);
        // A warp that fails goes on walking, without work, so that every ring moves on.
        auto fail = [&] {
            raise_flag(p.status, GQAQ_DEV_TIMEOUT);
            *abort_flag = 1;
        };
        const uint64_t seg_ns = 2 * p.timeout_ns + kLandNs;  // above what a failing warp needs to move on
        auto segment = [&](int i) -> P8Segment<D> & { return *reinterpret_cast<P8Segment<D> *>(smem8 + C::AT_SEG + (i % C::NSEG) * C::SEG); };
        auto seg_wait = [&](int i) {  // a thread; false: the range is done
            return mbar_wait(at + C::SEG_FULL + 8 * (i % C::NSEG), (uint32_t)(i / C::NSEG) & 1u, seg_ns, nullptr) && segment(i).more != 0;
        };
        auto seg_next = [&](int i) { return __all_sync(0xffffffffu, seg_wait(i)) != 0; };  // a warp
        auto seg_far = [&](int i) {  // a thread
            return mbar_wait(at + C::FAR_FULL + 8 * (i % C::NSEG), (uint32_t)(i / C::NSEG) & 1u, seg_ns, nullptr) && segment(i).far != 0;
        };
        auto seg_done = [&](int i) { mbar_arrive(at + C::SEG_EMPTY + 8 * (i % C::NSEG)); };

        if (warp >= 16) {
            // the launch's 80 registers for each of 768 threads: 96 for the softmax warps, 48 for these
            asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
            if (warp == 18) {
                // ---- walker ----
                PagedWalk w;
                bool more = w.init(p.w, *sched);
                for (int i = 0;; ++i) {
                    bool ok = true;
                    if (i >= C::NSEG) ok = lane != 0 || mbar_wait(at + C::SEG_EMPTY + 8 * (i % C::NSEG), ((uint32_t)(i / C::NSEG) & 1u) ^ 1u, seg_ns, nullptr);
                    if (!__all_sync(0xffffffffu, ok)) {
                        if (lane == 0) fail();
                        break;
                    }
                    P8Segment<D> &s = segment(i);
                    if (lane == 0) {
                        s.w = w;
                        s.more = more;
                        mbar_arrive(at + C::SEG_FULL + 8 * (i % C::NSEG));
                    }
                    if (!more) break;
                    const bool far = segment_far(p, w, lane);
                    if (lane == 0) {
                        s.far = far;
                        mbar_arrive(at + C::FAR_FULL + 8 * (i % C::NSEG));
                    }
                    more = w.advance(p.w);
                }
                __syncwarp();
            } else if (warp == 16) {
                // ---- loader: a lane per page ----
                const uint64_t pol = l2_policy_evict_first();
                const int ppt = kPagedTile >> p.w.shift, per = 32 / ppt;  // pages of a tile, tiles of a batch of entries
                const uint32_t box = (uint32_t)D << p.w.shift;
                const int nr = p.one_tile ? C::NR1 : C::NR, at_r = C::AT_R - (p.one_tile ? (C::NR1 - C::NR) * C::RAW : 0);
                bool ok = !p.test_stall;
                int n_q = 0;               // Q tiles asked for
                int i = 0, rs = 0, fs = 0;  // raw tiles asked for; slots
                uint32_t rp = 1;
                for (int sg = 0; seg_next(sg); ++sg) {
                    if (ok) {
                        const PagedWalk &w = segment(sg).w;
                        const int n = w.seg_len(), rows = min(TB, w.s.m - w.rb * TB) * p.G;
                        if (sg > 0) ok = warp_mbar_wait_slow(at + C::QEMPTY, (uint32_t)(sg - 1) & 1u, p.timeout_ns, abort_flag);
                        if (ok) {
                            ++n_q;
                            if (lane == 0) {
                                const int nq = rows > 128 ? 2 : 1;
                                mbar_arrive_expect_tx(at + C::QFULL, (uint32_t)(nq * C::TILE));
                                for (int x = 0; x < nq; ++x)
                                    for (int kh = 0; kh < C::KH; ++kh)
                                        tma_load_3d(at + x * C::TILE + kh * C::BLK, &qmap, 64 * kh, w.kv * p.G,
                                                    w.s.q0 + w.rb * TB + x * (TB / 2), at + C::QFULL, pol);
                            }
                            PageFeed<P8Params> feed;
                            feed.start(p, w, lane);
                            for (int t = 0, x = 0; t < n && ok; ++t, ++x) {
                                if (x == per) {
                                    feed.step(p);
                                    x = 0;
                                }
                                const int from = x * ppt + lane;
                                const int row = __shfl_sync(0xffffffffu, feed.row, from);
                                // factors of the tile's groups of eight tokens, whatever the page size (a table by pages cost registers for its offsets)
                                const int group = x * ppt + ((lane & 15) << 3 >> p.w.shift);
                                const int ke = __shfl_sync(0xffffffffu, feed.ke, group), ve = __shfl_sync(0xffffffffu, feed.ve, group);
#pragma unroll 1
                                for (int kv = 0; kv < 2; ++kv) {
                                    if (i >= nr) ok = warp_mbar_wait_slow(at + C::REMPTY + 8 * rs, rp, p.timeout_ns, abort_flag);
                                    if (!ok) break;
                                    const uint32_t fb = at + C::RFULL + 8 * rs;
                                    if (lane == 0) mbar_arrive_expect_tx(fb, (uint32_t)C::RAW);
                                    __syncwarp();
                                    if (lane < ppt)
                                        tma_load_2d(at + at_r + (uint32_t)(rs * C::RAW) + (uint32_t)lane * box, kv ? &vmap : &kmap, 0, row, fb, pol);
                                    if (kv == 0) {
                                        if (lane < 16) reinterpret_cast<float4 *>(smem8 + C::AT_F)[fs * 16 + lane] = page_factors(ke, ve);
                                        __syncwarp();
                                        if (lane == 0) mbar_arrive(at + C::FFULL + 8 * fs);
                                        if (++fs == C::NF) fs = 0;
                                    }
                                    ++i;
                                    if (++rs == nr) {
                                        rs = 0;
                                        rp ^= 1u;
                                    }
                                }
                            }
                        }
                        if (!ok && lane == 0) fail();
                    }
                    __syncwarp();
                    if (lane == 0) seg_done(sg);
                }
                if (lane == 0) {
                    // every copy issued lands before this CTA may retire, also where another warp has given up on it
                    for (int it = i > nr ? i - nr : 0; it < i; ++it)
                        mbar_wait(at + C::RFULL + 8 * (it % nr), (uint32_t)(it / nr) & 1u, kLandNs, nullptr);
                    if (n_q > 0) mbar_wait(at + C::QFULL, (uint32_t)(n_q - 1) & 1u, kLandNs, nullptr);
                }
                __syncwarp();
            } else if (warp == 17) {
                // ---- MMA issuer: as in paged_attn_tc.cu, over the widened tiles ----
                constexpr uint32_t IDESC_S = umma_idesc(128, 128, 0);
                constexpr uint32_t IDESC_O = umma_idesc(128, D, 1), IDESC_FAR = umma_idesc(128, D, 1, 1);
                const uint64_t qdesc0 = umma_desc(at, 16);
                const uint64_t kdesc0 = umma_desc(at + C::AT_K, 16);
                const uint64_t vdesc0 = umma_desc(at + C::AT_V, C::BLK);
                int ks = 0, vs = 0;             // ring slots and their phases
                uint32_t kp = 0, vp = 0;
                uint32_t pp = 0;                // phases of p_ready (bits 0, 1)
                uint32_t sp = 0;                // phase of the segment's barriers
                bool ok = true;
                auto wait = [&](uint32_t bar, uint32_t parity) {
                    return warp_mbar_wait(bar, parity, p.timeout_ns, abort_flag);
                };
                auto products = [&](auto dual_c, int sg, int ne) {
                    constexpr bool DUAL = decltype(dual_c)::value;
                    auto issue_s = [&](int e) {
                        const int x = e & 1;
                        if (!DUAL || x == 0) ok = wait(at + C::KFULL + 8 * ks, kp);
                        if (!ok) return;
                        tc_fence_after();
                        const uint64_t qd = qdesc0 + (uint64_t)(DUAL && x ? C::TILE >> 4 : 0);
                        const uint64_t kd = kdesc0 + (uint64_t)(ks * (C::TILE >> 4));
                        const uint32_t sd = tbase + C::S_COL + 128u * (uint32_t)x;
#pragma unroll
                        for (int kh = 0; kh < C::KH; ++kh)
                            warp_mma_ss4(sd, qd + (uint64_t)(kh * (C::BLK >> 4)), kd + (uint64_t)(kh * (C::BLK >> 4)), IDESC_S, kh > 0);
                        warp_commit(at + C::S_READY + 8 * x);
                        if (!DUAL || x == 1) {
                            warp_commit(at + C::KEMPTY + 8 * ks);
                            if (++ks == C::NK) {
                                ks = 0;
                                kp ^= 1u;
                            }
                        }
                        if (e == ne - 1) warp_commit(at + C::QEMPTY);
                    };
                    issue_s(0);
                    if (ok && ne > 1) issue_s(1);
                    auto pv = [&](auto far_c) {
#pragma unroll 1
                        for (int e = 0; e < ne && ok; ++e) {
                            const int x = e & 1;
                            if (!DUAL || x == 0) ok = wait(at + C::VFULL + 8 * vs, vp);
                            if (e == 0 && sg > 0) ok = ok && wait(at + C::O_FREE, sp ^ 1u);  // the last segment's O has been read
                            ok = ok && wait(at + C::P_READY + 8 * x, (pp >> x) & 1u);
                            if (!ok) break;
                            pp ^= 1u << x;
                            tc_fence_after();
                            const uint64_t vd = vdesc0 + (uint64_t)(vs * (C::TILE >> 4));
                            const uint32_t od = tbase + C::O_COL + 128u * (uint32_t)x, pd = tbase + C::S_COL + 128u * (uint32_t)x;
                            if constexpr (decltype(far_c)::value) {
#pragma unroll
                                for (uint32_t c = 0; c < 4; ++c)  // of tokens 32 c ..: columns 32 c ..
                                    warp_mma_far(od, pd + 32u * c, vd + 256u * c, IDESC_FAR, e > 1 || c > 0);
                            } else {
                                warp_mma_ts4(od, pd, vd, IDESC_O, e > 1);              // P of tokens 0-63: columns 0-31
                                warp_mma_ts4(od, pd + 64u, vd + 512u, IDESC_O, 1);     // of tokens 64-127: columns 64-95
                            }
                            if (!DUAL || x == 1) {
                                warp_commit(at + C::VEMPTY + 8 * vs);
                                if (++vs == C::NV) {
                                    vs = 0;
                                    vp ^= 1u;
                                }
                            }
                            if (e + 2 >= ne) warp_commit(at + C::O_DONE + 8 * x);
                            if (e + 2 < ne) issue_s(e + 2);
                        }
                    };
                    if (__any_sync(0xffffffffu, seg_far(sg))) pv(std::true_type());
                    else pv(std::false_type());
                };
                for (int sg = 0; seg_next(sg); ++sg) {
                    if (ok) {
                        const PagedWalk &w = segment(sg).w;
                        const int n = w.seg_len(), rows = min(TB, w.s.m - w.rb * TB) * p.G;
                        ok = wait(at + (BF16 ? C::QREADY : C::QFULL), sp);
                        if (ok) {
                            if (rows > 128) products(std::true_type(), sg, 2 * n);
                            else products(std::false_type(), sg, n);
                        }
                        if (!ok && lane == 0) fail();
                    }
                    sp ^= 1u;
                    __syncwarp();
                    if (lane == 0) seg_done(sg);
                }
                __syncwarp();
                warp_commit(at + C::DRAIN);  // every issued MMA completes before TMEM is released
                mbar_wait(at + C::DRAIN, 0u, kLandNs, nullptr);
                __syncwarp();
            } else if (warp == 19) {
                // ---- notifier: watches the S barriers (and that the factors are there) for the softmax warps ----
                uint32_t sph = 0, fp = 0;
                int fs = 0;
                bool ok = true;
                auto watch = [&](uint32_t bar, uint32_t parity) {
                    if (!ok) return;
                    ok = warp_mbar_wait(bar, parity, p.timeout_ns, abort_flag);
                    if (!ok && lane == 0) fail();
                };
                for (int sg = 0; seg_next(sg); ++sg) {
                    const PagedWalk &w = segment(sg).w;
                    const int n = w.seg_len();
                    const bool dual = min(TB, w.s.m - w.rb * TB) * p.G > 128;
                    const int ne = dual ? 2 * n : n;
                    for (int e = 0; e < ne; ++e) {
                        const int x = e & 1;
                        if (!dual || x == 0) {
                            watch(at + C::FFULL + 8 * fs, fp);
                            if (++fs == C::NF) {
                                fs = 0;
                                fp ^= 1u;
                            }
                        }
                        watch(at + C::S_READY + 8 * x, (sph >> x) & 1u);
                        sph ^= 1u << x;
                        tc_fence_after();
                        tc_fence_before();
                        named_bar_sync(10 + x, 288);  // also after a timeout: the groups pass once per tile
                    }
                    __syncwarp();
                    if (lane == 0) seg_done(sg);
                }
            } else {
                // ---- widening ----
                const int nr = p.one_tile ? C::NR1 : C::NR, at_r = C::AT_R - (p.one_tile ? (C::NR1 - C::NR) * C::RAW : 0);
                int rs = 0, ks = 0, vs = 0;
                uint32_t rp = 0, kp = 1, vp = 1;
                bool ok = true;
                auto wait = [&](uint32_t bar, uint32_t parity) {
                    return warp_mbar_wait_slow(bar, parity, p.timeout_ns, abort_flag);
                };
                auto turn = [&](bool far, uint32_t ring, int N, int &slot, uint32_t &ph, uint32_t full, uint32_t empty, int rows) {
                    ok = wait(at + C::RFULL + 8 * rs, rp) && wait(empty + 8 * slot, ph);
                    if (!ok) return;
                    widen_tile<D>(at + at_r + (uint32_t)(rs * C::RAW), ring + (uint32_t)(slot * C::TILE), warp - 20, lane, rows);
                    if (__builtin_expect(far, 0)) rewiden_tile<D>(ring + (uint32_t)(slot * C::TILE), warp - 20, lane);
                    fence_async_shared();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(full + 8 * slot);
                        mbar_arrive(at + C::REMPTY + 8 * rs);
                    }
                    if (++rs == nr) {
                        rs = 0;
                        rp ^= 1u;
                    }
                    if (++slot == N) {
                        slot = 0;
                        ph ^= 1u;
                    }
                };
                for (int sg = 0; seg_next(sg); ++sg) {
                    const PagedWalk &w = segment(sg).w;
                    const int n = w.seg_len(), first = w.local * kPagedTile, len = w.s.len;
                    const bool far = __any_sync(0xffffffffu, seg_far(sg));
                    for (int t = 0; t < n && ok; ++t) {
                        turn(false, at + C::AT_K, C::NK, ks, kp, at + C::KFULL, at + C::KEMPTY, 128);
                        if (ok) turn(far, at + C::AT_V, C::NV, vs, vp, at + C::VFULL, at + C::VEMPTY, len - (first + t * kPagedTile));
                        if (!ok && lane == 0) fail();
                    }
                    __syncwarp();
                    if (lane == 0) seg_done(sg);
                }
            }
        } else {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 96;");
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
            uint32_t oph = 0, qph = 0;  // phases of o_done and qfull
            int fs0 = 0;               // slot of the segment's first tile's factors
            bool ok = true;
            float *xchg = reinterpret_cast<float *>(smem8 + C::AT_X);  // [256]
            volatile int *more_s = reinterpret_cast<volatile int *>(smem8 + C::AT_MORE);
            const float4 *factors = reinterpret_cast<const float4 *>(smem8 + C::AT_F);  // [NF][16]
            auto wait = [&](uint32_t bar, uint32_t parity) {
                const bool r = warp_mbar_wait(bar, parity, p.timeout_ns, abort_flag);
                if (!r && lane == 0) fail();
                return r;
            };
            for (int sg = 0;; ++sg) {
                if (tid == 0) *more_s = seg_wait(sg);
                named_bar_sync(1, 512);
                if (!*more_s) break;
                const PagedWalk &w = segment(sg).w;
                const int n = w.seg_len();
                const int rows = min(TB, w.s.m - w.rb * TB) * p.G;
                const bool dual = rows > 128;
                const int nx = dual ? n : (n + 1 - g) / 2;          // this group's tiles
                const int r0 = dual ? 128 * g : 0;                  // its first row
                const int rho = r0 + row;                           // this thread's
                const bool live = rho < rows, warp_live = r0 + (warp & 3) * 32 < rows;
                // Of a tile, from its number jj in the segment on: a thread's tokens, and what it may see of them. From shared
                // memory where masks need them, so that the loop over tiles keeps one number for the warp.
                auto token = [&](int jj) { return (w.local + jj) * kPagedTile + 64 * h; };
                auto limit = [&] { return w.s.start + w.rb * TB + (rho >> p.gshift); };  // the row's own position
                const int masked_from = ((w.s.start + w.rb * TB + ((r0 + (warp & 3) * 32) >> p.gshift) - 63 - 64 * h) >> kPagedTileLog) + 1 - w.local;
                float mul = p.scale_log2;                           // any sign, not zero
                if (BF16) {
                    // Q to fp16, in place: eight lanes per row, each the same chunk of every 64-channel block
                    ok = ok && wait(at + C::QFULL, qph);
                    qph ^= 1u;
                    if (ok) {
                        for (int r = warp * 4 + (lane >> 3); r < (dual ? 256 : 128); r += 64) {
                            const uint32_t chunk = at + (uint32_t)((r >> 7) * C::TILE + (r & 127) * 128 + (lane & 7) * 16);
                            uint4 x[C::KH];
                            uint32_t top = 0u;  // bits of the row's largest finite magnitude
#pragma unroll
                            for (int kh = 0; kh < C::KH; ++kh) {
                                x[kh] = lds128(chunk + (uint32_t)(kh * C::BLK));
                                const uint32_t y[4] = {x[kh].x, x[kh].y, x[kh].z, x[kh].w};
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const uint32_t lo = y[e] & 0x7fffu, hi = (y[e] >> 16) & 0x7fffu;
                                    top = max(top, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
                                }
                            }
#pragma unroll
                            for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                            const int e2 = max((int)(top >> 7) - 127 - 14, -100);
                            const float by = pow2i(-e2);
#pragma unroll
                            for (int kh = 0; kh < C::KH; ++kh) {
                                uint32_t y[4] = {x[kh].x, x[kh].y, x[kh].z, x[kh].w};
#pragma unroll
                                for (int e = 0; e < 4; ++e) y[e] = pack2<false>(__uint_as_float(y[e] << 16) * by, __uint_as_float(y[e] & 0xffff0000u) * by);
                                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(chunk + (uint32_t)(kh * C::BLK)), "r"(y[0]), "r"(y[1]),
                                             "r"(y[2]), "r"(y[3])
                                             : "memory");
                            }
                            if ((lane & 7) == 0) xchg[r] = pow2i(e2);
                        }
                    }
                    fence_async_shared();
                    named_bar_sync(1, 512);
                    if (tid == 0) mbar_arrive(at + C::QREADY);
                    mul *= ok ? xchg[rho] : 1.f;
                    named_bar_sync(1, 512);  // xchg is free again
                }
                // times 2^-48 still not 0, so that a masked score's product stays -inf; what is this small moves no score by 2^-20
                mul = copysignf(fmaxf(fabsf(mul), 0x1p-100f), mul);
                // a row behind the item's weighs nothing and never has its reference moved, so that no other depends on it
                float ref = live ? -INFINITY : INFINITY, l = 0.f;
                int fs = fs0 + (dual ? 0 : g);
                if (fs >= C::NF) fs -= C::NF;
                auto tiles = [&](auto far_c) {
                    for (int k = 0; k < nx; ++k) {
                        const int jj = dual ? k : 2 * k + g;  // tile within the segment
                        named_bar_sync(10 + g, 288);  // S is complete (after a timeout it holds anything)
                        tc_fence_after();
                        if (warp_live) {
                            const bool mask = jj >= masked_from;  // some row of the warp does not see all of these tokens
                            const float4 *fac = factors + fs * 16 + 8 * h;  // of tokens 8 i .. of this thread's
                            uint32_t pk[32];
                            // P of these tokens against reference r; their sum, and the sum of each over 2^ve
                            auto exps = [&](float r, float &share) {
                                const float nref = r == -INFINITY ? 0.f : -r;
                                float sum = 0.f;
                                share = 0.f;
#pragma unroll
                                for (int c = 0; c < 2; ++c) {
                                    uint32_t x[32];
                                    tmem_ld32_async(scol + 32u * c, x);
                                    tmem_ld32_wait(x);
                                    if (__builtin_expect(mask, 0)) {
                                        const int seen = limit() - token(jj) - 32 * c;  // the last of these that the row sees
                                        const uint32_t hide = p.scale_log2 > 0.f ? 0xff800000u : 0x7f800000u;  // its product is -inf
#pragma unroll
                                        for (int e = 0; e < 32; ++e)
                                            if (e > seen) x[e] = hide;
                                    }
#pragma unroll
                                    for (int i = 0; i < 4; ++i) {
                                        const float4 f = fac[4 * c + i];
                                        const float m = finite32(mul * f.x), b = f.y + nref;
                                        const uint64_t m2 = pair32(m, m), b2 = pair32(b, b);
                                        uint64_t s8 = 0;
#pragma unroll
                                        for (int e = 8 * i; e < 8 * i + 8; e += 2) {
                                            const float2 y = unpair32(fma2(pair32(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), m2, b2));
                                            const float e0 = fast_exp2(y.x), e1 = fast_exp2(y.y);
                                            s8 = e == 8 * i ? pair32(e0, e1) : add2(s8, pair32(e0, e1));
                                            pk[16 * c + (e >> 1)] = pack2<false>(e0, e1);
                                        }
                                        const float2 t = unpair32(s8);
                                        sum += t.x + t.y;
                                        share = fmaf(t.x + t.y, f.z, share);
                                    }
                                }
                                return sum;
                            };
                            float cs = 0.f, share = 0.f;
                            const bool fresh = __all_sync(0xffffffffu, fabsf(ref) == INFINITY);  // of both warps: they share ref
                            // one copy of the exponentials serves both passes: the second, after a
                            // row's reference has moved, is rare, and code that is jumped over costs fetches
#pragma unroll 1
                            for (int pass = fresh ? 0 : 1;; ++pass) {
                                if (pass > 0) cs = exps(ref, share);
                                if (pass > 1) break;
                                const bool redo = (ref == -INFINITY && limit() >= (w.local + jj) * kPagedTile) || cs > kSumLimit;  // the row's first keys, or far above
                                if (__builtin_expect(!pair_any(pair_bar, redo), 1)) {
                                    if (pass == 0) {
#pragma unroll
                                        for (int e = 0; e < 32; ++e) pk[e] = 0u;  // every row of the pair is masked in this tile
                                    }
                                    break;
                                }
                                // the row's maximum over both halves becomes the reference
                                float top = -INFINITY;
#pragma unroll 1
                                for (int c = 0; c < 2; ++c) {
                                    uint32_t x[32];
                                    tmem_ld32_async(scol + 32u * c, x);
                                    tmem_ld32_wait(x);
                                    const int seen = limit() - token(jj) - 32 * c;
#pragma unroll
                                    for (int i = 0; i < 4; ++i) {
                                        const float4 f = fac[4 * c + i];
                                        const float m = finite32(mul * f.x);
#pragma unroll
                                        for (int e = 8 * i; e < 8 * i + 8; ++e)
                                            top = fmaxf(top, e > seen ? -INFINITY : fmaf(__uint_as_float(x[e]), m, f.y));
                                    }
                                }
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
                                        tmem_ld32_async(ocol + (uint32_t)c, o);
                                        tmem_ld32_wait(o);
#pragma unroll
                                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                                        tmem_st32(ocol + (uint32_t)c, o);
                                    }
                                }
                                pass = 1;  // the next pass is the last
                            }
                            l += share;
                            if constexpr (decltype(far_c)::value) {
                                // each P in two bfloat16 numbers, over the scores: of 16 tokens the first in eight columns, the second in eight
                                const float nref = ref == -INFINITY ? 0.f : -ref;
#pragma unroll 1
                                for (int c = 0; c < 4; ++c) {
                                    uint32_t x[16], y[16];
                                    tmem_ld16(scol + 16u * c, x);
                                    const int seen = limit() - token(jj) - 16 * c;
#pragma unroll
                                    for (int e = 0; e < 16; e += 2) {
                                        const float4 f = fac[2 * c + e / 8];
                                        const float m = finite32(mul * f.x), b = f.y + nref;
                                        const float e0 = e > seen ? 0.f : fast_exp2(fmaf(__uint_as_float(x[e]), m, b));
                                        const float e1 = e + 1 > seen ? 0.f : fast_exp2(fmaf(__uint_as_float(x[e + 1]), m, b));
                                        y[e / 2] = pack2<true>(e0, e1);
                                        y[8 + e / 2] = pack2<true>(e0 - __uint_as_float(y[e / 2] << 16), e1 - __uint_as_float(y[e / 2] & 0xffff0000u));
                                    }
                                    tmem_st16(scol + 16u * c, y);
                                }
                            } else {
                                tmem_st32(scol, pk);  // over the first half of the scores it read
                            }
                            tmem_wait_st();
                        }
                        fs += dual ? 1 : 2;
                        if (fs >= C::NF) fs -= C::NF;
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(at + C::P_READY + 8 * g);
                    }
                };
                if (__any_sync(0xffffffffu, seg_far(sg))) tiles(std::true_type());
                else tiles(std::false_type());
                fs0 = (fs0 + n) % C::NF;
                ptc_finish<D, BF16>(p, w, sched, xchg, at + C::O_DONE, at + C::O_FREE, tlane, g, h, row, n, nx, dual, live, warp_live, rho, ref, l, oph, ok, wait);
                named_bar_sync(1, 512);  // the segment has been read
                if (tid == 0) seg_done(sg);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 17) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tbase), "n"(512));
}

template <int D, bool BF16>
int launch_t(const PagedAttnArgs &a, const LaunchCtx &ctx) {
    using C = P8Cfg<D>;
    static std::atomic<uint64_t> ready{0};
    const int rc = allow_smem(reinterpret_cast<const void *>(paged_tc8_kernel<D, BF16>), C::SMEM, ready, ctx);
    if (rc != GQAQ_OK) return rc;
    static std::atomic<int> regs{0};  // the softmax warps would wait for ever for registers that the launch did not bring
    if (regs.load(std::memory_order_acquire) == 0) {
        cudaFuncAttributes attr;
        if (cudaFuncGetAttributes(&attr, paged_tc8_kernel<D, BF16>) != cudaSuccess) return GQAQ_ERR_CUDA;
        regs.store(attr.numRegs, std::memory_order_release);
    }
    if (regs.load(std::memory_order_acquire) * C::THREADS < 96 * 512 + 48 * (C::THREADS - 512)) return GQAQ_ERR_CUDA;
    const gqaq_paged_dims &d = *a.dims;
    const uint64_t rows = (uint64_t)d.num_pages * d.num_kv_heads * d.page_size;
    P8Params p;
    fill_ptc(a, ctx, p);
    p.k_exp = a.k_exp;
    p.v_exp = a.v_exp;
    p.begun = a.share == 2 ? reinterpret_cast<unsigned *>(a.workspace) + kPagedBegunWord : nullptr;
    p.one_tile = (int64_t)a.max_q_len * p.G <= 128;
    CUtensorMap qmap, kmap, vmap;
    if (!encode_tensor_map_heads(&qmap, a.q, d.max_tokens, d.num_q_heads, D, p.G, 128 / p.G)) return GQAQ_ERR_CUDA;
    if (!encode_tensor_map_u8(&kmap, a.k_pages, rows, D, d.page_size, D == 128 ? 128 : 0)) return GQAQ_ERR_CUDA;
    if (!encode_tensor_map_u8(&vmap, a.v_pages, rows, D, d.page_size, D == 128 ? 128 : 0)) return GQAQ_ERR_CUDA;
    const cudaError_t e = launch_kernel(paged_tc8_kernel<D, BF16>, dim3((unsigned)paged_tc_grid(ctx)), dim3(C::THREADS), C::SMEM, ctx, 0,
                                        qmap, kmap, vmap, p);
    return e == cudaSuccess ? GQAQ_OK : GQAQ_ERR_CUDA;
}

}  // namespace

int launch_paged_tc_e4m3(const PagedAttnArgs &a, const LaunchCtx &ctx) {
    if (a.dims->dtype == GQAQ_BF16) return a.dims->head_dim == 128 ? launch_t<128, true>(a, ctx) : launch_t<64, true>(a, ctx);
    return a.dims->head_dim == 128 ? launch_t<128, false>(a, ctx) : launch_t<64, false>(a, ctx);
}

}  // namespace gqaq
