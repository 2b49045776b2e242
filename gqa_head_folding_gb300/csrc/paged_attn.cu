// paged_attn.cu -- paged attention for single tokens and short drafts (at most
// eight rows per KV head), and the choice between it and the tensor-memory
// kernel.
//
// A request's q_len tokens and the G query heads of a KV head form at most
// eight rows, which are the N = 8 side of mma.sync m16n8k16; the tokens of the
// cache are the M side, so a K or V row is read from HBM once for all of them
// and no row of the tensor core's tile is padding of a 128-row block:
//   S^T [16 tokens x 8] = K Q^T,   O^T [D x 8] += V^T P^T
// with an online softmax in the log2 domain on the S^T fragments: the row
// maxima are gathered across lanes, and the sums and outputs rescaled, only
// when a tile holds a score 2^8 above the reference (P <= 2^8 keeps fp16
// exact enough). Sums and outputs are fp32; each P is rounded once.
//
// Kernel shape (persistent CTAs, one launch): the tiles of 128 tokens of all
// (request, KV head) items are split evenly (paged_sched.cuh); warp 8 gathers
// a tile from its pages with TMA, one box per page and operand, into a ring of
// three stages; warps 0-7 own 16 tokens of each tile. At the end of an item's
// segment the eight warps' states merge in shared memory; an item cut by a
// range boundary leaves an fp32 partial and the CTA that arrives last merges
// them.
//
// What bounds it: HBM (batch 8 at up to 64K, 8 KV heads of 128 channels: 224 us,
// 6.6 TB/s, 97% of the copy rate); with little data the chain of schedule (2
// us), first tile (1.3), tiles, state merge (0.6), arrival (1.1) and merge of
// the parts (one request at 4K, 8 KV heads of 64 channels: 10.3 us).
#include <math.h>

#include <atomic>

#include "attn_mma.cuh"
#include "paged_sched.cuh"

namespace gqaq {
namespace {

constexpr int kRows = 8;          // rows of an item: q_len * G at most
constexpr int kItemTiles = 1;     // what an item costs beside its tiles, in tiles
constexpr int kMinUnits = 2;      // tiles per CTA below which a small step uses fewer CTAs (8 KV heads of 64 channels over 4K tokens: two 10.4 us, four 11.7)

template <int D>
struct PdCfg {
    static constexpr int THREADS = 288;
    static constexpr int KBYTES = 128 * D * 2;
    static constexpr int STAGE = 2 * KBYTES;
    static constexpr int NSTAGE = 3;
    static constexpr int MROWS = 4;                       // rows merged at a time
    static constexpr int MERGE = 8 * MROWS * (D + 2) * 4;
    static constexpr int MISC = 512;
    static constexpr int SMEM = 1024 + NSTAGE * STAGE + MERGE + MISC;
    static constexpr int MIN_BLOCKS = D == 64 ? 2 : 1;
    static constexpr int PART = kRows * (D + 2);          // floats of a partial: (m, l, acc) per row
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
    __device__ __forceinline__ void begin(const PdParams &p, const PagedWalk &w) {
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
    // (m, l, acc) of rows first .. first + 3 to this warp's slot of the merge buffer.
    __device__ __forceinline__ void store(float *slot, int first) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float ls = l[i];
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, x);
            const int n = 2 * c + i - first;
            if (n < 0 || n >= PdCfg<D>::MROWS) continue;
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

// An item this CTA arrived at last, to be merged at the end of its range.
struct PdSplit {
    int64_t off, out;  // tile offset of the item; first element of its output
    int tiles, rows, last;
};

template <int D, bool BF16>
__global__ void __launch_bounds__(PdCfg<D>::THREADS, PdCfg<D>::MIN_BLOCKS)
    paged_decode_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                        const __grid_constant__ PdParams p) {
    using C = PdCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *stages = smem;
    float *merge = reinterpret_cast<float *>(stages + C::NSTAGE * C::STAGE);
    uint64_t *full = reinterpret_cast<uint64_t *>(reinterpret_cast<uint8_t *>(merge) + C::MERGE);
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
    pdl_wait_and_release();
    paged_schedule(p.w, sched, scratch, kMinUnits, 0);
    if (warp < 8) paged_zero_rows(p.w, reinterpret_cast<uint4 *>(p.out), p.Hq * D / 8, p.status, 256);
    if (sched->t_begin >= sched->t_end) return;
    PagedWalk w;
    if (!w.init(p.w, *sched)) return;

    if (warp == 8) {
        // ---- loader: a lane per page ----
        if (p.test_stall) return;
        const uint64_t pol = l2_policy_evict_first();
        const int ppt = kPagedTile >> p.w.shift;
        const uint32_t box = (uint32_t)(p.S * D * 2);
        int i = 0;
        bool ok = true;
        do {
            const int n = w.seg_len();
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
    PagedWarp<D, BF16> wa;
    wa.lane = lane;
    wa.r = lane >> 2;
    wa.c = lane & 3;
    int i = 0, nsplit = 0;
    do {
        const int n = w.seg_len();
        const bool whole = w.whole();
        const int rows = w.s.m << p.gshift;
        wa.begin(p, w);
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
                wa.tile(kb, kb + C::KBYTES, 16 * warp, tok0, rem < 16 ? rem : 16, tok0 + 15 > w.s.start, p.scale_log2);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&empty[s]));
        }

        // ---- merge the eight warps' states, four rows at a time ----
        const int64_t out0 = ((int64_t)w.s.q0 * p.Hq + (w.kv << p.gshift)) * D;
        float *part = p.part + ((int64_t)blockIdx.x * 2 + w.slot()) * C::PART;
        for (int first = 0; first < rows; first += C::MROWS) {
            wa.store(merge + warp * C::MROWS * (D + 2), first);
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

template <int D, bool BF16>
int decode_grid(const LaunchCtx &ctx) {
    using C = PdCfg<D>;
    // CTAs per SM, asked for once per device
    static std::atomic<int> occ[64] = {};
    if (ctx.device < 0 || ctx.device >= 64) return -1;
    int per_sm = occ[ctx.device].load(std::memory_order_acquire);
    if (per_sm == 0) {
        auto kern = paged_decode_kernel<D, BF16>;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, C::THREADS, C::SMEM) != cudaSuccess || per_sm < 1)
            return -1;
        if (per_sm > C::MIN_BLOCKS) per_sm = C::MIN_BLOCKS;
        occ[ctx.device].store(per_sm, std::memory_order_release);
    }
    const int grid = per_sm * ctx.num_sms;
    return ctx.max_ctas > 0 && ctx.max_ctas < grid ? ctx.max_ctas : grid;
}

template <int D, bool BF16>
int launch_decode(const PagedAttnArgs &a, const LaunchCtx &ctx) {
    using C = PdCfg<D>;
    const gqaq_paged_dims &d = *a.dims;
    const int grid = decode_grid<D, BF16>(ctx);
    if (grid < 1) return GQAQ_ERR_CUDA;
    const uint64_t rows = (uint64_t)d.num_pages * d.num_kv_heads * d.page_size;
    CUtensorMap kmap, vmap;
    if (!encode_tensor_map_kpage(&kmap, a.k_pages, rows, D, d.page_size)) return GQAQ_ERR_CUDA;
    if (!encode_tensor_map_kpage(&vmap, a.v_pages, rows, D, d.page_size)) return GQAQ_ERR_CUDA;
    const int G = d.num_q_heads / d.num_kv_heads;
    PdParams p;
    fill_paged_work(a, 23, 1 << 23, kItemTiles, p.w);  // one block: every token of a request
    p.q = static_cast<const uint16_t *>(a.q);
    p.out = static_cast<uint16_t *>(a.out);
    p.count = reinterpret_cast<unsigned *>(a.workspace);
    p.part = reinterpret_cast<float *>(static_cast<uint8_t *>(a.workspace) + kPagedCountBytes);
    p.status = ctx.status;
    p.gshift = G == 1 ? 0 : G == 2 ? 1 : G == 4 ? 2 : 3;
    p.Hq = d.num_q_heads;
    p.S = d.page_size;
    p.zero_row = (int)rows;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.timeout_ns = ctx.timeout_ns;
    p.test_stall = ctx.test_stall;
    const cudaError_t e = launch_kernel(paged_decode_kernel<D, BF16>, dim3((unsigned)grid), dim3(C::THREADS), C::SMEM, ctx, 0,
                                        kmap, vmap, p);
    return e == cudaSuccess ? GQAQ_OK : GQAQ_ERR_CUDA;
}

size_t decode_workspace_bytes(const gqaq_paged_dims *d, const LaunchCtx &ctx) {
    const size_t part = d->head_dim == 128 ? PdCfg<128>::MIN_BLOCKS * PdCfg<128>::PART : PdCfg<64>::MIN_BLOCKS * PdCfg<64>::PART;
    return kPagedCountBytes + (size_t)ctx.num_sms * 2 * part * sizeof(float);
}

}  // namespace

size_t paged_attn_workspace_bytes(const gqaq_paged_dims *d, const LaunchCtx &ctx) {
    const size_t a = paged_tc_workspace_bytes(d, ctx), b = decode_workspace_bytes(d, ctx);
    return a > b ? a : b;
}

int launch_paged_attn(const PagedAttnArgs &a, const LaunchCtx &ctx) {
    if (a.workspace_bytes < paged_attn_workspace_bytes(a.dims, ctx)) return GQAQ_ERR_WORKSPACE;
    // Up to eight rows per KV head: the decode kernel (32 query and 8 KV heads of 64 channels: one request at 4K 10.4 us
    // against 18.4, 32 requests of 1K to 4K 31.4 against 43.8); above, the tensor-memory kernel (16 requests of up to 9K with 3
    // to 6 drafted tokens, 12 to 24 rows: 44 to 65 us, where two and three N blocks of mma.sync took 52 to 196).
    if ((int64_t)a.max_q_len * (a.dims->num_q_heads / a.dims->num_kv_heads) > kRows) return launch_paged_tc(a, ctx);
    if (a.dims->dtype == GQAQ_BF16) return a.dims->head_dim == 128 ? launch_decode<128, true>(a, ctx) : launch_decode<64, true>(a, ctx);
    return a.dims->head_dim == 128 ? launch_decode<128, false>(a, ctx) : launch_decode<64, false>(a, ctx);
}

}  // namespace gqaq
