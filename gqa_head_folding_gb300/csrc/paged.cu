// paged.cu -- the paged cache around the attention: planning a step's pages
// and slots from request lengths, returning pages, and the pass between a
// layer's projection and its attention (per-head RMS norm, rotation, append).
#include <cuda_bf16.h>

#include <atomic>

#include "internal.h"

namespace gqaq {
namespace {

constexpr int kTabThreads = 1024;

// Every thread of the cluster comes here; .aligned wants a warp's threads together, which after loops of unlike length
// only __syncwarp promises.
__device__ __forceinline__ void cluster_sync_all() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Exclusive sum over the block's threads (in thread order) and the total.
// buf: 32 words of shared memory, free again on return.
__device__ __forceinline__ int64_t block_exclusive(int64_t v, int64_t *buf, int64_t &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    int64_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) buf[warp] = incl;
    __syncthreads();
    int64_t w = lane < nw ? buf[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    const int64_t base = warp > 0 ? __shfl_sync(0xffffffffu, w, warp - 1) : 0;
    __syncthreads();
    return base + incl - v;
}

// The b in [0, n) with cum[b] <= x < cum[b + 1] (cum ascending, cum[0] <= x < cum[n]).
__device__ __forceinline__ int owner_of(const int *cum, int n, int x) {
    int lo = 0, hi = n;  // cum[lo] <= x < cum[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cum[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

struct TablesParams {
    const int *cache_len, *new_len, *free_pages, *free_count;
    int *table, *kv_len, *cu_q, *positions, *slots, *free_count_out;
    int *status;
    int B, T, S, shift, num_pages, max_pages;
    int room;  // tokens of a request at most
};

// Every CTA repeats the two prefix sums over the requests (new
// rows, needed pages) from the same inputs, so that nothing but the final
// count has to be exchanged; the rows and the new table entries are then
// shared out over the grid's threads, each finding its request by a binary
// search of the sums in shared memory. A new page's index follows from the
// sums and the free list alone, so no thread waits for another's table entry.
// Latency bounds it: 4.9 us for 32 requests, 6.6 us for 256 requests and 37K rows (5.0
// and 9.1 with the count replaced in place, which keeps the grid to eight CTAs).
__global__ void __launch_bounds__(kTabThreads) paged_tables_kernel(const TablesParams p) {
    extern __shared__ int sm[];
    int *cu = sm;                // [B + 1] first row of each request, clamped to T
    int *np = cu + p.B + 1;      // [B + 1] new pages before each request
    int *base = np + p.B + 1;    // [B] tokens in the cache; -1: refused
    __shared__ int64_t buf[32];
    __shared__ int granted;      // new pages handed out
    const int tid = threadIdx.x, rank = (int)blockIdx.x;
    const int nthreads = (int)blockDim.x, nctas = (int)gridDim.x;
    if (tid == 0) granted = 0;
    pdl_wait_and_release();
    const int raw_count = *p.free_count;
    const int count = raw_count < 0 ? 0 : raw_count > p.num_pages ? p.num_pages : raw_count;
    int flags = count != raw_count ? GQAQ_DEV_BAD_LEN : 0;

    const int per = (p.B + nthreads - 1) / nthreads;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    int64_t rows = 0, all;
    for (int b = b0; b < b1; ++b) rows += max(p.new_len[b], 0);
    rows = block_exclusive(rows, buf, all);
    int64_t need = 0;
    for (int b = b0; b < b1; ++b) {
        const int64_t c = p.cache_len[b], n = max(p.new_len[b], 0);
        cu[b] = (int)min(rows, (int64_t)p.T);
        rows += n;
        bool ok = c >= 0 && p.new_len[b] >= 0 && c + n <= p.room;
        if (!ok) flags |= GQAQ_DEV_BAD_LEN;
        if (rows > p.T) {
            ok = false;
            flags |= GQAQ_DEV_BAD_POS;
        }
        base[b] = ok ? (int)c : -1;
        if (ok) need += ((c + n + p.S - 1) >> p.shift) - ((c + p.S - 1) >> p.shift);
    }
    if (tid == 0) cu[p.B] = (int)min(all, (int64_t)p.T);
    int64_t pages = block_exclusive(need, buf, all);
    int mine = 0;
    for (int b = b0; b < b1; ++b) {
        np[b] = (int)min(pages, (int64_t)count);
        if (base[b] < 0) continue;
        const int64_t c = base[b], n = max(p.new_len[b], 0);
        const int64_t want = ((c + n + p.S - 1) >> p.shift) - ((c + p.S - 1) >> p.shift);
        pages += want;
        if (want == 0) continue;  // needs nothing: runs, whatever the requests before it took
        if (pages > count) {      // and so is every later request that needs a page
            base[b] = -1;
            flags |= GQAQ_DEV_NO_PAGES;
        } else {
            mine = (int)pages;
        }
    }
    if (tid == 0) np[p.B] = (int)min(all, (int64_t)count);
    if (mine > 0) atomicMax(&granted, mine);
    __syncthreads();

    const int stride = nctas * nthreads, first = rank * nthreads + tid;
    for (int b = first; b < p.B; b += stride) {
        p.kv_len[b] = base[b] < 0 ? 0 : base[b] + p.new_len[b];
        p.cu_q[b + 1] = cu[b + 1];
        if (b == 0) p.cu_q[0] = 0;
    }
    for (int t = first; t < p.T; t += stride) {
        int pos = 0, slot = -1;
        if (t < cu[p.B]) {
            const int b = owner_of(cu, p.B, t);
            if (base[b] >= 0) {
                pos = base[b] + (t - cu[b]);
                const int pg = pos >> p.shift, held = (int)(((int64_t)base[b] + p.S - 1) >> p.shift);
                const int page = pg < held ? p.table[(int64_t)b * p.max_pages + pg]
                                           : p.free_pages[count - 1 - (np[b] + pg - held)];
                if (page >= 0 && page < p.num_pages) slot = page * p.S + (pos & (p.S - 1));
                else flags |= GQAQ_DEV_BAD_PAGE;
            }
        }
        p.positions[t] = pos;
        p.slots[t] = slot;
    }
    for (int j = first; j < granted; j += stride) {
        const int b = owner_of(np, p.B, j);
        const int page = p.free_pages[count - 1 - j];
        if (page < 0 || page >= p.num_pages) flags |= GQAQ_DEV_BAD_PAGE;
        const int held = (int)(((int64_t)base[b] + p.S - 1) >> p.shift);
        p.table[(int64_t)b * p.max_pages + held + (j - np[b])] = page;
    }
    if (flags) raise_flag(p.status, flags);
    // a count replaced in place: one cluster, whose CTAs have all read it (else a cluster is one CTA)
    cluster_sync_all();
    if (rank == 0 && tid == 0) *p.free_count_out = count - granted;
}

struct ReleaseParams {
    const int *kv_len, *keep_len, *table, *free_count;
    int *free_pages, *free_count_out;
    int *status;
    int B, S, shift, num_pages, max_pages;
};

// The same shape as the plan: every CTA sums the pages that
// leave, then each thread moves some of them (154K pages of 500 requests: 6.6
// us; 31 us in the one cluster of eight CTAs that a count in place takes).
__global__ void __launch_bounds__(kTabThreads) paged_release_kernel(const ReleaseParams p) {
    extern __shared__ int sm[];
    int *cum = sm;               // [B + 1] leaving pages before each request
    int *from = cum + p.B + 1;   // [B] first leaving page
    __shared__ int64_t buf[32];
    const int tid = threadIdx.x, rank = (int)blockIdx.x;
    const int nthreads = (int)blockDim.x, nctas = (int)gridDim.x;
    pdl_wait_and_release();
    const int raw_count = *p.free_count;
    const int count = raw_count < 0 ? 0 : raw_count > p.num_pages ? p.num_pages : raw_count;
    int flags = count != raw_count ? GQAQ_DEV_BAD_LEN : 0;
    const int per = (p.B + nthreads - 1) / nthreads;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    const int64_t room = (int64_t)p.max_pages * p.S;
    int64_t sum = 0, all;
    for (int b = b0; b < b1; ++b) {
        const int64_t len = p.kv_len[b], keep = p.keep_len[b];
        const bool ok = len >= 0 && len <= room && keep >= 0 && keep <= len;
        if (!ok) flags |= GQAQ_DEV_BAD_LEN;
        const int lo = ok ? (int)((keep + p.S - 1) >> p.shift) : 0, hi = ok ? (int)((len + p.S - 1) >> p.shift) : 0;
        from[b] = lo;
        cum[b] = hi - lo;
        sum += hi - lo;
    }
    int64_t at = block_exclusive(sum, buf, all);
    const int64_t space = p.num_pages - count;
    for (int b = b0; b < b1; ++b) {
        const int n = cum[b];
        cum[b] = (int)min(at, space);
        at += n;
    }
    const bool fits = all <= space;
    if (!fits) {
        flags |= GQAQ_DEV_BAD_LEN;
        all = space;
    }
    if (tid == 0) cum[p.B] = (int)all;
    __syncthreads();
    const int stride = nctas * nthreads;
    for (int j = rank * nthreads + tid; j < (int)all; j += stride) {
        const int b = owner_of(cum, p.B, j);
        int page = p.table[(int64_t)b * p.max_pages + from[b] + (j - cum[b])];
        if (fits && (page < 0 || page >= p.num_pages)) {  // its place stays, so that the others' follow from the sums alone
            page = -1;
            flags |= GQAQ_DEV_BAD_PAGE;
        }
        p.free_pages[count + j] = page;
    }
    if (flags) raise_flag(p.status, flags);
    cluster_sync_all();
    if (rank == 0 && tid == 0) *p.free_count_out = count + (int)all;
}

int log2_of(int s) {
    int k = 0;
    while ((1 << k) < s) ++k;
    return k;
}

// CTAs: one up to 2048 elements of work. A count replaced in place needs the
// cluster's barrier before it is written, hence at most eight CTAs; otherwise
// up to 64 (each repeats the sums, so more would add little).
int table_ctas(int64_t work, bool in_place) {
    int c = 1;
    while (c < (in_place ? 8 : 64) && (int64_t)c * 2 * kTabThreads < work) c *= 2;
    return c;
}

// The sums of the largest batch pass the 48 KB that a kernel has without asking (its static shared memory counts too).
// The limit belongs to the kernel and not to a call, so it is raised once per device, to what any batch takes.
template <typename P>
int launch_tables(void (*kern)(P), const P &p, int words, int most_words, int64_t work, bool in_place, std::atomic<uint64_t> &ready,
                  const LaunchCtx &ctx) {
    const size_t smem = (size_t)words * sizeof(int);
    const int rc = allow_smem(reinterpret_cast<const void *>(kern), most_words * (int)sizeof(int), ready, ctx);
    if (rc != GQAQ_OK) return rc;
    const int ctas = table_ctas(work, in_place);
    const cudaError_t e = launch_kernel(kern, dim3((unsigned)ctas), dim3(kTabThreads), smem, ctx, in_place ? ctas : 0, p);
    return e == cudaSuccess ? GQAQ_OK : GQAQ_ERR_CUDA;
}

// ---------------------------------------------------------------------------
// Norm, rotation and append
// ---------------------------------------------------------------------------
struct AppendPagedParams {
    const uint16_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    const int *positions, *slots;
    const uint16_t *q_weight, *k_weight;
    float eps;
    const float *cos_sin;
    uint16_t *q_out, *k_pages, *v_pages;
    int *status;
    int T, Hq, Hkv, S, shift, num_pages, rope, max_position;
    int stages, stage_bytes;  // the ring of tokens
    uint64_t timeout_ns;
};

// Eight channels as four register pairs of 32-bit floats.
template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4 &x, f32x2 (&y)[4]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (BF16) {
            y[i] = pair32(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        } else {
            const float2 f = half2_bits_to_float2(w[i]);
            y[i] = pair32(f.x, f.y);
        }
    }
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const f32x2 (&y)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpair32(y[i]);
        w[i] = pack2<BF16>(f.x, f.y);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Bytes of shared memory of a CTA's ring of tokens. Three CTAs per SM whose
// rings hold three tokens of 48 rows moved 8192 of them in 36 us (5.7 TB/s);
// rings of 64 and 110 KB took 44 and 50 us.
constexpr int kAppendRing = 40 * 1024;
constexpr int kAppendStages = 6;        // tokens in flight at most
constexpr int kAppendThreads = 256;     // consumer threads at most

// What the loader leaves beside a token's rows.
struct alignas(16) AppendToken {
    int slot;  // -1: padding, or refused
    int pad[3];
};

// Persistent CTAs over tokens; blockIdx.y takes a range of the token's rows
// (q heads, then k, then v) when they are too many for the ring. A loader warp
// brings whole tokens into a ring in shared memory with bulk copies, several
// ahead, so that the loads of every SM stay in flight while the consumers
// compute: with the next token's rows in registers instead the kernel kept 20
// KB per SM in flight and moved 4.1 TB/s.
// D/16 lanes share a head's row; a lane holds two blocks of eight channels:
// (8j, rope/2 + 8j), so that with the halves style both members of every pair
// sit in one lane, and two neighbouring blocks where nothing turns.
template <int D, bool BF16, bool INTER>
__global__ void __launch_bounds__(kAppendThreads + 32, 3) paged_append_kernel(const AppendPagedParams p) {
    constexpr int LPR = D / 16;                    // lanes per row
    extern __shared__ __align__(128) uint8_t sm_append[];
    __shared__ uint64_t full[kAppendStages], empty[kAppendStages];
    __shared__ AppendToken token[kAppendStages];
    __shared__ int abort_flag_s;
    volatile int *abort_flag = &abort_flag_s;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int consumers = (int)blockDim.x - 32, rpp = consumers / LPR;  // threads, rows per pass
    const int H = p.Hq + 2 * p.Hkv;
    const int h_lo = (int)((int64_t)H * blockIdx.y / gridDim.y), h_hi = (int)((int64_t)H * (blockIdx.y + 1) / gridDim.y);
    const int rows = h_hi - h_lo, R = p.rope;
    uint8_t *wq_s = sm_append, *wk_s = wq_s + 2 * D;   // norm weights
    uint8_t *ring = wk_s + 2 * D;                      // stages: rows, then cosines and sines
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), (uint32_t)consumers / 32);
        }
        abort_flag_s = 0;
        fence_mbar_init();
    }
    pdl_wait_and_release();
    if ((int)threadIdx.x < D / 8) {
        if (p.q_weight) reinterpret_cast<uint4 *>(wq_s)[threadIdx.x] = reinterpret_cast<const uint4 *>(p.q_weight)[threadIdx.x];
        if (p.k_weight) reinterpret_cast<uint4 *>(wk_s)[threadIdx.x] = reinterpret_cast<const uint4 *>(p.k_weight)[threadIdx.x];
    }
    __syncthreads();
    const int step = (int)gridDim.x, n_tok = (p.T - (int)blockIdx.x + step - 1) / step;

    if (warp == consumers / 32) {
        // ---- loader: 32 tokens' slots and positions at a time, a lane each ----
        // rows of q, k and v in this CTA's range: [lo, hi) of each tensor
        const int q_lo = min(h_lo, p.Hq), q_hi = min(h_hi, p.Hq);
        const int k_lo = min(max(h_lo - p.Hq, 0), p.Hkv), k_hi = min(max(h_hi - p.Hq, 0), p.Hkv);
        const int v_lo = max(h_lo - p.Hq - p.Hkv, 0), v_hi = max(h_hi - p.Hq - p.Hkv, 0);
        const uint32_t bytes = (uint32_t)(rows * D * 2 + 4 * R);
        int s = 0;
        uint32_t ph = 1;
        bool ok = true;
        int issued = 0;
        for (int i0 = 0; i0 < n_tok && ok; i0 += 32) {
            int my_slot = -1, my_pos = 0;
            if (i0 + lane < n_tok) {
                const int t = (int)blockIdx.x + (i0 + lane) * step;
                my_slot = p.slots[t];
                if (R > 0) my_pos = p.positions[t];
                int flags = 0;
                if (my_slot >= 0) {
                    if ((my_slot >> p.shift) >= p.num_pages) flags |= GQAQ_DEV_BAD_PAGE;
                    if (R > 0 && (my_pos < 0 || my_pos >= p.max_position)) flags |= GQAQ_DEV_BAD_POS;
                }
                if (flags) {
                    my_slot = -1;
                    if (blockIdx.y == 0) raise_flag(p.status, flags);
                }
            }
            for (int i = i0; i < min(i0 + 32, n_tok); ++i) {
                const int slot = __shfl_sync(0xffffffffu, my_slot, i - i0), pos = __shfl_sync(0xffffffffu, my_pos, i - i0);
                if (lane == 0) {
                    const int64_t t = (int64_t)blockIdx.x + (int64_t)i * step;
                    if (i >= p.stages) ok = mbar_wait(smem_u32(&empty[s]), ph, p.timeout_ns, abort_flag);
                    if (ok) {
                        token[s].slot = slot;
                        const uint32_t fb = smem_u32(&full[s]);
                        if (slot < 0) {
                            mbar_arrive(fb);
                        } else {
                            mbar_arrive_expect_tx(fb, bytes);
                            uint32_t dst = smem_u32(ring) + (uint32_t)s * (uint32_t)p.stage_bytes;
                            auto bulk = [&](const void *src, uint32_t n) {
                                if (n == 0) return;
                                bulk_load(dst, src, n, fb);
                                dst += n;
                            };
                            bulk(p.q + t * p.q_stride + q_lo * D, (uint32_t)(q_hi - q_lo) * D * 2);
                            bulk(p.k + t * p.k_stride + k_lo * D, (uint32_t)(k_hi - k_lo) * D * 2);
                            bulk(p.v + t * p.v_stride + v_lo * D, (uint32_t)(v_hi - v_lo) * D * 2);
                            bulk(p.cos_sin + (int64_t)pos * R, (uint32_t)(4 * R));
                        }
                        ++issued;
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                if (++s == p.stages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        if (lane == 0) {
            if (!ok) {
                raise_flag(p.status, GQAQ_DEV_TIMEOUT);
                *abort_flag = 1;
            }
            // every copy issued lands before this CTA may retire, also where a consumer has given up on it
            for (int i = issued > p.stages ? issued - p.stages : 0; i < issued; ++i)
                mbar_wait(smem_u32(&full[i % p.stages]), (uint32_t)(i / p.stages) & 1u, kLandNs, nullptr);
        }
        return;
    }

    // ---- consumers ----
    const int j = threadIdx.x % LPR, r0 = threadIdx.x / LPR;
    const bool turns = 16 * j < R;
    const int c0 = turns ? 8 * j : 16 * j, c1 = turns ? R / 2 + 8 * j : 16 * j + 8;
    // halves: pair i of both blocks is channel 8j + i; adjacent pairs: a block
    // of eight channels holds pairs c/2 .. c/2 + 3
    const int i0 = INTER ? c0 / 2 : 8 * j, i1 = INTER ? c1 / 2 : 8 * j + 4;
    int s = 0;
    uint32_t ph = 0;
    for (int i = 0; i < n_tok; ++i) {
        if (!mbar_wait(smem_u32(&full[s]), ph, p.timeout_ns, abort_flag)) {
            if (lane == 0) {
                raise_flag(p.status, GQAQ_DEV_TIMEOUT);
                *abort_flag = 1;
            }
            return;
        }
        const int slot = token[s].slot;
        if (slot >= 0) {
            const int64_t t = (int64_t)blockIdx.x + (int64_t)i * step;
            const uint8_t *stage = ring + s * p.stage_bytes;
            f32x2 cs[4], sn[4];
            if (turns) {
                const float *row = reinterpret_cast<const float *>(stage + rows * D * 2);
                const float4 a = *reinterpret_cast<const float4 *>(row + i0), b = *reinterpret_cast<const float4 *>(row + i1);
                const float4 c = *reinterpret_cast<const float4 *>(row + R / 2 + i0), d = *reinterpret_cast<const float4 *>(row + R / 2 + i1);
                cs[0] = pair32(a.x, a.y); cs[1] = pair32(a.z, a.w); cs[2] = pair32(b.x, b.y); cs[3] = pair32(b.z, b.w);
                sn[0] = pair32(c.x, c.y); sn[1] = pair32(c.z, c.w); sn[2] = pair32(d.x, d.y); sn[3] = pair32(d.z, d.w);
            }
            const int page = slot >> p.shift, row_in = slot & (p.S - 1);
            // whole passes, so that the shuffles see all lanes of a row's group
            for (int rb = 0; rb < rows; rb += rpp) {
                const int rl = rb + r0;
                const bool live = rl < rows;
                const int h = h_lo + rl;
                const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.Hkv;
                uint4 x0 = make_uint4(0u, 0u, 0u, 0u), x1 = x0;
                if (live) {
                    x0 = *reinterpret_cast<const uint4 *>(stage + (rl * D + c0) * 2);
                    x1 = *reinterpret_cast<const uint4 *>(stage + (rl * D + c1) * 2);
                }
                f32x2 a[4], b[4];
                unpack8<BF16>(x0, a);
                unpack8<BF16>(x1, b);
                f32x2 sq = mul2(a[0], a[0]);
#pragma unroll
                for (int e = 1; e < 4; ++e) sq = fma2(a[e], a[e], sq);
#pragma unroll
                for (int e = 0; e < 4; ++e) sq = fma2(b[e], b[e], sq);
                float ss = unpair32(sq).x + unpair32(sq).y;
#pragma unroll
                for (int o = 1; o < LPR; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                if (!live) continue;
                const bool norm = !is_v && (is_q ? p.q_weight : p.k_weight) != nullptr;
                if (norm) {
                    const float inv = rsqrtf(ss * (1.f / D) + p.eps);
                    const f32x2 inv2 = pair32(inv, inv);
                    const uint8_t *w = is_q ? wq_s : wk_s;
                    f32x2 u[4], v[4];
                    unpack8<BF16>(*reinterpret_cast<const uint4 *>(w + c0 * 2), u);
                    unpack8<BF16>(*reinterpret_cast<const uint4 *>(w + c1 * 2), v);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        a[e] = mul2(mul2(a[e], inv2), u[e]);
                        b[e] = mul2(mul2(b[e], inv2), v[e]);
                    }
                }
                const bool turn = turns && !is_v;
                if (turn) {
                    if (INTER) {
                        // (x, y) -> (x cos - y sin, y cos + x sin), a pair of channels per register pair
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 xa = unpair32(a[e]), xb = unpair32(b[e]);
                            const float2 ca = unpair32(cs[e >> 1]), sa = unpair32(sn[e >> 1]);
                            const float2 cb = unpair32(cs[2 + (e >> 1)]), sb = unpair32(sn[2 + (e >> 1)]);
                            const float c = (e & 1) ? ca.y : ca.x, d = (e & 1) ? sa.y : sa.x;
                            const float f = (e & 1) ? cb.y : cb.x, g = (e & 1) ? sb.y : sb.x;
                            a[e] = fma2(pair32(-xa.y, xa.x), pair32(d, d), mul2(a[e], pair32(c, c)));
                            b[e] = fma2(pair32(-xb.y, xb.x), pair32(g, g), mul2(b[e], pair32(f, f)));
                        }
                    } else {
                        const f32x2 minus = pair32(-1.f, -1.f);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const f32x2 u = a[e], v = b[e];
                            a[e] = fma2(mul2(v, minus), sn[e], mul2(u, cs[e]));
                            b[e] = fma2(u, sn[e], mul2(v, cs[e]));
                        }
                    }
                }
                if (norm || turn) {  // else the bits as they are
                    x0 = pack8<BF16>(a);
                    x1 = pack8<BF16>(b);
                }
                const int hk = is_v ? h - p.Hq - p.Hkv : h - p.Hq;
                uint16_t *dst = is_q ? p.q_out + (t * p.Hq + h) * D
                                     : (is_v ? p.v_pages : p.k_pages) + (((int64_t)page * p.Hkv + hk) * p.S + row_in) * D;
                *reinterpret_cast<uint4 *>(dst + c0) = x0;
                *reinterpret_cast<uint4 *>(dst + c1) = x1;
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&empty[s]));
        if (++s == p.stages) {
            s = 0;
            ph ^= 1u;
        }
    }
}

template <int D, bool BF16>
int launch_append_t(AppendPagedParams &p, bool inter, const LaunchCtx &ctx) {
    auto kern = inter ? paged_append_kernel<D, BF16, true> : paged_append_kernel<D, BF16, false>;
    // A token's rows are split over gy CTAs until two of them fit the ring.
    const int H = p.Hq + 2 * p.Hkv, angles = 4 * p.rope;
    int gy = 1;
    auto stage = [&](int n) { return (H + n - 1) / n * D * 2 + angles; };
    while (2 * stage(gy) > kAppendRing) ++gy;
    p.stage_bytes = stage(gy);
    p.stages = kAppendRing / p.stage_bytes < kAppendStages ? kAppendRing / p.stage_bytes : kAppendStages;
    const size_t smem = 4 * D + (size_t)p.stages * p.stage_bytes;
    static std::atomic<uint64_t> ready[2] = {};
    const int rc = allow_smem(reinterpret_cast<const void *>(kern), 4 * D + kAppendRing, ready[inter], ctx);
    if (rc != GQAQ_OK) return rc;
    // consumers: the rows in as few passes as 256 threads allow, all full
    const int rows = (H + gy - 1) / gy, lanes = D / 16, passes = (rows * lanes + kAppendThreads - 1) / kAppendThreads;
    const int threads = ((rows + passes - 1) / passes * lanes + 31) / 32 * 32 + 32;
    // CTAs per SM, asked for once per shape (the driver's answer costs more than the launch)
    static std::atomic<uint64_t> known[2][64] = {};
    const uint64_t shape = ((uint64_t)smem << 32) | ((uint64_t)threads << 8);
    uint64_t got = known[inter][ctx.device].load(std::memory_order_relaxed);
    if ((got & ~0xffull) != shape) {
        int n = 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, smem) != cudaSuccess || n < 1) return GQAQ_ERR_CUDA;
        got = shape | (uint64_t)n;
        known[inter][ctx.device].store(got, std::memory_order_relaxed);
    }
    const int per_sm = (int)(got & 0xffu);
    int gx = per_sm * ctx.num_sms / gy;
    gx = gx < 1 ? 1 : gx < p.T ? gx : p.T;
    const cudaError_t e = launch_kernel(kern, dim3((unsigned)gx, (unsigned)gy), dim3((unsigned)threads), smem, ctx, 0, p);
    return e == cudaSuccess ? GQAQ_OK : GQAQ_ERR_CUDA;
}

}  // namespace

int launch_paged_tables(const PagedTablesArgs &a, const LaunchCtx &ctx) {
    const gqaq_paged_dims &d = *a.dims;
    TablesParams p;
    p.cache_len = a.cache_len;
    p.new_len = a.new_len;
    p.free_pages = a.free_pages;
    p.free_count = a.free_count;
    p.table = a.block_table;
    p.kv_len = a.kv_len;
    p.cu_q = a.cu_q;
    p.positions = a.positions;
    p.slots = a.slots;
    p.free_count_out = a.free_count_out;
    p.status = ctx.status;
    p.B = d.batch;
    p.T = d.max_tokens;
    p.S = d.page_size;
    p.shift = log2_of(d.page_size);
    p.num_pages = d.num_pages;
    p.max_pages = d.max_pages;
    const int held = d.max_pages * d.page_size;
    p.room = d.max_len > 0 && d.max_len < held ? d.max_len : held;
    static std::atomic<uint64_t> ready{0};
    return launch_tables(paged_tables_kernel, p, 3 * d.batch + 2, 3 * kPagedMaxBatch + 2, (int64_t)d.max_tokens + d.batch,
                         a.free_count == a.free_count_out, ready, ctx);
}

int launch_paged_release(const PagedReleaseArgs &a, const LaunchCtx &ctx) {
    const gqaq_paged_dims &d = *a.dims;
    ReleaseParams p;
    p.kv_len = a.kv_len;
    p.keep_len = a.keep_len;
    p.table = a.block_table;
    p.free_count = a.free_count;
    p.free_pages = a.free_pages;
    p.free_count_out = a.free_count_out;
    p.status = ctx.status;
    p.B = d.batch;
    p.S = d.page_size;
    p.shift = log2_of(d.page_size);
    p.num_pages = d.num_pages;
    p.max_pages = d.max_pages;
    const int64_t table = (int64_t)d.batch * d.max_pages;  // at most this many pages leave, and at most the pool
    static std::atomic<uint64_t> ready{0};
    return launch_tables(paged_release_kernel, p, 2 * d.batch + 1, 2 * kPagedMaxBatch + 1, table < d.num_pages ? table : d.num_pages,
                         a.free_count == a.free_count_out, ready, ctx);
}

int launch_paged_append(const PagedAppendArgs &a, const LaunchCtx &ctx) {
    const gqaq_paged_dims &d = *a.dims;
    AppendPagedParams p;
    p.q = static_cast<const uint16_t *>(a.q);
    p.k = static_cast<const uint16_t *>(a.k);
    p.v = static_cast<const uint16_t *>(a.v);
    p.q_stride = a.q_stride;
    p.k_stride = a.k_stride;
    p.v_stride = a.v_stride;
    p.positions = a.positions;
    p.slots = a.slots;
    p.q_weight = static_cast<const uint16_t *>(a.q_weight);
    p.k_weight = static_cast<const uint16_t *>(a.k_weight);
    p.eps = a.eps;
    p.cos_sin = a.cos_sin;
    p.q_out = static_cast<uint16_t *>(a.q_out);
    p.k_pages = static_cast<uint16_t *>(a.k_pages);
    p.v_pages = static_cast<uint16_t *>(a.v_pages);
    p.status = ctx.status;
    p.T = d.max_tokens;
    p.Hq = d.num_q_heads;
    p.Hkv = d.num_kv_heads;
    p.S = d.page_size;
    p.shift = log2_of(d.page_size);
    p.num_pages = d.num_pages;
    p.rope = a.rope_dim;
    p.max_position = a.max_position;
    p.timeout_ns = ctx.timeout_ns;
    const bool inter = a.interleaved != 0;
    if (d.dtype == GQAQ_BF16)
        return d.head_dim == 128 ? launch_append_t<128, true>(p, inter, ctx) : launch_append_t<64, true>(p, inter, ctx);
    return d.head_dim == 128 ? launch_append_t<128, false>(p, inter, ctx) : launch_append_t<64, false>(p, inter, ctx);
}

}  // namespace gqaq
