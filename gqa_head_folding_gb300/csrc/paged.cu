// paged.cu -- the paged cache around the attention: planning a step's pages
// and slots from request lengths, returning pages, and the pass between a
// layer's projection and its attention (per-head RMS norm, rotation, append).
#include <cuda_bf16.h>

#include "internal.h"

namespace gqaq {
namespace {

constexpr int kTabThreads = 1024;

__device__ __forceinline__ void cluster_sync_all() {
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
};

// Every CTA repeats the two prefix sums over the requests (new
// rows, needed pages) from the same inputs, so that nothing but the final
// count has to be exchanged; the rows and the new table entries are then
// shared out over the grid's threads, each finding its request by a binary
// search of the sums in shared memory. A new page's index follows from the
// sums and the free list alone, so no thread waits for another's table entry.
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
    const int64_t room = (int64_t)p.max_pages * p.S;
    int64_t rows = 0, all;
    for (int b = b0; b < b1; ++b) rows += max(p.new_len[b], 0);
    rows = block_exclusive(rows, buf, all);
    int64_t need = 0;
    for (int b = b0; b < b1; ++b) {
        const int64_t c = p.cache_len[b], n = max(p.new_len[b], 0);
        cu[b] = (int)min(rows, (int64_t)p.T);
        rows += n;
        bool ok = c >= 0 && p.new_len[b] >= 0 && c + n <= room;
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
// leave, then each thread moves some of them.
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
    if (all > space) {
        flags |= GQAQ_DEV_BAD_LEN;
        all = space;
    }
    if (tid == 0) cum[p.B] = (int)all;
    __syncthreads();
    const int stride = nctas * nthreads;
    for (int j = rank * nthreads + tid; j < (int)all; j += stride) {
        const int b = owner_of(cum, p.B, j);
        p.free_pages[count + j] = p.table[(int64_t)b * p.max_pages + from[b] + (j - cum[b])];
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

template <typename P>
int launch_tables(void (*kern)(P), const P &p, int words, int64_t work, bool in_place, const LaunchCtx &ctx) {
    const size_t smem = (size_t)words * sizeof(int);
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return GQAQ_ERR_CUDA;
    const int ctas = table_ctas(work, in_place);
    const cudaError_t e = launch_kernel(kern, dim3((unsigned)ctas), dim3(kTabThreads), smem, ctx, in_place ? ctas : 0, p);
    return e == cudaSuccess ? GQAQ_OK : GQAQ_ERR_CUDA;
}

// ---------------------------------------------------------------------------
// Norm, rotation and append
// ---------------------------------------------------------------------------
constexpr int kAppendRows = 2;  // rows of a token per thread

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
};

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4 &x, float (&y)[8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (BF16) {
            y[2 * i] = __uint_as_float(w[i] << 16);
            y[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        } else {
            const float2 f = half2_bits_to_float2(w[i]);
            y[2 * i] = f.x;
            y[2 * i + 1] = f.y;
        }
    }
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    if (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&y)[8]) {
    return make_uint4(pack2<BF16>(y[0], y[1]), pack2<BF16>(y[2], y[3]), pack2<BF16>(y[4], y[5]), pack2<BF16>(y[6], y[7]));
}

// D/16 lanes share a head's row; a lane holds two blocks of eight channels:
// (8j, rope/2 + 8j), so that with the halves style both members of every pair
// sit in one lane, and two neighbouring blocks where nothing turns. A thread
// owns the same two rows (heads) of every token its CTA takes, so the norm
// weights stay in registers, a token's angles serve both rows, and the next
// token's rows are loaded while this one's are computed: the kernel moves each
// byte once and is bound by HBM (see launch_append_t for the shape).
template <int D, bool BF16, bool INTER>
__global__ void __launch_bounds__(256) paged_append_kernel(const AppendPagedParams p) {
    constexpr int LPR = D / 16;         // lanes per row
    constexpr int NP = kAppendRows;     // rows per thread
    pdl_wait_and_release();
    const int rpp = (int)blockDim.x / LPR;  // rows per pass
    const int j = threadIdx.x % LPR, r0 = threadIdx.x / LPR;
    const int R = p.rope;
    const bool turns = 16 * j < R;
    const int c0 = turns ? 8 * j : 16 * j, c1 = turns ? R / 2 + 8 * j : 16 * j + 8;
    // halves: pair i of both blocks is channel 8j + i; adjacent pairs: a block
    // of eight channels holds pairs c/2 .. c/2 + 3
    const int i0 = INTER ? c0 / 2 : 8 * j, i1 = INTER ? c1 / 2 : 8 * j + 4;
    const int H = p.Hq + 2 * p.Hkv;
    int head[NP], kind[NP];             // head within its tensor; 0 q, 1 k, 2 v, 3 none
    uint4 wa[NP], wb[NP];
    bool norm[NP];
#pragma unroll
    for (int n = 0; n < NP; ++n) {
        const int h = ((int)blockIdx.y * NP + n) * rpp + r0;
        kind[n] = h < p.Hq ? 0 : h < p.Hq + p.Hkv ? 1 : h < H ? 2 : 3;
        head[n] = kind[n] == 0 ? h : kind[n] == 1 ? h - p.Hq : h - p.Hq - p.Hkv;
        const uint16_t *w = kind[n] == 0 ? p.q_weight : kind[n] == 1 ? p.k_weight : nullptr;
        norm[n] = w != nullptr;
        wa[n] = wb[n] = make_uint4(0u, 0u, 0u, 0u);
        if (norm[n]) {
            wa[n] = *reinterpret_cast<const uint4 *>(w + c0);
            wb[n] = *reinterpret_cast<const uint4 *>(w + c1);
        }
    }
    // a token's place, or -1: padding, or refused
    auto place = [&](int t, int &pos) {
        const int slot = p.slots[t];
        pos = R > 0 ? p.positions[t] : 0;
        int flags = 0;
        if (slot < 0) return -1;
        if ((slot >> p.shift) >= p.num_pages) flags |= GQAQ_DEV_BAD_PAGE;
        if (R > 0 && (pos < 0 || pos >= p.max_position)) flags |= GQAQ_DEV_BAD_POS;
        if (flags == 0) return slot;
        if (threadIdx.x == 0 && blockIdx.y == 0) raise_flag(p.status, flags);
        return -1;
    };
    auto load = [&](int t, uint4 (&x0)[NP], uint4 (&x1)[NP]) {
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            if (kind[n] == 3) continue;
            const uint16_t *src = (kind[n] == 0 ? p.q + t * p.q_stride : kind[n] == 1 ? p.k + t * p.k_stride : p.v + t * p.v_stride) + head[n] * D;
            x0[n] = *reinterpret_cast<const uint4 *>(src + c0);
            x1[n] = *reinterpret_cast<const uint4 *>(src + c1);
        }
    };
    uint4 x0[NP], x1[NP], y0[NP], y1[NP];
#pragma unroll
    for (int n = 0; n < NP; ++n) x0[n] = x1[n] = y0[n] = y1[n] = make_uint4(0u, 0u, 0u, 0u);
    int pos = 0, next_pos = 0;
    int slot = place(blockIdx.x, pos);
    if (slot >= 0) load(blockIdx.x, x0, x1);
    for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
        const int tn = t + (int)gridDim.x;
        int next = -1;
        if (tn < p.T) {
            next = place(tn, next_pos);
            if (next >= 0) load(tn, y0, y1);
        }
        if (slot >= 0) {  // the same for the whole CTA
            float cs[8], sn[8];
            if (turns) {
                const float *row = p.cos_sin + (int64_t)pos * R;
                const float4 a = *reinterpret_cast<const float4 *>(row + i0), b = *reinterpret_cast<const float4 *>(row + i1);
                const float4 c = *reinterpret_cast<const float4 *>(row + R / 2 + i0), d = *reinterpret_cast<const float4 *>(row + R / 2 + i1);
                cs[0] = a.x; cs[1] = a.y; cs[2] = a.z; cs[3] = a.w; cs[4] = b.x; cs[5] = b.y; cs[6] = b.z; cs[7] = b.w;
                sn[0] = c.x; sn[1] = c.y; sn[2] = c.z; sn[3] = c.w; sn[4] = d.x; sn[5] = d.y; sn[6] = d.z; sn[7] = d.w;
            }
            const int page = slot >> p.shift, row_in = slot & (p.S - 1);
#pragma unroll
            for (int n = 0; n < NP; ++n) {
                float a[8], b[8];
                unpack8<BF16>(x0[n], a);
                unpack8<BF16>(x1[n], b);
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) ss += a[e] * a[e] + b[e] * b[e];
#pragma unroll
                for (int o = 1; o < LPR; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                if (kind[n] == 3) continue;
                if (norm[n]) {
                    const float inv = rsqrtf(ss * (1.f / D) + p.eps);
                    float u[8], v[8];
                    unpack8<BF16>(wa[n], u);
                    unpack8<BF16>(wb[n], v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        a[e] = a[e] * inv * u[e];
                        b[e] = b[e] * inv * v[e];
                    }
                }
                const bool turn = turns && kind[n] != 2;
                if (turn) {
                    if (INTER) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float u = a[2 * e], v = a[2 * e + 1], y = b[2 * e], z = b[2 * e + 1];
                            a[2 * e] = u * cs[e] - v * sn[e];
                            a[2 * e + 1] = v * cs[e] + u * sn[e];
                            b[2 * e] = y * cs[4 + e] - z * sn[4 + e];
                            b[2 * e + 1] = z * cs[4 + e] + y * sn[4 + e];
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float u = a[e], v = b[e];
                            a[e] = u * cs[e] - v * sn[e];
                            b[e] = v * cs[e] + u * sn[e];
                        }
                    }
                }
                uint16_t *dst = kind[n] == 0 ? p.q_out + ((int64_t)t * p.Hq + head[n]) * D
                                             : (kind[n] == 1 ? p.k_pages : p.v_pages) + (((int64_t)page * p.Hkv + head[n]) * p.S + row_in) * D;
                const bool same = !norm[n] && !turn;  // nothing computed: the bits as they are
                *reinterpret_cast<uint4 *>(dst + c0) = same ? x0[n] : pack8<BF16>(a);
                *reinterpret_cast<uint4 *>(dst + c1) = same ? x1[n] : pack8<BF16>(b);
            }
        }
        slot = next;
        pos = next_pos;
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            x0[n] = y0[n];
            x1[n] = y1[n];
        }
    }
}

template <int D, bool BF16>
int launch_append_t(const AppendPagedParams &p, bool inter, const LaunchCtx &ctx) {
    auto kern = inter ? paged_append_kernel<D, BF16, true> : paged_append_kernel<D, BF16, false>;
    const int H = p.Hq + 2 * p.Hkv, lanes = D / 16;
    // threads for half a token's rows (two rows each), in whole warps; more
    // heads than 256 threads hold take more CTAs per token
    int threads = ((H + kAppendRows - 1) / kAppendRows * lanes + 31) / 32 * 32;
    if (threads > 256) threads = 256;
    const int rows = threads / lanes * kAppendRows, gy = (H + rows - 1) / rows;
    int per_sm = 1;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, 0) != cudaSuccess || per_sm < 1) return GQAQ_ERR_CUDA;
    int gx = per_sm * ctx.num_sms / gy;
    gx = gx < 1 ? 1 : gx < p.T ? gx : p.T;
    const cudaError_t e = launch_kernel(kern, dim3((unsigned)gx, (unsigned)gy), dim3((unsigned)threads), 0, ctx, 0, p);
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
    return launch_tables(paged_tables_kernel, p, 3 * d.batch + 2, (int64_t)d.max_tokens + d.batch, a.free_count == a.free_count_out, ctx);
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
    return launch_tables(paged_release_kernel, p, 2 * d.batch + 1, table < d.num_pages ? table : d.num_pages,
                         a.free_count == a.free_count_out, ctx);
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
    const bool inter = a.interleaved != 0;
    if (d.dtype == GQAQ_BF16)
        return d.head_dim == 128 ? launch_append_t<128, true>(p, inter, ctx) : launch_append_t<64, true>(p, inter, ctx);
    return d.head_dim == 128 ? launch_append_t<128, false>(p, inter, ctx) : launch_append_t<64, false>(p, inter, ctx);
}

}  // namespace gqaq
