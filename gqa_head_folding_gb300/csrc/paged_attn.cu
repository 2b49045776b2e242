// paged_attn.cu -- attention of each request's new tokens over a paged cache.
//
// Request b owns rows cu_q[b] .. cu_q[b+1]-1 of q; token i of its q_len new
// tokens sits at position kv_len - q_len + i and attends to the tokens up to
// itself, whose rows lie in the pages of block_table[b].
#include <math.h>

#include <cuda_bf16.h>

#include "internal.h"

namespace gqaq {
namespace {

struct PagedAttnParams {
    const uint16_t *q, *k_pages, *v_pages;
    const int *table, *cu_q, *kv_len;
    uint16_t *out;
    int *status;
    int B, T, Hq, Hkv, S, num_pages, max_pages, max_q;
    float scale_log2;
};

template <bool BF16>
__device__ __forceinline__ float to_f32(uint16_t x) {
    return BF16 ? __uint_as_float((uint32_t)x << 16) : __half2float(__ushort_as_half(x));
}
template <bool BF16>
__device__ __forceinline__ uint16_t from_f32(float x) {
    return BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(x)) : __half_as_ushort(__float2half_rn(x));
}

// One warp per (token, query head): 32 keys at a time, a key per lane for the
// scores, D/32 channels per lane for the sum over values.
template <int D, bool BF16>
__global__ void __launch_bounds__(128) paged_attn_kernel(const PagedAttnParams p) {
    constexpr int EPL = D / 32;
    __shared__ float qs[4][D];
    pdl_wait_and_release();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * 4 + warp;
    if (blockIdx.x == 0) {
        for (int b = threadIdx.x; b < p.B; b += 128) {
            const int c0 = p.cu_q[b], c1 = p.cu_q[b + 1];
            int flags = 0;
            if (p.kv_len[b] < 0 || (int64_t)p.kv_len[b] > (int64_t)p.max_pages * p.S || c1 - c0 > p.max_q) flags |= GQAQ_DEV_BAD_LEN;
            if (c0 < 0 || c1 < c0 || c1 > p.T) flags |= GQAQ_DEV_BAD_POS;
            if (flags) raise_flag(p.status, flags);
        }
    }
    if (w >= (int64_t)p.T * p.Hq) return;
    const int t = (int)(w / p.Hq), h = (int)(w % p.Hq), kv = h / (p.Hq / p.Hkv);
    // the request of row t: the last b with cu_q[b] <= t
    if (t < p.cu_q[0] || t >= p.cu_q[p.B]) return;
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.cu_q[mid] <= t) lo = mid; else hi = mid;
    }
    const int b = lo, i = t - p.cu_q[b], n = p.cu_q[b + 1] - p.cu_q[b];
    if (i < 0 || i >= n || i >= p.max_q) return;
    const int len = (int)min((int64_t)max(p.kv_len[b], 0), (int64_t)p.max_pages * p.S);
    const int last = len - n + i;  // this token's position
    const uint16_t *qr = p.q + ((int64_t)t * p.Hq + h) * D;
    for (int d = lane; d < D; d += 32) qs[warp][d] = to_f32<BF16>(qr[d]);
    __syncwarp();
    float m = -INFINITY, l = 0.f, o[EPL];
#pragma unroll
    for (int e = 0; e < EPL; ++e) o[e] = 0.f;
    for (int k0 = 0; k0 <= last; k0 += 32) {
        const int key = k0 + lane;
        int64_t row = -1;
        float s = -INFINITY;
        if (key <= last) {
            const int page = p.table[(int64_t)b * p.max_pages + key / p.S];
            s = 0.f;
            if (page >= 0 && page < p.num_pages) {
                row = ((int64_t)page * p.Hkv + kv) * p.S + key % p.S;
                const uint16_t *kr = p.k_pages + row * D;
                for (int d = 0; d < D; ++d) s = fmaf(qs[warp][d], to_f32<BF16>(kr[d]), s);
                s *= p.scale_log2;
            } else {
                raise_flag(p.status, GQAQ_DEV_BAD_PAGE);
            }
        }
        float mx = s;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
        const float mn = fmaxf(m, mx), ref = mn == -INFINITY ? 0.f : mn;
        const float al = exp2f(m - ref), pr = exp2f(s - ref);
        m = mn;
        float ps = pr;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, x);
        l = l * al + ps;
#pragma unroll
        for (int e = 0; e < EPL; ++e) o[e] *= al;
        for (int j = 0; j < 32 && k0 + j <= last; ++j) {
            const float pj = __shfl_sync(0xffffffffu, pr, j);
            const int64_t rj = __shfl_sync(0xffffffffu, row, j);
            if (rj < 0) continue;
#pragma unroll
            for (int e = 0; e < EPL; ++e) o[e] = fmaf(pj, to_f32<BF16>(p.v_pages[rj * D + lane * EPL + e]), o[e]);
        }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    uint16_t *out = p.out + ((int64_t)t * p.Hq + h) * D + lane * EPL;
#pragma unroll
    for (int e = 0; e < EPL; ++e) out[e] = from_f32<BF16>(o[e] * inv);
}

template <int D, bool BF16>
int launch_t(const PagedAttnArgs &a, const LaunchCtx &ctx) {
    const gqaq_paged_dims &d = *a.dims;
    PagedAttnParams p;
    p.q = static_cast<const uint16_t *>(a.q);
    p.k_pages = static_cast<const uint16_t *>(a.k_pages);
    p.v_pages = static_cast<const uint16_t *>(a.v_pages);
    p.table = a.block_table;
    p.cu_q = a.cu_q;
    p.kv_len = a.kv_len;
    p.out = static_cast<uint16_t *>(a.out);
    p.status = ctx.status;
    p.B = d.batch;
    p.T = d.max_tokens;
    p.Hq = d.num_q_heads;
    p.Hkv = d.num_kv_heads;
    p.S = d.page_size;
    p.num_pages = d.num_pages;
    p.max_pages = d.max_pages;
    p.max_q = a.max_q_len;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    const int64_t warps = (int64_t)d.max_tokens * d.num_q_heads;
    const cudaError_t e = launch_kernel(paged_attn_kernel<D, BF16>, dim3((unsigned)((warps + 3) / 4)), dim3(128), 0, ctx, 0, p);
    return e == cudaSuccess ? GQAQ_OK : GQAQ_ERR_CUDA;
}

}  // namespace

size_t paged_attn_workspace_bytes(const gqaq_paged_dims *d, const LaunchCtx &ctx) { return paged_tc_workspace_bytes(d, ctx); }

int launch_paged_attn(const PagedAttnArgs &a, const LaunchCtx &ctx) {
    if (a.workspace_bytes < paged_attn_workspace_bytes(a.dims, ctx)) return GQAQ_ERR_WORKSPACE;
    if ((int64_t)a.max_q_len * (a.dims->num_q_heads / a.dims->num_kv_heads) > 8) return launch_paged_tc(a, ctx);
    if (a.dims->dtype == GQAQ_BF16) return a.dims->head_dim == 128 ? launch_t<128, true>(a, ctx) : launch_t<64, true>(a, ctx);
    return a.dims->head_dim == 128 ? launch_t<128, false>(a, ctx) : launch_t<64, false>(a, ctx);
}

}  // namespace gqaq
