// paged_append_e4m3.cu -- per-head RMS norm, rotation and append of a step's
// tokens to 8-bit pages (paged_e4m3.cuh).
//
// A run is the step's tokens of one page: consecutive rows whose slots ascend
// by one (one of them without an angle is skipped, and the run goes on). For each
// run and KV head, of keys and of values alike:
//   a    = the largest finite |y| of the run's rows (fp32, after norm and rotation)
//   e    = the least exponent with a <= 448 * 2^e; of a page that holds rows (the
//          run does not begin at its row 0) at least the exponent it has
//   code = nearest E4M3 code to y * 2^-e (one rounding from fp32)
// and where a page's exponent grows, the codes that it holds are rounded to the
// new one.
//
// Kernel shape: a CTA per (window of tokens, KV head): the window's query rows
// of the KV head's group, and the keys and values of the runs that begin in it,
// wherever they end. D/16 lanes share a row and keep one token, whose query rows
// all turn by the same angles; the keys and values are the rows from the
// window's first run on, as many as the window has in one pass (a page that lies
// across two windows takes no more: a run ends before the next one's first row),
// and more passes where a page is longer than the window. The query rows, asked
// for first, are worked on while the keys and values are on their way; these
// wait in registers for the runs' maxima (rows of later passes are read and
// computed again).
//
// What bounds it (8192 tokens, 32 query and 8 KV heads of 128 channels, pages of
// 16, normed and rotated: 44 us, 4.3 TB/s, 63% of the copy rate): a CTA's chain
// of slots, rows, maxima, exponents and codes, each of which waits for the one
// before, beside 17 instructions per channel (55% of the issue slots; a third
// are conversions and moves between register pairs). A small step is that chain
// once (32 single tokens 5.2 us; four chunks among 19 single tokens over pages of
// 64, which are two windows of 128 channels and computed twice, 9.0), where no
// page's exponent grows. A window's grown pages are rounded again by its one CTA,
// 16 bytes a thread after the other: where all pages of 32 single tokens grow, 8
// and 12 us (64 and 128 channels, pages of 16), 17 and 29 (of 64), 28 and 50 (of
// 128); of 256 single tokens 14 and 15, 38 and 42, 66 and 76; of 16 times 5 drafted
// tokens 9 and 8, 13 and 12, 18 and 17.
#include "paged_e4m3.cuh"
#include "paged_rows.cuh"

namespace gqaq {
namespace {

// Threads of a CTA, those of an SM, and the query rows that a lane has in flight. A step whose CTAs all run at once asks for
// all it needs at the start. A longer one gains more from half as long windows and six CTAs per SM, which are at different
// stages, though each has fewer rows in flight (32 query and 8 KV heads of 128 channels, pages of 16: 1024 tokens 7.1 us
// against 9.0, 1500 tokens 10.7 against 9.3, 8000 tokens 48.7 against 43.3). Pages longer than such a window stay with the long
// one: a run's rows beyond the first pass are read and computed twice (8192 tokens, long against short windows: 128 channels,
// pages of 32, 64 and 128 50, 54 and 59 us against 47, 52 and 61; 64 channels, of 64 and 128 26 and 29 against 27 and 32).
struct FewTokens {
    static constexpr int THREADS = 256, RESIDENT = 512, AHEAD = 4;
};
struct ManyTokens {
    static constexpr int THREADS = 128, RESIDENT = 768, AHEAD = 1;
};

struct Append8Params {
    const uint16_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    const int *positions, *slots;
    const uint16_t *q_weight, *k_weight;
    float eps;
    const float *cos_sin;
    uint16_t *q_out;
    uint8_t *k_pages, *v_pages;
    int8_t *k_exp, *v_exp;
    int *status;
    int T, Hq, Hkv, G, S, shift, num_pages, rope, max_position;
};

// Largest finite magnitude of eight 16-bit numbers and eight more, as the bits of a 32-bit float.
template <bool BF16>
__device__ __forceinline__ uint32_t largest16(const uint4 &x, const uint4 &y) {
    constexpr uint32_t INF = BF16 ? 0x7f80u : 0x7c00u;
    const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    uint32_t m = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = __vmaxu2(m, w[e] & 0x7fff7fffu);  // bits of non-negative numbers are ordered as they are
    m = max(m & 0xffffu, m >> 16);
    if (__builtin_expect(m >= INF, 0)) {
        m = 0u;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t lo = w[e] & 0x7fffu, hi = (w[e] >> 16) & 0x7fffu;
            m = max(m, max(lo < INF ? lo : 0u, hi < INF ? hi : 0u));
        }
    }
    return BF16 ? m << 16 : __float_as_uint(half2_bits_to_float2(m).x);
}
__device__ __forceinline__ uint32_t largest32(const f32x2 (&a)[4], const f32x2 (&b)[4]) {
    float m = 0.f;  // fmaxf passes NaN over
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 y = unpair32(a[e]), z = unpair32(b[e]);
        m = fmaxf(fmaxf(m, fmaxf(fabsf(y.x), fabsf(y.y))), fmaxf(fabsf(z.x), fabsf(z.y)));
    }
    if (__builtin_expect(m == INFINITY, 0)) {
        m = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 y = unpair32(a[e]), z = unpair32(b[e]);
            const float c[4] = {fabsf(y.x), fabsf(y.y), fabsf(z.x), fabsf(z.y)};
#pragma unroll
            for (int i = 0; i < 4; ++i) m = fmaxf(m, c[i] < INFINITY ? c[i] : 0.f);
        }
    }
    return __float_as_uint(m);
}

template <int D, bool BF16, bool INTER, typename Form>
__global__ void __launch_bounds__(Form::THREADS, Form::RESIDENT / Form::THREADS) paged_append_e4m3_kernel(const Append8Params p) {
    constexpr int kThreads = Form::THREADS, kAhead = Form::AHEAD;
    constexpr int LPR = D / 16;                      // lanes per row
    constexpr int W = kThreads / LPR;                // tokens of a window
    constexpr int WORDS = (1 + W + 127 + 31) / 32;   // of 32 tokens looked at, at most: one before, and a run's end
    __shared__ int slot_s[WORDS * 32];               // token t0 - 1 + i; -1: padding, or no such page
    __shared__ int pos_s[WORDS * 32];
    __shared__ uint32_t live_s[WORDS];               // bit i: the token has a slot and a position
    __shared__ uint32_t begins_s[WORDS], joins_s[WORDS];  // a run begins at the token; it goes on there
    __shared__ unsigned amax_s[2][W];                // keys, then values, of the run that begins at token t0 + i
    __shared__ int exp_s[2][W], grown_s[2][W];
    __shared__ int list_s[2 * W], listed_s;          // runs whose page's exponent grew
    const int tid = threadIdx.x, lane = tid & 31;
    const int win = blockIdx.x / p.Hkv, h = blockIdx.x - win * p.Hkv;
    const int64_t t0 = (int64_t)win * W;
    const int R = p.rope, look = 1 + W + p.S - 1, words = (look + 31) / 32;
    const int j = tid % LPR, r0 = tid / LPR;  // a lane's place in its row, its token in the window
    const RowLane w = RowLane::of<INTER>(j, R);
    const bool norm_k = p.k_weight != nullptr, norm_q = p.q_weight != nullptr;
    struct Raw {
        uint4 x0, x1;
    };
    auto load = [&](const uint16_t *row, bool here) {
        Raw x;
        x.x0 = x.x1 = make_uint4(0u, 0u, 0u, 0u);
        if (here) {
            x.x0 = *reinterpret_cast<const uint4 *>(row + w.c0);
            x.x1 = *reinterpret_cast<const uint4 *>(row + w.c1);
        }
        return x;
    };
    RowAngles angles;
    auto turn_to = [&](int pos, bool here) {
        if (w.turns && here) angles.load(p.cos_sin + (int64_t)pos * R, R, w);
    };
    pdl_wait_and_release();

    // ---- this lane's token: its first query rows and its angles, asked for ----
    bool live_q = false;
    int pos_q = 0;
    if (t0 + r0 < p.T) {
        const int slot = p.slots[t0 + r0];
        if (R > 0) pos_q = p.positions[t0 + r0];
        live_q = slot >= 0 && (slot >> p.shift) < p.num_pages && (R == 0 || (uint32_t)pos_q < (uint32_t)p.max_position);
    }
    const uint16_t *q_row = p.q + (t0 + r0) * p.q_stride + (int64_t)h * p.G * D;
    Raw q[kAhead];
#pragma unroll
    for (int x = 0; x < kAhead; ++x) q[x] = load(q_row + x * D, live_q && x < p.G);
    turn_to(pos_q, live_q);

    // ---- the window's runs ----
    for (int i = tid; i < words * 32; i += kThreads) {
        const int64_t t = t0 - 1 + i;
        int slot = -1, pos = 0, flags = 0;
        if (i < look && t >= 0 && t < p.T) {
            slot = p.slots[t];
            if (R > 0) pos = p.positions[t];
            if (slot >= 0 && (slot >> p.shift) >= p.num_pages) {
                slot = -1;
                flags |= GQAQ_DEV_BAD_PAGE;
            } else if (slot >= 0 && R > 0 && (uint32_t)pos >= (uint32_t)p.max_position) {
                flags |= GQAQ_DEV_BAD_POS;
            }
            if (flags && h == 0 && i > 0 && i <= W) raise_flag(p.status, flags);
        }
        slot_s[i] = slot;
        pos_s[i] = pos;
        const unsigned live = __ballot_sync(0xffffffffu, slot >= 0 && flags == 0);
        if (lane == 0) live_s[i >> 5] = live;
    }
    if (tid < 2 * W) amax_s[0][tid] = 0u;
    if (tid == 0) listed_s = 0;
    __syncthreads();
    for (int i = tid; i < words * 32; i += kThreads) {
        const int now = slot_s[i], before = i > 0 ? slot_s[i - 1] : -1;
        const bool joins = now >= 0 && before >= 0 && now == before + 1 && (now & (p.S - 1)) != 0;
        const unsigned jb = __ballot_sync(0xffffffffu, joins), bb = __ballot_sync(0xffffffffu, now >= 0 && !joins && i > 0);
        if (lane == 0) {
            joins_s[i >> 5] = jb;
            begins_s[i >> 5] = bb;
        }
    }
    __syncthreads();
    auto bit = [](const uint32_t *words, int i) { return (words[i >> 5] >> (i & 31)) & 1u; };
    // tokens first .. last: from the window's first run to its end, or to that of a run that goes on behind it
    int first = 1, last = 0;
    {
        int at = 0;
        uint32_t m = begins_s[0];
        while (m == 0u && at + 1 < words) m = begins_s[++at];
        const int f = 32 * at + __ffs((int)m) - 1;
        if (m != 0u && f <= W) {
            first = f;
            last = W + 1;  // the first token behind the window that joins no run
            uint32_t out = ~joins_s[last >> 5] >> (last & 31);
            while (out == 0u && (last | 31) + 1 < words * 32) {
                last = (last | 31) + 1;
                out = ~joins_s[last >> 5];
            }
            last = min(out == 0u ? look : last + __ffs((int)out) - 1, look) - 1;
        }
    }
    // the window's token (0 ..) whose run token i belongs to, or -1
    auto run_of = [&](int i) {
        if (!bit(live_s, i)) return -1;
        int x = i >> 5;
        uint32_t m = begins_s[x] & (uint32_t)((2ull << (i & 31)) - 1ull);
        while (m == 0u && x > 0) m = begins_s[--x];
        const int at = m == 0u ? 0 : 32 * x + 31 - __clz((int)m);
        return at >= 1 && at <= W ? at - 1 : -1;
    };
    auto k_row = [&](int i) { return p.k + (t0 - 1 + i) * p.k_stride + (int64_t)h * D; };
    auto v_row = [&](int i) { return p.v + (t0 - 1 + i) * p.v_stride + (int64_t)h * D; };
    const int i0 = first + r0;  // this lane's token of the first pass
    const int run0 = i0 <= last ? run_of(i0) : -1;
    const Raw k0 = load(k_row(i0), run0 >= 0), v0 = load(v_row(i0), run0 >= 0);

    // ---- queries ----
    uint16_t *q_dst = p.q_out + ((t0 + r0) * p.Hq + (int64_t)h * p.G) * D;
    for (int g = 0; g < p.G; g += kAhead) {
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
            if (g + x >= p.G) break;
            Raw y = q[x];
            if (g + x + kAhead < p.G) q[x] = load(q_row + (g + x + kAhead) * D, live_q);
            if (norm_q || w.turns) {  // else the bits as they are
                f32x2 a[4], b[4];
                unpack8<BF16>(y.x0, a);
                unpack8<BF16>(y.x1, b);
                if (norm_q) row_norm<D, BF16>(a, b, row_square_sum<D>(a, b), p.eps, reinterpret_cast<const uint8_t *>(p.q_weight), w);
                if (w.turns && live_q) row_turn<INTER>(a, b, angles);
                y.x0 = pack8<BF16>(a);
                y.x1 = pack8<BF16>(b);
            }
            if (live_q) {
                *reinterpret_cast<uint4 *>(q_dst + (g + x) * D + w.c0) = y.x0;
                *reinterpret_cast<uint4 *>(q_dst + (g + x) * D + w.c1) = y.x1;
            }
        }
    }
    if (last == 0) return;  // no run begins here (the whole CTA knows)

    // ---- keys and values: their runs' maxima ----
    auto key = [&](const Raw &x, bool here, f32x2 (&a)[4], f32x2 (&b)[4]) {  // whole warps call
        unpack8<BF16>(x.x0, a);
        unpack8<BF16>(x.x1, b);
        if (norm_k) row_norm<D, BF16>(a, b, row_square_sum<D>(a, b), p.eps, reinterpret_cast<const uint8_t *>(p.k_weight), w);
        if (w.turns && here) row_turn<INTER>(a, b, angles);
    };
    auto maximum = [&](uint32_t m, int run, int kind) {
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (j == 0 && run >= 0) atomicMax(&amax_s[kind][run], m);
    };
    if (first != 1) turn_to(pos_s[i0], run0 >= 0);
    f32x2 ka[4], kb[4];
    key(k0, run0 >= 0, ka, kb);
    maximum(largest32(ka, kb), run0, 0);
    maximum(largest16<BF16>(v0.x0, v0.x1), run0, 1);
    for (int i = i0 + W; i - r0 <= last; i += W) {
        const int run = i <= last ? run_of(i) : -1;
        const Raw k1 = load(k_row(i), run >= 0), v1 = load(v_row(i), run >= 0);
        turn_to(pos_s[run >= 0 ? i : 0], run >= 0);
        f32x2 a[4], b[4];
        key(k1, run >= 0, a, b);
        maximum(largest32(a, b), run, 0);
        maximum(largest16<BF16>(v1.x0, v1.x1), run, 1);
    }

    // ---- the runs' exponents ----
    __syncthreads();
    if (tid < 2 * W) {
        const int i = tid >> 1, kind = tid & 1;
        if (bit(begins_s, 1 + i)) {
            const int slot = slot_s[1 + i];
            int8_t *place = (kind ? p.v_exp : p.k_exp) + (int64_t)(slot >> p.shift) * p.Hkv + h;
            int e = page_exp_of(amax_s[kind][i]);
            if ((slot & (p.S - 1)) != 0) {
                const int old = min(max((int)*place, kLeastPageExp), kMostPageExp);
                e = max(e, old);
                grown_s[kind][i] = e - old;
                if (e > old) list_s[atomicAdd(&listed_s, 1)] = tid;
            }
            *place = (int8_t)e;
            exp_s[kind][i] = e;
        }
    }
    __syncthreads();

    // ---- codes ----
    auto store = [&](const f32x2 (&a)[4], const f32x2 (&b)[4], int slot, int run, int kind) {
        const float by = pow2i(-exp_s[kind][run]);
        const f32x2 by2 = pair32(by, by);
        uint8_t *dst = (kind ? p.v_pages : p.k_pages) + ((((int64_t)(slot >> p.shift) * p.Hkv + h) << p.shift) + (slot & (p.S - 1))) * D;
        *reinterpret_cast<uint2 *>(dst + w.c0) = make_uint2(f32x4_to_e4m3x4(mul2(a[0], by2), mul2(a[1], by2)), f32x4_to_e4m3x4(mul2(a[2], by2), mul2(a[3], by2)));
        *reinterpret_cast<uint2 *>(dst + w.c1) = make_uint2(f32x4_to_e4m3x4(mul2(b[0], by2), mul2(b[1], by2)), f32x4_to_e4m3x4(mul2(b[2], by2), mul2(b[3], by2)));
    };
    auto value = [&](const Raw &x, int slot, int run) {
        f32x2 a[4], b[4];
        unpack8<BF16>(x.x0, a);
        unpack8<BF16>(x.x1, b);
        store(a, b, slot, run, 1);
    };
    if (run0 >= 0) {
        store(ka, kb, slot_s[i0], run0, 0);
        value(v0, slot_s[i0], run0);
    }
    for (int i = i0 + W; i - r0 <= last; i += W) {
        const int run = i <= last ? run_of(i) : -1;
        const Raw k1 = load(k_row(i), run >= 0), v1 = load(v_row(i), run >= 0);
        turn_to(pos_s[run >= 0 ? i : 0], run >= 0);
        key(k1, run >= 0, ka, kb);
        if (run >= 0) {
            store(ka, kb, slot_s[i], run, 0);
            value(v1, slot_s[i], run);
        }
    }

    // ---- pages whose exponent grew: the codes of their other rows ----
    const int per = p.S * LPR;  // 16-byte words of a page
    for (int c = tid; c < listed_s * per; c += kThreads) {
        const int u = list_s[c / per], i = u >> 1, kind = u & 1, word = c % per, row = word / LPR;
        const int slot = slot_s[1 + i], row0 = slot & (p.S - 1);
        if (row >= row0 && run_of(1 + i + row - row0) == i) continue;  // written above
        const float by = pow2i(-grown_s[kind][i]);
        uint4 *at = reinterpret_cast<uint4 *>((kind ? p.v_pages : p.k_pages) + (((int64_t)(slot >> p.shift) * p.Hkv + h) << p.shift) * D) + word;
        const uint4 x = *at;
        *at = make_uint4(e4m3x4_shift(x.x, by), e4m3x4_shift(x.y, by), e4m3x4_shift(x.z, by), e4m3x4_shift(x.w, by));
    }
}

template <int D, bool BF16, typename Form>
int launch_form(Append8Params &p, bool inter, const LaunchCtx &ctx) {
    auto kern = inter ? paged_append_e4m3_kernel<D, BF16, true, Form> : paged_append_e4m3_kernel<D, BF16, false, Form>;
    constexpr int W = Form::THREADS / (D / 16);
    const int64_t ctas = (int64_t)((p.T + W - 1) / W) * p.Hkv;
    const cudaError_t e = launch_kernel(kern, dim3((unsigned)ctas), dim3(Form::THREADS), 0, ctx, 0, p);
    return e == cudaSuccess ? GQAQ_OK : GQAQ_ERR_CUDA;
}

template <int D, bool BF16>
int launch_t(Append8Params &p, bool inter, const LaunchCtx &ctx) {
    constexpr int LPR = D / 16;
    const int64_t threads = (int64_t)p.T * p.Hkv * LPR;
    const bool many = p.S <= ManyTokens::THREADS / LPR && threads > (int64_t)FewTokens::RESIDENT * ctx.num_sms;
    return many ? launch_form<D, BF16, ManyTokens>(p, inter, ctx) : launch_form<D, BF16, FewTokens>(p, inter, ctx);
}

}  // namespace

int launch_paged_append_e4m3(const PagedAppendArgs &a, const LaunchCtx &ctx) {
    const gqaq_paged_dims &d = *a.dims;
    Append8Params p;
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
    p.k_pages = static_cast<uint8_t *>(a.k_pages);
    p.v_pages = static_cast<uint8_t *>(a.v_pages);
    p.k_exp = a.k_exp;
    p.v_exp = a.v_exp;
    p.status = ctx.status;
    p.T = d.max_tokens;
    p.Hq = d.num_q_heads;
    p.Hkv = d.num_kv_heads;
    p.G = d.num_q_heads / d.num_kv_heads;
    p.S = d.page_size;
    p.shift = 0;
    while ((1 << p.shift) < d.page_size) ++p.shift;
    p.num_pages = d.num_pages;
    p.rope = a.rope_dim;
    p.max_position = a.max_position;
    const bool inter = a.interleaved != 0;
    if (d.dtype == GQAQ_BF16)
        return d.head_dim == 128 ? launch_t<128, true>(p, inter, ctx) : launch_t<64, true>(p, inter, ctx);
    return d.head_dim == 128 ? launch_t<128, false>(p, inter, ctx) : launch_t<64, false>(p, inter, ctx);
}

}  // namespace gqaq
