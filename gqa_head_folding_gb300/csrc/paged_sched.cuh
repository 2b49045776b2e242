// paged_sched.cuh -- how the paged attention kernels share out a ragged step.
//
// An item is (request, KV head, block of TB tokens); the G query heads of the
// KV head and the block's tokens form its rows, token outer: row r is token
// r / G, head r % G. An item's context is cut into tiles of 128 tokens, up to
// its last row's position. A tile costs one unit, or two where the block has
// more than `half` tokens (the tensor-memory kernel runs it for two row
// tiles), and an item costs as `extra` more tiles before its first, for what
// it takes beside its tiles (a batch of 30 short contexts and two chunks ended between
// 59 and 94 us without them). The units of all items, in the order (request, KV head, block,
// tile), are split into equal contiguous ranges, one per CTA, so a batch of
// unlike lengths loads all SMs alike; consecutive CTAs work on the same keys,
// which the L2 then serves. A tile is its first unit's owner's. An item whose
// tiles have several owners is merged by the one that finishes last.
#pragma once

#include "internal.h"

namespace gqaq {

constexpr int kPagedTileLog = 7, kPagedTile = 1 << kPagedTileLog;

struct PagedWorkParams {
    const int *table, *cu_q, *kv_len;
    int B, T, Hkv, max_q;
    int shift;             // log2 of the page size
    int tbs;               // log2 of TB, the tokens per block
    int half;              // tokens of a block above which its tiles cost two units
    int extra;             // what an item costs beside its tiles, in tiles
    int num_pages, max_pages;
    int64_t room;          // max_pages * page size
};

inline void fill_paged_work(const PagedAttnArgs &a, int tbs, int half, int extra, PagedWorkParams &w) {
    const gqaq_paged_dims &d = *a.dims;
    w.table = a.block_table;
    w.cu_q = a.cu_q;
    w.kv_len = a.kv_len;
    w.B = d.batch;
    w.T = d.max_tokens;
    w.Hkv = d.num_kv_heads;
    w.max_q = a.max_q_len;
    w.tbs = tbs;
    w.half = half;
    w.extra = extra;
    w.shift = 0;
    while ((1 << w.shift) < d.page_size) ++w.shift;
    w.num_pages = d.num_pages;
    w.max_pages = d.max_pages;
    w.room = (int64_t)d.max_pages * d.page_size;
}

// One request as the kernels see it, clamped to what the buffers hold.
struct PagedSeq {
    int q0;     // first row of its tokens
    int m;      // tokens computed: min(q_len, max_q)
    int start;  // position of its first new token (negative: tokens without a place)
    int len;    // tokens in the cache
    int flags;
    __device__ __forceinline__ void load(const PagedWorkParams &p, int b) {
        const int c0 = p.cu_q[b], c1 = p.cu_q[b + 1], raw = p.kv_len[b];
        flags = 0;
        q0 = min(max(c0, 0), p.T);
        const int q1 = min(max(c1, q0), p.T);
        if (q0 != c0 || q1 != c1) flags |= GQAQ_DEV_BAD_POS;
        len = (int)min((int64_t)max(raw, 0), p.room);
        if (len != raw) flags |= GQAQ_DEV_BAD_LEN;
        const int n = q1 - q0;
        m = min(n, p.max_q);
        if (m != n) flags |= GQAQ_DEV_BAD_LEN;
        start = len - n;
    }
};

// Tiles of block rb: those up to the position of its last token.
__device__ __forceinline__ int block_tiles(const PagedSeq &s, int rb, int tbs) {
    const int64_t end = (int64_t)s.start + min((int64_t)(rb + 1) << tbs, (int64_t)s.m);
    return end > 0 ? (int)((end + kPagedTile - 1) >> kPagedTileLog) : 0;
}

// sum_{i=1}^{n} ceil(i / 2^k)
__device__ __forceinline__ int64_t sum_ceil(int64_t n, int k) {
    const int64_t q = n >> k, r = n - (q << k);
    return ((q * (q + 1) / 2) << k) + r * (q + 1);
}

// Tiles of the first rb (whole) blocks. A block's tiles are
// ceil((start + (k + 1) TB) / 128): an arithmetic series when TB is a multiple
// of the tile, else a series in units of TB that rises every 128 / TB blocks.
__device__ __forceinline__ int64_t tiles_before(const PagedSeq &s, int64_t rb, int tbs) {
    if (rb <= 0) return 0;
    int64_t a = (int64_t)s.start + (1ll << tbs), n = rb;
    if (a <= 0) {  // blocks that end before position zero have no tile
        const int64_t skip = (-a >> tbs) + 1;
        if (skip >= n) return 0;
        a += skip << tbs;
        n -= skip;
    }
    if (tbs >= kPagedTileLog)
        return n * ((a + kPagedTile - 1) >> kPagedTileLog) + ((n * (n - 1) / 2) << (tbs - kPagedTileLog));
    const int64_t u = (a + (1ll << tbs) - 1) >> tbs;
    return sum_ceil(u + n - 1, kPagedTileLog - tbs) - sum_ceil(u - 1, kPagedTileLog - tbs);
}

// log2 of the units of a tile of block rb
__device__ __forceinline__ int unit_shift(const PagedSeq &s, int rb, const PagedWorkParams &p) {
    return s.m - (rb << p.tbs) > p.half ? 1 : 0;
}

// Units of the first rb blocks (each but a request's last is whole, hence of
// one kind), and of all blocks of a head.
__device__ __forceinline__ int64_t units_before(const PagedSeq &s, int rb, const PagedWorkParams &p) {
    const int empty = s.start < 0 ? min(rb, -s.start >> p.tbs) : 0;  // blocks that end before position zero
    return (tiles_before(s, rb, p.tbs) + (int64_t)p.extra * (rb - empty)) << unit_shift(s, 0, p);
}
__device__ __forceinline__ int64_t item_units(int tiles, int us, const PagedWorkParams &p) {
    return tiles > 0 ? (int64_t)(tiles + p.extra) << us : 0;
}
__device__ __forceinline__ int64_t head_units(const PagedSeq &s, const PagedWorkParams &p) {
    if (s.m <= 0) return 0;
    const int last = (s.m - 1) >> p.tbs;
    return units_before(s, last, p) + item_units(block_tiles(s, last, p.tbs), unit_shift(s, last, p), p);
}

// Up to 64 probes of a barrier's phase in the shortest loop there is: a
// waiting warp shares its scheduler with warps that compute (with a vote, a
// clock and a sleep between probes, waiting took half of all issue slots).
__device__ __forceinline__ bool mbar_probe64(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, c;\n\t.reg .u32 n;\n\tmov.u32 n, 16;\n"
        "AGAIN_%=:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE_%=;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE_%=;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE_%=;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE_%=;\n\t"
        "sub.u32 n, n, 1;\n\tsetp.ne.u32 c, n, 0;\n\t@c bra AGAIN_%=;\n"
        "DONE_%=:\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Bounded wait of a converged warp for the phase with parity `parity`; false
// on every lane when timeout_ns passed or *abort became nonzero first.
__device__ __forceinline__ bool warp_mbar_wait(uint32_t bar, uint32_t parity, uint64_t timeout_ns, const volatile int *abort) {
    if (__all_sync(0xffffffffu, mbar_probe64(bar, parity))) return true;
    const uint64_t t0 = global_timer_ns();
    while (true) {
        if (__all_sync(0xffffffffu, mbar_probe64(bar, parity))) return true;
        if (__any_sync(0xffffffffu, *abort != 0 || global_timer_ns() - t0 >= timeout_ns)) return false;
    }
}

// The same with sleeps between probes, for warps whose waits are not urgent.
__device__ __forceinline__ bool warp_mbar_wait_slow(uint32_t bar, uint32_t parity, uint64_t timeout_ns, const volatile int *abort) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const uint64_t t0 = global_timer_ns();
    while (true) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        if (__any_sync(0xffffffffu, *abort != 0 || global_timer_ns() - t0 >= timeout_ns)) return false;
    }
}

// First unit of CTA c's range, and the CTA whose range holds unit t: in 32 bits
// where they suffice (a 64-bit division is a long sequence, and these stand
// between the launch and the first load).
constexpr int64_t kSmallUnits = 1 << 22;
__device__ __forceinline__ int64_t unit_begin(int64_t c, int64_t T, int grid) {
    if (T < kSmallUnits && grid < 1024) return (uint32_t)c * (uint32_t)T / (uint32_t)grid;
    return tile_begin(c, T, grid);
}
__device__ __forceinline__ int64_t unit_owner(int64_t t, int64_t T, int grid) {
    if (T < kSmallUnits && grid < 1024) return (((uint32_t)t + 1u) * (uint32_t)grid - 1u) / (uint32_t)T;
    return tile_owner(t, T, grid);
}

// What a CTA knows of its range.
struct PagedSched {
    int64_t T, t_begin, t_end;  // units of all items; this CTA's range
    int64_t off_b;              // unit offset of request b
    int b;                      // request of the range's first unit
    int grid;                   // CTAs with work
    int abort;
    int last;                   // this CTA arrived last at the item
};

// The parts of a split item: its tiles' owners are CTAs lo .. lo + n - 1 (a
// range holds at least two units, so each owns one of its tiles). A CTA keeps
// one partial without the item's first tile (slot 0: of the item its range
// begins in) and one with it (slot 1: of the item its end cuts), so the first
// part lies in slot 1 and the others in slot 0.
struct PagedParts {
    int64_t lo;
    int n;
    // off: unit of the item's first tile
    __device__ __forceinline__ PagedParts(const PagedSched &w, int64_t off, int tiles, int us) {
        lo = unit_owner(off, w.T, w.grid);
        n = (int)(unit_owner(off + ((int64_t)(tiles - 1) << us), w.T, w.grid) - lo) + 1;
    }
};

// A CTA's place in its range: one item (segment) after the other.
struct PagedWalk {
    PagedSeq s;
    int b, kv, rb, local, tiles;  // tile `local` of the item's `tiles`
    int us;                       // log2 of the units of its tiles
    int64_t off, end;             // unit of the item's first tile; end of the range
    // False when the range holds no tile.
    __device__ __forceinline__ bool init(const PagedWorkParams &p, const PagedSched &w) {
        b = w.b;
        s.load(p, b);
        const int64_t head = head_units(s, p), rel = w.t_begin - w.off_b;
        kv = w.T < kSmallUnits ? (int)((uint32_t)rel / (uint32_t)head) : (int)(rel / head);
        const int64_t in_head = rel - kv * head;
        int lo = 0, hi = ((s.m - 1) >> p.tbs) + 1;  // the last block that begins at or before in_head
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (units_before(s, mid, p) <= in_head) lo = mid; else hi = mid;
        }
        rb = lo;
        us = unit_shift(s, rb, p);
        tiles = block_tiles(s, rb, p.tbs);
        off = w.off_b + kv * head + units_before(s, rb, p) + (p.extra << us);
        end = w.t_end;
        const int64_t past = w.t_begin - off;
        local = past <= 0 ? 0 : (int)((past + us) >> us);  // a tile begun in the last range is not this one's
        if (local >= tiles) return advance(p);
        return seg_len() > 0;
    }
    // Tiles of the item in this range, from `local` on.
    __device__ __forceinline__ int seg_len() const {
        const int64_t n = (end - off + us) >> us;
        return (int)(n < tiles ? n : tiles) - local;
    }
    __device__ __forceinline__ bool whole() const { return local == 0 && seg_len() == tiles; }
    __device__ __forceinline__ int slot() const { return local == 0 ? 1 : 0; }  // of its partial
    // To the next item with a tile in the range; false when there is none.
    __device__ __forceinline__ bool advance(const PagedWorkParams &p) {
        off += (int64_t)tiles << us;
        local = 0;
        do {
            if (((int64_t)(rb + 1) << p.tbs) < s.m) {
                ++rb;
            } else {
                rb = 0;
                if (++kv == p.Hkv) {
                    kv = 0;
                    do {
                        if (++b >= p.B) return false;
                        s.load(p, b);
                    } while (s.m <= 0 || s.start + s.m <= 0);
                }
            }
            tiles = block_tiles(s, rb, p.tbs);
        } while (tiles == 0);
        us = unit_shift(s, rb, p);
        off += p.extra << us;
        return off < end;
    }
};

// Threads 0 .. 255 (whole CTA must call; it has __syncthreads): the units of
// all items, and the request that holds the range's first unit. scratch: 12
// words of 64 bits. min_units: every CTA with work has at least this many.
// merge > 0: few long items are not cut into the smallest parts. n parts of u
// units each take u units' time, then n times a partial's reading by the CTA
// that merges them, so of an item of U units the best u is near the root of U
// times a part's cost in units (256 rows: 2 merge, 128 rows: 3/4 merge). A
// 104-token chunk of a 7K context on one KV head took 61 us in parts of one tile.
__device__ __forceinline__ void paged_schedule(const PagedWorkParams &p, PagedSched *sched, int64_t *scratch, int min_units,
                                               int merge) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.B + 255) / 256;
    int64_t mine = 0, incl = 0;
    int b0 = 0, b1 = 0;
    int *longest_s = reinterpret_cast<int *>(scratch + 8);
    if (tid < 256) {
        int longest = 0;  // of a request's items: units times four times a part's cost, over merge
        b0 = min(tid * per, p.B);
        b1 = min(b0 + per, p.B);
        for (int b = b0; b < b1; ++b) {
            PagedSeq s;
            s.load(p, b);
            mine += p.Hkv * head_units(s, p);
            if (merge > 0 && s.m > 0) {
                for (int rb = (s.m - 1) >> p.tbs, k = 0; rb >= 0 && k < 2; --rb, ++k) {  // the last block, and the last whole one
                    const int us = unit_shift(s, rb, p);
                    longest = max(longest, (int)min(item_units(block_tiles(s, rb, p.tbs), us, p), (int64_t)(1 << 24)) * (us ? 8 : 3));
                }
            }
        }
        if (merge > 0) {
            longest = (int)__reduce_max_sync(0xffffffffu, (unsigned)longest);
            if (lane == 0) longest_s[warp] = longest;
        }
        incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) scratch[warp] = incl;
    }
    __syncthreads();
    if (tid < 256) {
        int64_t total = 0, base = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            if (w < warp) base += scratch[w];
            total += scratch[w];
        }
        if (merge > 0) {
            int longest = 0;
#pragma unroll
            for (int w = 0; w < 8; ++w) longest = max(longest, longest_s[w]);
            min_units = max(min_units, (int)sqrtf((float)longest * (float)merge * 0.25f));
        }
        const int64_t most = total < kSmallUnits ? (int64_t)((uint32_t)total / (uint32_t)min_units) : total / min_units;
        const int grid = most < (int64_t)gridDim.x ? (most > 0 ? (int)most : 1) : (int)gridDim.x;
        int64_t tb = 0, te = 0;
        if (total > 0 && (int)blockIdx.x < grid) {
            tb = unit_begin(blockIdx.x, total, grid);
            te = unit_begin(blockIdx.x + 1, total, grid);
        }
        int64_t off = base + incl - mine;
        if (tid == 0) {
            sched->T = total;
            sched->grid = grid;
            sched->t_begin = tb;
            sched->t_end = te;
            sched->abort = 0;
            sched->last = 0;
        }
        if (tb < te && off <= tb && tb < off + mine) {  // one thread's requests hold unit tb
            for (int b = b0; b < b1; ++b) {
                int64_t n = mine;
                if (per > 1) {
                    PagedSeq s;
                    s.load(p, b);
                    n = p.Hkv * head_units(s, p);
                }
                if (tb < off + n) {
                    sched->b = b;
                    sched->off_b = off;
                    break;
                }
                off += n;
            }
        }
    }
    __syncthreads();
}

// Threads 0 .. nthreads-1: flags of bad lengths, and zeros for the tokens that
// have nothing to attend to (their items have no tile). Request b is CTA
// b % gridDim.x's. row_words: 16-byte words of a token's output (Hq * D * 2 / 16).
__device__ __forceinline__ void paged_zero_rows(const PagedWorkParams &p, uint4 *out, int row_words, int *status, int nthreads) {
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        PagedSeq s;
        s.load(p, b);
        if (threadIdx.x == 0 && s.flags) raise_flag(status, s.flags);
        if (s.start >= 0) continue;
        const int64_t n = (int64_t)min(s.m, -s.start) * row_words;
        uint4 *o = out + (int64_t)s.q0 * row_words;
        for (int64_t e = threadIdx.x; e < n; e += nthreads) o[e] = make_uint4(0u, 0u, 0u, 0u);
    }
}

}  // namespace gqaq
