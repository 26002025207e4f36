// tq_paged.cuh -- definitions shared by the translation units of the paged
// 4-bit cache: the handle, the packed format, the description of an
// attention call and the division of its work among CTAs.
//
// Format of a head vector of d channels (4.25 bits per value):
//   groups of 32 channels; a group's scale s is one byte, the upper eight of
//   the fifteen magnitude bits of a binary16 number (five exponent bits, three
//   mantissa bits): the smallest such number with max|x| <= 7.5 s, at most
//   7680.  A value is the code c = sign(x) floor(|x|/s + 1/2), held to
//   [-8, 7], stored as c + 8, and stands for c s.  So |x - c s| <= s/2 below
//   the cap, and c s (three bits times four) is exact in binary16, bfloat16
//   and float32: no later step rounds a stored value again.
// A page of one kv head: [page_size][d/2] code bytes (channel j in nibble
// j % 2 of byte j / 2), then [page_size][d/32] scale bytes.
#pragma once

#include <algorithm>
#include <atomic>

#include "tq_internal.cuh"

#define TQ_FLAG_INDEX 2u   // a slot, page number, length or query start was out of range

struct tq_paged {
    int d, page, device;
    unsigned long long *d_status;   // [2]: non-finite rows, error flags
};

constexpr int PG_GROUP = 32;             // channels of one scale
constexpr uint32_t PG_MAX_SCALE = 223;   // byte of 7680, so that 8 s is finite in binary16

// Everything an attention kernel needs to know about a call.
struct PagedAttn {
    const uint8_t *kc, *vc;
    int64_t n_pages, page_bytes;     // bytes of a page of one kv head
    int lg_page, Hkv, G, batch, total_q;
    const void *q;
    void *out;
    int64_t sqt, sqh, sot, soh;      // element strides of q and out: token, head
    int bf16;                        // type of q and out: 1 bfloat16, 0 binary16
    const int *table;
    int64_t table_stride;
    int max_tokens;                  // pages of a table row times the page size
    const int *lens, *starts;        // starts may be NULL: one query per sequence
    int window, sinks;
    float scale_log2;                // softmax scale times log2(e)
    float *part;                     // split partials: [2 * grid][rows (d + 2)]
    void *rec;                       // [grid] tqpaged::Joint
    unsigned long long *status;
    int item_cost;                   // what beginning an item costs, in units of its tiles
    int whole_tokens;                // items of at most so many tokens are not cut (by the kernel)
    int whole;                       // none is cut: nothing to join, no workspace
    int even;                        // and there are no more items than CTAs: each counts as one, and has its own
    int device;
    uint64_t inv_G;                  // ceil(2^64 / G), for rows / G (unused at G = 1)
    int out32;                       // rows of `out` start on 32-byte boundaries
};

namespace tqpaged {

// One sequence's queries and cached tokens, held to the buffers' bounds.
struct Seq {
    int q0, n, len;
};

__device__ __forceinline__ Seq load_seq(const PagedAttn &P, int b, bool &bad) {
    Seq s;
    int q0 = b, q1 = b + 1;
    if (P.starts) {
        q0 = P.starts[b];
        q1 = P.starts[b + 1];
    }
    int len = P.lens[b];
    bad |= q0 < 0 || q0 > P.total_q || q1 < q0 || q1 > P.total_q || len < 0 || len > P.max_tokens;
    s.q0 = min(max(q0, 0), P.total_q);
    s.n = min(max(q1, s.q0), P.total_q) - s.q0;
    s.len = min(max(len, 0), P.max_tokens);
    return s;
}

// row / G.  The reciprocal is at most G too large in 2^64, so the product's
// upper half is exact for every 32-bit row.
__device__ __forceinline__ int token_of(const PagedAttn &P, int row) {
    return P.G == 1 ? row : (int)__umul64hi((uint64_t)(uint32_t)row, P.inv_G);
}

// The tiles of TT tokens that the queries of one chunk of rows see: the
// sinks' tiles [0, ts), then the window's [tw, te).  A chunk that sees
// nothing has one tile, all of it masked, so that its rows are written.
struct Tiles {
    int ts, tw, n;
    int p_lo, p_hi;   // positions of the first and last query
};

template <int TT>
__device__ __forceinline__ Tiles chunk_tiles(const PagedAttn &P, const Seq &s, int row0, int row1) {
    Tiles t;
    const int base = s.len - s.n;
    t.p_lo = base + token_of(P, row0);
    t.p_hi = base + token_of(P, row1 - 1);
    const int hi = max(t.p_hi + 1, 0);
    int lo = 0, s_end = 0;
    if (P.window > 0) {
        lo = max(t.p_lo - P.window + 1, 0);
        s_end = min(min(P.sinks, lo), hi);
    }
    t.ts = (s_end + TT - 1) / TT;
    t.tw = max(lo / TT, t.ts);
    t.n = max(t.ts + max((hi + TT - 1) / TT - t.tw, 0), 1);
    return t;
}

// Whether some query of the chunk sees a token of [tok, tok + n): the windows of
// consecutive positions leave no gap.  Pages of other tokens are not looked up:
// a serving loop may have given them back.
__device__ __forceinline__ bool any_seen(const PagedAttn &P, const Tiles &t, int tok, int n) {
    return tok <= t.p_hi && (P.window <= 0 || tok + n - 1 > t.p_lo - P.window || tok < P.sinks);
}

__device__ __forceinline__ int tile_token(const Tiles &t, int i, int TT) {
    return (i < t.ts ? i : t.tw + (i - t.ts)) * TT;
}

// Chunks of R rows of one kv head of a sequence, and what one costs, in units
// of as many tiles as the kernel takes at a time.
template <int R>
__device__ __forceinline__ int chunks_of(const PagedAttn &P, const Seq &s) {
    return (int)(((long long)s.n * P.G + R - 1) / R);
}
template <int R, int TT, int UNIT>
__device__ __forceinline__ int units_of(const PagedAttn &P, const Seq &s, int chunk) {
    if (P.even) return 1;
    const int row0 = chunk * R;
    return (chunk_tiles<TT>(P, s, row0, min(s.n * P.G, row0 + R)).n + UNIT - 1) / UNIT + P.item_cost;
}

// This CTA's share of the call's work, counted in units sequence by sequence,
// kv head by kv head, chunk by chunk: [lo, hi) of the whole, and where `lo`
// falls.  Every CTA takes the same, so a batch of unlike lengths fills the
// GPU evenly; a chunk cut by a share's border is joined afterwards.  A chunk
// counts its units and, before them, item_cost for its queries and outputs: a
// border that falls there cuts nothing.  Where items stay whole, one belongs to
// the share in which it begins; where they are no more than the CTAs, each
// counts as one, since by their tiles two could begin in one share while
// another CTA had none (one prompt of 128 tokens, 32 query heads on 8, d =
// 128: 21.4 us; a decode step over 8 x 64..512 tokens, the same heads, d =
// 256: 17.6 us; 14.2 and 13.3 so).
struct Share {
    long long lo, hi, quota;
    int b;              // sequence in which lo falls
    long long into;     // units of that sequence before lo
    long long per_head; // units of one kv head of that sequence
};

// A thread counts a sequence of few chunks by itself; one of many is counted
// by its warp.  Call with whole warps.
template <int R, int TT, int UNIT>
__device__ __forceinline__ long long head_units(const PagedAttn &P, const Seq &s) {
    constexpr int FEW = 4;
    const int lane = threadIdx.x & 31, chunks = chunks_of<R>(P, s);
    long long sum = 0;
    if (chunks <= FEW)
        for (int c = 0; c < chunks; ++c) sum += units_of<R, TT, UNIT>(P, s, c);
    for (uint32_t many = __ballot_sync(0xffffffffu, chunks > FEW); many; many &= many - 1) {
        const int from = __ffs(many) - 1;
        const Seq t{0, __shfl_sync(0xffffffffu, s.n, from), __shfl_sync(0xffffffffu, s.len, from)};
        const int all = chunks_of<R>(P, t);
        long long part = 0;
        for (int c = lane; c < all; c += 32) part += units_of<R, TT, UNIT>(P, t, c);
#pragma unroll
        for (int o = 16; o; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
        if (lane == from) sum = part;
    }
    return sum;
}

template <int R, int TT, int UNIT, int THREADS>
__device__ __forceinline__ Share find_share(const PagedAttn &P, Share *s_share, long long *s_sum) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (P.batch + THREADS - 1) / THREADS, b0 = tid * per;
    bool bad = false;
    long long mine = 0, head = 0;
    for (int i = 0; i < per; ++i) {   // whole warps take the same number of turns
        const Seq s = b0 + i < P.batch ? load_seq(P, b0 + i, bad) : Seq{0, 0, 0};
        head = head_units<R, TT, UNIT>(P, s);
        mine += head * P.Hkv;
    }
    if (bad) atomicOr(reinterpret_cast<unsigned int *>(P.status + 1), TQ_FLAG_INDEX);
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) s_sum[warp] = inc;
    __syncthreads();
    long long before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += s_sum[w];
        total += s_sum[w];
    }
    const long long first = before + inc - mine;
    long long quota;
    if (total >> 32) quota = (total + gridDim.x - 1) / gridDim.x;
    else quota = ((uint32_t)total + gridDim.x - 1) / gridDim.x;
    quota = max(quota, 1ll);
    const long long lo = min(quota * blockIdx.x, total), hi = min(lo + quota, total);
    const bool here = lo < hi && lo >= first && lo < first + mine;
    if (per == 1) {
        if (here) *s_share = Share{lo, hi, quota, b0, lo - first, head};
    } else if (__any_sync(0xffffffffu, here)) {
        long long at = first;
        bool found = false;
        for (int i = 0; i < per; ++i) {
            const Seq s = b0 + i < P.batch ? load_seq(P, b0 + i, bad) : Seq{0, 0, 0};
            head = head_units<R, TT, UNIT>(P, s);
            if (here && !found && lo < at + head * P.Hkv) {
                *s_share = Share{lo, hi, quota, b0 + i, lo - at, head};
                found = true;
            }
            at += head * P.Hkv;
        }
    }
    __syncthreads();
    if (lo >= hi) return Share{lo, hi, quota, 0, 0, 1};
    return *s_share;
}

// A CTA's note for the joining kernel: the item that it took over from the
// CTA before it, if any.
struct Joint {
    int row0, rows, first, last;   // rows <= 0: none; CTAs that hold parts of it
    long long q0, h;               // its sequence's first query row, its kv head
};

// The items (chunk of R rows of one kv head of one sequence) that a share
// reaches, one after another, and the tiles [i0, i1) of each that are its.
// Whole warps call begin().
template <int R, int TT, int UNIT>
struct Walk {
    Seq s;
    Tiles tl;
    int b, h, row0, row1, i0, i1, units;
    long long at, hi;   // work done, end of the share
    int span;           // work of this item in the share
    long long start;    // where the item's work begins

    __device__ __forceinline__ void begin(const PagedAttn &P, const Share &sh) {
        bool bad = false;
        b = sh.b;
        s = load_seq(P, b, bad);
        at = sh.lo;
        hi = sh.hi;
        long long into = sh.into;
        h = (into | sh.per_head) >> 32 ? (int)(into / sh.per_head) : (int)((uint32_t)into / (uint32_t)sh.per_head);
        into -= h * sh.per_head;
        // the chunk in which the share begins, 32 at a time
        const int lane = threadIdx.x & 31, chunks = chunks_of<R>(P, s);
        int c0 = 0;
        for (; chunks > 1; c0 += 32) {
            const int mine = c0 + lane < chunks ? units_of<R, TT, UNIT>(P, s, c0 + lane) : 0;
            long long sum = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long v = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += v;
            }
            const uint32_t past = __ballot_sync(0xffffffffu, into < sum);
            if (past || c0 + 32 >= chunks) {
                const int at_lane = past ? __ffs(past) - 1 : 31;
                into -= __shfl_sync(0xffffffffu, sum - mine, at_lane);
                c0 += at_lane;
                break;
            }
            into -= __shfl_sync(0xffffffffu, sum, 31);
        }
        row0 = c0 * R;
        item(P, (int)into);
        if (P.whole && into > 0) next(P);   // the share before has it
    }
    __device__ __forceinline__ bool more() const { return at < hi; }
    __device__ __forceinline__ void item(const PagedAttn &P, int into) {
        row1 = min(s.n * P.G, row0 + R);
        tl = chunk_tiles<TT>(P, s, row0, row1);
        units = (tl.n + UNIT - 1) / UNIT;
        if (P.whole) {
            span = (P.even ? 1 : units + P.item_cost) - into;
            i0 = 0;
            i1 = tl.n;
            return;
        }
        span = (int)min((long long)(units + P.item_cost - into), hi - at);
        const int u0 = max(into - P.item_cost, 0), u1 = max(into + span - P.item_cost, 0);
        i0 = u0 * UNIT;
        i1 = min(u1 * UNIT, tl.n);
        start = at - into;
        if (u1 == u0) at = hi;   // the border falls before its first tile: the next CTA's
    }
    __device__ __forceinline__ void next(const PagedAttn &P) {
        at += span;
        if (at >= hi) return;
        row0 += R;
        if (row0 >= s.n * P.G) {
            row0 = 0;
            if (++h == P.Hkv) {
                h = 0;
                bool bad = false;
                do s = load_seq(P, ++b, bad);
                while (s.n == 0 && b < P.batch - 1);
            }
        }
        item(P, 0);
    }
    __device__ __forceinline__ bool begins() const { return i0 == 0; }
    __device__ __forceinline__ bool ends() const { return i1 == tl.n; }
    // the note on this share's first item
    __device__ __forceinline__ Joint joint(const PagedAttn &P, const Share &sh) const {
        const long long first = start + P.item_cost;   // where its first tile counts
        return Joint{row0, !more() || begins() ? 0 : row1 - row0, (int)(first / sh.quota), (int)((first + units - 1) / sh.quota), s.q0, h};
    }
};

// Copies of the codes and scales of TILES tiles, made by one warp: a lane
// looks after a part of a tile (a page, or what of a page is in the tile).
template <int D, int TT, int TILES>
struct TileLoad {
    static constexpr int SIDE = TT * (D / 2 + D / 32);   // keys, then values: each part's codes, then its scales
    static constexpr int TILE = 2 * SIDE, STAGE = TILES * TILE;
    static_assert(TILES * TT / 16 <= 32, "a lane for each part");

    int lg, parts, tile, part;   // tokens of a part (log2), parts of a tile; this lane's

    __device__ __forceinline__ TileLoad(const PagedAttn &P, int lane) {
        lg = min(P.lg_page, TT == 64 ? 6 : 5);
        parts = TT >> lg;
        tile = lane / parts;
        part = lane % parts;
    }
    // the token at which this lane's part begins, tiles from i on of [.., i1);
    // -1 for none, or where no query of the chunk sees it
    __device__ __forceinline__ int token(const PagedAttn &P, const Tiles &t, int i, int i1) const {
        const int tok = tile_token(t, i + tile, TT) + (part << lg);
        return tile < TILES && i + tile < i1 && any_seen(P, t, tok, 1 << lg) ? tok : -1;
    }
    static __device__ __forceinline__ int fetch(const PagedAttn &P, int b, int tok) {
        return tok < 0 ? -1 : __ldg(P.table + (int64_t)b * P.table_stride + (tok >> P.lg_page));
    }
    // Requests the tiles into `dst`, their parts that are there into *valid
    // (a bit each, tile by tile) before that; note(those) by whole warps.
    template <typename Note>
    __device__ __forceinline__ void request(const PagedAttn &P, int tok, int page, int h, int lane, uint8_t *dst,
                                            volatile uint32_t *valid, uint64_t *bar, Note note) const {
        const bool ok = tok >= 0 && page >= 0 && page < P.n_pages;
        if (tok >= 0 && !ok) atomicOr(reinterpret_cast<unsigned int *>(P.status + 1), TQ_FLAG_INDEX);
        const uint32_t got = __ballot_sync(0xffffffffu, ok);
        const uint32_t codes = (uint32_t)(D / 2) << lg, scales = (uint32_t)(D / 32) << lg;
        note(got);
        if (lane == 0) {
            *valid = got;
            tqdev::mbar_expect_tx(bar, (uint32_t)__popc(got) * 2u * (codes + scales));
        }
        __syncwarp();
        if (!ok) return;
        const int64_t src = ((int64_t)page * P.Hkv + h) * P.page_bytes;
        dst += tile * TILE + part * (codes + scales);
        if (P.lg_page == lg) {   // a whole page: codes and scales in one piece
            tqdev::bulk_load(dst, P.kc + src, codes + scales, bar);
            tqdev::bulk_load(dst + SIDE, P.vc + src, codes + scales, bar);
            return;
        }
        const int in = tok & ((1 << P.lg_page) - 1);
        const int64_t c0 = src + (int64_t)in * (D / 2);
        const int64_t s0 = src + ((int64_t)(D / 2) << P.lg_page) + (int64_t)in * (D / 32);
        tqdev::bulk_load(dst, P.kc + c0, codes, bar);
        tqdev::bulk_load(dst + codes, P.kc + s0, scales, bar);
        tqdev::bulk_load(dst + SIDE, P.vc + c0, codes, bar);
        tqdev::bulk_load(dst + SIDE + codes, P.vc + s0, scales, bar);
    }
    // byte offsets in a side of token r's codes and scales
    static __device__ __forceinline__ int codes_at(int r, int lg) { return r * (D / 2) + ((r >> lg) << lg) * (D / 32); }
    static __device__ __forceinline__ int scales_at(int r, int lg) {
        return (((r >> lg) + 1) << lg) * (D / 2) + r * (D / 32);
    }
};

__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ __half2 u2h(uint32_t u) { return *reinterpret_cast<__half2 *>(&u); }

__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t bits) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(bits));   // (w & mask) | bits
    return r;
}

// lo, hi += the two halves of h
__device__ __forceinline__ void add_halves(float &lo, float &hi, uint32_t h) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "add.rn.f32.f16 %0, a, %0;\n\tadd.rn.f32.f16 %1, b, %1;\n\t}"
        : "+f"(lo), "+f"(hi) : "r"(h));
}

// A scale as widen() takes it, two of them side by side (w: a scale byte in
// the low bits of each half).  Everything is 2^-7 of its true size: then
// 1032 s fits binary16 for every scale, and every value below is still exact,
// a multiple of 2^-24 with at most eleven bits.
struct Scale2 {
    __half2 s, m1032, m72;   // s, -1032 s, -72 s
};
constexpr float WIDE = 128.f;   // what widened values have to be multiplied by

__device__ __forceinline__ Scale2 scale2(uint32_t w) {
    const __half2 v = u2h(w << 7);
    return {__hmul2(v, __float2half2_rn(0.0078125f)), __hmul2(v, __float2half2_rn(-8.0625f)),
            __hmul2(v, __float2half2_rn(-0.5625f))};
}

// Pairs of codes in nibbles 0..3 of both halves of w, times the scales of
// the two halves: p[i] = 2^-7 ((nibble i of the low half) - 8) s.x, the same
// of the high half and s.y, exact.  A nibble is spliced into the mantissa of
// 1024 + c (at bit 0) or 64 + c (at bit 4); one fused operation takes off
// the offset and applies the scale.
__device__ __forceinline__ void widen(uint32_t w, const Scale2 &k, uint32_t (&p)[4]) {
    const uint32_t w8 = w >> 8;
    p[0] = h2u(__hfma2(u2h(and_or(w, 0x000F000Fu, 0x64006400u)), k.s, k.m1032));
    p[1] = h2u(__hfma2(u2h(and_or(w, 0x00F000F0u, 0x54005400u)), k.s, k.m72));
    p[2] = h2u(__hfma2(u2h(and_or(w8, 0x000F000Fu, 0x64006400u)), k.s, k.m1032));
    p[3] = h2u(__hfma2(u2h(and_or(w8, 0x00F000F0u, 0x54005400u)), k.s, k.m72));
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float RAISE = 8.f;   // the running maximum is raised when a score passes it by 2^8
constexpr float BIAS = 6.f;    // weights are 2^(s - m + 6): at most 2^14, and exact to 2^-20

// The factor (a power of two) that takes a bfloat16 row whose largest
// magnitude has the bits `m` into binary16, to [2^14, 2^15), and its inverse.
__device__ __forceinline__ void query_factor(uint32_t m, float &up, float &back) {
    const int e = min(max((int)(m >> 7), 15), 254);
    up = __uint_as_float((uint32_t)(268 - e) << 23);     // 2^(141 - e)
    back = __uint_as_float((uint32_t)(e - 14) << 23);    // 2^(e - 141)
}

__device__ __forceinline__ uint32_t amax4(uint4 w) {
    return __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu), __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
}

__device__ __forceinline__ uint4 bf16_to_half(uint4 w, float up) {
    uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        x[j] = h2u(__floats2half2_rn(__uint_as_float(x[j] << 16) * up, __uint_as_float(x[j] & 0xFFFF0000u) * up));
    return make_uint4(x[0], x[1], x[2], x[3]);
}

// Element offsets of row `row` of (sequence, kv head) in q and in out.
__device__ __forceinline__ int64_t query_at(const PagedAttn &P, const Seq &s, int h, int row) {
    const int tok = token_of(P, row), hg = row - tok * P.G;
    return (int64_t)(s.q0 + tok) * P.sqt + (int64_t)(h * P.G + hg) * P.sqh;
}
__device__ __forceinline__ int64_t out_at(const PagedAttn &P, const Seq &s, int h, int row) {
    const int tok = token_of(P, row), hg = row - tok * P.G;
    return (int64_t)(s.q0 + tok) * P.sot + (int64_t)(h * P.G + hg) * P.soh;
}

__device__ __forceinline__ uint32_t out_pair(const PagedAttn &P, float a, float b) {
    if (P.bf16) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&x);
    }
    return h2u(__floats2half2_rn(a, b));
}

}  // namespace tqpaged

// Allows a kernel `bytes` of dynamic shared memory, once on each device; it
// must have been compiled to `regs` registers a thread or more (a kernel whose
// warp groups trade registers would wait for what was never there).
template <typename K>
cudaError_t tq_paged_allow(K kern, int bytes, int regs, int device, std::atomic<uint64_t> &done) {
    const uint64_t bit = device < 64 ? 1ull << device : 0;
    if (bit && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    cudaFuncAttributes a;
    cudaError_t e = cudaFuncGetAttributes(&a, kern);
    if (e == cudaSuccess && a.numRegs < regs) e = cudaErrorLaunchOutOfResources;
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// CTAs of a call of at most `items` items of at most `units` units, and its
// workspace: notes for the joining kernel, and two parts of R rows a CTA.
struct PagedGrid {
    int ctas;
    size_t notes, bytes;
};

inline PagedGrid tq_paged_grid(PagedAttn &P, int64_t items, int64_t units, int most_ctas, int R, int D) {
    P.whole = P.max_tokens <= P.whole_tokens;
    P.even = P.whole && items <= most_ctas;
    const int64_t bound = P.whole || items >= most_ctas ? items : items * units;   // (at the limits the product passes 2^63)
    PagedGrid g{(int)std::max<int64_t>(1, std::min<int64_t>(most_ctas, bound)), 0, 0};
    if (g.ctas == 1) P.whole = 1;
    if (P.whole) return g;
    g.notes = ((size_t)g.ctas * sizeof(tqpaged::Joint) + 255) / 256 * 256;
    g.bytes = g.notes + (size_t)g.ctas * 2 * R * (D + 2) * sizeof(float);
    P.rec = P.part;
    if (P.part) P.part = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(P.part) + g.notes);
    return g;
}

// Kernels of a call: for few rows (queries times heads of a group) of each kv
// head, and for many; `need` non-null asks for the workspace's bytes only.
tq_status tq_launch_paged_prefill(int d, const PagedAttn &P, int max_q_len, int n_sms, cudaStream_t stream, size_t *need);
tq_status tq_launch_paged_join(int d, const PagedAttn &P, int grid, int rows, cudaStream_t stream);
tq_status tq_launch_paged_attention(const tq_paged *ctx, const PagedAttn &P, int max_q_len, int n_sms,
                                    cudaStream_t stream, size_t *need);
