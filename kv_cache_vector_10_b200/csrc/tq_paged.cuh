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
    int4 *rec;                       // [grid]: the split item that begins in this CTA
    unsigned long long *status;
    int min_tiles;                   // least tiles a CTA takes
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
    t.p_lo = base + row0 / P.G;
    t.p_hi = base + (row1 - 1) / P.G;
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

__device__ __forceinline__ int tile_token(const Tiles &t, int i, int TT) {
    return (i < t.ts ? i : t.tw + (i - t.ts)) * TT;
}

// Tiles of one kv head of a sequence, over its chunks of R rows.
template <int R, int TT>
__device__ __forceinline__ long long head_tiles(const PagedAttn &P, const Seq &s) {
    long long sum = 0;
    const long long rows = (long long)s.n * P.G;
    for (long long r = 0; r < rows; r += R)
        sum += chunk_tiles<TT>(P, s, (int)r, (int)min(rows, r + R)).n;
    return sum;
}

// This CTA's share of the call's tiles, counted sequence by sequence, kv head
// by kv head, chunk by chunk: [lo, hi) of the whole, and where `lo` falls.
// Every CTA takes the same number, so a batch of unlike lengths fills the
// GPU evenly; a chunk cut by a share's border is joined afterwards.
struct Share {
    long long lo, hi, quota;
    int b;             // sequence in which lo falls
    long long into;    // tiles of that sequence before lo
};

template <int R, int TT, int THREADS>
__device__ __forceinline__ Share find_share(const PagedAttn &P, Share *s_share, long long *s_sum) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (P.batch + THREADS - 1) / THREADS;
    const int b0 = min(tid * per, P.batch), b1 = min(b0 + per, P.batch);
    bool bad = false;
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += head_tiles<R, TT>(P, load_seq(P, b, bad)) * P.Hkv;
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
    long long quota = (total + gridDim.x - 1) / gridDim.x;
    quota = max(quota, (long long)P.min_tiles);
    const long long lo = min(quota * blockIdx.x, total), hi = min(lo + quota, total);
    if (tid == 0) *s_share = Share{lo, hi, quota, P.batch, 0};
    __syncthreads();
    if (lo < hi && mine > 0 && lo >= first && lo < first + mine) {
        long long at = first;
        for (int b = b0; b < b1; ++b) {
            const long long t = head_tiles<R, TT>(P, load_seq(P, b, bad)) * P.Hkv;
            if (lo < at + t) {
                *s_share = Share{lo, hi, quota, b, lo - at};
                break;
            }
            at += t;
        }
    }
    __syncthreads();
    return *s_share;
}

}  // namespace tqpaged

tq_status tq_launch_paged_attention(const tq_paged *ctx, const PagedAttn &P, int max_q_len, int n_sms,
                                    cudaStream_t stream, size_t *need);
