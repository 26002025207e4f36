// tq_paged_attend.cu -- attention over the paged 4-bit cache for few queries
// a sequence: decode steps, drafted tokens.
//
//   s_t = q . k_t / sqrt(d),  o = sum_t softmax(s)_t v_t  over the visible t:
//   t <= p, and, under a window W with S sinks, t > p - W or t < S,
// where p is the query's position and k_t, v_t are what the codes stand for.
//
// What bounds it: a token of one kv head is 17 d / 16 bytes (136 at d = 128)
// and is used by few rows (queries times query heads of the group), so the
// floor is the time to read the visible tokens.  At HBM rate an SM has about
// 94 cycles for 16 tokens, that is some 370 warp instructions to turn 4096
// codes into operands, multiply and take the softmax; it takes about 285,
// issued at 0.6 a cycle and scheduler whether 8 or 12 warps are on an SM (the
// integer pipe, which splices the codes, is the busiest, at 40%).  So each
// further 2^21 tokens of a kv head take 56 us at d = 128 (285 MB, 78% of the
// copy rate; d = 64: 37 us, 59%; d = 256: 119 us, 73%).  The line through
// calls of 2^18 to 2^21 tokens meets none at 13 us (d = 256: 19): a call of
// one round an item takes 9.4 us (start, shares, the first tiles' way from
// memory, the last's way through the warps, the join), and the rest of the
// line's start has not been taken apart.  4 sequences of 32768 tokens, 8 kv
// heads, 32 query heads, d = 128 (143 MB): 41 us, 53% of the copy rate; one
// sequence of 1024 tokens and one kv head, not split: 10.3 us.  Hence:
//   * codes go from shared memory into registers as the fragments of
//     mma.m16n8k16 (tokens or channels as the 16 rows, queries as the 8
//     columns) and are widened there: no operand is written back to shared
//     memory, which tcgen05 would need (64 KB for 128 tokens, more than the
//     shared-memory bandwidth allows at this rate);
//   * a lane takes consecutive code words, and the contraction runs over the
//     channels in the order that this gives; the query's fragments are built
//     in the same order;
//   * code pairs are spliced into the mantissa of 1024 + c or 64 + c and
//     brought to c s by one packed operation, exactly;
//   * one warp of a CTA requests the codes, a tile for each of the four that
//     compute, by bulk copies of whole (parts of) pages, and runs ahead of
//     them across items; those four meet only where an item ends;
//   * every CTA has the same share of all tiles, whatever the sequences'
//     lengths; an item cut by a share's border is joined by a second kernel.
//     Where all are short, none is cut and there is no second kernel.
// The probabilities are rounded to binary16 (error 2^-12 of each weight,
// half a rounding step of a binary16 output) and divided by the sum of what
// they are rounded to, at no cost in time (the sum of the unrounded ones: 1.55
// times the error of an unrounded softmax with binary16 outputs where one
// token outweighs the others, instead of 1.2; by a product with ones: 2%
// slower); queries are taken to binary16
// after a power-of-two scaling by their largest channel (bfloat16; exact
// unless a channel is below 2^-28 of the largest), keys and values are exact
// in binary16, and scores, maxima, sums and outputs are float32.
#include <algorithm>

#include "tq_paged.cuh"

namespace {

using namespace tqpaged;

constexpr int NW = 4;                  // warps of a CTA that compute; one more requests the codes
constexpr int THREADS = 32 * (NW + 1);

template <int D, int NT>
struct Cfg {
    static constexpr int TT = D == 256 ? 32 : 64;              // tokens of a tile
    static constexpr int NST = D == 64 ? 3 : 2;                // stages: a tile for each warp
    // CTAs of an SM: as many as the registers of the fragments allow (a third
    // one at d = 128, NT = 1 takes 48 us instead of 43.5 for 4 x 32768 tokens
    // and 22.1 instead of 20.0 for 4 x 8192).  d = 128, NT = 1 spills none of
    // them; the others do (stores and loads in bytes: d = 64, NT = 1 36 and 44,
    // NT = 2 288 and 372; d = 128, NT = 2 492 and 564; d = 256 204 and 276).
    static constexpr int CTAS = D == 64 ? 4 - NT / 2 : 2;
    using Load = TileLoad<D, TT, NW>;
    static constexpr int SMEM = NST * Load::STAGE;
};

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// WORDS consecutive 32-bit words of shared memory.
template <int WORDS>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t (&w)[WORDS]) {
    if constexpr (WORDS == 1) {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else if constexpr (WORDS == 2) {
        const uint2 x = *reinterpret_cast<const uint2 *>(p);
        w[0] = x.x, w[1] = x.y;
    } else {
#pragma unroll
        for (int i = 0; i < WORDS; i += 4) {
            const uint4 x = *reinterpret_cast<const uint4 *>(p + 4 * i);
            w[i] = x.x, w[i + 1] = x.y, w[i + 2] = x.z, w[i + 3] = x.w;
        }
    }
}

// The query fragments of an item's rows.  Lane (g, t) holds row 8 nt + g,
// channels [t D/4, (t + 1) D/4), in pairs (e, e + 4) of each eight: the order
// in which widen() gives the codes.  `mul[nt][c]` is what turns the product
// of column 2 t + c into a score in units of log2.
template <int D, int NT>
__device__ __forceinline__ void load_queries(const PagedAttn &P, const Seq &s, int h, int row0, int row1, int lane,
                                             uint32_t (&q)[NT][D / 8], float (&mul)[NT][2]) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int row = row0 + 8 * nt + g;
        uint4 w[D / 32];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) w[i] = make_uint4(0, 0, 0, 0);
        if (row < row1) {
            const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(P.q) + query_at(P, s, h, row) + t * (D / 4));
#pragma unroll
            for (int i = 0; i < D / 32; ++i) w[i] = __ldg(src + i);
        }
        float back = 1.f;
        if (P.bf16) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) m = __vmaxu2(m, amax4(w[i]));
            m = max(m >> 16, m & 0xFFFFu);
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
            float up;
            query_factor(m, up, back);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) w[i] = bf16_to_half(w[i], up);
        }
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {   // elements 0..7 of a word: pairs (0,4) (1,5) (2,6) (3,7)
            q[nt][4 * i + 0] = __byte_perm(w[i].x, w[i].z, 0x5410);
            q[nt][4 * i + 1] = __byte_perm(w[i].x, w[i].z, 0x7632);
            q[nt][4 * i + 2] = __byte_perm(w[i].y, w[i].w, 0x5410);
            q[nt][4 * i + 3] = __byte_perm(w[i].y, w[i].w, 0x7632);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) mul[nt][c] = __shfl_sync(0xffffffffu, back, (2 * t + c) * 4) * (P.scale_log2 * WIDE);
    }
}

__device__ __forceinline__ void store_out4(const PagedAttn &P, int64_t at, float4 v) {
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(P.out) + at) = make_uint2(out_pair(P, v.x, v.y), out_pair(P, v.z, v.w));
}

template <int D, int NT>
__global__ void __launch_bounds__(THREADS, Cfg<D, NT>::CTAS) tq_paged_decode_kernel(const __grid_constant__ PagedAttn P) {
    using C = Cfg<D, NT>;
    constexpr int TT = C::TT, NST = C::NST, R = 8 * NT, KW = D / 32, VW = D / 64, SUB = TT / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t full[NST], freed[NST];
    __shared__ uint32_t s_valid[NST];
    __shared__ float s_m[2][NW][R], s_l[2][NW][R];   // by the item's parity: a warp may be one item ahead
    __shared__ Share s_share;
    __shared__ long long s_sum[NW + 1];
    __shared__ int s_abort;
    static_assert(NW * R * D * 4 <= C::Load::STAGE, "a stage holds the warps' parts of an item");

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    tqdev::grid_dep_wait();
    if (tid == 0) {
        s_abort = tqdev::status_aborted(P.status) ? 1 : 0;
        for (int i = 0; i < NST; ++i) {
            tqdev::mbar_init(&full[i], 1);
            tqdev::mbar_init(&freed[i], NW);
        }
        tqdev::fence_barrier_init();
    }
    tqdev::grid_dep_trigger();
    const Share sh = find_share<R, TT, NW, THREADS>(P, &s_share, s_sum);
    if (s_abort || sh.lo >= sh.hi) {
        if (tid == 0 && !P.whole) static_cast<Joint *>(P.rec)[blockIdx.x].rows = 0;
        return;
    }
    bool failed = false;
    Walk<R, TT, NW> it;
    it.begin(P, sh);
    if (warp == NW) {
        // --------------------------------------------- requests, items ahead
        if (lane == 0 && !P.whole) static_cast<Joint *>(P.rec)[blockIdx.x] = it.joint(P, sh);
        const typename C::Load load(P, lane);
        int n = 0;
        for (; it.more() && !failed; it.next(P)) {
            int tok = load.token(P, it.tl, it.i0, it.i1), page = C::Load::fetch(P, it.b, tok);
            for (int i = it.i0; i < it.i1; i += NW, ++n) {
                const int st = n % NST, tok2 = load.token(P, it.tl, i + NW, it.i1), page2 = C::Load::fetch(P, it.b, tok2);
                if (n >= NST && !__all_sync(0xffffffffu, tqdev::mbar_wait_bounded(&freed[st], (uint32_t)(n / NST - 1) & 1u))) {
                    failed = true;
                    break;
                }
                load.request(P, tok, page, it.h, lane, smem + st * C::Load::STAGE, &s_valid[st], &full[st], [](uint32_t) {});
                tok = tok2;
                page = page2;
            }
        }
        // whatever became of the others: the copies in flight have landed
        for (int k = max(0, n - NST); k < n; ++k) failed |= !tqdev::mbar_wait_bounded(&full[k % NST], (uint32_t)(k / NST) & 1u);
        if (failed) atomicOr(reinterpret_cast<unsigned int *>(P.status + 1), TQ_FLAG_WAIT_TIMEOUT);
        return;
    }

    int n = 0;                        // stages consumed, over all items
    for (int items = 0; it.more(); it.next(P), ++items) {
        const Seq &s = it.s;
        const Tiles &tl = it.tl;
        const int lg_part = min(P.lg_page, TT == 64 ? 6 : 5), parts = TT >> lg_part;
        uint32_t q[NT][D / 8];
        float mul[NT][2], m_run[NT][2], l_run[NT][2], o[NT][D / 16][4];
        load_queries<D, NT>(P, s, it.h, it.row0, it.row1, lane, q, mul);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                m_run[nt][c] = -INFINITY;
                l_run[nt][c] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nt][j][e] = 0.f;
        }

        uint8_t *stage = smem;
        for (int i = it.i0; i < it.i1; i += NW, ++n) {
            const int st = n % NST;
            stage = smem + st * C::Load::STAGE;
            if (n > 0 && i > it.i0) {   // the stage before may be filled again (an item's last: after the join below)
                __syncwarp();
                if (lane == 0) tqdev::mbar_arrive(&freed[(n - 1) % NST]);
            }
            failed = failed || !__all_sync(0xffffffffu, tqdev::mbar_wait_bounded(&full[st], (uint32_t)(n / NST) & 1u));
            if (failed || i + warp >= it.i1) continue;
            uint8_t *const keys = stage + warp * C::Load::TILE, *const vals = keys + C::Load::SIDE;
            const int T0 = tile_token(tl, i + warp, TT);
            const uint32_t all = (1u << parts) - 1u;
            const uint32_t got = (*reinterpret_cast<volatile uint32_t *>(&s_valid[st]) >> (warp * parts)) & all;
            const bool whole = T0 + TT - 1 <= tl.p_lo && (P.window <= 0 || T0 > tl.p_hi - P.window || T0 + TT <= P.sinks) && got == all;

            // scores: 16 tokens a step; rows g and g + 8 of the fragment are
            // the tokens (g / 2) + 4 (g % 2) and that + 8, so that the
            // transposed weights come out in the order of the value loads
            float sc[NT][SUB][4];
            const int tok0 = (g >> 1) + 4 * (g & 1);
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                uint32_t w0[KW], w1[KW];
                const uint8_t *kc = keys + C::Load::codes_at(16 * u, lg_part), *ks = keys + C::Load::scales_at(16 * u, lg_part);
                const int ra = tok0, rb = tok0 + 8;
                load_words<KW>(kc + ra * (D / 2) + t * (D / 8), w0);
                load_words<KW>(kc + rb * (D / 2) + t * (D / 8), w1);
                constexpr int GW = D == 256 ? 4 : KW;   // words of a lane in one group
#pragma unroll
                for (int x = 0; x < KW; x += GW) {
                    const int grp = D == 64 ? t >> 1 : D == 128 ? t : 2 * t + x / 4;
                    const Scale2 s0 = scale2(ks[ra * (D / 32) + grp] * 0x00010001u);
                    const Scale2 s1 = scale2(ks[rb * (D / 32) + grp] * 0x00010001u);
#pragma unroll
                    for (int y = x; y < x + GW; ++y) {
                        uint32_t a[4], c[4];
                        widen(w0[y], s0, a);
                        widen(w1[y], s1, c);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if (y == 0) mma_first(sc[nt][u], a[0], c[0], a[1], c[1], q[nt][0], q[nt][1]);
                            else mma(sc[nt][u], a[0], c[0], a[1], c[1], q[nt][4 * y], q[nt][4 * y + 1]);
                            mma(sc[nt][u], a[2], c[2], a[3], c[3], q[nt][4 * y + 2], q[nt][4 * y + 3]);
                        }
                    }
                }
            }
            if (!whole) {
                // rows that no query of the chunk sees may hold anything: their
                // values become zeros here, in the few tiles that have such rows
                // (tested at the loads of every tile below, 4 x 32768 tokens took
                // 45.9 us instead of 42.3)
                for (int r = lane; r < TT; r += 32)
                    if (!(any_seen(P, tl, T0 + r, 1) && ((got >> (r >> lg_part)) & 1u))) {
                        uint8_t *at = vals + C::Load::scales_at(r, lg_part);
#pragma unroll
                        for (int x = 0; x < D / 32; x += 2) *reinterpret_cast<uint16_t *>(at + x) = 0;
                    }
                tqdev::fence_proxy_async_smem();   // the next copy into this stage comes after
                __syncwarp();
#pragma unroll
                for (int u = 0; u < SUB; ++u) {
                    const bool have = (got >> ((16 * u) >> lg_part)) & 1u;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int tok = T0 + 16 * u + tok0 + (e >= 2 ? 8 : 0);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const int p = s.len - s.n + token_of(P, it.row0 + 8 * nt + 2 * t + (e & 1));
                            const bool see = have && tok <= p && (P.window <= 0 || tok > p - P.window || tok < P.sinks);
                            if (!see) sc[nt][u][e] = -INFINITY;
                        }
                    }
                }
            }
            // softmax: raise the maximum only when some score passes it by RAISE
            float mx[NT][2];
            bool raise = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float m = fmaxf(sc[nt][0][c], sc[nt][0][c + 2]);
#pragma unroll
                    for (int u = 1; u < SUB; ++u) m = fmaxf(m, fmaxf(sc[nt][u][c], sc[nt][u][c + 2]));
                    mx[nt][c] = m * mul[nt][c];
                    raise |= mx[nt][c] > m_run[nt][c] + RAISE;
                }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float m = mx[nt][c];
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                        m = fmaxf(m, m_run[nt][c]);
                        const float f = m_run[nt][c] == -INFINITY ? 0.f : exp2_fast(m_run[nt][c] - m);
                        m_run[nt][c] = m;
                        l_run[nt][c] *= f;
#pragma unroll
                        for (int j = 0; j < D / 16; ++j) {
                            o[nt][j][c] *= f;
                            o[nt][j][c + 2] *= f;
                        }
                    }
            }
            uint32_t pw[NT][SUB][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float r0 = m_run[nt][0] == -INFINITY ? 0.f : m_run[nt][0] - BIAS;
                const float r1 = m_run[nt][1] == -INFINITY ? 0.f : m_run[nt][1] - BIAS;
#pragma unroll
                for (int u = 0; u < SUB; ++u) {
                    const float p0 = exp2_fast(fmaf(sc[nt][u][0], mul[nt][0], -r0)), p1 = exp2_fast(fmaf(sc[nt][u][1], mul[nt][1], -r1));
                    const float p2 = exp2_fast(fmaf(sc[nt][u][2], mul[nt][0], -r0)), p3 = exp2_fast(fmaf(sc[nt][u][3], mul[nt][1], -r1));
                    // summed as they are rounded: where few tokens carry a row,
                    // their rounding cancels
                    const uint32_t h0 = h2u(__floats2half2_rn(p0, p1)), h1 = h2u(__floats2half2_rn(p2, p3));
                    add_halves(l_run[nt][0], l_run[nt][1], h0);
                    add_halves(l_run[nt][0], l_run[nt][1], h1);
                    pw[nt][u][0] = transpose8(h0);
                    pw[nt][u][1] = transpose8(h1);
                }
            }
            // values: lane (g, t) takes channels [g D/8, (g + 1) D/8) of the
            // tokens t, t + 4, t + 8, t + 12 of each sixteen
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                const uint8_t *vc = vals + C::Load::codes_at(16 * u, lg_part), *vs = vals + C::Load::scales_at(16 * u, lg_part);
                uint32_t w[4][VW], sv[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = t + 4 * k;
                    load_words<VW>(vc + r * (D / 2) + g * (D / 16), w[k]);
                    sv[k] = vs[r * (D / 32) + (g * (D / 8)) / 32];
                }
                const Scale2 s0 = scale2(sv[0] | sv[1] << 16), s1 = scale2(sv[2] | sv[3] << 16);
#pragma unroll
                for (int y = 0; y < VW; ++y) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint32_t sel = half ? 0x7632u : 0x5410u;
                        uint32_t a[4], c[4];
                        widen(__byte_perm(w[0][y], w[1][y], sel), s0, a);
                        widen(__byte_perm(w[2][y], w[3][y], sel), s1, c);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma(o[nt][4 * y + 2 * half], a[0], a[1], c[0], c[1], pw[nt][u][0], pw[nt][u][1]);
                            mma(o[nt][4 * y + 2 * half + 1], a[2], a[3], c[2], c[3], pw[nt][u][0], pw[nt][u][1]);
                        }
                    }
                }
            }
        }

        // The warps' parts of this item, joined through the last stage used
        // (the next one is being filled meanwhile).
        float(*sm)[R] = s_m[items & 1], (*sl)[R] = s_l[items & 1];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float l = l_run[nt][c];
                l += __shfl_xor_sync(0xffffffffu, l, 4);
                l += __shfl_xor_sync(0xffffffffu, l, 8);
                l += __shfl_xor_sync(0xffffffffu, l, 16);
                if (g == 0) {
                    sm[warp][8 * nt + 2 * t + c] = m_run[nt][c];
                    sl[warp][8 * nt + 2 * t + c] = l;
                }
            }
        tqdev::named_sync(1, 32 * NW);
        float *all_parts = reinterpret_cast<float *>(stage);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int r = 8 * nt + 2 * t + c;
                float m = sm[0][r];
#pragma unroll
                for (int w = 1; w < NW; ++w) m = fmaxf(m, sm[w][r]);
                const float f = m_run[nt][c] == -INFINITY ? 0.f : exp2_fast(m_run[nt][c] - m) * WIDE;
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
                    *reinterpret_cast<float2 *>(all_parts + (warp * R + r) * D + g * (D / 8) + 8 * (j >> 2) + 2 * (j & 3)) =
                        make_float2(o[nt][j][c] * f, o[nt][j][c + 2] * f);
            }
        tqdev::named_sync(1, 32 * NW);
        const bool direct = it.begins() && it.ends();
        float *part = P.part + ((int64_t)blockIdx.x * 2 + (it.begins() ? 1 : 0)) * (R * (D + 2));
        for (int x = tid; x < R * D / 4; x += 32 * NW) {
            const int r = x / (D / 4), c4 = x % (D / 4);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float4 y = *reinterpret_cast<const float4 *>(all_parts + (w * R + r) * D + 4 * c4);
                v.x += y.x, v.y += y.y, v.z += y.z, v.w += y.w;
            }
            float m = sm[0][r], l = 0.f;
#pragma unroll
            for (int w = 1; w < NW; ++w) m = fmaxf(m, sm[w][r]);
#pragma unroll
            for (int w = 0; w < NW; ++w)   // (a part that saw nothing adds nothing; one of NaN alone has no maximum, but a sum)
                if (sm[w][r] != -INFINITY || sl[w][r] != 0.f) l += sl[w][r] * exp2_fast(sm[w][r] - m);
            if (direct) {
                if (it.row0 + r < it.row1) {
                    const float inv = l != 0.f ? 1.f / l : 0.f;
                    store_out4(P, out_at(P, s, it.h, it.row0 + r) + 4 * c4, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
                }
            } else {
                *reinterpret_cast<float4 *>(part + r * D + 4 * c4) = v;
                if (c4 == 0) {
                    part[R * D + r] = m;
                    part[R * D + R + r] = l;
                }
            }
        }
        tqdev::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tqdev::mbar_arrive(&freed[(n - 1) % NST]);
    }
    if (failed) atomicOr(reinterpret_cast<unsigned int *>(P.status + 1), TQ_FLAG_WAIT_TIMEOUT);
}

// Joins the parts of the items that were cut between CTAs.  The blocks
// (x, y) serve the item that CTA x took over from the one before; an item of
// n parts has n - 1 such x, and all their warps share its groups of four
// outputs.  A warp's lanes split a few of these and the parts, and add up in
// a fixed order.
constexpr int JOIN_WARPS = 4;

template <int D>
__global__ void __launch_bounds__(32 * JOIN_WARPS) tq_paged_join_kernel(const __grid_constant__ PagedAttn P, int R) {
    tqdev::grid_dep_wait();
    const Joint J = static_cast<const Joint *>(P.rec)[blockIdx.x];
    if (tqdev::status_aborted(P.status) || J.rows <= 0) return;
    const int lane = threadIdx.x & 31, slices = JOIN_WARPS * gridDim.y;
    const int n = J.last - J.first + 1, warps = (n - 1) * slices;
    const int me = (blockIdx.x - J.first - 1) * slices + blockIdx.y * JOIN_WARPS + (threadIdx.x >> 5);
    const int total = J.rows * (D / 4), each = (total + warps - 1) / warps;
    const int c0 = me * each, c1 = min(total, c0 + each);
    const int lg = each > 1 ? 32 - __clz(min(each, 32) - 1) : 0, groups = 32 >> lg;   // columns at once (log2), parts at once
    const int col = lane & ((1 << lg) - 1), grp = lane >> lg;
    const int64_t size = (int64_t)R * (D + 2);
    const Seq s{(int)J.q0, 0, 0};
    for (int c = c0; c < c1; c += 1 << lg) {
        const int x = min(c + col, c1 - 1), r = x / (D / 4), c4 = x % (D / 4);
        float m = -INFINITY, l = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](float mk, float lk, const float4 &y) {
            if (mk == -INFINITY && lk == 0.f) return;   // saw nothing; where all scores are NaN, l is NaN and the row becomes it
            const float to = fmaxf(m, mk), f = m == -INFINITY ? 0.f : exp2_fast(m - to), g = exp2_fast(mk - to);
            m = to;
            l = l * f + lk * g;
            v.x = v.x * f + y.x * g, v.y = v.y * f + y.y * g, v.z = v.z * f + y.z * g, v.w = v.w * f + y.w * g;
        };
        constexpr int B = 4;   // parts on their way at once
        for (int k0 = grp; k0 < n; k0 += B * groups) {
            float mk[B], lk[B];
            float4 y[B];
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const int k = k0 + b * groups;
                mk[b] = -INFINITY, lk[b] = 0.f;
                if (k < n) {
                    const float *p = P.part + ((int64_t)(J.first + k) * 2 + (k == 0 ? 1 : 0)) * size;
                    mk[b] = __ldcg(p + (int64_t)R * D + r);
                    lk[b] = __ldcg(p + (int64_t)R * D + R + r);
                    y[b] = __ldcg(reinterpret_cast<const float4 *>(p + (int64_t)r * D) + c4);
                }
            }
#pragma unroll
            for (int b = 0; b < B; ++b) add(mk[b], lk[b], y[b]);
        }
        for (int o = 16; o >= (1 << lg); o >>= 1) {
            const float mo = __shfl_xor_sync(0xffffffffu, m, o), lo = __shfl_xor_sync(0xffffffffu, l, o);
            const float4 z = make_float4(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o),
                                         __shfl_xor_sync(0xffffffffu, v.z, o), __shfl_xor_sync(0xffffffffu, v.w, o));
            add(mo, lo, z);
        }
        if (grp == 0 && c + col < c1) {
            const float inv = l != 0.f ? 1.f / l : 0.f;
            store_out4(P, out_at(P, s, (int)J.h, J.row0 + r) + 4 * c4, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
        }
    }
}

template <int D, int NT>
tq_status launch_decode(PagedAttn P, int64_t rows, int n_sms, cudaStream_t stream, size_t *need) {
    using C = Cfg<D, NT>;
    constexpr int R = 8 * NT;
    // Shares are counted in rounds of a tile for each of the four warps, since
    // a part of a round takes as long as a whole one (in single tiles: 8 x 4096
    // tokens of 32 kv heads 45.0 us instead of 43.6, drafted tokens 18.6
    // instead of 17.1, 4 x 32768 the same, but 32 windows of 1024, short
    // against a round, 23.6 instead of 24.6, and 8 x 4096 tokens at d = 256
    // 30.8 instead of 32.4).  An item's queries and the join
    // of its warps' parts take about a round (not counted: drafted tokens 18.6,
    // 4 x 32768 43.5 instead of 42.2, the others within 1%).
    P.item_cost = 1;
    // Uncut, a short item saves the second launch and the join; cut, its rounds
    // run side by side.  Kernel times in us, cut and whole, four query heads a
    // kv head, by tokens (rounds) and items (sequences times kv heads):
    //              d = 64             d = 128            d = 256
    //   rounds   8 items  64 items   8 items  64 items   8 items  64 items
    //     1      7.1  5.4  7.4  5.8   7.8  6.0  8.2  6.5   9.9  8.2 10.1  8.7
    //     2      8.0  6.6  8.8  7.0   8.8  7.4  9.9  8.0  11.5  9.9 13.8 10.3
    //     4      8.2  8.8  9.7  9.2   8.9 10.3 12.0 10.7  11.1 12.9 15.8 13.4
    //     8      8.4 13.5 11.9 14.0   9.2 15.8 13.0 16.4  11.4 19.3 16.5 19.7
    // and a call that is not replayed from a graph takes about 16 cut, 11.3 to
    // 13.8 whole up to four rounds, 13.8 to 20.2 at eight.  So: whole up to four
    // rounds, where calls gain 2 to 5 us, and a replayed step of few items loses
    // up to 2.3 us (at four rounds).  Of 768 items, more than the CTAs, whole
    // ones are the faster at up to two rounds; at four they take 27.6 us where
    // cut 26.1 (d = 64), 36.9 and 37.5 (128), 47.6 and 51.7 (256).
    P.whole_tokens = 4 * NW * C::TT;
    const int64_t items = (int64_t)P.batch * P.Hkv * ((rows + R - 1) / R);
    const PagedGrid grid = tq_paged_grid(P, items, P.max_tokens / (C::TT * NW) + 1, n_sms * C::CTAS, R, D);
    if (need) {
        *need = grid.bytes;
        return TQ_OK;
    }
    static std::atomic<uint64_t> allowed;
    cudaError_t e = tq_paged_allow(tq_paged_decode_kernel<D, NT>, C::SMEM, 0, P.device, allowed);
    if (e == cudaSuccess) {
        e = tq_launch_dependent(tq_paged_decode_kernel<D, NT>, dim3(grid.ctas), dim3(THREADS), C::SMEM, stream, P);
    }
    if (e != cudaSuccess || P.whole) return tq_check_cuda(e);
    return tq_launch_paged_join(D, P, grid.ctas, R, stream);
}

template <int D>
tq_status launch_dim(const PagedAttn &P, int max_q_len, int n_sms, cudaStream_t stream, size_t *need) {
    const int64_t rows = (int64_t)max_q_len * P.G;
    const int nt = (rows <= 8 || D == 256) ? 1 : 2;
    if constexpr (D != 256)
        if (nt == 2) return launch_decode<D, 2>(P, rows, n_sms, stream, need);
    return launch_decode<D, 1>(P, rows, n_sms, stream, need);
}

}  // namespace

tq_status tq_launch_paged_join(int d, const PagedAttn &P, int grid, int rows, cudaStream_t stream) {
    const auto kern = d == 64 ? tq_paged_join_kernel<64> : d == 128 ? tq_paged_join_kernel<128> : tq_paged_join_kernel<256>;
    return tq_check_cuda(tq_launch_dependent(kern, dim3(grid, std::max(1, rows / 8)), dim3(32 * JOIN_WARPS), 0, stream, P, rows));
}

tq_status tq_launch_paged_attention(const tq_paged *ctx, const PagedAttn &P, int max_q_len, int n_sms,
                                    cudaStream_t stream, size_t *need) {
    // Rows of a kv head (the most of a sequence) up to which the fragments of
    // this file are the faster: at 64 k tokens and 8 kv heads (d = 64) 32 rows
    // took 43 us here and 59 on the row blocks of 128, 64 rows 68 and 59; at
    // d = 128 32 rows 62 and 65, 64 rows 109 and 65; at d = 256 (16 k tokens)
    // 16 rows 37 and 40, 32 rows 53 and 41.
    const int64_t rows = (int64_t)max_q_len * P.G;
    if (rows > (ctx->d == 64 ? 48 : 4096 / ctx->d)) return tq_launch_paged_prefill(ctx->d, P, max_q_len, n_sms, stream, need);
    if (ctx->d == 64) return launch_dim<64>(P, max_q_len, n_sms, stream, need);
    if (ctx->d == 128) return launch_dim<128>(P, max_q_len, n_sms, stream, need);
    return launch_dim<256>(P, max_q_len, n_sms, stream, need);
}
