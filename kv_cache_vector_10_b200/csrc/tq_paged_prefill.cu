// tq_paged_prefill.cu -- attention over the paged 4-bit cache for many
// queries a sequence (chunks of a prompt, whole prompts), on the tcgen05
// tensor cores.  The mathematics is that of tq_paged_attend.cu.
//
// A CTA takes items of 128 NM rows (queries times the query heads of a kv
// head's group) and walks the tiles of 64 tokens that they see:
//   S[128 x 64] = Q K^T      Q (binary16, pre-scaled rows) in TMEM or, where TMEM is full, beside K in shared memory
//   P = 2^(S - m)            one thread a row: S read from TMEM, P written over it as binary16
//   O[128 x d] += P V        P from TMEM, V in shared memory (MN-major), O in TMEM
// What bounds it: 4 * 64 * d operations a row and tile on the tensor cores
// against 64 exponentials on the special-function units, which take as long
// at d = 128; and a tile's codes have to be widened to binary16 (about 1.4
// instructions a code), which is why two row blocks (NM = 2) share each
// widened tile while TMEM holds both (d <= 128).  Two tiles' scores of each
// row block take turns, so that the next is there when a softmax ends.
// Roles: NM x 4 softmax warps, 4 (NM = 2) or 8 widening warps, one warp that
// requests the codes (bulk copies of pages), one that issues the MMAs.
// Measured: 2048 queries over 8192 tokens, 32 query heads on 8 kv heads, d =
// 128: 272 to 277 us on several boxes, 870 to 885 TFLOP/s, 53% of the cuBLAS
// burst rate.  A tile of both row
// blocks takes 2150 cycles, of which the tensor cores need 1024 at their best
// and 1460 for products of 64 columns, shared memory some 1600 (the queries
// are read from it) and each softmax warp 1800.  Whole prompts of 1674, 3127
// and 4001 tokens under a window of 1024 with 4 sinks, 8 query heads on 2 kv
// heads, d = 256: 116 us, 530 TFLOP/s; tensor pipe 31% busy, integer pipe
// 37%, issue slots 42%: the items are short (14.7 tiles), and between them the
// tensor cores wait for the softmax warps, which also load the next queries
// and store the rows.  Registers are spilled at every size (stores and loads
// in bytes: NM = 2 404 and 504 at d = 128, 576 and 780 at d = 64; NM = 1 212
// to 224 and 152 to 156).
#include <algorithm>

#include "tq_paged.cuh"

namespace {

using namespace tqpaged;

constexpr int PT = 64;                 // tokens of a tile
constexpr int UNIT = 1;                // tiles that a CTA's share is counted in

template <int D, int NM>
struct Pre {
    static constexpr int SOFT_WARPS = 4 * NM, WIDEN_WARPS = NM == 1 ? 8 : 4;   // what 64 K registers allow
    // With two row blocks the softmax needs more registers than an equal
    // share: four warp groups start with 128 a thread and trade them.
    static constexpr bool TRADE = NM == 2;
    static constexpr int THREADS = TRADE ? 512 : 32 * (SOFT_WARPS + WIDEN_WARPS + 2);
    static constexpr int REGS_SOFT = 152, REGS_WIDEN = 104, REGS_REST = 104;
    static_assert(2 * REGS_SOFT + REGS_WIDEN + REGS_REST <= 512, "registers of the block");
    static constexpr int R = 128 * NM;
    static constexpr int NB = D == 256 ? 2 : 3;      // widened tiles in shared memory
    static constexpr int NC = 5;                     // code tiles in shared memory (keys run two tiles ahead of values)
    using Load = TileLoad<D, PT, 1>;
    static constexpr int KX = PT * 128;              // 64 channels of a tile: rows of 128 bytes, swizzled
    static constexpr int TILE = (D / 64) * KX;
    // TMEM columns: outputs, two tiles' scores of each row block, and the
    // queries where they fit (else in shared memory)
    static constexpr int COL_S = NM * D, COL_Q = COL_S + NM * 2 * PT;
    static constexpr bool QTMEM = COL_Q + NM * D / 2 <= 512;
    static constexpr int QX = 128 * 128;             // 64 channels of a row block's queries, swizzled
    static constexpr int OFF_V = NB * TILE, OFF_Q = 2 * NB * TILE, OFF_C = OFF_Q + (QTMEM ? 0 : NM * (D / 64) * QX);
    static constexpr int SMEM = OFF_C + NC * Load::STAGE + 1024;
    static_assert(COL_Q <= 512, "TMEM columns");
    static_assert(SMEM <= 232448 - 1024, "shared memory");
};

struct PreBars {
    uint64_t codes_full[5], codes_free[5];
    uint64_t k_full[3], k_free[3], v_full[3], v_free[3];
    uint64_t s_full[2][2], p_full[2][2];   // scores and weights of a row block, by the tile's parity
    uint64_t o_done[2][2], q_ready[2], done;   // o_done by the tile's parity too: two may be outstanding
};

// D[tmem] (+)= A[tmem] * B[smem desc]^T, kind::f16, one CTA.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// A value that is the same in all lanes, as the compiler can tell.
template <typename T>
__device__ __forceinline__ T uniform(T x) {
    return (T)__shfl_sync(0xffffffffu, (int)x, 0);
}

// True in one lane of the (whole) warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// Descriptor of an MN-major operand in 128-byte swizzled atoms: rows of 64
// consecutive MN elements, one row per K index, 64-element MN blocks `lbo`
// bytes apart, 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, uint32_t lbo) {
    uint64_t desc = 0;
    desc |= (uint64_t)((saddr >> 4) & 0x3FFF);
    desc |= (uint64_t)((lbo >> 4) & 0x3FFF) << 16;
    desc |= (uint64_t)(1024 >> 4) << 32;
    desc |= (uint64_t)1 << 46;
    desc |= (uint64_t)2 << 61;
    return desc;
}

__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t phase) {
    return __all_sync(0xffffffffu, tqdev::mbar_wait_bounded(bar, phase));
}

// Pairs of float32, handled by one instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t r, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ void store32(void *p, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e, uint32_t f,
                                        uint32_t g, uint32_t h) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(a), "r"(b), "r"(c), "r"(d), "r"(e), "r"(f),
                 "r"(g), "r"(h)
                 : "memory");
}

// Bit c of the result: token T0 + c is seen from position p.
__device__ __forceinline__ uint64_t seen_bits(const PagedAttn &P, int T0, int p, uint32_t got, int lg_part) {
    const int hi = p - T0;
    uint64_t see = hi < 0 ? 0ull : hi >= 63 ? ~0ull : (2ull << hi) - 1ull;
    if (P.window > 0) {
        const int lo = p - P.window + 1 - T0, ns = P.sinks - T0;
        const uint64_t win = lo <= 0 ? ~0ull : lo >= 64 ? 0ull : ~0ull << lo;
        see &= win | (ns <= 0 ? 0ull : ns >= 64 ? ~0ull : (1ull << ns) - 1ull);
    }
    const uint64_t part = lg_part >= 6 ? ~0ull : (1ull << (1 << lg_part)) - 1ull;
    for (int j = 0; j < (PT >> lg_part); ++j)
        if (!((got >> j) & 1u)) see &= ~(part << (j << lg_part));
    return see;
}

template <int D, int NM>
__global__ void __launch_bounds__(Pre<D, NM>::THREADS, 1) tq_paged_prefill_kernel(const __grid_constant__ PagedAttn P) {
    using C = Pre<D, NM>;
    constexpr int NB = C::NB, NC = C::NC, R = C::R, SW = C::SOFT_WARPS, WIDEN_WARPS = C::WIDEN_WARPS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) PreBars bars;
    __shared__ Share s_share;
    __shared__ long long s_sum[C::THREADS / 32];
    __shared__ uint32_t s_tmem, s_valid[16], s_seen[16][2];   // which parts of a tile were there, which rows are seen: 16 tiles back
    __shared__ int s_abort;

    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    tqdev::grid_dep_wait();
    tqdev::grid_dep_trigger();
    if (tid == 0) {
        for (int i = 0; i < NC; ++i) {
            tqdev::mbar_init(&bars.codes_full[i], 1);
            tqdev::mbar_init(&bars.codes_free[i], WIDEN_WARPS);
        }
        for (int i = 0; i < 3; ++i) {
            tqdev::mbar_init(&bars.k_full[i], WIDEN_WARPS / 2);
            tqdev::mbar_init(&bars.k_free[i], 1);
            tqdev::mbar_init(&bars.v_full[i], WIDEN_WARPS / 2);
            tqdev::mbar_init(&bars.v_free[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            for (int j = 0; j < 2; ++j) {
                tqdev::mbar_init(&bars.s_full[i][j], 1);
                tqdev::mbar_init(&bars.p_full[i][j], 4);
                tqdev::mbar_init(&bars.o_done[i][j], 1);
            }
            tqdev::mbar_init(&bars.q_ready[i], 4);
        }
        tqdev::mbar_init(&bars.done, 1);
        s_abort = tqdev::status_aborted(P.status) ? 1 : 0;
        tqdev::fence_barrier_init();
    }
    const Share sh = find_share<R, PT, UNIT, C::THREADS>(P, &s_share, s_sum);
    if (s_abort || sh.lo >= sh.hi) {
        if (tid == 0 && !P.whole) static_cast<Joint *>(P.rec)[blockIdx.x].rows = 0;
        return;
    }
    if (warp == 0) tqdev::tmem_alloc(&s_tmem, 512);
    tqdev::tc_fence_before();
    __syncthreads();
    tqdev::tc_fence_after();
    const uint32_t tmem = uniform(s_tmem);
    const int lg_part = min(P.lg_page, 6), parts = PT >> lg_part;
    const uint32_t all_parts = (1u << parts) - 1u;
    bool failed = false;
    Walk<R, PT, UNIT> it;
    it.begin(P, sh);
    if (tid == 0 && !P.whole) static_cast<Joint *>(P.rec)[blockIdx.x] = it.joint(P, sh);

    if (warp < SW) {
        if constexpr (C::TRADE) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_SOFT));
        // ------------------------------------------------------------- softmax
        const int m = warp >> 2, r = 128 * m + 32 * (warp & 3) + lane;
        const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t t_o = lanes + m * D, t_q = lanes + C::COL_Q + m * (D / 2);
        // what an item's rows need to know: position of this row's query and
        // of the row block's first and last, factor of its scores, output
        int pos = 0, p_lo = 0, p_hi = 0;
        float mul = 1.f;
        uint16_t *out = nullptr;   // NULL: no such row
        auto enter = [&]() {
            const int row = it.row0 + r, tok = token_of(P, row), hg = row - tok * P.G, base = it.s.len - it.s.n;
            const bool active = row < it.row1;
            pos = base + tok;
            p_lo = base + token_of(P, it.row0 + 128 * m);
            p_hi = base + token_of(P, it.row0 + 128 * m + 127);
            const int64_t t64 = it.s.q0 + tok, h64 = it.h * P.G + hg;
            out = active ? static_cast<uint16_t *>(P.out) + t64 * P.sot + h64 * P.soh : nullptr;
            // this row's query: binary16, channels in the order of widen()
            const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(P.q) + (active ? t64 * P.sqt + h64 * P.sqh : 0));
            constexpr bool ONCE = D <= 128;   // a row in registers between its maximum and its conversion
            uint4 qr[ONCE ? D / 8 : 1];
            float up = 1.f;
            mul = 1.f;
            if (ONCE) {
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
                    qr[ONCE ? i : 0] = active ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
            }
            if (P.bf16 && active) {
                uint32_t a = 0;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) a = __vmaxu2(a, amax4(ONCE ? qr[ONCE ? i : 0] : __ldg(src + i)));
                query_factor(max(a >> 16, a & 0xFFFFu), up, mul);
            }
            mul *= P.scale_log2 * WIDE;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                float x[32];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint4 w = ONCE ? qr[ONCE ? 8 * c + i : 0] : active ? __ldg(src + 8 * c + i) : make_uint4(0, 0, 0, 0);
                    if (P.bf16) w = bf16_to_half(w, up);
                    const uint4 o = make_uint4(__byte_perm(w.x, w.z, 0x5410), __byte_perm(w.x, w.z, 0x7632),
                                               __byte_perm(w.y, w.w, 0x5410), __byte_perm(w.y, w.w, 0x7632));
                    if (C::QTMEM) {
                        x[4 * i + 0] = __uint_as_float(o.x);
                        x[4 * i + 1] = __uint_as_float(o.y);
                        x[4 * i + 2] = __uint_as_float(o.z);
                        x[4 * i + 3] = __uint_as_float(o.w);
                    } else {
                        const int rr = r & 127;
                        *reinterpret_cast<uint4 *>(sm + C::OFF_Q + (m * (D / 64) + c) * C::QX + rr * 128 + ((i ^ (rr & 7)) << 4)) = o;
                    }
                }
                if (C::QTMEM) tqdev::tmem_st_32x32b_x32(t_q + 32 * c, x);
            }
            if (C::QTMEM) {
                tqdev::tmem_wait_st();
                tqdev::tc_fence_before();
            } else {
                tqdev::fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) tqdev::mbar_arrive(&bars.q_ready[m]);
        };
        int n = 0;
        if (it.more()) enter();
        while (it.more()) {
            float m_run = -INFINITY, l_run = 0.f;
            for (int i = it.i0; i < it.i1; ++i, ++n) {
                const uint32_t t_s = lanes + C::COL_S + (2 * m + (n & 1)) * PT;
                if (!wait_warp(&bars.s_full[m][n & 1], (uint32_t)(n >> 1) & 1u)) {
                    failed = true;
                    break;
                }
                tqdev::tc_fence_after();
                float x[2][32];
                tqdev::tmem_ld_32x32b_x32_nowait(t_s, x[0]);
                tqdev::tmem_ld_32x32b_x32(t_s + 32, x[1]);
                const int T0 = tile_token(it.tl, i, PT);
                const uint32_t got = *reinterpret_cast<volatile uint32_t *>(&s_valid[n & 15]);
                const bool whole = T0 + PT - 1 <= p_lo && (P.window <= 0 || T0 > p_hi - P.window || T0 + PT <= P.sinks) && got == all_parts;
                if (!whole) {
                    const uint64_t see = seen_bits(P, T0, pos, got, lg_part);
                    const uint32_t lo = (uint32_t)see, hi = (uint32_t)(see >> 32);
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        if (!((lo >> c) & 1u)) x[0][c] = -INFINITY;
                        if (!((hi >> c) & 1u)) x[1][c] = -INFINITY;
                    }
                }
                float mc[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) mc[c] = fmaxf(x[0][c], x[1][c]);
#pragma unroll
                for (int c = 4; c < 32; ++c) mc[c & 3] = max3(mc[c & 3], x[0][c], x[1][c]);
                const float mx = fmaxf(max3(mc[0], mc[1], mc[2]), mc[3]) * mul;
                const bool raise = mx > m_run + RAISE;
                if (__any_sync(0xffffffffu, raise)) {
                    const float to = fmaxf(m_run, mx);
                    const float f = m_run == -INFINITY ? 0.f : exp2_fast(m_run - to);
                    m_run = to;
                    l_run *= f;
                    if (i > it.i0) {   // the output of the tiles before, once it is complete
                        if (!wait_warp(&bars.o_done[m][(n - 1) & 1], (uint32_t)((n - 1) >> 1) & 1u)) {
                            failed = true;
                            break;
                        }
                        tqdev::tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            float o[32];
                            tqdev::tmem_ld_32x32b_x32(t_o + c, o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] *= f;
                            tqdev::tmem_st_32x32b_x32(t_o + c, o);
                        }
                    }
                }
                const float ref = m_run == -INFINITY ? 0.f : m_run - BIAS;
                float w[32];
                const uint64_t mul2 = pack2(mul, mul), ref2 = pack2(-ref, -ref);
                // the sum of the weights as they are rounded: where few tokens
                // carry a row, their rounding cancels
                float l[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    float a, b;
                    unpack2(fma2(pack2(x[c >> 4][2 * (c & 15)], x[c >> 4][2 * (c & 15) + 1]), mul2, ref2), a, b);
                    a = exp2_fast(a);
                    b = exp2_fast(b);
                    const uint32_t h = h2u(__floats2half2_rn(a, b));
                    add_halves(l[2 * (c & 1)], l[2 * (c & 1) + 1], h);
                    w[c] = __uint_as_float(h);
                }
                l_run += (l[0] + l[1]) + (l[2] + l[3]);
                tqdev::tmem_st_32x32b_x32(t_s, w);
                tqdev::tmem_wait_st();
                tqdev::tc_fence_before();
                __syncwarp();
                if (lane == 0) tqdev::mbar_arrive(&bars.p_full[m][n & 1]);
            }
            if (failed) break;
            // the next item's queries first, so that its scores are on their
            // way while this item's rows (or this CTA's part of them) go out
            const bool direct = it.begins() && it.ends();
            const float inv = !direct ? WIDE : l_run != 0.f ? WIDE / l_run : 0.f;
            uint16_t *to = out;
            float *part = P.part + ((int64_t)blockIdx.x * 2 + (it.begins() ? 1 : 0)) * (R * (D + 2));
            it.next(P);
            if (it.more()) enter();
            if (!wait_warp(&bars.o_done[m][(n - 1) & 1], (uint32_t)((n - 1) >> 1) & 1u)) {
                failed = true;
                break;
            }
            tqdev::tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                float o[32];
                tqdev::tmem_ld_32x32b_x32(t_o + c, o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] *= inv;
                // columns 0..7 hold channels 0 4 1 5 2 6 3 7
                if (!direct) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        store32(part + (int64_t)r * D + c + e, __float_as_uint(o[e]), __float_as_uint(o[e + 2]), __float_as_uint(o[e + 4]),
                                __float_as_uint(o[e + 6]), __float_as_uint(o[e + 1]), __float_as_uint(o[e + 3]),
                                __float_as_uint(o[e + 5]), __float_as_uint(o[e + 7]));
                } else if (to && P.out32) {
#pragma unroll
                    for (int e = 0; e < 32; e += 16)
                        store32(to + c + e, out_pair(P, o[e], o[e + 2]), out_pair(P, o[e + 4], o[e + 6]), out_pair(P, o[e + 1], o[e + 3]),
                                out_pair(P, o[e + 5], o[e + 7]), out_pair(P, o[e + 8], o[e + 10]), out_pair(P, o[e + 12], o[e + 14]),
                                out_pair(P, o[e + 9], o[e + 11]), out_pair(P, o[e + 13], o[e + 15]));
                } else if (to) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        *reinterpret_cast<uint4 *>(to + c + e) = make_uint4(out_pair(P, o[e], o[e + 2]), out_pair(P, o[e + 4], o[e + 6]),
                                                                             out_pair(P, o[e + 1], o[e + 3]), out_pair(P, o[e + 5], o[e + 7]));
                }
            }
            if (!direct) {
                part[R * D + r] = m_run;
                part[R * D + R + r] = l_run;
            }
            tqdev::tc_fence_before();
        }
    } else if (warp < SW + WIDEN_WARPS) {
        if constexpr (C::TRADE) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_WIDEN));
        // ------------------------------------------------------------ widening
        // A lane takes a group (32 channels) of a token: four words of codes
        // to four swizzled sixteen-byte chunks of an operand row.  The lanes
        // of a warp take the groups of consecutive tokens in order, and each
        // begins at another of its words, so that neither the words that are
        // read at once nor the chunks that eight lanes write fall into the
        // same banks.  (Shared memory is what the tensor cores, the copies
        // and this share: at d = 256 a tile takes 1350 cycles of it, and took
        // 1750 with whole groups read at once.)
        // Half of the warps take the keys, half the values: the keys run two
        // tiles ahead of the scores and must not wait for the weights, and a
        // warp makes its writes visible to the MMAs once a tile.
        constexpr int SIDE_WARPS = WIDEN_WARPS / 2, ROWS = PT / SIDE_WARPS, GROUPS = D / 32, STEP = 32 / GROUPS;
        const int kv = uniform((warp - SW) / SIDE_WARPS), e = (warp - SW) % SIDE_WARPS, grp = lane % GROUPS;
        uint64_t *full = kv ? bars.v_full : bars.k_full, *freed = kv ? bars.v_free : bars.k_free;
        int n = 0;
        for (; it.more() && !failed; it.next(P)) {
            for (int i = it.i0; i < it.i1; ++i, ++n) {
                const int cs = n % NC, b = n % NB;
                if (!wait_warp(&bars.codes_full[cs], (uint32_t)(n / NC) & 1u) ||
                    (n >= NB && !wait_warp(&freed[b], (uint32_t)(n / NB - 1) & 1u))) {
                    failed = true;
                    break;
                }
                const uint8_t *codes = sm + C::OFF_C + cs * C::Load::STAGE + kv * C::Load::SIDE;
                uint8_t *tile = sm + (kv ? C::OFF_V : 0) + b * C::TILE;
                // this warp's rows that some query sees, a bit each; the others may hold anything
                const uint32_t seen = *reinterpret_cast<volatile uint32_t *>(&s_seen[n & 15][ROWS * e / 32]) >> (ROWS * e % 32);
#pragma unroll
                for (int g = 0; g < ROWS; g += STEP) {
                    const int tr = ROWS * e + g + lane / GROUPS;   // this lane's token
                    const uint8_t *src = codes + C::Load::codes_at(tr, lg_part) + 16 * grp;
                    const Scale2 sc = scale2(((seen >> (g + lane / GROUPS)) & 1u ? codes[C::Load::scales_at(tr, lg_part) + grp] : 0u) * 0x00010001u);
                    uint8_t *dst = tile + (grp >> 1) * C::KX + tr * 128;
                    const int first = D == 256 ? (grp >> 1) + tr : D == 128 ? 2 * (grp >> 1) + (tr >> 1) : tr >> 2;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int k = (first + j) & 3;
                        uint32_t p[4];
                        widen(*reinterpret_cast<const uint32_t *>(src + 4 * k), sc, p);
                        *reinterpret_cast<uint4 *>(dst + (((4 * (grp & 1) + k) ^ (tr & 7)) << 4)) = make_uint4(p[0], p[1], p[2], p[3]);
                    }
                }
                tqdev::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tqdev::mbar_arrive(&full[b]);
                    tqdev::mbar_arrive(&bars.codes_free[cs]);
                }
            }
        }
    } else {
        if constexpr (C::TRADE) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_REST));
    }
    if (warp == SW + WIDEN_WARPS) {
        // ------------------------------------------------- requests of the codes
        const typename C::Load load(P, lane);
        int n = 0;
        for (; it.more() && !failed; it.next(P)) {
            int tok = load.token(P, it.tl, it.i0, it.i1), page = C::Load::fetch(P, it.b, tok);
            for (int i = it.i0; i < it.i1; ++i, ++n) {
                const int cs = n % NC, tok2 = load.token(P, it.tl, i + 1, it.i1), page2 = C::Load::fetch(P, it.b, tok2);
                if (n >= NC && !wait_warp(&bars.codes_free[cs], (uint32_t)(n / NC - 1) & 1u)) {
                    failed = true;
                    break;
                }
                // (the rows that are seen are found here, once a tile and off
                // the widening warps' way, where it took windowed prompts of
                // d = 256 119 us instead of 115)
                load.request(P, tok, page, it.h, lane, sm + C::OFF_C + cs * C::Load::STAGE, &s_valid[n & 15], &bars.codes_full[cs],
                             [&](uint32_t got) {
#pragma unroll
                                 for (int x = 0; x < 2; ++x) {
                                     const int row = 32 * x + lane;
                                     const uint32_t rows = __ballot_sync(0xffffffffu, any_seen(P, it.tl, tile_token(it.tl, i, PT) + row, 1) && ((got >> (row >> lg_part)) & 1u));
                                     if (lane == 0) *reinterpret_cast<volatile uint32_t *>(&s_seen[n & 15][x]) = rows;
                                 }
                             });
                tok = tok2;
                page = page2;
            }
        }
        // whatever happened to the others: the copies in flight have landed
        for (int k = max(0, n - NC); k < n; ++k) tqdev::mbar_wait_bounded(&bars.codes_full[k % NC], (uint32_t)(k / NC) & 1u);
    } else if (warp == SW + WIDEN_WARPS + 1) {
        // ----------------------------------------------------------------- MMAs
        // The whole warp walks the loop, on values that the compiler knows to
        // be the same in all lanes, and an elected lane issues: the operands
        // of the instructions are then uniform registers.  With the loop in
        // one lane an issue took 84 cycles, more than the product itself (44
        // to 65).
        constexpr uint32_t id_s = tqdev::idesc_f16_f32(PT), id_o = tqdev::idesc_f16_f32(D) | (1u << 16);   // V is MN-major
        const uint32_t k0 = tqdev::smem_u32(sm);
        const uint64_t kd0 = tqdev::smem_desc_sw128(k0), qd0 = tqdev::smem_desc_sw128(k0 + C::OFF_Q), vd0 = desc_mn(k0 + C::OFF_V, C::KX);
        auto scores = [&](int kn, int kb, int m) {
            const uint32_t t_s = tmem + C::COL_S + (2 * m + (kn & 1)) * PT;
            const uint64_t kd = kd0 + (uint32_t)(kb * (C::TILE >> 4));
            if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint64_t b = kd + (uint32_t)(((ks >> 2) * C::KX + (ks & 3) * 32) >> 4);
                    if (C::QTMEM) mma_ts(t_s, tmem + C::COL_Q + m * (D / 2) + 8 * ks, b, id_s, ks != 0);
                    else tqdev::mma_f16_ss(t_s, qd0 + (uint32_t)(((m * (D / 64) + (ks >> 2)) * C::QX + (ks & 3) * 32) >> 4), b, id_s, ks != 0);
                }
                tqdev::mma_commit(&bars.s_full[m][kn & 1]);
            }
            __syncwarp();
        };
        auto outputs = [&](int vn, int vb, int m, bool first) {
            const uint32_t t_p = tmem + C::COL_S + (2 * m + (vn & 1)) * PT;
            const uint64_t vd = vd0 + (uint32_t)(vb * (C::TILE >> 4));
            if (elect_one()) {
                mma_ts(tmem + m * D, t_p, vd, id_o, !first);
#pragma unroll
                for (int ks = 1; ks < PT / 16; ++ks) mma_ts(tmem + m * D, t_p + 8 * ks, vd + (uint32_t)((2048 * ks) >> 4), id_o, 1u);
                tqdev::mma_commit(&bars.o_done[m][vn & 1]);
            }
            __syncwarp();
        };
        auto commit = [&](uint64_t *bar) {
            if (elect_one()) tqdev::mma_commit(bar);
            __syncwarp();
        };
        // buffers and phases of the next tile to score (k) and to weigh (v)
        int n = 0, kn = 0, kb = 0, vb = 0, items = 0;
        uint32_t kph = 0, vph = 0;
        auto next_scores = [&]() {
            if (++kb == NB) {
                kb = 0;
                kph ^= 1;
            }
            ++kn;
        };
        bool ok = true;
        for (; uniform(it.more()) && ok; it.next(P), ++items) {
            const int nt = uniform(it.i1 - it.i0);
            for (int m = 0; m < NM && ok; ++m) ok = wait_warp(&bars.q_ready[m], (uint32_t)items & 1u);
            if (!ok) break;
            tqdev::tc_fence_after();
            for (int j = 0; j < 2 && j < nt; ++j) {   // two tiles' scores ahead
                if (!(ok = wait_warp(&bars.k_full[kb], kph))) break;
                tqdev::tc_fence_after();
                for (int m = 0; m < NM; ++m) scores(kn, kb, m);
                commit(&bars.k_free[kb]);
                next_scores();
            }
            for (int i = 0; i < nt && ok; ++i, ++n) {
                const bool more = i + 2 < nt;
                for (int m = 0; m < NM && ok; ++m) {
                    ok = wait_warp(&bars.p_full[m][n & 1], (uint32_t)(n >> 1) & 1u) && (m > 0 || wait_warp(&bars.v_full[vb], vph));
                    if (!ok) break;
                    tqdev::tc_fence_after();
                    outputs(n, vb, m, i == 0);
                    if (more) {
                        if (m == 0) {
                            if (!(ok = wait_warp(&bars.k_full[kb], kph))) break;
                            tqdev::tc_fence_after();
                        }
                        scores(kn, kb, m);
                    }
                }
                if (!ok) break;
                commit(&bars.v_free[vb]);
                if (++vb == NB) {
                    vb = 0;
                    vph ^= 1;
                }
                if (more) {
                    commit(&bars.k_free[kb]);
                    next_scores();
                }
            }
        }
        failed = !ok;
        commit(&bars.done);
        if (!wait_warp(&bars.done, 0u)) failed = true;
    }
    if (failed) atomicOr(reinterpret_cast<unsigned int *>(P.status + 1), TQ_FLAG_WAIT_TIMEOUT);
    tqdev::tc_fence_before();
    __syncthreads();
    tqdev::tc_fence_after();
    if (warp == 0) tqdev::tmem_dealloc(tmem, 512);
}

template <int D, int NM>
tq_status launch_prefill(PagedAttn P, int64_t rows, int n_sms, cudaStream_t stream, size_t *need) {
    using C = Pre<D, NM>;
    // queries into TMEM and outputs out of it take about as long as eight
    // tiles: ragged prompts under a window 182 us without, 120 with 4, 112
    // with 8, 117 with 16; 2048 tokens over 8192 the same within 2%
    P.item_cost = 8;
    // uncut, whole prompts, 32 query heads on 8, kernel times cut and whole: at
    // d = 128 one of 64 tokens 14.0 and 12.4 us, of 128 16.4 and 14.2, of 512
    // 28.4 and 20.9, of 1024 39.2 and 30.6, eight of 512 72.8 and 63.4; at d =
    // 256 one of 512 37.7 and 22.1, of 1024 57.7 and 55.9; on a single kv head,
    // d = 128, one of 512 21.2 and 20.1, of 1024 23.0 and 28.9: the bound
    P.whole_tokens = 512;
    const int64_t items = (int64_t)P.batch * P.Hkv * ((rows + C::R - 1) / C::R);
    const PagedGrid grid = tq_paged_grid(P, items, P.max_tokens / (4 * PT) + 1, n_sms, C::R, D);
    if (need) {
        *need = grid.bytes;
        return TQ_OK;
    }
    static std::atomic<uint64_t> allowed;
    cudaError_t e = tq_paged_allow(tq_paged_prefill_kernel<D, NM>, C::SMEM, C::TRADE ? 128 : 0, P.device, allowed);
    if (e == cudaSuccess) {
        e = tq_launch_dependent(tq_paged_prefill_kernel<D, NM>, dim3(grid.ctas), dim3(C::THREADS), C::SMEM, stream, P);
    }
    if (e != cudaSuccess || P.whole) return tq_check_cuda(e);
    return tq_launch_paged_join(D, P, grid.ctas, C::R, stream);
}

}  // namespace

tq_status tq_launch_paged_prefill(int d, const PagedAttn &P, int max_q_len, int n_sms, cudaStream_t stream, size_t *need) {
    const int64_t rows = (int64_t)max_q_len * P.G;
    const int nm = rows > 128 && d != 256 ? 2 : 1;
    if (d == 64) return nm == 2 ? launch_prefill<64, 2>(P, rows, n_sms, stream, need) : launch_prefill<64, 1>(P, rows, n_sms, stream, need);
    if (d == 128) return nm == 2 ? launch_prefill<128, 2>(P, rows, n_sms, stream, need) : launch_prefill<128, 1>(P, rows, n_sms, stream, need);
    return launch_prefill<256, 1>(P, rows, n_sms, stream, need);
}
