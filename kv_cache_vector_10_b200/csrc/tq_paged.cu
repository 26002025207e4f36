// tq_paged.cu -- the paged 4-bit cache: handle, argument checks, and the two
// kernels that write rows into pages and read rows back (tq_paged.cuh gives
// the format; the attention kernels are in tq_paged_attend.cu).
//
// Both kernels move bytes: 4.25 bits of packed row against 16 (or 32) bits of
// plain value, some ten instructions for each value.  A thread owns sixteen
// consecutive channels of a row: one 32-byte load or store of 16-bit values
// and one 8-byte word of codes, so a warp moves whole sectors, addresses and
// scales are worked out once for sixteen values, and two lanes share a scale.
#include <climits>
#include <cmath>
#include <cstring>
#include <new>

#include "tq_paged.cuh"

int tq_device_sms(int dev);

namespace {

constexpr int RW_THREADS = 256;

struct RowsArg {
    const void *k, *v;          // plain rows in (write)
    void *ko, *vo;              // plain rows out (read; stored values of a write), contiguous
    uint8_t *kc, *vc;           // pages
    const int64_t *slots;
    int64_t skt, skh, svt, svh; // element strides of k and v: token, head
    int64_t n_rows;             // tokens * heads
    int64_t n_slots, page_bytes;
    uint64_t inv_H;             // ceil(2^32 / H): r / H for r < 2^16
    int H, lg_page;
    unsigned long long *status;
};

__device__ __forceinline__ float scale_value(uint32_t byte) {
    return __half2float(__ushort_as_half((unsigned short)(byte << 7)));
}

// The smallest scale byte with amax <= 7.5 s.  7.5 times a scale has eight
// bits, so the comparison is exact; the quotient is only a first guess, made
// a little too small: at most one step for values of up to eleven bits (the
// distance of amax / 7.5 from a scale that it is not equal to is then more
// than the guess is off), two for float32.
template <int STEPS>
__device__ __forceinline__ uint32_t scale_byte(float amax) {
    const float y = amax * (0.13333333f * (1.f - 1.f / 1048576.f));
    uint32_t b = y < 6.103515625e-05f ? (uint32_t)(y * 131072.f) : (__float_as_uint(y) >> 20) - 896u;
    b = min(b, PG_MAX_SCALE);
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
        if (b < PG_MAX_SCALE && 7.5f * scale_value(b) < amax) ++b;
    return b;
}

// 32 bytes at once, from and to global memory.  Rows to be written are read
// once, and the values given back with them are as long as the rows: both
// are marked to leave L2 first, before the pages (32768 x 32 rows: 224 us,
// 236 without, 245 with the loads alone marked).
__device__ __forceinline__ void load32(const void *p, uint32_t (&w)[8]) {
    asm volatile("ld.global.nc.L1::no_allocate.L2::evict_first.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
}
template <bool PASSING>
__device__ __forceinline__ void store32(void *p, const uint32_t (&w)[8]) {
    if (PASSING)
        asm volatile("st.global.L1::no_allocate.L2::evict_first.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]),
                     "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    else
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                     "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
}
// The same by halves, where only 16-byte alignment is known.
__device__ __forceinline__ void load32_16(const void *p, uint32_t (&w)[8]) {
    const uint4 a = __ldg(static_cast<const uint4 *>(p)), b = __ldg(static_cast<const uint4 *>(p) + 1);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
}

// Plain values of a type: W words hold sixteen of them.
template <typename T>
struct Plain {
    static constexpr int W = sizeof(T) * 4;
    static constexpr uint32_t LIMIT = sizeof(T) == 4 ? 0x7F800000u : 0;   // |bits| of a value that is not finite
};
template <>
struct Plain<__half> {
    static constexpr int W = 8;
    static constexpr uint32_t LIMIT = 0x7C00u;
    static __device__ __forceinline__ float from_bits(uint32_t b) { return __half2float(__ushort_as_half((unsigned short)b)); }
    static __device__ __forceinline__ float2 pair(uint32_t w) { return __half22float2(tqpaged::u2h(w)); }
};
template <>
struct Plain<__nv_bfloat16> {
    static constexpr int W = 8;
    static constexpr uint32_t LIMIT = 0x7F80u;
    static __device__ __forceinline__ float from_bits(uint32_t b) { return __uint_as_float(b << 16); }
    static __device__ __forceinline__ float2 pair(uint32_t w) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
};

// |bits| of the largest magnitude; integer order is that of the magnitudes,
// and infinities and NaN come last.
template <typename T>
__device__ __forceinline__ uint32_t amax_bits(const uint32_t (&w)[Plain<T>::W]) {
    uint32_t m = 0;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 16; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
        return m;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
        return max(m >> 16, m & 0xFFFFu);
    }
}

template <typename T>
__device__ __forceinline__ float value(const uint32_t (&w)[Plain<T>::W], int i) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else {
        const float2 p = Plain<T>::pair(w[i >> 1]);
        return (i & 1) ? p.y : p.x;
    }
}

// The values of eight codes, exact in every type, as words in their order.
// A nibble is spliced into the mantissa of 1024 + n or 64 + n (binary16), or
// of 128 + n (bfloat16, whose 136 s has eight bits: 17 times four).
template <typename T>
__device__ __forceinline__ void unpack8(uint32_t w, uint32_t byte, uint32_t *o) {
    using namespace tqpaged;
    if constexpr (sizeof(T) == 2 && Plain<T>::LIMIT == 0x7F80u) {
        const __nv_bfloat162 s = __float2bfloat162_rn(scale_value(byte)), m136 = __float2bfloat162_rn(-136.f * scale_value(byte));
        uint32_t p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t n = and_or(w >> (4 * i), 0x000F000Fu, 0x43004300u);
            const __nv_bfloat162 v = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&n), s, m136);
            p[i] = *reinterpret_cast<const uint32_t *>(&v);
        }
        o[0] = __byte_perm(p[0], p[1], 0x5410);
        o[1] = __byte_perm(p[2], p[3], 0x5410);
        o[2] = __byte_perm(p[0], p[1], 0x7632);
        o[3] = __byte_perm(p[2], p[3], 0x7632);
    } else {
        // offset and scale in two steps: 72 s can pass the largest binary16
        const __half2 s = u2h(byte * 0x00800080u), m72 = __float2half2_rn(-72.f), m1032 = __float2half2_rn(-1032.f);
        const uint32_t w8 = w >> 8;
        const uint32_t p0 = h2u(__hmul2(__hadd2(u2h(and_or(w, 0x000F000Fu, 0x64006400u)), m1032), s));
        const uint32_t p1 = h2u(__hmul2(__hadd2(u2h(and_or(w, 0x00F000F0u, 0x54005400u)), m72), s));
        const uint32_t p2 = h2u(__hmul2(__hadd2(u2h(and_or(w8, 0x000F000Fu, 0x64006400u)), m1032), s));
        const uint32_t p3 = h2u(__hmul2(__hadd2(u2h(and_or(w8, 0x00F000F0u, 0x54005400u)), m72), s));
        const uint32_t q[4] = {__byte_perm(p0, p1, 0x5410), __byte_perm(p2, p3, 0x5410), __byte_perm(p0, p1, 0x7632),
                               __byte_perm(p2, p3, 0x7632)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 2) {
                o[i] = q[i];
            } else {
                const float2 f = __half22float2(u2h(q[i]));
                o[2 * i] = __float_as_uint(f.x);
                o[2 * i + 1] = __float_as_uint(f.y);
            }
        }
    }
}

// Sixteen values (two words of codes) to plain rows.
template <typename T, bool PASSING>
__device__ __forceinline__ void store_values(T *dst, uint2 w, uint32_t byte) {
    uint32_t o[Plain<T>::W];
    unpack8<T>(w.x, byte, o);
    unpack8<T>(w.y, byte, o + Plain<T>::W / 2);
#pragma unroll
    for (int i = 0; i < Plain<T>::W; i += 8)
        store32<PASSING>(reinterpret_cast<uint32_t *>(dst) + i, *reinterpret_cast<const uint32_t(*)[8]>(o + i));
}

// Where a thread's row `base + local` is.
struct Place {
    int64_t token;
    int head;
};

__device__ __forceinline__ Place place_of(const RowsArg &A, int64_t base_token, int base_head, int local) {
    const uint32_t r = (uint32_t)(base_head + local);   // < H + rows of a block < 2^16
    const uint32_t t = (uint32_t)(((uint64_t)r * A.inv_H) >> 32);
    return {base_token + t, (int)(r - t * (uint32_t)A.H)};
}

// Quantise one thread's sixteen values (two lanes share a group, D / 16 a
// row) and store codes, scale and, if `so`, the stored values.
template <typename T, int D>
__device__ __forceinline__ void quantise_store(uint32_t (&x)[Plain<T>::W], bool live, bool kept, uint8_t *page, int t,
                                               int lg_page, int j, T *so, unsigned &bad_rows) {
    constexpr int LANES = D / 16;
    const int lane = threadIdx.x & 31;
    uint32_t m = amax_bits<T>(x);
    // a row with a value that is not finite is stored as zeros
    const uint32_t row_mask = (uint32_t)(((1ull << LANES) - 1) << (lane & ~(LANES - 1)));
    if (__ballot_sync(0xffffffffu, m >= Plain<T>::LIMIT) & row_mask) {
#pragma unroll
        for (int i = 0; i < Plain<T>::W; ++i) x[i] = 0;
        m = 0;
        if (kept && j == 0) ++bad_rows;   // (padding may hold anything)
    }
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    float amax;
    if constexpr (sizeof(T) == 4) amax = __uint_as_float(m);
    else amax = Plain<T>::from_bits(m);
    const uint32_t byte = scale_byte<sizeof(T) == 4 ? 2 : 1>(amax);
    const float s = scale_value(byte);
    // Rounding by a first product: x / s of a value with at most 11 bits is
    // either a half-way point n + 1/2 or at least 2^-12 of itself away from
    // one (s has four bits), so a reciprocal made 2^-16 too large rounds
    // half-way points away from zero and moves nothing else.  A float32 value
    // is compared with (n +- 1/2) s, which is exact.
    const float inv = byte ? __fdividef(1.f, s) * (1.f + 1.f / 65536.f) : 0.f;
    constexpr float MAGIC = 12582920.f;   // 1.5 * 2^23 + 8: the sum's low bits are the code + 8
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t acc = 0;
#pragma unroll
        for (int i = 7; i >= 0; --i) {
            const float xi = value<T>(x, 8 * h + i);
            float c = fminf(fmaxf(fmaf(xi, inv, MAGIC), MAGIC - 8.f), MAGIC + 7.f);
            if (sizeof(T) == 4 && byte) {
                const float n = fabsf(c - MAGIC), a = fabsf(xi), sg = xi < 0.f ? -1.f : 1.f;
                if (a < (n - 0.5f) * s) c -= sg;
                else if (a >= (n + 0.5f) * s) c = fminf(fmaxf(c + sg, MAGIC - 8.f), MAGIC + 7.f);
            }
            acc = acc * 16u + __float_as_uint(c);
        }
        // every term but the nibbles: the bits of 1.5 * 2^23, times 16^i
        w[h] = acc - 0x4B400000u * 0x11111111u;
    }
    if (kept) {
        *reinterpret_cast<uint2 *>(page + (int64_t)t * (D / 2) + 8 * j) = make_uint2(w[0], w[1]);
        if ((j & 1) == 0) page[((int64_t)(D / 2) << lg_page) + t * (D / PG_GROUP) + (j >> 1)] = (uint8_t)byte;
    }
    if (so && live) store_values<T, true>(so, make_uint2(w[0], w[1]), byte);
}

// A thread's row, and where it lies in the cache.
struct Row {
    int64_t row, at;   // row of the call; byte offset of its page of this head
    Place p;
    int t;             // token of the page
    bool live, kept;   // whether there is such a row, and whether it has a place in the cache
};

template <int D>
__device__ __forceinline__ Row row_of(const RowsArg &A) {
    constexpr int STEP = RW_THREADS / (D / 16);   // rows of a block
    const int64_t base = (int64_t)blockIdx.x * STEP, base_token = base / A.H;
    Row r;
    r.row = base + threadIdx.x / (D / 16);
    r.live = r.row < A.n_rows;
    r.p = place_of(A, base_token, (int)(base - base_token * A.H), (int)(r.row - base));
    const int64_t slot = r.live ? __ldg(A.slots + r.p.token) : -1;
    r.kept = slot >= 0 && slot < A.n_slots;
    r.t = r.kept ? (int)(slot & ((1 << A.lg_page) - 1)) : 0;
    r.at = r.kept ? ((slot >> A.lg_page) * A.H + r.p.head) * A.page_bytes : 0;
    if (slot >= A.n_slots) atomicOr(reinterpret_cast<unsigned int *>(A.status + 1), TQ_FLAG_INDEX);
    return r;
}

// Rows -> pages.  Each thread holds sixteen channels of a row's key and value,
// both loaded before either is used.  WIDE: every row starts on a 32-byte
// boundary.  More rows a thread do not help (two: the same at 32768 x 32
// rows, 5% slower at 8191 x 8 of 64 channels).
template <typename T, int D, bool WIDE>
__global__ void __launch_bounds__(RW_THREADS) tq_paged_write_kernel(const __grid_constant__ RowsArg A) {
    constexpr int W = Plain<T>::W;
    const int j = threadIdx.x % (D / 16);
    tqdev::grid_dep_wait();
    const Row r = row_of<D>(A);
    const T *k = static_cast<const T *>(A.k), *v = static_cast<const T *>(A.v);
    T *ko = static_cast<T *>(A.ko), *vo = static_cast<T *>(A.vo);
    uint32_t xk[W], xv[W];
    auto load = [&](const T *p, uint32_t(&x)[W]) {
#pragma unroll
        for (int i = 0; i < W; i += 8) {
            auto &part = *reinterpret_cast<uint32_t(*)[8]>(x + i);
            if (WIDE) load32(reinterpret_cast<const uint32_t *>(p) + i, part);
            else load32_16(reinterpret_cast<const uint32_t *>(p) + i, part);
        }
    };
#pragma unroll
    for (int e = 0; e < W; ++e) xk[e] = xv[e] = 0;
    if (r.live) {
        if (k) load(k + r.p.token * A.skt + r.p.head * A.skh + 16 * j, xk);
        if (v) load(v + r.p.token * A.svt + r.p.head * A.svh + 16 * j, xv);
    }
    unsigned bad_rows = 0;
    if (k) quantise_store<T, D>(xk, r.live, r.kept, A.kc + r.at, r.t, A.lg_page, j, ko ? ko + r.row * D + 16 * j : nullptr, bad_rows);
    if (v) quantise_store<T, D>(xv, r.live, r.kept, A.vc + r.at, r.t, A.lg_page, j, vo ? vo + r.row * D + 16 * j : nullptr, bad_rows);
    if (bad_rows) atomicAdd(A.status, (unsigned long long)bad_rows);
}

// Pages -> rows (exact in every type).  A slot outside the cache gives a row
// of zeros.
template <typename T, int D>
__global__ void __launch_bounds__(RW_THREADS) tq_paged_read_kernel(const __grid_constant__ RowsArg A) {
    const int j = threadIdx.x % (D / 16);
    tqdev::grid_dep_wait();
    const Row r = row_of<D>(A);
    T *out[2] = {static_cast<T *>(A.ko), static_cast<T *>(A.vo)};
    uint2 w[2];
    uint32_t sb[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint8_t *c = (h ? A.vc : A.kc) + r.at;
        w[h] = make_uint2(0x88888888u, 0x88888888u);
        sb[h] = 0;
        if (r.kept && out[h]) {
            w[h] = __ldg(reinterpret_cast<const uint2 *>(c + (int64_t)r.t * (D / 2)) + j);
            sb[h] = __ldg(c + ((int64_t)(D / 2) << A.lg_page) + r.t * (D / PG_GROUP) + (j >> 1));
        }
    }
    if (!r.live) return;
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (out[h]) store_values<T, false>(out[h] + r.row * D + 16 * j, w[h], sb[h]);
}

template <typename T, int D>
cudaError_t launch_rows(bool write, bool wide, const RowsArg &A, cudaStream_t stream) {
    constexpr int STEP = RW_THREADS / (D / 16);
    // a kernel may be on its way while the one before it ends (it waits for
    // that one before it reads)
    const dim3 grid((unsigned)((A.n_rows + STEP - 1) / STEP)), block(RW_THREADS);
    if (!write) return tq_launch_dependent(tq_paged_read_kernel<T, D>, grid, block, 0, stream, A);
    return wide ? tq_launch_dependent(tq_paged_write_kernel<T, D, true>, grid, block, 0, stream, A)
                : tq_launch_dependent(tq_paged_write_kernel<T, D, false>, grid, block, 0, stream, A);
}

template <typename T>
cudaError_t launch_rows_d(int d, bool write, bool wide, const RowsArg &A, cudaStream_t stream) {
    if (d == 64) return launch_rows<T, 64>(write, wide, A, stream);
    if (d == 128) return launch_rows<T, 128>(write, wide, A, stream);
    return launch_rows<T, 256>(write, wide, A, stream);
}

bool dtype_ok(tq_dtype t) { return t == TQ_F32 || t == TQ_F16 || t == TQ_BF16; }

bool misaligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

int log2_of(int x) {
    int l = 0;
    while ((1 << l) < x) ++l;
    return l;
}

tq_status check_paged_device(const tq_paged *c) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return TQ_ERR_CUDA;
    return dev == c->device ? TQ_OK : TQ_ERR_DEVICE;
}

int64_t page_bytes_of(const tq_paged *c) { return (int64_t)c->page * (c->d / 2 + c->d / PG_GROUP); }

tq_status check_pages(const tq_paged *c, const tq_pages *p, bool need_k, bool need_v) {
    if (!c || !p) return TQ_ERR_NULL;
    if ((need_k && !p->k) || (need_v && !p->v)) return TQ_ERR_NULL;
    if (p->n_kv_heads <= 0 || p->n_pages <= 0) return TQ_ERR_EMPTY;
    if (p->n_kv_heads > TQ_MAX_HEADS || p->n_pages > INT_MAX) return TQ_ERR_LIMIT;
    if ((need_k && misaligned(p->k, 16)) || (need_v && misaligned(p->v, 16))) return TQ_ERR_ALIGN;
    return TQ_OK;
}

tq_status run_rows(tq_paged *ctx, bool write, const tq_pages *pages, RowsArg &A, const int64_t *slots, int64_t n_tokens,
                   tq_dtype dtype, void *stream) {
    if (!dtype_ok(dtype) || n_tokens < 0) return TQ_ERR_DIM_MISMATCH;
    tq_status st = check_paged_device(ctx);
    if (st != TQ_OK) return st;
    if (n_tokens == 0) return TQ_OK;
    if (!slots) return TQ_ERR_NULL;
    if (misaligned(slots, 8)) return TQ_ERR_ALIGN;
    if (n_tokens > INT_MAX || n_tokens * pages->n_kv_heads > (int64_t)INT_MAX * 4) return TQ_ERR_LIMIT;
    A.kc = static_cast<uint8_t *>(pages->k);
    A.vc = static_cast<uint8_t *>(pages->v);
    A.slots = slots;
    A.H = pages->n_kv_heads;
    A.inv_H = ((1ull << 32) + A.H - 1) / A.H;
    A.lg_page = log2_of(ctx->page);
    A.n_rows = n_tokens * A.H;
    A.n_slots = pages->n_pages * ctx->page;
    A.page_bytes = page_bytes_of(ctx);
    A.status = ctx->d_status;
    const int64_t es = dtype == TQ_F32 ? 4 : 2;
    const bool wide = !misaligned(A.k, 32) && !misaligned(A.v, 32) && (A.skt | A.skh | A.svt | A.svh) * es % 32 == 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == TQ_F32) return tq_check_cuda(launch_rows_d<float>(ctx->d, write, wide, A, s));
    if (dtype == TQ_F16) return tq_check_cuda(launch_rows_d<__half>(ctx->d, write, wide, A, s));
    return tq_check_cuda(launch_rows_d<__nv_bfloat16>(ctx->d, write, wide, A, s));
}

}  // namespace

extern "C" {

tq_status tq_paged_create(int head_dim, int page_size, tq_paged **out) {
    if (!out) return TQ_ERR_NULL;
    *out = nullptr;
    if (head_dim == 0) return TQ_ERR_ZERO_DIM;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return TQ_ERR_DIM;
    if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1))) return TQ_ERR_DIM_MISMATCH;
    int dev = -1, major = 0, minor = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return TQ_ERR_CUDA;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
        return TQ_ERR_CUDA;
    if (major != 10 || minor != 0) return TQ_ERR_DEVICE;
    unsigned long long *status = nullptr;
    tq_status st = tq_check_cuda(cudaMalloc(&status, 2 * sizeof(unsigned long long)));
    if (st == TQ_OK) st = tq_check_cuda(cudaMemset(status, 0, 2 * sizeof(unsigned long long)));
    if (st == TQ_OK) st = tq_check_cuda(cudaDeviceSynchronize());
    tq_paged *c = st == TQ_OK ? new (std::nothrow) tq_paged{head_dim, page_size, dev, status} : nullptr;
    if (!c) {
        cudaFree(status);
        return st == TQ_OK ? TQ_ERR_LIMIT : st;
    }
    *out = c;
    return TQ_OK;
}

void tq_paged_destroy(tq_paged *ctx) {
    if (!ctx) return;
    int dev = -1;
    cudaGetDevice(&dev);
    if (dev != ctx->device) cudaSetDevice(ctx->device);
    cudaDeviceSynchronize();
    cudaFree(ctx->d_status);
    if (dev >= 0 && dev != ctx->device) cudaSetDevice(dev);
    delete ctx;
}

int64_t tq_paged_page_bytes(const tq_paged *ctx) { return ctx ? page_bytes_of(ctx) : 0; }

tq_status tq_paged_write(tq_paged *ctx, const void *k, const void *v, tq_dtype dtype, int64_t n_tokens,
                         int64_t stride_kt, int64_t stride_kh, int64_t stride_vt, int64_t stride_vh,
                         const int64_t *slots, const tq_pages *pages, void *k_stored, void *v_stored, void *stream) {
    if (!ctx || !pages) return TQ_ERR_NULL;
    if (n_tokens != 0 && !k && !v) return TQ_ERR_NULL;
    if ((k_stored && !k) || (v_stored && !v)) return TQ_ERR_NULL;
    tq_status st = check_pages(ctx, pages, k != nullptr, v != nullptr);
    if (st != TQ_OK) return st;
    if (!dtype_ok(dtype)) return TQ_ERR_DIM_MISMATCH;
    const int64_t es = dtype == TQ_F32 ? 4 : 2;
    if (misaligned(k, 16) || misaligned(v, 16) || misaligned(k_stored, 32) || misaligned(v_stored, 32) ||
        (k && (stride_kt * es % 16 || stride_kh * es % 16)) || (v && (stride_vt * es % 16 || stride_vh * es % 16)))
        return TQ_ERR_ALIGN;
    RowsArg A = {};
    A.k = k;
    A.v = v;
    A.ko = k_stored;
    A.vo = v_stored;
    A.skt = stride_kt;
    A.skh = stride_kh;
    A.svt = stride_vt;
    A.svh = stride_vh;
    return run_rows(ctx, true, pages, A, slots, n_tokens, dtype, stream);
}

tq_status tq_paged_read(tq_paged *ctx, const tq_pages *pages, const int64_t *slots, int64_t n_tokens, void *k_out,
                        void *v_out, tq_dtype dtype, void *stream) {
    if (!ctx || !pages) return TQ_ERR_NULL;
    if (n_tokens != 0 && !k_out && !v_out) return TQ_ERR_NULL;
    tq_status st = check_pages(ctx, pages, k_out != nullptr, v_out != nullptr);
    if (st != TQ_OK) return st;
    if (misaligned(k_out, 32) || misaligned(v_out, 32)) return TQ_ERR_ALIGN;
    RowsArg A = {};
    A.ko = k_out;
    A.vo = v_out;
    return run_rows(ctx, false, pages, A, slots, n_tokens, dtype, stream);
}

}  // extern "C"

// The checks of an attention call, and its description for the kernels.
static tq_status describe(const tq_paged *ctx, const tq_pages *pages, const void *q, tq_dtype dtype, int64_t total_q,
                          int n_q_heads, int64_t stride_qt, int64_t stride_qh, const int32_t *page_table,
                          int64_t table_stride, int64_t max_pages, const int32_t *seq_lens, const int32_t *q_starts,
                          int batch, int max_q_len, int window, int sinks, float scale, void *out, int64_t stride_ot,
                          int64_t stride_oh, PagedAttn &P) {
    tq_status st = check_pages(ctx, pages, true, true);
    if (st != TQ_OK) return st;
    if (dtype != TQ_F16 && dtype != TQ_BF16) return TQ_ERR_DIM_MISMATCH;
    if (batch <= 0 || n_q_heads <= 0 || max_q_len <= 0) return TQ_ERR_EMPTY;
    if (n_q_heads % pages->n_kv_heads || total_q < 0 || (!q_starts && total_q != batch)) return TQ_ERR_DIM_MISMATCH;
    if (max_pages < 0 || table_stride < max_pages || window < 0 || sinks < 0 || !std::isfinite(scale) || scale < 0.f)
        return TQ_ERR_DIM_MISMATCH;
    if (n_q_heads > TQ_MAX_HEADS || batch > TQ_MAX_PAGED_SEQS || total_q > INT_MAX || total_q * n_q_heads > INT_MAX / 2 ||
        max_pages > INT_MAX || max_pages * ctx->page > INT_MAX / 2 || window > INT_MAX / 2)
        return TQ_ERR_LIMIT;
    if (total_q > 0) {
        if (!q || !out || !seq_lens || (!page_table && max_pages > 0)) return TQ_ERR_NULL;
        if (misaligned(q, 16) || misaligned(out, 16) || stride_qt % 8 || stride_qh % 8 || stride_ot % 8 || stride_oh % 8 ||
            misaligned(page_table, 4) || misaligned(seq_lens, 4) || misaligned(q_starts, 4))
            return TQ_ERR_ALIGN;
    }
    P = PagedAttn{};
    P.kc = static_cast<const uint8_t *>(pages->k);
    P.vc = static_cast<const uint8_t *>(pages->v);
    P.n_pages = pages->n_pages;
    P.page_bytes = page_bytes_of(ctx);
    P.lg_page = log2_of(ctx->page);
    P.Hkv = pages->n_kv_heads;
    P.G = n_q_heads / pages->n_kv_heads;
    P.batch = batch;
    P.total_q = (int)total_q;
    P.q = q;
    P.out = out;
    P.sqt = stride_qt;
    P.sqh = stride_qh;
    P.sot = stride_ot;
    P.soh = stride_oh;
    P.bf16 = dtype == TQ_BF16;
    P.table = page_table;
    P.table_stride = table_stride;
    P.max_tokens = (int)(max_pages * ctx->page);
    P.lens = seq_lens;
    P.starts = q_starts;
    P.window = window;
    P.sinks = sinks;
    P.scale_log2 = (scale > 0.f ? scale : 1.f / std::sqrt((float)ctx->d)) * 1.4426950408889634f;
    P.status = ctx->d_status;
    P.device = ctx->device;
    P.inv_G = P.G > 1 ? ~0ull / (uint64_t)P.G + 1 : 0;
    P.out32 = !misaligned(out, 32) && (stride_ot | stride_oh) % 16 == 0;
    return TQ_OK;
}

extern "C" {

size_t tq_paged_workspace_bytes(const tq_paged *ctx, int n_q_heads, int n_kv_heads, int batch, int64_t max_pages,
                                int max_q_len) {
    if (!ctx || n_q_heads <= 0 || n_kv_heads <= 0 || n_q_heads % n_kv_heads || batch <= 0 || max_pages < 0 ||
        max_q_len <= 0 || max_pages > INT_MAX || max_pages * ctx->page > INT_MAX / 2)
        return 0;
    PagedAttn P = {};
    P.Hkv = n_kv_heads;
    P.G = n_q_heads / n_kv_heads;
    P.batch = batch;
    P.max_tokens = (int)(max_pages * ctx->page);
    size_t need = 0;
    tq_launch_paged_attention(ctx, P, max_q_len, tq_device_sms(ctx->device), nullptr, &need);
    return need;
}

tq_status tq_paged_attention(tq_paged *ctx, const tq_pages *pages, const void *q, tq_dtype dtype, int64_t total_q,
                             int n_q_heads, int64_t stride_qt, int64_t stride_qh, const int32_t *page_table,
                             int64_t table_stride, int64_t max_pages, const int32_t *seq_lens, const int32_t *q_starts,
                             int batch, int max_q_len, int window, int sinks, float scale, void *out,
                             int64_t stride_ot, int64_t stride_oh, void *workspace, size_t ws_bytes, void *stream) {
    if (!ctx || !pages) return TQ_ERR_NULL;
    PagedAttn P;
    tq_status st = describe(ctx, pages, q, dtype, total_q, n_q_heads, stride_qt, stride_qh, page_table, table_stride,
                            max_pages, seq_lens, q_starts, batch, max_q_len, window, sinks, scale, out, stride_ot,
                            stride_oh, P);
    if (st != TQ_OK) return st;
    if ((st = check_paged_device(ctx)) != TQ_OK) return st;
    if (total_q == 0) return TQ_OK;
    const size_t need = tq_paged_workspace_bytes(ctx, n_q_heads, pages->n_kv_heads, batch, max_pages, max_q_len);
    if (need && (!workspace || ws_bytes < need)) return TQ_ERR_WORKSPACE;
    if (misaligned(workspace, 32)) return TQ_ERR_ALIGN;
    P.part = static_cast<float *>(workspace);
    return tq_launch_paged_attention(ctx, P, max_q_len, tq_device_sms(ctx->device), static_cast<cudaStream_t>(stream),
                                     nullptr);
}

tq_status tq_paged_get_status(tq_paged *ctx, void *stream, uint64_t *nonfinite_rows, uint32_t *error_flags) {
    if (!ctx) return TQ_ERR_NULL;
    unsigned long long h[2] = {0, 0};
    tq_status st = tq_check_cuda(cudaStreamSynchronize(static_cast<cudaStream_t>(stream)));
    if (st == TQ_OK) st = tq_check_cuda(cudaMemcpy(h, ctx->d_status, sizeof(h), cudaMemcpyDeviceToHost));
    if (st != TQ_OK) return st;
    if (nonfinite_rows) *nonfinite_rows = h[0];
    if (error_flags) *error_flags = (uint32_t)h[1];
    return TQ_OK;
}

tq_status tq_paged_reset_status(tq_paged *ctx, void *stream) {
    if (!ctx) return TQ_ERR_NULL;
    return tq_check_cuda(
        cudaMemsetAsync(ctx->d_status, 0, 2 * sizeof(unsigned long long), static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
