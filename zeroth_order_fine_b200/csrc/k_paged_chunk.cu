// Attention of chunks of new tokens over the paged cache on the 5th-generation tensor cores: bf16,
// head_dim 64 or 128.
//
// 4 hd flops per (query row, key) against 4 hd bytes per key and 256 rows: the tensor cores and
// the exponentials bound it, HBM only when a chunk is short.  A work item is (256 query rows of one
// request and kv head -- new tokens x the g heads that share it, token-major -- and that head's
// keys); it is processed as two row tiles A and B of 128 against each 128-key unit, so that a key
// tile fetched once serves 256 rows.  The units of all items form one line, cut into equal
// stretches, one per SM; an item cut by a stretch's end is written as partial (m, l, o) and joined
// by a second kernel in key order.
//   warp 0       TMA producer: keys and values of a unit, page by page, into a ring of tiles; one
//                box (64 columns of up to 128 rows) per lane, so the table lookups run in parallel
//   warp 1       TMEM allocator and the single thread that issues tcgen05.mma:
//                  S_t = Q_t K^T  (M 128, N 128, K hd), O_t (+)= P_t V (A from TMEM, N hd)
//                in the order P_A V, Q_A K, P_B V, Q_B K: while one tile's softmax runs, the tensor
//                cores work for the other
//   warps 4..7   softmax of tile A, one row per thread (= its TMEM lane), 8..11 of tile B:
//                P = exp2(S c - m) in bf16 back into TMEM over S's own columns (head_dim 128 fills
//                the 512 columns with S_A S_B O_A O_B), so S_t of the next unit waits for P_t V
// The running reference m of a row moves only when its maximum grows by more than 2^8: sums and
// outputs stay exact in fp32 (P up to 2^8, the same relative rounding) and O is rarely rescaled.
// Keys a row may not see get probability exactly 0.  A row whose scores have a NaN or +infinity is NaN (seen
// by the maximum: the exponentials on the FMA pipe would hide it).  Value rows behind the item's last key (the
// rest of a page, or what an earlier tile left) are not multiplied: the product takes the 16-key
// steps that hold keys, and the rest of the last step is cleared in shared memory.
// Every wait is bounded; on expiry the kernel records the error word, lets what it issued land,
// frees its tensor memory and returns.
//
// Measured: 1024 tokens over 16111 cached, 32 query and 8 kv heads of 128 (279 GFLOP): 264 us, 1.06
// PFLOP/s, 0.65 of the measured burst peak; back to back under the power cap 304 us.  168 registers a
// thread, with 32 bytes of spills (head_dim 64: 28 or 32).  Of the ~3640
// cycles of a unit (clock64 in the roles) each tile's softmax warps work 1670 and wait 1670 for S; the
// MMAs' own time is 2048, and those of Q K, with both operands in shared memory, take all of its 128
// bytes a cycle while the next tiles land there.  So the chain softmax -> P V -> Q K of a tile bounds
// it, the other tile's MMAs filling its gaps; a second S per tile, which would cut the chain, does not
// fit the tensor memory at head_dim 128.  Slower: two issuing warps, one a tile (343 us); 64-key halves
// with S twice (304); both softmax groups on one tile with an exchange of maxima (292); all
// exponentials on the MUFU pipe (282).
#include <float.h>

#include <type_traits>

#include "paged.cuh"

namespace zo {

namespace {

constexpr int RB = 256, UK = 128;                    // rows of an item, keys of a unit
constexpr int THREADS = 384;
constexpr int ATOM = 128 * 128;                      // 64 columns of 128 rows
constexpr int GROUPS = 1024;
constexpr int MAX_CTAS = 148;
constexpr uint32_t DRAIN_POLLS = 1u << 24;
constexpr uint32_t IDESC_QK = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(UK >> 3) << 17) |
                              ((uint32_t)(128 >> 4) << 24);
using Line = PagedLine<true, RB, UK>;

__device__ int g_chunk_error = 0;

template <int HD>
struct Geo {
    static constexpr int NA = HD / 64;               // column halves
    static constexpr int TILE = NA * ATOM;           // bytes of 128 rows of q, k or v
    static constexpr int STAGES = HD == 128 ? 5 : 8;
    static constexpr int TAIL = 512;
    static constexpr int SMEM = (2 + STAGES) * TILE + 1024 + TAIL;
    static constexpr uint32_t IDESC_PV = (IDESC_QK & ~(0x3Fu << 17)) | ((uint32_t)(HD >> 3) << 17) |
                                         (1u << 16);
};

// Pairs of a row's 16 scores whose exponentials go to the FMA pipe instead of the special function
// unit, which for 128 x 128 scores of a tile is busy as long as the tensor cores: a quarter.
// Measured at 1024 new tokens over 16111 (none, 1/8, 1/4, 3/8, 1/2): 277, 263, 261, 274, 286 us.
__device__ __forceinline__ constexpr bool on_fma(int j) { return (j >> 1) % 8 < 2; }
template <int HD>
struct Part {                                        // one piece of an item
    float4 o[HD / 4][RB];
    float m[RB], l[RB];
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// K-major operand: 128-byte rows in 8-row groups of 1024 bytes, 128-byte swizzle
__device__ __forceinline__ uint64_t desc_k(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)1u << 16) | ((uint64_t)(1024u >> 4) << 32) |
           ((uint64_t)1u << 46) | ((uint64_t)2u << 61);
}
// MN-major operand (values as loaded): 64-column blocks ATOM apart
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((uint32_t)ATOM >> 4) << 16) |
           ((uint64_t)(1024u >> 4) << 32) | ((uint64_t)1u << 46) | ((uint64_t)2u << 61);
}
// suspends the thread for ~1 us at most, so that a waiting one looks at its clock regularly
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(1000u)
        : "memory");
    return ok != 0;
}
// Bounded wait, by itself for each lane; false when the bound ended it or another role gave up.  The bound
// lies LIMIT_AT ints behind the flag: a register for it would be one too many in the softmax.
constexpr int LIMIT_AT = 9;
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_f) {
    if (bar_try(bar, parity)) return true;
    const long long t0 = clock64(), limit = *reinterpret_cast<volatile long long*>(abort_f + LIMIT_AT);
    do {
        if (*abort_f) return false;
        if (clock64() - t0 > limit) {
            *abort_f = 1;
            atomicOr(&g_chunk_error, 1);
            return false;
        }
    } while (!bar_try(bar, parity));
    return true;
}
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok));
    return ok != 0;
}
__device__ __forceinline__ void drain_bar(uint32_t bar, uint32_t parity) {
    for (uint32_t i = 0; i < DRAIN_POLLS && !bar_try(bar, parity); ++i) __nanosleep(128);
}
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count));
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                 : "memory");
}
__device__ __forceinline__ void fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_async() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// 32 columns of the thread's TMEM lane, without waiting for them
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
// Waits for the thread's TMEM loads; v: the registers of one of them, which nothing may read before
__device__ __forceinline__ void tmem_wait_ld(uint32_t* v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]),
                 "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]),
                 "+r"(v[14]), "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]),
                 "+r"(v[21]), "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]),
                 "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
        "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]),
        "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld16(uint32_t* v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]),
                   "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]),
                   "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
                 :
                 : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// the larger of two, NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// two fp32 operations in one instruction, each rounded as by itself
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// 2^x of two values on the FMA pipe, for x >= -126 (below, and for NaN: 2^-126; the caller looks for
// scores that are NaN or infinite by their maximum), relative error 2.7e-6: x = n + f with
// n the nearest integer (from the low mantissa bits of x + 1.5 2^23), 2^f on [-1/2, 1/2] by the
// degree-4 polynomial of least maximal relative error (fitted by linear programming over a
// Chebyshev grid), n added to its exponent.
__device__ __forceinline__ float2 exp2_fma(float2 v) {
    const uint64_t x = pair(fmaxf(v.x, -126.f), fmaxf(v.y, -126.f));
    const uint64_t t = add2(x, pair(12582912.f, 12582912.f));
    const uint64_t n = add2(t, pair(-12582912.f, -12582912.f));
    const uint64_t f = fma2(n, pair(-1.f, -1.f), x);
    uint64_t p = fma2(f, pair(0.009567738510668278f, 0.009567738510668278f),
                      pair(0.05591749772429466f, 0.05591749772429466f));
    p = fma2(p, f, pair(0.24024811387062073f, 0.24024811387062073f));
    p = fma2(p, f, pair(0.6931219100952148f, 0.6931219100952148f));
    p = fma2(p, f, pair(0.9999992251396179f, 0.9999992251396179f));
    const float2 tf = unpair(t), pf = unpair(p);
    return make_float2(__int_as_float(__float_as_int(pf.x) + (__float_as_int(tf.x) << 23)),
                       __int_as_float(__float_as_int(pf.y) + (__float_as_int(tf.y) << 23)));
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
}

// One MMA per 16 of the summed dimension.  The descriptors are a base plus constants, so that the
// issuing thread spends no more on an MMA than the tensor cores do (rebuilt from addresses each time
// they cost it ~117 cycles a piece, against 64 on the tensor cores).
template <int HD>
__device__ __forceinline__ void mma_qk(uint32_t d, uint64_t q, uint64_t k) {
#pragma unroll
    for (int kk = 0; kk < HD / 16; ++kk) {
        const uint64_t off = (uint64_t)(((kk >> 2) * ATOM + (kk & 3) * 32) >> 4);
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(q + off), "l"(k + off), "r"(IDESC_QK), "r"(kk > 0 ? 1u : 0u)
            : "memory");
    }
}
// steps of 16 keys: P from TMEM (bf16 pairs, 8 columns a step), V from shared memory
template <int HD>
__device__ __forceinline__ void mma_pv(uint32_t d, uint32_t p, uint64_t v, int steps, bool accum) {
#pragma unroll
    for (int kk = 0; kk < UK / 16; ++kk)
        if (kk < steps)
            asm volatile(
                "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
                "r"(p + kk * 8), "l"(v + (uint64_t)(kk * 2048 >> 4)), "r"(Geo<HD>::IDESC_PV),
                "r"(kk > 0 ? 1u : (uint32_t)accum)
                : "memory");
}

// A stretch's part of one item: units [c0, c1) of it; n[t]: units that tile t's rows see any key
// of, from 0 (none of the rows exist: 0).
struct Piece {
    int c0, c1, n[2], kend;
    __device__ __forceinline__ bool active(int t, int c) const { return c < n[t]; }
    __device__ __forceinline__ int end(int t) const { return min(c1, n[t]); }
    __device__ __forceinline__ bool any(int t) const { return c0 < n[t]; }
    // keys of unit c that the product takes
    __device__ __forceinline__ int valid(int c) const { return min(UK, kend - c * UK); }
};
__device__ __forceinline__ Piece piece_of(const PagedArgs& a, const Line::Cursor& k, long long left) {
    Piece p;
    p.c0 = k.unit;
    p.c1 = (int)min((long long)k.units, k.unit + left);
    const int row0 = k.tile * RB;
    p.kend = Line::keys(a, k.q, row0 + RB);
#pragma unroll
    for (int t = 0; t < 2; ++t)
        p.n[t] = row0 + 128 * t >= k.q.rows ? 0
                 : k.q.bad                  ? 1
                                            : (Line::keys(a, k.q, row0 + 128 * (t + 1)) + UK - 1) / UK;
    return p;
}

template <int HD>
__global__ void __launch_bounds__(THREADS, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap map, PagedArgs a, int box_rows,
                       PagedDesc* __restrict__ desc, Part<HD>* __restrict__ part) {
    using G = Geo<HD>;
    constexpr int STAGES = G::STAGES, TILE = G::TILE;
    extern __shared__ uint8_t raw[];
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    uint8_t* g = raw + (base - smem_u32(raw));
    const uint32_t ring = base + 2 * TILE;
    uint8_t* tail = g + (2 + STAGES) * TILE;
    const uint32_t bar0 = smem_u32(tail);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (STAGES + s); };
    auto q_full = [&](int t) { return bar0 + 8u * (2 * STAGES + t); };
    auto s_full = [&](int t) { return bar0 + 8u * (2 * STAGES + 2 + t); };
    auto p_full = [&](int t) { return bar0 + 8u * (2 * STAGES + 4 + t); };
    auto pv_done = [&](int t) { return bar0 + 8u * (2 * STAGES + 6 + t); };
    auto o_free = [&](int t) { return bar0 + 8u * (2 * STAGES + 8 + t); };
    const uint32_t drain = bar0 + 8u * (2 * STAGES + 10);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(tail + 256);
    volatile int* abort_f = reinterpret_cast<volatile int*>(tail + 260);
    volatile int* bad_unit = reinterpret_cast<volatile int*>(tail + 264);          // [8]
    Line::Cursor* first = reinterpret_cast<Line::Cursor*>(tail + 304);
    static_assert((260 + 4 * LIMIT_AT) % 8 == 0 && 260 + 4 * LIMIT_AT + 8 <= 304 && 4 * LIMIT_AT >= 36, "limit");
    static_assert(8 * (2 * STAGES + 11) <= 256 && 304 + sizeof(Line::Cursor) <= G::TAIL, "tail");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) {
            bar_init(full(s), 1);
            bar_init(empty(s), 1);
        }
        for (int t = 0; t < 2; ++t) {
            bar_init(q_full(t), 4);
            bar_init(s_full(t), 1);
            bar_init(p_full(t), 4);
            bar_init(pv_done(t), 1);
            bar_init(o_free(t), 4);
        }
        bar_init(drain, 1);
        *abort_f = 0;
        *reinterpret_cast<volatile long long*>(abort_f + LIMIT_AT) = a.wait_cycles;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    grid_dep_launch();                                // the joining kernel may be scheduled
    // the prefix sums lie in the ring until the stretch is known
    long long* cum = reinterpret_cast<long long*>(g + 2 * TILE);
    long long* wsum = cum + GROUPS + 1;
    const long long L = Line::prefix(a, GROUPS, cum, wsum);
    const int w = blockIdx.x;
    const long long stretch = div_ll(L + gridDim.x - 1, gridDim.x);
    long long u0 = stretch * w;
    const long long u1 = min(L, u0 + stretch);
    if (tid == 0) desc[w].pieces = 0;
    if (u0 >= u1) return;                             // the whole CTA
    if (warp == 0) {
        const Line::Cursor k = Line::locate(a, GROUPS, cum, u0);
        if (lane == 0) *first = k;
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tslot))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_async();                                    // the ring's first use was by plain accesses
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *tslot;
    auto t_s = [&](int t) { return tmem + (uint32_t)(t * 128); };
    auto t_o = [&](int t) { return tmem + (uint32_t)(256 + t * 128); };
    Line::Cursor k = *first;

    int loads = 0;                                    // producer: ring tiles asked for
    bool issued = false;                              // issuer: any MMA
    if (warp == 0) {
        // ---------------- keys and values ----------------
        const int n_pages = (int)(a.n_slots >> a.page_shift);
        const int boxes = UK / box_rows;              // row boxes of a tile
        int unit = 0;
        bool ok = true;
        for (long long u = u0; u < u1 && ok;) {
            const Piece p = piece_of(a, k, u1 - u);
            const int* table = a.block_table + (size_t)k.r * a.max_blocks;
            for (int c = p.c0; c < p.c1 && ok; ++c, ++unit) {
                // lane l of a box row-major list: row box l / NA, column half l % NA
                const int rb = lane / G::NA, half = lane % G::NA;
                const int key = c * UK + rb * box_rows;
                const bool want = rb < boxes && key < p.kend;
                int row = -1;
                if (want) {
                    const int page = table[key >> a.page_shift];
                    if ((unsigned)page < (unsigned)n_pages)
                        row = (page << a.page_shift) + (key & ((1 << a.page_shift) - 1));
                }
                const unsigned have = __ballot_sync(0xffffffffu, row >= 0);
                const unsigned asked = __ballot_sync(0xffffffffu, want);
                const uint32_t bytes = (uint32_t)__popc(have) * (uint32_t)(box_rows * 128);
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    const int s = loads % STAGES;
                    if (!whole_warp(wait_bar(empty(s), ((loads / STAGES) & 1) ^ 1u, abort_f))) { ok = false; break; }
                    if (lane == 0) {
                        if (kv == 0) bad_unit[unit & 7] = k.q.bad || have != asked;
                        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(full(s)),
                                     "r"(bytes)
                                     : "memory");
                    }
                    __syncwarp();
                    if (row >= 0)
                        asm volatile(
                            "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
                            " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(
                                ring + (uint32_t)(s * TILE + half * ATOM + rb * box_rows * 128)),
                            "l"(reinterpret_cast<uint64_t>(&map)), "r"(full(s)), "r"(0), "r"(row),
                            "r"(k.head * G::NA + half), "r"(kv)
                            : "memory");
                    ++loads;
                }
            }
            u += p.c1 - p.c0;
            Line::advance(a, k, p.c1 - p.c0, u < u1);
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer ----------------
        // the whole warp runs the loop, so that its counters stay uniform; one lane issues, and no lane
        // needs another, so each takes its own waits' verdicts
        const bool leader = elect_one();
        {
            const uint64_t dq = desc_k(base), dk = desc_k(ring), dv = desc_mn(ring);
            // Steps run over the stretch's units; at step i tile t's P V of unit i - 1 comes before
            // its Q K of unit i.  P V waits for the softmax.  Q K writes the columns that P lies in
            // and is issued straight behind P V: the MMAs of a CTA run in the order of issue.
            // (A wait for P V in between left the tensor cores idle for ~250 cycles a tile.)
            Piece prev, cur;
            bool have_prev = false, ok = true;
            int prev_c = 0, ks = 0, vs = 0;
            uint32_t kp = 0, vp = 0;
            int qi[2] = {0, 0};                       // pieces begun: q_full and o_free phases
            int pi[2] = {0, 0};                       // P V issued
            long long u = u0;
            bool more = true;
            cur = piece_of(a, k, u1 - u);
            int c = cur.c0;
            while (ok) {
                // ring tiles: keys of this unit (ks, parity kp), values of the one before (vs, vp)
                if (more && !wait_bar(full(ks), kp, abort_f)) break;
                if (have_prev && !wait_bar(full(vs), vp, abort_f)) break;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (have_prev && prev.active(t, prev_c)) {
                        if (!wait_bar(p_full(t), pi[t] & 1, abort_f)) { ok = false; break; }
                        const bool head = prev_c == prev.c0;
                        if (head && qi[t] > 1 && !wait_bar(o_free(t), qi[t] & 1, abort_f)) { ok = false; break; }
                        fence_after();
                        const int valid = prev.valid(prev_c);
                        if (leader) {
                            mma_pv<HD>(t_o(t), t_s(t), dv + (uint64_t)(vs * TILE >> 4), (valid + 15) / 16, !head);
                            commit(pv_done(t));
                        }
                        issued = true;
                        ++pi[t];
                    }
                    if (more && cur.active(t, c)) {
                        if (c == cur.c0) {
                            if (!wait_bar(q_full(t), qi[t] & 1, abort_f)) { ok = false; break; }
                            ++qi[t];
                        }
                        fence_after();
                        if (leader) {
                            mma_qk<HD>(t_s(t), dq + (uint64_t)(t * TILE >> 4), dk + (uint64_t)(ks * TILE >> 4));
                            commit(s_full(t));
                        }
                        issued = true;
                    }
                }
                if (!ok) break;
                if (have_prev && leader) commit(empty(vs));
                if (!more) break;
                if (leader) commit(empty(ks));
                have_prev = true;
                prev = cur;
                prev_c = c;
                vs = ks + 1 == STAGES ? 0 : ks + 1;
                vp = ks + 1 == STAGES ? kp ^ 1u : kp;
                ks = vs + 1 == STAGES ? 0 : vs + 1;
                kp = vs + 1 == STAGES ? vp ^ 1u : vp;
                if (++c == cur.c1) {
                    u += cur.c1 - cur.c0;
                    more = u < u1;
                    Line::advance(a, k, cur.c1 - cur.c0, more);
                    if (more) {
                        cur = piece_of(a, k, u1 - u);
                        c = cur.c0;
                    }
                }
            }
            if (leader && issued) {
                commit(drain);                        // every MMA retires before TMEM is freed
                drain_bar(drain, 0);
            }
        }
    } else if (warp >= 4) {
        // ---------------- softmax and outputs ----------------
        const int t = (warp - 4) >> 2;
        const int row = (warp & 3) * 32 + lane;       // row of the tile = TMEM lane
        const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
        const float sl2 = a.scale * 1.4426950408889634f;
        uint8_t* qs = g + t * TILE;
        const uint32_t ts = t_s(t) + lane_addr, to = t_o(t) + lane_addr;
        auto load_q = [&](const Line::Cursor& at) {
            const int r = at.tile * RB + t * 128 + row;
            const bool live = r < at.q.rows;
            const int rr = live ? r : 0;
            const uint4* q = reinterpret_cast<const uint4*>(
                static_cast<const __nv_bfloat16*>(a.q) + (size_t)(at.q.start + by_g(a, rr)) * a.ld_q +
                (size_t)(at.head * a.g + mod_g(a, rr)) * HD);
#pragma unroll 8
            for (int ch = 0; ch < HD / 8; ++ch)
                *reinterpret_cast<uint4*>(qs + (ch >> 3) * ATOM + row * 128 + (((ch & 7) ^ (row & 7)) << 4)) =
                    live ? __ldg(q + ch) : make_uint4(0u, 0u, 0u, 0u);
            fence_async();
            __syncwarp();
            if (lane == 0) bar_arrive(q_full(t));
        };
        int unit = 0, ns = 0;                         // ring position; S tiles consumed
        bool ok = true;
        long long u = u0;
        Piece p = piece_of(a, k, u1 - u);
        if (p.any(t)) load_q(k);
        while (ok) {
            const Line::Cursor it = k;
            float m = -FLT_MAX, raw = -FLT_MAX;       // the reference, scaled and as a score
            uint64_t l[4] = {0ull, 0ull, 0ull, 0ull};  // eight running sums
            bool bad = it.q.bad;
            const int r = it.tile * RB + t * 128 + row;
            const bool live = r < it.q.rows;
            // keys below lim are seen by this row
            const int lim = it.q.bad || !live ? 0 : it.q.ctx + by_g(a, r) + 1;
            const int e = p.end(t);
            const uint64_t c2 = pair(sl2, sl2);
            for (int c = p.c0; c < e; ++c) {
                const bool there = wait_bar(s_full(t), ns & 1, abort_f);     // (the whole warp's verdict below)
                ++ns;
                fence_after();
                bad |= bad_unit[(unit + c - p.c0) & 7] != 0;
                // One pass over the row's scores, 16 at a time with the next 16 on their way: the
                // exponentials are taken against the reference as it stands while the maximum is
                // looked for.  Only when the maximum turns out to be over 2^8 above the reference
                // (a piece's first unit, rarely later) does it move, and the pass is repeated; the
                // scores are still there, since P goes out at the end.
                const int cut = lim - c * UK;
                uint32_t pk[64];
                uint64_t ln[4];
                for (;;) {
                    // The usual pass scales a score and takes the reference off in one rounding.  The
                    // reference has its own, which with scores of 2^31 and more is over 2^7 in the
                    // exponent: no weight left, or none finite.  So the other pass, the one with the masks, takes
                    // the reference off before it scales.
                    const bool plain = there && cut >= UK && (fabsf(m) <= 0x1p20f || m == -FLT_MAX);
                    const bool masked = !whole_warp(plain);
                    if (masked && !whole_warp(there)) { ok = false; break; }
                    const uint64_t m2 = pair(-m, -m), r2 = pair(-raw, -raw);
                    uint32_t sv[2][16];
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < 4; ++i) ln[i] = l[i];
                    auto pass = [&](auto mask) {
                        tmem_ld16(ts, sv[0]);
#pragma unroll
                        for (int h = 0; h < 8; ++h) {
                            uint32_t* v = sv[h & 1];
                            tmem_wait_ld16(v);
                            if (h < 7) tmem_ld16(ts + (h + 1) * 16, sv[(h + 1) & 1]);
                            if (mask) {
#pragma unroll
                                for (int j = 0; j < 16; ++j)
                                    if (h * 16 + j >= cut) v[j] = __float_as_uint(-INFINITY);
                            }
#pragma unroll
                            for (int j = 0; j < 16; j += 2) {
                                const float s0 = __uint_as_float(v[j]), s1 = __uint_as_float(v[j + 1]);
                                mx[(j >> 1) & 3] = max_nan(mx[(j >> 1) & 3], max_nan(s0, s1));
                                const float2 x = unpair(mask ? mul2(add2(pair(s0, s1), r2), c2) : fma2(pair(s0, s1), c2, m2));
                                const float2 e = !mask && on_fma(j) ? exp2_fma(x) : make_float2(ex2(x.x), ex2(x.y));
                                ln[(j >> 1) & 3] = add2(ln[(j >> 1) & 3], pair(e.x, e.y));
                                pk[h * 8 + j / 2] = pack2(e.x, e.y);
                            }
                        }
                    };
                    if (masked) pass(std::true_type{});
                    else pass(std::false_type{});
                    // NaN if any score is, and then the row's result, as with a score of +infinity
                    const float most = max_nan(max_nan(mx[0], mx[1]), max_nan(mx[2], mx[3])), top = most * sl2;
                    bad |= !(top < INFINITY);
                    const bool move = top > m + 8.f;
                    if (!__any_sync(0xffffffffu, move)) break;
                    const float mn = move ? top : m;
                    const float f = ex2(m - mn);      // 1 where it stays; 0 from the start value
                    if (c > p.c0) {
                        // the tile's P V before this unit has retired: the commit that signalled
                        // this S covers all that was issued before it
#pragma unroll 1
                        for (int j = 0; j < HD / 32; ++j) {
                            uint32_t v[32];
                            tmem_ld32(to + j * 32, v);
                            tmem_wait_ld(v);
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
                            tmem_st32(to + j * 32, v);
                        }
                    }
                    const uint64_t f2 = pair(f, f);
#pragma unroll
                    for (int i = 0; i < 4; ++i) l[i] = fma2(l[i], f2, 0ull);
                    m = mn;
                    if (move) raw = most;
                }
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < 4; ++i) l[i] = ln[i];
                tmem_st32(ts, pk);
                tmem_st32(ts + 32, pk + 32);
                tmem_wait_st();
                const int valid = p.valid(c);
                if (valid < UK && (valid & 15)) {
                    // the value rows behind the last key, up to the end of its 16-key step
                    const int vt = 2 * (unit + c - p.c0) + 1, vs = vt % STAGES;
                    if (!whole_warp(wait_bar(full(vs), (vt / STAGES) & 1, abort_f))) { ok = false; break; }
                    const int rows = 16 - (valid & 15);
                    for (int i = (warp & 3) * 32 + lane; i < rows * (HD / 8); i += 128) {
                        const int vr = valid + i / (HD / 8), ch = i % (HD / 8);
                        *reinterpret_cast<uint4*>(g + (2 + vs) * TILE + (ch >> 3) * ATOM + vr * 128 +
                                                  ((ch & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_async();
                }
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(p_full(t));
            }
            if (!ok) break;
            unit += p.c1 - p.c0;
            u += p.c1 - p.c0;
            const bool more = u < u1;
            const Piece done = p;
            Line::advance(a, k, p.c1 - p.c0, more);
            if (more) {
                // the next piece's rows: every Q K of this one has retired (its last S was read)
                p = piece_of(a, k, u1 - u);
                if (p.any(t)) load_q(k);
            }
            const bool whole = done.c0 == 0 && done.c1 == it.units;
            const float2 l2 = unpair(add2(add2(l[0], l[1]), add2(l[2], l[3])));
            // m still at its start: no score of the piece is above -infinity, and what the exponentials on
            // the FMA pipe have left in l is no weight (a whole item's row is then 0 / 0)
            const float lt = bad || (whole && m == -FLT_MAX) ? __int_as_float(0x7fc00000)
                             : m == -FLT_MAX                 ? 0.f
                                                             : l2.x + l2.y;
            Part<HD>* slot = part + 2 * w + (done.c0 == 0 ? 1 : 0);
            if (!whole) {
                slot->m[t * 128 + row] = m;
                slot->l[t * 128 + row] = lt;
                if (t == 0 && row == 0 && done.c0 == 0) {
                    const long long last = u - (done.c1 - done.c0) + it.units - 1;
                    PagedDesc d;
                    d.pieces = (int)(last / stretch) - w + 1;
                    d.start = it.q.start;
                    d.row0 = it.tile * RB;
                    d.rows = min(RB, it.q.rows - it.tile * RB);
                    d.kvh = it.head;
                    desc[w] = d;
                }
            }
            if (done.any(t)) {
                if (!whole_warp(wait_bar(pv_done(t), (ns - 1) & 1, abort_f))) { ok = false; break; }
                fence_after();
                const float inv = 1.f / lt;
                __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) +
                                     (size_t)(it.q.start + by_g(a, r)) * a.ld_out +
                                     (size_t)(it.head * a.g + mod_g(a, r)) * HD;
#pragma unroll 1
                for (int j = 0; j < HD / 32; ++j) {
                    uint32_t v[32];
                    tmem_ld32(to + j * 32, v);
                    tmem_wait_ld(v);
                    if (live && whole) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            auto pr = [&](int x) {
                                return pack2(__uint_as_float(v[8 * i + 2 * x]) * inv,
                                             __uint_as_float(v[8 * i + 2 * x + 1]) * inv);
                            };
                            *reinterpret_cast<uint4*>(out + j * 32 + i * 8) = make_uint4(pr(0), pr(1), pr(2), pr(3));
                        }
                    } else if (live) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            slot->o[j * 8 + i][t * 128 + row] =
                                make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]),
                                            __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3]));
                    }
                }
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(o_free(t));
            }
            if (!more) break;
        }
    }
    __syncthreads();                                  // every role has left its loop
    if (*abort_f && warp == 0 && lane == 0)
        for (int i = loads - 1; i >= 0 && i >= loads - STAGES; --i)
            drain_bar(full(i % STAGES), (i / STAGES) & 1);
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// Adds the pieces of the item that worker blockIdx.x's stretch ended inside, in key order: one row
// per thread; a piece whose keys a row does not see has l = 0 and no output.
constexpr int JOIN_ROWS = 32, JOIN_THREADS = 256;
template <int HD>
__global__ void __launch_bounds__(JOIN_THREADS)
    paged_chunk_join_kernel(PagedArgs a, const PagedDesc* __restrict__ desc, const Part<HD>* __restrict__ part) {
    grid_dep_wait();
    const int w = blockIdx.x;
    const PagedDesc d = desc[w];
    const int row = blockIdx.y * JOIN_ROWS + (threadIdx.x & 31), dg = threadIdx.x >> 5;
    if (d.pieces <= 0 || row >= d.rows) return;
    constexpr int DG = HD / 4 / (JOIN_THREADS / 32);  // float4 groups of a thread
    constexpr int N = 4;                              // pieces in flight together
    float m = -FLT_MAX, l = 0.f;
    float4 o[DG];
#pragma unroll
    for (int j = 0; j < DG; ++j) o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < d.pieces; i0 += N) {
        float pm[N], pl[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const Part<HD>* p = part + 2 * (w + i0 + i) + (i0 + i == 0 ? 1 : 0);
            pm[i] = i0 + i < d.pieces ? p->m[row] : -FLT_MAX;
            pl[i] = i0 + i < d.pieces ? p->l[row] : 0.f;
        }
        float mn = m;
#pragma unroll
        for (int i = 0; i < N; ++i) mn = fmaxf(mn, pm[i]);
        const float g = ex2(m - mn);
        m = mn;
        l *= g;
#pragma unroll
        for (int j = 0; j < DG; ++j) {
            o[j].x *= g;
            o[j].y *= g;
            o[j].z *= g;
            o[j].w *= g;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (pl[i] == 0.f) continue;
            const Part<HD>* p = part + 2 * (w + i0 + i) + (i0 + i == 0 ? 1 : 0);
            const float f = ex2(pm[i] - m);
            l = fmaf(f, pl[i], l);
#pragma unroll
            for (int j = 0; j < DG; ++j) {
                const float4 v = p->o[dg * DG + j][row];
                o[j].x = fmaf(f, v.x, o[j].x);
                o[j].y = fmaf(f, v.y, o[j].y);
                o[j].z = fmaf(f, v.z, o[j].z);
                o[j].w = fmaf(f, v.w, o[j].w);
            }
        }
    }
    const float inv = 1.f / l;
    const int q = d.row0 + row;
    uint2* out = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) +
                                          (size_t)(d.start + by_g(a, q)) * a.ld_out +
                                          (size_t)(d.kvh * a.g + mod_g(a, q)) * HD) + dg * DG;
#pragma unroll
    for (int j = 0; j < DG; ++j)
        out[j] = make_uint2(pack2(o[j].x * inv, o[j].y * inv), pack2(o[j].z * inv, o[j].w * inv));
}

template <int HD>
cudaError_t launch_chunk(const PagedArgs& a, cudaStream_t st) {
    CUtensorMap map;
    const int box_rows = min(UK, 1 << a.page_shift);
    if (!paged_cache_map(&map, a, box_rows, 1, 1)) return cudaErrorNotSupported;
    static std::atomic<uint64_t> attr{0};
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
        e = smem_limit(reinterpret_cast<const void*>(paged_chunk_kernel<HD>), Geo<HD>::SMEM, attr);
    if (e != cudaSuccess) return e;
    const int grid = min(sms, MAX_CTAS);
    PagedDesc* desc = static_cast<PagedDesc*>(a.ws);
    auto* part = reinterpret_cast<Part<HD>*>(static_cast<char*>(a.ws) + MAX_CTAS * sizeof(PagedDesc));
    paged_chunk_kernel<HD><<<grid, THREADS, Geo<HD>::SMEM, st>>>(map, a, box_rows, desc, part);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_pdl(paged_chunk_join_kernel<HD>, dim3(grid, RB / JOIN_ROWS), dim3(JOIN_THREADS), 0, st, a,
                      static_cast<const PagedDesc*>(desc), static_cast<const Part<HD>*>(part));
}

}  // namespace

size_t paged_chunk_workspace(int hd) {
    const size_t p = hd == 128 ? sizeof(Part<128>) : sizeof(Part<64>);
    return MAX_CTAS * (sizeof(PagedDesc) + 2 * p);
}

cudaError_t launch_paged_chunk(PagedArgs a, cudaStream_t st) {
    if (a.n_tokens <= 0 || a.n_rows <= 0) return cudaSuccess;
    a.line_heads = a.Hkv;
    return a.hd == 128 ? launch_chunk<128>(a, st) : launch_chunk<64>(a, st);
}

int paged_chunk_error_word() {
    int v = 0;
    const int zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_chunk_error, sizeof(int)) != cudaSuccess) return -1;
    cudaMemcpyToSymbol(g_chunk_error, &zero, sizeof(int));
    return v;
}

}  // namespace zo
