// Attention of a few query rows per request over the paged cache (decode steps): bf16, head_dim
// 64 or 128, on the tensor cores' warp-level path.
//
// A decode step reads every cached key and value once and computes 4 g flops per element, so
// HBM bounds it and the products only have to keep out of the way.  That decides the form:
//
// * The work of a call is one line of units -- 16 keys (with their values) of one (request, tile
//   of query rows, team of kv heads) -- and every team of warps takes an equal stretch of that
//   line, whatever lengths the requests have.  A team has a warp per head, gcd(Hkv, 8) of them,
//   so its warps read neighbouring columns of the same cache rows at about the same time: whole
//   rows come from HBM together.  A warp works alone: its own ring of shared-memory
//   stages, its own barriers, running maxima, sums and outputs, no block-wide synchronisation.
//   An item cut by a stretch's end is written as a partial (m, l, o) and the pieces are added in
//   key order by a small second kernel.
// * One TMA copy brings a unit: 16 rows of a page, k and v, as a 4-d box (64 columns, rows,
//   column halves, k/v), 128-byte-swizzled, so each warp has STAGES x 8 KB (head_dim 128) in
//   flight and an SM 192 KB.
// * The products are transposed so that no row is padding: S^T = K Q^T takes 16 keys as the
//   16-row side and up to 8 query rows per 8-column block, O^T += V^T P^T takes 16 of the head's
//   dims; P^T turns from accumulator to operand layout by an 8x8 transpose in registers
//   (movmatrix).  With m16n8k16 the MMAs of a 64 KB round of an SM's warps take well under the
//   time HBM needs for those 64 KB.
// * Softmax statistics, outputs and partials are fp32; P is rounded to bf16 for its product, as
//   the packed attention does (the sum l is of the unrounded values).
// Keys a query may not see get probability exactly 0; value rows behind the tile's last key are
// cleared in registers (0 x NaN would not be 0).
//
// Measured: 61 requests of 300-4000 tokens, 32 query and 8 kv heads of 128: 100 us, 5.5 TB/s of the
// cache, 0.85 of the measured HBM rate, of which the join takes 5.  32 requests of 15-160 tokens, 40
// heads: 24.4 us for 60 MB.  The kernel's 13 us of those are 2.5 us before the first copy (lengths,
// prefix sums, the table), 8.5 us at 6.9 TB/s and a tail where CTAs change requests; launch and join
// take the rest.  A team per head instead of per 8 (team = 1): 25.1 and 101.2 us against 24.4 and
// 100.8, as cache rows then come in pieces.
#include <float.h>

#include "paged.cuh"

namespace zo {

namespace {

constexpr int WARPS = 8, THREADS = WARPS * 32;
constexpr int UK = 16;                               // keys per unit
constexpr int GROUPS = 1024;                         // prefix entries kept in shared memory
constexpr int MAX_CTAS = 148;
constexpr int MAX_WORKERS = MAX_CTAS * WARPS;
constexpr uint32_t DRAIN_POLLS = 1u << 24;

__device__ int g_step_error = 0;                     // bit 0: a bounded wait expired

template <int HD>
struct Geo {
    static constexpr int NH = HD / 64;               // 64-column halves of a head
    static constexpr int STAGE = UK * HD * 2 * 2;    // bytes of a unit: k and v
    static constexpr int STAGES = HD == 128 ? 3 : 6;
    static constexpr int SMEM = WARPS * STAGES * STAGE + 1024;
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
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
// one look of a wait: under a bound that is less than a suspension, without one
__device__ __forceinline__ bool bar_poll(uint32_t bar, uint32_t parity, long long limit) {
    return limit < 4000 ? bar_test(bar, parity) : bar_try(bar, parity);
}
// Bounded wait of a whole warp for a unit's copy.
__device__ __forceinline__ bool wait_unit(uint32_t bar, uint32_t parity, long long limit) {
    bool there = bar_poll(bar, parity, limit);
    if (!there) {
        const long long t0 = clock64();
        while (!(there = bar_poll(bar, parity, limit)))
            if (clock64() - t0 > limit) {
                atomicOr(&g_step_error, 1);
                break;
            }
    }
    return whole_warp(there);
}
__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t* r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, const uint32_t* b) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// Slots of partial results, in the accumulator's own layout: slot 2 w: the piece with which team
// w's stretch begins (an item begun by an earlier team); 2 w + 1: the one it ends with (an item
// that goes on); each with a part per warp of the team.  desc[w] describes the item of slot
// 2 w + 1.
template <int HD, int NB>
struct Part {
    float4 o[HD / 16][NB][32];
    float m[NB * 8], l[NB * 8];
};

// 16-dim tiles mt0 .. mt0 + MT - 1 of the rows
template <int HD, int NB, int MT>
__device__ __forceinline__ void store_rows(const PagedArgs& a, int start, int row0, int rows, int kvh,
                                           int mt0, const float (*o)[NB][4], const float (*inv)[2], int lane) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int n = nb * 8 + 2 * (lane & 3) + e;
            if (n >= rows) continue;
            const int row = row0 + n;
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) +
                                 (size_t)(start + by_g(a, row)) * a.ld_out +
                                 (size_t)(kvh * a.g + mod_g(a, row)) * HD + mt0 * 16 + (lane >> 2);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                out[mt * 16] = __float2bfloat16_rn(o[mt][nb][e] * inv[nb][e]);
                out[mt * 16 + 8] = __float2bfloat16_rn(o[mt][nb][2 + e] * inv[nb][e]);
            }
        }
}

template <int HD, int NB>
__global__ void __launch_bounds__(THREADS, 1)
    paged_step_kernel(const __grid_constant__ CUtensorMap map, PagedArgs a, int box_rows,
                      PagedDesc* __restrict__ desc, Part<HD, NB>* __restrict__ part) {
    using G = Geo<HD>;
    constexpr int RB = NB * 8, NH = G::NH, STAGES = G::STAGES;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t bars[WARPS * STAGES];
    __shared__ long long cum[GROUPS + 1];
    __shared__ long long wsum[WARPS];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t ring = ((smem_u32(raw) + 1023u) & ~1023u) + (uint32_t)(warp * STAGES * G::STAGE);
    const uint32_t bar0 = smem_u32(bars + warp * STAGES);
    if (lane == 0)
        for (int s = 0; s < STAGES; ++s)
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar0 + 8u * s));
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (tid == 0) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&map)) : "memory");
    grid_dep_launch();                                // the joining kernel may be scheduled

    // The tables and the queries into L2, a line per thread over the grid: both are read where the
    // copies and the products would wait for DRAM.
    {
        const long long i = (long long)blockIdx.x * THREADS + tid;
        if (i < ((long long)a.n_rows * a.max_blocks + 31) / 32) prefetch_l2(a.block_table + i * 32);
        const int per_row = (a.g * a.Hkv * HD + 63) / 64;
        if (i < (long long)a.n_tokens * per_row) {
            const int t = (int)((unsigned)i / (unsigned)per_row);
            prefetch_l2(static_cast<const __nv_bfloat16*>(a.q) + (size_t)t * a.ld_q + ((int)i - t * per_row) * 64);
        }
    }
    using Line = PagedLine<false, RB, UK>;
    const long long L = Line::prefix(a, GROUPS, cum, wsum);
    const int team = min(WARPS, a.Hkv & -a.Hkv);      // a power of two, as WARPS is
    const int workers = gridDim.x * (WARPS / team), w = blockIdx.x * (WARPS / team) + warp / team;
    const int mate = warp % team;                     // the warp's head within the team's
    const long long stretch = div_ll(L + workers - 1, workers);      // units per worker
    long long u0 = stretch * w;
    const long long u1 = min(L, u0 + stretch);
    if (mate == 0 && lane == 0) desc[w].pieces = 0;
    if (u0 >= u1) return;                             // nothing to do, nothing in flight

    const int count = (int)(u1 - u0);                 // units of this stretch
    struct Place {
        typename Line::Cursor c;
        int kend;                                     // the tile's keys
    };
    Place con;
    con.c = Line::locate(a, GROUPS, cum, u0);
    con.kend = Line::keys(a, con.c.q, (con.c.tile + 1) * RB);
    Place pro = con;
    // to the next unit; true: it belongs to another tile.  `more`: the stretch goes on
    auto advance = [&](Place& p, bool more) {
        if (++p.c.unit < p.c.units) return false;
        p.c.unit = 0;
        if (++p.c.head < a.line_heads) return false;
        p.c.head = 0;
        if (!more) return false;
        Line::next_tile(a, p.c);
        p.kend = Line::keys(a, p.c.q, (p.c.tile + 1) * RB);
        return true;
    };

    // ---- producer side of the warp: unit `pro` into stage ps ----
    const int n_pages = (int)(a.n_slots >> a.page_shift);
    int ids = 0, ids_at = -1, ids_r = -1;             // 32 table entries, one per lane
    uint32_t bad_stage = 0;
    auto page_of = [&](int idx) {
        if (ids_r != pro.c.r || idx < ids_at || idx >= ids_at + 32) {
            ids_r = pro.c.r;
            ids_at = idx;
            ids = idx + lane < a.max_blocks ? a.block_table[(size_t)pro.c.r * a.max_blocks + idx + lane] : -1;
        }
        return __shfl_sync(0xffffffffu, ids, idx - ids_at);
    };
    auto issue = [&](int ps) {
        const uint32_t dst = ring + (uint32_t)(ps * G::STAGE), bar = bar0 + 8u * ps;
        const int kbase = pro.c.unit * UK;
        uint32_t bytes = 0;
        int row[2] = {-1, -1};
        bool bad = pro.c.q.bad;
        if (!bad) {
            const int subs = UK / box_rows;           // boxes per unit: 1, or 2 with pages of 8
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int k = kbase + s * box_rows;
                if (s < subs && k < pro.kend) {
                    const int page = page_of(k >> a.page_shift);
                    if ((unsigned)page < (unsigned)n_pages) {
                        row[s] = (page << a.page_shift) + (k & ((1 << a.page_shift) - 1));
                        bytes += (uint32_t)(box_rows * HD * 4);
                    } else {
                        bad = true;
                    }
                }
            }
        }
        bad_stage = bad ? bad_stage | (1u << ps) : bad_stage & ~(1u << ps);
        if (lane == 0) {
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                         : "memory");
#pragma unroll
            for (int s = 0; s < 2; ++s)
                if (row[s] >= 0)
                    asm volatile(
                        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
                        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst + (uint32_t)(s * box_rows * HD * 4)),
                        "l"(reinterpret_cast<uint64_t>(&map)), "r"(bar), "r"(0), "r"(row[s]),
                        "r"((pro.c.head * team + mate) * NH), "r"(0)
                        : "memory");
        }
    };
    int issued = 0;
    for (int s = 0; s < STAGES && issued < count; ++s) {
        issue(s);
        ++issued;
        advance(pro, issued < count);
    }

    // ---- consumer side ----
    const float sl2 = a.scale * 1.4426950408889634f;
    // lane-dependent parts of the operand addresses: k rows by (lane & 7) + 8 * bit 3, value rows
    // by (lane & 7) + 8 * bit 4; rows of 128 bytes, 16-byte chunks swizzled by the row
    const uint32_t half_st = (uint32_t)box_rows * 128u;          // between column halves
    const uint32_t v_st = half_st * NH;                          // from k to v
    const uint32_t sub_st = box_rows == 16 ? 1024u : 2u * v_st;  // between the two 8-row groups
    const uint32_t k_row = (uint32_t)(lane & 7) * 128u + ((lane >> 3) & 1) * sub_st;
    const uint32_t v_row = v_st + (uint32_t)(lane & 7) * 128u + (lane >> 4) * sub_st;
    const uint32_t k_chunk = lane >> 4, v_chunk = (lane >> 3) & 1, swz = lane & 7;

    uint32_t qf[HD / 16][NB][2];
    float o[HD / 16][NB][4], m[NB][2], l[NB][2];      // m in units of ln 2 of the scaled scores
    int lim[NB][2], lim_min = 0, first_unit = 0;
    size_t q_at[NB], out_at[NB][2];                   // the lane's query and output rows, head 0
    uint32_t q_live = 0;
    bool bad = false, fresh = true, new_tile = true, alive = true;
    int stage = 0;
    uint32_t phase = 0;
    for (int u = 0; u < count; ++u) {
        if (new_tile) {                               // the tile's rows and masks
            new_tile = false;
            const int row0 = con.c.tile * RB;
            lim_min = con.c.q.bad ? 0 : con.c.q.ctx + by_g(a, row0) + 1;
            q_live = 0;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const int row = row0 + nb * 8 + (lane >> 2);
                const int rr = row < con.c.q.rows ? row : row0;
                if (row < con.c.q.rows) q_live |= 1u << nb;
                q_at[nb] = (size_t)(con.c.q.start + by_g(a, rr)) * a.ld_q + (size_t)(mod_g(a, rr)) * HD + 2 * (lane & 3);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int n = row0 + nb * 8 + 2 * (lane & 3) + e, nr = min(n, con.c.q.rows - 1);
                    lim[nb][e] = n < con.c.q.rows ? con.c.q.ctx + by_g(a, nr) + 1 : con.kend;
                    out_at[nb][e] = (size_t)(con.c.q.start + by_g(a, nr)) * a.ld_out + (size_t)(mod_g(a, nr)) * HD + (lane >> 2);
                }
            }
        }
        if (fresh) {                                  // a new item: its queries
            fresh = false;
            first_unit = con.c.unit;
            bad = con.c.q.bad;
            const size_t head = (size_t)((con.c.head * team + mate) * a.g) * HD;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const uint32_t* q = reinterpret_cast<const uint32_t*>(
                    static_cast<const __nv_bfloat16*>(a.q) + q_at[nb] + head);
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk) {
                    qf[kk][nb][0] = (q_live >> nb) & 1u ? __ldg(q + kk * 8) : 0u;
                    qf[kk][nb][1] = (q_live >> nb) & 1u ? __ldg(q + kk * 8 + 4) : 0u;
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    m[nb][e] = -FLT_MAX;
                    l[nb][e] = 0.f;
                }
            }
#pragma unroll
            for (int mt = 0; mt < HD / 16; ++mt)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[mt][nb][e] = 0.f;
        }
        if (!wait_unit(bar0 + 8u * stage, phase, a.wait_cycles)) {
            alive = false;
            break;
        }
        bad |= (bad_stage >> stage) & 1u;
        const uint32_t at = ring + (uint32_t)(stage * G::STAGE);
        const int kbase = con.c.unit * UK;
        float s[NB][4], s1[NB][4];                    // two chains of products
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nb][e] = s1[nb][e] = 0.f;
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk) {
            uint32_t kf[4];
            const uint32_t ch = (kk & 3) * 2 + k_chunk;
            ldsm4(kf, at + k_row + (kk >> 2) * half_st + ((ch ^ swz) << 4));
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) mma16816(kk & 1 ? s1[nb] : s[nb], kf, qf[kk][nb]);
        }
        const int left = con.kend - kbase;            // keys of the unit that exist for the tile
        uint32_t pf[NB][2];
        bool move = false;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 4; ++e)               // (rounded by itself, as the reference is, whatever its size)
                s[nb][e] = __fmul_rn(s[nb][e] + s1[nb][e], sl2);
        if (kbase + UK > lim_min) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = kbase + (lane >> 2) + (e >> 1) * 8;
                    if (key >= min(lim[nb][e & 1], con.kend)) s[nb][e] = -INFINITY;
                }
        }
        // a row's reference moves only when a score is over 2^8 above it: then to the row's maximum
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) move |= fmaxf(s[nb][e], s[nb][e + 2]) > m[nb][e] + 8.f;
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = fmaxf(s[nb][e], s[nb][e + 2]);
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                    const float mn = fmaxf(m[nb][e], mx), f = ex2(m[nb][e] - mn);
                    m[nb][e] = mn;
                    l[nb][e] *= f;
#pragma unroll
                    for (int mt = 0; mt < HD / 16; ++mt) {
                        o[mt][nb][e] *= f;
                        o[mt][nb][e + 2] *= f;
                    }
                }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nb][e] = ex2(s[nb][e] - m[nb][e & 1]);
#pragma unroll
            for (int e = 0; e < 2; ++e) l[nb][e] += s[nb][e] + s[nb][e + 2];
            pf[nb][0] = transpose8x8(pack2(s[nb][0], s[nb][1]));
            pf[nb][1] = transpose8x8(pack2(s[nb][2], s[nb][3]));
        }
        // value rows behind the last key: cleared, the two keys of a register one by one
        const int k2 = 2 * (lane & 3);
        const uint32_t keep0 = (k2 < left ? 0xffffu : 0u) | (k2 + 1 < left ? 0xffff0000u : 0u);
        const uint32_t keep1 = (k2 + 8 < left ? 0xffffu : 0u) | (k2 + 9 < left ? 0xffff0000u : 0u);
#pragma unroll
        for (int mt = 0; mt < HD / 16; ++mt) {
            uint32_t vf[4];
            const uint32_t ch = (mt & 3) * 2 + v_chunk;
            ldsm4t(vf, at + v_row + (mt >> 2) * half_st + ((ch ^ swz) << 4));
            if (left < UK) {
                vf[0] &= keep0;
                vf[1] &= keep0;
                vf[2] &= keep1;
                vf[3] &= keep1;
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) mma16816(o[mt][nb], vf, pf[nb]);
        }
        __syncwarp();                                 // every lane has read the stage
        if (issued < count) {
            issue(stage);
            ++issued;
            advance(pro, issued < count);
        }
        if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
        }

        const bool item_end = con.c.unit + 1 == con.c.units;
        if (item_end || u + 1 == count) {
            fresh = true;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) l[nb][e] += __shfl_xor_sync(0xffffffffu, l[nb][e], d);
                    if (bad) l[nb][e] = __int_as_float(0x7fc00000);
                }
            const int row0 = con.c.tile * RB, rows = min(RB, con.c.q.rows - row0);
            if (first_unit == 0 && item_end) {
                __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + (size_t)((con.c.head * team + mate) * a.g) * HD;
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (nb * 8 + 2 * (lane & 3) + e >= rows) continue;
                        const float inv = 1.f / l[nb][e];
#pragma unroll
                        for (int mt = 0; mt < HD / 16; ++mt) {
                            out[out_at[nb][e] + mt * 16] = __float2bfloat16_rn(o[mt][nb][e] * inv);
                            out[out_at[nb][e] + mt * 16 + 8] = __float2bfloat16_rn(o[mt][nb][2 + e] * inv);
                        }
                    }
            } else {
                Part<HD, NB>& p = part[(2 * w + (first_unit == 0 ? 1 : 0)) * team + mate];
#pragma unroll
                for (int mt = 0; mt < HD / 16; ++mt)
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
                        p.o[mt][nb][lane] = make_float4(o[mt][nb][0], o[mt][nb][1], o[mt][nb][2], o[mt][nb][3]);
                if (lane < 4)
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            p.m[nb * 8 + 2 * lane + e] = m[nb][e];
                            p.l[nb * 8 + 2 * lane + e] = l[nb][e];
                        }
                if (first_unit == 0 && mate == 0 && lane == 0) {
                    // the item's last unit is (units - 1) behind its first, which is u - unit
                    const long long last = u0 + u - con.c.unit + con.c.units - 1;
                    PagedDesc d;
                    d.pieces = (int)div_ll(last, stretch) - w + 1;
                    d.start = con.c.q.start;
                    d.row0 = row0;
                    d.rows = rows;
                    d.kvh = con.c.head * team;
                    desc[w] = d;
                }
            }
        }
        new_tile = advance(con, u + 1 < count);
    }
    if (!alive) {
        // the copies still in flight land (or the bound ends) before the memory goes away
        const int n = min(STAGES, issued);
        for (int s = 0; s < n; ++s) {
            const uint32_t ph = (uint32_t)(((issued - 1 - s) / STAGES) & 1);
            const uint32_t bar = bar0 + 8u * (uint32_t)((issued - 1 - s) % STAGES);
            for (uint32_t i = 0; i < DRAIN_POLLS && !bar_try(bar, ph); ++i) __nanosleep(128);
        }
    }
}

// Adds the pieces of the item that team blockIdx.x's stretch ended inside, in key order, in the
// partials' own layout, one CTA per head of the team: each warp takes a quarter of the dims of every
// PARTS-th piece.  The statistics of up to JOIN pieces are fetched by all threads at once and the
// outputs of several pieces are in flight together, so that the chain of dependent loads grows little
// with the pieces.  PARTS: 4 where an item has 8 pieces and more on average (one request over 16000
// tokens, 143 pieces: 31 us, 37 with 2 parts, 49 with 1), else 1 (32 short requests, 1 to 3 pieces:
// 24.7 us, 26.1 with 2 parts, whose larger CTAs take longer to start).
constexpr int JOIN = 64;                              // pieces in shared memory at a time
template <int HD, int NB, int PARTS>
__global__ void __launch_bounds__(128 * PARTS) paged_step_join_kernel(PagedArgs a, const PagedDesc* __restrict__ desc,
                                                              const Part<HD, NB>* __restrict__ part) {
    constexpr int MT = HD / 64;                       // 16-dim tiles of a warp
    __shared__ float sm[JOIN][NB * 8], sl[JOIN][NB * 8];
    __shared__ float so[PARTS > 1 ? PARTS - 1 : 1][MT * NB * 4 + NB * 2][PARTS > 1 ? 128 : 1];
    grid_dep_wait();
    const int w = blockIdx.x, lane = threadIdx.x & 31, of = threadIdx.x >> 7, at = threadIdx.x & 127;
    const int warp = at >> 5;
    const PagedDesc d = desc[w];
    if (d.pieces <= 0) return;
    const int c = 2 * (lane & 3);
    float o[MT][NB][4], m[NB][2], l[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            m[nb][e] = -FLT_MAX;
            l[nb][e] = 0.f;
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[mt][nb][e] = 0.f;
    }
    for (int i0 = 0; i0 < d.pieces; i0 += JOIN) {
        const int n = min(JOIN, d.pieces - i0);
        auto piece = [&](int i) {
            return part + (size_t)(2 * (w + i0 + i) + (i0 + i == 0 ? 1 : 0)) * gridDim.y + blockIdx.y;
        };
        __syncthreads();
        for (int i = threadIdx.x; i < n * NB * 8; i += 128 * PARTS) {
            sm[i / (NB * 8)][i % (NB * 8)] = piece(i / (NB * 8))->m[i % (NB * 8)];
            sl[i / (NB * 8)][i % (NB * 8)] = piece(i / (NB * 8))->l[i % (NB * 8)];
        }
        __syncthreads();
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mn = m[nb][e];
                for (int i = 0; i < n; ++i) mn = fmaxf(mn, sm[i][nb * 8 + c + e]);
                const float f = ex2(m[nb][e] - mn);
                l[nb][e] *= f;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    o[mt][nb][e] *= f;
                    o[mt][nb][e + 2] *= f;
                }
                m[nb][e] = mn;
            }
#pragma unroll 8
        for (int i = of; i < n; i += PARTS) {
            const Part<HD, NB>* p = piece(i);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                float f[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    f[e] = ex2(sm[i][nb * 8 + c + e] - m[nb][e]);
                    l[nb][e] = fmaf(f[e], sl[i][nb * 8 + c + e], l[nb][e]);
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const float4 v = p->o[warp * MT + mt][nb][lane];
                    o[mt][nb][0] = fmaf(f[0], v.x, o[mt][nb][0]);
                    o[mt][nb][1] = fmaf(f[1], v.y, o[mt][nb][1]);
                    o[mt][nb][2] = fmaf(f[0], v.z, o[mt][nb][2]);
                    o[mt][nb][3] = fmaf(f[1], v.w, o[mt][nb][3]);
                }
            }
        }
    }
    if constexpr (PARTS > 1) {                        // the parts have the same maxima: their sums add up
        if (of > 0) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
                for (int e = 0; e < 2; ++e) so[of - 1][MT * NB * 4 + nb * 2 + e][at] = l[nb][e];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) so[of - 1][(mt * NB + nb) * 4 + e][at] = o[mt][nb][e];
            }
        }
        __syncthreads();
        if (of > 0) return;
        for (int p = 0; p < PARTS - 1; ++p)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
                for (int e = 0; e < 2; ++e) l[nb][e] += so[p][MT * NB * 4 + nb * 2 + e][at];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[mt][nb][e] += so[p][(mt * NB + nb) * 4 + e][at];
            }
    }
    float inv[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) inv[nb][e] = 1.f / l[nb][e];
    store_rows<HD, NB, MT>(a, d.start, d.row0, d.rows, d.kvh + blockIdx.y, warp * MT, o, inv, lane);
}

template <int HD, int NB>
cudaError_t launch_step(const PagedArgs& a, cudaStream_t st) {
    CUtensorMap map;
    const int box_rows = min(UK, 1 << a.page_shift);
    if (!paged_cache_map(&map, a, box_rows, HD / 64, 2)) return cudaErrorNotSupported;
    static std::atomic<uint64_t> attr{0};
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
        e = smem_limit(reinterpret_cast<const void*>(paged_step_kernel<HD, NB>), Geo<HD>::SMEM, attr);
    if (e != cudaSuccess) return e;
    const int grid = min(sms, MAX_CTAS), team = min(WARPS, a.Hkv & -a.Hkv);
    PagedDesc* desc = static_cast<PagedDesc*>(a.ws);
    auto* part = reinterpret_cast<Part<HD, NB>*>(static_cast<char*>(a.ws) + MAX_WORKERS * sizeof(PagedDesc));
    paged_step_kernel<HD, NB><<<grid, THREADS, Geo<HD>::SMEM, st>>>(map, a, box_rows, desc, part);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int workers = grid * (WARPS / team);
    const bool many = (long long)a.n_rows * a.line_heads * 8 <= workers;
    return launch_pdl(many ? paged_step_join_kernel<HD, NB, 4> : paged_step_join_kernel<HD, NB, 1>,
                      dim3(workers, team), dim3(many ? 512 : 128), 0, st, a,
                      static_cast<const PagedDesc*>(desc), static_cast<const Part<HD, NB>*>(part));
}

}  // namespace

size_t paged_step_workspace(int hd) {
    const size_t p = hd == 128 ? sizeof(Part<128, 2>) : sizeof(Part<64, 2>);
    return MAX_WORKERS * (sizeof(PagedDesc) + 2 * p);
}

bool paged_tc_supported(const PagedArgs& a) {
    const uintptr_t mix = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.cache) |
                          reinterpret_cast<uintptr_t>(a.out);
    return a.dtype == E_BF16 && (a.hd == 64 || a.hd == 128) && a.g <= 128 && mix % 16 == 0 &&
           a.ld_q % 8 == 0 && a.ld_out % 8 == 0;
}

cudaError_t launch_paged_step(PagedArgs a, cudaStream_t st) {
    if (a.n_tokens <= 0 || a.n_rows <= 0) return cudaSuccess;
    a.line_heads = a.Hkv / min(WARPS, a.Hkv & -a.Hkv);
    const bool one = (long long)a.max_new * a.g <= 8;
    if (a.hd == 128) return one ? launch_step<128, 1>(a, st) : launch_step<128, 2>(a, st);
    return one ? launch_step<64, 1>(a, st) : launch_step<64, 2>(a, st);
}

int paged_step_error_word() {
    int v = 0;
    const int zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_step_error, sizeof(int)) != cudaSuccess) return -1;
    cudaMemcpyToSymbol(g_step_error, &zero, sizeof(int));
    return v;
}

}  // namespace zo
