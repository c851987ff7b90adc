// The paged key/value cache of served requests: block tables and slot maps from request
// lengths, the cache write, and the CUDA-core attention over the pages (fp32, and the head
// sizes the tensor-core kernels do not take).
#include <float.h>

#include <type_traits>

#include "paged.cuh"

namespace zo {

namespace {

// ---- block tables and slot maps -----------------------------------------------------------
// Integers only: grow_r = max(0, ceil(new_r / P) - ceil(old_r / P)) pages are taken from the
// ring at head + sum_{i < r} grow_i, drop_r (the reverse difference) go back at head + count +
// sum_{i < r} drop_i.  The state is read from one array and written to another, pages given back
// land behind the pages that can be taken, and a new page's id is read from the ring wherever it
// is needed: so no CTA waits for another, and one launch does the whole step.  Every CTA sums the
// lengths of all requests itself (a few KB from L2) and then serves its own few requests.  The
// work is a few bytes a token: launch and one or two dependent loads bound it (64 requests 4.2 us, 509
// requests with 59000 new tokens 6.3 us).
constexpr int BT_THREADS = 256;

struct Sum3 {
    long long grow, drop, toks;
};
__device__ __forceinline__ Sum3 add3(Sum3 a, Sum3 b) {
    return {a.grow + b.grow, a.drop + b.drop, a.toks + b.toks};
}

__global__ void __launch_bounds__(BT_THREADS)
    block_tables_kernel(const int* __restrict__ old_lens, const int* __restrict__ new_lens, int R,
                        int shift, int* __restrict__ table, int max_blocks, int* ring, int n_pages,
                        const int* __restrict__ state, int* __restrict__ state_out,
                        int* __restrict__ cu_new, int* __restrict__ slots, int max_tokens,
                        int rows_per_cta) {
    __shared__ long long red[BT_THREADS / 32][6];
    __shared__ int bad_s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int P = 1 << shift;
    const int head = state[0], count = state[1];
    const int r0 = blockIdx.x * rows_per_cta;
    const int r1 = min(R, r0 + rows_per_cta);
    if (tid == 0) bad_s = 0;
    __syncthreads();
    // sums over the requests before this CTA's, and over all of them
    const long long cap = (long long)max_blocks << shift;
    auto diff = [&](int o, int n) {
        Sum3 d;
        const long long a = ((long long)o + P - 1) >> shift, b = ((long long)n + P - 1) >> shift;
        d.grow = b > a ? b - a : 0;
        d.drop = a > b ? a - b : 0;
        d.toks = n > o ? (long long)n - o : 0;
        return d;
    };
    Sum3 before = {0, 0, 0}, all = {0, 0, 0};
    bool bad = false;
    for (int r = tid; r < R; r += BT_THREADS) {
        const int o = old_lens[r], n = new_lens[r];
        bad |= o < 0 || n < 0 || o > cap || n > cap;
        const Sum3 d = diff(o, n);
        all = add3(all, d);
        if (r < r0) before = add3(before, d);
    }
    if (bad) bad_s = 1;
    long long v[6] = {before.grow, before.drop, before.toks, all.grow, all.drop, all.toks};
#pragma unroll
    for (int i = 0; i < 6; ++i) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        if (lane == 0) red[warp][i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 6; ++i) {
        v[i] = 0;
        for (int w = 0; w < BT_THREADS / 32; ++w) v[i] += red[w][i];
    }
    int status = 0;
    if (head < 0 || head >= n_pages || count < 0 || count > n_pages) status = -4;
    else if (bad_s) status = -1;
    else if (v[5] > max_tokens) status = -2;
    else if (count + v[4] > n_pages) status = -3;
    else if (v[3] > count) status = (int)min(v[3] - count, 0x7fffffffll);
    const int total = status ? 0 : (int)v[5];
    if (blockIdx.x == 0 && tid == 0) {
        state_out[0] = status ? head : (int)((head + v[3]) % n_pages);
        state_out[1] = status ? count : (int)(count - v[3] + v[4]);
        state_out[2] = status;
        state_out[3] = 0;
        cu_new[R] = total;
    }
    // slots behind the last new token
    for (long long t = total + (long long)blockIdx.x * BT_THREADS + tid; t < max_tokens;
         t += (long long)gridDim.x * BT_THREADS)
        slots[t] = -1;
    if (status) {
        for (int r = r0 + tid; r < r1; r += BT_THREADS) cu_new[r] = 0;
        return;
    }
    Sum3 at = {v[0], v[1], v[2]};
    for (int r = r0; r < r1; ++r) {
        const int o = old_lens[r], n = new_lens[r];
        const Sum3 d = diff(o, n);
        const int have = (int)(((long long)o + P - 1) >> shift);
        const int want = (int)(((long long)n + P - 1) >> shift);
        int* row = table + (size_t)r * max_blocks;
        if (tid == 0) cu_new[r] = (int)at.toks;
        auto taken = [&](int j) { return ring[(head + at.grow + (j - have)) % n_pages]; };
        for (int j = have + tid; j < want; j += BT_THREADS) row[j] = taken(j);
        for (int j = want + tid; j < have; j += BT_THREADS)
            ring[(head + count + at.drop + (j - want)) % n_pages] = row[j];
        for (int i = tid; i < (int)d.toks; i += BT_THREADS) {
            const int pos = o + i, j = pos >> shift;
            const int page = j < have ? row[j] : taken(j);
            slots[at.toks + i] = page * P + (pos & (P - 1));
        }
        at = add3(at, d);
    }
}

// ---- cache write ---------------------------------------------------------------------------
// One CTA per packed row: its k|v columns go to the row's slot.  A copy: bound by HBM (9001 rows of
// 20 KB: 59.4 us, 6.2 TB/s, 0.96 of the measured rate).
constexpr int KW_THREADS = 256;

template <typename V>
__global__ void __launch_bounds__(KW_THREADS)
    kv_write_kernel(const char* __restrict__ kv, size_t ld_bytes, const int* __restrict__ slots,
                    char* __restrict__ cache, long long n_slots, int row_bytes) {
    const int t = blockIdx.x;
    const int slot = slots[t];
    if (slot < 0 || slot >= n_slots) return;
    const V* s = reinterpret_cast<const V*>(kv + (size_t)t * ld_bytes);
    V* d = reinterpret_cast<V*>(cache + (size_t)slot * row_bytes);
    for (int i = threadIdx.x; i < row_bytes / (int)sizeof(V); i += KW_THREADS) d[i] = s[i];
}

// ---- attention over the pages, CUDA cores ----------------------------------------------------
// A work item is (tile of 64 query rows of one request, kv head).  A request's query rows for a kv
// head are its new tokens times the g query heads that share the head, token-major: row i is token
// i / g, head kvh * g + i % g.  Keys stream through shared memory in chunks of 64 with an online
// softmax in fp32; keys a row may not see get probability 0 and value rows behind the request's
// end are staged as zeros, so what lies there is never part of a result.  The chunks of all items
// form one line, cut into equal stretches, one per CTA that fits on the SMs; an item cut by a
// stretch's end is written as partial (m, l, o) and joined by a second kernel in key order.  The
// stretches are equal in time, not in chunks: a chunk of a tile of n rows weighs 3 + ceil(n / 8), as
// measured for head_dim 64 and 128 (8 rows take 0.35-0.45 of 64 rows' time, 32 rows 0.65; a mixed batch
// of 7 requests took 91 us with equal numbers of chunks, 71 with equal weights).
// fp32's floor is the FMA rate.  With 64 rows the FMA pipe is 56 % busy (issue slots 44 %): the rest
// are the pairs of P that fma.f32x2 wants twice, the softmax and waits that 16 warps an SM at 128
// registers do not cover.  7 requests of 105-515 tokens, 1-93 of them new, 32 heads of 64: 69 us.
constexpr int AQ = 64, AK = 64, A_THREADS = 256;
constexpr int RT = 4;                      // query rows of a thread, 16 threads side by side on 64 keys
constexpr int A_GROUPS = 1024;             // prefix entries, in the chunk buffers before their use
using Line = PagedLine<false, AQ, AK, 3>;

// Floats of a partial result: o [AQ][hd], m [AQ], l [AQ].
__host__ __device__ constexpr int part_floats(int hd) { return AQ * (hd + 2); }
// CTAs on an SM: by the registers, and the chunk buffers of the wide heads
constexpr int paged_ctas(int hd) { return 148 * (hd <= 64 ? 2 : 1); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// two fp32 operations to an instruction, each rounded as by itself
__device__ __forceinline__ uint64_t pair_of(float v) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ void fma_pair(uint64_t& acc, uint64_t a, uint64_t b) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float half_of(uint64_t v, int i) {
    return __uint_as_float((unsigned)(i ? v >> 32 : v));
}

// chunks of keys and values in shared memory: two where they fit and come by themselves
template <int HD, bool FAST>
constexpr int paged_stages() { return FAST && HD <= 128 ? 2 : 1; }

// Bytes `bytes` of 16 (the rest zeros) to shared memory, asynchronously.
__device__ __forceinline__ void copy16(void* dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src), "r"(bytes)
                 : "memory");
}

// FAST: fp32 with 16-byte rows: keys and values come by asynchronous 16-byte copies, the next
// chunk's beside the work on this one; otherwise element by element.
template <int HD, bool FAST>
__global__ void __launch_bounds__(A_THREADS, HD <= 64 ? 2 : 1)
    paged_attention_kernel(PagedArgs a, PagedDesc* __restrict__ desc, float* __restrict__ part) {
    extern __shared__ __align__(16) float sm[];
    constexpr int LD = HD + 4;             // padded rows: 16-byte reads without bank clashes
    constexpr int STAGES = paged_stages<HD, FAST>();
    constexpr int PLD = AK + 4;
    float* Qs = sm;                        // [AQ][LD]
    float* Ps = Qs + AQ * LD;              // [AQ][PLD]
    float* KVs = Ps + AQ * PLD;            // [STAGES][2][AK][LD]
    __shared__ int bad_s;
    // 16 threads of the same parity in a warp share their rows: neighbouring lanes then read the same
    // keys and values, and a 16-byte read of a warp takes half the passes
    const int tid = threadIdx.x, tx = (tid >> 1) & 15, ty = 2 * (tid >> 5) + (tid & 1);
    grid_dep_launch();
    long long* cum = reinterpret_cast<long long*>(KVs);
    const long long L = Line::prefix(a, A_GROUPS, cum, cum + A_GROUPS + 1);
    const int w = blockIdx.x;
    const long long stretch = max(div_ll(L + gridDim.x - 1, gridDim.x), (long long)Line::WMAX);
    const long long u1 = min(L, stretch * (w + 1));
    long long u = stretch * w;
    if (tid == 0) desc[w].pieces = 0;
    if (u >= u1) return;
    Line::Cursor k = Line::locate(a, A_GROUPS, cum, u);
    if (u >= u1) return;                   // no unit begins here
    if (k.unit == k.units) Line::advance(a, k, 0, true);

    const float sl2 = a.scale * 1.4426950408889634f;      // scores in units of ln 2
    const int n_pages = (int)(a.n_slots >> a.page_shift);
    const size_t ldc = (size_t)2 * a.Hkv * HD;
    constexpr int PER = HD / 4;            // a chunk's keys and values: 4 threads to a row
    const int jr = tid >> 2, lane_col = (tid & 3) * PER;
    // output dims of a thread: VW at tx * VW + 16 VW * i
    constexpr int VW = HD >= 64 ? 4 : 2, NV = HD / (16 * VW);
    while (u < u1) {
        const int row0 = k.tile * AQ, rows = min(AQ, k.q.rows - row0), kvh = k.head;
        const int wt = Line::weight(k.q, k.tile);
        const int first = k.unit, chunks = (int)min((long long)k.units, k.unit + div_ll(u1 - u + wt - 1, wt));
        const int kend = Line::keys(a, k.q, row0 + AQ);
        const int* table = a.block_table + (size_t)k.r * a.max_blocks;
        __syncthreads();                   // what the piece before (or the search) read is free
        if (tid == 0) bad_s = 0;
        __syncthreads();
        // the page of the thread's row in the next chunk to load, fetched a chunk ahead
        auto page_at = [&](int c) { return c * AK + jr < kend ? table[(c * AK + jr) >> a.page_shift] : 0; };
        int next_page = page_at(first);
        auto load = [&](int c) {
            float* kd = KVs + (size_t)(c % STAGES) * 2 * AK * LD + jr * LD + lane_col;
            float* vd = kd + AK * LD;
            const int pos = c * AK + jr;
            const int page = next_page;
            next_page = page_at(c + 1);
            size_t b = 0;
            bool live = false;
            if (pos < kend) {
                live = (unsigned)page < (unsigned)n_pages;
                if (!live) bad_s = 1;
                else
                    b = (((size_t)page << a.page_shift) + (pos & ((1 << a.page_shift) - 1))) * ldc +
                        (size_t)kvh * HD + lane_col;
            }
            if (FAST) {
                const float* src = static_cast<const float*>(a.cache) + b;
#pragma unroll
                for (int d = 0; d < PER; d += 4) {
                    copy16(kd + d, src + d, live ? 16 : 0);
                    copy16(vd + d, src + (live ? (size_t)a.Hkv * HD : 0) + d, live ? 16 : 0);
                }
            } else {
                for (int d = 0; d < PER; ++d) {
                    kd[d] = live ? ld_elem(a.cache, b + d, a.dtype) : 0.f;
                    vd[d] = live ? ld_elem(a.cache, b + (size_t)a.Hkv * HD + d, a.dtype) : 0.f;
                }
            }
        };
        if (STAGES > 1) load(first);
        // few rows: 2 or 4 groups of warps, each with all rows and its part of every chunk's keys
        const int groups = rows > AQ / 2 ? 1 : rows > AQ / 4 ? 2 : 4, span = AQ / groups;
        const int kg = ty * RT / span, r0 = RT * ty - kg * span;      // the thread's keys and rows
        for (int i = tid; i < span * HD; i += A_THREADS) {
            const int q = i / HD, d = i % HD;
            float v = 0.f;
            if (q < rows) {
                const int t = by_g(a, row0 + q), h = kvh * a.g + mod_g(a, row0 + q);
                v = ld_elem(a.q, (size_t)(k.q.start + t) * a.ld_q + (size_t)h * HD + d, a.dtype) * sl2;
            }
            Qs[q * LD + d] = v;
        }
        float m[RT], l[RT];
        uint64_t o[RT][NV][VW / 2];        // pairs of neighbouring dims
        int lim[RT];                       // keys below lim are seen by the thread's rows
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            m[i] = -FLT_MAX;
            l[i] = 0.f;
            lim[i] = min(kend, k.q.ctx + by_g(a, row0 + r0 + i) + 1);
#pragma unroll
            for (int d = 0; d < NV; ++d)
#pragma unroll
                for (int e = 0; e < VW / 2; ++e) o[i][d][e] = 0ull;
        }
        // a warp's rows past the tile's take no part in the products
        const bool warp_live = (r0 & ~(2 * RT - 1)) < rows;

        // a chunk for the thread's 16 NJ keys
        auto attend = [&](int c, auto nj) {
            constexpr int NJ = decltype(nj)::value;
            const int key0 = 16 * NJ * kg;
            const float* Ks = KVs + (size_t)(c % STAGES) * 2 * AK * LD;
            const float* Vs = Ks + AK * LD;
            float s[RT][NJ];
            {
                uint64_t s2[RT][NJ];        // sums over the even and over the odd dims
#pragma unroll
                for (int i = 0; i < RT; ++i)
#pragma unroll
                    for (int j = 0; j < NJ; ++j) s2[i][j] = 0ull;
#pragma unroll 4
                for (int d = 0; d < HD; d += 4) {
                    ulonglong2 qv[RT], kv[NJ];
#pragma unroll
                    for (int i = 0; i < RT; ++i)
                        qv[i] = *reinterpret_cast<const ulonglong2*>(Qs + (r0 + i) * LD + d);
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
                        kv[j] = *reinterpret_cast<const ulonglong2*>(Ks + (key0 + tx + 16 * j) * LD + d);
#pragma unroll
                    for (int i = 0; i < RT; ++i)
#pragma unroll
                        for (int j = 0; j < NJ; ++j) {
                            fma_pair(s2[i][j], qv[i].x, kv[j].x);
                            fma_pair(s2[i][j], qv[i].y, kv[j].y);
                        }
                }
#pragma unroll
                for (int i = 0; i < RT; ++i)
#pragma unroll
                    for (int j = 0; j < NJ; ++j) s[i][j] = half_of(s2[i][j], 0) + half_of(s2[i][j], 1);
            }
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                bool see[NJ];
                float mx = -FLT_MAX;
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    see[j] = c * AK + key0 + tx + 16 * j < lim[i];
                    if (see[j]) mx = fmaxf(mx, s[i][j]);
                }
#pragma unroll
                for (int x = 16; x > 1; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
                const float mn = fmaxf(m[i], mx);
                const float corr = ex2(m[i] - mn);
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    const float p = see[j] ? ex2(s[i][j] - mn) : 0.f;
                    sum += p;
                    Ps[(r0 + i) * PLD + key0 + tx + 16 * j] = p;
                }
#pragma unroll
                for (int x = 16; x > 1; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
                l[i] = l[i] * corr + sum;
                m[i] = mn;
                const uint64_t cc = pair_of(corr);
#pragma unroll
                for (int d = 0; d < NV; ++d)
#pragma unroll
                    for (int e = 0; e < VW / 2; ++e) o[i][d][e] = mul_pair(o[i][d][e], cc);
            }
            __syncwarp();                  // a row's P is written and read by one warp
            const int keys = min(key0 + 16 * NJ, kend - c * AK);
#pragma unroll 2
            for (int j0 = key0; j0 < keys; j0 += 4) {       // (P and V behind the last key are zeros)
                uint64_t pe[RT][4];
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    const float4 t = *reinterpret_cast<const float4*>(Ps + (r0 + i) * PLD + j0);
                    pe[i][0] = pair_of(t.x); pe[i][1] = pair_of(t.y);
                    pe[i][2] = pair_of(t.z); pe[i][3] = pair_of(t.w);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int d = 0; d < NV; ++d) {
                        uint64_t v[VW / 2];
                        const float* src = Vs + (j0 + j) * LD + tx * VW + 16 * VW * d;
                        if constexpr (VW == 4) {
                            const ulonglong2 t = *reinterpret_cast<const ulonglong2*>(src);
                            v[0] = t.x; v[1] = t.y;
                        } else {
                            v[0] = *reinterpret_cast<const uint64_t*>(src);
                        }
#pragma unroll
                        for (int e = 0; e < VW / 2; ++e)
#pragma unroll
                            for (int i = 0; i < RT; ++i) fma_pair(o[i][d][e], pe[i][j], v[e]);
                    }
            }
            __syncwarp();
        };

        for (int c = first; c < chunks; ++c) {
            if (STAGES == 1) {
                __syncthreads();
                load(c);
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncthreads();               // chunk c is there; chunk c - 1 has been read
            if (STAGES > 1 && c + 1 < chunks) load(c + 1);
            if (!warp_live) continue;
            if (groups == 1) attend(c, std::integral_constant<int, 4>());
            else if (groups == 2) attend(c, std::integral_constant<int, 2>());
            else attend(c, std::integral_constant<int, 1>());
        }
        __syncthreads();                   // bad_s is final
        const bool bad = k.q.bad || bad_s;
        if (groups > 1) {                  // the groups' partial results into the first one's
            float* os = KVs;               // [groups - 1][span][LD], then their m and l
            float* ms = os + (size_t)(AQ - span) * LD;
            if (kg > 0 && warp_live) {
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    const int at = (kg - 1) * span + r0 + i;
#pragma unroll
                    for (int d = 0; d < NV; ++d)
#pragma unroll
                        for (int e = 0; e < VW / 2; ++e)
                            *reinterpret_cast<uint64_t*>(os + at * LD + tx * VW + 16 * VW * d + 2 * e) = o[i][d][e];
                    if (tx == 0) {
                        ms[at] = m[i];
                        ms[AQ + at] = l[i];
                    }
                }
            }
            __syncthreads();
            if (kg == 0 && warp_live) {
                for (int x = 0; x < groups - 1; ++x)
#pragma unroll
                    for (int i = 0; i < RT; ++i) {
                        const int at = x * span + r0 + i;
                        const float mn = fmaxf(m[i], ms[at]), f = ex2(m[i] - mn), f2 = ex2(ms[at] - mn);
                        m[i] = mn;
                        l[i] = fmaf(l[i], f, ms[AQ + at] * f2);
                        const uint64_t ff = pair_of(f), ff2 = pair_of(f2);
#pragma unroll
                        for (int d = 0; d < NV; ++d)
#pragma unroll
                            for (int e = 0; e < VW / 2; ++e) {
                                uint64_t t = mul_pair(o[i][d][e], ff);
                                fma_pair(t, ff2, *reinterpret_cast<const uint64_t*>(os + at * LD + tx * VW +
                                                                                    16 * VW * d + 2 * e));
                                o[i][d][e] = t;
                            }
                    }
            }
        }
        const bool whole = first == 0 && chunks == k.units;
        float* p = part + (size_t)(2 * w + (first == 0 ? 1 : 0)) * part_floats(HD);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int q = r0 + i;
            if (kg > 0 || q >= rows) continue;
            if (bad) l[i] = __int_as_float(0x7fc00000);
            if (!whole && tx == 0) {
                p[AQ * HD + q] = m[i];
                p[AQ * HD + AQ + q] = l[i];
            }
            const int t = by_g(a, row0 + q), h = kvh * a.g + mod_g(a, row0 + q);
            const size_t out = (size_t)(k.q.start + t) * a.ld_out + (size_t)h * HD;
            const float inv = 1.f / l[i];
#pragma unroll
            for (int d = 0; d < NV; ++d)
#pragma unroll
                for (int e = 0; e < VW; ++e) {
                    const int col = tx * VW + 16 * VW * d + e;
                    const float v = half_of(o[i][d][e / 2], e & 1);
                    if (whole) st_elem(a.out, out + col, a.dtype, v * inv);
                    else p[q * HD + col] = v;
                }
        }
        if (!whole && first == 0 && tid == 0) {
            PagedDesc d;
            d.pieces = (int)div_ll(u + (long long)(k.units - 1) * wt, stretch) - w + 1;
            d.start = k.q.start;
            d.row0 = row0;
            d.rows = rows;
            d.kvh = kvh;
            desc[w] = d;
        }
        u += (long long)(chunks - first) * wt;
        Line::advance(a, k, chunks - first, u < u1);
    }
}

// Adds the pieces of the item that CTA blockIdx.x's stretch ended inside, in key order: 4 dims of a
// row per thread and turn.
template <int HD>
__global__ void __launch_bounds__(A_THREADS)
    paged_attention_join_kernel(PagedArgs a, const PagedDesc* __restrict__ desc, const float* __restrict__ part) {
    grid_dep_wait();
    const int w = blockIdx.x;
    const PagedDesc t = desc[w];
    if (t.pieces <= 0) return;
    auto piece = [&](int i) { return part + (size_t)(2 * (w + i) + (i == 0 ? 1 : 0)) * part_floats(HD); };
    constexpr int V = HD / 4;
    for (int i = threadIdx.x; i < t.rows * V; i += A_THREADS) {
        const int q = i / V, d = i % V * 4;
        float m = -FLT_MAX, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int z = 0; z < t.pieces; ++z) m = fmaxf(m, piece(z)[AQ * HD + q]);
#pragma unroll 4
        for (int z = 0; z < t.pieces; ++z) {
            const float* s = piece(z);
            const float f = ex2(s[AQ * HD + q] - m);
            const float4 v = *reinterpret_cast<const float4*>(s + q * HD + d);
            l = fmaf(f, s[AQ * HD + AQ + q], l);
            o[0] = fmaf(f, v.x, o[0]); o[1] = fmaf(f, v.y, o[1]);
            o[2] = fmaf(f, v.z, o[2]); o[3] = fmaf(f, v.w, o[3]);
        }
        const int tok = by_g(a, t.row0 + q), h = t.kvh * a.g + mod_g(a, t.row0 + q);
        for (int e = 0; e < 4; ++e)
            st_elem(a.out, (size_t)(t.start + tok) * a.ld_out + (size_t)h * HD + d + e, a.dtype, o[e] / l);
    }
}

template <int HD, bool FAST>
cudaError_t launch_paged_hd(const PagedArgs& a, cudaStream_t st) {
    const size_t smem = sizeof(float) * (AQ * (HD + 4) + AQ * (AK + 4) +
                                         (size_t)paged_stages<HD, FAST>() * 2 * AK * (HD + 4));
    static_assert(2 * AK * (HD + 4) * 4 >= (A_GROUPS + 1 + A_THREADS / 32) * 8, "room for the prefix sums");
    static std::atomic<uint64_t> attr{0};
    cudaError_t e = smem_limit(reinterpret_cast<const void*>(paged_attention_kernel<HD, FAST>), (int)smem, attr);
    if (e != cudaSuccess) return e;
    const int grid = paged_ctas(HD);
    PagedDesc* desc = static_cast<PagedDesc*>(a.ws);
    float* part = reinterpret_cast<float*>(static_cast<char*>(a.ws) + grid * sizeof(PagedDesc));
    paged_attention_kernel<HD, FAST><<<grid, A_THREADS, smem, st>>>(a, desc, part);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_pdl(paged_attention_join_kernel<HD>, dim3(grid), dim3(A_THREADS), 0, st, a,
                      static_cast<const PagedDesc*>(desc), static_cast<const float*>(part));
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = []() -> EncodeTiledFn {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<EncodeTiledFn>(p);
        return nullptr;
    }();
    return fn;
}

}  // namespace

bool paged_cache_map(CUtensorMap* m, const PagedArgs& a, int rows, int halves, int kvs) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t kv = (cuuint64_t)a.Hkv * a.hd * 2;          // bytes of a row's keys
    const cuuint64_t dims[4] = {64, (cuuint64_t)a.n_slots, (cuuint64_t)(a.Hkv * a.hd / 64), 2};
    const cuuint64_t strides[3] = {2 * kv, 128, kv};
    const cuuint32_t box[4] = {64, (cuuint32_t)rows, (cuuint32_t)halves, (cuuint32_t)kvs};
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(a.cache), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_block_tables(const int* old_lens, const int* new_lens, int R, int page_shift,
                                int* table, int max_blocks, int* ring, int n_pages, const int* state,
                                int* state_out, int* cu_new, int* slots, int max_tokens,
                                cudaStream_t st) {
    // a CTA per request up to 4 per SM; above that each CTA takes several requests, so that the
    // lengths are not summed by more CTAs than run at once (592 requests of 100 new tokens: 6.2 us, 8.3
    // with several a CTA; 1200: 8.2 and 12.4 with one; 4096: 16.4 and 55.4)
    const int rows_per_cta = R <= 592 ? 1 : (R + 591) / 592;
    const int grid = R > 0 ? (R + rows_per_cta - 1) / rows_per_cta : 1;
    block_tables_kernel<<<grid, BT_THREADS, 0, st>>>(old_lens, new_lens, R, page_shift, table, max_blocks,
                                                     ring, n_pages, state, state_out, cu_new, slots,
                                                     max_tokens, rows_per_cta);
    return cudaGetLastError();
}

cudaError_t launch_kv_write(const void* kv, long long ld_bytes, const int* slots, int n_tokens,
                            void* cache, long long n_slots, int row_bytes, cudaStream_t st) {
    if (n_tokens <= 0) return cudaSuccess;
    const char* s = static_cast<const char*>(kv);
    char* c = static_cast<char*>(cache);
    const uintptr_t mix = reinterpret_cast<uintptr_t>(kv) | reinterpret_cast<uintptr_t>(cache) |
                          (uintptr_t)ld_bytes | (uintptr_t)row_bytes;
    if (mix % 16 == 0)
        kv_write_kernel<uint4><<<n_tokens, KW_THREADS, 0, st>>>(s, ld_bytes, slots, c, n_slots, row_bytes);
    else
        kv_write_kernel<uint16_t><<<n_tokens, KW_THREADS, 0, st>>>(s, ld_bytes, slots, c, n_slots, row_bytes);
    return cudaGetLastError();
}

size_t paged_attention_workspace(int hd) {
    return paged_ctas(hd) * (sizeof(PagedDesc) + (size_t)2 * part_floats(hd) * sizeof(float));
}

cudaError_t launch_paged_attention(PagedArgs a, cudaStream_t st) {
    if (a.n_tokens <= 0 || a.n_rows <= 0) return cudaSuccess;
    a.line_heads = a.Hkv;
    a.step_tokens = 0x7fffffff;            // every request
    const bool fast = a.dtype == E_F32 && reinterpret_cast<uintptr_t>(a.cache) % 16 == 0;
    switch (a.hd) {
        case 32: return fast ? launch_paged_hd<32, true>(a, st) : launch_paged_hd<32, false>(a, st);
        case 64: return fast ? launch_paged_hd<64, true>(a, st) : launch_paged_hd<64, false>(a, st);
        case 128: return fast ? launch_paged_hd<128, true>(a, st) : launch_paged_hd<128, false>(a, st);
        case 256: return fast ? launch_paged_hd<256, true>(a, st) : launch_paged_hd<256, false>(a, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace zo
