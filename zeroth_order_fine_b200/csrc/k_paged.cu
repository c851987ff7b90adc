// The paged key/value cache of served requests: block tables and slot maps from request
// lengths, the cache write, and the CUDA-core attention over the pages (fp32, and the head
// sizes the tensor-core kernels do not take).
#include <float.h>

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
// work is a few bytes a token: launch and one or two dependent loads bound it.
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
// One CTA per packed row: its k|v columns go to the row's slot.  A copy: bound by HBM.
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
// One CTA per (tile of 32 query rows of one request, kv head).  A request's query rows for a kv
// head are its new tokens times the g query heads that share the head, token-major: row i is token
// i / g, head kvh * g + i % g.  Keys stream through shared memory in chunks of 64 with an online
// softmax in fp32; keys a row may not see get probability 0 and value rows behind the request's
// end are staged as zeros, so what lies there is never part of a result.
constexpr int AQ = 32, AK = 64, A_THREADS = 256;

struct TileAt {
    int req, tile;                         // request and its tile, or req < 0: past the last
};

// Request and tile of the i-th tile, when request r has ceil(n_r * g / rows) of them.  All
// threads of the block take part; the answer is in shared memory (out).
__device__ __forceinline__ int tile_count(const PagedArgs& a, int r, int rows) {
    const int s = a.cu_new[r], e = a.cu_new[r + 1];
    if (s < 0 || e < s || e > a.n_tokens) return 0;
    return (int)(((long long)(e - s) * a.g + rows - 1) / rows);
}

__device__ __forceinline__ void find_tile(const PagedArgs& a, int i, int rows, TileAt* out,
                                          int* wsum) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
    if (tid == 0) out->req = -1;
    int base = 0;
    for (int r0 = 0; r0 < a.n_rows; r0 += blockDim.x) {
        __syncthreads();                   // wsum free, out written
        const int r = r0 + tid;
        const int c = r < a.n_rows ? tile_count(a, r, rows) : 0;
        int incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        if (lane == 31) wsum[warp] = incl;
        __syncthreads();
        int total = 0, before = 0;
        for (int w = 0; w < nw; ++w) {
            if (w < warp) before += wsum[w];
            total += wsum[w];
        }
        const int excl = base + before + incl - c;
        if (c > 0 && i >= excl && i < excl + c) {
            out->req = r;
            out->tile = i - excl;
        }
        base += total;
        if (i < base) break;               // uniform: every thread has the same base
    }
    __syncthreads();
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
__global__ void __launch_bounds__(A_THREADS) paged_attention_kernel(PagedArgs a) {
    extern __shared__ __align__(16) float sm[];
    constexpr int LD = HD + 4;             // padded rows: 16-byte reads without bank clashes
    constexpr int STAGES = paged_stages<HD, FAST>();
    constexpr int PLD = AK + 4;
    float* Qs = sm;                        // [AQ][LD]
    float* Ps = Qs + AQ * LD;              // [AQ][PLD]
    float* KVs = Ps + AQ * PLD;            // [STAGES][2][AK][LD]
    __shared__ TileAt at;
    __shared__ int wsum[A_THREADS / 32];
    __shared__ int bad_s;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    if (tid == 0) bad_s = 0;
    find_tile(a, blockIdx.x, AQ, &at, wsum);   // (synchronises the block)
    if (at.req < 0) return;
    const int r = at.req, kvh = blockIdx.y;
    const int start = a.cu_new[r], n = a.cu_new[r + 1] - start, len = a.lens[r];
    const int row0 = at.tile * AQ;
    const int rows = min(AQ, (int)min((long long)n * a.g - row0, (long long)AQ));
    const bool bad_len = len < n || (long long)len > ((long long)a.max_blocks << a.page_shift);
    const int* table = a.block_table + (size_t)r * a.max_blocks;
    const int n_pages = (int)(a.n_slots >> a.page_shift);
    const int ctx = len - n;
    // the last key any row of the tile sees, plus one
    const int kend = bad_len ? 0 : ctx + (row0 + rows - 1) / a.g + 1;
    const size_t ldc = (size_t)2 * a.Hkv * HD;
    const int chunks = (kend + AK - 1) / AK;

    // a chunk's keys and values: 4 threads to a row
    constexpr int PER = HD / 4;            // elements of a thread
    const int jr = tid >> 2, part = (tid & 3) * PER;
    auto load = [&](int c) {
        float* kd = KVs + (size_t)(c % STAGES) * 2 * AK * LD + jr * LD + part;
        float* vd = kd + AK * LD;
        const int pos = c * AK + jr;
        size_t b = 0;
        bool live = false;
        if (pos < kend) {
            const int page = table[pos >> a.page_shift];
            live = (unsigned)page < (unsigned)n_pages;
            if (!live) bad_s = 1;
            else
                b = (((size_t)page << a.page_shift) + (pos & ((1 << a.page_shift) - 1))) * ldc +
                    (size_t)kvh * HD + part;
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
    if (STAGES > 1 && chunks > 0) load(0);
    for (int i = tid; i < AQ * HD; i += A_THREADS) {
        const int q = i / HD, d = i % HD;
        float v = 0.f;
        if (q < rows) {
            const int t = (row0 + q) / a.g, h = kvh * a.g + (row0 + q) % a.g;
            v = ld_elem(a.q, (size_t)(start + t) * a.ld_q + (size_t)h * HD + d, a.dtype) * a.scale;
        }
        Qs[q * LD + d] = v;
    }
    // output dims of a thread: V at tx * VW + 16 VW * i
    constexpr int VW = HD >= 64 ? 4 : 2, NV = HD / (16 * VW);
    float m[2] = {-FLT_MAX, -FLT_MAX}, l[2] = {0.f, 0.f}, o[2][NV][VW];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int d = 0; d < NV; ++d)
#pragma unroll
            for (int e = 0; e < VW; ++e) o[i][d][e] = 0.f;
    int lim[2];                            // keys below lim are seen by the thread's rows
#pragma unroll
    for (int i = 0; i < 2; ++i) lim[i] = min(kend, ctx + (row0 + 2 * ty + i) / a.g + 1);
    // a warp's rows past the tile's take no part in the products
    const bool warp_live = 4 * (tid >> 5) < rows;

    for (int c = 0; c < chunks; ++c) {
        if (STAGES == 1) {
            __syncthreads();
            load(c);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();                   // chunk c is there; chunk c - 1 has been read
        if (STAGES > 1 && c + 1 < chunks) load(c + 1);
        const float* Ks = KVs + (size_t)(c % STAGES) * 2 * AK * LD;
        const float* Vs = Ks + AK * LD;
        if (!warp_live) continue;
        float s[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
        for (int d = 0; d < HD; d += 4) {
            float4 qv[2], kv[4];
#pragma unroll
            for (int i = 0; i < 2; ++i) qv[i] = *reinterpret_cast<const float4*>(Qs + (2 * ty + i) * LD + d);
#pragma unroll
            for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4*>(Ks + (tx + 16 * j) * LD + d);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = fmaf(qv[i].x, kv[j].x, s[i][j]);
                    s[i][j] = fmaf(qv[i].y, kv[j].y, s[i][j]);
                    s[i][j] = fmaf(qv[i].z, kv[j].z, s[i][j]);
                    s[i][j] = fmaf(qv[i].w, kv[j].w, s[i][j]);
                }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            bool see[4];
            float mx = -FLT_MAX;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                see[j] = c * AK + tx + 16 * j < lim[i];
                if (see[j]) mx = fmaxf(mx, s[i][j]);
            }
#pragma unroll
            for (int w = 8; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
            const float mn = fmaxf(m[i], mx);
            const float corr = expf(m[i] - mn);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = see[j] ? expf(s[i][j] - mn) : 0.f;
                sum += p;
                Ps[(2 * ty + i) * PLD + tx + 16 * j] = p;
            }
#pragma unroll
            for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
            l[i] = l[i] * corr + sum;
            m[i] = mn;
#pragma unroll
            for (int d = 0; d < NV; ++d)
#pragma unroll
                for (int e = 0; e < VW; ++e) o[i][d][e] *= corr;
        }
        __syncwarp();                      // a row's P is written and read by one half-warp
        const int keys = min(AK, kend - c * AK);
#pragma unroll 2
        for (int j0 = 0; j0 < keys; j0 += 4) {       // (P and V behind the last key are zeros)
            float4 pv[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) pv[i] = *reinterpret_cast<const float4*>(Ps + (2 * ty + i) * PLD + j0);
            const float pe[2][4] = {{pv[0].x, pv[0].y, pv[0].z, pv[0].w}, {pv[1].x, pv[1].y, pv[1].z, pv[1].w}};
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int d = 0; d < NV; ++d) {
                    float v[VW];
                    const float* src = Vs + (j0 + j) * LD + tx * VW + 16 * VW * d;
                    if constexpr (VW == 4) {
                        const float4 t = *reinterpret_cast<const float4*>(src);
                        v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
                    } else {
                        const float2 t = *reinterpret_cast<const float2*>(src);
                        v[0] = t.x; v[1] = t.y;
                    }
#pragma unroll
                    for (int e = 0; e < VW; ++e) {
                        o[0][d][e] = fmaf(pe[0][j], v[e], o[0][d][e]);
                        o[1][d][e] = fmaf(pe[1][j], v[e], o[1][d][e]);
                    }
                }
        }
        __syncwarp();
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int q = 2 * ty + i;
        if (q >= rows) continue;
        const int t = (row0 + q) / a.g, h = kvh * a.g + (row0 + q) % a.g;
        const float inv = (bad_len || bad_s) ? __int_as_float(0x7fc00000) : 1.f / l[i];
#pragma unroll
        for (int d = 0; d < NV; ++d)
#pragma unroll
            for (int e = 0; e < VW; ++e)
                st_elem(a.out, (size_t)(start + t) * a.ld_out + (size_t)h * HD + tx * VW + 16 * VW * d + e,
                        a.dtype, o[i][d][e] * inv);
    }
}

template <int HD, bool FAST>
cudaError_t launch_paged_hd(const PagedArgs& a, cudaStream_t st) {
    const size_t smem = sizeof(float) * (AQ * (HD + 4) + AQ * (AK + 4) +
                                         (size_t)paged_stages<HD, FAST>() * 2 * AK * (HD + 4));
    static std::atomic<uint64_t> attr{0};
    cudaError_t e = smem_limit(reinterpret_cast<const void*>(paged_attention_kernel<HD, FAST>), (int)smem, attr);
    if (e != cudaSuccess) return e;
    const long long tiles = ((long long)a.n_tokens * a.g + AQ - 1) / AQ + a.n_rows;
    paged_attention_kernel<HD, FAST><<<dim3((unsigned)tiles, a.Hkv), A_THREADS, smem, st>>>(a);
    return cudaGetLastError();
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
    // lengths are not summed by more CTAs than run at once
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

cudaError_t launch_paged_attention(const PagedArgs& a, cudaStream_t st) {
    if (a.n_tokens <= 0 || a.n_rows <= 0) return cudaSuccess;
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
