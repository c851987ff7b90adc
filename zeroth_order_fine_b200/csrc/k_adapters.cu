// One linear layer for rows of many requests, each row under an adapter of its own:
//   y[m] = act(x[m] W^T + b + scale[a] (x[m] A_a^T) B_a^T),  a = row_adapter[m].
//
// Tensor-core forms (bf16).  Which one: DIRECT below.
//   direct: few output tiles (decode steps, M <= 128 rows always), where the product is a stream
//     of W over split K slices: the rows' shrink S in fp32 runs beside it on CUDA cores, and the
//     slices' reduction adds S[m] B_a^T from the row's own factors before bias and activation.
//   tiles: the expand runs as extra K blocks of the product's tcgen05 GEMM (S masked per row,
//     zeros for other adapters), each 256-row block with only the 64-column blocks of B that its
//     rows' adapters touch, and of those only the 16-column steps.
//
// CUDA-core form (fp32, and shapes the tensor cores do not take): the rows' shrink
// S[m, j] = scale[a] x[m] . A_a[j] goes to the workspace in fp32, then a tiled GEMM adds
// S[m] B_a^T to each of its tiles before the bias, activation and rounding.
#include <cstring>

#include "common.cuh"
#include "kernels.h"

namespace zo {

namespace {

constexpr int SH_WARPS = 8;

// S[m, j] for the rank rows of row m's own adapter: one warp per (m, j), the dot summed over the
// lanes in a fixed tree.  Rows without an adapter are not written (nor read later).
__global__ void __launch_bounds__(SH_WARPS * 32) adapter_shrink_kernel(AdapterArgs a, float* S) {
    const int m = blockIdx.x, lane = threadIdx.x & 31;
    const int j = blockIdx.y * SH_WARPS + (threadIdx.x >> 5);
    const int id = a.ids[m];
    if (id < 0 || id >= a.n_adapters || j >= a.rank) return;
    const size_t xr = (size_t)m * a.K, ar = ((size_t)id * a.rank + j) * a.K;
    const int t = a.dtype;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    int k = lane;
    for (; k + 96 < a.K; k += 128)
#pragma unroll
        for (int u = 0; u < 4; ++u)
            s[u] = fmaf(ld_elem(a.x, xr + k + 32 * u, t), ld_elem(a.A, ar + k + 32 * u, t), s[u]);
    for (; k < a.K; k += 32) s[0] = fmaf(ld_elem(a.x, xr + k, t), ld_elem(a.A, ar + k, t), s[0]);
    const float v = warp_sum((s[0] + s[1]) + (s[2] + s[3]));
    if (lane == 0) S[(size_t)m * a.rank + j] = v * a.scale[id];
}

constexpr int BM = 64, BN = 64, BK = 16;

__global__ void __launch_bounds__(256) adapter_gemm_kernel(AdapterArgs a, const float* __restrict__ S) {
    __shared__ __align__(16) float As[BK][BM + 4];
    __shared__ __align__(16) float Bs[BK][BN + 4];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int m0 = blockIdx.y * BM, n0 = blockIdx.x * BN;
    float acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
    const int lr = tid >> 2, lk = (tid & 3) * 4;
    for (int k0 = 0; k0 < a.K; k0 += BK) {
        const int m = m0 + lr, n = n0 + lr;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = k0 + lk + i;
            As[lk + i][lr] = (m < a.M && k < a.K) ? ld_elem(a.x, (size_t)m * a.K + k, a.dtype) : 0.f;
            Bs[lk + i][lr] = (n < a.N && k < a.K) ? ld_elem(a.W, (size_t)n * a.K + k, a.dtype) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < BK; ++kk) {
            const float4 x = *reinterpret_cast<const float4*>(&As[kk][ty * 4]);
            const float4 w = *reinterpret_cast<const float4*>(&Bs[kk][tx * 4]);
            const float xv[4] = {x.x, x.y, x.z, x.w}, wv[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xv[i], wv[j], acc[i][j]);
        }
        __syncthreads();
    }
    const size_t ldb = (size_t)a.n_adapters * a.rank;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = m0 + ty * 4 + i;
        if (m >= a.M) continue;
        const int id = a.ids[m];
        const bool live = id >= 0 && id < a.n_adapters;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + tx * 4 + j;
            if (n >= a.N) continue;
            float v = acc[i][j];
            if (live)
                for (int c = 0; c < a.rank; ++c)
                    v = fmaf(S[(size_t)m * a.rank + c],
                             ld_elem(a.B, (size_t)n * ldb + (size_t)id * a.rank + c, a.dtype), v);
            else if (id != -1)
                v = __int_as_float(0x7fc00000);
            if (a.bias) v += a.bias[n];
            const size_t ci = (size_t)m * a.N + n;
            if (a.accumulate) {
                static_cast<float*>(a.y)[ci] += v;
            } else {
                // not fmaxf, which would turn a NaN into 0
                if (a.act == 1) v = v < 0.f ? 0.f : v;
                st_elem(a.y, ci, a.dtype, v);
            }
        }
    }
}


// ---- tensor-core forms ----------------------------------------------------------------------

__device__ __forceinline__ void bf8(const uint4& u, float* f) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = __bfloat1622float2(h[i]);
        f[2 * i] = t.x;
        f[2 * i + 1] = t.y;
    }
}

// The fp32 shrink of the rows' own adapters (direct form): one warp per (m, j), 16-byte loads;
// the warps of a CTA share row m through L1.  The CTAs behind those (FETCH_CTAS of them) ask L2 for
// the rows' expand factors, output row by output row, while the product streams W: the reduction
// reads them in 2 rank-byte pieces, which from HBM, each by itself, took it 15 us instead of 6 (48
// rows, 32 adapters of rank 16, OPT-13B q|k|v).
constexpr int FETCH_CTAS = 148;
__global__ void __launch_bounds__(SH_WARPS * 32) adapter_shrink_rows_kernel(AdapterArgs a, float* S) {
    grid_dep_launch();                 // the product does not read S: it may start now
    const int lane = threadIdx.x & 31, groups = (a.rank + SH_WARPS - 1) / SH_WARPS;
    const int fetch = (int)blockIdx.x - a.M * groups;
    if (fetch >= 0) {
        const size_t ldb = (size_t)a.n_adapters * a.rank * 2;
        for (int m0 = 0; m0 < a.M; m0 += 32) {
            const int id = m0 + lane < a.M ? a.ids[m0 + lane] : -1;
            // one lane per adapter of these rows
            const unsigned same = __match_any_sync(0xffffffffu, id);
            if (id < 0 || id >= a.n_adapters || (same & ((1u << lane) - 1u))) continue;
            const char* b = static_cast<const char*>(a.B) + (size_t)id * a.rank * 2;
            for (int n = fetch * SH_WARPS + (threadIdx.x >> 5); n < a.N; n += FETCH_CTAS * SH_WARPS)
                for (int c = 0; c < a.rank * 2; c += 32)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(b + (size_t)n * ldb + c));
        }
        return;
    }
    const int m = (int)blockIdx.x / groups;
    const int j = (int)blockIdx.x % groups * SH_WARPS + (threadIdx.x >> 5);
    const int id = a.ids[m];
    if (id < 0 || id >= a.n_adapters || j >= a.rank) return;
    const uint4* x = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.x) + (size_t)m * a.K);
    const uint4* f = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.A) +
                                                    ((size_t)id * a.rank + j) * a.K);
    const int n8 = a.K / 8;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int k = lane; k < n8; k += 32) {
        float xv[8], fv[8];
        bf8(__ldg(x + k), xv);
        bf8(__ldg(f + k), fv);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i & 3] = fmaf(xv[i], fv[i], s[i & 3]);
    }
    const float v = warp_sum((s[0] + s[1]) + (s[2] + s[3]));
    if (lane == 0) S[(size_t)m * a.rank + j] = v * a.scale[id];
}

// Output of 4 columns n.. of row m from the product's sums y.
__device__ __forceinline__ void adapter_store4(const AdapterArgs& a, int m, int n, const float* y) {
    const size_t at = (size_t)m * a.N + n;
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = y[i] + (a.bias ? a.bias[n + i] : 0.f);
        if (a.act == 1) v[i] = v[i] < 0.f ? 0.f : v[i];       // a NaN stays
    }
    if (a.accumulate) {
        float4* c = reinterpret_cast<float4*>(static_cast<float*>(a.y) + at);
        float4 o = *c;
        o.x += v[0]; o.y += v[1]; o.z += v[2]; o.w += v[3];
        *c = o;
    } else {
        __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]), hi = __floats2bfloat162_rn(v[2], v[3]);
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.y) + at) =
            make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
    }
}

// The slices' reduction of the direct form: a CTA takes 512 columns of a row.  First the expand
// S[m] B_a[n]^T of its columns into shared memory: LPR lanes share a row of B (LPR 16-byte loads side
// by side, so that a warp's load takes whole sectors), their sums joined by shuffles.  Then
// each thread adds the slices of 4 columns in split order, the expand, bias and activation.
template <int LPR>
__device__ __forceinline__ void adapter_expand(const AdapterArgs& a, const float* __restrict__ s,
                                               const __nv_bfloat16* __restrict__ b, size_t ldb, int n0,
                                               int n1, float* e) {
    constexpr int ROWS = 32 / LPR;            // rows of B per warp and load
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = lane % LPR;
#pragma unroll 4
    for (int i = 0; i < 128; i += ROWS) {
        const int n = n0 + warp * 128 + i + lane / LPR;
        float y = 0.f;
        if (n < n1)
            for (int c = part * 8; c < a.rank; c += LPR * 8) {
                float bv[8];
                bf8(__ldg(reinterpret_cast<const uint4*>(b + n * ldb + c)), bv);
#pragma unroll
                for (int q = 0; q < 8; ++q) y = fmaf(s[c + q], bv[q], y);
            }
#pragma unroll
        for (int d = LPR / 2; d > 0; d >>= 1) y += __shfl_xor_sync(0xffffffffu, y, d);
        if (part == 0) e[warp * 128 + i + lane / LPR] = y;
    }
}

__global__ void __launch_bounds__(128)
    adapter_reduce_kernel(AdapterArgs a, const float* __restrict__ S, const float* __restrict__ ws, int ks) {
    __shared__ __align__(16) float e[512];
    __shared__ float s[256];
    const int m = blockIdx.y, n0 = blockIdx.x * 512, n = n0 + threadIdx.x * 4;
    const int id = a.ids[m];
    const bool live = id >= 0 && id < a.n_adapters;
    grid_dep_wait();
    float y[4] = {0.f, 0.f, 0.f, 0.f};
    if (n < a.N)
        for (int k = 0; k < ks; ++k) {
            const float4 w = *reinterpret_cast<const float4*>(ws + ((size_t)k * a.M + m) * a.N + n);
            y[0] += w.x; y[1] += w.y; y[2] += w.z; y[3] += w.w;
        }
    if (live) {
        for (int c = threadIdx.x; c < a.rank; c += 128) s[c] = S[(size_t)m * a.rank + c];
        __syncthreads();
        const size_t ldb = (size_t)a.n_adapters * a.rank;
        const __nv_bfloat16* b = static_cast<const __nv_bfloat16*>(a.B) + (size_t)id * a.rank;
        const int n1 = min(a.N, n0 + 512);
        if (a.rank % 64 == 0) {
            adapter_expand<8>(a, s, b, ldb, n0, n1, e);
        } else if (a.rank % 16 == 0) {
            adapter_expand<2>(a, s, b, ldb, n0, n1, e);
        } else if (a.rank % 8 == 0) {
            adapter_expand<1>(a, s, b, ldb, n0, n1, e);
        } else {
            for (int i = threadIdx.x; n0 + i < n1; i += 128) {
                float v = 0.f;
                for (int c = 0; c < a.rank; ++c) v = fmaf(s[c], __bfloat162float(b[(n0 + i) * ldb + c]), v);
                e[i] = v;
            }
        }
        __syncthreads();
        if (n < a.N) {
            const float4 v = *reinterpret_cast<const float4*>(e + threadIdx.x * 4);
            y[0] += v.x; y[1] += v.y; y[2] += v.z; y[3] += v.w;
        }
    } else if (id != -1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = __int_as_float(0x7fc00000);
    }
    if (n < a.N) adapter_store4(a, m, n, y);
}

// The tiles form's lists: CTA = a block of 256 rows, thread = a row.  A block's list holds the
// 64-column blocks of the factors that its rows' adapters touch, ascending, with the mask of the
// 16-column steps they touch.
__global__ void __launch_bounds__(256)
    adapter_lists_kernel(const int* __restrict__ ids, int M, int n_adapters, int rank, int* __restrict__ cnt,
                         int* __restrict__ list, int n_list) {
    __shared__ unsigned steps[4096 / 32];       // one bit per 16-column step of 65536 columns
    __shared__ int wsum[8];
    grid_dep_launch();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < 4096 / 32; i += 256) steps[i] = 0u;
    __syncthreads();
    const int m = blockIdx.x * 256 + tid;
    const int id = m < M ? ids[m] : -1;
    if (id >= 0 && id < n_adapters) {
        const int s0 = id * rank / 16, s1 = ((id + 1) * rank - 1) / 16;
        for (int s = s0; s <= s1; ++s)
            if (!((steps[s >> 5] >> (s & 31)) & 1u)) atomicOr(&steps[s >> 5], 1u << (s & 31));
    }
    __syncthreads();
    int base = 0;
    for (int b0 = 0; b0 < n_list; b0 += 256) {
        const int b = b0 + tid;
        const int mask = b < n_list ? (int)((steps[b >> 3] >> (4 * (b & 7))) & 15u) : 0;
        const unsigned have = __ballot_sync(0xffffffffu, mask != 0);
        if (lane == 0) wsum[warp] = __popc(have);
        __syncthreads();
        int at = base, total = 0;
        for (int w = 0; w < 8; ++w) {
            if (w < warp) at += wsum[w];
            total += wsum[w];
        }
        if (mask) list[(size_t)blockIdx.x * n_list + at + __popc(have & ((1u << lane) - 1u))] = b | (mask << 16);
        base += total;
        __syncthreads();
    }
    if (tid == 0) cnt[blockIdx.x] = base;
}

// Chunks of 32 rows x 32 columns that the product's epilogue marked, and rows whose id names no
// adapter: marked chunks are computed anew from the rows' own factors, one warp per output, and
// rows without an adapter to name become NaN.  On finite weights nothing is marked and the kernel
// only reads the marks.
constexpr int FIX_THREADS = 256;
__global__ void __launch_bounds__(FIX_THREADS)
    adapter_repair_kernel(AdapterArgs a, const __nv_bfloat16* __restrict__ S, int ldS,
                          const uint8_t* __restrict__ odd) {
    grid_dep_wait();
    const int chunks = (a.N + 31) / 32, m0 = blockIdx.x * 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int id_l = m0 + lane < a.M ? a.ids[m0 + lane] : -1;
    const unsigned none = __ballot_sync(0xffffffffu, id_l < -1 || id_l >= a.n_adapters);
    // usually nothing is marked: all of the CTA's marks in one look
    int any = none != 0u;
    for (int c = threadIdx.x; c < chunks; c += FIX_THREADS) any |= odd[(size_t)blockIdx.x * chunks + c];
    if (!__syncthreads_or(any)) return;
    for (int c = warp; c < chunks; c += FIX_THREADS / 32) {
        const bool marked = odd[(size_t)blockIdx.x * chunks + c] != 0;
        if (!marked && !none) continue;
        for (int r = 0; r < 32 && m0 + r < a.M; ++r) {
            const int m = m0 + r;
            const int id = __shfl_sync(0xffffffffu, id_l, r);
            const bool bad = (none >> r) & 1u;
            if (!marked && !bad) continue;
            float mine = __int_as_float(0x7fc00000);
            if (!bad)
                for (int j = 0; j < 32 && c * 32 + j < a.N; ++j) {
                    const int n = c * 32 + j;
                    const uint4* x = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.x) + (size_t)m * a.K);
                    const uint4* w = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.W) + (size_t)n * a.K);
                    float v = 0.f;
                    for (int k = lane; k < a.K / 8; k += 32) {
                        float xv[8], wv[8];
                        bf8(__ldg(x + k), xv);
                        bf8(__ldg(w + k), wv);
#pragma unroll
                        for (int i = 0; i < 8; ++i) v = fmaf(xv[i], wv[i], v);
                    }
                    if (id >= 0) {
                        const size_t col = (size_t)id * a.rank;
                        const size_t ldb = (size_t)a.n_adapters * a.rank;
                        for (int k = lane; k < a.rank; k += 32)
                            v = fmaf(__bfloat162float(S[(size_t)m * ldS + col + k]),
                                     __bfloat162float(static_cast<const __nv_bfloat16*>(a.B)[(size_t)n * ldb + col + k]), v);
                    }
                    v = warp_sum(v);
                    if (lane == j) mine = v;
                }
            const int n = c * 32 + lane;
            if (n >= a.N) continue;
            float v = mine + (a.bias ? a.bias[n] : 0.f);
            if (a.act == 1) v = v < 0.f ? 0.f : v;
            const size_t at = (size_t)m * a.N + n;
            if (a.accumulate) static_cast<float*>(a.y)[at] += v;
            else static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v);
        }
    }
}

// DIRECT: at most 128 rows, where the swapped single-SM product streams W, or too few 256 x 256
// output tiles to give every SM pair two.
bool direct_form(int M, int N) {
    const long long tiles = (long long)((M + 255) / 256) * ((N + 255) / 256);
    return M <= 128 || (N > 128 && tiles < 37);
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Slices of the direct form: room for up to 16 splits, 64 MB at most unless one slice is more.
size_t slice_floats(int M, int N) {
    const size_t one = (size_t)M * N;
    const size_t most = ((size_t)64 << 20) / 4 / one;
    return one * (most < 1 ? 1 : most > 16 ? 16 : most);
}

// Rows of one pass of the tiles form: the masked shrink stays within 256 MB.
int pass_rows(int M, int K2) {
    const size_t ld = ((size_t)K2 + 63) / 64 * 64;
    size_t rows = ((size_t)256 << 20) / (ld * 2) / 256 * 256;
    rows = rows < 256 ? 256 : rows > 262144 ? 262144 : rows;
    return (size_t)M < rows ? M : (int)rows;
}
struct TileSpace {
    size_t list, s, odd, total;           // offsets
    int blocks, n_list, ld;
};
TileSpace tile_space(int M, int N, int K2) {
    TileSpace t;
    const int rows = pass_rows(M, K2);
    t.blocks = (rows + 255) / 256;
    t.n_list = (K2 + 63) / 64;
    t.ld = t.n_list * 64;
    t.list = up256((size_t)t.blocks * 4);
    t.s = t.list + up256((size_t)t.blocks * t.n_list * 4);
    t.odd = t.s + up256((size_t)rows * t.ld * 2);
    t.total = t.odd + up256((size_t)((rows + 31) / 32) * ((N + 31) / 32));
    return t;
}

}  // namespace

size_t adapter_workspace(int M, int N, int K, int n_adapters, int rank, int dtype) {
    (void)K;
    const size_t s = up256((size_t)M * rank * 4) + 256;
    if (dtype != E_BF16 || M == 0) return s;
    if (direct_form(M, N)) return s + up256(slice_floats(M, N) * 4);
    const size_t t = tile_space(M, N, n_adapters * rank).total;
    return t > s ? t : s;
}

cudaError_t launch_linear_adapters_simt(const AdapterArgs& a, cudaStream_t st) {
    float* S = static_cast<float*>(a.ws);
    adapter_shrink_kernel<<<dim3(a.M, cdiv(a.rank, SH_WARPS)), SH_WARPS * 32, 0, st>>>(a, S);
    adapter_gemm_kernel<<<dim3(cdiv(a.N, BN), cdiv(a.M, BM)), 256, 0, st>>>(a, S);
    return cudaGetLastError();
}

cudaError_t launch_adapter_reduce(const AdapterArgs& a, const float* S, const float* ws, int ks,
                                  cudaStream_t st, bool pdl) {
    const dim3 grid(cdiv(a.N, 512), a.M);
    if (pdl) return launch_pdl(adapter_reduce_kernel, grid, dim3(128), 0, st, a, S, ws, ks);
    adapter_reduce_kernel<<<grid, 128, 0, st>>>(a, S, ws, ks);
    return cudaGetLastError();
}

bool linear_adapters_tc_supported(const AdapterArgs& a) {
    const uintptr_t mix = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.W) |
                          reinterpret_cast<uintptr_t>(a.A) | reinterpret_cast<uintptr_t>(a.B) |
                          reinterpret_cast<uintptr_t>(a.y) | reinterpret_cast<uintptr_t>(a.bias);
    return a.dtype == E_BF16 && a.K % 8 == 0 && a.N % 8 == 0 && (a.n_adapters * a.rank) % 8 == 0 &&
           mix % 16 == 0;
}

cudaError_t launch_linear_adapters_tc(const AdapterArgs& a, cudaStream_t st) {
    char* ws = static_cast<char*>(a.ws);
    if (direct_form(a.M, a.N)) {
        float* S = reinterpret_cast<float*>(ws);
        GemmArgs g;
        memset(&g, 0, sizeof(g));
        g.A = a.x; g.lda = a.K; g.a_type = E_BF16;
        g.B = a.W; g.ldb = a.K; g.b_type = E_BF16;
        g.M = a.M; g.N = a.N; g.K = a.K;
        g.epi = a.accumulate ? EPI_RESID : a.act ? EPI_STORE_RELU : EPI_STORE;
        g.bias = a.bias;
        g.C = a.y; g.ldc = a.N; g.c_type = a.accumulate ? E_F32 : E_BF16;
        g.ws = reinterpret_cast<float*>(ws + up256((size_t)a.M * a.rank * 4));
        g.ws_floats = slice_floats(a.M, a.N);
        g.adapt = &a;
        g.adapt_S = S;
        if (!gemm_tc_supported(g)) return cudaErrorNotSupported;
        adapter_shrink_rows_kernel<<<a.M * cdiv(a.rank, SH_WARPS) + FETCH_CTAS, SH_WARPS * 32, 0, st>>>(a, S);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        return gemm_tc(g, st) ? cudaErrorUnknown : cudaSuccess;
    }
    const int K2 = a.n_adapters * a.rank;
    const TileSpace t = tile_space(a.M, a.N, K2);
    const int rows = pass_rows(a.M, K2);
    for (int m0 = 0; m0 < a.M; m0 += rows) {
        AdapterArgs b = a;
        b.M = a.M - m0 < rows ? a.M - m0 : rows;
        b.x = static_cast<const __nv_bfloat16*>(a.x) + (size_t)m0 * a.K;
        b.ids = a.ids + m0;
        b.y = static_cast<char*>(a.y) + (size_t)m0 * a.N * (a.accumulate ? 4 : 2);
        AdapterTiles at;
        at.cnt = reinterpret_cast<int*>(ws);
        at.list = reinterpret_cast<int*>(ws + t.list);
        at.n_list = t.n_list;
        at.S = ws + t.s;
        at.ldS = t.ld;
        at.odd = reinterpret_cast<uint8_t*>(ws + t.odd);
        adapter_lists_kernel<<<cdiv(b.M, 256), 256, 0, st>>>(b.ids, b.M, b.n_adapters, b.rank,
                                                            const_cast<int*>(at.cnt), const_cast<int*>(at.list),
                                                            at.n_list);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        if (gemm_tc_adapters(b, at, st)) return cudaErrorUnknown;
        e = launch_pdl(adapter_repair_kernel, dim3(cdiv(b.M, 32)), dim3(FIX_THREADS), 0, st, b,
                       static_cast<const __nv_bfloat16*>(at.S), at.ldS, static_cast<const uint8_t*>(at.odd));
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace zo
