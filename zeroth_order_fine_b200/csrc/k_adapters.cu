// One linear layer for rows of many requests, each row under an adapter of its own:
//   y[m] = act(x[m] W^T + b + scale[a] (x[m] A_a^T) B_a^T),  a = row_adapter[m].
//
// CUDA-core form (fp32, and shapes the tensor cores do not take): the rows' shrink
// S[m, j] = scale[a] x[m] . A_a[j] goes to the workspace in fp32, then a tiled GEMM adds
// S[m] B_a^T to each of its tiles before the bias, activation and rounding.
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

}  // namespace

size_t adapter_workspace(int M, int N, int K, int n_adapters, int rank, int dtype) {
    (void)N; (void)K; (void)n_adapters; (void)dtype;
    return ((size_t)M * rank * 4 + 255) / 256 * 256 + 256;
}

cudaError_t launch_linear_adapters_simt(const AdapterArgs& a, cudaStream_t st) {
    float* S = static_cast<float*>(a.ws);
    adapter_shrink_kernel<<<dim3(a.M, cdiv(a.rank, SH_WARPS)), SH_WARPS * 32, 0, st>>>(a, S);
    adapter_gemm_kernel<<<dim3(cdiv(a.N, BN), cdiv(a.M, BM)), 256, 0, st>>>(a, S);
    return cudaGetLastError();
}

}  // namespace zo
