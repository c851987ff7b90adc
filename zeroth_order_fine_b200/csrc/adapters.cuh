// Shared by the adapter kernels: what a row's output is, one element at a time.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace zo {

__device__ __forceinline__ void bf8(const uint4& u, float* f) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = __bfloat1622float2(h[i]);
        f[2 * i] = t.x;
        f[2 * i + 1] = t.y;
    }
}

// Lanes `lane`, lane + lanes, .. of x[m] . W[n] + S[m] . B_a[n] with the row's own adapter (none: the
// first part), by plain fp32 sums: the slow way, for elements that the tensor cores' zeros of other
// adapters have made non-finite.  S is the masked shrink, bf16 [.. x ldS].
__device__ inline float adapter_element(const AdapterArgs& a, const __nv_bfloat16* S, int ldS, int m, int n,
                                        int id, int lane, int lanes) {
    const uint4* x = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.x) + (size_t)m * a.K);
    const uint4* w = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.W) + (size_t)n * a.K);
    float v = 0.f;
#pragma unroll 4
    for (int k = lane; k < a.K / 8; k += lanes) {
        float xv[8], wv[8];
        bf8(__ldg(x + k), xv);
        bf8(__ldg(w + k), wv);
#pragma unroll
        for (int i = 0; i < 8; ++i) v = fmaf(xv[i], wv[i], v);
    }
    if (id >= 0) {
        const size_t col = (size_t)id * a.rank, ldb = (size_t)a.n_adapters * a.rank;
        for (int k = lane; k < a.rank; k += lanes)
            v = fmaf(__bfloat162float(S[(size_t)m * ldS + col + k]),
                     __bfloat162float(static_cast<const __nv_bfloat16*>(a.B)[(size_t)n * ldb + col + k]), v);
    }
    return v;
}

// bias and activation (a NaN stays) and the store of one element
template <typename T = __nv_bfloat16>
__device__ __forceinline__ void adapter_store(const AdapterArgs& a, int m, int n, float v) {
    if (a.bias) v += a.bias[n];
    if (a.act == 1) v = v < 0.f ? 0.f : v;
    const size_t at = (size_t)m * a.N + n;
    if (a.accumulate) static_cast<float*>(a.y)[at] += v;
    else static_cast<T*>(a.y)[at] = static_cast<T>(v);          // to the nearest
}

}  // namespace zo
