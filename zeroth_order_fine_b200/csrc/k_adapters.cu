// One linear layer for rows of many requests, each row under an adapter of its own:
//   y[m] = act(x[m] W^T + b + scale[a] (x[m] A_a^T) B_a^T),  a = row_adapter[m].
//
// Tensor-core forms (bf16, from three rows on): the expand runs as extra K blocks of the product's tcgen05 GEMM, with the
// rows' shrink S masked to their own adapter (zeros in the others' columns); of the factors' 64-column
// blocks, and of those the 16-column steps, only those that the rows at hand touch.
//   one or two rows (fp32: up to 24): W streamed by CUDA cores with S beside it.
//   decode steps (up to 128 rows, and more of small layers): the product is a stream of W, the weights on the tensor cores'
//     128-row side; S comes from a CUDA-core kernel beside its first blocks.
//   more rows: per 256-row block a list of blocks, S from a tcgen05 shrink, 256 x 256 output tiles.
// An output that the zeros have made non-finite (0 times another adapter's infinity) is computed anew
// from the row's own factors.
//
// CUDA-core form (fp32, and shapes the tensor cores do not take): the rows' shrink
// S[m, j] = scale[a] x[m] . A_a[j] goes to the workspace in fp32, then a tiled GEMM adds
// S[m] B_a^T to each of its tiles before the bias, activation and rounding.
#include <cstring>

#include "adapters.cuh"

namespace zo {

namespace {

constexpr int SH_WARPS = 8;

// S[m, j] for the rank rows of row m's own adapter: one warp per (m, j), the dot summed over the
// lanes in a fixed tree.  Rows without an adapter are not written (nor read later).  VEC: fp32 with
// 16-byte rows.
template <bool VEC>
__global__ void __launch_bounds__(SH_WARPS * 32) adapter_shrink_kernel(AdapterArgs a, float* S) {
    grid_dep_launch();                         // the fp32 product does not read S
    const int m = blockIdx.x, lane = threadIdx.x & 31;
    const int j = blockIdx.y * SH_WARPS + (threadIdx.x >> 5);
    const int id = a.ids[m];
    if (id < 0 || id >= a.n_adapters || j >= a.rank) return;
    const size_t xr = (size_t)m * a.K, ar = ((size_t)id * a.rank + j) * a.K;
    const int t = a.dtype;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (VEC) {
        const float4* x = reinterpret_cast<const float4*>(static_cast<const float*>(a.x) + xr);
        const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(a.A) + ar);
#pragma unroll 4
        for (int q = lane; q < a.K / 4; q += 32) {
            const float4 u = __ldg(x + q), v = __ldg(f + q);
            s[0] = fmaf(u.x, v.x, s[0]);
            s[1] = fmaf(u.y, v.y, s[1]);
            s[2] = fmaf(u.z, v.z, s[2]);
            s[3] = fmaf(u.w, v.w, s[3]);
        }
    }
    int k = VEC ? a.K : lane;
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


// ---- fp32 -----------------------------------------------------------------------------------
// The product in fp32 on CUDA cores, bound by their FMA rate (2 M N K flops at ~70 TFLOP/s; 301 x 2048 x
// 2048 with its adapters 74 us, of which this kernel ~65: the FMA pipe is 63 % busy while an SM works
// and the SMs work 91 % of the time; 48-byte spills at 128 registers for a fourth CTA gave nothing): 64 x 64
// tiles, 8 x 4 outputs a thread, K in 32-deep stages by asynchronous 16-byte copies.  The tiles stay
// as they lie in memory (K contiguous, rows padded to 36 floats): a thread reads 4 of K at a time of
// its 8 rows and 4 columns, 12 16-byte reads for 128 FMAs, without bank clashes, two FMAs to an
// instruction (neighbouring k).  K is also split over CTAs where the tiles alone would leave the
// last round of SMs half empty; each split writes a slice, and the slices are added in order by the
// kernel that adds the expand.
constexpr int FM = 64, FK = 32, FLD = FK + 4, FSTAGES = 3, F_THREADS = 128;
constexpr int F_SMEM = FSTAGES * 2 * FM * FLD * 4;

__device__ __forceinline__ void cp16(uint32_t dst, const float* src, bool live) {
    const int n = live ? 16 : 0;               // 0: zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

__global__ void __launch_bounds__(F_THREADS)
    gemm_f32_kernel(const float* __restrict__ A, const float* __restrict__ B, int M, int N, int K, int ks,
                    float* __restrict__ slices) {
    extern __shared__ __align__(16) float fsm[];
    grid_dep_launch();
    // neighbouring lanes read the same columns: a 16-byte read of a warp takes half the passes
    const int tid = threadIdx.x, tx = (tid >> 1) & 15, ty = 2 * (tid >> 5) + (tid & 1);
    const int m0 = blockIdx.y * FM, n0 = blockIdx.x * FM, split = blockIdx.z;
    const int blocks = (K + FK - 1) / FK, per = (blocks + ks - 1) / ks;
    const int b0 = split * per, b1 = min(blocks, b0 + per);
    const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(fsm));
    // 8 copies a thread and stage: 4 of each operand's 16-row steps, 4 columns of K
    const int lr = tid / (FK / 4), lc = tid % (FK / 4) * 4;
    const float *pa = A + (size_t)(m0 + lr) * K + lc, *pb = B + (size_t)(n0 + lr) * K + lc;
    const uint32_t to = base + (uint32_t)(lr * FLD + lc) * 4;
    auto load = [&](int b) {
        const uint32_t st = to + (uint32_t)((b - b0) % FSTAGES) * (2 * FM * FLD * 4);
        const int k = b * FK;
#pragma unroll
        for (int i = 0; i < 2 * FM / 16; ++i) {
            const int r = i % (FM / 16) * 16;
            const bool live = (i < FM / 16 ? m0 : n0) + lr + r < (i < FM / 16 ? M : N) && k + lc < K;
            const float* src = (i < FM / 16 ? pa : pb) + (live ? (size_t)r * K + k : 0);
            cp16(st + (uint32_t)(i * 16 * FLD) * 4, live ? src : A, live);
        }
    };
    uint64_t acc[8][4];                        // sums over the even and over the odd k
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0ull;
#pragma unroll
    for (int s = 0; s < FSTAGES - 1; ++s) {
        if (b0 + s < b1) load(b0 + s);
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    for (int b = b0; b < b1; ++b) {
        asm volatile("cp.async.wait_group %0;" ::"n"(FSTAGES - 2) : "memory");
        __syncthreads();                       // stage b is there, and b - 1 has been read
        if (b + FSTAGES - 1 < b1) load(b + FSTAGES - 1);
        asm volatile("cp.async.commit_group;" ::: "memory");
        const float* as = fsm + (size_t)((b - b0) % FSTAGES) * (2 * FM * FLD) + ty * FLD;
        const float* bs = fsm + (size_t)((b - b0) % FSTAGES) * (2 * FM * FLD) + (FM + tx) * FLD;
#pragma unroll
        for (int k = 0; k < FK; k += 4) {
            ulonglong2 x[8], w[4];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = *reinterpret_cast<const ulonglong2*>(as + i * 8 * FLD + k);
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = *reinterpret_cast<const ulonglong2*>(bs + j * 16 * FLD + k);
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc[i][j]) : "l"(x[i].x), "l"(w[j].x));
                    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc[i][j]) : "l"(x[i].y), "l"(w[j].y));
                }
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    float* out = slices + (size_t)split * M * N;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int m = m0 + ty + 8 * i;
        if (m >= M) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + tx + 16 * j;
            const float2 v = *reinterpret_cast<const float2*>(&acc[i][j]);
            if (n < N) out[(size_t)m * N + n] = v.x + v.y;
        }
    }
    grid_dep_wait();                           // the shrink before: what follows reads both
}

// y = act(slices + S[m] B_a^T + b): a CTA takes 4 rows and 128 columns, a thread a column.  Rows of
// one request lie together, so the factors of a column are read once for a run of rows with the same
// adapter.
constexpr int ER = 4;
__global__ void __launch_bounds__(128)
    adapter_expand_f32_kernel(AdapterArgs a, const float* __restrict__ S, const float* __restrict__ slices, int ks) {
    __shared__ __align__(16) float s[ER][256];
    const int m0 = blockIdx.x * ER, n = blockIdx.y * 128 + threadIdx.x, rows = min(ER, a.M - m0);
    int id[ER];
#pragma unroll
    for (int i = 0; i < ER; ++i) id[i] = i < rows ? a.ids[m0 + i] : -1;
    grid_dep_wait();
    for (int i = threadIdx.x; i < rows * a.rank; i += 128) s[i / a.rank][i % a.rank] = S[(size_t)m0 * a.rank + i];
    __syncthreads();
    if (n >= a.N) return;
    float y[ER];
#pragma unroll
    for (int i = 0; i < ER; ++i) {
        y[i] = 0.f;
        if (i < rows)
#pragma unroll 4
            for (int k = 0; k < ks; ++k) y[i] += slices[((size_t)k * a.M + m0 + i) * a.N + n];
    }
    const float* B = static_cast<const float*>(a.B) + (size_t)n * a.n_adapters * a.rank;
    const bool vec = a.rank % 4 == 0 && reinterpret_cast<uintptr_t>(a.B) % 16 == 0;
#pragma unroll
    for (int i = 0; i < ER; ++i) {
        // the run that begins at row i
        if (i >= rows || id[i] < 0 || id[i] >= a.n_adapters || (i > 0 && id[i] == id[i > 0 ? i - 1 : 0])) continue;
        int end = i + 1;
        while (end < rows && a.ids[m0 + end] == id[i]) ++end;
        const float* b = B + (size_t)id[i] * a.rank;
        int c = 0;
        if (vec)
#pragma unroll 4
            for (; c < a.rank; c += 4) {
                const float4 v = __ldg(reinterpret_cast<const float4*>(b + c));
#pragma unroll
                for (int q = i; q < ER; ++q) {
                    if (q >= end) continue;
                    const float4 f = *reinterpret_cast<const float4*>(&s[q][c]);
                    y[q] = fmaf(f.w, v.w, fmaf(f.z, v.z, fmaf(f.y, v.y, fmaf(f.x, v.x, y[q]))));
                }
            }
        for (; c < a.rank; ++c) {
            const float v = __ldg(b + c);
#pragma unroll
            for (int q = i; q < ER; ++q)
                if (q < end) y[q] = fmaf(s[q][c], v, y[q]);
        }
    }
#pragma unroll
    for (int i = 0; i < ER; ++i) {
        if (i >= rows) continue;
        float v = y[i];
        if (id[i] < -1 || id[i] >= a.n_adapters) v = __int_as_float(0x7fc00000);
        if (a.bias) v += a.bias[n];
        if (a.act == 1) v = v < 0.f ? 0.f : v;
        float* o = static_cast<float*>(a.y) + (size_t)(m0 + i) * a.N + n;
        *o = a.accumulate ? *o + v : v;
    }
}

// K splits of the fp32 product: the fewest whose last round of SMs is full enough.  301 x 2048 x 2048 under
// 5 adapters (160 tiles) takes 133 us unsplit, 103 in 2, 88 in 4 and 84 in 8.  Each split costs a slice,
// written and read: a fiftieth of a round there, and in proportion to the tiles and against K where
// that is more, so that many full rounds are not split for the last one (2048 x 8192 x 2048: 1.59 ms, 1.62
// in 4; 4093 x 20480 x 5120: 19.8, 20.2 in 5); 64 MB of slices at most, as in the decode form.
constexpr size_t SLICES_MOST = (size_t)64 << 20;
int f32_splits(int M, int N, int K) {
    const long long tiles = (long long)((M + FM - 1) / FM) * ((N + FM - 1) / FM);
    const int blocks = (K + FK - 1) / FK;
    int best = 1;
    double least = 1e300;
    for (int k = 1; k <= 8 && k <= (blocks + 3) / 4; ++k) {
        const int per = (blocks + k - 1) / k;
        if ((blocks + per - 1) / per != k) continue;
        if (k > 1 && (size_t)M * N * k * 4 > SLICES_MOST) break;
        const double slice = 0.256 * (double)tiles / K;
        const double cost = (double)((tiles * k + 147) / 148) * per / blocks + (slice > 0.02 ? slice : 0.02) * k;
        if (cost < least) {
            least = cost;
            best = k;
        }
    }
    return best;
}

// Rows of one pass of the fp32 form: a pass's slice stays within 256 MB, in whole tiles.
int f32_pass_rows(int M, int N) {
    size_t rows = ((size_t)256 << 20) / 4 / N / FM * FM;
    if (rows < FM) rows = FM;
    return (size_t)M < rows ? M : (int)rows;
}
size_t f32_slice_floats(int M, int N, int K) {
    const int rows = f32_pass_rows(M, N), last = M % rows;
    const size_t a = (size_t)f32_splits(rows, N, K) * rows * N;
    const size_t b = last ? (size_t)f32_splits(last, N, K) * last * N : 0;
    return a > b ? a : b;
}

// ---- tensor-core forms ----------------------------------------------------------------------

// The rows' shrink for the decode form: S[m, j] = scale[a] x[m] . A_a[j] in fp32, rounded to bf16
// into row m of the masked S (the products' extension operand, which the tensor cores take in bf16:
// half a step of S, as the plain form in bf16 has), whose other columns become zeros in the blocks
// that any row uses.  KW warps share a dot, each with its part of K: a whole CTA per dot while the
// CTAs are about two a SM, since the chain of loads is what takes time (16 rows of rank 16, K = 5120,
// the whole call: 16.9 us against 18.0), a warp per dot above (48 rows: 18.5 us against 19.1; 128 rows
// of rank 64: 35.8 against 45.4).  16-byte loads; the warps of a CTA share row m through L1.  The
// first CTA also writes the list of blocks: those that the rows' adapters touch, with the mask of
// their 16-column steps.
template <int KW>
__global__ void __launch_bounds__(SH_WARPS * 32)
    adapter_shrink_rows_kernel(AdapterArgs a, __nv_bfloat16* __restrict__ S, int ldS, int* __restrict__ cnt,
                               int* __restrict__ list) {
    __shared__ unsigned steps[4096 / 32];      // one bit per 16-column step of 65536 columns
    grid_dep_launch();                         // the product reads S and the list only at its end
    constexpr int PER_CTA = SH_WARPS / KW;               // rows of the adapter per CTA
    static_assert(KW == 1 || KW == SH_WARPS, "a whole CTA per dot, or a warp");
    __shared__ float parts[SH_WARPS];
    const int groups = (a.rank + PER_CTA - 1) / PER_CTA;
    const int m = (int)blockIdx.x / groups, grp = (int)blockIdx.x % groups;
    const int lane = threadIdx.x & 31, n_list = ldS / 64;
    const int id = a.ids[m];
    const bool live = id >= 0 && id < a.n_adapters;
    if (grp == 0) {
        for (int i = threadIdx.x; i < (n_list + 7) / 8; i += blockDim.x) steps[i] = 0u;
        __syncthreads();
        for (int i = threadIdx.x; i < a.M; i += blockDim.x) {
            const int r = a.ids[i];
            if (r >= 0 && r < a.n_adapters)
                for (int s = r * a.rank / 16; s <= ((r + 1) * a.rank - 1) / 16; ++s)
                    if (!((steps[s >> 5] >> (s & 31)) & 1u)) atomicOr(&steps[s >> 5], 1u << (s & 31));
        }
        __syncthreads();
        const int lo = live ? id * a.rank : 0, hi = live ? lo + a.rank : 0;
        for (int b = threadIdx.x; b < n_list; b += blockDim.x) {
            const int mask = (int)((steps[b >> 3] >> (4 * (b & 7))) & 15u);
            if (!mask) continue;
            for (int c = b * 64; c < b * 64 + 64; c += 8) {
                __nv_bfloat16* p = S + (size_t)m * ldS + c;
                if (c + 8 <= lo || c >= hi) {
                    *reinterpret_cast<uint4*>(p) = make_uint4(0u, 0u, 0u, 0u);
                } else {
                    for (int i = 0; i < 8; ++i)
                        if (c + i < lo || c + i >= hi) p[i] = __float2bfloat16_rn(0.f);
                }
            }
        }
        if (m == 0 && threadIdx.x < 32) {              // the list, ascending
            int used = 0;
            for (int b0 = 0; b0 < n_list; b0 += 32) {
                const int b = b0 + lane;
                const int mask = b < n_list ? (int)((steps[b >> 3] >> (4 * (b & 7))) & 15u) : 0;
                const unsigned have = __ballot_sync(0xffffffffu, mask != 0);
                if (mask) list[used + __popc(have & ((1u << lane) - 1u))] = b | (mask << 16);
                used += __popc(have);
            }
            if (lane == 0) *cnt = used;
        }
    }
    const int warp = (int)(threadIdx.x >> 5), kpart = warp % KW;
    const int j = grp * PER_CTA + warp / KW;
    if (!live || j >= a.rank) return;          // (with KW > 1 the whole CTA)
    const uint4* x = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.x) + (size_t)m * a.K);
    const uint4* f = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.A) +
                                                    ((size_t)id * a.rank + j) * a.K);
    float s[2] = {0.f, 0.f};
#pragma unroll 4
    for (int k = kpart * 32 + lane; k < a.K / 8; k += 32 * KW) {
        float xv[8], fv[8];
        bf8(__ldg(x + k), xv);
        bf8(__ldg(f + k), fv);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i & 1] = fmaf(xv[i], fv[i], s[i & 1]);
    }
    float v = warp_sum(s[0] + s[1]);
    if (KW > 1) {
        if (lane == 0) parts[warp] = v;
        __syncthreads();
        v = 0.f;
        for (int w = 0; w < KW; ++w) v += parts[w];
    }
    if (lane == 0 && kpart == 0)
        S[(size_t)m * ldS + (size_t)id * a.rank + j] = __float2bfloat16_rn(v * a.scale[id]);
}

template <int KW>
cudaError_t launch_shrink_rows(const AdapterArgs& a, __nv_bfloat16* S, int ldS, int* cnt, int* list,
                               cudaStream_t st) {
    static std::atomic<uint64_t> share{0};
    const cudaError_t e = smem_share(reinterpret_cast<const void*>(adapter_shrink_rows_kernel<KW>), share);
    if (e != cudaSuccess) return e;
    adapter_shrink_rows_kernel<KW>
        <<<a.M * cdiv(a.rank, SH_WARPS / KW), SH_WARPS * 32, 0, st>>>(a, S, ldS, cnt, list);
    return cudaGetLastError();
}

// ---- a few rows --------------------------------------------------------------------------------
// A decode step of one request is 2 flops per weight and row: CUDA cores stream W as fast as HBM gives
// it, without the swapped product's splits, slices and tensor maps.  A CTA takes an equal range of W's
// rows; the steps of that range (two rows by 2 KB of K) are one line that its 16 warps share equally,
// each with the next step's 4 KB in flight (64 KB an SM besides what it works on).  A row's dots are
// summed over a warp's lanes together (each step halves what a lane holds) and over the warps through
// shared memory in warp order, with fp32 sums throughout.  S, fp32, comes from a small kernel beside it
// and is needed only at the end, where 8 threads take an output: the warps' sums, S B_a^T, bias,
// activation.  HBM bounds it: bf16, 4096 x 4096, rank 16: 11.7 us (2.9 TB/s with launch and ramp), 15360
// x 5120: 29 us (5.4 TB/s).
// bf16, one row against the swapped product: 4096 x 4096 12.0 and 15.9 us, 15360 x 5120 29 and 33, 5120
// x 20480 36 and 43, 20480 x 5120 rank 64 39 and 47; two rows: 14.0 and 15.8, 33.4 and 33.1, 40 and 43,
// 44 and 47; four rows (17.7 and 16.1, 47 and 34, 57 and 43, 67 and 49) are the product's.
// fp32, in groups of up to 8 rows, against the tiled product: 4096 x 4096, 1 row 16 and 71 us, 8 rows
// 26 and 84, 24 rows 68 and 89, 32 rows 89 and 89; 2048 x 2048: 8.5 and 24, 13 and 29, 30 and 32, 38
// and 33.
constexpr int ROWS_MOST = 2, ROWS_MOST_F32 = 24;
constexpr int ROW_WARPS = 16;

// the elements of 16 bytes, in fp32
template <typename T>
__device__ __forceinline__ void floats_of(const uint4& u, float* f);
template <>
__device__ __forceinline__ void floats_of<__nv_bfloat16>(const uint4& u, float* f) { bf8(u, f); }
template <>
__device__ __forceinline__ void floats_of<float>(const uint4& u, float* f) {
    f[0] = __uint_as_float(u.x);
    f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z);
    f[3] = __uint_as_float(u.w);
}

template <typename T>
__global__ void __launch_bounds__(SH_WARPS * 32) adapter_row_shrink_kernel(AdapterArgs a, float* __restrict__ S) {
    __shared__ float parts[SH_WARPS];
    grid_dep_launch();
    const int m = blockIdx.x / a.rank, j = blockIdx.x % a.rank;
    const int id = a.ids[m], lane = threadIdx.x & 31;
    if (id < 0 || id >= a.n_adapters) return;
    constexpr int E = 16 / sizeof(T);
    const uint4* x = reinterpret_cast<const uint4*>(static_cast<const T*>(a.x) + (size_t)m * a.K);
    const uint4* f = reinterpret_cast<const uint4*>(static_cast<const T*>(a.A) + ((size_t)id * a.rank + j) * a.K);
    float s[2] = {0.f, 0.f};
#pragma unroll 4
    for (int k = threadIdx.x; k < a.K / E; k += SH_WARPS * 32) {
        float xv[E], fv[E];
        floats_of<T>(__ldg(x + k), xv);
        floats_of<T>(__ldg(f + k), fv);
#pragma unroll
        for (int i = 0; i < E; ++i) s[i & 1] = fmaf(xv[i], fv[i], s[i & 1]);
    }
    const float v = warp_sum(s[0] + s[1]);
    if (lane == 0) parts[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        float t = 0.f;
        for (int w = 0; w < SH_WARPS; ++w) t += parts[w];
        S[(size_t)m * a.rank + j] = t * a.scale[id];
    }
}

__device__ __forceinline__ uint4 load_once(const uint4* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

template <typename T, int MR>
__global__ void __launch_bounds__(ROW_WARPS * 32, 1)
    adapter_rows_kernel(AdapterArgs a, const float* __restrict__ S, int per) {
    constexpr int RB = 2, U = 4, V = MR * RB;          // rows and 512-byte chunks of K of a step
    constexpr int E = 16 / sizeof(T), PASS = MR <= 4 ? 128 : 64;      // W rows between two looks at S
    __shared__ float red[ROW_WARPS][PASS * MR];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, KE = a.K / E;
    const int m0 = (int)blockIdx.y * MR, mr = min(MR, a.M - m0);      // the CTA's rows of x
    const int first = (int)blockIdx.x * per, last = min(a.N, first + per);
    const int groups = (KE + 32 * U - 1) / (32 * U);
    const uint4* W = static_cast<const uint4*>(a.W);
    const uint4* X = static_cast<const uint4*>(a.x);
    const size_t ldb = (size_t)a.n_adapters * a.rank;
    for (int p0 = first; p0 < last; p0 += PASS) {
        const int rows = min(PASS, last - p0), line = (rows + RB - 1) / RB * groups;
        const int share = (line + ROW_WARPS - 1) / ROW_WARPS;
        const int s0 = min(line, warp * share), steps = min(line, s0 + share) - s0;
        for (int i = lane; i < rows * MR; i += 32) red[warp][i] = 0.f;
        __syncwarp();
        uint4 w[2][RB * U];
        int lr = s0 / groups * RB, lg = s0 % groups;   // the next load's rows and chunks
        auto load = [&](uint4* to) {
#pragma unroll
            for (int i = 0; i < RB; ++i)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int k = (lg * U + u) * 32 + lane;
                    to[i * U + u] = lr + i < rows && k < KE ? load_once(W + (size_t)(p0 + lr + i) * KE + k)
                                                            : make_uint4(0u, 0u, 0u, 0u);
                }
            if (++lg == groups) {
                lg = 0;
                lr += RB;
            }
        };
        int r = lr, g = lg;                            // the next step to use
        float acc[V];
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.f;
        auto use = [&](const uint4* from, bool end) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = (g * U + u) * 32 + lane;
                float wv[RB][E];
#pragma unroll
                for (int i = 0; i < RB; ++i) floats_of<T>(from[i * U + u], wv[i]);
#pragma unroll
                for (int m = 0; m < MR; ++m) {
                    float xv[E];
                    floats_of<T>(k < KE && m < mr ? __ldg(X + (size_t)(m0 + m) * KE + k) : make_uint4(0u, 0u, 0u, 0u), xv);
#pragma unroll
                    for (int i = 0; i < RB; ++i)
#pragma unroll
                        for (int q = 0; q < E; ++q) acc[i * MR + m] = fmaf(xv[q], wv[i][q], acc[i * MR + m]);
                }
            }
            if (++g < groups && !end) return;
            // the lanes' sums: a lane keeps the half of its dots that its bit of the step names
            int at = 0;
#pragma unroll
            for (int n = V / 2, o = 16; o > 0; n >>= 1, o >>= 1) {
                if (n > 0) {
                    const bool hi = lane & o;
                    at = at * 2 + (hi ? 1 : 0);
#pragma unroll
                    for (int i = 0; i < n; ++i) {
                        const float send = hi ? acc[i] : acc[i + n], keep = hi ? acc[i + n] : acc[i];
                        acc[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                    }
                } else {
                    acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], o);
                }
            }
            if (lane % (32 / V) == 0 && r + at / MR < rows) red[warp][r * MR + at] = acc[0];
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = 0.f;
            g = 0;
            r += RB;
        };
        if (steps > 0) load(w[0]);
        for (int step = 0; step < steps; step += 2) {
            if (step + 1 < steps) load(w[1]);
            use(w[0], step + 1 == steps);
            if (step + 1 < steps) {
                if (step + 2 < steps) load(w[0]);
                use(w[1], step + 2 == steps);
            }
        }
        grid_dep_wait();                               // S
        __syncthreads();
        for (int q = tid >> 3; q < rows * MR; q += ROW_WARPS * 4) {
            const int n = p0 + q / MR, m = q % MR, l8 = tid & 7;
            const int id = m < mr ? a.ids[m0 + m] : -1;
            float v = red[l8][q] + red[l8 + 8][q];
            if (id >= 0 && id < a.n_adapters) {
                const T* b = static_cast<const T*>(a.B) + (size_t)n * ldb + (size_t)id * a.rank;
                for (int j = l8; j < a.rank; j += 8)
                    v = fmaf(S[(size_t)(m0 + m) * a.rank + j], (float)b[j], v);
            }
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffu << (lane & 24), v, o);
            if (id < -1 || id >= a.n_adapters) v = __int_as_float(0x7fc00000);
            if (l8 == 0 && m < mr) adapter_store<T>(a, m0 + m, n, v);
        }
        __syncthreads();
    }
}

template <typename T, int MR>
cudaError_t launch_rows(const AdapterArgs& a, cudaStream_t st) {
    float* S = static_cast<float*>(a.ws);
    adapter_row_shrink_kernel<T><<<a.M * a.rank, SH_WARPS * 32, 0, st>>>(a, S);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int per = (a.N + 147) / 148;
    return launch_pdl(adapter_rows_kernel<T, MR>, dim3(cdiv(a.N, per), cdiv(a.M, MR)), dim3(ROW_WARPS * 32), 0, st, a,
                      static_cast<const float*>(S), per);
}

// The slices' reduction of the decode form: one thread per 4 columns of a row adds them in split
// order, with bias and activation; sums that are not finite are taken anew from the row's own factors.
__global__ void __launch_bounds__(128)
    adapter_reduce_kernel(AdapterArgs a, const __nv_bfloat16* __restrict__ S, int ldS,
                          const float* __restrict__ ws, int ks) {
    const int m = blockIdx.y, n = (blockIdx.x * blockDim.x + threadIdx.x) * 4;
    const int id = a.ids[m];
    grid_dep_wait();
    if (n >= a.N) return;
    float y[4] = {0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < ks; ++k) {
        const float4 w = *reinterpret_cast<const float4*>(ws + ((size_t)k * a.M + m) * a.N + n);
        y[0] += w.x; y[1] += w.y; y[2] += w.z; y[3] += w.w;
    }
    const bool none = id < -1 || id >= a.n_adapters;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (none) y[i] = __int_as_float(0x7fc00000);
        else if (!isfinite(y[i])) y[i] = adapter_element(a, S, ldS, m, n + i, id, 0, 1);
        if (a.bias) y[i] += a.bias[n + i];
        if (a.act == 1) y[i] = y[i] < 0.f ? 0.f : y[i];       // a NaN stays
    }
    const size_t at = (size_t)m * a.N + n;
    if (a.accumulate) {
        float4* c = reinterpret_cast<float4*>(static_cast<float*>(a.y) + at);
        float4 o = *c;
        o.x += y[0]; o.y += y[1]; o.z += y[2]; o.w += y[3];
        *c = o;
    } else {
        __nv_bfloat162 lo = __floats2bfloat162_rn(y[0], y[1]), hi = __floats2bfloat162_rn(y[2], y[3]);
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.y) + at) =
            make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
    }
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

// Elements that the product's epilogue named, in the chunks of 32 rows x 32 columns that it marked, and rows
// whose id names no adapter: the elements are computed anew from the rows' own factors, and rows without an
// adapter to name become NaN.  On finite weights nothing is marked and the kernel only reads the
// marks.  A warp takes a chunk, lists its elements and computes 8 at a time, so that 16 loads are in
// flight (4093 rows, 20480 x 5120, 0.63 ms: one NaN row, all of its outputs, 0.5 ms more; in CTAs of 128
// chunks instead of 32 4.3 ms more and 2 us less when nothing is marked; whole chunks of 32 rows computed
// element by element 229 ms more, and with other bits in the 31 rows beside it).
constexpr int FIX_THREADS = 256, FIX_CHUNKS = 32, FIX_N = 8;
__global__ void __launch_bounds__(FIX_THREADS)
    adapter_repair_kernel(AdapterArgs a, const __nv_bfloat16* __restrict__ S, int ldS,
                          const uint8_t* __restrict__ odd, const uint32_t* __restrict__ bits) {
    grid_dep_wait();
    __shared__ uint16_t elems[FIX_THREADS / 32][1024];           // row << 5 | column
    const int chunks = (a.N + 31) / 32, m0 = blockIdx.x * 32;
    const int c0 = blockIdx.y * FIX_CHUNKS, c1 = min(chunks, c0 + FIX_CHUNKS);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int id_l = m0 + lane < a.M ? a.ids[m0 + lane] : -1;
    const unsigned none = __ballot_sync(0xffffffffu, id_l < -1 || id_l >= a.n_adapters);
    // usually nothing is marked: all of the CTA's marks in one look
    int any = none != 0u;
    for (int c = c0 + (int)threadIdx.x; c < c1; c += FIX_THREADS) any |= odd[(size_t)blockIdx.x * chunks + c];
    if (!__syncthreads_or(any)) return;
    for (int c = c0 + warp; c < c1; c += FIX_THREADS / 32) {
        const int n0 = c * 32;
        for (unsigned rows = none; rows; rows &= rows - 1)
            if (n0 + lane < a.N) adapter_store(a, m0 + __ffs(rows) - 1, n0 + lane, __int_as_float(0x7fc00000));
        if (!odd[(size_t)blockIdx.x * chunks + c]) continue;
        uint32_t mine = m0 + lane < a.M && !((none >> lane) & 1u) ? bits[(size_t)(m0 + lane) * chunks + c] : 0u;
        if (a.N - n0 < 32) mine &= (1u << (a.N - n0)) - 1u;
        int end = __popc(mine);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, end, o);
            if (lane >= o) end += v;
        }
        const int total = __shfl_sync(0xffffffffu, end, 31);
        __syncwarp();                          // the list before has been read
        for (int at = end - __popc(mine); mine; mine &= mine - 1) elems[warp][at++] = (uint16_t)(lane << 5 | (__ffs(mine) - 1));
        __syncwarp();
        for (int e0 = 0; e0 < total; e0 += FIX_N) {
            const uint4 *x[FIX_N], *w[FIX_N];
            const __nv_bfloat16 *s[FIX_N], *f[FIX_N];
            bool has[FIX_N];
            float v[FIX_N];
#pragma unroll
            for (int i = 0; i < FIX_N; ++i) {
                const int e = elems[warp][min(e0 + i, total - 1)];
                x[i] = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.x) + (size_t)(m0 + (e >> 5)) * a.K);
                w[i] = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.W) + (size_t)(n0 + (e & 31)) * a.K);
                v[i] = 0.f;
            }
            for (int k = lane; k < a.K / 8; k += 32) {
                uint4 xu[FIX_N], wu[FIX_N];
#pragma unroll
                for (int i = 0; i < FIX_N; ++i) {
                    xu[i] = __ldg(x[i] + k);
                    wu[i] = __ldg(w[i] + k);
                }
#pragma unroll
                for (int i = 0; i < FIX_N; ++i) {
                    float xv[8], wv[8];
                    bf8(xu[i], xv);
                    bf8(wu[i], wv);
#pragma unroll
                    for (int q = 0; q < 8; ++q) v[i] = fmaf(xv[q], wv[q], v[i]);
                }
            }
            // the expand, the row's own factors (rows of a chunk may have several adapters)
#pragma unroll
            for (int i = 0; i < FIX_N; ++i) {
                const int e = elems[warp][min(e0 + i, total - 1)], id = __shfl_sync(0xffffffffu, id_l, e >> 5);
                s[i] = S + (size_t)(m0 + (e >> 5)) * ldS + (size_t)max(id, 0) * a.rank;
                f[i] = static_cast<const __nv_bfloat16*>(a.B) + (size_t)(n0 + (e & 31)) * a.n_adapters * a.rank +
                       (size_t)max(id, 0) * a.rank;
                has[i] = id >= 0;
            }
            for (int k = lane; k < a.rank; k += 32)
#pragma unroll
                for (int i = 0; i < FIX_N; ++i)
                    if (has[i]) v[i] = fmaf(__bfloat162float(s[i][k]), __bfloat162float(f[i][k]), v[i]);
#pragma unroll
            for (int i = 0; i < FIX_N; ++i) {
                const float y = warp_sum(v[i]);
                const int e = elems[warp][min(e0 + i, total - 1)];
                if (lane == i && e0 + i < total) adapter_store(a, m0 + (e >> 5), n0 + (e & 31), y);
            }
        }
    }
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Where the decode form is taken: up to 128 rows, and up to 1024 while its 128 x 128 tiles are at most
// one a SM, the factors' columns, all of whose listed blocks every tile goes through, no more than K's,
// and the shrink, here on CUDA cores, 24576 dots at most.  It splits K over the SMs that the tiles leave idle; the tiles form has 256 x 256 tiles for SM
// pairs and no split.  128 rows of the OPT-13B FFN input under 32 adapters of rank 16: 68 us, the tiles
// form 101; under 8 adapters, 2048 x 2048: 256 rows 17 and 41, 1024 rows (128 tiles) 36 and 42; 4096 x
// 4096: 256 rows 28 and 56, 512 rows (128 tiles) 43 and 57, 768 rows (192) 60 and 57; 6144 x 4096 under
// 32: 384 rows (144) 43 and 59, 768 rows (288) 74 and 60; 15360 x 5120: 256 rows (240) 74 and 70.  By
// the dots, 4096 x 4096 under rank 64: 384 rows (24576) 52 and 58, 512 rows (32768) 65 and 59; 2048 x
// 2048, rank 32: 768 rows (24576) 37 and 43, 1024 rows (32768) 45 and 43.
bool step_form(int M, int N, int K, int K2, int rank) {
    if (M <= 128) return true;
    return M <= 1024 && M * rank <= 24576 && K2 <= K &&
           (long long)((M + 127) / 128) * ((N + 127) / 128) <= 148;
}

// Slices of the decode form: room for up to 16 splits, 64 MB at most unless one slice is more.
size_t slice_floats(int M, int N) {
    const size_t one = (size_t)M * N;
    const size_t most = SLICES_MOST / 4 / one;
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
    size_t list, s, odd, bits, total;     // offsets
    int blocks, n_list, ld;
};
TileSpace tile_space(int M, int N, int K2) {
    TileSpace t;
    const int rows = pass_rows(M, K2);
    t.blocks = (rows + 255) / 256;
    const int blocks = (K2 + 63) / 64;
    t.n_list = (blocks + 7) / 8 * 8;      // lists are read 8 entries at a time
    t.ld = blocks * 64;
    t.list = up256((size_t)t.blocks * 4);
    t.s = t.list + up256((size_t)t.blocks * t.n_list * 4);
    t.odd = t.s + up256((size_t)rows * t.ld * 2);
    t.bits = t.odd + up256((size_t)((rows + 31) / 32) * ((N + 31) / 32));
    t.total = t.bits + up256((size_t)rows * ((N + 31) / 32) * 4);
    return t;
}

}  // namespace

size_t adapter_workspace(int M, int N, int K, int n_adapters, int rank, int dtype) {
    const size_t s = up256((size_t)M * rank * 4) + 256;
    if (M == 0) return s;
    if (dtype != E_BF16) return s + up256(f32_slice_floats(M, N, K) * 4);
    size_t t = tile_space(M, N, n_adapters * rank).total;
    if (step_form(M, N, K, n_adapters * rank, rank)) t += up256(slice_floats(M, N) * 4);
    return t > s ? t : s;
}

template <bool VEC>
static cudaError_t launch_shrink(const AdapterArgs& a, float* S, cudaStream_t st) {
    static std::atomic<uint64_t> share{0};
    const cudaError_t e = smem_share(reinterpret_cast<const void*>(adapter_shrink_kernel<VEC>), share);
    if (e != cudaSuccess) return e;
    adapter_shrink_kernel<VEC><<<dim3(a.M, cdiv(a.rank, SH_WARPS)), SH_WARPS * 32, 0, st>>>(a, S);
    return cudaGetLastError();
}

cudaError_t launch_linear_adapters_simt(const AdapterArgs& a, cudaStream_t st) {
    float* S = static_cast<float*>(a.ws);
    const uintptr_t mix = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.W) |
                          reinterpret_cast<uintptr_t>(a.A);
    const bool rows16 = a.dtype == E_F32 && a.K % 4 == 0 && mix % 16 == 0;       // 16-byte loads
    if (rows16 && a.M <= ROWS_MOST_F32)
        return a.M == 1   ? launch_rows<float, 1>(a, st)
               : a.M == 2 ? launch_rows<float, 2>(a, st)
               : a.M <= 4 ? launch_rows<float, 4>(a, st)
                          : launch_rows<float, 8>(a, st);
    cudaError_t e;
    if (rows16) {
        static std::atomic<uint64_t> attr{0};
        e = smem_limit(reinterpret_cast<const void*>(gemm_f32_kernel), F_SMEM, attr);
        if (e != cudaSuccess) return e;
        float* slices = reinterpret_cast<float*>(static_cast<char*>(a.ws) + up256((size_t)a.M * a.rank * 4));
        const int rows = f32_pass_rows(a.M, a.N);
        for (int m0 = 0; m0 < a.M; m0 += rows) {
            AdapterArgs b = a;
            b.M = a.M - m0 < rows ? a.M - m0 : rows;
            b.x = static_cast<const float*>(a.x) + (size_t)m0 * a.K;
            b.ids = a.ids + m0;
            b.y = static_cast<float*>(a.y) + (size_t)m0 * a.N;
            e = launch_shrink<true>(b, S, st);
            if (e != cudaSuccess) return e;
            const int ks = f32_splits(b.M, a.N, a.K);
            // The product beside the shrink, unless the shrink is long: then the two fight for L1 and the
            // shrink reads x again and again from L2 (301 rows, 1544 x 1000: rank 8 45 us beside and 48
            // behind, rank 64 100 and 66; 2048 x 2048, rank 32: 84 and 88, with adapters changing from row to
            // row 107 and 103).
            const dim3 grid(cdiv(a.N, FM), cdiv(b.M, FM), ks);
            const float *x = static_cast<const float*>(b.x), *W = static_cast<const float*>(a.W);
            if (a.N >= 64 * a.rank) {
                e = launch_pdl(gemm_f32_kernel, grid, dim3(F_THREADS), F_SMEM, st, x, W, b.M, a.N, a.K, ks, slices);
            } else {
                gemm_f32_kernel<<<grid, F_THREADS, F_SMEM, st>>>(x, W, b.M, a.N, a.K, ks, slices);
                e = cudaGetLastError();
            }
            if (e != cudaSuccess) return e;
            e = launch_pdl(adapter_expand_f32_kernel, dim3(cdiv(b.M, ER), cdiv(a.N, 128)), dim3(128), 0, st, b,
                           static_cast<const float*>(S), static_cast<const float*>(slices), ks);
            if (e != cudaSuccess) return e;
        }
        return cudaSuccess;
    }
    e = launch_shrink<false>(a, S, st);
    if (e != cudaSuccess) return e;
    adapter_gemm_kernel<<<dim3(cdiv(a.N, BN), cdiv(a.M, BM)), 256, 0, st>>>(a, S);
    return cudaGetLastError();
}

cudaError_t launch_adapter_reduce(const AdapterArgs& a, const AdapterTiles& t, const float* ws, int ks,
                                  cudaStream_t st, bool pdl) {
    const dim3 grid(cdiv(a.N / 4, 128), a.M);
    const __nv_bfloat16* S = static_cast<const __nv_bfloat16*>(t.S);
    if (pdl) return launch_pdl(adapter_reduce_kernel, grid, dim3(128), 0, st, a, S, t.ldS, ws, ks);
    adapter_reduce_kernel<<<grid, 128, 0, st>>>(a, S, t.ldS, ws, ks);
    return cudaGetLastError();
}

bool linear_adapters_tc_supported(const AdapterArgs& a) {
    const uintptr_t mix = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.W) |
                          reinterpret_cast<uintptr_t>(a.A) | reinterpret_cast<uintptr_t>(a.B) |
                          reinterpret_cast<uintptr_t>(a.y) | reinterpret_cast<uintptr_t>(a.bias);
    return a.dtype == E_BF16 && a.K % 8 == 0 && a.N % 8 == 0 && (a.n_adapters * a.rank) % 8 == 0 &&
           mix % 16 == 0;
}

cudaError_t launch_linear_adapters_tc(const AdapterArgs& a, cudaStream_t st, bool few) {
    if (few && a.M <= ROWS_MOST)
        return a.M == 1 ? launch_rows<__nv_bfloat16, 1>(a, st) : launch_rows<__nv_bfloat16, 2>(a, st);
    char* ws = static_cast<char*>(a.ws);
    const int K2 = a.n_adapters * a.rank;
    const TileSpace t = tile_space(a.M, a.N, K2);
    AdapterTiles at;
    int* cnt = reinterpret_cast<int*>(ws);
    int* list = reinterpret_cast<int*>(ws + t.list);
    at.cnt = cnt;
    at.list = list;
    at.n_list = t.n_list;
    at.S = ws + t.s;
    at.ldS = t.ld;
    at.odd = reinterpret_cast<uint8_t*>(ws + t.odd);
    at.bits = reinterpret_cast<uint32_t*>(ws + t.bits);
    if (step_form(a.M, a.N, a.K, K2, a.rank)) {
        GemmArgs g;
        memset(&g, 0, sizeof(g));
        g.A = a.x; g.lda = a.K; g.a_type = E_BF16;
        g.B = a.W; g.ldb = a.K; g.b_type = E_BF16;
        g.M = a.M; g.N = a.N; g.K = a.K;
        g.epi = a.accumulate ? EPI_RESID : a.act ? EPI_STORE_RELU : EPI_STORE;
        g.bias = a.bias;
        g.C = a.y; g.ldc = a.N; g.c_type = a.accumulate ? E_F32 : E_BF16;
        g.ws = reinterpret_cast<float*>(ws + t.total);
        g.ws_floats = slice_floats(a.M, a.N);
        g.adapt = &a;
        g.adapt_tiles = &at;
        if (!gemm_tc_supported(g)) return cudaErrorNotSupported;
        __nv_bfloat16* S = static_cast<__nv_bfloat16*>(at.S);
        const cudaError_t e = a.M * a.rank <= 2 * 148 ? launch_shrink_rows<SH_WARPS>(a, S, t.ld, cnt, list, st)
                                                      : launch_shrink_rows<1>(a, S, t.ld, cnt, list, st);
        if (e != cudaSuccess) return e;
        return gemm_tc(g, st) ? cudaErrorUnknown : cudaSuccess;
    }
    const int rows = pass_rows(a.M, K2);
    for (int m0 = 0; m0 < a.M; m0 += rows) {
        AdapterArgs b = a;
        b.M = a.M - m0 < rows ? a.M - m0 : rows;
        b.x = static_cast<const __nv_bfloat16*>(a.x) + (size_t)m0 * a.K;
        b.ids = a.ids + m0;
        b.y = static_cast<char*>(a.y) + (size_t)m0 * a.N * (a.accumulate ? 4 : 2);
        adapter_lists_kernel<<<cdiv(b.M, 256), 256, 0, st>>>(b.ids, b.M, b.n_adapters, b.rank, cnt, list, at.n_list);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        if (gemm_tc_adapters(b, at, st)) return cudaErrorUnknown;
        e = launch_pdl(adapter_repair_kernel, dim3(cdiv(b.M, 32), cdiv(cdiv(b.N, 32), FIX_CHUNKS)),
                       dim3(FIX_THREADS), 0, st, b, static_cast<const __nv_bfloat16*>(at.S), at.ldS,
                       static_cast<const uint8_t*>(at.odd), static_cast<const uint32_t*>(at.bits));
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace zo
