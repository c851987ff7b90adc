// Kernel-level entry points (include/zo_ops.h): argument checks and launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdlib>
#include <cstring>
#include <algorithm>
#include <string>
#include <vector>

#include "../../include/zo.h"
#include "../../include/zo_ops.h"
#include "kernels.h"

using namespace zo;

namespace {
thread_local std::string t_op_err;

// ZO_OK, or ZO_ERR_CUDA with the CUDA error (a failed launch, or an earlier asynchronous
// error the launch ran into) kept for zo_op_last_error
int op_status() {
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) return ZO_OK;
    t_op_err = std::string(cudaGetErrorName(e)) + ": " + cudaGetErrorString(e);
    return ZO_ERR_CUDA;
}
int op_fail(const char* what) {
    const cudaError_t e = cudaGetLastError();
    t_op_err = what;
    if (e != cudaSuccess) t_op_err += std::string(" (") + cudaGetErrorName(e) + ")";
    return ZO_ERR_CUDA;
}

bool use_tc(int32_t impl, int dtype) {
    if (impl == ZO_IMPL_CUDA_CORES) return false;
    return dtype == ZO_DTYPE_BF16;
}

// the exponent of a cache page size (8, 16, .. 256 tokens), or -1
int page_shift(int32_t page_size) {
    for (int s = 3; s <= 8; ++s)
        if (page_size == 1 << s) return s;
    return -1;
}
}  // namespace

extern "C" {

int zo_op_quantize_rows_e4m3(const void* x, int32_t dtype, int32_t rows, int32_t cols,
                             uint8_t* q, float* scale, void* stream) {
    if (!x || !q || !scale || rows < 0 || cols <= 0) return ZO_ERR_ARG;
    if (dtype != ZO_DTYPE_FP32 && dtype != ZO_DTYPE_BF16) return ZO_ERR_ARG;
    launch_quant_rows_e4m3(x, dtype == ZO_DTYPE_BF16 ? E_BF16 : E_F32, rows, cols, (size_t)cols, q,
                           (size_t)cols, scale, static_cast<cudaStream_t>(stream));
    return op_status();
}

int zo_op_linear_fp8(const uint8_t* xq, const float* sx, const uint8_t* wq, const float* sw,
                     const float* bias, void* y, int32_t M, int32_t N, int32_t K, int32_t act,
                     void* stream) {
    if (!xq || !sx || !wq || !sw || !y || M < 0 || N <= 0 || K <= 0) return ZO_ERR_ARG;
    if (act != ZO_ACT_NONE && act != ZO_ACT_RELU) return ZO_ERR_ARG;
    GemmArgs g;
    memset(&g, 0, sizeof(g));
    g.A = xq; g.lda = K; g.a_type = E_FP8;
    g.B = wq; g.ldb = K; g.b_type = E_FP8;
    g.a_scale = sx; g.b_scale = sw;
    g.M = M; g.N = N; g.K = K;
    g.bias = bias;
    g.epi = act == ZO_ACT_RELU ? EPI_STORE_RELU : EPI_STORE;
    g.C = y; g.ldc = N; g.c_type = E_BF16;
    if (M == 0) return ZO_OK;
    if (!gemm_tc_supported(g)) return ZO_ERR_UNSUPPORTED;
    if (gemm_tc(g, static_cast<cudaStream_t>(stream))) return op_fail("tensor-core GEMM launch failed");
    return op_status();
}

int zo_op_linear(const void* x, const void* W, const float* bias, void* y, int32_t M, int32_t N,
                 int32_t K, int32_t dtype, int32_t act, int32_t accumulate, int32_t impl,
                 void* stream) {
    if (!x || !W || !y || M < 0 || N <= 0 || K <= 0) return ZO_ERR_ARG;
    if (dtype != ZO_DTYPE_FP32 && dtype != ZO_DTYPE_BF16) return ZO_ERR_ARG;
    if (act != ZO_ACT_NONE && act != ZO_ACT_RELU) return ZO_ERR_ARG;
    if (accumulate && act != ZO_ACT_NONE) return ZO_ERR_ARG;
    GemmArgs g;
    memset(&g, 0, sizeof(g));
    const int t = dtype == ZO_DTYPE_BF16 ? E_BF16 : E_F32;
    g.A = x; g.lda = K; g.a_type = t;
    g.B = W; g.ldb = K; g.b_type = t;
    g.M = M; g.N = N; g.K = K;
    g.bias = bias;
    g.epi = accumulate ? EPI_RESID : (act == ZO_ACT_RELU ? EPI_STORE_RELU : EPI_STORE);
    g.C = y; g.ldc = N; g.c_type = accumulate ? E_F32 : t;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (M == 0) return ZO_OK;
    if (use_tc(impl, dtype)) {
        if (gemm_tc_supported(g)) {
            if (gemm_tc(g, st)) return op_fail("tensor-core GEMM launch failed");
            return op_status();
        }
        if (impl == ZO_IMPL_TENSOR_CORES) return ZO_ERR_UNSUPPORTED;
    } else if (impl == ZO_IMPL_TENSOR_CORES) {
        return ZO_ERR_UNSUPPORTED;
    }
    gemm_simt(g, st);
    return op_status();
}

int zo_op_linear_decode(const void* x, const void* W, const float* bias, void* y, int32_t M,
                        int32_t N, int32_t K, int32_t act, int32_t accumulate, float* ws,
                        size_t ws_floats, void* stream) {
    if (M < 0 || N <= 0 || K <= 0) return ZO_ERR_ARG;
    if (act != ZO_ACT_NONE && act != ZO_ACT_RELU) return ZO_ERR_ARG;
    if (accumulate && act != ZO_ACT_NONE) return ZO_ERR_ARG;
    if (M == 0) return ZO_OK;
    if (!x || !W || !y || !ws || ws_floats < (size_t)M * N) return ZO_ERR_ARG;
    if (K % 8 || N % 4) return ZO_ERR_UNSUPPORTED;
    GemmArgs g;
    memset(&g, 0, sizeof(g));
    g.A = x; g.lda = K; g.a_type = E_BF16;
    g.B = W; g.ldb = K; g.b_type = E_BF16;
    g.M = M; g.N = N; g.K = K;
    g.bias = bias;
    g.epi = accumulate ? EPI_RESID : (act == ZO_ACT_RELU ? EPI_STORE_RELU : EPI_STORE);
    g.C = y; g.ldc = N; g.c_type = accumulate ? E_F32 : E_BF16;
    g.ws = ws; g.ws_floats = ws_floats;
    if (!gemm_tc_supported(g)) return ZO_ERR_UNSUPPORTED;
    if (gemm_tc(g, static_cast<cudaStream_t>(stream))) return op_fail("tensor-core GEMM launch failed");
    return op_status();
}

size_t zo_op_lm_head_workspace(int32_t n_rows, int32_t vocab, int32_t impl) {
    (void)impl;
    const size_t tiles = (size_t)gemm_lse_col_tiles(vocab);
    const size_t part = ((size_t)n_rows * tiles * 4 + 255) / 256 * 256;
    const size_t tg = ((size_t)n_rows * 4 + 255) / 256 * 256;
    return 2 * part + tg;
}

int zo_op_lm_head_logprob(const void* h, const void* E, const int32_t* targets, int32_t n_rows,
                          int32_t vocab, int32_t d, int32_t dtype, float* logprob,
                          void* workspace, size_t workspace_bytes, int32_t impl, void* stream) {
    if (!h || !E || !targets || !logprob || n_rows < 0 || vocab <= 0 || d <= 0) return ZO_ERR_ARG;
    if (dtype != ZO_DTYPE_FP32 && dtype != ZO_DTYPE_BF16) return ZO_ERR_ARG;
    if (n_rows == 0) return ZO_OK;
    const size_t need = zo_op_lm_head_workspace(n_rows, vocab, impl);
    if (!workspace || workspace_bytes < need) return ZO_ERR_ARG;
    if (reinterpret_cast<uintptr_t>(workspace) % 256) return ZO_ERR_ARG;
    const int tiles = gemm_lse_col_tiles(vocab);   // the larger count: both paths fit
    const size_t part = ((size_t)n_rows * tiles * 4 + 255) / 256 * 256;
    char* ws = static_cast<char*>(workspace);
    float* pmax = reinterpret_cast<float*>(ws);
    float* psum = reinterpret_cast<float*>(ws + part);
    float* tgt = reinterpret_cast<float*>(ws + 2 * part);
    const int t = dtype == ZO_DTYPE_BF16 ? E_BF16 : E_F32;
    GemmArgs g;
    memset(&g, 0, sizeof(g));
    g.A = h; g.lda = d; g.a_type = t;
    g.B = E; g.ldb = d; g.b_type = t;
    g.M = n_rows; g.N = vocab; g.K = d;
    g.epi = EPI_LSE;
    g.targets = targets; g.part_max = pmax; g.part_sum = psum; g.tgt_logit = tgt;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool tc = use_tc(impl, dtype) && gemm_tc_supported(g);
    if (impl == ZO_IMPL_TENSOR_CORES && !tc) return ZO_ERR_UNSUPPORTED;
    g.n_col_tiles = tc ? gemm_tc_col_tiles(vocab) : tiles;
    if (tc) {
        if (gemm_tc(g, st)) return op_fail("tensor-core GEMM launch failed");
    } else {
        gemm_simt(g, st);
    }
    launch_lse_merge(pmax, psum, tgt, n_rows, g.n_col_tiles, logprob, st);
    return op_status();
}

int zo_op_attention(const void* qkv, void* out, const int32_t* seq_lens, int32_t n_rows,
                    int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, int32_t dtype,
                    void* workspace, size_t workspace_bytes, int32_t impl, void* stream) {
    if (!qkv || !out || !seq_lens || n_rows < 0 || n_heads <= 0 || n_kv_heads <= 0) return ZO_ERR_ARG;
    if (n_heads % n_kv_heads) return ZO_ERR_ARG;
    if (head_dim != 32 && head_dim != 64 && head_dim != 128 && head_dim != 256)
        return ZO_ERR_UNSUPPORTED;
    if (dtype != ZO_DTYPE_FP32 && dtype != ZO_DTYPE_BF16) return ZO_ERR_ARG;
    if (n_rows == 0) return ZO_OK;
    if (n_rows >= 32768) return ZO_ERR_ARG;
    std::vector<int> meta(n_rows + 1);
    meta[0] = 0;
    const bool tc = use_tc(impl, dtype) && (head_dim == 64 || head_dim == 128);
    if (impl == ZO_IMPL_TENSOR_CORES && !tc) return ZO_ERR_UNSUPPORTED;
    const int qtile = tc ? 128 : 64;
    std::vector<int> tiles;
    for (int r = 0; r < n_rows; ++r) {
        if (seq_lens[r] < 1 || seq_lens[r] > 65535 * 64) return ZO_ERR_ARG;
        meta[r + 1] = meta[r] + seq_lens[r];
        for (int q = 0; q < (seq_lens[r] + qtile - 1) / qtile; ++q) tiles.push_back((r << 16) | q);
    }
    // attention CTAs are issued in item order: longest (most key chunks) first
    if (tc)
        std::stable_sort(tiles.begin(), tiles.end(),
                         [](int x, int y) { return (x & 0xFFFF) > (y & 0xFFFF); });
#ifdef ZO_DEBUG
    // test hook of the debug build: ZO_DEBUG_PLANT=attention_tile makes the last work tile
    // name a row past the batch; the kernels' bounds checks must report it and skip it
    if (const char* plant = std::getenv("ZO_DEBUG_PLANT"))
        if (!std::strcmp(plant, "attention_tile") && !tiles.empty())
            tiles.back() = (n_rows << 16) | (tiles.back() & 0xFFFF);
#endif
    const size_t need = (meta.size() + tiles.size()) * 4;
    if (!workspace || workspace_bytes < need) return ZO_ERR_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int* w = static_cast<int*>(workspace);
    meta.insert(meta.end(), tiles.begin(), tiles.end());
    if (cudaMemcpyAsync(w, meta.data(), meta.size() * 4, cudaMemcpyHostToDevice, st) != cudaSuccess)
        return op_fail("copy of the row metadata failed");
    // the host vector must outlive the copy
    if (cudaStreamSynchronize(st) != cudaSuccess) return op_fail("stream synchronisation failed");
    AttnArgs a;
    memset(&a, 0, sizeof(a));
    a.qkv = qkv; a.ld_qkv = (n_heads + 2 * n_kv_heads) * head_dim;
    a.out = out; a.ld_out = n_heads * head_dim;
    a.dtype = dtype == ZO_DTYPE_BF16 ? E_BF16 : E_F32;
    a.cu_seqlens = w;
    a.tiles = w + n_rows + 1;
    a.n_tiles = (int)tiles.size();
    a.H = n_heads; a.Hkv = n_kv_heads; a.hd = head_dim;
    a.scale = (float)(1.0 / std::sqrt((double)head_dim));
    a.n_tokens = meta[n_rows];
    a.n_rows = n_rows;
    if (tc && attention_tc_supported(a)) {
        if (!launch_attention_tc(a, st)) return op_fail("tensor-core attention setup failed");
    } else if (impl == ZO_IMPL_TENSOR_CORES) {
        return ZO_ERR_UNSUPPORTED;
    } else {
        launch_attention(a, st);
    }
    return op_status();
}

int zo_op_linear_ext(const void* x, const void* W, const float* bias, const void* x2,
                     const void* W2, int32_t K2, void* y, int32_t ldy, int32_t M, int32_t N,
                     int32_t K, int32_t epi, const zo_qk_norm_rope_args* qk, void* stream) {
    if (!x || !W || !y || M < 0 || N <= 0 || K <= 0 || K2 < 0 || ldy <= 0) return ZO_ERR_ARG;
    if (K2 > 0 && (!x2 || !W2)) return ZO_ERR_ARG;
    GemmArgs g;
    memset(&g, 0, sizeof(g));
    switch (epi) {
        case ZO_EPI_STORE: g.epi = EPI_STORE; g.c_type = E_BF16; break;
        case ZO_EPI_RELU: g.epi = EPI_STORE_RELU; g.c_type = E_BF16; break;
        case ZO_EPI_RESID: g.epi = EPI_RESID; g.c_type = E_F32; break;
        case ZO_EPI_SWIGLU:
            if (N % 256) return ZO_ERR_UNSUPPORTED;
            g.epi = EPI_SWIGLU; g.c_type = E_BF16;
            if (ldy < N / 2) return ZO_ERR_ARG;
            break;
        case ZO_EPI_QK_NORM_ROPE:
            if (!qk || !qk->tok_pos || !qk->q_norm || !qk->k_norm || !qk->rope_cos ||
                !qk->rope_sin || qk->n_q_heads <= 0 || qk->n_kv_heads <= 0)
                return ZO_ERR_ARG;
            if (bias) return ZO_ERR_UNSUPPORTED;
            g.epi = EPI_QKNR; g.c_type = E_BF16;
            g.tok_pos = qk->tok_pos; g.qn = qk->q_norm; g.kn = qk->k_norm;
            g.rope_cos = qk->rope_cos; g.rope_sin = qk->rope_sin; g.norm_eps = qk->eps;
            g.n_q_heads = qk->n_q_heads; g.n_qk_heads = qk->n_q_heads + qk->n_kv_heads;
            if ((int64_t)(g.n_qk_heads + qk->n_kv_heads) * 128 != N) return ZO_ERR_ARG;
            break;
        default: return ZO_ERR_ARG;
    }
    if (epi != ZO_EPI_SWIGLU && ldy < N) return ZO_ERR_ARG;
    g.A = x; g.lda = K; g.a_type = E_BF16;
    g.B = W; g.ldb = K; g.b_type = E_BF16;
    if (K2 > 0) {
        g.A2 = x2; g.lda2 = K2; g.a2_type = E_BF16;
        g.B2 = W2; g.ldb2 = K2; g.b2_type = E_BF16;
        g.K2 = K2;
    }
    g.M = M; g.N = N; g.K = K;
    g.bias = bias;
    g.C = y; g.ldc = ldy;
    if (M == 0) return ZO_OK;
    if (!gemm_tc_supported(g)) return ZO_ERR_UNSUPPORTED;
    if (gemm_tc(g, static_cast<cudaStream_t>(stream))) return op_fail("tensor-core GEMM launch failed");
    return op_status();
}

int zo_op_rope_table(float* cos_t, float* sin_t, int32_t max_pos, int32_t head_dim, double theta,
                     void* stream) {
    if (!cos_t || !sin_t || max_pos <= 0 || head_dim <= 0 || head_dim % 2 || !(theta > 0.0))
        return ZO_ERR_ARG;
    launch_rope_table(cos_t, sin_t, max_pos, head_dim, theta, static_cast<cudaStream_t>(stream));
    return op_status();
}

int zo_op_block_tables(const int32_t* old_lens, const int32_t* new_lens, int32_t n_rows,
                       int32_t page_size, int32_t* block_table, int32_t max_blocks,
                       int32_t* free_ring, int32_t n_pages, const int32_t* state,
                       int32_t* state_out, int32_t* cu_new, int32_t* slot_map,
                       int32_t max_tokens, void* stream) {
    const int shift = page_shift(page_size);
    if (shift < 0 || n_rows < 0 || max_blocks < 1 || n_pages < 1 || max_tokens < 0) return ZO_ERR_ARG;
    if (((int64_t)n_pages << shift) > 0x7fffffffLL) return ZO_ERR_ARG;
    if (!free_ring || !state || !state_out || !cu_new || state == state_out) return ZO_ERR_ARG;
    if (n_rows > 0 && (!old_lens || !new_lens || !block_table)) return ZO_ERR_ARG;
    if (max_tokens > 0 && !slot_map) return ZO_ERR_ARG;
    if (launch_block_tables(old_lens, new_lens, n_rows, shift, block_table, max_blocks, free_ring,
                            n_pages, state, state_out, cu_new, slot_map, max_tokens,
                            static_cast<cudaStream_t>(stream)) != cudaSuccess)
        return op_fail("block table launch failed");
    return ZO_OK;
}

int zo_op_kv_write(const void* qkv, int64_t ld_qkv, const int32_t* slot_map, int32_t n_tokens,
                   void* cache, int64_t n_slots, int32_t n_heads, int32_t n_kv_heads,
                   int32_t head_dim, int32_t dtype, void* stream) {
    if (n_tokens < 0 || n_slots < 1 || n_heads < 0 || n_kv_heads < 1 || head_dim < 1) return ZO_ERR_ARG;
    if (dtype != ZO_DTYPE_FP32 && dtype != ZO_DTYPE_BF16) return ZO_ERR_ARG;
    const int64_t es = dtype == ZO_DTYPE_BF16 ? 2 : 4;
    const int64_t q = (int64_t)n_heads * head_dim, kv = (int64_t)2 * n_kv_heads * head_dim;
    if (ld_qkv < q + kv || kv * es > 0x7fffffffLL) return ZO_ERR_ARG;
    if (n_tokens == 0) return ZO_OK;
    if (!qkv || !slot_map || !cache) return ZO_ERR_ARG;
    if (launch_kv_write(static_cast<const char*>(qkv) + q * es, ld_qkv * es, slot_map, n_tokens, cache,
                        n_slots, (int)(kv * es), static_cast<cudaStream_t>(stream)) != cudaSuccess)
        return op_fail("cache write launch failed");
    return ZO_OK;
}

size_t zo_op_attention_paged_workspace(int32_t n_tokens, int32_t n_rows, int32_t n_heads,
                                       int32_t n_kv_heads, int32_t head_dim, int32_t dtype) {
    if (n_tokens < 0 || n_rows < 0 || n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads || head_dim < 1)
        return 0;
    size_t n = paged_attention_workspace(head_dim);
    if (dtype == ZO_DTYPE_BF16 && (head_dim == 64 || head_dim == 128))
        n = std::max(n, std::max(paged_step_workspace(head_dim), paged_chunk_workspace(head_dim)));
    return n;
}

int zo_op_attention_paged(const void* q, int64_t ld_q, const void* cache, int64_t n_slots,
                          const int32_t* block_table, int32_t max_blocks, int32_t page_size,
                          const int32_t* cu_new, const int32_t* lens, int32_t n_rows,
                          int32_t n_tokens, int32_t max_new, int32_t n_heads,
                          int32_t n_kv_heads, int32_t head_dim, int32_t dtype, void* out,
                          int64_t ld_out, void* ws, size_t ws_bytes, int32_t impl, void* stream) {
    const int shift = page_shift(page_size);
    if (shift < 0 || n_rows < 0 || n_tokens < 0 || max_new < 0 || max_blocks < 1) return ZO_ERR_ARG;
    if (n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads || head_dim < 1) return ZO_ERR_ARG;
    if (dtype != ZO_DTYPE_FP32 && dtype != ZO_DTYPE_BF16) return ZO_ERR_ARG;
    if (impl < ZO_IMPL_AUTO || impl > ZO_IMPL_TENSOR_CORES) return ZO_ERR_ARG;
    if (ld_q < (int64_t)n_heads * head_dim || ld_out < (int64_t)n_heads * head_dim) return ZO_ERR_ARG;
    if (n_slots < page_size || n_slots % page_size || n_slots > 0x7fffffffLL) return ZO_ERR_ARG;
    if (head_dim != 32 && head_dim != 64 && head_dim != 128 && head_dim != 256)
        return ZO_ERR_UNSUPPORTED;
    if (n_kv_heads > 65535 || (int64_t)n_tokens * (n_heads / n_kv_heads) > (1 << 30))
        return ZO_ERR_UNSUPPORTED;
    if (n_rows == 0 || n_tokens == 0) return ZO_OK;
    if (!q || !cache || !block_table || !cu_new || !lens || !out) return ZO_ERR_ARG;
    if (!ws || reinterpret_cast<uintptr_t>(ws) % 16 ||
        ws_bytes < zo_op_attention_paged_workspace(n_tokens, n_rows, n_heads, n_kv_heads, head_dim, dtype))
        return ZO_ERR_ARG;
    PagedArgs a;
    memset(&a, 0, sizeof(a));
    a.q = q; a.ld_q = ld_q;
    a.cache = cache; a.n_slots = n_slots;
    a.block_table = block_table; a.max_blocks = max_blocks; a.page_shift = shift;
    a.cu_new = cu_new; a.lens = lens;
    a.n_rows = n_rows; a.n_tokens = n_tokens; a.max_new = max_new;
    a.H = n_heads; a.Hkv = n_kv_heads; a.g = n_heads / n_kv_heads; a.hd = head_dim;
    for (a.g_shift = 31; (1ll << (a.g_shift - 31)) < a.g;) ++a.g_shift;
    a.g_mul = ((1ull << a.g_shift) + a.g - 1) / a.g;
    a.scale = (float)(1.0 / std::sqrt((double)head_dim));
    a.dtype = dtype == ZO_DTYPE_BF16 ? E_BF16 : E_F32;
    a.out = out; a.ld_out = ld_out;
    a.ws = ws;
    a.wait_cycles = gemm_tc_wait_cycles();
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (impl != ZO_IMPL_CUDA_CORES && paged_tc_supported(a)) {
        // Requests of up to 16 query rows per kv head: the decode-step kernel; others: the chunk
        // kernel.  A request alone is the one that max_new speaks of (and the chunk kernel takes any).
        const bool chunks = (int64_t)max_new * a.g > 16;
        a.step_tokens = !chunks ? 0x7fffffff : n_rows == 1 ? 0 : 16 / a.g;
        if (a.step_tokens > 0 && launch_paged_step(a, st) != cudaSuccess)
            return op_fail("paged attention launch failed");
        if (chunks && launch_paged_chunk(a, st) != cudaSuccess)
            return op_fail("paged attention launch failed");
        return ZO_OK;
    }
    if (impl == ZO_IMPL_TENSOR_CORES) return ZO_ERR_UNSUPPORTED;
    if (launch_paged_attention(a, st) != cudaSuccess) return op_fail("paged attention launch failed");
    return ZO_OK;
}

size_t zo_op_linear_adapters_workspace(int32_t M, int32_t N, int32_t K, int32_t n_adapters,
                                       int32_t rank, int32_t dtype) {
    if (M < 0 || N < 1 || K < 1 || n_adapters < 1 || rank < 1) return 0;
    return adapter_workspace(M, N, K, n_adapters, rank, dtype == ZO_DTYPE_BF16 ? E_BF16 : E_F32);
}

int zo_op_linear_adapters(const void* x, const void* W, const float* bias, const void* A,
                          const void* B, const int32_t* row_adapter, const float* scale,
                          int32_t n_adapters, int32_t rank, void* y, int32_t M, int32_t N,
                          int32_t K, int32_t dtype, int32_t act, int32_t accumulate, void* ws,
                          size_t ws_bytes, int32_t impl, void* stream) {
    if (M < 0 || N < 1 || K < 1 || n_adapters < 1 || rank < 1 || rank > 256) return ZO_ERR_ARG;
    if ((int64_t)n_adapters * rank > 65536) return ZO_ERR_ARG;
    if (dtype != ZO_DTYPE_FP32 && dtype != ZO_DTYPE_BF16) return ZO_ERR_ARG;
    if (act != ZO_ACT_NONE && act != ZO_ACT_RELU) return ZO_ERR_ARG;
    if (accumulate && act != ZO_ACT_NONE) return ZO_ERR_ARG;
    if (impl < ZO_IMPL_AUTO || impl > ZO_IMPL_TENSOR_CORES) return ZO_ERR_ARG;
    if (M == 0) return ZO_OK;
    if (!x || !W || !A || !B || !row_adapter || !scale || !y) return ZO_ERR_ARG;
    if (!ws || reinterpret_cast<uintptr_t>(ws) % 256 ||
        ws_bytes < zo_op_linear_adapters_workspace(M, N, K, n_adapters, rank, dtype))
        return ZO_ERR_ARG;
    if (M > 65535 * 64) return ZO_ERR_UNSUPPORTED;
    AdapterArgs a;
    memset(&a, 0, sizeof(a));
    a.x = x; a.W = W; a.bias = bias; a.A = A; a.B = B;
    a.ids = row_adapter; a.scale = scale;
    a.n_adapters = n_adapters; a.rank = rank;
    a.y = y; a.M = M; a.N = N; a.K = K;
    a.dtype = dtype == ZO_DTYPE_BF16 ? E_BF16 : E_F32;
    a.act = act; a.accumulate = accumulate;
    a.ws = ws; a.ws_bytes = ws_bytes;
    if (impl != ZO_IMPL_CUDA_CORES && linear_adapters_tc_supported(a)) {
        if (launch_linear_adapters_tc(a, static_cast<cudaStream_t>(stream), impl == ZO_IMPL_AUTO) != cudaSuccess)
            return op_fail("adapter linear launch failed");
        return ZO_OK;
    }
    if (impl == ZO_IMPL_TENSOR_CORES) return ZO_ERR_UNSUPPORTED;
    if (launch_linear_adapters_simt(a, static_cast<cudaStream_t>(stream)) != cudaSuccess)
        return op_fail("adapter linear launch failed");
    return ZO_OK;
}

int64_t zo_op_set_wait_limit(int64_t cycles) {
    return (int64_t)gemm_tc_set_wait_cycles((long long)cycles);
}

/* Error word of the tensor-core kernels (bit 0: a bounded wait expired);
 * synchronises the device and clears the word. */
int zo_op_error_word(void) {
    if (cudaDeviceSynchronize() != cudaSuccess) return -1;
    const int v = gemm_tc_error_word();
    const int w = attention_tc_error_word();
    const int s = paged_step_error_word();
    const int c = paged_chunk_error_word();
    if (v < 0 || w < 0 || s < 0 || c < 0) return -1;
    return v | w | s | c;
}

int zo_debug_build(void) {
#ifdef ZO_DEBUG
    return 1;
#else
    return 0;
#endif
}

uint32_t zo_debug_word(int32_t clear) {
    return debug_word_attention_tc(clear != 0) | debug_word_attention(clear != 0) |
           debug_word_decode(clear != 0) | debug_word_reduce(clear != 0) |
           debug_word_gemm(clear != 0);
}

const char* zo_op_last_error(void) { return t_op_err.c_str(); }

}  // extern "C"
