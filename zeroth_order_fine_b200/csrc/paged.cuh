// Shared by the tensor-core kernels of the paged attention: requests, the line of work units, and
// the TMA map over the cache.
#pragma once

#include <cuda.h>

#include "common.cuh"
#include "kernels.h"

namespace zo {

// a / b for a >= 0, b > 0: a 32-bit division wherever that does (a 64-bit one is ~5 times slower)
__device__ __forceinline__ long long div_ll(long long a, long long b) {
    return ((a | b) >> 32) ? a / b : (long long)((unsigned)a / (unsigned)b);
}

// a row's token (x / g) and its head of the group
__device__ __forceinline__ int by_g(const PagedArgs& a, int x) {
    return (int)((unsigned long long)(unsigned)x * a.g_mul >> a.g_shift);
}
__device__ __forceinline__ int mod_g(const PagedArgs& a, int x) { return x - by_g(a, x) * a.g; }

// A kernel takes the requests of at most step_tokens new tokens (BIG false) or the others (BIG
// true); the rest have no rows for it.  RB query rows (new tokens x g of one kv head) make a tile,
// UK keys a unit; a place on the line stands for line_heads-th parts of the kv heads.
// W0 > 0: a unit of a tile of n rows is W0 + ceil(n / 8) steps of the line and not one, where a unit
// of few rows takes less time; a stretch has the units that begin in it and is at least WMAX long,
// so that every stretch inside an item has some of its units.
template <bool BIG, int RB, int UK, int W0 = 0>
struct PagedLine {
    static constexpr int WMAX = W0 ? W0 + RB / 8 : 1;
    struct Req {
        int start, rows, ctx;             // first packed row, rows per kv head, tokens before
        bool bad;                         // the length cannot be used: NaN rows
    };
    // a place on the line: units of a (request, tile, group of kv heads) in key order, then groups
    // (line_heads of them), tiles, requests
    struct Cursor {
        Req q;
        int r, tile, head, unit, units;
    };
    static __device__ __forceinline__ Req get(const PagedArgs& a, int r) {
        Req q;
        const int s = a.cu_new[r], e = a.cu_new[r + 1], len = a.lens[r];
        const int n = e - s;
        const bool in = s >= 0 && e >= s && e <= a.n_tokens;
        q.start = s;
        q.rows = in && (n > a.step_tokens) == BIG ? n * a.g : 0;
        // (the last 256 lengths of an int: a unit's end would not fit)
        q.bad = len < n || len > 0x7fffff00 || (long long)len > ((long long)a.max_blocks << a.page_shift);
        q.ctx = len - n;
        return q;
    }
    // keys that the rows before `end` of a request see, and units of its tile t
    static __device__ __forceinline__ int keys(const PagedArgs& a, const Req& q, int end) {
        return q.bad ? 0 : q.ctx + by_g(a, min(end, q.rows) - 1) + 1;
    }
    static __device__ __forceinline__ int units(const PagedArgs& a, const Req& q, int t) {
        return q.bad ? 1 : (keys(a, q, (t + 1) * RB) + UK - 1) / UK;
    }
    static __device__ __forceinline__ int weight(const Req& q, int t) {       // steps of a unit of tile t
        return W0 ? W0 + (min(RB, q.rows - t * RB) + 7) / 8 : 1;
    }
    static __device__ __forceinline__ long long req_units(const PagedArgs& a, int r) {
        const Req q = get(a, r);
        long long u = 0;
        for (int t = 0; t * RB < q.rows; ++t) u += (long long)units(a, q, t) * weight(q, t);
        return u * a.line_heads;
    }
    // Prefix sums of the requests' units in groups of ceil(n_rows / max_groups) requests: cum[0 ..
    // groups]; every thread of the block takes part and gets the total.  wsum: one per warp.
    static __device__ __forceinline__ long long prefix(const PagedArgs& a, int max_groups, long long* cum,
                                                       long long* wsum) {
        const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nw = blockDim.x >> 5;
        const int c = (a.n_rows + max_groups - 1) / max_groups;
        const int groups = c == 1 ? a.n_rows : (a.n_rows + c - 1) / c;
        long long base = 0;
        for (int g0 = 0; g0 < groups; g0 += blockDim.x) {
            const int gi = g0 + tid;
            long long u = 0;
            if (gi < groups)
                for (int r = gi * c; r < min(a.n_rows, (gi + 1) * c); ++r) u += req_units(a, r);
            long long incl = u;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            if (lane == 31) wsum[warp] = incl;
            __syncthreads();
            long long before = 0, total = 0;
            for (int w = 0; w < nw; ++w) {
                if (w < warp) before += wsum[w];
                total += wsum[w];
            }
            if (gi < groups) cum[gi + 1] = base + before + incl;
            base += total;
            __syncthreads();
        }
        if (tid == 0) cum[0] = 0;
        __syncthreads();
        return base;
    }
    // The place of the first unit that begins at step u (below the total) or behind it, u then moved
    // there; with W0 it may be unit = units, the end of an item.  A whole warp calls it with the same
    // u, max_groups <= 1024.
    static __device__ __forceinline__ Cursor locate(const PagedArgs& a, int max_groups,
                                                    const long long* cum, long long& u) {
        const int c = (a.n_rows + max_groups - 1) / max_groups;
        const int groups = c == 1 ? a.n_rows : (a.n_rows + c - 1) / c, lane = threadIdx.x & 31;
        int lo = 0;                                    // the last group with cum <= u
        for (int step = groups > 32 ? 32 : 1;; step >>= 5) {
            const int at = lo + lane * step;
            const unsigned le = __ballot_sync(0xffffffffu, at < groups && cum[at] <= u);
            lo += (31 - __clz(le)) * step;             // cum does not fall: the bits set are the low ones
            if (step == 1) break;
        }
        long long rest = u - cum[lo];
        Cursor k;
        k.r = lo * c;
        if (c > 1)
            for (;; ++k.r) {
                const long long n = req_units(a, k.r);
                if (rest < n) break;
                rest -= n;
            }
        k.q = get(a, k.r);
        k.tile = 0;
        int wt;
        for (;;) {
            k.units = units(a, k.q, k.tile);
            wt = weight(k.q, k.tile);
            const long long n = (long long)k.units * wt * a.line_heads;
            if (rest < n) break;
            rest -= n;
            ++k.tile;
        }
        k.head = (int)div_ll(rest, (long long)k.units * wt);
        rest -= (long long)k.head * k.units * wt;
        k.unit = W0 ? (int)div_ll(rest + wt - 1, wt) : (int)rest;
        u += (long long)k.unit * wt - rest;
        return k;
    }
    // On by n units of the same (request, tile, head), n <= units - unit; `more`: the line goes on
    // behind them.
    static __device__ __forceinline__ void advance(const PagedArgs& a, Cursor& k, int n, bool more) {
        k.unit += n;
        if (k.unit < k.units) return;
        k.unit = 0;
        if (++k.head < a.line_heads) return;
        k.head = 0;
        if (more) next_tile(a, k);
    }
    // To the next tile, of the next request that has rows here if need be (there is one).
    static __device__ __forceinline__ void next_tile(const PagedArgs& a, Cursor& k) {
        if (++k.tile * RB >= k.q.rows) {
            k.tile = 0;
            do {
                ++k.r;
                k.q = get(a, k.r);
            } while (k.q.rows == 0 && k.r + 1 < a.n_rows);
        }
        k.units = units(a, k.q, k.tile);
    }
};

// An item (request, tile, kv head) that a worker's stretch of the line ended inside: workers w ..
// w + pieces - 1 hold its pieces (pieces 0: none).
struct PagedDesc {
    int pieces;
    int start, row0, rows;            // first packed row; first and number of the request's rows
    int kvh, pad[3];
};

// The cache [n_slots][2][Hkv][hd] as (64 columns, rows, column halves of all heads, k/v), 128-byte
// swizzled boxes of 64 x rows x halves x kvs.
bool paged_cache_map(CUtensorMap* m, const PagedArgs& a, int rows, int halves, int kvs);

}  // namespace zo
