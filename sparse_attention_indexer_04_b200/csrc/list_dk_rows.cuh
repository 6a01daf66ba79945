// dK from the rows that the dQ pass leaves, for lists that cover little of the prefix.
//
// The dQ pass (kListGradRows) writes, for every usable place j of query t, the row
// R[t,j] = sum_h G[t,j,h] q[t,h] (fp32); dK[s] is the sum of the rows whose place lists s.  The rows
// are stored by key: those of key s lie together, in the order of their queries, so that one warp
// sums a key's rows as one stream, in registers and in a fixed order.  Where they lie is worked out
// beforehand from one bit per (key, query): set bits below a query's are the rows before its own.
// Two times 512 bytes a listed pair at d = 128 (written, then read) are what this costs: the sum reads
// them at 6.0 TB/s (721 us for 4096 queries of 2048 places, in five launches).
// (Rows stored by query and picked out by the warp that owns a block of keys: 2.6 ms instead of the
// stream for 4096 queries of 2048 places, bound by the look-ups.)
#pragma once

#include "list.cuh"

namespace dsa {

constexpr int kBitsPlaces = 512;   // list places of a warp of the marking kernel

// bits[w][n_k]: bit b of word w of key row s: query t0 + 32 w + b lists it.  A warp per kBitsPlaces places
// of a query (blockIdx.y: which).
__global__ void __launch_bounds__(256) list_bits_kernel(const int32_t* lists, int32_t k, const RowDesc* rows,
                                                        const int32_t* k_off, int32_t t0, int32_t t1, int32_t n_k,
                                                        uint32_t* bits, uint32_t* status)
{
    const int t = t0 + blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (t >= t1) return;
    const RowDesc r = rows[t];
    const int i0 = blockIdx.y * kBitsPlaces, i1 = min(r.ncols, i0 + kBitsPlaces);
    const int32_t* l = lists + (int64_t)t * k;
    uint32_t* word = bits + (int64_t)((t - t0) >> 5) * n_k;
    const uint32_t bit = 1u << ((t - t0) & 31);
    const int kb = k_off[r.seq];
#pragma unroll 8
    for (int i = i0 + lane; i < i1; i += 32) {
        const int s = kb + __ldg(l + i);
        if (DSA_CHECK(s >= 0 && s < n_k, status, 117)) atomicOr(word + s, bit);
    }
}

// Exclusive sum of v over the CTA's threads (a power of two of warps), and the total.
template <int NT>
__device__ __forceinline__ uint32_t cta_exclusive_sum(uint32_t v, uint32_t* red, uint32_t* total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
    }
    __syncthreads();   // red is free
    if (lane == 31) red[warp] = s;
    __syncthreads();
    uint32_t before = 0, all = 0;
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += red[w];
        all += red[w];
    }
    *total = all;
    return before + s - v;
}

// Per key: pre[w][n_k], its rows before word w; count[n_k]; off[n_k], its first row within the CTA's keys,
// whose number goes to base[blockIdx.x].
__global__ void __launch_bounds__(kPosBlock) list_count_kernel(const uint32_t* bits, int32_t words, int32_t n_k,
                                                              uint16_t* pre, uint32_t* count, uint32_t* off,
                                                              uint32_t* base)
{
    __shared__ uint32_t red[32];
    const int s = blockIdx.x * kPosBlock + threadIdx.x;
    uint32_t n = 0;
    if (s < n_k) {
        constexpr int U = 16;   // words read together
        for (int w0 = 0; w0 < words; w0 += U) {
            uint32_t b[U];
#pragma unroll
            for (int u = 0; u < U; ++u) b[u] = w0 + u < words ? bits[(int64_t)(w0 + u) * n_k + s] : 0u;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (w0 + u < words) pre[(int64_t)(w0 + u) * n_k + s] = (uint16_t)n;
                n += __popc(b[u]);
            }
        }
        count[s] = n;
    }
    uint32_t total;
    const uint32_t at = cta_exclusive_sum<kPosBlock>(n, red, &total);
    if (s < n_k) off[s] = at;
    if (threadIdx.x == 0) base[blockIdx.x] = total;
}

// base[i] becomes the number of rows before key block i (one CTA).
__global__ void __launch_bounds__(1024) list_base_kernel(uint32_t* base, int32_t n)
{
    __shared__ uint32_t red[32];
    uint32_t sum = 0;
    for (int i0 = 0; i0 < n; i0 += 1024) {
        const int i = i0 + threadIdx.x;
        const uint32_t v = i < n ? base[i] : 0u;
        uint32_t total;
        const uint32_t at = cta_exclusive_sum<1024>(v, red, &total);
        if (i < n) base[i] = sum + at;
        sum += total;
    }
}

struct DkRowsArgs {
    const float* part;      // rows by key
    const uint32_t* count;  // [n_k]
    const uint32_t* off;    // [n_k]
    const uint32_t* base;   // [blocks of kPosBlock keys]
    float* acc;             // [n_k][D] sums of earlier and later launches (not used by a single one)
    __nv_bfloat16* dK;
    int32_t n_k;
    int32_t first, last;    // of the launches
};

constexpr int kRowsWarps = 8;   // keys of a CTA: one a warp

template <int D>
__global__ void __launch_bounds__(kRowsWarps * 32) list_dk_rows_kernel(const __grid_constant__ DkRowsArgs a)
{
    constexpr int V = D / 32;   // columns of a lane
    const int lane = threadIdx.x & 31, s = blockIdx.x * kRowsWarps + (threadIdx.x >> 5);
    grid_dep_wait();
    if (s >= a.n_k) return;
    const int n = a.count[s];
    if (n == 0 && !a.first && !a.last) return;
    const float* r = a.part + ((int64_t)a.base[s / kPosBlock] + a.off[s]) * D + lane * V;
    const int64_t at = (int64_t)s * D + lane * V;
    float sum[V];
#pragma unroll
    for (int c = 0; c < V; ++c) sum[c] = a.first ? 0.f : a.acc[at + c];
#pragma unroll 8
    for (int i = 0; i < n; ++i, r += D) {
        if constexpr (V == 4) {
            const float4 x = __ldcs(reinterpret_cast<const float4*>(r));
            sum[0] += x.x; sum[1] += x.y; sum[2] += x.z; sum[3] += x.w;
        } else if constexpr (V == 2) {
            const float2 x = __ldcs(reinterpret_cast<const float2*>(r));
            sum[0] += x.x; sum[1] += x.y;
        } else {
            sum[0] += __ldcs(r);
        }
    }
#pragma unroll
    for (int c = 0; c < V; ++c) {
        if (a.last) a.dK[at + c] = __float2bfloat16_rn(sum[c]);
        else a.acc[at + c] = sum[c];
    }
}

}  // namespace dsa
