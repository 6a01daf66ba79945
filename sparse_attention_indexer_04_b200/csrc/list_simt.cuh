// Indexer scores at listed keys and their backward pass, on the fp32 pipes.
//
// Query t lists keys l(t, j); s[t, j] = sum_h w[t,h] max(0, q[t,h] . k[l(t,j)]).  Backward, with
// e = ds and G[t,j,h] = e[t,j] w[t,h] where q[t,h] . k > 0 (else 0):
//   dW[t,h] = sum_j e max(0, q . k),  dQ[t,h] = sum_j G k[l(t,j)],  dK[s] = sum over listing (t, h) of G q[t,h].
#pragma once

#include <math_constants.h>

#include "common.cuh"

namespace dsa {

struct ListArgs {
    const RowDesc* rows;          // row t: sequence and number of usable list places
    const __nv_bfloat16* Q;
    const __nv_bfloat16* K;
    const float* W;
    const int32_t* lists;         // [n_q, k]
    const float* ds;              // [n_q, k]
    float* scores;                // [n_q, k]
    __nv_bfloat16* dQ;
    __nv_bfloat16* dK;
    float* dW;
    const int32_t* q_off;
    const int32_t* k_off;
    uint32_t* status;
    int32_t n_seqs, n_q, n_k, H, k;
};

// Usable list places of every query (one warp each): strictly ascending keys of the sequence up to
// the first -1, of which those within the query's prefix count.  A key outside the sequence, not
// above its predecessor or behind the padding ends the list and records kErrBadRow (detail t).
__global__ void list_rows_kernel(const int32_t* lists, int32_t k, const int32_t* q_off, const int32_t* k_off,
                                 const int32_t* q_pos, int32_t n_seqs, int32_t n_q, RowDesc* rows, uint32_t* status)
{
    const int t = blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (t >= n_q) return;
    const int seq = find_seq(q_off, n_seqs, t);
    const int L = k_off[seq + 1] - k_off[seq];
    const int lim = eligible_count(q_pos[t], L);
    const int32_t* l = lists + (int64_t)t * k;
    int first_end = k, first_bad = k, first_far = k;
    for (int i = lane; i < k; i += 32) {
        const int32_t v = l[i];
        const int32_t prev = i > 0 ? l[i - 1] : -1;
        if (v < 0) { first_end = min(first_end, i); continue; }
        if (v >= L || (i > 0 && (prev < 0 || prev >= v))) first_bad = min(first_bad, i);
        if (v >= lim) first_far = min(first_far, i);
    }
    first_end = __reduce_min_sync(0xffffffffu, first_end);
    first_bad = __reduce_min_sync(0xffffffffu, first_bad);
    first_far = __reduce_min_sync(0xffffffffu, first_far);
    if (lane == 0) {
        if (first_bad < k) record_error(status, kErrBadRow, (uint32_t)t);
        rows[t] = RowDesc{t, seq, min(min(first_end, first_bad), first_far), t};
    }
}

constexpr int kListThreads = 128;

template <int D>
__device__ __forceinline__ float list_dot(const float* q, const float* key)
{
    float s = 0.f;
#pragma unroll 8
    for (int i = 0; i < D; ++i) s = fmaf(q[i], key[i], s);
    return s;
}

// One thread per list place; the query's heads in shared memory.
template <int D>
__global__ void __launch_bounds__(kListThreads) list_scores_simt_kernel(const __grid_constant__ ListArgs a)
{
    extern __shared__ float sm[];
    const int t = blockIdx.x, j = blockIdx.y * kListThreads + threadIdx.x;
    const RowDesc r = a.rows[t];
    for (int i = threadIdx.x; i < a.H * D; i += kListThreads) sm[i] = __bfloat162float(a.Q[(int64_t)t * a.H * D + i]);
    __syncthreads();
    if (j >= a.k) return;
    float s = -CUDART_INF_F;
    if (j < r.ncols) {
        const int64_t row = (int64_t)a.k_off[r.seq] + a.lists[(int64_t)t * a.k + j];
        if (DSA_CHECK(row >= 0 && row < a.n_k, a.status, 110)) {
            float key[D];
#pragma unroll
            for (int i = 0; i < D; ++i) key[i] = __bfloat162float(a.K[row * D + i]);
            s = 0.f;
            for (int h = 0; h < a.H; ++h)
                s = fmaf(a.W[(int64_t)t * a.H + h], fmaxf(list_dot<D>(sm + h * D, key), 0.f), s);
        }
    }
    a.scores[(int64_t)t * a.k + j] = s;
}

constexpr int kListTile = 32;   // keys staged at once

// dQ and dW of one query per CTA, its listed keys staged 32 at a time.
template <int D>
__global__ void __launch_bounds__(kListThreads) list_dq_simt_kernel(const __grid_constant__ ListArgs a)
{
    extern __shared__ float sm[];
    const int H = a.H;
    float* sQ = sm;                        // [H][D]
    float* sK = sQ + H * D;                // [tile][D + 1]
    float* sS = sK + kListTile * (D + 1);  // [tile][H] products, then G
    const int t = blockIdx.x;
    const RowDesc r = a.rows[t];
    for (int i = threadIdx.x; i < H * D; i += kListThreads) sQ[i] = __bfloat162float(a.Q[(int64_t)t * H * D + i]);
    constexpr int kMax = 64 * D / kListThreads;
    float acc[kMax];
#pragma unroll
    for (int i = 0; i < kMax; ++i) acc[i] = 0.f;
    float dw = 0.f;
    for (int j0 = 0; j0 < r.ncols; j0 += kListTile) {
        __syncthreads();
        for (int i = threadIdx.x; i < kListTile * D; i += kListThreads) {
            const int j = j0 + i / D;
            float v = 0.f;
            if (j < r.ncols) {
                const int64_t row = (int64_t)a.k_off[r.seq] + a.lists[(int64_t)t * a.k + j];
                if (DSA_CHECK(row >= 0 && row < a.n_k, a.status, 111)) v = __bfloat162float(a.K[row * D + i % D]);
            }
            sK[(i / D) * (D + 1) + i % D] = v;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < kListTile * H; i += kListThreads)
            sS[i] = list_dot<D>(sQ + (i % H) * D, sK + (i / H) * (D + 1));
        __syncthreads();
        if ((int)threadIdx.x < H)
            for (int j = 0; j < kListTile && j0 + j < r.ncols; ++j) {
                const float e = a.ds[(int64_t)t * a.k + j0 + j], s = sS[j * H + threadIdx.x];
                dw = fmaf(e, fmaxf(s, 0.f), dw);
                sS[j * H + threadIdx.x] = s > 0.f ? e * a.W[(int64_t)t * H + threadIdx.x] : 0.f;
            }
        __syncthreads();
        const int m = min(kListTile, r.ncols - j0);
#pragma unroll
        for (int i = 0; i < kMax; ++i) {
            const int o = i * kListThreads + threadIdx.x;
            if (o >= H * D) break;
            for (int j = 0; j < m; ++j) acc[i] = fmaf(sS[j * H + o / D], sK[j * (D + 1) + o % D], acc[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < kMax; ++i) {
        const int o = i * kListThreads + threadIdx.x;
        if (o < H * D && a.dQ) a.dQ[(int64_t)t * H * D + o] = __float2bfloat16_rn(acc[i]);
    }
    if ((int)threadIdx.x < H && a.dW) a.dW[(int64_t)t * H + threadIdx.x] = dw;
}

// First place of an ascending list of n whose key is at least s.
__device__ __forceinline__ int list_lower_bound(const int32_t* l, int n, int s)
{
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (l[mid] < s) lo = mid + 1; else hi = mid;
    }
    return lo;
}

// dK of kListTile keys of one sequence per CTA, over the sequence's queries in order (no atomics:
// the sum's order does not depend on the launch).  blockIdx.x: key tile over all key rows.
template <int D>
__global__ void __launch_bounds__(kListThreads) list_dk_simt_kernel(const __grid_constant__ ListArgs a)
{
    extern __shared__ float sm[];
    const int H = a.H;
    float* sQ = sm;                        // [H][D]
    float* sK = sQ + H * D;                // [tile][D + 1]
    float* sS = sK + kListTile * (D + 1);  // [tile][H]: G
    const int row0 = blockIdx.x * kListTile, row1 = min(row0 + kListTile, a.n_k);
    for (int i = threadIdx.x; i < (row1 - row0) * D; i += kListThreads)
        sK[(i / D) * (D + 1) + i % D] = __bfloat162float(a.K[(int64_t)(row0) * D + i]);
    constexpr int kMax = kListTile * D / kListThreads;
    float acc[kMax];
#pragma unroll
    for (int i = 0; i < kMax; ++i) acc[i] = 0.f;
    // the sequences that own rows of this tile (a tile may cross their borders)
    for (int b = find_seq(a.k_off, a.n_seqs, row0); b < a.n_seqs && a.k_off[b] < row1; ++b) {
        const int kb = a.k_off[b];
        const int s0 = max(row0 - kb, 0), s1 = min(row1, a.k_off[b + 1]) - kb;   // keys of the sequence
        if (s1 <= s0) continue;
        for (int t = a.q_off[b]; t < a.q_off[b + 1]; ++t) {
            const int32_t* l = a.lists + (int64_t)t * a.k;
            const int n = a.rows[t].ncols;
            const int lo = list_lower_bound(l, n, s0), hi = lo + list_lower_bound(l + lo, n - lo, s1);
            if (lo == hi) continue;
            __syncthreads();
            for (int i = threadIdx.x; i < H * D; i += kListThreads)
                sQ[i] = __bfloat162float(a.Q[(int64_t)t * H * D + i]);
            __syncthreads();
            for (int i = threadIdx.x; i < (hi - lo) * H; i += kListThreads) {
                const int h = i % H, key = kb + l[lo + i / H] - row0;
                if (!DSA_CHECK(key >= 0 && key < kListTile, a.status, 112)) continue;
                const float s = list_dot<D>(sQ + h * D, sK + key * (D + 1));
                sS[key * H + h] = s > 0.f ? a.ds[(int64_t)t * a.k + lo + i / H] * a.W[(int64_t)t * H + h] : 0.f;
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kMax; ++i) {
                const int o = i * kListThreads + threadIdx.x;
                const int key = row0 + o / D - kb;
                const int j = lo + list_lower_bound(l + lo, hi - lo, key);
                if (j == hi || l[j] != key) continue;
                for (int h = 0; h < H; ++h) acc[i] = fmaf(sS[(o / D) * H + h], sQ[h * D + o % D], acc[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kMax; ++i) {
        const int o = i * kListThreads + threadIdx.x;
        if (row0 + o / D < row1) a.dK[(int64_t)row0 * D + o] = __float2bfloat16_rn(acc[i]);
    }
}

}  // namespace dsa
