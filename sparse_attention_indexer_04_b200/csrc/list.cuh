// Indexer scores at listed keys and their backward pass: arguments and set-up.
//
// Query t lists keys l(t, j); s[t, j] = sum_h w[t,h] max(0, q[t,h] . k[l(t,j)]).  Backward, with
// e = ds and G[t,j,h] = e[t,j] w[t,h] where q[t,h] . k > 0 (else 0):
//   dW[t,h] = sum_j e max(0, q . k),  dQ[t,h] = sum_j G k[l(t,j)],  dK[s] = sum over listing (t, h) of G q[t,h].
#pragma once

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

constexpr int kPosBlock = 256;  // keys that share a base of row positions
constexpr int kDkKeys = 256;   // keys of a block of the dense dK pass

// Key blocks over all sequences: sequence b's first is unit_base(b), which leaves it at least as many
// as it has, without a table.  find_unit: the sequence of a block.
__device__ __forceinline__ int unit_base(const int32_t* k_off, int b) { return k_off[b] / kDkKeys + b; }

__device__ __forceinline__ int find_unit(const int32_t* k_off, int n_seqs, int unit)
{
    int lo = 0, hi = n_seqs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (unit_base(k_off, mid) <= unit) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// One warp per query.  rows[t]: the usable list places, which are strictly ascending keys of the
// sequence up to the first -1, of which those within the query's prefix count; a key outside the
// sequence, not above its predecessor or behind the padding ends the list and records kErrBadRow
// (detail t).  edge (may be NULL): per block of kDkKeys keys the first usable place at or behind the
// block's start, edge[b][n_q] for blocks 0 .. n_blocks.  `quads`: rows are read four places at a time.
__global__ void __launch_bounds__(256) list_rows_kernel(const int32_t* lists, int32_t k, int32_t quads,
                                                        const int32_t* q_off, const int32_t* k_off,
                                                        const int32_t* q_pos, int32_t n_seqs, int32_t n_q,
                                                        RowDesc* rows, uint16_t* edge, int32_t n_blocks,
                                                        uint32_t* status)
{
    const int t = blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (t >= n_q) return;
    const int seq = find_seq(q_off, n_seqs, t);
    const int L = k_off[seq + 1] - k_off[seq];
    const int lim = eligible_count(q_pos[t], L);
    const int32_t* l = lists + (int64_t)t * k;
    int first_end = k, first_bad = k, first_far = k, carry = -1;
    // place i holds v behind prev (the sequence's start: -1 < 0 passes for place 0)
    auto look = [&](int i, int v, int prev) {
        if (v < 0) { first_end = min(first_end, i); return; }
        if (v >= L || (i > 0 && (prev < 0 || prev >= v))) first_bad = min(first_bad, i);
        if (v >= lim) first_far = min(first_far, i);
    };
    // the block borders between place i - 1 and place i
    auto borders = [&](int i, int v, int prev) {
        const int lo = i > 0 ? prev / kDkKeys + 1 : 0, hi = v / kDkKeys;
        for (int b = lo; b <= hi; ++b) edge[(int64_t)b * n_q + t] = (uint16_t)i;
    };
    auto sweep = [&](auto&& f, int n) {
        carry = -1;
        if (quads) {
#pragma unroll 4
            for (int i0 = 0; i0 < n; i0 += 128) {
                const int i = i0 + 4 * lane;
                const int4 v = i < k ? __ldg(reinterpret_cast<const int4*>(l + i)) : make_int4(-1, -1, -1, -1);
                const int up = __shfl_up_sync(0xffffffffu, v.w, 1);
                const int prev = lane == 0 ? carry : up;
                carry = __shfl_sync(0xffffffffu, v.w, 31);
                if (i < n) f(i, v.x, prev);
                if (i + 1 < n) f(i + 1, v.y, v.x);
                if (i + 2 < n) f(i + 2, v.z, v.y);
                if (i + 3 < n) f(i + 3, v.w, v.z);
            }
        } else {
#pragma unroll 4
            for (int i0 = 0; i0 < n; i0 += 32) {
                const int i = i0 + lane;
                const int v = i < k ? __ldg(l + i) : -1;
                const int up = __shfl_up_sync(0xffffffffu, v, 1);
                const int prev = lane == 0 ? carry : up;
                carry = __shfl_sync(0xffffffffu, v, 31);
                if (i < n) f(i, v, prev);
            }
        }
    };
    sweep(look, k);
    first_end = __reduce_min_sync(0xffffffffu, first_end);
    first_bad = __reduce_min_sync(0xffffffffu, first_bad);
    first_far = __reduce_min_sync(0xffffffffu, first_far);
    const int n = min(min(first_end, first_bad), first_far);
    if (lane == 0) {
        if (first_bad < k) record_error(status, kErrBadRow, (uint32_t)t);
        rows[t] = RowDesc{t, seq, n, t};
    }
    if (!edge) return;
    sweep(borders, n);   // from L1 or L2
    const int last = n > 0 ? l[n - 1] / kDkKeys + 1 : 0;
    for (int b = last + lane; b <= n_blocks; b += 32) edge[(int64_t)b * n_q + t] = (uint16_t)n;
}

// scores[t][j] = S[t][lists[t][j]] for the usable places (as list_rows_kernel finds them), -inf in the others;
// S [n_q][ld] holds every eligible score.  One warp per query, `quads`: four places a lane.
template <int PER>
__global__ void __launch_bounds__(256) list_pick_kernel(const int32_t* lists, int32_t k, const int32_t* q_off,
                                                        const int32_t* k_off, const int32_t* q_pos, int32_t n_seqs,
                                                        int32_t n_q, const float* S, int64_t ld, float* scores,
                                                        uint32_t* status)
{
    const int t = blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (t >= n_q) return;
    const int seq = find_seq(q_off, n_seqs, t);
    const int L = k_off[seq + 1] - k_off[seq];
    const int lim = eligible_count(q_pos[t], L);
    const int32_t* l = lists + (int64_t)t * k;
    const float* row = S + (int64_t)t * ld;
    float* out = scores + (int64_t)t * k;
    int stop = k, carry = -1;
    bool bad = false;
    int v[PER], next[PER];
    auto read = [&](int i) {
        if constexpr (PER == 4) {
            const int4 x = i < k ? __ldg(reinterpret_cast<const int4*>(l + i)) : make_int4(-1, -1, -1, -1);
            next[0] = x.x; next[1] = x.y; next[2] = x.z; next[3] = x.w;
        } else {
            next[0] = i < k ? __ldg(l + i) : -1;
        }
    };
    read(PER * lane);
    for (int i0 = 0; i0 < k; i0 += 32 * PER) {
        const int i = i0 + PER * lane;
#pragma unroll
        for (int e = 0; e < PER; ++e) v[e] = next[e];
        read(i + 32 * PER);
        const int up = __shfl_up_sync(0xffffffffu, v[PER - 1], 1);
        int prev = lane == 0 ? carry : up, mine = k;
        carry = __shfl_sync(0xffffffffu, v[PER - 1], 31);
#pragma unroll
        for (int e = PER - 1; e >= 0; --e) {
            const int before = e > 0 ? v[e - 1] : prev;
            const bool wrong = v[e] >= 0 && (v[e] >= L || (i + e > 0 && (before < 0 || before >= v[e])));
            bad |= wrong && i + e < k;
            if (v[e] < 0 || wrong || v[e] >= lim) mine = min(mine, i + e);
        }
        stop = min(stop, (int)__reduce_min_sync(0xffffffffu, (unsigned)mine));
        float s[PER];
#pragma unroll
        for (int e = 0; e < PER; ++e)
            s[e] = i + e < stop && DSA_CHECK(v[e] >= 0 && v[e] < lim, status, 119) ? __ldg(row + v[e]) : __int_as_float(0xff800000);
        if (i < k) {
            if constexpr (PER == 4) *reinterpret_cast<float4*>(out + i) = make_float4(s[0], s[1], s[2], s[3]);
            else out[i] = s[0];
        }
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) record_error(status, kErrBadRow, (uint32_t)t);
}

}  // namespace dsa
