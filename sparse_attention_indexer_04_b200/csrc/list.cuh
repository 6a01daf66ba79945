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

}  // namespace dsa
