// dK of the scores at listed keys on the tensor cores: dK[s] = sum over (t, h) of G[t,s,h] q[t,h],
// G = ds w where q . k > 0 and t lists s, else 0.
//
// The sum runs over queries, so the keys stay: a CTA owns 256 consecutive keys of a sequence (two
// tiles of 128, resident in shared memory, their dK accumulators in TMEM for the CTA's whole life)
// and passes over the queries that list any of them, NQ = up to 128 / H at a time:
//   S[128 keys x ROWS] = K_tile . Q^T      (ROWS = NQ * H query-head rows)
//   G = S > 0 ? ds w : 0                    (bf16, in TMEM over S; ds scattered from the list's places)
//   dK_tile += G . Q                        (A = G from TMEM, B = Q MN-major as it lies)
// (G in shared memory had the products read 8 KB an MMA there, which its bandwidth, not the tensor
// cores, paced: 92 clocks an MMA of 64.)
// No atomics: each (key tile, query) product is dense, keys that the query does not list have G = 0.
// That does 1 / density of the needed work at the tensor cores' rate (2.15 us for 256 keys x 2 queries
// of 64 heads on every SM: 1.16 PFLOP/s, 0.83 of the sustained bf16 rate; 3.6 ms for 4096 queries of
// 32K keys); where lists cover little, list_dk_rows.cuh costs less (dk_by_rows).  The queries of a
// sequence are dealt to `parts` CTAs per key block when there are few key blocks; their fp32 partial
// sums are added in order by a second kernel.
// Roles: warps 0..2 load (one stage each: query rows, weights and the block's ds), warp 4 issues the
// MMAs, warps 5..20 are four sets of four: a key tile and half of the query-head rows each.  Every
// wait is bounded.
#pragma once

#include "list_tc.cuh"

namespace dsa {

constexpr int kDkThreads = 672;
constexpr int kDkMaxList = 8192;   // queries of one CTA at most

template <int D, int H>
struct DkShape {
    static constexpr int NQ = H >= 8 ? 128 / H : 16;               // queries of a block
    static constexpr int ROWS = NQ * H;                            // 16, 32, 64 or 128
    static constexpr int CW = ROWS >= 64 ? 32 : ROWS / 2;          // columns of S a thread takes at a time
    static constexpr uint32_t ROWB = D * 2 >= 128 ? 128 : 64;
    static constexpr int BOXC = ROWB / 2;
    static constexpr int NBOX = D / BOXC;
    static constexpr uint32_t KBOX = 128u * ROWB;
    static constexpr uint32_t KTILE = KBOX * NBOX;
    static constexpr uint32_t QBOX = (uint32_t)ROWS * ROWB;
    static constexpr uint32_t QTILE = QBOX * NBOX;
    static constexpr int NS = 3;                                   // stages of queries
    // TMEM columns of G inside the tile's S: CW values packed in pairs over S columns that the same
    // threads have read; 16 rows are one MMA's k and need adjacent columns (free ones)
    static constexpr int g_chunk(int c0) { return ROWS == 16 ? 32 + c0 / 2 : c0; }
    static constexpr int g_step(int kk) { return ROWS >= 64 ? (kk / 2) * 32 + (kk % 2) * 8 : ROWS == 32 ? kk * 16 : 32; }
    static constexpr uint32_t E_BYTES = (uint32_t)NQ * kDkKeys * 4;
    static constexpr uint32_t q_off = 2 * KTILE;
    static constexpr uint32_t e_off = q_off + NS * QTILE;
    static constexpr uint32_t w_off = e_off + NS * E_BYTES;
    static constexpr uint32_t list_off = w_off + NS * ROWS * 4;
    static constexpr uint32_t bar_off = list_off + kDkMaxList * 2;
    static constexpr uint32_t bytes = bar_off + 512;
    static_assert(NS <= 4 && list_off % 8 == 0 && ROWS % (32 / (D / 8)) == 0);
    static_assert(q_off % 1024 == 0 && bytes <= 232448, "shared memory of the dK kernel");
};

struct DkArgs {
    ListArgs l;
    const uint16_t* edge;   // [max blocks + 1][n_q]
    float* part;            // [parts][n_k][D] (parts > 1)
    int32_t parts;
};

template <int D, int H>
__global__ void __launch_bounds__(kDkThreads, 1)
    list_dk_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ DkArgs a)
{
    using SH = DkShape<D, H>;
    constexpr int NQ = SH::NQ, ROWS = SH::ROWS, NS = SH::NS;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint32_t* status = a.l.status;
    if (smem_u32(smem) & 1023u) {
        if (threadIdx.x == 0) record_error(status, kErrListAlign, blockIdx.x);
        return;
    }
    const int unit = blockIdx.x / a.parts, part = blockIdx.x % a.parts;
    const int seq = find_unit(a.l.k_off, a.l.n_seqs, unit);
    const int blk = unit - unit_base(a.l.k_off, seq);
    const int kb = a.l.k_off[seq], L = a.l.k_off[seq + 1] - kb;
    const int s0 = blk * kDkKeys;
    if (s0 >= L) return;   // a unit without keys
    const int q0 = a.l.q_off[seq], nq = a.l.q_off[seq + 1] - q0;

    uint8_t* sK = smem;
    uint8_t* sQ = smem + SH::q_off;
    float* sE = reinterpret_cast<float*>(smem + SH::e_off);
    float* sW = reinterpret_cast<float*>(smem + SH::w_off);
    uint16_t* sList = reinterpret_cast<uint16_t*>(smem + SH::list_off);
    uint64_t* kfull = reinterpret_cast<uint64_t*>(smem + SH::bar_off);
    uint64_t* qfull = kfull + 1;          // [NS] query rows have landed
    uint64_t* qfree = qfull + NS;         // [NS] both products have read them
    uint64_t* efull = qfree + NS;         // [NS] ds and weights are written
    uint64_t* efree = efull + NS;         // [NS] and read
    uint64_t* sfull = efree + NS;         // [tile] S is complete
    uint64_t* sfree = sfull + 2;          // [tile] G, which lies over S, has been read
    uint64_t* gfull = sfree + 2;          // [tile] G is written
    uint64_t* dkfull = gfull + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(dkfull + 1);
    volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(tmem_slot + 1);
    int32_t* sCount = reinterpret_cast<int32_t*>(tmem_slot + 2);   // [21] per-warp counts

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(kfull, 1);
        for (int i = 0; i < NS; ++i) {
            mbar_init(&qfull[i], 32);
            mbar_init(&qfree[i], 1);
            mbar_init(&efull[i], 32);
            mbar_init(&efree[i], 512);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sfull[i], 1);
            mbar_init(&sfree[i], 1);
            mbar_init(&gfull[i], 256);
        }
        mbar_init(dkfull, 1);
        *abort_flag = 0;
        fence_barrier_init();
        prefetch_tensormap(&tmK);
    }
    if (warp == 4) tmem_alloc(tmem_slot, 512);
    grid_dep_wait();   // the edges and lists' lengths come from earlier kernels

    // the part's queries that list a key of the block, in order (query part + ordinal * parts)
    const uint16_t* e0 = a.edge + (int64_t)blk * a.l.n_q + q0;
    const uint16_t* e1 = e0 + a.l.n_q;
    const int n_cand = nq > part ? (nq - part + a.parts - 1) / a.parts : 0;
    int m = 0;
    for (int c0 = 0; c0 < n_cand; c0 += kDkThreads) {
        const int c = c0 + threadIdx.x, t = part + c * a.parts;
        const bool on = c < n_cand && e1[t] > e0[t];
        const uint32_t vote = __ballot_sync(0xffffffffu, on);
        if (lane == 0) sCount[warp] = __popc(vote);
        __syncthreads();
        int before = m, total = 0;
        for (int w = 0; w < kDkThreads / 32; ++w) {
            if (w < warp) before += sCount[w];
            total += sCount[w];
        }
        if (on && DSA_CHECK(before + __popc(vote & lanemask_lt()) < kDkMaxList, status, 114))
            sList[before + __popc(vote & lanemask_lt())] = (uint16_t)c;
        m += total;
        __syncthreads();
    }
    const int nb = (m + NQ - 1) / NQ;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tDK = tmem, tS = tmem + 256;   // dK: tile * D; S: tile * 128

    if (warp < 4) {
        // -------------------------------------------------------- loaders
        constexpr int CPR = D / 8, RPI = 32 / CPR, CPB = SH::ROWB / 16;
        const int chunk = lane % CPR, rsub = lane / CPR, cc = chunk % CPB;
        const uint32_t coff = (uint32_t)(chunk / CPB) * SH::QBOX;
        // GL lanes per query of the block; a lane's list places are read PF at a time, the first ahead
        constexpr int GL = 32 / NQ, PF = 8;
        const int q = lane / GL, sub = lane % GL;
        bool alive = true;
        struct Next {
            int t, lo, hi;   // the lane's query and its places in the block (none past the unit's queries)
        };
        auto look = [&](int j) {
            const int ord = j * NQ + q;   // past the end: the last query again, counting for nothing
            Next x{part + (int)sList[min(ord, m - 1)] * a.parts, 0, 0};
            if (ord < m) {
                x.lo = e0[x.t];
                x.hi = e1[x.t];
            }
            return x;
        };
        Next nx{0, 0, 0};
        if (warp < NS && warp < nb) nx = look(warp);
        // warp w fills stage w every time: a stage's next filling waits for its last one's release,
        // which a parity tells apart only for one waiter that never runs ahead
        for (int j = warp; j < nb && warp < NS; j += NS) {
            const int s = warp;
            const uint32_t ph = (uint32_t)((j / NS) & 1);
            const Next c = nx;
            // everything this block needs from memory is asked for before the first wait
            const int32_t* lp = a.l.lists + (int64_t)(q0 + c.t) * a.l.k;
            const float* dp = a.l.ds + (int64_t)(q0 + c.t) * a.l.k;
            int key[PF];
            float ds[PF];
            auto read = [&](int i0) {
#pragma unroll
                for (int x = 0; x < PF; ++x) {
                    const int i = i0 + x * GL;
                    key[x] = i < c.hi ? __ldg(lp + i) : -1;
                    ds[x] = i < c.hi ? __ldg(dp + i) : 0.f;
                }
            };
            read(c.lo + sub);
            float wv[(ROWS + 31) / 32];
#pragma unroll
            for (int x = 0; x < (ROWS + 31) / 32; ++x) {
                const int row = x * 32 + lane, wq = min(row / H, NQ - 1);
                const int t = __shfl_sync(0xffffffffu, c.t, wq * GL);
                wv[x] = row < ROWS && j * NQ + wq < m ? a.l.W[(int64_t)(q0 + t) * H + row % H] : 0.f;
            }
            if (j + NS < nb) nx = look(j + NS);
            alive = tc_wait_warp(&qfree[s], ph ^ 1u, status, 41, abort_flag, alive);
            if (!alive) break;
            const uint32_t dst = smem_u32(sQ + s * SH::QTILE) + coff;
#pragma unroll
            for (int x = 0; x < ROWS / RPI; ++x) {
                const int row = x * RPI + rsub;
                const int t = __shfl_sync(0xffffffffu, c.t, row / H * GL);
                const int sw = SH::ROWB == 128 ? cc ^ (row & 7) : cc ^ ((row >> 1) & 3);
                cp_async16(dst + row * SH::ROWB + sw * 16, a.l.Q + ((int64_t)(q0 + t) * H + row % H) * D + chunk * 8);
            }
            cp_async_arrive(&qfull[s]);
            alive = tc_wait_warp(&efree[s], ph ^ 1u, status, 42, abort_flag, alive);
            if (!alive) break;
            float* w = sW + s * ROWS;
#pragma unroll
            for (int x = 0; x < (ROWS + 31) / 32; ++x)
                if (x * 32 + lane < ROWS) w[x * 32 + lane] = wv[x];
            float* e = sE + s * NQ * kDkKeys;
            for (int x = lane; x < NQ * kDkKeys / 4; x += 32)
                reinterpret_cast<float4*>(e)[x] = make_float4(0.f, 0.f, 0.f, 0.f);
            __syncwarp();
            e += q * kDkKeys;
            for (int i = c.lo + sub;;) {
#pragma unroll
                for (int x = 0; x < PF; ++x)
                    if (key[x] >= 0 && DSA_CHECK(key[x] >= s0 && key[x] < s0 + kDkKeys, status, 115)) e[key[x] - s0] = ds[x];
                if ((i += PF * GL) >= c.hi) break;
                read(i);
            }
            __syncwarp();
            mbar_arrive(&efull[s]);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
    } else if (warp == 4) {
        // -------------------------------------------------------- MMA issuer
        if (nb > 0) {   // (nothing listed: the epilogue writes zeros)
            if (elect_one()) {
                mbar_arrive_expect_tx(kfull, 2 * SH::KTILE);
                for (int x = 0; x < 2; ++x)
                    for (int bx = 0; bx < SH::NBOX; ++bx)
                        tma_load_2d(sK + x * SH::KTILE + bx * SH::KBOX, &tmK, bx * SH::BOXC, kb + s0 + x * 128, kfull);
            }
            __syncwarp();
            const uint32_t idS = idesc_bf16_f32(128, ROWS);
            const uint32_t idK = idesc_bf16_f32(128, D) | kIdescBMn;
            const uint64_t dKs = smem_desc_kmajor(smem_u32(sK), SH::ROWB), dQs = smem_desc_kmajor(smem_u32(sQ), SH::ROWB);
            const uint64_t dQt = smem_desc_mnmajor(smem_u32(sQ), SH::ROWB, SH::QBOX);
            const uint32_t tbase = __shfl_sync(0xffffffffu, tmem, 0);
            bool alive = __all_sync(0xffffffffu, mbar_wait(kfull, 0, status, 43));
            if (!alive) *abort_flag = 1;
            auto flush = [&](int j, int x) {   // dK += G . Q of block j, tile x
                const int s = j % NS;
                const uint64_t bd = dQt + s * (SH::QTILE >> 4);
                alive = tc_wait_warp(&gfull[x], j & 1, status, 44, abort_flag, alive);
                if (!alive) return;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < ROWS / 16; ++kk)
                        tc_mma_ta(tbase + x * D, tbase + 256 + x * 128 + SH::g_step(kk), bd + kk * SH::ROWB, idK,
                                  kk > 0 || j > 0 ? 1u : 0u);
                    tc_commit(&sfree[x]);
                    if (x == 1) tc_commit(&qfree[s]);
                }
                __syncwarp();
            };
            // the two tiles take turns: one's S, then the other's dK, so that a tile's epilogue runs
            // beside the other tile's products
            for (int j = 0; j < nb && alive; ++j) {
                const int s = j % NS;
                alive = tc_wait_warp(&qfull[s], (j / NS) & 1, status, 45, abort_flag, alive);
                if (!alive) break;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the copies, for the MMA's reads
                const uint64_t bd = dQs + s * (SH::QTILE >> 4);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    alive = tc_wait_warp(&sfree[x], (j & 1) ^ 1u, status, 46, abort_flag, alive);
                    if (!alive) break;
                    tc_fence_after();
                    const uint64_t ad = dKs + x * (SH::KTILE >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const int bx = kk / (SH::BOXC / 16);
                            const uint32_t ko = (kk % (SH::BOXC / 16)) * 2;
                            tc_mma(tbase + 256 + x * 128, ad + bx * (SH::KBOX >> 4) + ko, bd + bx * (SH::QBOX >> 4) + ko,
                                   idS, kk > 0 ? 1u : 0u);
                        }
                        tc_commit(&sfull[x]);
                    }
                    __syncwarp();
                    if (x == 1) flush(j, 0);
                    else if (j > 0) flush(j - 1, 1);
                }
            }
            if (alive) flush(nb - 1, 1);
            if (elect_one()) tc_commit(dkfull);   // every MMA issued so far
            __syncwarp();
            mbar_wait(dkfull, 0, status, 47);
            if (!alive) mbar_wait(kfull, 0, status, 48);   // the key tiles have landed before the CTA leaves
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------- epilogue
        const int quarter = warp & 3, set = (warp - 5) >> 3, half = ((warp - 5) >> 2) & 1;
        const int lrow = quarter * 32 + lane;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        constexpr int CW = SH::CW;
        bool alive = true;
        for (int j = 0; j < nb; ++j) {
            const int s = j % NS;
            alive = tc_wait_warp(&efull[s], (j / NS) & 1, status, 49, abort_flag, alive);
            alive = tc_wait_warp(&sfull[set], j & 1, status, 50, abort_flag, alive);
            if (!alive) break;
            tc_fence_after();
            const float* e = sE + s * NQ * kDkKeys + set * 128 + lrow;
#pragma unroll
            for (int x = 0; x < ROWS / 2; x += CW) {
                const int c0 = half * (ROWS / 2) + x;   // query-head rows (columns of S) c0 .. c0 + CW - 1
                float v[CW];
                tmem_load<CW>(tS + set * 128 + c0 + lanes, v);
                const float* w = sW + s * ROWS + c0;
                float eq[CW > H ? CW / H : 1];
#pragma unroll
                for (int q = 0; q < (CW > H ? CW / H : 1); ++q) eq[q] = e[(c0 / H + q) * kDkKeys];
                uint32_t g[CW / 2];
#pragma unroll
                for (int c = 0; c < CW; c += 4) {
                    const float4 w4 = *reinterpret_cast<const float4*>(w + c);
                    const float wv[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                    for (int y = 0; y < 4; ++y) v[c + y] = v[c + y] > 0.f ? eq[CW > H ? (c + y) / H : 0] * wv[y] : 0.f;
                    g[c / 2] = pack_bf16x2(v[c], v[c + 1]);
                    g[c / 2 + 1] = pack_bf16x2(v[c + 2], v[c + 3]);
                }
                tmem_store<CW / 2>(tS + set * 128 + SH::g_chunk(c0) + lanes, g);
            }
            tc_fence_before();
            mbar_arrive(&gfull[set]);
            mbar_arrive(&efree[s]);
        }
        // the finished rows
        if (nb > 0) {
            alive = tc_wait_warp(dkfull, 0, status, 52, abort_flag, alive);
            tc_fence_after();
        }
        const int key = s0 + set * 128 + lrow;
        const int64_t row = (int64_t)kb + key;
#pragma unroll
        for (int x0 = 0; x0 < D / 2; x0 += 16) {   // each set half of the dimensions
            const int x = half * (D / 2) + x0;
            float v[16];
            if (nb > 0 && alive) {
                tmem_load<16>(tDK + set * D + x + lanes, v);
            } else {
#pragma unroll
                for (int c = 0; c < 16; ++c) v[c] = 0.f;
            }
            if (key < L) {
                if (a.parts > 1) {
                    float* out = a.part + ((int64_t)part * a.l.n_k + row) * D + x;
#pragma unroll
                    for (int c = 0; c < 16; c += 4)
                        *reinterpret_cast<float4*>(out + c) = make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]);
                } else {
                    __nv_bfloat16* out = a.l.dK + row * D + x;
#pragma unroll
                    for (int c = 0; c < 16; c += 8)
                        *reinterpret_cast<uint4*>(out + c) =
                            make_uint4(pack_bf16x2(v[c], v[c + 1]), pack_bf16x2(v[c + 2], v[c + 3]),
                                       pack_bf16x2(v[c + 4], v[c + 5]), pack_bf16x2(v[c + 6], v[c + 7]));
                }
            }
            __syncwarp();   // the next load is the whole warp's
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 4) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// dK = the parts' sums added in order, rounded once.  n4 groups of four values.
__global__ void __launch_bounds__(256) list_dk_join_kernel(const float4* part, int32_t parts, int64_t n4, uint2* dK)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    grid_dep_wait();
    if (i >= n4) return;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int U = 8;   // parts read together
    for (int p0 = 0; p0 < parts; p0 += U) {
        float4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = p0 + u < parts ? part[(p0 + u) * n4 + i] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            s.x += v[u].x; s.y += v[u].y; s.z += v[u].z; s.w += v[u].w;
        }
    }
    dK[i] = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
}

}  // namespace dsa
