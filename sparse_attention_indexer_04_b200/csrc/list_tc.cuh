// Indexer scores at listed keys and their backward pass on the tensor cores (tcgen05 / TMEM).
//
// One query at a time per CTA: its listed keys pass by in tiles of 128, gathered by
// asynchronous copies, and
//   S[128 keys x HP heads] = K_tile . Q^T                 (A = keys, B = heads, both K-major over d)
//   scores: s[j] = sum_h w_h max(0, S[j,h])               (registers; one key per thread)
//   backward, with e = ds[j]:
//     G[j,h] = e w_h where S > 0, else 0, in bf16 in shared memory,
//     dQ^T[d x HP] += K_tile^T . G                        (both operands MN-major: the gathered tile and G as they lie)
//     dW_h = sum_j e max(0, S[j,h])                       (fp32 registers, joined once per query)
//     R[j] = G[j,:] . Q                                   (kListGradRows: rows that dK is summed from)
// G is the one value rounded below fp32 (to the operands' type, once, after e w in fp32): independent
// errors of 2^-9 that leave dQ and dK about 1.4 times their own rounding to bf16 off.
//
// What bounds it (d = 128, H = 64, 4096 queries of 2048 keys out of 32K):
//   scores 250 us: the gather, 256 bytes a listed pair out of L2 at 8.4 TB/s (tensor pipe 25 %);
//   dQ, dW 346 us: shared memory, of whose bandwidth a tile of 128 keys takes 1150 of 1450 clocks (32 KB
//     gathered, 48 KB read by S, 48 KB by dQ, 16 KB of G written); tensor pipe 36 %, issue 58 %;
//   with rows 1146 us: 512 bytes a pair written, 3.7 TB/s (960 threads leave 64 registers each: at H = 64,
//     d = 128 it spills 134 bytes a thread, which has not been weighed apart).
// Roles: warp 0 and three late ones gather; warp 1 issues S, a late one dQ (and R); the warps between are
// the epilogue, the last eight (kListGradRows) store R.  S is double-buffered, so a tile's product runs
// while the tile before is worked on.  HP = max(16, H): heads above H have zero rows in the query tile.
// Every wait is bounded.
#pragma once

#include <math_constants.h>

#include "list.cuh"
#include "ptx.cuh"

namespace dsa {

// Epilogue warps: two groups on alternate tiles, of four warps (forward) or of eight (backward: two sets,
// half of the heads each).  Backward measured 421 us for a packed batch of 8K queries with 16 heads a
// thread in one group, 400 us so (and 373 with the other steps since).
constexpr int kListTcProducers = 4;
constexpr int list_sets(int mode) { return mode ? 4 : 2; }
constexpr int list_threads(int mode)
{
    return 32 * (1 + kListTcProducers + (mode ? 1 : 0) + (mode == 2 ? 8 : 0)) + 128 * list_sets(mode);
}
constexpr uint32_t kErrListAlign = 3;

// Shared-memory matrix descriptor of an MN-major operand: rows of the K dimension are row_bytes
// (64 or 128) long, swizzled to match, 8-row groups contiguous; blocks of row_bytes along M or N
// are mn_stride bytes apart.
__device__ __forceinline__ uint64_t smem_desc_mnmajor(uint32_t addr, uint32_t row_bytes, uint32_t mn_stride)
{
    uint64_t d = 0;
    d |= (uint64_t)((addr >> 4) & 0x3FFFu);
    d |= (uint64_t)((mn_stride >> 4) & 0x3FFFu) << 16;
    d |= (uint64_t)(((8u * row_bytes) >> 4) & 0x3FFFu) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)(row_bytes == 128 ? 2u : 4u) << 61;
    return d;
}

constexpr uint32_t kIdescAMn = 1u << 15, kIdescBMn = 1u << 16;   // operand is MN-major

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v)
{
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float* v)
{
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_ld4(uint32_t taddr, float* v)
{
    uint32_t r[4];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
}

// N (4, 8, 16, 32 or 64) consecutive columns of this thread's TMEM lane; waits for them.
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t taddr, float* v)
{
    if constexpr (N == 4) {
        tmem_ld4(taddr, v);
    } else if constexpr (N == 8) {
        tmem_ld8(taddr, v);
    } else if constexpr (N == 16) {
        tmem_ld16(taddr, v);
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 32) tmem_ld32(taddr + i, v + i);
    }
    tmem_ld_wait();
    tmem_regs_ready<N>(v);
}

// tc_wait by a whole warp with one answer (the warp's next steps are warp-wide); false stays false.
__device__ __forceinline__ bool tc_wait_warp(uint64_t* bar, uint32_t parity, uint32_t* status, uint32_t where,
                                             volatile int32_t* abort_flag, bool alive)
{
    return __all_sync(0xffffffffu, alive && tc_wait(bar, parity, status, where, abort_flag));
}

// Stores N (4, 8 or 16) consecutive 32-bit columns of this thread's TMEM lane and waits for them.
template <int N>
__device__ __forceinline__ void tmem_store(uint32_t taddr, const uint32_t* r)
{
    static_assert(N == 4 || N == 8 || N == 16);
    if constexpr (N == 4) {
        asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                     "r"(r[2]), "r"(r[3])
                     : "memory");
    } else if constexpr (N == 8) {
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                     "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                     : "memory");
    } else {
        asm volatile(
            "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
            "%15, %16};" ::"r"(taddr),
            "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
            "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
            : "memory");
    }
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// tc_mma with the A operand in TMEM: lane = row, two bf16 of consecutive k a column.
__device__ __forceinline__ void tc_mma_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// True in one lane of the warp, the same one every time.  The issuing warp runs its loops whole and
// only the MMAs and commits under this, so that descriptors stay in uniform registers: built by a
// single diverged lane they cost about 150 clocks an MMA.
__device__ __forceinline__ bool elect_one()
{
    uint32_t on;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(on));
    return on != 0;
}

__device__ __forceinline__ void named_barrier(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Copies 16 bytes to shared memory, past L1.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// One of the barrier's expected arrivals, made when this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <int D, int HP>
struct ListShape {
    static constexpr uint32_t ROWB = D * 2 >= 128 ? 128 : 64;
    static constexpr int BOXC = ROWB / 2;
    static constexpr int NBOX = D / BOXC;
    static constexpr uint32_t KBOX = 128u * ROWB;
    static constexpr uint32_t KTILE = KBOX * NBOX;
    static constexpr uint32_t QBOX = (uint32_t)HP * ROWB;
    static constexpr uint32_t QTILE = QBOX * NBOX;
    static constexpr uint32_t GTILE = 128u * 128u;   // rows of 128 bytes, the first HP heads used
    static constexpr uint32_t W_BYTES = 4u * 2u * HP * 4;         // [set][parity][head]
    static constexpr uint32_t DW_BYTES = 2u * 8u * HP * 4;        // [parity][group][quarter][head]
    static constexpr uint32_t BAR_BYTES = 512;
    static constexpr uint32_t align1k(uint32_t x) { return (x + 1023u) & ~1023u; }
    // key stages, query tiles, G tiles, then the small arrays.  An operand tile narrower than the
    // MMA's 128 rows (d < 128) reads past itself into what follows: rows nobody looks at.
    static constexpr uint32_t q_off(int stages) { return stages * KTILE; }
    static constexpr uint32_t g_off(int stages) { return q_off(stages) + align1k(2 * QTILE); }
    static constexpr uint32_t w_off(int stages) { return g_off(stages) + 2 * GTILE; }
    static constexpr uint32_t x_off(int stages) { return w_off(stages) + W_BYTES + DW_BYTES + BAR_BYTES; }
    // rows: 4 KB a writing warp (eight), a 32 x 32 tile of dK on its way to memory
    static constexpr uint32_t bytes(int stages, bool rows) { return x_off(stages) + (rows ? 8u * 4096u : 0u); }
};

struct ListTcArgs {
    ListArgs l;
    int32_t n_stages;
    int32_t t0, t1;        // queries of the launch
    int32_t splits;        // kListScores: CTAs of a query, which take its tiles in turn (1: every CTA several queries)
    // kListGradRows: the rows sum_h G[t,j,h] q[t,h], stored by key.  Key row s lists its rows from
    // base[s / keys of a block] + off[s] on; before query t's come pre + the bits below t's.
    float* part;
    const uint32_t* bits;  // [words][n_k]
    const uint16_t* pre;   // [words][n_k]
    const uint32_t* off;   // [n_k]
    const uint32_t* base;
};

// The bf16 pair (e w where s > 0, else 0) of two products s: 0 - s has its sign bit set exactly where
// s > 0 (zeros of either sign give +0), and that bit, spread over 16 bits, masks the rounded e w.
__device__ __forceinline__ uint32_t relu_grad_pair(float s0, float s1, uint64_t ee, uint64_t ww)
{
    float n0, n1, g0, g1;
    unpack_f32x2(fma_f32x2(pack_f32x2(s0, s1), pack_f32x2(-1.f, -1.f), 0), n0, n1);
    unpack_f32x2(mul_f32x2(ee, ww), g0, g1);
    uint32_t m;   // bytes 0, 1: the sign of n0 eight times over; 2, 3: of n1
    asm("prmt.b32 %0, %1, %2, 0xFFBB;" : "=r"(m) : "r"(__float_as_uint(n0)), "r"(__float_as_uint(n1)));
    return pack_bf16x2(g0, g1) & m;
}

// Sums N (at most 32) per-lane values over the warp: lane i < N ends with the sum of value i in v[0].
// Each step halves the number of values, so N values cost about N shuffles.
template <int N>
__device__ __forceinline__ void warp_transpose_sum(float* v, int lane)
{
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float send = up ? v[i] : v[i + o];
            const float keep = up ? v[i + o] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
#pragma unroll
    for (int o = N; o < 32; o <<= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
}

// What a launch makes: scores; dQ and dW; those and the rows G . Q that dK is summed from.
enum : int { kListScores = 0, kListGrad = 1, kListGradRows = 2 };

template <int D, int HP, int MODE>
__global__ void __launch_bounds__(list_threads(MODE), 1)
    list_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ ListTcArgs a)
{
    constexpr bool BWD = MODE != kListScores, ROWS = MODE == kListGradRows;
    using SH = ListShape<D, HP>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint32_t* status = a.l.status;
    if (smem_u32(smem) & 1023u) {
        if (threadIdx.x == 0) record_error(status, kErrListAlign, blockIdx.x);
        return;
    }
    const int n_stages = a.n_stages;
    uint8_t* sK = smem;
    uint8_t* sQ = smem + SH::q_off(n_stages);
    uint8_t* sG = smem + SH::g_off(n_stages);
    float* sW = reinterpret_cast<float*>(smem + SH::w_off(n_stages));
    float* sDW = sW + SH::W_BYTES / 4;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + SH::w_off(n_stages) + SH::W_BYTES + SH::DW_BYTES);
    uint64_t* kempty = full + n_stages;   // the tile's products have read it
    uint64_t* qfull = kempty + n_stages;       // [2] the query tile has landed
    uint64_t* qempty = qfull + 2;              // [2] its last product has read it
    uint64_t* sfull = qempty + 2;              // [2] S is complete
    uint64_t* sfree = sfull + 2;               // [2] S has been read
    uint64_t* gfull = sfree + 2;               // [2] G is written
    uint64_t* gfree = gfull + 2;               // [2] G has been read
    uint64_t* dqfull = gfree + 2;              // [2] dQ of a query is complete
    uint64_t* dqfree = dqfull + 2;             // [2] dQ has been read
    uint64_t* dkfull = dqfree + 2;             // [2] a tile's rows of dK are complete
    uint64_t* dkfree = dkfull + 2;             // [2] and read
    uint64_t* drain = dkfree + 2;              // [2] one per issuing warp
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
    volatile int32_t* abort_flag = reinterpret_cast<volatile int32_t*>(tmem_slot + 1);

    constexpr int kEpi = 4 * list_sets(MODE);   // epilogue warps 2 .. kEpi + 1
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < n_stages; ++i) mbar_init(&full[i], kListTcProducers * 32);
        for (int i = 0; i < n_stages; ++i) mbar_init(&kempty[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&qfull[i], 1);
            mbar_init(&qempty[i], 1);
            mbar_init(&sfull[i], 1);
            mbar_init(&sfree[i], BWD ? 256 : 128);
            mbar_init(&gfull[i], 256);
            mbar_init(&gfree[i], 1);
            mbar_init(&dqfull[i], 1);
            mbar_init(&dqfree[i], 512);
            mbar_init(&dkfull[i], 1);
            mbar_init(&dkfree[i], 128);
        }
        for (int i = 0; i < 2; ++i) mbar_init(&drain[i], 1);
        *abort_flag = 0;
        fence_barrier_init();
        prefetch_tensormap(&tmQ);
    }
    // heads above H: zero rows that no load overwrites
    for (uint32_t i = threadIdx.x; i < SH::align1k(2 * SH::QTILE) / 4; i += list_threads(MODE))
        reinterpret_cast<uint32_t*>(sQ)[i] = 0u;
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    constexpr uint32_t kCols = ROWS ? 512 : 256;   // S 2 x 64, dQ 2 x 64, rows of dK 2 x 128
    if (warp == 1) tmem_alloc(tmem_slot, kCols);
    grid_dep_wait();   // the rows come from the set-up kernel
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tS = tmem, tDQ = tmem + 128;
    const int P = BWD ? 1 : a.splits, p = BWD ? 0 : blockIdx.x % P;
    const int t0 = a.t0 + blockIdx.x / P, n_q = a.t1, H = a.l.H, k = a.l.k, step = gridDim.x / P;
    // this CTA's tiles of a list: p, p + P, ...
    auto tiles = [&](int ncols) {
        const int nt = (ncols + 127) >> 7;
        return BWD ? nt : nt > p ? (nt - p + P - 1) / P : 0;
    };
    const RowDesc none{0, 0, 0, 0};

    if (warp == 0 || (warp >= 2 + kEpi && warp < 5 + kEpi)) {
        // ------------------------------------------------------ producers
        // Four warps of 32 tile rows each, 16 bytes a lane (asynchronous copies, two rows of 256 bytes
        // an instruction at d = 128): 1050 clocks a tile, the L2's pace; TMA (gather4) took 2400.
        const int pw = warp == 0 ? 0 : warp - 1 - kEpi;
        constexpr int CPR = D / 8;             // 16-byte chunks of a row
        constexpr int RPI = 32 / CPR;          // rows per instruction
        constexpr int CPB = SH::ROWB / 16;     // chunks of a box row
        const int chunk = lane % CPR, rsub = lane / CPR;
        const uint32_t coff = (uint32_t)(chunk / CPB) * SH::KBOX;
        const int cc = chunk % CPB;
        const uint32_t sk = smem_u32(sK);
        int stage = 0, it = 0;
        uint32_t phase = 0;
        int q_issued = 0;
        bool alive = true;
        // rows two queries ahead; the next query's first keys and its sequence's first key row one ahead, so
        // that queries of one tile do not wait for them in turn
        RowDesc nx = t0 < n_q ? a.l.rows[t0] : none, nx2 = t0 + step < n_q ? a.l.rows[t0 + step] : none;
        int key_next = 0, kb_next = 0;
        auto ask = [&](int t, const RowDesc& r) {
            if (t >= n_q || r.ncols == 0) return;
            // places behind the last take its key again
            key_next = __ldg(a.l.lists + (int64_t)t * k + min(p * 128 + pw * 32 + lane, r.ncols - 1));
            kb_next = a.l.k_off[r.seq];
        };
        ask(t0, nx);
        for (int t = t0; t < n_q && alive; t += step) {
            const RowDesc r = nx;
            nx = nx2;
            if (t + 2 * step < n_q) nx2 = a.l.rows[t + 2 * step];
            int key = key_next;
            const int kb = kb_next;
            ask(t + step, nx);
            const int nt = tiles(r.ncols);
            if (nt == 0) continue;
            const int qb = it & 1;
            const int32_t* l = a.l.lists + (int64_t)t * k + pw * 32 + lane;
            const int last = r.ncols - 1 - pw * 32 - lane;
            if (pw == 0) {
                int ok = 1;
                if (lane == 0) {
                    ok = tc_wait(&qempty[qb], ((it >> 1) & 1) ^ 1u, status, 21, abort_flag) ? 1 : 0;
                    if (ok) {
                        mbar_arrive_expect_tx(&qfull[qb], (uint32_t)H * D * 2);
                        for (int bx = 0; bx < SH::NBOX; ++bx)
                            tma_load_2d(sQ + qb * SH::QTILE + bx * SH::QBOX, &tmQ, bx * SH::BOXC, t * H, &qfull[qb]);
                    }
                }
                if (!__shfl_sync(0xffffffffu, ok, 0)) break;
                ++q_issued;
            }
            ++it;
            const __nv_bfloat16* kbase = a.l.K + (int64_t)kb * D + chunk * 8;
            [[maybe_unused]] const int n_seq = a.l.k_off[r.seq + 1] - a.l.k_off[r.seq];
            for (int i = 0; i < nt; ++i) {
                const int mine = DSA_CHECK(key >= 0 && key < n_seq, status, 113) ? key : 0;
                if (i + 1 < nt) key = __ldg(l + min((p + (i + 1) * P) * 128, last));
                alive = tc_wait_warp(&kempty[stage], phase ^ 1u, status, 22, abort_flag, alive);
                if (!alive) break;
                const uint32_t tile = sk + stage * SH::KTILE + coff;
#pragma unroll
                for (int x = 0; x < 32 / RPI; ++x) {
                    const int row = pw * 32 + x * RPI + rsub;
                    const int s = __shfl_sync(0xffffffffu, mine, x * RPI + rsub);
                    const int sw = SH::ROWB == 128 ? cc ^ (row & 7) : cc ^ ((row >> 1) & 3);
                    cp_async16(tile + row * SH::ROWB + sw * 16, kbase + (int64_t)s * D);
                }
                cp_async_arrive(&full[stage]);
                if (++stage == n_stages) { stage = 0; phase ^= 1u; }
            }
        }
        // every copy this warp started lands before the CTA leaves
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (pw == 0 && lane == 0 && *abort_flag)
            for (int back = 1; back <= 2 && back <= q_issued; ++back) {
                const int i = q_issued - back;
                mbar_wait(&qfull[i & 1], (uint32_t)((i >> 1) & 1), status, 23);
            }
        __syncwarp();
    } else if (warp == 1) {
        // -------------------------------------------------------- S issuer
        const uint32_t idS = idesc_bf16_f32(128, HP);
        // operands at stage 0 / buffer 0; the address field counts 16-byte units
        const uint64_t dKs = smem_desc_kmajor(smem_u32(sK), SH::ROWB), dQs = smem_desc_kmajor(smem_u32(sQ), SH::ROWB);
        const uint32_t tbase = __shfl_sync(0xffffffffu, tmem, 0);
        int stage = 0;
        uint32_t phase = 0;
        int n = 0, it = 0;     // tiles and non-empty queries so far
        bool alive = true;
        int nx = t0 < n_q ? a.l.rows[t0].ncols : 0, nx2 = t0 + step < n_q ? a.l.rows[t0 + step].ncols : 0;
        for (int t = t0; t < n_q && alive; t += step) {
            const int nt = __shfl_sync(0xffffffffu, tiles(nx), 0);
            nx = nx2;
            if (t + 2 * step < n_q) nx2 = a.l.rows[t + 2 * step].ncols;
            if (nt == 0) continue;
            const int qb = it & 1;
            alive = tc_wait_warp(&qfull[qb], (it >> 1) & 1, status, 27, abort_flag, alive);
            for (int i = 0; i < nt && alive; ++i, ++n) {
                const int b = n & 1;
                alive = tc_wait_warp(&full[stage], phase, status, 28, abort_flag, alive);
                alive = tc_wait_warp(&sfree[b], ((n >> 1) & 1) ^ 1u, status, 29, abort_flag, alive);
                if (!alive) break;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the copies, for the MMA's reads
                tc_fence_after();
                const uint64_t ad = dKs + stage * (SH::KTILE >> 4), bd = dQs + qb * (SH::QTILE >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const int bx = kk / (SH::BOXC / 16);
                        const uint32_t ko = (kk % (SH::BOXC / 16)) * 2;   // 16 values of a row: 32 bytes
                        tc_mma(tbase + b * 64, ad + bx * (SH::KBOX >> 4) + ko, bd + bx * (SH::QBOX >> 4) + ko, idS,
                               kk > 0 ? 1u : 0u);
                    }
                    tc_commit(&sfull[b]);
                    if (!ROWS && i == nt - 1) tc_commit(&qempty[qb]);
                    if (!BWD) tc_commit(&kempty[stage]);
                }
                __syncwarp();
                if (++stage == n_stages) { stage = 0; phase ^= 1u; }
            }
            ++it;
        }
        if (elect_one()) tc_commit(&drain[0]);   // every MMA issued has completed before TMEM is released
        __syncwarp();
        mbar_wait(&drain[0], 0, status, 30);
        __syncwarp();
    } else if (BWD && warp == 5 + kEpi) {
        // -------------------------------------------------------- dQ issuer
        // A warp of its own: its waits and the S issuer's overlap (one issuer left the tensor cores
        // idle for about 550 clocks a tile).
        const uint32_t idQ = idesc_bf16_f32(128, HP) | kIdescAMn | kIdescBMn;
        const uint64_t dKt = smem_desc_mnmajor(smem_u32(sK), SH::ROWB, SH::KBOX);
        const uint64_t dGt = smem_desc_mnmajor(smem_u32(sG), 128, 0);
        [[maybe_unused]] const uint32_t idK = idesc_bf16_f32(128, D) | kIdescBMn;
        [[maybe_unused]] const uint64_t dGk = smem_desc_kmajor(smem_u32(sG), 128);
        [[maybe_unused]] const uint64_t dQt = smem_desc_mnmajor(smem_u32(sQ), SH::ROWB, SH::QBOX);
        const uint32_t tbase = __shfl_sync(0xffffffffu, tmem, 0) + 128;
        int stage = 0, n = 0, it = 0;
        bool alive = true;
        int nx = t0 < n_q ? a.l.rows[t0].ncols : 0, nx2 = t0 + step < n_q ? a.l.rows[t0 + step].ncols : 0;
        for (int t = t0; t < n_q && alive; t += step) {
            const int nt = __shfl_sync(0xffffffffu, (nx + 127) >> 7, 0);
            nx = nx2;
            if (t + 2 * step < n_q) nx2 = a.l.rows[t + 2 * step].ncols;
            if (nt == 0) continue;
            const int qb = it & 1;
            alive = tc_wait_warp(&dqfree[qb], ((it >> 1) & 1) ^ 1u, status, 26, abort_flag, alive);
            for (int i = 0; i < nt && alive; ++i, ++n) {
                const int b = n & 1;
                // (G is written from this tile's S: the tile has landed, and the S issuer saw it)
                alive = tc_wait_warp(&gfull[b], (n >> 1) & 1, status, 25, abort_flag, alive);
                if (!alive) break;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                tc_fence_after();
                const uint64_t ad = dKt + stage * (SH::KTILE >> 4), bd = dGt + b * (SH::GTILE >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)   // 16 keys each
                        tc_mma(tbase + qb * 64, ad + kk * SH::ROWB, bd + kk * 128, idQ, kk > 0 || i > 0 ? 1u : 0u);
                    tc_commit(&kempty[stage]);
                    if (!ROWS) tc_commit(&gfree[b]);
                    if (i == nt - 1) tc_commit(&dqfull[qb]);
                }
                __syncwarp();
                if constexpr (ROWS) {   // the tile's rows of dK: G [keys x heads] . Q [heads x d]
                    alive = tc_wait_warp(&dkfree[b], ((n >> 1) & 1) ^ 1u, status, 35, abort_flag, alive);
                    if (!alive) break;
                    tc_fence_after();
                    const uint64_t gd = dGk + b * (SH::GTILE >> 4), qd = dQt + qb * (SH::QTILE >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < HP / 16; ++kk)
                            tc_mma(tbase + 128 + b * 128, gd + kk * 2, qd + kk * SH::ROWB, idK, kk > 0 ? 1u : 0u);
                        tc_commit(&gfree[b]);
                        tc_commit(&dkfull[b]);
                        if (i == nt - 1) tc_commit(&qempty[qb]);
                    }
                    __syncwarp();
                }
                if (++stage == n_stages) stage = 0;
            }
            ++it;
        }
        if (elect_one()) tc_commit(&drain[1]);
        __syncwarp();
        mbar_wait(&drain[1], 0, status, 34);
        __syncwarp();
    } else if (ROWS && warp >= 6 + kEpi) {
        // ------------------------------------------------- rows of dK to memory
        // two groups of four on alternate tiles
        const int quarter = warp & 3, lrow = quarter * 32 + lane, grp = (warp - 6 - kEpi) >> 2;
        int n = 0;
        bool alive = true;
        RowDesc nx = t0 < n_q ? a.l.rows[t0] : none;
        for (int t = t0; t < n_q && alive; t += step) {
            const RowDesc r = nx;
            const int nt = (r.ncols + 127) >> 7;
            if (t + step < n_q) nx = a.l.rows[t + step];
            const int32_t* l = a.l.lists + (int64_t)t * k;
            const int kb = a.l.k_off[r.seq];
            const int64_t word = (int64_t)((t - a.t0) >> 5) * a.l.n_k;
            const uint32_t below = (1u << ((t - a.t0) & 31)) - 1u;
            // the next tile's place is looked up while this one is stored: key two tiles ahead
            auto key_row = [&](int i) {
                const int j = i * 128 + lrow;
                const int s = kb + (j < r.ncols ? __ldg(l + j) : 0);
                return DSA_CHECK(s >= 0 && s < a.l.n_k, status, 118) ? s : 0;
            };
            auto place = [&](int s) {
                return __ldg(a.base + s / kPosBlock) + __ldg(a.off + s) + __ldg(a.pre + word + s) +
                       __popc(__ldg(a.bits + word + s) & below);
            };
            const int i0 = (n & 1) == grp ? 0 : 1;   // the group's first tile
            uint32_t at = i0 < nt ? place(key_row(i0)) : 0u;
            int s_next = i0 + 2 < nt ? key_row(i0 + 2) : 0;
            for (int i = i0; i < nt && alive; i += 2) {
                const uint32_t mine = at;
                if (i + 2 < nt) at = place(s_next);
                if (i + 4 < nt) s_next = key_row(i + 4);
                alive = tc_wait_warp(&dkfull[grp], ((n + i) >> 1) & 1, status, 36, abort_flag, alive);
                if (!alive) break;
                tc_fence_after();
                // Through shared memory, so that eight lanes store a whole 128-byte line: a lane storing its
                // own row took four times the requests (1.58 ms for 4096 queries of 2048 places).
                float4* tile = reinterpret_cast<float4*>(smem + SH::x_off(n_stages)) + (grp * 4 + quarter) * 256;
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    float v[32];
                    tmem_load<32>(tmem + 256 + grp * 128 + c + ((uint32_t)(quarter * 32) << 16), v);
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        tile[lane * 8 + (x ^ (lane & 7))] = make_float4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
                    __syncwarp();
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        const int row = y * 4 + lane / 8, x = lane & 7;
                        const float4 o = tile[row * 8 + (x ^ (row & 7))];
                        const uint32_t to = __shfl_sync(0xffffffffu, mine, row);
                        if (i * 128 + quarter * 32 + row < r.ncols)
                            *reinterpret_cast<float4*>(a.part + (int64_t)to * D + c + 4 * x) = o;
                    }
                    __syncwarp();
                }
                tc_fence_before();
                mbar_arrive(&dkfree[grp]);
            }
            n += nt;
        }
    } else {
        // ---------------------------------------------------------- epilogue
        // Named barriers are met by all threads of a set whatever an abort makes of the waits, so the
        // loops run to their end with `alive` false instead of leaving.
        const int quarter = warp & 3;           // TMEM lanes this warp may read
        const int set = (warp - 2) >> 2;
        const int lrow = quarter * 32 + lane;   // key of the tile
        const int st = threadIdx.x - 64 - set * 128;   // thread of the set
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        // head h's part of a score; the zero rows above H give NaN with an infinite key
        [[maybe_unused]] auto relu = [&](int h, float x) { return relu_nan(HP > 16 || h < H ? x : 0.f); };
        int n = 0, it = 0, all = 0;
        bool alive = true;
        int nx = t0 < n_q ? a.l.rows[t0].ncols : 0, nx2 = t0 + step < n_q ? a.l.rows[t0 + step].ncols : 0;
        float wnext = st < H && t0 < n_q ? a.l.W[(int64_t)t0 * H + st] : 0.f;
        // With few heads dQ of a query is read a query later, when its last product has long been made
        // (4096 queries of 512 keys, H = 4: 82 us at once, 74 so; with 64 heads the registers that it
        // takes cost more than the wait: 373 us at once, 403 so)
        constexpr bool LATE = HP < 64;
        [[maybe_unused]] int held = -1;
        [[maybe_unused]] auto readout = [&](int t, int i) {   // query t, the i-th with a list
            constexpr int NR = HP / 4;     // heads whose dQ a set writes
            const int r0 = set * NR, qb = i & 1;
            alive = tc_wait_warp(&dqfull[qb], (i >> 1) & 1, status, 33, abort_flag, alive);
            if (!alive) return;
            tc_fence_after();
            float v[NR];
            tmem_load<NR>(tDQ + qb * 64 + r0 + lanes, v);
            tc_fence_before();
            mbar_arrive(&dqfree[qb]);
            if (a.l.dQ && lrow < D) {
                __nv_bfloat16* out = a.l.dQ + ((int64_t)t * H + r0) * D + lrow;
#pragma unroll
                for (int c = 0; c < NR; ++c)
                    if (r0 + c < H) out[c * D] = __float2bfloat16_rn(v[c]);
            }
            __syncwarp();
        };
        // ds of a query's first tile of this set's group
        [[maybe_unused]] float first = 0.f;
        [[maybe_unused]] auto ask = [&](int t, int n, int ncols) {
            const int j = ((n & 1) == (set >> 1) ? 0 : 128) + lrow;
            first = t < n_q && j < ncols ? a.l.ds[(int64_t)t * k + j] : 0.f;
        };
        if (BWD) ask(t0, 0, nx);
        for (int t = t0; t < n_q; t += step, ++all) {
            const int ncols = nx;
            nx = nx2;
            if (t + 2 * step < n_q) nx2 = a.l.rows[t + 2 * step].ncols;
            float* w = sW + (set * 2 + (all & 1)) * HP;
            if (st < HP) w[st] = wnext;
            if (t + step < n_q) wnext = st < H ? a.l.W[(int64_t)(t + step) * H + st] : 0.f;
            named_barrier(1 + set, 128);
            const int nt = tiles(ncols);
            if constexpr (!BWD) {
                for (int i = (n & 1) == set ? 0 : 1; i < nt; i += 2) {   // the set's tiles
                    const int g = n + i;   // the CTA's tile number
                    alive = tc_wait_warp(&sfull[set], (g >> 1) & 1, status, 31, abort_flag, alive);
                    if (!alive) continue;
                    tc_fence_after();
                    float v[HP];
                    tmem_load<HP>(tS + set * 64 + lanes, v);
                    tc_fence_before();
                    mbar_arrive(&sfree[set]);
                    const int j = (p + i * P) * 128 + lrow;
                    uint64_t acc = 0;   // even heads and odd heads
#pragma unroll
                    for (int h = 0; h < HP; h += 4) {
                        const float4 w4 = *reinterpret_cast<const float4*>(w + h);
                        acc = fma_f32x2(pack_f32x2(w4.x, w4.y), pack_f32x2(relu(h, v[h]), relu(h + 1, v[h + 1])), acc);
                        acc = fma_f32x2(pack_f32x2(w4.z, w4.w), pack_f32x2(relu(h + 2, v[h + 2]), relu(h + 3, v[h + 3])), acc);
                    }
                    float s0, s1;
                    unpack_f32x2(acc, s0, s1);
                    if (j < k) a.l.scores[(int64_t)t * k + j] = j < ncols ? (s0 + s1) + 0.f : -CUDART_INF_F;
                }
                if (set == 0 && p == 0)   // places behind the last tile
                    for (int j = ((ncols + 127) & ~127) + st; j < k; j += 128) a.l.scores[(int64_t)t * k + j] = -CUDART_INF_F;
            } else {
                constexpr int NC = HP / 2;     // heads (columns) of a set
                const int grp = set >> 1, half = set & 1, c0 = half * NC;
                uint64_t dw[NC / 2];           // pairs of heads
#pragma unroll
                for (int h = 0; h < NC / 2; ++h) dw[h] = 0;
                const float* ds = a.l.ds + (int64_t)t * k + lrow;
                int i = (n & 1) == grp ? 0 : 1;   // the group's first tile
                float e = first;
                for (; i < nt; i += 2) {
                    const uint32_t use = (uint32_t)((n + i) >> 1) & 1u;
                    // a place behind the list's end repeats the last key: its products count for nothing (e = 0)
                    const uint64_t ee = pack_f32x2(e, e);
                    e = (i + 2) * 128 + lrow < ncols ? ds[(i + 2) * 128] : 0.f;
                    alive = tc_wait_warp(&sfull[grp], use, status, 31, abort_flag, alive);
                    alive = tc_wait_warp(&gfree[grp], use ^ 1u, status, 32, abort_flag, alive);
                    if (!alive) continue;
                    tc_fence_after();
                    uint8_t* grow = sG + grp * SH::GTILE + lrow * 128;
                    constexpr int CW = NC < 16 ? NC : 16;   // columns in registers at once
                    float v[CW];
#pragma unroll
                    for (int h = 0; h < NC; h += 8) {
                        if (h % CW == 0) {
                            tmem_load<CW>(tS + grp * 64 + c0 + h + lanes, v);
                            if (h + CW == NC) {
                                tc_fence_before();
                                mbar_arrive(&sfree[grp]);
                            }
                        }
                        uint32_t p[4];
#pragma unroll
                        for (int x = 0; x < 8; x += 4) {
                            const ulonglong2 w2 = *reinterpret_cast<const ulonglong2*>(w + c0 + h + x);
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const float s0 = v[h % CW + x + 2 * y], s1 = v[h % CW + x + 2 * y + 1];
                                uint64_t& acc = dw[(h + x) / 2 + y];
                                acc = fma_f32x2(ee, pack_f32x2(relu_nan(s0), relu_nan(s1)), acc);
                                p[x / 2 + y] = relu_grad_pair(s0, s1, ee, y ? w2.y : w2.x);
                            }
                        }
                        *reinterpret_cast<uint4*>(grow + (((c0 + h) / 8 ^ (lrow & 7)) << 4)) = make_uint4(p[0], p[1], p[2], p[3]);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    mbar_arrive(&gfull[grp]);
                }
                ask(t + step, n + nt, nx);   // under the joining of dW
                float dv[NC];
#pragma unroll
                for (int h = 0; h < NC / 2; ++h) unpack_f32x2(dw[h], dv[2 * h], dv[2 * h + 1]);
                warp_transpose_sum<NC>(dv, lane);
                float* part = sDW + (all & 1) * 8 * HP;
                if (lane < NC) part[(grp * 4 + quarter) * HP + c0 + lane] = dv[0];
                named_barrier(5, 512);
                const int h = threadIdx.x - 64;
                if (a.l.dW && h < H) {
                    float s = 0.f;
#pragma unroll
                    for (int x = 0; x < 8; ++x) s += part[x * HP + h];
                    a.l.dW[(int64_t)t * H + h] = s;
                }
                if (nt > 0) {
                    if (!LATE) {
                        readout(t, it);
                    } else {
                        if (held >= 0) readout(held, it - 1);
                        held = t;
                    }
                } else if (a.l.dQ) {   // nothing listed: zero gradients
                    for (int o = threadIdx.x - 64; o < H * D; o += 512)
                        a.l.dQ[(int64_t)t * H * D + o] = __float2bfloat16_rn(0.f);
                }
            }
            n += nt;
            if (nt > 0) ++it;
        }
        if (BWD && LATE && held >= 0) readout(held, it - 1);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kCols);
    }
}

}  // namespace dsa
