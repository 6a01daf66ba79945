// libdsaidx C ABI of the operators an indexer is trained with: layer norm, the distillation loss and
// the indexer's scores at listed keys, with their gradients.  Contract: include/dsa_index.h.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/dsa_index.h"
#include "distill.cuh"
#include "host.cuh"
#include "list_dk_rows.cuh"
#include "list_dk_tc.cuh"
#include "list_tc.cuh"
#include "norm.cuh"

using namespace dsa;

namespace {

constexpr int32_t kNormMaxWidth = 16384;

bool type_ok(int32_t t) { return t == DSA_FP32 || t == DSA_BF16; }
int64_t type_size(int32_t t) { return t == DSA_FP32 ? 4 : 2; }

// A row matrix: rows of d values of the given type, ld values apart.
dsa_status check_rows(const void* p, int32_t type, int64_t ld, int64_t n, int32_t d)
{
    if (!type_ok(type)) return DSA_ERR_UNSUPPORTED;
    if (n > 0 && !p) return DSA_ERR_INVALID_ARG;
    if (n > 1 && ld < d) return DSA_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(p) & (type_size(type) - 1)) return DSA_ERR_INVALID_ARG;
    return DSA_OK;
}

// Whether every row of the matrix starts on a 16-byte boundary.
bool rows_aligned(const void* p, int32_t type, int64_t ld, int64_t n)
{
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (n <= 1 || (ld * type_size(type)) % 16 == 0);
}

// ------------------------------------------------------------- layer norm

// CTAs of the backward pass with `threads` threads that take `groups` rows at once: as many as are
// resident, fewer where that leaves a CTA under 8 rows a group, since each CTA's partial sums (8 bytes
// a column) are written and read once more.
int32_t norm_bwd_ctas(int64_t n, int32_t groups, int32_t threads)
{
    const int64_t resident = int64_t(148) * norm_bwd_per_sm(threads);
    return (int32_t)std::max<int64_t>(1, std::min((n + 8 * groups - 1) / (8 * groups), resident));
}

// The most CTAs of any backward launch: those of 128 threads.
constexpr int64_t kNormMaxCtas = 148 * norm_bwd_per_sm(128);

template <typename TX, typename TY, int VEC, int T, int NV, int NT>
dsa_status norm_launch(const NormArgs& a, bool backward, int32_t* n_part, cudaStream_t st)
{
    constexpr int G = NT / T;
    if (backward) {
        *n_part = norm_bwd_ctas(a.n, G, NT);
        DSA_LAUNCH(kProfNorm, st, layer_norm_bwd_kernel<TX, TY, VEC, T, NV, NT><<<*n_part, NT, 0, st>>>(a));
        return launched();
    }
    // narrow rows: four a group in flight once that still fills the GPU (32768 x 128: 9.0 us with one)
    constexpr int R = NV * VEC <= 8 && T <= 32 ? 4 : 1;
    if (R == 1 || a.n < int64_t(148) * G * R) {
        DSA_LAUNCH(kProfNorm, st,
                   layer_norm_kernel<TX, TY, VEC, T, NV, NT, 1><<<(unsigned)((a.n + G - 1) / G), NT, 0, st>>>(a));
    } else {
        DSA_LAUNCH(kProfNorm, st, layer_norm_kernel<TX, TY, VEC, T, NV, NT, R>
                   <<<(unsigned)((a.n + G * R - 1) / (G * R)), NT, 0, st>>>(a));
    }
    return launched();
}

// The row group of a width: as few threads as hold the row in 8 registers a thread or so, so a
// narrow row costs no cross-warp step (128 values of a key: 16 lanes with one 16-byte load each).
template <typename TX, typename TY>
dsa_status norm_pick(const NormArgs& a, bool vec, bool bwd, int32_t* np, cudaStream_t st)
{
    if (vec) {
        if (a.d <= 32) return norm_launch<TX, TY, 8, 4, 1, 256>(a, bwd, np, st);
        if (a.d <= 64) return norm_launch<TX, TY, 8, 8, 1, 256>(a, bwd, np, st);
        if (a.d <= 128) return norm_launch<TX, TY, 8, 16, 1, 256>(a, bwd, np, st);
        if (a.d <= 256) return norm_launch<TX, TY, 8, 32, 1, 256>(a, bwd, np, st);
        if (a.d <= 1024) return norm_launch<TX, TY, 8, 128, 1, 128>(a, bwd, np, st);
        if (a.d <= 2048) return norm_launch<TX, TY, 8, 256, 1, 256>(a, bwd, np, st);
        if (a.d <= 4096) return norm_launch<TX, TY, 8, 512, 1, 512>(a, bwd, np, st);
        if (a.d <= 8192) return norm_launch<TX, TY, 8, 1024, 1, 1024>(a, bwd, np, st);
        return norm_launch<TX, TY, 8, 1024, 2, 1024>(a, bwd, np, st);
    }
    if (a.d <= 32) return norm_launch<TX, TY, 1, 32, 1, 256>(a, bwd, np, st);
    if (a.d <= 128) return norm_launch<TX, TY, 1, 32, 4, 256>(a, bwd, np, st);
    if (a.d <= 256) return norm_launch<TX, TY, 1, 32, 8, 256>(a, bwd, np, st);
    if (a.d <= 1024) return norm_launch<TX, TY, 1, 256, 4, 256>(a, bwd, np, st);
    if (a.d <= 2048) return norm_launch<TX, TY, 1, 512, 4, 512>(a, bwd, np, st);
    // a kernel per 1024 columns, which the backward's registers count: with the 8-column one (which spills) for
    // all from 4097 on, 4099 x 4500 fp32 100 us against 48, 4099 x 5121 104 and 68, 3000 x 7167 88 and 66
    if (a.d <= 5120) return norm_launch<TX, TY, 1, 1024, 5, 1024>(a, bwd, np, st);
    if (a.d <= 6144) return norm_launch<TX, TY, 1, 1024, 6, 1024>(a, bwd, np, st);
    if (a.d <= 7168) return norm_launch<TX, TY, 1, 1024, 7, 1024>(a, bwd, np, st);
    if (a.d <= 8192) return norm_launch<TX, TY, 1, 1024, 8, 1024>(a, bwd, np, st);
    return norm_launch<TX, TY, 1, 1024, 16, 1024>(a, bwd, np, st);
}

dsa_status norm_dispatch(const NormArgs& a, int32_t tx, int32_t ty, bool vec, bool bwd, int32_t* np, cudaStream_t st)
{
    if (tx == DSA_FP32)
        return ty == DSA_FP32 ? norm_pick<float, float>(a, vec, bwd, np, st)
                              : norm_pick<float, __nv_bfloat16>(a, vec, bwd, np, st);
    return ty == DSA_FP32 ? norm_pick<__nv_bfloat16, float>(a, vec, bwd, np, st)
                          : norm_pick<__nv_bfloat16, __nv_bfloat16>(a, vec, bwd, np, st);
}

// Partial sums of the weight's and the bias's gradient, one row of each per CTA: norm_bwd_ctas of any row group
// is at most one CTA per 8 rows, and kNormMaxCtas.
size_t norm_part_floats(int64_t n, int32_t d)
{
    return size_t(std::min<int64_t>(std::max<int64_t>(1, (n + 7) / 8), kNormMaxCtas)) * 2 * d;
}

size_t norm_ws_bytes(int64_t n, int32_t d)
{
    Carver c{nullptr};
    c.take<float>(norm_part_floats(n, d));
    return c.off;
}

// ------------------------------------------------------------ distillation

// 2^-64 and 2^64: factors of it, and differences of scores of its size in units of 2^24, stay normal numbers.
constexpr float kMinTemperature = 5.42101086e-20f, kMaxTemperature = 1.84467441e19f;

template <typename TT, bool WEIGHTS, int VEC, bool EDGE, int T, int NV, int NT>
dsa_status distill_launch(const DistillArgs& a, cudaStream_t st)
{
    constexpr int R = NT / T;
    DSA_LAUNCH(kProfDistill, st, distill_kernel<TT, WEIGHTS, VEC, EDGE, T, NV, NT>
               <<<(unsigned)((int64_t(a.n) + R - 1) / R), NT, 0, st>>>(a));
    return launched();
}

template <typename TT, bool WEIGHTS, bool EDGE, int NV, int NT, int CTAS = 1>
dsa_status distill_ring(const DistillArgs& a, cudaStream_t st)
{
    const auto kern = distill_ring_kernel<TT, WEIGHTS, EDGE, NV, NT, CTAS>;
    const size_t smem = size_t(NV) * NT * (16 + 4 * sizeof(TT) + (a.list ? 16 : 0));
    // the limit counts lists either way: calls at the same time may set it to one value only
    dsa_status s = set_smem(kern, std::min(size_t(NV) * NT * (32 + 4 * sizeof(TT)), size_t(200) * 1024));
    if (s != DSA_OK) return s;
    // lists and fp32 teachers: three quarters of the CTAs and of the shared memory, since rows of 192 KB
    // together leave the L1 too little for their loads and stores (9000 x 2000: 66 us, so 50; the other
    // types' rows come to 128 or 160 KB: 38 and 46 us, and no faster with fewer)
    const bool wide = CTAS > 1 && a.list && sizeof(TT) == 4;
    const int ctas = wide ? CTAS * 3 / 4 : CTAS;
    const int share = wide ? int(ctas * (smem + 2048) * 100 / (228 * 1024)) + 1 : (int)cudaSharedmemCarveoutDefault;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, share) != cudaSuccess)
        return DSA_ERR_CUDA;
    DSA_LAUNCH(kProfDistill, st, kern<<<std::min(a.n, 148 * ctas), NT, smem, st>>>(a));
    return launched();
}

template <typename TT, bool WEIGHTS, int VEC, bool EDGE>
dsa_status distill_pick(const DistillArgs& a, cudaStream_t st)
{
    // 16 places a thread or so: with 8 the two joint reductions were a third of the instructions
    constexpr int U = 4 / VEC;   // registers' worth of a 4-wide load
    const int64_t k = int64_t(a.k) + (EDGE ? 3 : 0);   // columns from the boundary before the row
    if (k <= 128) return distill_launch<TT, WEIGHTS, VEC, EDGE, 32, 1 * U, 256>(a, st);
    if (k <= 512) return distill_launch<TT, WEIGHTS, VEC, EDGE, 32, 4 * U, 256>(a, st);
    // many rows: the next one read ahead, with as many CTAs an SM as hold rows of 64 KB together
    // (18000 x 1000: 46.2 us without, 37.7 with, 9000 x 2000 47.7 and 38.2, 2250 x 8000 55.5 and 41.0, fp32);
    // not for rows off the 16-byte boundaries, whose end vectors cost more there (9765 x 2049: 78 us
    // without, 88 with)
    if constexpr (VEC == 4 && !EDGE) {
        if (k > 512 && k <= 1024 && a.n > 148 * 16) return distill_ring<TT, WEIGHTS, EDGE, 4, 64, 16>(a, st);
        if (k > 1024 && k <= 2048 && a.n > 148 * 8) return distill_ring<TT, WEIGHTS, EDGE, 4, 128, 8>(a, st);
        if (k > 2048 && k <= 4096 && a.n > 148 * 4) return distill_ring<TT, WEIGHTS, EDGE, 4, 256, 4>(a, st);
        if (k > 4096 && k <= 8192 && a.n > 148 * 2) return distill_ring<TT, WEIGHTS, EDGE, 4, 512, 2>(a, st);
    }
    if (k <= 1024) return distill_launch<TT, WEIGHTS, VEC, EDGE, 64, 4 * U, 64>(a, st);
    if (k <= 2048) return distill_launch<TT, WEIGHTS, VEC, EDGE, 128, 4 * U, 128>(a, st);
    if (k <= 4096) return distill_launch<TT, WEIGHTS, VEC, EDGE, 256, 4 * U, 256>(a, st);
    if (k <= 8192) return distill_launch<TT, WEIGHTS, VEC, EDGE, 512, 4 * U, 512>(a, st);
    // longer rows, as long as shared memory holds, read ahead: 192 KB of fp32 scores and teacher are 24,576 places,
    // with lists 16,384 (900 x 23001: 108 us in two sweeps, 68 so; 1200 x 15001 with lists: 92 us without, 69 so;
    // 1000 x 20480: 97 and 51; 1100 x 17000: 103 and 52); few rows with lists the register form takes in less
    // (8 x 16000: 6.3 us, 7.1 so)
    if constexpr (VEC == 4) {
        if (k <= 12288) return distill_ring<TT, WEIGHTS, EDGE, 6, 512>(a, st);
        if (k <= 16384 && (!a.list || a.n > 148)) return distill_ring<TT, WEIGHTS, EDGE, 8, 512>(a, st);
        if (k <= 20480 && !a.list) return distill_ring<TT, WEIGHTS, EDGE, 10, 512>(a, st);
        if (k <= 24576 && !a.list) return distill_ring<TT, WEIGHTS, EDGE, 12, 512>(a, st);
    }
    if (k <= 16384) return distill_launch<TT, WEIGHTS, VEC, EDGE, 1024, 4 * U, 1024>(a, st);
    if (k <= kDistillRegCols) return distill_launch<TT, WEIGHTS, VEC, EDGE, 1024, 5 * U, 1024>(a, st);
    DSA_LAUNCH(kProfDistill, st, distill_long_kernel<TT, WEIGHTS, 512><<<a.n, 512, 0, st>>>(a));
    return launched();
}

template <typename TT, bool WEIGHTS>
dsa_status distill_rows(const DistillArgs& a, bool vec, bool edge, cudaStream_t st)
{
    if (!vec) return distill_pick<TT, WEIGHTS, 1, false>(a, st);
    return edge ? distill_pick<TT, WEIGHTS, 4, true>(a, st) : distill_pick<TT, WEIGHTS, 4, false>(a, st);
}

// ----------------------------------------------------- scores at listed keys

struct ListPlan {
    RowDesc* rows;
    uint16_t* edge;     // backward: list places at the borders of the key blocks
    float* part;        // backward: partial dK of the query parts
    int32_t key_blocks; // of the longest sequence
    int32_t units;      // key blocks over all sequences (an upper bound)
    int32_t parts;
    float* S;           // forward, by picking: every eligible score
    char* dense;        // and its launch's plan
    bool picking;
    bool by_rows;       // dK from the dQ pass's rows (list_dk_rows.cuh), not from dense key blocks
    int32_t chunk;      // by_rows: queries of one launch
    int32_t words;      // by_rows: 32-query words of a launch
    uint32_t* bits;     // by_rows: where each key's rows lie (list_dk_rows.cuh)
    uint16_t* pre;
    uint32_t *count, *off, *base;
    float* acc;         // by_rows, more than one launch: sums so far
};

// Bytes of dK rows kept between two launches (888 queries of 2048 places at d = 128, six a CTA), and of
// the bits and counts that place them (6 bytes per key and 32 queries).
constexpr size_t kRowsBudget = size_t(1024) << 20;
constexpr int32_t kRowsMaxQueries = 32768;   // (counts of 16 bits)
// Bytes of partial dK of the dense form at most.
constexpr size_t kPartsBudget = size_t(4096) << 20;

// What a batch's lists hold, as far as the host knows: the queries of a sequence taken as its last ones
// (a training batch: all of them; a chunk at the end of a context), those above its keys' number with the
// whole of it.
struct ListWork {
    double listed = 0;   // listed (query, key) pairs
    double empty = 0;    // places of the tiles of 128 that lists end in, behind their ends
    double dense = 0;    // eligible pairs
    double blocks = 0;   // (query, key block) pairs with a listed key
};

ListWork list_work(const dsa_batch* b, int32_t k)
{
    ListWork w;
    for (int i = 0; i < b->num_seqs; ++i) {
        const double L = b->k_offsets_host[i + 1] - b->k_offsets_host[i];
        const double all = b->q_offsets_host[i + 1] - b->q_offsets_host[i], nq = std::min(all, L);
        const double p0 = L - nq + 1, p1 = L;   // prefix lengths from p0 to p1
        // sums over p0 .. p1 of p, of min(k, p) and of the blocks they touch
        const auto sum = [](double lo, double hi) { return hi < lo ? 0. : (lo + hi) * (hi - lo + 1) / 2; };
        const double m = std::min<double>(k, p1), dense = sum(p0, p1);
        const double whole = std::max(0., p1 - std::max(p0 - 1, m));   // queries of k places
        const double listed = sum(p0, std::min(m, p1)) + whole * k;
        const double full = std::min<double>(k, L);   // places of a query with the whole prefix
        const auto rest = [](double places) { return std::ceil(places / 128) * 128 - places; };
        w.dense += dense + (all - nq) * L;
        w.listed += listed + (all - nq) * full;
        w.empty += whole * rest(k) + (nq - whole) * 64 + (all - nq) * rest(full);
        w.blocks += std::min(listed, dense / kDkKeys + nq / 2) + (all - nq) * std::min(full, std::ceil(L / kDkKeys));
    }
    return w;
}

// Whether dK is summed from one row per listed pair or from dense products over whole key blocks.
// Measured both ways over 35 sizes (512 to 33,000 queries, 600 to 32K keys, 1 to 512 places) with H, d of
// 4, 32; 4, 128; 16, 64 and 64, 128, in ns: a row 0.2 at d = 128 (written by the dQ pass, read once), an empty
// place of a tile 0.02 and as much again at d = 128, the bits and counts of a (query, key) 0.00005 (10 bytes for
// 32 queries of a batch and any of its keys: 24 sequences of 4096 with 64 places and 8 heads 2.2 ms by rows, 1.7
// dense); a (query, block) product 0.3 and 4.3 with 64 heads, a block's CTA 150 and 350 at d = 128.  The form
// taken so is 0.5 % slower than the better one on average, 21 % at most.
bool dk_by_rows(const dsa_batch* b, int32_t k)
{
    const ListWork w = list_work(b, k);
    const double units = b->num_keys / kDkKeys + b->num_seqs, d = b->head_dim / 128.;
    const double bits = 5e-5 * b->num_queries * b->num_keys;
    return w.listed * 0.2 * d + w.empty * (0.02 + 0.02 * d) + bits <
           w.blocks * (0.3 + 4.3 * b->num_heads / 64.) + units * (150 + 350 * d);
}

// Whether the listed scores are picked from all scores of the prefix or computed from gathered keys.
// Measured at d = 128, in ns: a gathered pair 0.033; a dense one 0.014 with 64 heads and 0.002 to write and
// read it, two more launches 8000.
bool scores_by_picking(const dsa_batch* b, const HostInfo& hi, int32_t k)
{
    if (size_t(b->num_queries) * dense_scores_ld(hi.max_k) * 4 > (size_t(4) << 30)) return false;
    const ListWork w = list_work(b, k);
    const double d = b->head_dim / 128.;
    return w.dense * (0.002 + 0.014 * d * b->num_heads / 64.) + 8000 < w.listed * 0.033 * d;
}

// CTAs that share a key block's queries: enough for three waves over the GPU (a block's work is its
// queries', so early blocks of a causal sequence have the most), no more than there are groups of 16
// queries, and enough that a CTA's queries fit its list.
int32_t dk_parts(int32_t units, int32_t max_q)
{
    const int32_t fill = (3 * 148 + units - 1) / std::max(1, units);
    const int32_t most = std::max(1, std::min(32, max_q / 16));
    return std::max((max_q + kDkMaxList - 1) / kDkMaxList, std::max(1, std::min(fill, most)));
}

size_t list_plan(char* base, const dsa_batch* b, const HostInfo& hi, int32_t k, bool backward, ListPlan* p)
{
    Carver c{base};
    *p = ListPlan{};
    p->picking = !backward && scores_by_picking(b, hi, k);
    if (p->picking) {
        p->S = c.take<float>(size_t(b->num_queries) * dense_scores_ld(hi.max_k));
        p->dense = c.take<char>(dense_scores_plan_bytes(b, hi));
        return c.off;
    }
    p->rows = c.take<RowDesc>(std::max(1, b->num_queries));
    if (!backward) return c.off;
    p->key_blocks = (hi.max_k + kDkKeys - 1) / kDkKeys;
    p->units = b->num_keys / kDkKeys + b->num_seqs;
    p->parts = dk_parts(p->units, hi.max_q);
    p->by_rows = dk_by_rows(b, k) || (p->parts > 1 && size_t(p->parts) * b->num_keys * b->head_dim * 4 > kPartsBudget);
    if (p->by_rows) {
        const int64_t row = std::min(k, std::max(1, hi.max_k));   // places of a query at most
        const int64_t fit = int64_t(kRowsBudget / (size_t(row) * b->head_dim * 4));
        const int64_t words = std::max<int64_t>(1, int64_t(kRowsBudget / (6 * size_t(std::max(1, b->num_keys)))));
        const int64_t most = std::min({fit, 32 * words, int64_t(kRowsMaxQueries)});
        p->chunk = (int32_t)std::min<int64_t>(b->num_queries, most > 148 ? most / 148 * 148 : std::max<int64_t>(1, most));
        p->words = (p->chunk + 31) / 32;
        p->part = c.take<float>(size_t(p->chunk) * row * b->head_dim);
        p->bits = c.take<uint32_t>(size_t(p->words) * b->num_keys);
        p->pre = c.take<uint16_t>(size_t(p->words) * b->num_keys);
        p->count = c.take<uint32_t>(b->num_keys);
        p->off = c.take<uint32_t>(b->num_keys);
        p->base = c.take<uint32_t>((b->num_keys + kPosBlock - 1) / kPosBlock);
        if (p->chunk < b->num_queries) p->acc = c.take<float>(size_t(b->num_keys) * b->head_dim);
        return c.off;
    }
    p->edge = c.take<uint16_t>(size_t(p->key_blocks + 1) * std::max(1, b->num_queries));
    if (p->parts > 1) p->part = c.take<float>(size_t(p->parts) * b->num_keys * b->head_dim);
    return c.off;
}

dsa_status list_check(const dsa_batch* b, HostInfo* hi, int32_t k)
{
    dsa_status s = check_batch(b, hi);
    if (s != DSA_OK) return s;
    return k < 1 || k > kMaxK ? DSA_ERR_UNSUPPORTED : DSA_OK;
}

ListArgs list_args(const dsa_batch* b, const void* Q, const void* K, const float* W, int32_t k, const int32_t* lists,
                   const ListPlan& p, void* ws)
{
    ListArgs a{};
    a.rows = p.rows;
    a.Q = static_cast<const __nv_bfloat16*>(Q);
    a.K = static_cast<const __nv_bfloat16*>(K);
    a.W = W;
    a.lists = lists;
    a.q_off = b->q_offsets;
    a.k_off = b->k_offsets;
    a.status = static_cast<uint32_t*>(ws);
    a.n_seqs = b->num_seqs;
    a.n_q = b->num_queries;
    a.n_k = b->num_keys;
    a.H = b->num_heads;
    a.k = k;
    return a;
}

// The usable lists; with edges also the list places at the borders of the key blocks.
dsa_status list_rows(const dsa_batch* b, int32_t k, const int32_t* lists, const ListPlan& p, bool edges, void* ws,
                     cudaStream_t st)
{
    dsa_status s = clear_status(ws, st);
    if (s != DSA_OK || b->num_queries == 0) return s;
    const int32_t quads = k % 4 == 0 && (reinterpret_cast<uintptr_t>(lists) & 15) == 0;
    DSA_LAUNCH(kProfSetup, st, list_rows_kernel<<<(b->num_queries + 7) / 8, 256, 0, st>>>(
        lists, k, quads, b->q_offsets, b->k_offsets, b->q_pos, b->num_seqs, b->num_queries, p.rows,
        edges ? p.edge : nullptr, p.key_blocks, static_cast<uint32_t*>(ws)));
    return launched();
}

constexpr int kSmemMax = 232448;   // dynamic shared memory of one CTA

template <int D, int HP, int MODE>
dsa_status list_tc_launch(const ListArgs& l, int32_t t0, int32_t t1, const ListPlan& p, cudaStream_t st)
{
    using SH = ListShape<D, HP>;
    CUtensorMap mq;
    if (!make_tile_map(&mq, l.Q, int64_t(l.n_q) * l.H, D, l.H)) return DSA_ERR_CUDA;
    // few queries: several CTAs each, as many as fill the GPU once and find at least two tiles
    const int splits = MODE == kListScores ? std::max(1, std::min(148 / (t1 - t0), (l.k + 255) / 256)) : 1;
    const ListTcArgs a{l, std::min(8, int((kSmemMax - SH::bytes(0, MODE == kListGradRows)) / SH::KTILE)), t0, t1, splits,
                       p.part, p.bits, p.pre, p.off, p.base};
    const int smem = std::max<int>(SH::bytes(a.n_stages, MODE == kListGradRows), 120 * 1024);   // one CTA an SM
    dsa_status s = set_smem(list_tc_kernel<D, HP, MODE>, smem);
    if (s != DSA_OK) return s;
    DSA_LAUNCH(MODE ? kProfListDq : kProfListScores, st,
               launch_pdl(true, list_tc_kernel<D, HP, MODE>, std::min((t1 - t0) * splits, 148), list_threads(MODE), smem, st, mq, a));
    return launched();
}

template <int D, int MODE>
dsa_status list_tc(const ListArgs& a, int32_t t0, int32_t t1, const ListPlan& p, cudaStream_t st)
{
    if (a.H <= 16) return list_tc_launch<D, 16, MODE>(a, t0, t1, p, st);
    if (a.H <= 32) return list_tc_launch<D, 32, MODE>(a, t0, t1, p, st);
    return list_tc_launch<D, 64, MODE>(a, t0, t1, p, st);
}

template <int D>
dsa_status list_scores_d(const ListArgs& a, const ListPlan& p, cudaStream_t st)
{
    return list_tc<D, kListScores>(a, 0, a.n_q, p, st);
}

template <int D, int H>
dsa_status list_dk_launch(const ListArgs& l, const ListPlan& p, cudaStream_t st)
{
    using SH = DkShape<D, H>;
    CUtensorMap mk;
    if (!make_tile_map(&mk, l.K, l.n_k, D, 128)) return DSA_ERR_CUDA;
    const DkArgs a{l, p.edge, p.part, p.parts};
    const int smem = std::max<int>(SH::bytes, 120 * 1024);   // one CTA an SM: each takes all of TMEM
    dsa_status s = set_smem(list_dk_tc_kernel<D, H>, smem);
    if (s != DSA_OK) return s;
    DSA_LAUNCH(kProfListDk, st, launch_pdl(true, list_dk_tc_kernel<D, H>, (unsigned)p.units * p.parts, kDkThreads, smem, st, mk, a));
    if ((s = launched()) != DSA_OK || p.parts == 1) return s;
    const int64_t n4 = int64_t(l.n_k) * D / 4;
    DSA_LAUNCH(kProfListDk, st, launch_pdl(true, list_dk_join_kernel, (unsigned)((n4 + 255) / 256), 256, 0, st,
                                           reinterpret_cast<const float4*>(p.part), p.parts, n4,
                                           reinterpret_cast<uint2*>(l.dK)));
    return launched();
}

template <int D>
dsa_status list_dk(const ListArgs& a, const ListPlan& p, cudaStream_t st)
{
    switch (a.H) {
    case 1: return list_dk_launch<D, 1>(a, p, st);
    case 2: return list_dk_launch<D, 2>(a, p, st);
    case 4: return list_dk_launch<D, 4>(a, p, st);
    case 8: return list_dk_launch<D, 8>(a, p, st);
    case 16: return list_dk_launch<D, 16>(a, p, st);
    case 32: return list_dk_launch<D, 32>(a, p, st);
    default: return list_dk_launch<D, 64>(a, p, st);
    }
}

template <int D>
dsa_status list_backward_d(const ListArgs& a, const ListPlan& p, cudaStream_t st)
{
    dsa_status s;
    const bool want_k = a.n_k > 0 && a.dK;
    if (a.n_q == 0)   // nothing lists a key
        return !want_k || cudaMemsetAsync(a.dK, 0, size_t(a.n_k) * D * 2, st) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
    if (!want_k || !p.by_rows) {
        if ((a.dQ || a.dW) && (s = list_tc<D, kListGrad>(a, 0, a.n_q, p, st)) != DSA_OK) return s;
        return want_k ? list_dk<D>(a, p, st) : DSA_OK;
    }
    for (int32_t t0 = 0; t0 < a.n_q; t0 += p.chunk) {
        const int32_t t1 = std::min(t0 + p.chunk, a.n_q), words = (t1 - t0 + 31) / 32;
        const int32_t blocks = (a.n_k + kPosBlock - 1) / kPosBlock;
        if (cudaMemsetAsync(p.bits, 0, size_t(words) * a.n_k * 4, st) != cudaSuccess) return DSA_ERR_CUDA;
        const dim3 marks((t1 - t0 + 7) / 8, (a.k + kBitsPlaces - 1) / kBitsPlaces);
        DSA_LAUNCH(kProfSetup, st, list_bits_kernel<<<marks, 256, 0, st>>>(a.lists, a.k, a.rows, a.k_off, t0, t1, a.n_k,
                                                                           p.bits, a.status));
        DSA_LAUNCH(kProfSetup, st, list_count_kernel<<<blocks, kPosBlock, 0, st>>>(p.bits, words, a.n_k, p.pre, p.count,
                                                                                  p.off, p.base));
        DSA_LAUNCH(kProfSetup, st, list_base_kernel<<<1, 1024, 0, st>>>(p.base, blocks));
        if ((s = launched()) != DSA_OK) return s;
        if ((s = list_tc<D, kListGradRows>(a, t0, t1, p, st)) != DSA_OK) return s;
        const DkRowsArgs r{p.part, p.count, p.off, p.base, p.acc, a.dK, a.n_k, t0 == 0, t1 == a.n_q};
        DSA_LAUNCH(kProfListDk, st, launch_pdl(true, list_dk_rows_kernel<D>, (a.n_k + kRowsWarps - 1) / kRowsWarps,
                                               kRowsWarps * 32, 0, st, r));
        if ((s = launched()) != DSA_OK) return s;
    }
    return DSA_OK;
}

}  // namespace

extern "C" {

// ------------------------------------------------------------- layer norm
dsa_status dsa_layer_norm(int64_t n, int32_t d, const void* x, int32_t x_type, int64_t ld_x, const float* weight,
                          const float* bias, float eps, void* y, int32_t y_type, int64_t ld_y, float* mean,
                          float* rstd, void* stream)
{
    if (n < 0 || d < 1 || !(eps >= 0.f)) return DSA_ERR_INVALID_ARG;
    if (d > kNormMaxWidth) return DSA_ERR_UNSUPPORTED;
    dsa_status s;
    if ((s = check_rows(x, x_type, ld_x, n, d)) != DSA_OK) return s;
    if ((s = check_rows(y, y_type, ld_y, n, d)) != DSA_OK) return s;
    if ((reinterpret_cast<uintptr_t>(weight) | reinterpret_cast<uintptr_t>(bias) | reinterpret_cast<uintptr_t>(mean) |
         reinterpret_cast<uintptr_t>(rstd)) & 3)
        return DSA_ERR_INVALID_ARG;
    if (n == 0) return DSA_OK;
    NormArgs a{};
    a.x = x; a.ld_x = ld_x; a.out = y; a.ld_out = ld_y; a.w = weight; a.b = bias;
    a.mean = mean; a.rstd = rstd; a.n = n; a.d = d; a.eps = eps;
    const bool vec = d % 8 == 0 && rows_aligned(x, x_type, ld_x, n) && rows_aligned(y, y_type, ld_y, n) &&
                     ((reinterpret_cast<uintptr_t>(weight) | reinterpret_cast<uintptr_t>(bias)) & 15) == 0;
    int32_t unused = 0;
    return norm_dispatch(a, x_type, y_type, vec, false, &unused, static_cast<cudaStream_t>(stream));
}

size_t dsa_layer_norm_backward_workspace(int64_t n, int32_t d)
{
    if (n < 0 || d < 1 || d > kNormMaxWidth) return 0;
    return norm_ws_bytes(n, d);
}

dsa_status dsa_layer_norm_backward(int64_t n, int32_t d, const void* dy, int32_t dy_type, int64_t ld_dy,
                                   const void* x, int32_t x_type, int64_t ld_x, const float* weight,
                                   const float* mean, const float* rstd, void* dx, int64_t ld_dx, float* dweight,
                                   float* dbias, void* ws, size_t ws_bytes, void* stream)
{
    if (n < 0 || d < 1) return DSA_ERR_INVALID_ARG;
    if (d > kNormMaxWidth) return DSA_ERR_UNSUPPORTED;
    dsa_status s;
    if ((s = check_rows(dy, dy_type, ld_dy, n, d)) != DSA_OK) return s;
    if ((s = check_rows(x, x_type, ld_x, n, d)) != DSA_OK) return s;
    if (dx && (s = check_rows(dx, x_type, ld_dx, n, d)) != DSA_OK) return s;
    if (n > 0 && (!mean || !rstd)) return DSA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(weight) | reinterpret_cast<uintptr_t>(mean) | reinterpret_cast<uintptr_t>(rstd) |
         reinterpret_cast<uintptr_t>(dweight) | reinterpret_cast<uintptr_t>(dbias)) & 3)
        return DSA_ERR_INVALID_ARG;
    if ((s = check_ws(ws, ws_bytes, norm_ws_bytes(n, d))) != DSA_OK) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // no sums, whose kernel clears the status otherwise
    if ((n == 0 || (!dweight && !dbias)) && cudaMemsetAsync(ws, 0, kStatusBytes, st) != cudaSuccess) return DSA_ERR_CUDA;
    if (n == 0) {   // sums over no rows
        if ((dweight && cudaMemsetAsync(dweight, 0, size_t(d) * 4, st) != cudaSuccess) ||
            (dbias && cudaMemsetAsync(dbias, 0, size_t(d) * 4, st) != cudaSuccess))
            return DSA_ERR_CUDA;
        return DSA_OK;
    }
    if (!dx && !dweight && !dbias) return DSA_OK;
    Carver c{static_cast<char*>(ws)};
    NormArgs a{};
    a.x = x; a.ld_x = ld_x; a.dy = dy; a.ld_dy = ld_dy; a.out = dx; a.ld_out = ld_dx; a.w = weight;
    a.mean_in = mean; a.rstd_in = rstd; a.n = n; a.d = d;
    a.part = dweight || dbias ? c.take<float>(norm_part_floats(n, d)) : nullptr;
    const bool vec = d % 8 == 0 && rows_aligned(x, x_type, ld_x, n) && rows_aligned(dy, dy_type, ld_dy, n) &&
                     (!dx || rows_aligned(dx, x_type, ld_dx, n)) && (reinterpret_cast<uintptr_t>(weight) & 15) == 0;
    int32_t n_part = 0;
    if ((s = norm_dispatch(a, x_type, dy_type, vec, true, &n_part, st)) != DSA_OK || !a.part) return s;
    DSA_LAUNCH(kProfNorm, st, launch_pdl(true, layer_norm_dw_kernel, (2 * d + 31) / 32, 1024, 0, st,
                                         (const float*)a.part, n_part, d, dweight, dbias, static_cast<uint32_t*>(ws)));
    return launched();
}

// ------------------------------------------------------------ distillation
dsa_status dsa_distill_topk(int32_t n, int32_t k, const float* scores, int64_t ld_scores, const int32_t* lists,
                            int64_t ld_lists, const void* teacher, int32_t teacher_type, int64_t ld_teacher,
                            int32_t teacher_kind, float temperature, const float* grad_loss, float* loss,
                            float* dscores, int64_t ld_dscores, void* stream)
{
    if (n < 0 || k < 1 || !(temperature >= kMinTemperature && temperature <= kMaxTemperature)) return DSA_ERR_INVALID_ARG;
    if (teacher_kind != DSA_TEACHER_LOGITS && teacher_kind != DSA_TEACHER_WEIGHTS) return DSA_ERR_INVALID_ARG;
    dsa_status s;
    if ((s = check_rows(scores, DSA_FP32, ld_scores, n, k)) != DSA_OK) return s;
    if ((s = check_rows(teacher, teacher_type, ld_teacher, n, k)) != DSA_OK) return s;
    if (lists && (s = check_rows(lists, DSA_FP32, ld_lists, n, k)) != DSA_OK) return s;
    if (dscores && (s = check_rows(dscores, DSA_FP32, ld_dscores, n, k)) != DSA_OK) return s;
    if ((reinterpret_cast<uintptr_t>(grad_loss) | reinterpret_cast<uintptr_t>(loss)) & 3) return DSA_ERR_INVALID_ARG;
    if (n == 0 || (!loss && !dscores)) return DSA_OK;
    DistillArgs a{};
    a.s = scores; a.ld_s = ld_scores; a.list = lists; a.ld_list = ld_lists; a.t = teacher; a.ld_t = ld_teacher;
    a.g = grad_loss; a.loss = loss; a.ds = dscores; a.ld_ds = ld_dscores; a.n = n; a.k = k;
    a.inv_tau = 1.f / temperature;
    a.scale = (float)(1.4426950408889634 * kDistillUnit / (double)temperature);
    a.unit_log2 = (float)(0.69314718055994531 / kDistillUnit * (double)temperature);
    // four places a load where the arrays' rows lie alike against 4-place boundaries
    const auto place = [](const void* p, int64_t size) { return int32_t(reinterpret_cast<uintptr_t>(p) / size % 4); };
    a.off0 = place(scores, 4);
    a.off_step = int32_t(ld_scores % 4);
    const auto alike = [&](const void* p, int64_t size, int64_t ld) {
        return !p || (place(p, size) == a.off0 && (n == 1 || int32_t(ld % 4) == a.off_step));
    };
    const bool vec = alike(teacher, type_size(teacher_type), ld_teacher) && alike(lists, 4, ld_lists) &&
                     alike(dscores, 4, ld_dscores);
    const bool edge = k % 4 != 0 || a.off0 != 0 || (n > 1 && a.off_step != 0);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool weights = teacher_kind == DSA_TEACHER_WEIGHTS;
    if (teacher_type == DSA_FP32)
        return weights ? distill_rows<float, true>(a, vec, edge, st) : distill_rows<float, false>(a, vec, edge, st);
    return weights ? distill_rows<__nv_bfloat16, true>(a, vec, edge, st)
                   : distill_rows<__nv_bfloat16, false>(a, vec, edge, st);
}

// ----------------------------------------------------- scores at listed keys
size_t dsa_list_scores_workspace(const dsa_batch* b, int32_t k)
{
    HostInfo hi;
    ListPlan p;
    return list_check(b, &hi, k) == DSA_OK ? list_plan(nullptr, b, hi, k, false, &p) : 0;
}

dsa_status dsa_list_scores(const dsa_batch* b, const void* Q, const void* K, const float* W, int32_t k,
                           const int32_t* lists, float* scores, void* ws, size_t ws_bytes, void* stream)
{
    HostInfo hi;
    dsa_status s = list_check(b, &hi, k);
    if (s != DSA_OK) return s;
    if ((s = check_tensors(b, Q, K, W)) != DSA_OK) return s;
    if (b->num_queries > 0 && (!lists || !scores)) return DSA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(lists) | reinterpret_cast<uintptr_t>(scores)) & 3) return DSA_ERR_INVALID_ARG;
    ListPlan p;
    if ((s = check_ws(ws, ws_bytes, list_plan(nullptr, b, hi, k, false, &p))) != DSA_OK) return s;
    list_plan(static_cast<char*>(ws), b, hi, k, false, &p);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (p.picking) {
        uint32_t* status = static_cast<uint32_t*>(ws);
        if ((s = clear_status(ws, st)) != DSA_OK) return s;
        if ((s = dense_scores(b, hi, Q, K, W, p.S, p.dense, status, st)) != DSA_OK) return s;
        const bool quads = k % 4 == 0 && ((reinterpret_cast<uintptr_t>(lists) | reinterpret_cast<uintptr_t>(scores)) & 15) == 0;
        const auto pick = quads ? list_pick_kernel<4> : list_pick_kernel<1>;
        DSA_LAUNCH(kProfListScores, st, pick<<<(b->num_queries + 7) / 8, 256, 0, st>>>(
            lists, k, b->q_offsets, b->k_offsets, b->q_pos, b->num_seqs, b->num_queries, p.S, dense_scores_ld(hi.max_k),
            scores, status));
        return launched();
    }
    if ((s = list_rows(b, k, lists, p, false, ws, st)) != DSA_OK || b->num_queries == 0) return s;
    ListArgs a = list_args(b, Q, K, W, k, lists, p, ws);
    a.scores = scores;
    switch (b->head_dim) {
    case 32: return list_scores_d<32>(a, p, st);
    case 64: return list_scores_d<64>(a, p, st);
    default: return list_scores_d<128>(a, p, st);
    }
}

size_t dsa_list_scores_backward_workspace(const dsa_batch* b, int32_t k)
{
    HostInfo hi;
    ListPlan p;
    return list_check(b, &hi, k) == DSA_OK ? list_plan(nullptr, b, hi, k, true, &p) : 0;
}

dsa_status dsa_list_scores_backward(const dsa_batch* b, const void* Q, const void* K, const float* W, int32_t k,
                                    const int32_t* lists, const float* dscores, void* dQ, void* dK, float* dW,
                                    void* ws, size_t ws_bytes, void* stream)
{
    HostInfo hi;
    dsa_status s = list_check(b, &hi, k);
    if (s != DSA_OK) return s;
    if ((s = check_tensors(b, Q, K, W)) != DSA_OK) return s;
    if (b->num_queries > 0 && (!lists || !dscores)) return DSA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(lists) | reinterpret_cast<uintptr_t>(dscores) | reinterpret_cast<uintptr_t>(dW)) & 3)
        return DSA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(dQ) | reinterpret_cast<uintptr_t>(dK)) & 15) return DSA_ERR_INVALID_ARG;
    ListPlan p;
    if ((s = check_ws(ws, ws_bytes, list_plan(nullptr, b, hi, k, true, &p))) != DSA_OK) return s;
    list_plan(static_cast<char*>(ws), b, hi, k, true, &p);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if ((s = list_rows(b, k, lists, p, dK != nullptr && !p.by_rows, ws, st)) != DSA_OK) return s;
    ListArgs a = list_args(b, Q, K, W, k, lists, p, ws);
    a.ds = dscores;
    a.dQ = static_cast<__nv_bfloat16*>(dQ);
    a.dK = static_cast<__nv_bfloat16*>(dK);
    a.dW = dW;
    switch (b->head_dim) {
    case 32: return list_backward_d<32>(a, p, st);
    case 64: return list_backward_d<64>(a, p, st);
    default: return list_backward_d<128>(a, p, st);
    }
}

}  // extern "C"
