// Host side shared by the library's translation units: argument checks, the
// workspace carve-out, launch helpers, launch accounting and tensor maps.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <mutex>
#include <vector>

#include "../../include/dsa_index.h"
#include "common.cuh"

namespace dsa {

constexpr int32_t kMaxK = 16384;

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Workspace header: the status word (kStatusBytes), then two counters per row of the split-row
// select (kSplitMaxRows rows).  Each call clears the header once before its first launch.
constexpr int32_t kSplitMaxRows = 512;
constexpr size_t kHeaderBytes = kStatusBytes + size_t(kSplitMaxRows) * 2 * sizeof(uint32_t);

// Sequential carve-out of a workspace; a dry run (base == nullptr) sizes it.
struct Carver {
    char* base;
    size_t off = kHeaderBytes;
    template <typename T>
    T* take(size_t count)
    {
        T* p = base ? reinterpret_cast<T*>(base + off) : nullptr;
        off = align256(off + count * sizeof(T));
        return p;
    }
};

inline bool head_dim_ok(int d) { return d == 32 || d == 64 || d == 128; }
inline bool heads_ok(int h) { return h >= 1 && h <= 64 && (h & (h - 1)) == 0; }

struct HostInfo {
    int32_t max_q = 0;   // longest query run of a sequence
    int32_t max_k = 0;   // longest key run of a sequence
};

inline dsa_status check_batch(const dsa_batch* b, HostInfo* info)
{
    if (!b) return DSA_ERR_INVALID_ARG;
    if (b->num_seqs < 1 || b->num_queries < 0 || b->num_keys < 0) return DSA_ERR_INVALID_ARG;
    if (!heads_ok(b->num_heads) || !head_dim_ok(b->head_dim)) return DSA_ERR_UNSUPPORTED;
    if (!b->q_offsets || !b->k_offsets || !b->q_offsets_host || !b->k_offsets_host)
        return DSA_ERR_INVALID_ARG;
    if (b->num_queries > 0 && !b->q_pos) return DSA_ERR_INVALID_ARG;
    const int32_t* qo = b->q_offsets_host;
    const int32_t* ko = b->k_offsets_host;
    if (qo[0] != 0 || ko[0] != 0) return DSA_ERR_INVALID_ARG;
    for (int i = 0; i < b->num_seqs; ++i) {
        if (qo[i + 1] < qo[i] || ko[i + 1] < ko[i]) return DSA_ERR_INVALID_ARG;
        info->max_q = std::max(info->max_q, qo[i + 1] - qo[i]);
        info->max_k = std::max(info->max_k, ko[i + 1] - ko[i]);
    }
    if (qo[b->num_seqs] != b->num_queries || ko[b->num_seqs] != b->num_keys) return DSA_ERR_INVALID_ARG;
    return DSA_OK;
}

inline dsa_status check_tensors(const dsa_batch* b, const void* Q, const void* K, const float* W)
{
    if (b->num_queries > 0 && (!Q || !W)) return DSA_ERR_INVALID_ARG;
    if (b->num_keys > 0 && !K) return DSA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(Q) | reinterpret_cast<uintptr_t>(K)) & 15) return DSA_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(W) & 3) return DSA_ERR_INVALID_ARG;
    return DSA_OK;
}

inline dsa_status check_ws(void* ws, size_t ws_bytes, size_t need)
{
    if (!ws || ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & 255)) return DSA_ERR_WORKSPACE;
    return DSA_OK;
}

// The status word of the entry point running on this host thread: select launches hand it to their
// kernels (checked builds record index errors there).  Set by every entry point before its launches.
inline thread_local uint32_t* g_status = nullptr;

inline dsa_status launched()
{
    return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

// Launches a kernel, with programmatic stream serialization when `pdl`: it may then be
// scheduled while the previous kernel on the stream still runs, and must call grid_dep_wait()
// before it touches memory an earlier kernel writes or reads.
template <typename... KArgs, typename... Args>
void launch_pdl(bool pdl, void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                Args... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    (void)cudaLaunchKernelEx(&cfg, kern, args...);   // errors surface through launched()
}

// Launches a kernel as clusters of `cluster` CTAs along x (with programmatic stream
// serialization, as launch_pdl).
template <typename... KArgs, typename... Args>
void launch_clustered(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, int cluster, cudaStream_t st,
                      Args... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    (void)cudaLaunchKernelEx(&cfg, kern, args...);   // errors surface through launched()
}

// Programmatic launch pays off for the short kernels of decode (it hides each launch's latency
// behind the previous kernel) and cost the multi-wave prefill kernels ~4% when measured, so it
// is used when the grids involved fit in about two waves.
inline bool latency_bound(int64_t ctas) { return ctas <= 2 * 148; }

// ------------------------------------------------------------- profiling
// Kernel kinds timed by the optional profiler (dsa_profile_*).
enum ProfKind : int32_t {
    kProfSetup = 0, kProfScoreSimt, kProfSelect, kProfPool, kProfProxy, kProfScoreTc, kProfFill, kProfNorm,
    kProfDistill, kProfListScores, kProfListDq, kProfListDk, kProfKinds
};
inline const char* const kProfNames[kProfKinds] = {"setup", "score_simt", "select_topk", "hisa_pool", "pivot_proxy",
                                            "score_tc", "fill", "layer_norm", "distill", "list_scores", "list_dq", "list_dk"};

struct ProfRec {
    int32_t kind;
    cudaEvent_t start, stop;
};
inline std::mutex g_prof_mu;
inline std::atomic<bool> g_prof_on{false};
inline std::vector<ProfRec> g_prof;
inline std::atomic<uint64_t> g_launches{0};

#define DSA_LAUNCH(kind, st, ...)      \
    do {                               \
        LaunchScope _ls((kind), (st)); \
        __VA_ARGS__;                   \
    } while (0)

// Counts one kernel launch; when profiling is on, brackets it with events on its stream.
struct LaunchScope {
    int32_t kind;
    cudaStream_t st;
    cudaEvent_t start = nullptr;
    LaunchScope(int32_t k, cudaStream_t s) : kind(k), st(s)
    {
        g_launches.fetch_add(1, std::memory_order_relaxed);
        if (g_prof_on.load(std::memory_order_relaxed) && cudaEventCreate(&start) == cudaSuccess)
            cudaEventRecord(start, st);
    }
    ~LaunchScope()
    {
        if (!start) return;
        cudaEvent_t stop;
        if (cudaEventCreate(&stop) != cudaSuccess) { cudaEventDestroy(start); return; }
        cudaEventRecord(stop, st);
        std::lock_guard<std::mutex> lk(g_prof_mu);
        g_prof.push_back(ProfRec{kind, start, stop});
    }
};

template <typename Kern>
dsa_status set_smem(Kern kern, size_t smem)
{
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) == cudaSuccess
               ? DSA_OK
               : DSA_ERR_CUDA;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled from the driver, found through the runtime (no link against libcuda).
inline EncodeTiledFn encode_tiled()
{
    static std::once_flag once;
    static EncodeTiledFn fn = nullptr;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// Tensor map of a row-major [rows, D] bf16 matrix, loaded in boxes of box_rows
// rows x (64 or 128 bytes) with the matching shared-memory swizzle; rows past
// the end read as zeros.
inline bool make_tile_map(CUtensorMap* m, const void* base, int64_t rows, int D, int box_rows)
{
    EncodeTiledFn enc = encode_tiled();
    if (!enc || rows <= 0 || rows > INT32_MAX) return false;
    const int row_bytes = D * 2 >= 128 ? 128 : 64;
    cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)D * 2};
    cuuint32_t box[2] = {(cuuint32_t)(row_bytes / 2), (cuuint32_t)box_rows};
    cuuint32_t elem[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, elem,
               CU_TENSOR_MAP_INTERLEAVE_NONE, row_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline dsa_status clear_status(void* ws, cudaStream_t st)
{
    g_status = static_cast<uint32_t*>(ws);
    return cudaMemsetAsync(ws, 0, kHeaderBytes, st) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

// Scores of every eligible key in one tensor-core launch, without filling the others (api.cu):
// S [n_q][dense_scores_ld] fp32; plan: dense_scores_plan_bytes of workspace, 256-byte aligned; status: the
// call's status word.
int64_t dense_scores_ld(int32_t max_k);
size_t dense_scores_plan_bytes(const dsa_batch* b, const HostInfo& hi);
dsa_status dense_scores(const dsa_batch* b, const HostInfo& hi, const void* Q, const void* K, const float* W, float* S,
                        char* plan, uint32_t* status, cudaStream_t st);

}  // namespace dsa
