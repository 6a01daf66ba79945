// Distillation of listed scores from a teacher's top logits or weights: the loss and its gradient in
// one pass over the rows.
//
// Row with student scores s_j, teacher values t_j, temperature tau; counted places C = those whose
// list entry is not negative and whose s_j is above -inf.  Over C
//   q = softmax(s / tau);  p = softmax(t / tau) (logits) or t / sum t (weights);
//   loss = sum p (log p - log q);  ds_j = (g / tau) (q_j - p_j), 0 outside C.
// With a_j = (s_j - max s) / tau, z = sum e^a, and the teacher's unnormalised weights f_j with
// logarithm c_j (c_j = (t_j - max t) / tau, f = e^c; or f = t, c = log t) and y = sum f:
//   loss = (sum f (c - a)) / y + log z - log y,
// so two joint reductions over the row (the maxima, then z, y and the cross sum) give everything.
// Bound by memory: a row is read once into registers and its gradient written once.  Rows longer
// than the registers of a CTA hold (kDistillRegCols) are swept three times, the later sweeps from L2.
#pragma once

#include <math_constants.h>

#include "common.cuh"

namespace dsa {

constexpr int kDistillRegCols = 16384;

struct DistillArgs {
    const float* s;
    int64_t ld_s;
    const int32_t* list;   // NULL: every place whose score is above -inf counts
    int64_t ld_list;
    const void* t;
    int64_t ld_t;
    const float* g;        // NULL: ones
    float* loss;           // NULL: not written
    float* ds;             // NULL: not written
    int64_t ld_ds;
    int32_t n, k;
    int32_t weights;       // the teacher's values: 0 logits, 1 weights
    float inv_tau;
};

template <int VEC>
__device__ __forceinline__ void distill_load(const float* p, float* v)
{
    if constexpr (VEC == 4) {
        const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    } else {
        v[0] = __ldcs(p);
    }
}

template <int VEC>
__device__ __forceinline__ void distill_load(const __nv_bfloat16* p, float* v)
{
    if constexpr (VEC == 4) {
        const uint2 a = __ldcs(reinterpret_cast<const uint2*>(p));
        v[0] = __uint_as_float(a.x << 16); v[1] = __uint_as_float(a.x & 0xffff0000u);
        v[2] = __uint_as_float(a.y << 16); v[3] = __uint_as_float(a.y & 0xffff0000u);
    } else {
        v[0] = __bfloat162float(*p);
    }
}

template <int VEC>
__device__ __forceinline__ void distill_load(const int32_t* p, int32_t* v)
{
    if constexpr (VEC == 4) {
        const int4 a = __ldcs(reinterpret_cast<const int4*>(p));
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    } else {
        v[0] = __ldcs(p);
    }
}

// Joint reductions over the T threads of a row: a warp's lanes (T = 32) or the whole CTA.
template <int T>
__device__ __forceinline__ void distill_max2(float& a, float& b, float4* red)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, o));
    }
    if constexpr (T > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float4(a, b, 0.f, 0.f);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < T / 32; ++i) {
            a = fmaxf(a, red[i].x);
            b = fmaxf(b, red[i].y);
        }
    }
}

template <int T>
__device__ __forceinline__ void distill_sum3(float& a, float& b, float& c, float4* red)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
        c += __shfl_xor_sync(0xffffffffu, c, o);
    }
    if constexpr (T > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float4(a, b, c, 0.f);
        __syncthreads();
        a = b = c = 0.f;
#pragma unroll
        for (int i = 0; i < T / 32; ++i) {
            const float4 v = red[i];
            a += v.x;
            b += v.y;
            c += v.z;
        }
    }
}

// The teacher's unnormalised weight of a counted place and the logarithm that goes with it.
__device__ __forceinline__ float distill_weight(float t, float mt, const DistillArgs& a, float& c)
{
    if (a.weights) {
        c = logf(t);
        return t;
    }
    c = (t - mt) * a.inv_tau;
    return expf(c);
}

// What a row's sums say: the loss, and the factors of e^a and f in the gradient.
struct DistillRow {
    float loss, cs, ct;
};

__device__ __forceinline__ DistillRow distill_row(float z, float y, float x, float g, const DistillArgs& a)
{
    DistillRow r{0.f, 0.f, 0.f};
    if (y == 0.f || z == 0.f) return r;   // no counted place, or none that the teacher weighs: nothing to learn
    r.loss = x / y + (logf(z) - logf(y));
    r.cs = g * a.inv_tau / z;
    r.ct = g * a.inv_tau / y;
    return r;
}

// One row per group of T threads (T = 32: NT / 32 rows per CTA; else T == NT), in registers.
template <typename TT, int VEC, int T, int NV, int NT>
__global__ void __launch_bounds__(NT) distill_kernel(const __grid_constant__ DistillArgs a)
{
    __shared__ float4 red1[32], red2[32];
    const int t = threadIdx.x % T;
    const int row = blockIdx.x * (NT / T) + threadIdx.x / T;
    if (row >= a.n) return;   // whole warps (T = 32) or whole CTAs
    const float* sp = a.s + (int64_t)row * a.ld_s;
    const TT* tp = static_cast<const TT*>(a.t) + (int64_t)row * a.ld_t;
    const int32_t* lp = a.list ? a.list + (int64_t)row * a.ld_list : nullptr;
    float s[NV][VEC], f[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * T + t) * VEC;
        if (c < a.k) {
            distill_load<VEC>(sp + c, s[i]);
            distill_load<VEC>(tp + c, f[i]);
            if (lp) {
                int32_t l[VEC];
                distill_load<VEC>(lp + c, l);
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (l[e] < 0) s[i][e] = -CUDART_INF_F;
            }
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) s[i][e] = -CUDART_INF_F;
        }
    }
    float ms = -CUDART_INF_F, mt = -CUDART_INF_F;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            if (s[i][e] == -CUDART_INF_F) f[i][e] = a.weights ? 0.f : -CUDART_INF_F;   // not counted: no value either
            ms = fmaxf(ms, s[i][e]);
            mt = fmaxf(mt, f[i][e]);
        }
    distill_max2<T>(ms, mt, red1);
    float z = 0.f, y = 0.f, x = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const bool in = s[i][e] != -CUDART_INF_F;
            const float d = (s[i][e] - ms) * a.inv_tau;
            s[i][e] = in ? expf(d) : 0.f;
            z += s[i][e];
            float c = 0.f, w = 0.f;
            if (in && mt != -CUDART_INF_F) w = distill_weight(f[i][e], mt, a, c);
            f[i][e] = w;
            y += w;
            if (w != 0.f) x = fmaf(w, c - d, x);
        }
    distill_sum3<T>(z, y, x, red2);
    const DistillRow r = distill_row(z, y, x, a.g ? a.g[row] : 1.f, a);
    if (t == 0 && a.loss) a.loss[row] = r.loss;
    if (!a.ds) return;
    float* dp = a.ds + (int64_t)row * a.ld_ds;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * T + t) * VEC;
        if (c >= a.k) continue;
        float v[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e)   // 0 where neither has weight, whatever a NaN elsewhere made of the factors
            v[e] = s[i][e] == 0.f && f[i][e] == 0.f ? 0.f : s[i][e] * r.cs - f[i][e] * r.ct;
        if constexpr (VEC == 4)
            *reinterpret_cast<float4*>(dp + c) = make_float4(v[0], v[1], v[2], v[3]);
        else
            dp[c] = v[0];
    }
}

// Rows of any length: one CTA per row, three sweeps (maxima, sums, gradient).
template <typename TT, int NT>
__global__ void __launch_bounds__(NT) distill_long_kernel(const __grid_constant__ DistillArgs a)
{
    __shared__ float4 red1[32], red2[32];
    const int row = blockIdx.x;
    const float* sp = a.s + (int64_t)row * a.ld_s;
    const TT* tp = static_cast<const TT*>(a.t) + (int64_t)row * a.ld_t;
    const int32_t* lp = a.list ? a.list + (int64_t)row * a.ld_list : nullptr;
    auto score = [&](int c) { return lp && lp[c] < 0 ? -CUDART_INF_F : sp[c]; };
    auto teacher = [&](int c) {
        if constexpr (sizeof(TT) == 2) return __bfloat162float(tp[c]);
        else return (float)tp[c];
    };
    float ms = -CUDART_INF_F, mt = -CUDART_INF_F;
#pragma unroll 4
    for (int c = threadIdx.x; c < a.k; c += NT) {
        const float s = score(c);
        const float v = teacher(c);
        ms = fmaxf(ms, s);
        if (s != -CUDART_INF_F) mt = fmaxf(mt, v);
    }
    distill_max2<NT>(ms, mt, red1);
    float z = 0.f, y = 0.f, x = 0.f;
#pragma unroll 4
    for (int c = threadIdx.x; c < a.k; c += NT) {
        const float s = score(c);
        const float v = teacher(c);
        if (s == -CUDART_INF_F) continue;
        const float d = (s - ms) * a.inv_tau;
        z += expf(d);
        if (mt == -CUDART_INF_F) continue;
        float lg;
        const float w = distill_weight(v, mt, a, lg);
        y += w;
        if (w != 0.f) x = fmaf(w, lg - d, x);
    }
    distill_sum3<NT>(z, y, x, red2);
    const DistillRow r = distill_row(z, y, x, a.g ? a.g[row] : 1.f, a);
    if (threadIdx.x == 0 && a.loss) a.loss[row] = r.loss;
    if (!a.ds) return;
    float* dp = a.ds + (int64_t)row * a.ld_ds;
#pragma unroll 4
    for (int c = threadIdx.x; c < a.k; c += NT) {
        const float s = score(c);
        const float v = teacher(c);
        float lg, out = 0.f;
        if (s != -CUDART_INF_F && mt != -CUDART_INF_F)
            out = expf((s - ms) * a.inv_tau) * r.cs - distill_weight(v, mt, a, lg) * r.ct;
        dp[c] = out;
    }
}

}  // namespace dsa
