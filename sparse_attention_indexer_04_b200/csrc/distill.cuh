// Distillation of listed scores from a teacher's top logits or weights: the loss and its gradient in
// one pass over the rows.
//
// Row with student scores s_j, teacher values t_j, temperature tau; counted places C = those whose
// list entry is not negative and whose s_j is above -inf.  Over C
//   q = softmax(s / tau);  p = softmax(t / tau) (logits) or t / sum t (weights);
//   loss = sum p (log p - log q);  ds_j = (g / tau) (q_j - p_j), 0 outside C.
// With a_j = (s_j - max s) / tau, z = sum e^a, and the teacher's unnormalised weights f_j with
// logarithm c_j (c_j = (t_j - max t) / tau, f = e^c; or f = t times the power of two that brings
// max t to 1 .. 2, c = log f: weights and their sum may lie below and above fp32's normal range) and y = sum f:
//   loss = (sum f (c - a)) / y + log z - log y,
// so two joint reductions over the row (the maxima, then z, y and the cross sum) give everything.
// Differences from the maxima are taken in units of 2^24 (exact, one fma each) and the cross sum is kept
// in those: a score masked with the type's lowest value is 3.4e38 below the maximum, which neither the
// factor log2(e) / tau nor a sum over millions of such places may carry past fp32.
// Bound by memory: a row is read once into registers and its gradient written once.  Exponentials
// are base 2, one multiply and one instruction each (with expf and logf the arithmetic took as long
// as the memory: 61.6 us for 8192 x 2048).  Rows that neither the registers of a CTA (kDistillRegCols) nor
// its shared memory hold are swept twice, the second time mostly from L2.
#pragma once

#include <math_constants.h>

#include <type_traits>

#include "common.cuh"

namespace dsa {

constexpr int kDistillRegCols = 20480;   // 1024 threads x 20 places, two values each in 64 registers

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
    float inv_tau;
    float scale;           // 2^24 log2(e) / tau: exponents are taken to base 2, of differences in units of 2^24
    float unit_log2;       // tau ln 2 / 2^24: a base-2 logarithm in those units
    int32_t off0, off_step; // VEC 4: row r starts (off0 + r * off_step) % 4 places behind a 4-place boundary
};

// Places c .. c + VEC - 1 of a row of k (VEC 4: p + c on a 4-element boundary); with EDGE places outside
// the row are not touched, else there are none.
template <int VEC, bool EDGE, typename X, typename V>
__device__ __forceinline__ void distill_load(const X* p, int c, int k, V* v)
{
    if (VEC == 4 && (!EDGE || (c >= 0 && c + 3 < k))) {
        if constexpr (sizeof(X) == 2) {
            const uint2 a = *reinterpret_cast<const uint2*>(p + c);
            v[0] = __uint_as_float(a.x << 16); v[1] = __uint_as_float(a.x & 0xffff0000u);
            v[2] = __uint_as_float(a.y << 16); v[3] = __uint_as_float(a.y & 0xffff0000u);
        } else if constexpr (sizeof(V) == sizeof(int32_t) && V(0.5f) == V(0)) {
            const int4 a = *reinterpret_cast<const int4*>(p + c);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        } else {
            const float4 a = *reinterpret_cast<const float4*>(p + c);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = !EDGE || (c + e >= 0 && c + e < k) ? (V)p[c + e] : V(0);
    }
}

template <int BYTES>
__device__ __forceinline__ void distill_copy(void* dst, const void* src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
                 "n"(BYTES)
                 : "memory");
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
        constexpr int NW = T / 32;
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float4(a, b, 0.f, 0.f);
        __syncthreads();
        const float4 v = red[threadIdx.x & (NW - 1)];
        a = v.x;
        b = v.y;
#pragma unroll
        for (int o = NW / 2; o > 0; o >>= 1) {
            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
            b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, o));
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
        constexpr int NW = T / 32;
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float4(a, b, c, 0.f);
        __syncthreads();
        const float4 v = red[threadIdx.x & (NW - 1)];
        a = v.x;
        b = v.y;
        c = v.z;
#pragma unroll
        for (int o = NW / 2; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
            c += __shfl_xor_sync(0xffffffffu, c, o);
        }
    }
}

// 2^x to about 2 units in the last place, log2 x to 2^-22 absolute around 1.
__device__ __forceinline__ float distill_exp2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float distill_log2(float x)
{
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What brings the largest weight m to 1 .. 2 (up to 4 from 2^127 on; a subnormal one to 2^-23 or more): a power of two.
__device__ __forceinline__ float distill_factor(float m)
{
    const int e = (__float_as_uint(m) >> 23) & 255;
    return __uint_as_float((uint32_t)max(254 - max(e, 1), 1) << 23);
}

constexpr float kDistillUnit = 16777216.f;   // 2^24

// x - max in units of 2^24; unit_max = -max / 2^24.
__device__ __forceinline__ float distill_below(float x, float unit_max) { return fmaf(x, 1.f / kDistillUnit, unit_max); }

// What distill_weight takes of the row's largest teacher value.
template <bool WEIGHTS>
__device__ __forceinline__ float distill_teacher(float mt) { return WEIGHTS ? distill_factor(mt) : -mt / kDistillUnit; }

// The teacher's unnormalised weight of a place and its logarithm c, times tau / 2^24 (a logit of -inf: 0 and -inf).
template <bool WEIGHTS>
__device__ __forceinline__ float distill_weight(float t, float teacher, const DistillArgs& a, float& c)
{
    if constexpr (WEIGHTS) {
        const float f = t * teacher;
        c = distill_log2(f) * a.unit_log2;
        return f;
    } else {
        c = distill_below(t, teacher);
        return distill_exp2(c * a.scale);
    }
}

// N places in registers: s scores (-inf where a place does not count), f the teacher's values (then 0 or
// -inf).  Raises the row's maxima.
template <bool WEIGHTS, int N>
__device__ __forceinline__ void distill_maxima(const float* s, float* f, float& ms, float& mt)
{
#pragma unroll
    for (int e = 0; e < N; ++e) {
        if (s[e] == -CUDART_INF_F) f[e] = WEIGHTS ? 0.f : -CUDART_INF_F;
        ms = fmaxf(ms, s[e]);
        mt = fmaxf(mt, f[e]);
    }
}

// From the row's maxima (0 in place of -inf, so that -inf gives weight 0): s becomes e^a, f the teacher's
// weight; their sums and the cross sum grow (that in units of 2^24 / tau).
template <bool WEIGHTS, int N>
__device__ __forceinline__ void distill_sums(float* s, float* f, float ms, float mt, const DistillArgs& a, float& z,
                                             float& y, float& x)
{
    const float um = -ms / kDistillUnit, ut = distill_teacher<WEIGHTS>(mt);
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const float d = distill_below(s[e], um);
        s[e] = distill_exp2(d * a.scale);
        z += s[e];
        float c;
        f[e] = distill_weight<WEIGHTS>(f[e], ut, a, c);
        y += f[e];
        if (f[e] != 0.f) x = fmaf(f[e], c - d, x);
    }
}

// What a row's sums say: the loss, and the factors of e^a and f in the gradient.
struct DistillRow {
    float loss, cs, ct;
    bool sound;   // the factors are finite
};

__device__ __forceinline__ DistillRow distill_row(float z, float y, float x, float g, const DistillArgs& a)
{
    DistillRow r{0.f, 0.f, 0.f, true};
    if (y == 0.f || z == 0.f) return r;   // no counted place, or none that the teacher weighs: nothing to learn
    r.loss = x / y * kDistillUnit * a.inv_tau + (logf(z) - logf(y));
    r.cs = g * a.inv_tau / z;
    r.ct = g * a.inv_tau / y;
    r.sound = isfinite(r.cs) && isfinite(r.ct);
    return r;
}

// A place's gradient: 0 where neither has weight, whatever a NaN elsewhere in the row made of the factors.
__device__ __forceinline__ float distill_grad(float s, float f, const DistillRow& r)
{
    return r.sound ? s * r.cs - f * r.ct : s == 0.f && f == 0.f ? 0.f : s * r.cs - f * r.ct;
}

// One row per group of T threads (T = 32: NT / 32 rows per CTA; else T == NT), in registers.
template <typename TT, bool WEIGHTS, int VEC, bool EDGE, int T, int NV, int NT>
__global__ void __launch_bounds__(NT) distill_kernel(const __grid_constant__ DistillArgs a)
{
    __shared__ float4 red1[32], red2[32];
    const int t = threadIdx.x % T;
    const int row = blockIdx.x * (NT / T) + threadIdx.x / T;
    if (row >= a.n) return;   // whole warps (T = 32) or whole CTAs
    const float* sp = a.s + (int64_t)row * a.ld_s;
    const TT* tp = static_cast<const TT*>(a.t) + (int64_t)row * a.ld_t;
    const int32_t* lp = a.list ? a.list + (int64_t)row * a.ld_list : nullptr;
    // columns are taken from the 4-place boundary at or before the row's start, so that rows of an odd
    // stride still move 16 bytes at a time (single places cost twice the time)
    const int c0 = EDGE ? -int((a.off0 + (int64_t)row * a.off_step) & 3) : 0;
    float s[NV][VEC], f[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = c0 + (i * T + t) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) s[i][e] = -CUDART_INF_F;
        if (c >= a.k) continue;
        distill_load<VEC, EDGE>(sp, c, a.k, s[i]);
        distill_load<VEC, EDGE>(tp, c, a.k, f[i]);
        int32_t l[VEC];
        if (lp) distill_load<VEC, EDGE>(lp, c, a.k, l);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            if ((EDGE && (c + e < 0 || c + e >= a.k)) || (lp && l[e] < 0)) s[i][e] = -CUDART_INF_F;
    }
    float ms = -CUDART_INF_F, mt = -CUDART_INF_F;
#pragma unroll
    for (int i = 0; i < NV; ++i) distill_maxima<WEIGHTS, VEC>(s[i], f[i], ms, mt);
    distill_max2<T>(ms, mt, red1);
    ms = ms == -CUDART_INF_F ? 0.f : ms;
    mt = mt == -CUDART_INF_F ? 0.f : mt;
    float z = 0.f, y = 0.f, x = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) distill_sums<WEIGHTS, VEC>(s[i], f[i], ms, mt, a, z, y, x);
    distill_sum3<T>(z, y, x, red2);
    const DistillRow r = distill_row(z, y, x, a.g ? a.g[row] : 1.f, a);
    if (t == 0 && a.loss) a.loss[row] = r.loss;
    if (!a.ds) return;
    float* dp = a.ds + (int64_t)row * a.ld_ds;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = c0 + (i * T + t) * VEC;
        if (c >= a.k) continue;
        float v[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = distill_grad(s[i][e], f[i][e], r);
        if (VEC == 4 && (!EDGE || (c >= 0 && c + 3 < a.k))) {
            *reinterpret_cast<float4*>(dp + c) = make_float4(v[0], v[VEC / 4], v[VEC / 2], v[VEC - 1]);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (!EDGE || (c + e >= 0 && c + e < a.k)) dp[c + e] = v[e];
        }
    }
}

// One row at a time per CTA, of at most NT * 4 * NV places, with the next row's places on
// their way to shared memory while this one is worked on (a CTA per row holds so many registers that
// it is alone on its SM, and its loads, sums and stores then follow one another: 78 us for
// 1021 x 20011).  A thread copies the places that it reads itself, so it waits for its own copies alone;
// vectors that hang over a row's ends are loaded when they are needed.
template <typename TT, bool WEIGHTS, bool EDGE, int NV, int NT, int CTAS>
__global__ void __launch_bounds__(NT, CTAS) distill_ring_kernel(const __grid_constant__ DistillArgs a)
{
    extern __shared__ __align__(16) uint8_t dyn[];
    __shared__ float4 red1[NT / 32], red2[NT / 32];
    const int t = threadIdx.x;
    float4* ss = reinterpret_cast<float4*>(dyn);                                    // [NV][NT] scores
    int4* sl = reinterpret_cast<int4*>(ss + NV * NT);                               // [NV][NT] lists, if given
    using Quad = typename std::conditional<sizeof(TT) == 2, uint2, float4>::type;
    Quad* st = reinterpret_cast<Quad*>(a.list ? sl + NV * NT : sl);                 // [NV][NT] teacher
    auto start = [&](int64_t row) { return EDGE ? -int((a.off0 + row * a.off_step) & 3) : 0; };
    auto whole = [&](int c) { return !EDGE || (c >= 0 && c + 3 < a.k); };
    auto fetch = [&](int64_t row) {
        if (row < a.n) {
            const int c0 = start(row);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = c0 + (i * NT + t) * 4;
                if (c >= a.k || !whole(c)) continue;
                distill_copy<16>(ss + i * NT + t, a.s + row * a.ld_s + c);
                distill_copy<sizeof(Quad)>(st + i * NT + t, static_cast<const TT*>(a.t) + row * a.ld_t + c);
                if (a.list) distill_copy<16>(sl + i * NT + t, a.list + row * a.ld_list + c);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    fetch(blockIdx.x);
    for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        const int c0 = start(row);
        float s[NV][4], f[NV][4];
        float ms = -CUDART_INF_F, mt = -CUDART_INF_F;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + (i * NT + t) * 4;
            int32_t l[4] = {0, 0, 0, 0};
            if (c >= a.k) {
#pragma unroll
                for (int e = 0; e < 4; ++e) { s[i][e] = -CUDART_INF_F; f[i][e] = 0.f; }
            } else if (whole(c)) {
                distill_load<4, false>(reinterpret_cast<const float*>(ss + i * NT + t), 0, 4, s[i]);
                distill_load<4, false>(reinterpret_cast<const TT*>(st + i * NT + t), 0, 4, f[i]);
                if (a.list) distill_load<4, false>(reinterpret_cast<const int32_t*>(sl + i * NT + t), 0, 4, l);
            } else {
                distill_load<4, true>(a.s + row * a.ld_s, c, a.k, s[i]);
                distill_load<4, true>(static_cast<const TT*>(a.t) + row * a.ld_t, c, a.k, f[i]);
                if (a.list) distill_load<4, true>(a.list + row * a.ld_list, c, a.k, l);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c + e < 0 || c + e >= a.k) s[i][e] = -CUDART_INF_F;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (l[e] < 0) s[i][e] = -CUDART_INF_F;
            distill_maxima<WEIGHTS, 4>(s[i], f[i], ms, mt);
        }
        distill_max2<NT>(ms, mt, red1);
        fetch(row + gridDim.x);   // behind the barrier: every value has left shared memory
        ms = ms == -CUDART_INF_F ? 0.f : ms;
        mt = mt == -CUDART_INF_F ? 0.f : mt;
        float z = 0.f, y = 0.f, x = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) distill_sums<WEIGHTS, 4>(s[i], f[i], ms, mt, a, z, y, x);
        distill_sum3<NT>(z, y, x, red2);
        const DistillRow r = distill_row(z, y, x, a.g ? a.g[row] : 1.f, a);
        if (t == 0 && a.loss) a.loss[row] = r.loss;
        if (!a.ds) continue;
        float* dp = a.ds + row * a.ld_ds;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + (i * NT + t) * 4;
            if (c >= a.k) continue;
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = distill_grad(s[i][e], f[i][e], r);
            if (whole(c)) {
                *reinterpret_cast<float4*>(dp + c) = make_float4(v[0], v[1], v[2], v[3]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c + e >= 0 && c + e < a.k) dp[c + e] = v[e];
            }
        }
    }
}

// Rows of any length: one CTA per row, two sweeps.  In the first a thread keeps running maxima and the
// sums z and y, rescaled when a batch of places raises a maximum (by 0 where that is out of reach); the
// CTA then brings its threads' sums to the row's maxima and joins them.  The second writes the gradient
// and adds up the cross sum: it needs the row's maxima, since a running one would carry terms of places
// whose weight the row's maximum makes zero (f = 0 times an infinite rescaling is no number).  The next
// batch's loads are under way behind the current one's arithmetic: 128 x 131072 fp32 79 us, 207 without
// (one row a CTA: the loads' latency was the time); 512 x 32768 83 us.
template <typename TT, bool WEIGHTS, int NT>
__global__ void __launch_bounds__(NT) distill_long_kernel(const __grid_constant__ DistillArgs a)
{
    __shared__ float4 red1[32], red2[32];
    const int row = blockIdx.x;
    const float* sp = a.s + (int64_t)row * a.ld_s;
    const TT* tp = static_cast<const TT*>(a.t) + (int64_t)row * a.ld_t;
    const int32_t* lp = a.list ? a.list + (int64_t)row * a.ld_list : nullptr;
    constexpr int BATCH = 8;
    float s[BATCH], v[BATCH], sn[BATCH];
    TT vn[BATCH];
    int32_t ln[BATCH];
    auto ask = [&](int64_t c0) {   // the batch at c0
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int64_t c = c0 + (int64_t)i * NT;
            sn[i] = -CUDART_INF_F;
            vn[i] = TT(0.f);
            ln[i] = 0;
            if (c < a.k) {
                sn[i] = sp[c];
                vn[i] = tp[c];
                if (lp) ln[i] = lp[c];
            }
        }
    };
    auto take = [&](int64_t next) {   // the batch asked for, into s and v; the one at `next` is asked for
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            s[i] = ln[i] < 0 ? -CUDART_INF_F : sn[i];
            v[i] = s[i] == -CUDART_INF_F ? (WEIGHTS ? 0.f : -CUDART_INF_F) : (float)vn[i];
        }
        ask(next);
    };
    // maxima with 0 in place of -inf (so that -inf gives weight 0)
    auto finite = [](float m) { return m == -CUDART_INF_F ? 0.f : m; };
    // to maxima m and n; nothing is summed while one is -inf
    float ms = -CUDART_INF_F, mt = -CUDART_INF_F, z = 0.f, y = 0.f;
    auto raise = [&](float m, float n) {
        if (m > ms) {
            if (ms != -CUDART_INF_F) z *= distill_exp2(distill_below(ms, -m / kDistillUnit) * a.scale);
            ms = m;
        }
        if (n > mt) {
            if (mt != -CUDART_INF_F)
                y *= WEIGHTS ? distill_factor(n) / distill_factor(mt)
                             : distill_exp2(distill_below(mt, -n / kDistillUnit) * a.scale);
            mt = n;
        }
    };
    ask(threadIdx.x);
    for (int64_t c0 = threadIdx.x; c0 < a.k; c0 += (int64_t)BATCH * NT) {
        take(c0 + (int64_t)BATCH * NT);
        float m = ms, n = mt;
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            m = fmaxf(m, s[i]);
            n = fmaxf(n, v[i]);
        }
        raise(m, n);
        const float um = -finite(ms) / kDistillUnit, ut = distill_teacher<WEIGHTS>(finite(mt));
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            z += distill_exp2(distill_below(s[i], um) * a.scale);
            float c;
            y += distill_weight<WEIGHTS>(v[i], ut, a, c);
        }
    }
    float m = ms, n = mt, x = 0.f;
    distill_max2<NT>(m, n, red1);
    raise(m, n);
    distill_sum3<NT>(z, y, x, red2);
    const float g = a.g ? a.g[row] : 1.f;
    DistillRow r = distill_row(z, y, x, g, a);
    const float um = -finite(ms) / kDistillUnit, ut = distill_teacher<WEIGHTS>(finite(mt));
    float* dp = a.ds ? a.ds + (int64_t)row * a.ld_ds : nullptr;
    ask(threadIdx.x);
    for (int64_t c0 = threadIdx.x; c0 < a.k; c0 += (int64_t)BATCH * NT) {
        take(c0 + (int64_t)BATCH * NT);
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int64_t c = c0 + (int64_t)i * NT;
            if (c >= a.k) continue;
            const float d = distill_below(s[i], um), e = distill_exp2(d * a.scale);
            float lg;
            const float w = distill_weight<WEIGHTS>(v[i], ut, a, lg);
            if (w != 0.f) x = fmaf(w, lg - d, x);
            if (dp) dp[c] = distill_grad(e, w, r);
        }
    }
    if (!a.loss) return;
    float unused1 = 0.f, unused2 = 0.f;
    distill_sum3<NT>(x, unused1, unused2, red1);
    if (threadIdx.x == 0) a.loss[row] = distill_row(z, y, x, g, a).loss;
}

}  // namespace dsa
