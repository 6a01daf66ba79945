// Layer norm of rows and its backward pass.
//
// Forward, per row x of d values: mu = mean(x), v = mean((x - mu)^2), r = 1/sqrt(v + eps),
// y = (x - mu) r w + b.  Backward with xh = (x - mu) r and g = dy w:
// dx = r (g - mean(g) - xh mean(g xh)), dw = sum over rows of dy xh, db = sum over rows of dy.
//
// Both passes are bound by memory: each input is read once and each output written once.  A row is
// held in the registers of a group of T threads (T * E >= d), so the variance is the two-pass one
// (centred before it is squared) at no extra read; the sums are fp32.  The weight's gradient is
// summed in two levels of fixed order: a thread keeps the same columns for every row it handles and
// adds them up in registers, a CTA joins its row groups through shared memory and writes one
// partial row, and a second kernel adds the partial rows column by column.
#pragma once

#include "ptx.cuh"

namespace dsa {

struct NormArgs {
    const void* x;
    int64_t ld_x;
    const void* dy;     // backward
    int64_t ld_dy;
    void* out;          // y, or dx
    int64_t ld_out;
    const float* w;     // NULL: ones
    const float* b;     // NULL: zeros
    const float* mean_in;
    const float* rstd_in;
    float* mean;        // NULL: not written
    float* rstd;
    float* part;        // [gridDim.x][2][d] partial sums of the weight's and the bias's gradient
    int64_t n;
    int32_t d;
    float eps;
};

// VEC consecutive elements as loaded (VEC 8: 16-byte aligned rows; VEC 1: any), and as fp32.
template <typename TX, int VEC>
struct NormRaw {
    TX v;
    __device__ __forceinline__ void zero() { v = TX(0.f); }
    __device__ __forceinline__ void load(const TX* p) { v = *p; }
    __device__ __forceinline__ void get(float* f) const { f[0] = (float)v; }
};

template <>
struct NormRaw<float, 8> {
    float4 a, b;
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void load(const float* p)
    {
        a = *reinterpret_cast<const float4*>(p);
        b = *reinterpret_cast<const float4*>(p + 4);
    }
    __device__ __forceinline__ void get(float* f) const
    {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
};

template <>
struct NormRaw<__nv_bfloat16, 8> {
    uint4 a;
    __device__ __forceinline__ void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void get(float* f) const
    {
        const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
};

template <int VEC, typename TX>
__device__ __forceinline__ void norm_load_vec(const TX* p, float* f)
{
    NormRaw<TX, VEC> r;
    r.load(p);
    r.get(f);
}

template <int VEC>
__device__ __forceinline__ void norm_store_vec(float* p, const float* v)
{
    if constexpr (VEC == 8) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *p = v[0];
    }
}

template <int VEC>
__device__ __forceinline__ void norm_store_vec(__nv_bfloat16* p, const float* v)
{
    if constexpr (VEC == 8) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
        *p = __float2bfloat16_rn(v[0]);
    }
}

// Arithmetic on N values in registers, two to an instruction where N is even: with one value an
// instruction, 16-bit rows were bound by the issue of instructions (two thirds of the slots), not by
// memory.  Every element is rounded as in the plain form.

// v += s
template <int N>
__device__ __forceinline__ void norm_shift(float* v, float s)
{
    if constexpr (N % 2 == 0) {
        const uint64_t ss = pack_f32x2(s, s);
#pragma unroll
        for (int i = 0; i < N; i += 2) unpack_f32x2(add_f32x2(pack_f32x2(v[i], v[i + 1]), ss), v[i], v[i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += s;
    }
}

// v *= s
template <int N>
__device__ __forceinline__ void norm_scale(float* v, float s)
{
    if constexpr (N % 2 == 0) {
        const uint64_t ss = pack_f32x2(s, s);
#pragma unroll
        for (int i = 0; i < N; i += 2) unpack_f32x2(mul_f32x2(pack_f32x2(v[i], v[i + 1]), ss), v[i], v[i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] *= s;
    }
}

// v *= w
template <int N>
__device__ __forceinline__ void norm_times(float* v, const float* w)
{
    if constexpr (N % 2 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 2)
            unpack_f32x2(mul_f32x2(pack_f32x2(v[i], v[i + 1]), pack_f32x2(w[i], w[i + 1])), v[i], v[i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] *= w[i];
    }
}

// acc += v
template <int N>
__device__ __forceinline__ void norm_add(float* acc, const float* v)
{
    if constexpr (N % 2 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 2)
            unpack_f32x2(add_f32x2(pack_f32x2(acc[i], acc[i + 1]), pack_f32x2(v[i], v[i + 1])), acc[i], acc[i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] += v[i];
    }
}

// acc = a * b + acc
template <int N>
__device__ __forceinline__ void norm_fma(float* acc, const float* a, const float* b)
{
    if constexpr (N % 2 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 2)
            unpack_f32x2(fma_f32x2(pack_f32x2(a[i], a[i + 1]), pack_f32x2(b[i], b[i + 1]), pack_f32x2(acc[i], acc[i + 1])),
                         acc[i], acc[i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = fmaf(a[i], b[i], acc[i]);
    }
}

// acc = a * s + acc
template <int N>
__device__ __forceinline__ void norm_fma(float* acc, const float* a, float s)
{
    if constexpr (N % 2 == 0) {
        const uint64_t ss = pack_f32x2(s, s);
#pragma unroll
        for (int i = 0; i < N; i += 2)
            unpack_f32x2(fma_f32x2(pack_f32x2(a[i], a[i + 1]), ss, pack_f32x2(acc[i], acc[i + 1])), acc[i], acc[i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = fmaf(a[i], s, acc[i]);
    }
}

// Sum of (a, b) over the T threads of a row group: lanes of one warp, or the whole CTA (T == NT).
// `red` (32 entries) must not be in use by a sum that some thread may still be reading: callers
// alternate between two.
template <int T>
__device__ __forceinline__ void norm_group_sum(float& a, float& b, float2* red)
{
#pragma unroll
    for (int o = (T < 32 ? T : 32) / 2; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if constexpr (T > 32) {
        constexpr int NW = T / 32;   // a power of two: every warp adds the same tree, every lane ends with the sum
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(a, b);
        __syncthreads();
        const float2 v = red[threadIdx.x & (NW - 1)];
        a = v.x;
        b = v.y;
#pragma unroll
        for (int o = NW / 2; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
        }
    }
}

// NT threads per CTA in groups of T; element e of thread t of a group: column ((e / VEC) * T + t) * VEC + e % VEC.
// A group takes R rows (NT / T apart), all asked for before the first is used.
template <typename TX, typename TY, int VEC, int T, int NV, int NT, int R>
__global__ void __launch_bounds__(NT) layer_norm_kernel(const __grid_constant__ NormArgs a)
{
    __shared__ float2 red[2][32];
    constexpr int G = NT / T;   // rows of a CTA at once
    const int t = threadIdx.x % T, g = threadIdx.x / T;
    const float inv_d = 1.f / (float)a.d;
    const int64_t row0 = (int64_t)blockIdx.x * (G * R) + g;
    NormRaw<TX, VEC> raw[R][NV];
#pragma unroll
    for (int k = 0; k < R; ++k)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t row = row0 + k * G;
            const int c = (i * T + t) * VEC;
            raw[k][i].zero();   // (what lies outside the row counts for nothing)
            if (row < a.n && c < a.d) raw[k][i].load(static_cast<const TX*>(a.x) + row * a.ld_x + c);
        }
    constexpr int S = VEC == 8 ? 2 : 1;   // running sums of a thread
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int64_t row = row0 + k * G;
        float v[NV][VEC];
        float s[S], q[S], unused = 0.f;
#pragma unroll
        for (int e = 0; e < S; ++e) s[e] = q[e] = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            raw[k][i].get(v[i]);
#pragma unroll
            for (int e = 0; e < VEC; e += S) norm_add<S>(s, v[i] + e);
        }
        float sum = S == 2 ? s[0] + s[S - 1] : s[0];
        norm_group_sum<T>(sum, unused, red[0]);
        const float mu = sum * inv_d;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            norm_shift<VEC>(v[i], -mu);
            if ((i * T + t) * VEC < a.d)
#pragma unroll
                for (int e = 0; e < VEC; e += S) norm_fma<S>(q, v[i] + e, v[i] + e);
        }
        sum = S == 2 ? q[0] + q[S - 1] : q[0];
        unused = 0.f;
        norm_group_sum<T>(sum, unused, red[1]);
        const float r = 1.f / sqrtf(fmaf(sum, inv_d, a.eps));
        if (row >= a.n) continue;
        if (t == 0) {
            if (a.mean) a.mean[row] = mu;
            if (a.rstd) a.rstd[row] = r;
        }
        TY* y = static_cast<TY*>(a.out) + row * a.ld_out;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * T + t) * VEC;
            if (c >= a.d) continue;
            float w[VEC], b[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) { w[e] = 1.f; b[e] = 0.f; }
            if (a.w) norm_load_vec<VEC>(a.w + c, w);
            if (a.b) norm_load_vec<VEC>(a.b + c, b);
            norm_scale<VEC>(v[i], r);
            norm_fma<VEC>(b, v[i], w);
            norm_store_vec<VEC>(y + c, b);
        }
    }
}

// CTAs of the backward kernel an SM holds: 768 threads of up to 80 registers (1024 of 64 spill, and CTAs
// past the resident ones ran as a second wave: 131072 x 128 fp32 45 us against 38), or one of 1024
// (whose launch bounds name no count: given 1, the compiler moved the loads behind the sums, 74 us
// against 56 for 4099 x 5001).
constexpr int norm_bwd_per_sm(int threads) { return threads >= 1024 ? 1 : 768 / threads; }

// TX: the type of x and dx, TY: of dy.  A group walks its rows with the next one's loads in flight
// behind the current one's sums: without that, a group waits out the memory's latency once a row.
template <typename TX, typename TY, int VEC, int T, int NV, int NT>
__global__ void __launch_bounds__(NT, NT < 1024 ? norm_bwd_per_sm(NT) : 0) layer_norm_bwd_kernel(const __grid_constant__ NormArgs a)
{
    __shared__ float2 red[2][32];
    constexpr int G = NT / T;
    const int t = threadIdx.x % T, g = threadIdx.x / T;
    const float inv_d = 1.f / (float)a.d;
    float dw[NV][VEC], db[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) dw[i][e] = db[i][e] = 0.f;
    NormRaw<TX, VEC> rx[NV];
    NormRaw<TY, VEC> ry[NV];
    float mu_next = 0.f, r_next = 0.f;
    auto read = [&](int64_t row) {
        if constexpr (VEC == 8) {   // places outside the rows are zeros in dy, which keeps them out of every sum
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                rx[i].zero();
                ry[i].zero();
            }
        }
        if (row >= a.n) return;
        const TX* x = static_cast<const TX*>(a.x) + row * a.ld_x;
        const TY* dy = static_cast<const TY*>(a.dy) + row * a.ld_dy;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * T + t) * VEC;
            if (c < a.d) {
                rx[i].load(x + c);
                ry[i].load(dy + c);
            }
        }
        mu_next = a.mean_in[row];
        r_next = a.rstd_in[row];
    };
    const int64_t step = (int64_t)gridDim.x * G;
    read((int64_t)blockIdx.x * G + g);
    int odd = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * G; row0 < a.n; row0 += step, odd ^= 1) {
        const int64_t row = row0 + g;
        const bool live = row < a.n;
        float xh[NV][VEC], gy[NV][VEC];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            rx[i].get(xh[i]);
            ry[i].get(gy[i]);
        }
        const float mu = mu_next, r = r_next;
        read(row + step);
        constexpr int S = VEC == 8 ? 2 : 1;
        float a1[S], a2[S];   // sums of g and of g xh
#pragma unroll
        for (int e = 0; e < S; ++e) a1[e] = a2[e] = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * T + t) * VEC;
            if constexpr (VEC == 8) {
                norm_shift<VEC>(xh[i], -mu);
                norm_scale<VEC>(xh[i], r);
                norm_fma<VEC>(dw[i], gy[i], xh[i]);
                norm_add<VEC>(db[i], gy[i]);
                if (a.w && c < a.d) {
                    float w[VEC];
                    norm_load_vec<VEC>(a.w + c, w);   // from L1 after the first row
                    norm_times<VEC>(gy[i], w);
                }
#pragma unroll
                for (int e = 0; e < VEC; e += S) {
                    norm_add<S>(a1, gy[i] + e);
                    norm_fma<S>(a2, gy[i] + e, xh[i] + e);
                }
            } else {
                const bool in = live && c < a.d;
                float w = 1.f;
                if (a.w && c < a.d) w = a.w[c];
                xh[i][0] = in ? (xh[i][0] - mu) * r : 0.f;
                gy[i][0] = in ? gy[i][0] : 0.f;
                dw[i][0] = fmaf(gy[i][0], xh[i][0], dw[i][0]);
                db[i][0] += gy[i][0];
                gy[i][0] *= w;
                a1[0] += gy[i][0];
                a2[0] = fmaf(gy[i][0], xh[i][0], a2[0]);
            }
        }
        float s1 = S == 2 ? a1[0] + a1[S - 1] : a1[0], s2 = S == 2 ? a2[0] + a2[S - 1] : a2[0];
        norm_group_sum<T>(s1, s2, red[odd]);
        const float m1 = s1 * inv_d, m2 = s2 * inv_d;
        if (!live || !a.out) continue;
        TX* dx = static_cast<TX*>(a.out) + row * a.ld_out;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * T + t) * VEC;
            if (c >= a.d) continue;
            if constexpr (VEC == 8) {
                norm_shift<VEC>(gy[i], -m1);
                norm_fma<VEC>(gy[i], xh[i], -m2);
                norm_scale<VEC>(gy[i], r);
            } else {
                gy[i][0] = r * (gy[i][0] - m1 - xh[i][0] * m2);
            }
            norm_store_vec<VEC>(dx + c, gy[i]);
        }
    }
    grid_dep_launch();   // the summing kernel may start its prologue
    if (!a.part) return;
    // join the CTA's row groups in order of their number, then one partial row per CTA
    float* out = a.part + (int64_t)blockIdx.x * 2 * a.d;
    if constexpr (G == 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * T + t) * VEC;
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (c + e < a.d) {
                    out[c + e] = dw[i][e];
                    out[a.d + c + e] = db[i][e];
                }
        }
    } else {
        // groups that share a warp are joined by shuffles, warps through shared memory
        constexpr int NW = NT / 32, CW = (T < 32 ? T : 32) * NV * VEC;   // columns held by a warp
        __shared__ float sh[NW][2][CW];
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                float p = dw[i][e], q = db[i][e];
#pragma unroll
                for (int o = 16; o >= T; o >>= 1) {
                    p += __shfl_xor_sync(0xffffffffu, p, o);
                    q += __shfl_xor_sync(0xffffffffu, q, o);
                }
                if ((threadIdx.x & 31) < T) {
                    sh[threadIdx.x >> 5][0][(i * T + t) * VEC + e] = p;
                    sh[threadIdx.x >> 5][1][(i * T + t) * VEC + e] = q;
                }
            }
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * a.d; c += NT) {
            const int which = c >= a.d, col = c - which * a.d;
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < NW; ++i) s += sh[i][which][col];
            out[c] = s;
        }
    }
}

// Column sums of part [n_part][2][d]: 32 columns per CTA, 32 threads down each column, joined in order.  Clears the
// workspace's status words (a line in the first kernel costs 4099 x 5001 fp32, whose registers are full, 7 us).
__global__ void __launch_bounds__(1024) layer_norm_dw_kernel(const float* part, int32_t n_part, int32_t d,
                                                             float* dw, float* db, uint32_t* status)
{
    __shared__ float sh[32][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + tx;
    grid_dep_wait();
    if (blockIdx.x == 0 && threadIdx.x < kStatusBytes / 4) status[threadIdx.x] = 0;
    float s = 0.f;
    constexpr int U = 8;   // rows read together
    if (c < 2 * d)
        for (int i0 = ty; i0 < n_part; i0 += 32 * U) {
            float v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = i0 + 32 * u < n_part ? part[(int64_t)(i0 + 32 * u) * 2 * d + c] : 0.f;
#pragma unroll
            for (int u = 0; u < U; ++u) s += v[u];
        }
    sh[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && c < 2 * d) {
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) z += sh[i][tx];
        float* out = c < d ? dw : db;
        if (out) out[c < d ? c : c - d] = z;
    }
}

}  // namespace dsa
