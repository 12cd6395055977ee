// gc_norm.h -- geometry and arithmetic shared by the group-norm kernels.
//
//   hat = (x - mean) * rstd,  z = gamma * hat + beta,  y = act(z)
//   g = dy * act'(z),  dbeta = sum g,  dgamma = sum g * hat
//   dx = rstd * (gamma*g - c1 - hat*c2),   c1 = mean over the group of gamma*g,
//                                          c2 = mean over the group of gamma*g*hat
#pragma once

#include "../../include/gc.h"
#include "gc_vec.h"

namespace gc {

struct NormGeom {
    int B, C, HW, G, Cg;   // Cg = C / G channels of a group
    int nhwc;              // 0: [B][C][HW], 1: [B][HW][C]
    int act;               // gc_act
    int pf32;              // gamma, beta and their gradients in fp32 (else the storage type)
    float eps;
    int64_t img;           // C*HW, elements of an image (below 2^31)
    FastDiv fd_HW, fd_Cg;
};

template <typename T>
__device__ __forceinline__ float param(const NormGeom &g, const void *p, int c, float none)
{
    if (!p) return none;
    return g.pf32 ? static_cast<const float *>(p)[c] : to_f32(static_cast<const T *>(p)[c]);
}

template <typename T>
__device__ __forceinline__ void set_param(const NormGeom &g, void *p, int c, float v)
{
    if (!p) return;
    if (g.pf32) static_cast<float *>(p)[c] = v;
    else static_cast<T *>(p)[c] = from_f32<T>(v);
}

// gamma (or beta) of K neighbouring channels, each for N/K elements of v in a row.  One
// wide load: lanes whose channels lie a vector apart would make a memory line of every
// few lanes of each element load (50,000 x 128 x 1 x 2 bf16 forward 29 us that way, 16 this).
template <int K, typename T, int N>
__device__ __forceinline__ void near_params(const NormGeom &g, const void *p, int c, float none, float (&v)[N])
{
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = none;
    if (!p) return;
    if (g.pf32) {
        const Vec<float, K> w = load_vec<float, K>(static_cast<const float *>(p) + c);
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = w.get(j / (N / K));
    } else {
        const Vec<T, K> w = load_vec<T, K>(static_cast<const T *>(p) + c);
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = w.get(j / (N / K));
    }
}

__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.f + __expf(-z)); }

// Phi(z), the normal distribution function, and e = exp(-z^2/2): Abramowitz and
// Stegun 7.1.26 for erf(|z|/sqrt 2), absolute error at most 1.5e-7 (half of that
// in Phi), whose exponential is the density's.
__device__ __forceinline__ float phi(float z, float &e)
{
    const float u = fabsf(z) * 0.70710678f;
    e = __expf(-u * u);
    const float t = __builtin_amdgcn_rcpf(fmaf(0.3275911f, u, 1.f));
    float p = fmaf(1.061405429f, t, -1.453152027f);
    p = fmaf(p, t, 1.421413741f);
    p = fmaf(p, t, -0.284496736f);
    p = fmaf(p, t, 0.254829592f);
    const float tail = 0.5f * p * t * e;   // Phi(-|z|)
    return z < 0.f ? tail : 1.f - tail;
}

__device__ __forceinline__ float norm_z(float x, float mean, float rstd, float gamma, float beta)
{
    return fmaf((x - mean) * rstd, gamma, beta);
}

// act(z); a NaN stays one
template <int N>
__device__ __forceinline__ void activate(int act, float (&z)[N])
{
    if (act == GC_ACT_RELU) {
#pragma unroll
        for (int j = 0; j < N; ++j) z[j] = z[j] <= 0.f ? 0.f : z[j];
    } else if (act == GC_ACT_SILU) {
#pragma unroll
        for (int j = 0; j < N; ++j) z[j] *= sigmoid(z[j]);
    } else if (act == GC_ACT_GELU) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float e;
            z[j] *= phi(z[j], e);
        }
    }
}

// dy[j] becomes g = dy * act'(z); x[j] becomes hat
template <int N, int NC>
__device__ __forceinline__ void act_grad(int act, float (&x)[N], float (&dy)[N], const float (&mean)[NC],
                                         const float (&rstd)[NC], const float (&gamma)[NC],
                                         const float (&beta)[NC])
{
    static_assert(NC == 1 || NC == N, "constants of one channel or of each element");
    if (act == GC_ACT_RELU) {
        // 0 where z <= 0.  z in fp32 is off by less than 2^-21 of its product term;
        // nearer to the kink than that (an element in a million) its sign is taken in fp64.
        uint32_t off = 0, near = 0;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int k = NC == 1 ? 0 : j;
            const float z = norm_z(x[j], mean[k], rstd[k], gamma[k], beta[k]);
            off |= z <= 0.f ? 1u << j : 0u;
            near |= fabsf(z) <= 4.8e-7f * fabsf(z - beta[k]) ? 1u << j : 0u;
        }
        while (near) {   // one at a time: unrolled, fp64 would take 30 to 70 registers
            const int i = __builtin_ctz(near);
            near &= near - 1;
            float v[5];
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int k = NC == 1 ? 0 : j;
                if (j == i) {
                    v[0] = x[j];
                    v[1] = mean[k];
                    v[2] = rstd[k];
                    v[3] = gamma[k];
                    v[4] = beta[k];
                }
            }
            const double z = (double(v[0]) - v[1]) * v[2] * v[3] + v[4];
            off = (off & ~(1u << i)) | (z <= 0.0 ? 1u << i : 0u);
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int k = NC == 1 ? 0 : j;
            if (off >> j & 1) dy[j] = 0.f;
            x[j] = (x[j] - mean[k]) * rstd[k];
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = (x[j] - mean[NC == 1 ? 0 : j]) * rstd[NC == 1 ? 0 : j];
    if (act == GC_ACT_SILU) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float z = fmaf(x[j], gamma[NC == 1 ? 0 : j], beta[NC == 1 ? 0 : j]);
            const float s = sigmoid(z);
            dy[j] *= s * fmaf(z, 1.f - s, 1.f);
        }
    } else if (act == GC_ACT_GELU) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float z = fmaf(x[j], gamma[NC == 1 ? 0 : j], beta[NC == 1 ? 0 : j]);
            float e;
            const float p = phi(z, e);
            dy[j] *= fmaf(z * 0.39894228f, e, p);
        }
    }
}

}  // namespace gc
