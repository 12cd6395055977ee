// norm_res_small.hip -- group norm with an activation for small groups whose vectors
// hold several channels: positions fewer than a vector's elements in NCHW (1 x 2 after
// the policy's second convolution, or none at all), and channels last with few
// elements a group.
//
// A team of L <= 64 lanes owns a group, so all sums are lane exchanges; consecutive
// teams own consecutive groups, so a wave reads consecutive memory.  Channel constants
// are held per element of a vector.
//   NCHW: lane's vectors are lane, lane + L, ... of the group's M = Cg*HW
//     contiguous elements, the last one moved back to end with the group (its first
//     `skip` elements are another vector's).
//   Channels last (LAST): a row of the group is cv = Cg/N vectors, a power of two; a
//     lane keeps one column of them and takes every (L/cv)-th row, so its constants
//     are shared by its vectors.
// The backward (NCHW: channels last the LDS sums of norm_res_nhwc.hip are faster, 32
// against 40 us for 8000 x 128 x 3 x 4 bf16) walks images slot, slot + slots, ... as in the
// other resident kernels, and joins a workgroup's slots of a group in one row of
// partials.  Bound by memory: 50,000 x 128 x 1 x 2 fp32 forward 21 us (5.1 TB/s), backward 30
// (5.4) and 4 for the rows of partials.
#include <type_traits>

#include "gc_norm_res.h"

namespace gc {
namespace {

template <int N, bool LAST>
struct Lane {
    int first, step, count;   // the lane's vectors: first, first + step, ... below count
    int col;                  // LAST: its column
};

template <int N, bool LAST>
__device__ __forceinline__ Lane<N, LAST> lane_of(const NormGeom &g, const NormResPlan &q, int lane)
{
    if (LAST) {
        const int cv = g.Cg / N;
        return {lane / cv, q.L / cv, g.HW, lane & (cv - 1)};
    }
    return {lane, q.L, (g.Cg * g.HW + N - 1) / N, 0};
}

// offset of vector v from the group's first element, and its leading elements to skip
template <int N, bool LAST>
__device__ __forceinline__ int64_t vector_at(const NormGeom &g, const Lane<N, LAST> &w, int v, int &skip)
{
    skip = 0;
    if (LAST) return int64_t(v) * g.C + w.col * N;
    const int at = min(v * N, g.Cg * g.HW - N);
    skip = v * N - at;
    return at;
}

// the group's first element: image b, group gg
template <bool LAST>
__device__ __forceinline__ int64_t group_at(const NormGeom &g, int64_t b, int gg)
{
    return b * g.img + int64_t(gg) * g.Cg * (LAST ? 1 : g.HW);
}

// constants of a vector that holds whole channels, planes of S, 2S, ... positions: S divides
// N, so every vector starts with a channel.  Wide loads, see near_params (planes of 4, 20,000
// x 128 x 2 x 2 bf16 forward: 13.6 us, a load an element 16.7).
template <typename T, int N, int S>
__device__ __forceinline__ bool whole_channels(const NormGeom &g, int c0, const void *gamma, const void *beta,
                                               float (&a)[N], float (&b)[N])
{
    if (g.HW == S) {
        near_params<N / S, T>(g, gamma, c0, 1.f, a);
        near_params<N / S, T>(g, beta, c0, 0.f, b);
        return true;
    }
    if constexpr (2 * S < N) return whole_channels<T, N, 2 * S>(g, c0, gamma, beta, a, b);
    return false;
}

// constants of a vector's elements
template <typename T, int N, bool LAST>
__device__ __forceinline__ void element_params(const NormGeom &g, const Lane<N, LAST> &w, int gg, int at,
                                               const void *gamma, const void *beta, float (&a)[N], float (&b)[N])
{
    const int c0 = gg * g.Cg + (LAST ? w.col * N : int(fdiv(uint32_t(at), g.fd_HW)));
    if (LAST) {
        near_params<N, T>(g, gamma, c0, 1.f, a);
        near_params<N, T>(g, beta, c0, 0.f, b);
        return;
    }
    if (whole_channels<T, N, 1>(g, c0, gamma, beta, a, b)) return;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int c = gg * g.Cg + int(fdiv(uint32_t(at + j), g.fd_HW));
        a[j] = param<T>(g, gamma, c, 1.f);
        b[j] = param<T>(g, beta, c, 0.f);
    }
}

template <typename T, int N, int NV, bool LAST, bool PAST>
__global__ void __launch_bounds__(kResThreads)
    res_small_fwd(NormGeom g, NormResPlan q, const T *__restrict__ x, const void *__restrict__ gamma,
                 const void *__restrict__ beta, T *__restrict__ y, float *__restrict__ mean_out,
                 float *__restrict__ rstd_out)
{
    const int64_t block = blockIdx.x;
    const int lane = threadIdx.x & (q.L - 1);
    const Lane<N, LAST> w = lane_of<N, LAST>(g, q, lane);
    const int64_t k = block * q.teams + threadIdx.x / q.L;
    const bool live = k < int64_t(g.B) * g.G;
    const int gg = int(k % g.G);
    const int64_t base = group_at<LAST>(g, k / g.G, gg);
    Vec<T, N> v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        int skip;
        const int idx = w.first + i * w.step;
        if (live && idx < w.count) v[i] = load_vec<T, N>(x + base + vector_at(g, w, idx, skip));
        else v[i] = Vec<T, N>{};
    }
    float s[1] = {};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        int skip;
        vector_at(g, w, w.first + i * w.step, skip);
        if (w.first + i * w.step >= w.count) continue;
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (LAST || j >= skip) s[0] += v[i].get(j);
    }
    s[0] = lanes_sum(s[0], q.L);
    const float n = 1.f / (float(g.Cg) * float(g.HW)), m0 = s[0] * n;
    float t[2] = {};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        int skip;
        vector_at(g, w, w.first + i * w.step, skip);
        if (w.first + i * w.step >= w.count) continue;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (!LAST && j < skip) continue;
            const float d = v[i].get(j) - m0;
            t[0] += d;
            t[1] = fmaf(d, d, t[1]);
        }
    }
    t[0] = lanes_sum(t[0], q.L);
    t[1] = lanes_sum(t[1], q.L);
    if (!live) return;
    const float off = t[0] * n, mean = m0 + off;
    const float var = fmaxf(fmaf(-off, off, t[1] * n), 0.f);
    const float rstd = t[1] != t[1] ? t[1] : 1.f / sqrtf(var + g.eps);
    if (lane == 0) {
        if (mean_out) mean_out[k] = mean;
        if (rstd_out) rstd_out[k] = rstd;
    }
    float a[N], b[N];
    if (LAST) element_params<T, N, LAST>(g, w, gg, 0, gamma, beta, a, b);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        int skip;
        const int idx = w.first + i * w.step;
        if (idx >= w.count) continue;
        const int64_t at = vector_at(g, w, idx, skip);
        if (!LAST) element_params<T, N, LAST>(g, w, gg, int(at), gamma, beta, a, b);
        float z[N];
#pragma unroll
        for (int j = 0; j < N; ++j) z[j] = norm_z(v[i].get(j), mean, rstd, a[j], b[j]);
        activate(g.act, z);
        Vec<T, N> o;
        o.put(z);
        put_vec<PAST>(y + base + at, o);
    }
}

template <typename T, int N, int NV, bool PAST>
__global__ void __launch_bounds__(kResThreads)
    res_small_bwd(NormGeom g, NormResPlan q, const T *__restrict__ x, const T *__restrict__ dy,
                  const void *__restrict__ gamma, const void *__restrict__ beta, const float *__restrict__ mean,
                  const float *__restrict__ rstd, T *__restrict__ dx, float *__restrict__ part)
{
    extern __shared__ float lds[];
    const int lane = threadIdx.x & (q.L - 1), team = threadIdx.x / q.L;
    const int64_t unit = int64_t(blockIdx.x) * q.teams + team;   // (slot, group)
    const int gg = int(unit % g.G), slot = int(unit / g.G);
    const Lane<N, false> w = lane_of<N, false>(g, q, lane);
    const float n = 1.f / (float(g.Cg) * float(g.HW));

    float a[NV][N], b[NV][N], sg[NV][N] = {}, st[NV][N] = {};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        int skip;
        const int idx = min(w.first + i * w.step, w.count - 1);
        element_params<T, N, false>(g, w, gg, int(vector_at(g, w, idx, skip)), gamma, beta, a[i], b[i]);
    }
    for (int img = slot < q.images ? slot : g.B; img < g.B; img += q.images) {
        const int64_t k = int64_t(img) * g.G + gg, base = group_at<false>(g, img, gg);
        const float mk = mean[k], rk = rstd[k];
        float h[NV][N], d[NV][N], m[N], r[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            m[j] = mk;
            r[j] = rk;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            int skip;
            const int idx = w.first + i * w.step;
            Vec<T, N> vx{}, vd{};
            if (idx < w.count) {
                const int64_t at = base + vector_at(g, w, idx, skip);
                vx = load_vec<T, N>(x + at);
                vd = load_vec<T, N>(dy + at);
            }
#pragma unroll
            for (int j = 0; j < N; ++j) {
                h[i][j] = vx.get(j);
                d[i][j] = vd.get(j);
            }
        }
        float c[2] = {};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            int skip;
            const int idx = w.first + i * w.step;
            if (idx >= w.count) continue;
            vector_at(g, w, idx, skip);
            act_grad<N, N>(g.act, h[i], d[i], m, r, a[i], b[i]);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                if (j < skip) continue;
                const float p = d[i][j] * h[i][j];
                sg[i][j] += d[i][j];
                st[i][j] += p;
                c[0] = fmaf(a[i][j], d[i][j], c[0]);
                c[1] = fmaf(a[i][j], p, c[1]);
            }
        }
        const float c1 = lanes_sum(c[0], q.L) * n, c2 = lanes_sum(c[1], q.L) * n;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            int skip;
            const int idx = w.first + i * w.step;
            if (idx >= w.count) continue;
            float o[N];
#pragma unroll
            for (int j = 0; j < N; ++j) o[j] = rk * (fmaf(a[i][j], d[i][j], -c1) - h[i][j] * c2);
            Vec<T, N> ov;
            ov.put(o);
            put_vec<PAST>(dx + base + vector_at(g, w, idx, skip), ov);
        }
    }
    if (!part) return;
    const int M = g.Cg * g.HW;
    float *mine = lds + team * M * 2;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        int skip;
        const int idx = w.first + i * w.step;
        if (idx >= w.count) continue;
        const int at = int(vector_at(g, w, idx, skip));
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (j < skip) continue;
            mine[(at + j) * 2] = sg[i][j];
            mine[(at + j) * 2 + 1] = st[i][j];
        }
    }
    __syncthreads();
    // a channel's elements, and with `join` (a multiple of G teams a workgroup) over the
    // workgroup's slots of a group, in order
    const int from = q.join ? threadIdx.x : lane, step = q.join ? kResThreads : q.L;
    const int channels = q.join ? g.C : g.Cg;
    if (!q.join && slot >= q.images) return;
    float *row = part + (q.join ? int64_t(blockIdx.x) * g.C : int64_t(slot) * g.C + gg * g.Cg) * 2;
    for (int c = from; c < channels; c += step) {
        const int first = q.join ? int(fdiv(uint32_t(c), g.fd_Cg)) : team;   // the first team with its group
        const int e0 = (q.join ? c - first * g.Cg : c) * g.HW;
        float s = 0, t = 0;
        for (int r = first; r < q.teams; r += q.join ? g.G : q.teams)
            for (int e = e0; e < e0 + g.HW; ++e) {
                s += lds[(r * M + e) * 2];
                t += lds[(r * M + e) * 2 + 1];
            }
        row[c * 2] = s;
        row[c * 2 + 1] = t;
    }
}

}  // namespace

template <typename T>
hipError_t launch_norm_res_small_fwd(const NormGeom &g, const NormResPlan &q, const void *x, const void *gamma,
                                     const void *beta, void *y, float *mean, float *rstd, hipStream_t s)
{
    constexpr int N = kVec<T>;
    return with_nv<small_vectors(N, true)>(q.NV, [&](auto nv) {
        return with_past<true>(q.past, [&](auto past) {
            constexpr int NV = decltype(nv)::value;
            constexpr bool P = decltype(past)::value;
            if (g.nhwc)
                hipLaunchKernelGGL((res_small_fwd<T, N, NV, true, P>), dim3(unsigned(q.grid)), dim3(q.threads), 0, s,
                                   g, q, (const T *)x, gamma, beta, (T *)y, mean, rstd);
            else if constexpr (NV <= small_vectors(N, false))
                hipLaunchKernelGGL((res_small_fwd<T, N, NV, false, P>), dim3(unsigned(q.grid)), dim3(q.threads), 0, s,
                                   g, q, (const T *)x, gamma, beta, (T *)y, mean, rstd);
            else
                return hipErrorInvalidValue;
            return hipGetLastError();
        });
    });
}

template <typename T>
hipError_t launch_norm_res_small_bwd(const NormGeom &g, const NormResPlan &q, const void *x, const void *gamma,
                                     const void *beta, const void *dy, const float *mean, const float *rstd, void *dx,
                                     float *part, hipStream_t s)
{
    constexpr int N = kVec<T>;
    return with_nv<small_vectors(N, false)>(q.NV, [&](auto nv) {
        return with_past<true>(q.past, [&](auto past) {
            hipLaunchKernelGGL((res_small_bwd<T, N, decltype(nv)::value, decltype(past)::value>), dim3(unsigned(q.grid)),
                               dim3(q.threads), q.lds_bytes, s, g, q, (const T *)x, (const T *)dy, gamma, beta, mean,
                               rstd, (T *)dx, part);
            return hipGetLastError();
        });
    });
}

#define GC_RES_SMALL(T)                                                                                              \
    template hipError_t launch_norm_res_small_fwd<T>(const NormGeom &, const NormResPlan &, const void *,            \
                                                     const void *, const void *, void *, float *, float *, hipStream_t); \
    template hipError_t launch_norm_res_small_bwd<T>(const NormGeom &, const NormResPlan &, const void *,            \
                                                     const void *, const void *, const void *, const float *,        \
                                                     const float *, void *, float *, hipStream_t);
GC_RES_SMALL(float)
GC_RES_SMALL(bf16_t)

}  // namespace gc
