// norm_res_nchw.hip -- group norm with an activation over NCHW tensors, for
// groups that fit the registers of one team of threads.
//
// A group's M = Cg*HW elements are contiguous.  A team of L threads (a power
// of two; below a wave several teams share one) reads them as vectors
// lane, lane + L, ..., holds them, and needs no second pass over memory.  Two
// vector shapes: N divides HW, so a vector lies in one channel; or HW >= N and a
// vector meets at most two channels, the last one of the group being moved
// back to end with it (its first `skip` elements are another vector's).
//
// The forward takes the mean, then the squares around it (with the remaining
// sum, so the mean's own rounding drops out).  The backward's team keeps its
// group's channel constants, walks images slot, slot + slots, ..., and adds
// each vector's g and g*hat to running sums of its own; only after its last
// image are those added up by channel, in LDS, into one row of partials a slot.
// Bound by memory where the call is large: 32,768 x 128 x 3 x 4 bf16 forward 38 us (5.3 TB/s),
// backward 52 (5.9), 300 x 32 x 32 x 32 fp32 forward 13.4 (5.9).  1024 x 128 x 3 x 4 is one round
// of loads and two dependent sums: fp32 forward 5.7 us for 13 MB, bf16 backward 6.7 for 11.
#include <type_traits>

#include "gc_norm_res.h"

namespace gc {
namespace {

template <int N, bool TWO>
struct Where {
    int at;       // first element in the group
    int c;        // its channel in the group
    int cut;      // TWO: elements before `cut` are channel c, the others c + 1
    int skip;     // TWO: leading elements that another vector holds
};

template <int N, bool TWO>
__device__ __forceinline__ Where<N, TWO> where(const NormGeom &g, int idx, int M)
{
    Where<N, TWO> w;
    w.at = TWO ? min(idx * N, M - N) : idx * N;
    w.skip = idx * N - w.at;
    w.c = int(fdiv(uint32_t(w.at), g.fd_HW));
    w.cut = (w.c + 1) * g.HW - w.at;
    return w;
}

// value of a vector's element j from those of its two channels
template <bool TWO>
__device__ __forceinline__ float pick(const float (&v)[2], int j, int cut)
{
    return TWO && j >= cut ? v[1] : v[0];
}

template <typename T, int N, int NV, bool TWO, bool PAST>
__global__ void __launch_bounds__(res_threads_fwd(N * NV))
    res_nchw_fwd(NormGeom g, NormResPlan q, const T *__restrict__ x, const void *__restrict__ gamma,
                 const void *__restrict__ beta, T *__restrict__ y, float *__restrict__ mean_out,
                 float *__restrict__ rstd_out)
{
    __shared__ float red[32];
    const int64_t block = blockIdx.x;
    const int lane = threadIdx.x & (q.L - 1);
    const int M = g.Cg * g.HW, nvec = (M + N - 1) / N;
    const int64_t k = block * q.teams + threadIdx.x / q.L;
    const bool live = k < int64_t(g.B) * g.G;
    const T *xp = x + k * M;
    Vec<T, N> v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int idx = lane + i * q.L;
        if (live && idx < nvec) v[i] = load_vec<T, N>(xp + (TWO ? min(idx * N, M - N) : idx * N));
        else v[i] = Vec<T, N>{};
    }
    float s[1] = {};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int idx = lane + i * q.L;
        const int skip = TWO && idx == nvec - 1 ? nvec * N - M : 0;
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (!TWO || j >= skip) s[0] += v[i].get(j);
    }
    team_sum(s, q.L, red);
    keep_packed(v);
    const float n = 1.f / float(M), m0 = s[0] * n;
    float t[2] = {};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int idx = lane + i * q.L;
        const int skip = TWO && idx == nvec - 1 ? nvec * N - M : 0;
        if (idx >= nvec) continue;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (TWO && j < skip) continue;
            const float d = v[i].get(j) - m0;
            t[0] += d;
            t[1] = fmaf(d, d, t[1]);
        }
    }
    team_sum(t, q.L, red);
    keep_packed(v);
    if (!live) return;
    const float off = t[0] * n, mean = m0 + off;
    const float var = fmaxf(fmaf(-off, off, t[1] * n), 0.f);
    const float rstd = t[1] != t[1] ? t[1] : 1.f / sqrtf(var + g.eps);
    if (lane == 0) {
        if (mean_out) mean_out[k] = mean;
        if (rstd_out) rstd_out[k] = rstd;
    }
    const int c0 = int(k % g.G) * g.Cg;
    T *yp = y + k * M;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int idx = lane + i * q.L;
        if (idx >= nvec) continue;
        const Where<N, TWO> w = where<N, TWO>(g, idx, M);
        float a[2], b[2], z[N];
        a[0] = param<T>(g, gamma, c0 + w.c, 1.f);
        b[0] = param<T>(g, beta, c0 + w.c, 0.f);
        if (TWO && w.cut < N) {
            a[1] = param<T>(g, gamma, c0 + w.c + 1, 1.f);
            b[1] = param<T>(g, beta, c0 + w.c + 1, 0.f);
        } else {
            a[1] = a[0];
            b[1] = b[0];
        }
#pragma unroll
        for (int j = 0; j < N; ++j)
            z[j] = norm_z(v[i].get(j), mean, rstd, pick<TWO>(a, j, w.cut), pick<TWO>(b, j, w.cut));
        activate(g.act, z);
        Vec<T, N> o;
        o.put(z);
        put_vec<PAST>(yp + w.at, o);
    }
}

template <typename T, int N, int NV, bool TWO, bool PAST>
__global__ void __launch_bounds__(res_threads_bwd(N * NV))
    res_nchw_bwd(NormGeom g, NormResPlan q, const T *__restrict__ x, const T *__restrict__ dy,
                 const void *__restrict__ gamma, const void *__restrict__ beta, const float *__restrict__ mean,
                 const float *__restrict__ rstd, T *__restrict__ dx, float *__restrict__ part)
{
    constexpr int NC = TWO ? 2 : 1;   // channels of a vector
    extern __shared__ float lds[];
    const int lane = threadIdx.x & (q.L - 1), team = threadIdx.x / q.L;
    const int64_t unit = int64_t(blockIdx.x) * q.teams + team;   // (slot, group)
    const int gg = int(unit % g.G);
    const int slot = int(unit / g.G);
    const int M = g.Cg * g.HW, nvec = (M + N - 1) / N;
    const float n = 1.f / float(M);

    float a[NV][2], b[NV][2], sg[NV][NC] = {}, st[NV][NC] = {};
    Where<N, TWO> w[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int idx = min(lane + i * q.L, nvec - 1);
        w[i] = where<N, TWO>(g, idx, M);
        const int c = gg * g.Cg + w[i].c;
        a[i][0] = param<T>(g, gamma, c, 1.f);
        b[i][0] = param<T>(g, beta, c, 0.f);
        const int c1 = TWO && w[i].cut < N ? c + 1 : c;
        a[i][1] = TWO ? param<T>(g, gamma, c1, 1.f) : a[i][0];
        b[i][1] = TWO ? param<T>(g, beta, c1, 0.f) : b[i][0];
    }
    // the teams of a workgroup larger than a wave are one: its trips are uniform
    for (int img = slot < q.images ? slot : g.B; img < g.B; img += q.images) {
        const int64_t k = int64_t(img) * g.G + gg;
        const T *xp = x + k * M, *dp = dy + k * M;
        const float m[1] = {mean[k]}, r[1] = {rstd[k]};
        float h[NV][N], d[NV][N];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Vec<T, N> vx{}, vd{};
            if (lane + i * q.L < nvec) {
                vx = load_vec<T, N>(xp + w[i].at);
                vd = load_vec<T, N>(dp + w[i].at);
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
            if (lane + i * q.L >= nvec) continue;
            if constexpr (TWO) {
                float ma[N], ra[N], ga[N], ba[N];
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    ma[j] = m[0];
                    ra[j] = r[0];
                    ga[j] = pick<TWO>(a[i], j, w[i].cut);
                    ba[j] = pick<TWO>(b[i], j, w[i].cut);
                }
                act_grad<N, N>(g.act, h[i], d[i], ma, ra, ga, ba);
            } else {
                const float ga[1] = {a[i][0]}, ba[1] = {b[i][0]};
                act_grad<N, 1>(g.act, h[i], d[i], m, r, ga, ba);
            }
            float s[2] = {}, t[2] = {};
#pragma unroll
            for (int j = 0; j < N; ++j) {
                if (TWO && j < w[i].skip) continue;
                const bool hi = TWO && j >= w[i].cut;
                const float p = d[i][j] * h[i][j];
                if (TWO) {
                    s[0] += hi ? 0.f : d[i][j];
                    t[0] += hi ? 0.f : p;
                    s[1] += hi ? d[i][j] : 0.f;
                    t[1] += hi ? p : 0.f;
                } else {
                    s[0] += d[i][j];
                    t[0] = fmaf(d[i][j], h[i][j], t[0]);
                }
            }
#pragma unroll
            for (int e = 0; e < NC; ++e) {
                sg[i][e] += s[e];
                st[i][e] += t[e];
                c[0] = fmaf(a[i][e], s[e], c[0]);
                c[1] = fmaf(a[i][e], t[e], c[1]);
            }
        }
        team_sum(c, q.L, lds);
        const float c1 = c[0] * n, c2 = c[1] * n;
        T *op = dx + k * M;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (lane + i * q.L >= nvec) continue;
            float o[N];
#pragma unroll
            for (int j = 0; j < N; ++j)
                o[j] = r[0] * (fmaf(pick<TWO>(a[i], j, w[i].cut), d[i][j], -c1) - h[i][j] * c2);
            Vec<T, N> ov;
            ov.put(o);
            put_vec<PAST>(op + w[i].at, ov);
        }
    }
    if (!part) return;
    // a channel's vectors start at its first element or after: lo[v] is what vector
    // v holds of its first channel, hi[v] of its second
    __syncthreads();
    float *mine = lds + team * nvec * 2 * NC;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int idx = lane + i * q.L;
        if (idx >= nvec) continue;
#pragma unroll
        for (int e = 0; e < NC; ++e) {
            mine[(idx * NC + e) * 2] = sg[i][e];
            mine[(idx * NC + e) * 2 + 1] = st[i][e];
        }
    }
    __syncthreads();
    if (slot >= q.images) return;
    const int sub = lane & (q.P - 1);
    for (int c = lane / q.P; c < g.Cg; c += q.L / q.P) {
        const int v0 = (c * g.HW + N - 1) / N;
        const int v1 = min(((c + 1) * g.HW + N - 1) / N, nvec);
        float s = 0, t = 0;
        for (int v = v0 + sub; v < v1; v += q.P) {
            s += mine[v * NC * 2];
            t += mine[v * NC * 2 + 1];
        }
        if (TWO && sub == 0 && c * g.HW % N) {
            const int v = c * g.HW / N;
            s += mine[(v * NC + 1) * 2];
            t += mine[(v * NC + 1) * 2 + 1];
        }
        s = lanes_sum(s, q.P);
        t = lanes_sum(t, q.P);
        if (sub == 0) {
            float *o = part + (int64_t(slot) * g.C + gg * g.Cg + c) * 2;
            o[0] = s;
            o[1] = t;
        }
    }
}

}  // namespace

template <typename T>
hipError_t launch_norm_res_nchw_fwd(const NormGeom &g, const NormResPlan &q, const void *x, const void *gamma,
                                    const void *beta, void *y, float *mean, float *rstd, hipStream_t s)
{
    return with_n<T>(q.N, [&](auto n) {
        return with_nv<16>(q.NV, [&](auto nv) {
            constexpr int N = decltype(n)::value, NV = decltype(nv)::value;
            return with_past<(sizeof(T) * N >= 8)>(q.past, [&](auto past) {
            constexpr bool P = decltype(past)::value;
            if (q.two) {
                if constexpr (N == kVec<T>)
                    hipLaunchKernelGGL((res_nchw_fwd<T, N, NV, true, P>), dim3(unsigned(q.grid)), dim3(q.threads), 0, s, g, q, (const T *)x, gamma, beta, (T *)y, mean, rstd);
                else
                    return hipErrorInvalidValue;
            } else {
                hipLaunchKernelGGL((res_nchw_fwd<T, N, NV, false, P>), dim3(unsigned(q.grid)), dim3(q.threads), 0, s, g, q, (const T *)x, gamma, beta, (T *)y, mean, rstd);
            }
            return hipGetLastError();
            });
        });
    });
}

template <typename T>
hipError_t launch_norm_res_nchw_bwd(const NormGeom &g, const NormResPlan &q, const void *x, const void *gamma,
                                    const void *beta, const void *dy, const float *mean, const float *rstd, void *dx,
                                    float *part, hipStream_t s)
{
    return with_n<T>(q.N, [&](auto n) {
        return with_nv<(decltype(n)::value > 1 ? kHeldMost / decltype(n)::value : 16)>(q.NV, [&](auto nv) {
            constexpr int N = decltype(n)::value, NV = decltype(nv)::value;
            return with_past<(sizeof(T) * N >= 8)>(q.past, [&](auto past) {
            constexpr bool P = decltype(past)::value;
            if (q.two) {
                if constexpr (N == kVec<T>)
                    hipLaunchKernelGGL((res_nchw_bwd<T, N, NV, true, P>), dim3(unsigned(q.grid)), dim3(q.threads), q.lds_bytes, s, g, q, (const T *)x, (const T *)dy, gamma, beta, mean, rstd,
                                       (T *)dx, part);
                else
                    return hipErrorInvalidValue;
            } else {
                hipLaunchKernelGGL((res_nchw_bwd<T, N, NV, false, P>), dim3(unsigned(q.grid)), dim3(q.threads), q.lds_bytes, s, g, q, (const T *)x, (const T *)dy, gamma, beta, mean, rstd,
                                   (T *)dx, part);
            }
            return hipGetLastError();
            });
        });
    });
}

#define GC_RES_NCHW(T)                                                                                              \
    template hipError_t launch_norm_res_nchw_fwd<T>(const NormGeom &, const NormResPlan &, const void *, const void *, \
                                                    const void *, void *, float *, float *, hipStream_t);           \
    template hipError_t launch_norm_res_nchw_bwd<T>(const NormGeom &, const NormResPlan &, const void *, const void *, \
                                                    const void *, const void *, const float *, const float *, void *, \
                                                    float *, hipStream_t);
GC_RES_NCHW(float)
GC_RES_NCHW(bf16_t)

}  // namespace gc
