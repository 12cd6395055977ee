// norm_res_nhwc.hip -- group norm with an activation over channels-last tensors,
// for images (or slabs of whole groups of an image's channels) that fit the
// registers of one team of threads.
//
// A team is one wave or a workgroup.  Thread (slot, col) owns the N channels of
// vector col of the slab and holds positions slot, slot + slots, ..., so its
// channel constants stay in registers and a row is read by neighbouring threads.
// Group sums go through LDS: one entry a thread where a vector lies in one
// group (kOne), else one for each of its channels (kMixed), added up by P lanes a
// group in a fixed order.  A slab that is one group need not be whole vectors wide: the
// last one of a row is moved back to end with it (kTail; its first `skip` elements are
// another vector's).  The forward takes the mean, then the squares around it (with
// the remaining sum, so the mean's own rounding drops out).  The backward's
// team walks images slot, slot + images, ..., keeping the channels' running sums of g
// and g*hat in registers; the teams of a workgroup join them at the end into one
// row of partials.  Bound by memory: 32,768 x 128 x 3 x 4 bf16 backward 57 us (5.4 TB/s), 1000 x 64
// x 11 x 15 fp32 forward 15 us (5.8 TB/s); with few large images by the 64-byte rows of their
// slabs (16 x 256 x 64 x 64 bf16 forward 22 us, 3.1 TB/s); where vectors mix groups or end inside
// them by the sums of single channels in LDS (1000 x 59 x 11 x 15 in one group, bf16 backward 29 us
// for 59 MB).
#include <type_traits>

#include "gc_norm_res.h"

namespace gc {
namespace {

enum { kMixed, kOne, kTail };

struct Place {
    int tt, team, slot, col, c;   // thread of the team, team, row slot, vector, first channel
    int skip;                     // kTail: leading elements that another vector holds
    bool live;
};

template <int N, int MIX>
__device__ __forceinline__ Place place(const NormResPlan &q, int slab)
{
    Place p;
    p.team = threadIdx.x / q.L;
    p.tt = threadIdx.x - p.team * q.L;
    uint32_t s, c;
    fdivmod(uint32_t(p.tt), q.fd_cols, s, c);
    p.slot = int(s);
    p.col = int(c);
    p.live = p.slot < q.slots;
    const int at = p.live ? MIX == kTail ? min(p.col * N, q.CW - N) : p.col * N : 0;
    p.skip = MIX == kTail && p.live ? p.col * N - at : 0;
    p.c = slab * q.CW + at;
    return p;
}

template <typename T, int N, int NV, int MIX, bool PAST>
__global__ void __launch_bounds__(res_threads_fwd(N * NV))
    res_nhwc_fwd(NormGeom g, NormResPlan q, const T *__restrict__ x, const void *__restrict__ gamma,
                 const void *__restrict__ beta, T *__restrict__ y, float *__restrict__ mean_out,
                 float *__restrict__ rstd_out)
{
    extern __shared__ float lds[];
    const int64_t block = q.slabs > 1 ? die_order(blockIdx.x, gridDim.x) : blockIdx.x;
    constexpr bool ONE = MIX != kMixed;
    constexpr int E = ONE ? 1 : N;
    const int64_t unit = block * q.teams + threadIdx.x / q.L;   // (image, slab)
    const int slab = int(unit % q.slabs);
    const int64_t b = unit / q.slabs;
    const Place p = place<N, MIX>(q, slab);
    const bool live = p.live && b < g.B;
    float *red = lds + p.team * q.team_lds, *stat = red + 2 * q.slots * q.width;
    const T *xp = x + b * g.img + p.c;
    Vec<T, N> v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int row = p.slot + i * q.slots;
        if (live && row < g.HW) v[i] = load_vec<T, N>(xp + int64_t(row) * g.C);
        else v[i] = Vec<T, N>{};
    }
    float a[N], be[N];
    int ge[E];   // groups of the thread's entries, within the slab
#pragma unroll
    for (int e = 0; e < E; ++e) ge[e] = int(fdiv(uint32_t(p.c + e), g.fd_Cg)) - slab * q.Gs;
    near_params<N, T>(g, gamma, p.c, 1.f, a);
    near_params<N, T>(g, beta, p.c, 0.f, be);

    const float n = 1.f / (float(g.Cg) * float(g.HW));
    float m0[E], mean[E], rstd[E];
    {
        float s[1][E] = {};
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (MIX != kTail || j >= p.skip) s[0][ONE ? 0 : j] += v[i].get(j);
        team_groups<1, E>(q, p.live, p.tt, p.slot, p.col, s, red, stat);
#pragma unroll
        for (int e = 0; e < E; ++e) m0[e] = stat[ge[e]] * n;
    }
    keep_packed(v);
    {
        float s[2][E] = {};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (p.slot + i * q.slots >= g.HW) continue;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                if (MIX == kTail && j < p.skip) continue;
                const float d = v[i].get(j) - m0[ONE ? 0 : j];
                s[0][ONE ? 0 : j] += d;
                s[1][ONE ? 0 : j] = fmaf(d, d, s[1][ONE ? 0 : j]);
            }
        }
        team_groups<2, E>(q, p.live, p.tt, p.slot, p.col, s, red, stat);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float off = stat[ge[e]] * n, sq = stat[q.Gs + ge[e]];
            mean[e] = m0[e] + off;
            const float var = fmaxf(fmaf(-off, off, sq * n), 0.f);
            rstd[e] = sq != sq ? sq : 1.f / sqrtf(var + g.eps);
        }
    }
    keep_packed(v);
    if (!live) return;
    // the thread with a group's first channel in the first row writes its statistics
    if (p.slot == 0) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int64_t k = b * g.G + slab * q.Gs + ge[e];
            if (int(slab * q.Gs + ge[e]) * g.Cg != p.c + e) continue;
            if (mean_out) mean_out[k] = mean[e];
            if (rstd_out) rstd_out[k] = rstd[e];
        }
    }
    T *yp = y + b * g.img + p.c;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int row = p.slot + i * q.slots;
        if (row >= g.HW) continue;
        float z[N];
#pragma unroll
        for (int j = 0; j < N; ++j) z[j] = norm_z(v[i].get(j), mean[ONE ? 0 : j], rstd[ONE ? 0 : j], a[j], be[j]);
        activate(g.act, z);
        Vec<T, N> o;
        o.put(z);
        put_vec<PAST>(yp + int64_t(row) * g.C, o);
    }
}

template <typename T, int N, int NV, int MIX, bool PAST>
__global__ void __launch_bounds__(res_threads_bwd(N * NV))
    res_nhwc_bwd(NormGeom g, NormResPlan q, const T *__restrict__ x, const T *__restrict__ dy,
                 const void *__restrict__ gamma, const void *__restrict__ beta, const float *__restrict__ mean,
                 const float *__restrict__ rstd, T *__restrict__ dx, float *__restrict__ part)
{
    constexpr bool ONE = MIX != kMixed;
    constexpr int E = ONE ? 1 : N;
    extern __shared__ float lds[];
    // a workgroup: one slab, `teams` image slots
    const uint32_t id = q.slabs > 1 ? die_order(blockIdx.x, gridDim.x) : blockIdx.x;
    const int slab = int(id % q.slabs);
    const int row0 = int(id / q.slabs);
    const Place p = place<N, MIX>(q, slab);
    const int first = row0 * q.teams + p.team;
    float *red = lds + p.team * q.team_lds, *stat = red + 2 * q.slots * q.width;
    float a[N], be[N], sg[N] = {}, st[N] = {};
    int ge[E];
#pragma unroll
    for (int e = 0; e < E; ++e) ge[e] = int(fdiv(uint32_t(p.c + e), g.fd_Cg)) - slab * q.Gs;
    near_params<N, T>(g, gamma, p.c, 1.f, a);
    near_params<N, T>(g, beta, p.c, 0.f, be);
    const float n = 1.f / (float(g.Cg) * float(g.HW));
    // a team that is a workgroup makes uniform trips; one that is a wave syncs by itself
    for (int img = first; img < g.B; img += q.images) {
        const int64_t base = int64_t(img) * g.img + p.c;
        float m[N], r[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int64_t k = int64_t(img) * g.G + slab * q.Gs + ge[ONE ? 0 : j];
            if (!ONE || j == 0) {
                m[j] = mean[k];
                r[j] = rstd[k];
            } else {
                m[j] = m[0];
                r[j] = r[0];
            }
        }
        float h[NV][N], d[NV][N];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int row = p.slot + i * q.slots;
            Vec<T, N> vx{}, vd{};
            if (p.live && row < g.HW) {
                vx = load_vec<T, N>(x + base + int64_t(row) * g.C);
                vd = load_vec<T, N>(dy + base + int64_t(row) * g.C);
            }
#pragma unroll
            for (int j = 0; j < N; ++j) {
                h[i][j] = vx.get(j);
                d[i][j] = vd.get(j);
            }
        }
        float s[N] = {}, t[N] = {};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (p.slot + i * q.slots >= g.HW) continue;
            act_grad<N, N>(g.act, h[i], d[i], m, r, a, be);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                if (MIX == kTail && j < p.skip) continue;
                s[j] += d[i][j];
                t[j] = fmaf(d[i][j], h[i][j], t[j]);
            }
        }
        float c[2][E] = {};
#pragma unroll
        for (int j = 0; j < N; ++j) {
            sg[j] += s[j];
            st[j] += t[j];
            c[0][ONE ? 0 : j] = fmaf(a[j], s[j], c[0][ONE ? 0 : j]);
            c[1][ONE ? 0 : j] = fmaf(a[j], t[j], c[1][ONE ? 0 : j]);
        }
        team_groups<2, E>(q, p.live, p.tt, p.slot, p.col, c, red, stat);
        float c1[E], c2[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            c1[e] = stat[ge[e]] * n;
            c2[e] = stat[q.Gs + ge[e]] * n;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int row = p.slot + i * q.slots;
            if (!p.live || row >= g.HW) continue;
            float o[N];
#pragma unroll
            for (int j = 0; j < N; ++j)
                o[j] = r[j] * (fmaf(a[j], d[i][j], -c1[ONE ? 0 : j]) - h[i][j] * c2[ONE ? 0 : j]);
            Vec<T, N> ov;
            ov.put(o);
            put_vec<PAST>(dx + base + int64_t(row) * g.C, ov);
        }
    }
    if (!part) return;
    __syncthreads();
    if (p.live) {
        float *mine = lds + ((p.team * q.slots + p.slot) * q.CW + p.c - slab * q.CW) * 2;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (MIX == kTail && j < p.skip) continue;
            mine[2 * j] = sg[j];
            mine[2 * j + 1] = st[j];
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * q.CW; e += blockDim.x) {
        float s = 0;
        for (int r = 0; r < q.teams * q.slots; ++r) s += lds[r * q.CW * 2 + e];
        part[(int64_t(row0) * g.C + slab * q.CW) * 2 + e] = s;
    }
}

}  // namespace

template <typename T>
hipError_t launch_norm_res_nhwc_fwd(const NormGeom &g, const NormResPlan &q, const void *x, const void *gamma,
                                    const void *beta, void *y, float *mean, float *rstd, hipStream_t s)
{
    return with_n<T>(q.N, [&](auto n) {
        return with_nv<16>(q.NV, [&](auto nv) {
            constexpr int N = decltype(n)::value, NV = decltype(nv)::value;
            return with_past<(sizeof(T) * N >= 8)>(q.past, [&](auto past) {
            constexpr bool P = decltype(past)::value;
            if (q.mix == kOne) {
                hipLaunchKernelGGL((res_nhwc_fwd<T, N, NV, kOne, P>), dim3(unsigned(q.grid)), dim3(q.threads), q.lds_bytes, s,
                                   g, q, (const T *)x, gamma, beta, (T *)y, mean, rstd);
            } else if (q.mix == kTail) {
                if constexpr (N > 1)
                    hipLaunchKernelGGL((res_nhwc_fwd<T, N, NV, kTail, P>), dim3(unsigned(q.grid)), dim3(q.threads), q.lds_bytes, s,
                                   g, q, (const T *)x, gamma, beta, (T *)y, mean, rstd);
                else
                    return hipErrorInvalidValue;
            } else {
                if constexpr (N > 1 && NV <= kMixedMost)
                    hipLaunchKernelGGL((res_nhwc_fwd<T, N, NV, kMixed, P>), dim3(unsigned(q.grid)), dim3(q.threads), q.lds_bytes, s,
                                   g, q, (const T *)x, gamma, beta, (T *)y, mean, rstd);
                else
                    return hipErrorInvalidValue;
            }
            return hipGetLastError();
            });
        });
    });
}

template <typename T>
hipError_t launch_norm_res_nhwc_bwd(const NormGeom &g, const NormResPlan &q, const void *x, const void *gamma,
                                    const void *beta, const void *dy, const float *mean, const float *rstd, void *dx,
                                    float *part, hipStream_t s)
{
    return with_n<T>(q.N, [&](auto n) {
        return with_nv<kHeldMost / decltype(n)::value>(q.NV, [&](auto nv) {
            constexpr int N = decltype(n)::value, NV = decltype(nv)::value;
            return with_past<(sizeof(T) * N >= 8)>(q.past, [&](auto past) {
            constexpr bool P = decltype(past)::value;
            if (q.mix == kOne) {
                hipLaunchKernelGGL((res_nhwc_bwd<T, N, NV, kOne, P>), dim3(unsigned(q.grid)), dim3(q.threads), q.lds_bytes, s,
                                   g, q, (const T *)x, (const T *)dy, gamma, beta, mean, rstd, (T *)dx, part);
            } else if (q.mix == kTail) {
                if constexpr (N > 1)
                    hipLaunchKernelGGL((res_nhwc_bwd<T, N, NV, kTail, P>), dim3(unsigned(q.grid)), dim3(q.threads), q.lds_bytes, s,
                                   g, q, (const T *)x, (const T *)dy, gamma, beta, mean, rstd, (T *)dx, part);
                else
                    return hipErrorInvalidValue;
            } else {
                if constexpr (N > 1)
                    hipLaunchKernelGGL((res_nhwc_bwd<T, N, NV, kMixed, P>), dim3(unsigned(q.grid)), dim3(q.threads), q.lds_bytes, s,
                                   g, q, (const T *)x, (const T *)dy, gamma, beta, mean, rstd, (T *)dx, part);
                else
                    return hipErrorInvalidValue;
            }
            return hipGetLastError();
            });
        });
    });
}

#define GC_RES_NHWC(T)                                                                                              \
    template hipError_t launch_norm_res_nhwc_fwd<T>(const NormGeom &, const NormResPlan &, const void *, const void *, \
                                                    const void *, void *, float *, float *, hipStream_t);           \
    template hipError_t launch_norm_res_nhwc_bwd<T>(const NormGeom &, const NormResPlan &, const void *, const void *, \
                                                    const void *, const void *, const float *, const float *, void *, \
                                                    float *, hipStream_t);
GC_RES_NHWC(float)
GC_RES_NHWC(bf16_t)

}  // namespace gc
