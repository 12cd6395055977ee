// norm_rows.hip -- layer norm of rows, the residual stream's addition with it, and the
// backward pass with the gradients of its weights.
//
//   s = x + residual,  hat = (s - mean) * rstd,  y = gamma * hat + beta
//   w = gamma * dy,  dx = dtotal + rstd * (w - mean(w) - hat * mean(w*hat))
//   dgamma = sum over rows of dy*hat,  dbeta = sum over rows of dy
//
// Memory bound: a row is read once into the registers of a team of threads, which adds up
// its sums by lane exchanges (a team of one wave) or through LDS, and writes its outputs.  Teams
// walk rows, so gamma and beta are read once a team, and the backward's sums over rows
// stay in registers until a team's last row; its next row's loads fly while a row is
// worked on.  A second launch adds up the workgroups' sums.  Rows past a workgroup's
// registers (16,384 values forward, 8192 backward) are walked in several passes.
//
// With inputs from HBM, here and below: 32,768 rows of 1760 bf16 with a residual 88 us forward (462 MB,
// 5.2 TB/s); 8191 rows of 4096 bf16, with the stream's gradient, 60 us backward (269 MB, 4.5 TB/s) and 5 for the
// sums; 1024 rows of 1760 fp32 12.6 and 4.0 us, the latency of a row's loads, its sums, and the join.
#include <algorithm>
#include <type_traits>

#include "gc_core.h"
#include "gc_norm_res.h"

namespace gc {
namespace {

// N neighbouring values of gamma or beta in fp32.
template <typename T, int N>
__device__ __forceinline__ void params_at(const RowsGeom &g, const void *p, int at, float none, float (&v)[N])
{
    if (!p) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = none;
    } else if (g.pf32) {
        const Vec<float, N> w = load_vec<float, N>(static_cast<const float *>(p) + at);
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = w.get(j);
    } else {
        const Vec<T, N> w = load_vec<T, N>(static_cast<const T *>(p) + at);
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = w.get(j);
    }
}

// Sums over the L threads of a team, the same value for all: lanes of a wave, or whole
// waves of a workgroup that may hold several such teams (`red` 16*K values, which the next call must
// not use: it may begin before all have read them).
template <int K>
__device__ __forceinline__ void rows_sum(float (&v)[K], int L, float *red)
{
    const int w = L < 64 ? L : 64;
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = lanes_sum(v[k], w);
    if (L <= 64) return;
    const int wave = threadIdx.x >> 6, nw = L >> 6, first = wave & ~(nw - 1);
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) red[k * 16 + wave] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float s = red[k * 16 + first];
        for (int i = 1; i < nw; ++i) s += red[k * 16 + first + i];
        v[k] = s;
    }
}

// ----------------------------------------------------------------- forward --
// The values of a row stay in fp32, 32 a thread at most.  The mean first, then the squares around
// it, so a mean far from zero costs no precision.
template <typename T, int N, int NV, bool RES, bool PAST>
__global__ void __launch_bounds__(512) rows_fwd(RowsGeom g, int L, const T *x, const T *res,
                                                 const void *__restrict__ gamma, const void *__restrict__ beta,
                                                 T *y, T *total, float *__restrict__ mean, float *__restrict__ rstd)
{
    __shared__ float red[2][16];
    const int tt = threadIdx.x & (L - 1), teams = blockDim.x / L;
    float gm[NV][N], bt[NV][N];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const Place<N> at(i * L + tt, g.D);
        params_at<T, N>(g, gamma, at.at, 1.f, gm[i]);
        params_at<T, N>(g, beta, at.at, 0.f, bt[i]);
    }
    const float inv = 1.f / float(g.D);
    // every team of a workgroup takes as many turns, for the barriers; one without a row reads the last again
    for (int64_t turn = int64_t(blockIdx.x) * teams; turn < g.rows; turn += int64_t(gridDim.x) * teams) {
        const bool own = turn + threadIdx.x / L < g.rows;
        const int64_t row = own ? turn + threadIdx.x / L : g.rows - 1;
        const T *xr = x + row * g.ld_x;
        Vec<T, N> xv[NV], rv[RES ? NV : 1];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Place<N> at(i * L + tt, g.D);
            xv[i] = load_vec<T, N>(xr + at.at);
            if (RES) rv[i] = load_vec<T, N>(res + row * g.ld_res + at.at);
        }
        float v[NV][N];
        float sum[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Place<N> at(i * L + tt, g.D);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                v[i][j] = xv[i].get(j);
                if (RES) v[i][j] += rv[i].get(j);
                sum[0] += j >= at.skip ? v[i][j] : 0.f;
            }
        }
        rows_sum<1>(sum, L, red[0]);
        const float m = sum[0] * inv;
        float sq[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Place<N> at(i * L + tt, g.D);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float off = v[i][j] - m;
                sq[0] += j >= at.skip ? off * off : 0.f;
            }
        }
        rows_sum<1>(sq, L, red[1]);
        const float r = 1.f / sqrtf(sq[0] * inv + g.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Place<N> at(i * L + tt, g.D);
            if (!at.live || !own) continue;
            Vec<T, N> out;
            if (total) {
                out.put(v[i]);
                put_own<PAST, T, N>(total + row * g.ld_total + at.at, out, at.skip);
            }
            float z[N];
#pragma unroll
            for (int j = 0; j < N; ++j) z[j] = (v[i][j] - m) * r * gm[i][j] + bt[i][j];
            out.put(z);
            put_own<PAST, T, N>(y + row * g.ld_y + at.at, out, at.skip);
        }
        if (tt == 0 && own) {
            if (mean) mean[row] = m;
            if (rstd) rstd[row] = r;
        }
    }
}

// A row past the registers: three passes over it by one workgroup.
template <typename T, int N>
__global__ void __launch_bounds__(1024) rows_fwd_loop(RowsGeom g, const T *x, const T *res,
                                                      const void *__restrict__ gamma, const void *__restrict__ beta,
                                                      T *y, T *total, float *__restrict__ mean,
                                                      float *__restrict__ rstd)
{
    __shared__ float red[16];
    const int nv = vectors(g.D, N);
    const float inv = 1.f / float(g.D);
    for (int64_t row = blockIdx.x; row < g.rows; row += gridDim.x) {
        const T *xr = x + row * g.ld_x, *rr = res ? res + row * g.ld_res : nullptr;
        auto values = [&](int at, float (&v)[N]) {
            const Vec<T, N> a = load_vec<T, N>(xr + at);
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] = a.get(j);
            if (!rr) return;
            const Vec<T, N> b = load_vec<T, N>(rr + at);
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] += b.get(j);
        };
        float sum = 0.f, sq = 0.f, v[N];
        for (int i = threadIdx.x; i < nv; i += blockDim.x) {
            const Place<N> at(i, g.D);
            values(at.at, v);
#pragma unroll
            for (int j = 0; j < N; ++j) sum += j >= at.skip ? v[j] : 0.f;
        }
        const float m = block_sum(sum, red) * inv;
        for (int i = threadIdx.x; i < nv; i += blockDim.x) {
            const Place<N> at(i, g.D);
            values(at.at, v);
#pragma unroll
            for (int j = 0; j < N; ++j) sq += j >= at.skip ? (v[j] - m) * (v[j] - m) : 0.f;
        }
        const float r = 1.f / sqrtf(block_sum(sq, red) * inv + g.eps);
        for (int i = threadIdx.x; i < nv; i += blockDim.x) {
            const Place<N> at(i, g.D);
            values(at.at, v);
            float gm[N], bt[N];
            params_at<T, N>(g, gamma, at.at, 1.f, gm);
            params_at<T, N>(g, beta, at.at, 0.f, bt);
            Vec<T, N> out;
            if (total) {
                out.put(v);
                put_own<false, T, N>(total + row * g.ld_total + at.at, out, at.skip);
            }
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] = (v[j] - m) * r * gm[j] + bt[j];
            out.put(v);
            put_own<false, T, N>(y + row * g.ld_y + at.at, out, at.skip);
        }
        if (threadIdx.x == 0) {
            if (mean) mean[row] = m;
            if (rstd) rstd[row] = r;
        }
    }
}

// ---------------------------------------------------------------- backward --
// Adds up the running sums of a workgroup's teams and writes them as one row of partials, D of dbeta's and
// D of dgamma's: teams within a wave by lane exchanges, the others in order from LDS.
template <int N, int NV>
__device__ __forceinline__ void write_part(int D, int L, float (&db)[NV][N], float (&dg)[NV][N], float *all, float *part)
{
    const int tt = threadIdx.x & (L - 1);
    for (int m = 32; m >= L; m >>= 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j) {
                db[i][j] += __shfl_xor(db[i][j], m, 64);
                dg[i][j] += __shfl_xor(dg[i][j], m, 64);
            }
    }
    const int wide = L < 64 ? 64 : L, turns = blockDim.x / wide;
    if (int(threadIdx.x) % wide < L) {
        float *to = turns > 1 ? all + int(threadIdx.x) / wide * 2 * D : part;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Place<N> at(i * L + tt, D);
            if (!at.live) continue;
            Vec<float, N> b, g;
            b.put(db[i]);
            g.put(dg[i]);
            put_own<false, float, N>(to + at.at, b, at.skip);
            put_own<false, float, N>(to + D + at.at, g, at.skip);
        }
    }
    if (turns == 1) return;
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * D; e += blockDim.x) {
        float s = all[e];
        for (int w = 1; w < turns; ++w) s += all[w * 2 * D + e];
        part[e] = s;
    }
}

// A row's inputs, as they lie in memory.
template <typename T, int N, int NV>
struct RowIn {
    Vec<T, N> x[NV], d[NV], t[NV];
    float mean, rstd;
};

// AHEAD rows' loads fly while one is worked on.
template <typename T, int N, int NV, int AHEAD, bool PAST>
__global__ void __launch_bounds__(512) rows_bwd(RowsGeom g, int L, const T *x, const void *__restrict__ gamma,
                                                const T *dy, const T *dtotal, const float *__restrict__ mean,
                                                const float *__restrict__ rstd, T *dx, float *__restrict__ part)
{
    __shared__ float red[2][32];
    extern __shared__ float joined[];
    const int tt = threadIdx.x & (L - 1), teams = blockDim.x / L, team = threadIdx.x / L;
    // every team of a workgroup takes as many turns, for the barriers; one without a row reads the last again
    auto row_of = [&](int64_t turn) { return min(turn + team, g.rows - 1); };
    auto fetch = [&](int64_t row) {
        RowIn<T, N, NV> in;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Place<N> at(i * L + tt, g.D);
            in.x[i] = load_vec<T, N>(x + row * g.ld_x + at.at);
            in.d[i] = load_vec<T, N>(dy + row * g.ld_y + at.at);
            if (dtotal) in.t[i] = load_vec<T, N>(dtotal + row * g.ld_total + at.at);
        }
        in.mean = mean[row];
        in.rstd = rstd[row];
        return in;
    };
    const int64_t stride = int64_t(gridDim.x) * teams, first = int64_t(blockIdx.x) * teams;
    RowIn<T, N, NV> next[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
        if (first + k * stride < g.rows) next[k] = fetch(row_of(first + k * stride));
    float gm[NV][N], dg[NV][N] = {}, db[NV][N] = {};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const Place<N> at(i * L + tt, g.D);
        params_at<T, N>(g, gamma, at.at, 1.f, gm[i]);
    }
    const float inv = 1.f / float(g.D);
    int half = 0;
    for (int64_t turn = first; turn < g.rows; turn += stride, half ^= 1) {
        const bool own = turn + team < g.rows;
        const int64_t row = row_of(turn);
        const RowIn<T, N, NV> in = next[0];
#pragma unroll
        for (int k = 1; k < AHEAD; ++k) next[k - 1] = next[k];
        if (turn + AHEAD * stride < g.rows) next[AHEAD - 1] = fetch(row_of(turn + AHEAD * stride));
        float c[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Place<N> at(i * L + tt, g.D);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float hat = (in.x[i].get(j) - in.mean) * in.rstd;
                const float d = own && j >= at.skip ? in.d[i].get(j) : 0.f;
                const float dh = own && j >= at.skip ? d * hat : 0.f;
                db[i][j] += d;
                dg[i][j] += dh;
                c[0] += gm[i][j] * d;
                c[1] += gm[i][j] * dh;
            }
        }
        rows_sum<2>(c, L, red[half]);
        const float c1 = c[0] * inv, c2 = c[1] * inv;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const Place<N> at(i * L + tt, g.D);
            if (!at.live || !own) continue;
            float z[N];
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float hat = (in.x[i].get(j) - in.mean) * in.rstd;
                z[j] = in.rstd * (gm[i][j] * in.d[i].get(j) - c1 - hat * c2);
                if (dtotal) z[j] += in.t[i].get(j);
            }
            Vec<T, N> out;
            out.put(z);
            put_own<PAST, T, N>(dx + row * g.ld_res + at.at, out, at.skip);
        }
    }
    if (part) write_part<N, NV>(g.D, L, db, dg, joined, part + int64_t(blockIdx.x) * 2 * g.D);
}

// dbeta and dgamma from the rows of partials: a workgroup takes 64 columns, its threads every 32nd row
// of two columns each.
constexpr int kSumCols = 64, kSumSlots = 32;
template <typename T>
__global__ void __launch_bounds__(1024) rows_params(RowsGeom g, int parts, const float *__restrict__ part,
                                                    void *__restrict__ dgamma, void *__restrict__ dbeta)
{
    __shared__ float red[kSumSlots][kSumCols];
    constexpr int U = 8;      // rows whose loads fly together
    const int col = threadIdx.x % (kSumCols / 2) * 2, slot = threadIdx.x / (kSumCols / 2);
    const int e = blockIdx.x * kSumCols + col;
    float s0 = 0.f, s1 = 0.f;
    if (e < 2 * g.D)
        for (int r = slot; r < parts; r += U * kSumSlots) {
            Vec<float, 2> v[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (r + u * kSumSlots < parts) v[u] = load_vec<float, 2>(part + int64_t(r + u * kSumSlots) * 2 * g.D + e);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (r + u * kSumSlots < parts) {
                    s0 += v[u].get(0);
                    s1 += v[u].get(1);
                }
        }
    red[slot][col] = s0;
    red[slot][col + 1] = s1;
    __syncthreads();
    const int k = blockIdx.x * kSumCols + threadIdx.x;
    if (threadIdx.x >= kSumCols || k >= 2 * g.D) return;
    float s = red[0][threadIdx.x];
#pragma unroll
    for (int i = 1; i < kSumSlots; ++i) s += red[i][threadIdx.x];
    void *to = k < g.D ? dbeta : dgamma;
    const int at = k < g.D ? k : k - g.D;
    if (!to) return;
    if (g.pf32) static_cast<float *>(to)[at] = s;
    else static_cast<T *>(to)[at] = from_f32<T>(s);
}

// Rows past the registers: the sums over rows first, by columns (dx may take dy's place),
// then dx in two passes over a row.
template <typename T>
__global__ void __launch_bounds__(256) rows_bwd_columns(RowsGeom g, const T *__restrict__ x, const T *__restrict__ dy,
                                                        const float *__restrict__ mean, const float *__restrict__ rstd,
                                                        float *__restrict__ part)
{
    const int e = blockIdx.x * 256 + threadIdx.x;
    if (e >= g.D) return;
    float db = 0.f, dg = 0.f;
    for (int64_t row = blockIdx.y; row < g.rows; row += gridDim.y) {
        const float d = to_f32(dy[row * g.ld_y + e]);
        db += d;
        dg += d * ((to_f32(x[row * g.ld_x + e]) - mean[row]) * rstd[row]);
    }
    float *to = part + int64_t(blockIdx.y) * 2 * g.D + e;
    to[0] = db;
    to[g.D] = dg;
}

template <typename T, int N>
__global__ void __launch_bounds__(1024) rows_bwd_loop(RowsGeom g, const T *x, const void *__restrict__ gamma,
                                                      const T *dy, const T *dtotal, const float *__restrict__ mean,
                                                      const float *__restrict__ rstd, T *dx)
{
    __shared__ float red[32];
    const int nv = vectors(g.D, N);
    const float inv = 1.f / float(g.D);
    for (int64_t row = blockIdx.x; row < g.rows; row += gridDim.x) {
        const T *xr = x + row * g.ld_x, *dr = dy + row * g.ld_y;
        const float m = mean[row], r = rstd[row];
        float c[2] = {0.f, 0.f}, gm[N];
        for (int i = threadIdx.x; i < nv; i += blockDim.x) {
            const Place<N> at(i, g.D);
            params_at<T, N>(g, gamma, at.at, 1.f, gm);
            const Vec<T, N> xv = load_vec<T, N>(xr + at.at), dv = load_vec<T, N>(dr + at.at);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float w = j >= at.skip ? gm[j] * dv.get(j) : 0.f;
                c[0] += w;
                c[1] += j >= at.skip ? w * ((xv.get(j) - m) * r) : 0.f;
            }
        }
        rows_sum<2>(c, 1024, red);
        __syncthreads();
        const float c1 = c[0] * inv, c2 = c[1] * inv;
        for (int i = threadIdx.x; i < nv; i += blockDim.x) {
            const Place<N> at(i, g.D);
            params_at<T, N>(g, gamma, at.at, 1.f, gm);
            const Vec<T, N> xv = load_vec<T, N>(xr + at.at), dv = load_vec<T, N>(dr + at.at);
            float z[N];
#pragma unroll
            for (int j = 0; j < N; ++j) z[j] = r * (gm[j] * dv.get(j) - c1 - (xv.get(j) - m) * r * c2);
            if (dtotal) {
                const Vec<T, N> tv = load_vec<T, N>(dtotal + row * g.ld_total + at.at);
#pragma unroll
                for (int j = 0; j < N; ++j) z[j] += tv.get(j);
            }
            Vec<T, N> out;
            out.put(z);
            put_own<false, T, N>(dx + row * g.ld_res + at.at, out, at.skip);
        }
    }
}

constexpr int kFwdHeld = 32, kBwdHeld = 16;   // values of a row that a thread holds, at most

// Calls f(N, NV) with the plan's vector as compile-time constants.
template <typename T, int MOST, typename F>
hipError_t with_vectors(const RowsPlan &q, F f)
{
    if (q.N == 1) return f(std::integral_constant<int, 1>(), std::integral_constant<int, 1>());
    return with_nv<MOST / kVec<T>>(q.NV, [&](auto nv) { return f(std::integral_constant<int, kVec<T>>(), nv); });
}

}  // namespace

void plan_rows(const RowsGeom &g, int dtype, bool bwd, bool more, RowsPlan &q)
{
    q = RowsPlan{};
    const int vec = dtype == GC_F32 ? 4 : 8, held = bwd ? kBwdHeld : kFwdHeld;
    const int threads = 512;
    q.N = g.D < vec ? 1 : vec;
    const int64_t nv = vectors(g.D, q.N);
    const int most = q.N == 1 ? 1 : held / vec;
    q.loop = nv > int64_t(threads) * most;
    const int64_t rows = std::max<int64_t>(1, g.rows);
    if (q.loop) {
        q.N = vec;
        q.NV = 1;
        q.L = q.threads = 1024;
        q.grid = std::min<int64_t>(rows, 4 * kCUs);
        q.parts = std::min<int64_t>(rows, 64);
    } else {
        // The smallest team that holds a row; while there are fewer teams than the chip takes, twice the threads.
        // The backward's workgroups are one a CU: with two, twice the rows of partial sums cost more than the
        // overlap gains (8191 x 4096 bf16 72 us against 63).
        q.L = 1;
        while (int64_t(q.L) * most < nv) q.L *= 2;
        while (q.L < threads && q.L < nv && rows * q.L < 1024 * kCUs / 4) q.L *= 2;
        q.NV = int((nv + q.L - 1) / q.L);
        while (!(q.NV <= 4 || q.NV == 8)) ++q.NV;   // the instances there are
        q.threads = bwd ? 512 : std::max(256, q.L);
        const int teams = q.threads / q.L;
        q.grid = std::min<int64_t>((rows + teams - 1) / teams, bwd ? kCUs * 512 / q.threads : kCUs * 2048 / q.threads);
        q.parts = q.grid;
        const int turns = q.threads / std::max(64, q.L);
        q.lds_bytes = bwd && turns > 1 ? size_t(turns) * g.D * 8 : 0;
    }
    const size_t bytes = size_t(rows) * g.D * (dtype == GC_F32 ? 4 : 2) * ((bwd ? 3 : 2) + (more ? (bwd ? 1 : 2) : 0));
    q.past = !q.loop && q.N > 1 && bytes >= kStreamBytes;
    q.ws_bytes = bwd ? (size_t(q.parts) * g.D * 8 + 255) & ~size_t(255) : 0;
}

template <typename T>
hipError_t launch_rows_fwd(const RowsGeom &g, const RowsPlan &q, const void *x, const void *res, const void *gamma,
                           const void *beta, void *y, void *total, float *mean, float *rstd, hipStream_t s)
{
    const T *xt = static_cast<const T *>(x), *rt = static_cast<const T *>(res);
    T *yt = static_cast<T *>(y), *tt = static_cast<T *>(total);
    if (q.loop) {
        hipLaunchKernelGGL((rows_fwd_loop<T, kVec<T>>), dim3(unsigned(q.grid)), dim3(q.threads), 0, s, g, xt, rt, gamma,
                           beta, yt, tt, mean, rstd);
        return hipGetLastError();
    }
    return with_vectors<T, kFwdHeld>(q, [&](auto n, auto nv) {
        constexpr int N = decltype(n)::value, NV = decltype(nv)::value;
        auto go = [&](auto r) {
            return with_past<(N > 1)>(q.past, [&](auto past) {
                hipLaunchKernelGGL((rows_fwd<T, N, NV, decltype(r)::value, decltype(past)::value>), dim3(unsigned(q.grid)),
                                   dim3(q.threads), 0, s, g, q.L, xt, rt, gamma, beta, yt, tt, mean, rstd);
                return hipGetLastError();
            });
        };
        return rt ? go(std::true_type()) : go(std::false_type());
    });
}

template <typename T>
hipError_t launch_rows_bwd(const RowsGeom &g, const RowsPlan &q, const void *x, const void *gamma, const void *dy,
                           const void *dtotal, const float *mean, const float *rstd, void *dx, void *dgamma,
                           void *dbeta, float *part, hipStream_t s)
{
    const T *xt = static_cast<const T *>(x), *dt = static_cast<const T *>(dy), *tt = static_cast<const T *>(dtotal);
    T *out = static_cast<T *>(dx);
    const bool sums = dgamma || dbeta;
    if (g.rows) {
        hipError_t e;
        if (q.loop) {
            if (sums) {
                hipLaunchKernelGGL((rows_bwd_columns<T>), dim3(unsigned((g.D + 255) / 256), unsigned(q.parts)), dim3(256), 0,
                                   s, g, xt, dt, mean, rstd, part);
                if (e = hipGetLastError(); e != hipSuccess) return e;
            }
            hipLaunchKernelGGL((rows_bwd_loop<T, kVec<T>>), dim3(unsigned(q.grid)), dim3(q.threads), 0, s, g, xt, gamma, dt,
                               tt, mean, rstd, out);
            e = hipGetLastError();
        } else {
            e = with_vectors<T, kBwdHeld>(q, [&](auto n, auto nv) {
                constexpr int N = decltype(n)::value, NV = decltype(nv)::value;
                auto go = [&](auto ahead) {
                    return with_past<(N > 1)>(q.past, [&](auto past) {
                        hipLaunchKernelGGL((rows_bwd<T, N, NV, decltype(ahead)::value, decltype(past)::value>),
                                           dim3(unsigned(q.grid)), dim3(q.threads), q.lds_bytes, s, g, q.L, xt, gamma, dt, tt,
                                           mean, rstd, out, sums ? part : nullptr);
                        return hipGetLastError();
                    });
                };
                // Two rows ahead where registers allow it and teams of several waves wait for each other: 8191 x 4096
                // bf16 62.9 us, with one 70.3; teams within a wave lose by it (65,536 x 256 34.0 and 33.1).
                if constexpr (NV * N * sizeof(T) == 32 && N > 1)
                    if (q.L > 64) return go(std::integral_constant<int, 2>());
                return go(std::integral_constant<int, 1>());
            });
        }
        if (e != hipSuccess) return e;
    }
    if (!sums) return hipSuccess;
    hipLaunchKernelGGL((rows_params<T>), dim3(unsigned((2 * g.D + kSumCols - 1) / kSumCols)), dim3(1024), 0, s, g,
                       g.rows ? int(q.parts) : 0, part, dgamma, dbeta);
    return hipGetLastError();
}

#define GC_ROWS_INSTANCES(T)                                                                                          \
    template hipError_t launch_rows_fwd<T>(const RowsGeom &, const RowsPlan &, const void *, const void *, const void *, \
                                           const void *, void *, void *, float *, float *, hipStream_t);               \
    template hipError_t launch_rows_bwd<T>(const RowsGeom &, const RowsPlan &, const void *, const void *, const void *, \
                                           const void *, const float *, const float *, void *, void *, void *, float *, \
                                           hipStream_t);
GC_ROWS_INSTANCES(float)
GC_ROWS_INSTANCES(bf16_t)

}  // namespace gc
