// norm_split.hip -- group norm with an activation, forward and backward, for
// groups too large to stay on one compute unit: three launches each.
//
//   1. channel sums over a chunk of positions, partial[image][chunk][channel]:
//      forward (x, x^2) in fp64, so that the variance can be a difference of two large
//      sums; fp64 is entered once for the kUnroll vectors that a thread has in flight, summed
//      in fp32 around their mean.  Around the first of 32 vectors' values the time is the same
//      within 5 % (64 x 64 x 128 x 128 fp32 135 us, 16 x 320 x 64 x 64 channels last bf16 35),
//      but a first value far from the others put 3e-5 on rstd.  Backward (g, g*hat) in fp32;
//   2. per (image, group) the statistics (forward: mean, rstd; backward: c1, c2),
//      one workgroup each, and for the backward dgamma and dbeta, one workgroup for 4
//      channels, all in fixed orders;
//   3. the elementwise pass over the same chunks.
//
// Work in 1 and 3 is laid out by channels.  NCHW: a wave walks positions of one
// channel plane.  Channels last: a thread owns the channels of one vector and
// walks positions, the threads of a row reading whole rows.  Either way the
// channel constants stay in registers.  The inputs are read twice (the second
// time from the 256 MB cache where they fit), and the middle launches take 3 to 5 us each, 11
// where one workgroup adds up a whole image (60 x 424 x 8 x 50 in one group).  30 x 64 x 72 x 72
// fp32 in 8 groups, channels last: forward 9.4, 3.3 and 14.0 us for 40, 1 and 80 MB, backward
// 15.3, 3.9, 20.2 and 5.5; 64 x 64 x 128 x 128 fp32 forward 47 (5.7 TB/s), 5 and 84 (6.4).
#include <algorithm>

#include "gc_norm.h"
#include "gc_train.h"

namespace gc {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kUnroll = 4;     // vectors a thread has in flight

// Positions [p0, p1) of image b and the channels this thread works on.
template <int N, bool NHWC>
struct Part {
    bool live;
    int c;             // channel (NHWC: the first of N)
    int p, p1, step;   // first position, end, distance between visits
    int64_t base;      // element offset of (image, channel c, position 0)
    int chunk, slot;   // NHWC: the thread's row slot
    int mine;          // NHWC: first of the N channels that no other vector holds
};

template <int N, bool NHWC>
__device__ __forceinline__ Part<N, NHWC> part_of(const NormGeom &g, const NormSplitPlan &q, int &b)
{
    Part<N, NHWC> w;
    uint32_t unit = blockIdx.x;
    const int lane = threadIdx.x & 63;
    if (NHWC) {
        // unit = (image, chunk, block of columns)
        const int block = unit % q.blocks;
        unit /= q.blocks;
        w.chunk = unit % q.chunks;
        b = unit / q.chunks;
        w.slot = threadIdx.x / q.cols;
        const int col = block * q.cols + threadIdx.x % q.cols;
        w.live = w.slot < q.slots && col * N < g.C;
        // the last vector of a row is moved back to end with it
        w.c = min(col * N, g.C - N);
        w.mine = col * N - w.c;
        w.p = w.chunk * q.len + w.slot;
        w.step = q.slots;
        w.base = int64_t(b) * g.img + w.c;
    } else {
        // a wave's unit = (image, chunk, channel)
        uint64_t k = uint64_t(unit) * kWaves + (threadIdx.x >> 6);
        w.c = int(k % g.C);
        k /= g.C;
        w.chunk = int(k % q.chunks);
        k /= q.chunks;
        w.live = k < uint64_t(g.B);
        b = int(k);
        w.slot = w.mine = 0;
        w.p = w.chunk * q.len + lane * N;
        w.step = 64 * N;
        w.base = int64_t(b) * g.img + int64_t(w.c) * g.HW;
    }
    w.p1 = min(g.HW, (w.chunk + 1) * q.len);
    return w;
}

// Elements of the vector at position p: where it starts (the last one of a
// plane is moved back to end with it) and how many leading elements an earlier
// vector already holds.  Chunks but the last are whole vectors long.
template <int N>
__device__ __forceinline__ int pulled_back(int p, int p1, int &skip)
{
    const int at = min(p, p1 - N);
    skip = p - at;
    return at;
}

// A workgroup's per-channel pairs to partial[b][chunk][c].
template <typename V, int N, bool NHWC>
__device__ __forceinline__ void write_sums(const NormGeom &g, const NormSplitPlan &q, const Part<N, NHWC> &w,
                                           int b, V (&s)[NHWC ? N : 1], V (&t)[NHWC ? N : 1], V *__restrict__ part)
{
    if (NHWC) {
        extern __shared__ char lds[];
        V *red = reinterpret_cast<V *>(lds);   // [slot][cols*N][2]
        const int width = q.cols * N;
        const int c0 = int(blockIdx.x % q.blocks) * width;
        if (w.live) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                if (j < w.mine) continue;
                const int e = (w.slot * width + w.c - c0 + j) * 2;
                red[e] = s[NHWC ? j : 0];
                red[e + 1] = t[NHWC ? j : 0];
            }
        }
        __syncthreads();
        for (int e = threadIdx.x; e < 2 * width; e += kThreads) {
            const int c = c0 + e / 2;
            if (c >= g.C) continue;
            V v = 0;
            for (int r = 0; r < q.slots; ++r) v += red[r * 2 * width + e];
            part[((int64_t(b) * q.chunks + w.chunk) * g.C + c) * 2 + e % 2] = v;
        }
    } else {
        const V a = lanes_sum(s[0], 64), d = lanes_sum(t[0], 64);
        if (w.live && (threadIdx.x & 63) == 0) {
            V *o = part + ((int64_t(b) * q.chunks + w.chunk) * g.C + w.c) * 2;
            o[0] = a;
            o[1] = d;
        }
    }
}

// ---------------------------------------------------------------- forward --
template <typename T, int N, bool NHWC>
__global__ void __launch_bounds__(kThreads) norm_stats(NormGeom g, NormSplitPlan q, const T *__restrict__ x,
                                                       double *__restrict__ part)
{
    constexpr int NC = NHWC ? N : 1;
    int b;
    const Part<N, NHWC> w = part_of<N, NHWC>(g, q, b);
    double s[NC] = {}, t[NC] = {};
    if (w.live) {
        for (int p = w.p; p < w.p1; p += kUnroll * w.step) {
            Vec<T, N> v[kUnroll];
            int skip[kUnroll];
            float n = 0;
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                skip[u] = N;   // nothing there
                v[u] = Vec<T, N>{};
                if (p + u * w.step < w.p1) {
                    skip[u] = 0;
                    const int at = NHWC ? p + u * w.step : pulled_back<N>(p + u * w.step, w.p1, skip[u]);
                    v[u] = load_vec<T, N>(x + w.base + (NHWC ? int64_t(at) * g.C : at));
                }
                n += NHWC ? (skip[u] ? 0.f : 1.f) : float(N - skip[u]);
            }
            // sum of x = n*o + fs, of x^2 = n*o^2 + 2*o*fs + ft, o the mean of these n values (or
            // nearly: its own rounding drops out).  n*o^2 is at most their sum of squares whatever
            // they are, so what fp32 rounds here is small against the sum.
            const float each = __builtin_amdgcn_rcpf(n);
            float o[NC] = {}, fs[NC] = {}, ft[NC] = {};
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
#pragma unroll
                for (int j = 0; j < N; ++j)
                    if (j >= skip[u]) o[NC == 1 ? 0 : j] = fmaf(v[u].get(j), each, o[NC == 1 ? 0 : j]);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const int e = NC == 1 ? 0 : j;
                    const float d = j < skip[u] ? 0.f : v[u].get(j) - o[e];
                    fs[e] += d;
                    ft[e] = fmaf(d, d, ft[e]);
                }
#pragma unroll
            for (int e = 0; e < NC; ++e) {
                const double od = o[e], sd = fs[e], nd = n;
                s[e] += fma(nd, od, sd);
                t[e] += fma(od, fma(nd, od, 2 * sd), double(ft[e]));
            }
        }
    }
    write_sums<double, N, NHWC>(g, q, w, b, s, t, part);
}

// One workgroup per (image, group): sums of w(c) * pair over the group's channels and
// chunks, in a fixed order.
template <typename V, typename W>
__device__ __forceinline__ void group_pair(const NormGeom &g, int chunks, const V *__restrict__ part, int64_t b,
                                           int c0, W w, V *red, V &s, V &t)
{
    s = t = 0;
    for (int i = threadIdx.x; i < chunks * g.Cg; i += kThreads) {
        uint32_t k, c;
        fdivmod(uint32_t(i), g.fd_Cg, k, c);
        const V *p = part + ((b * chunks + k) * g.C + c0 + c) * 2;
        const V v = w(c0 + int(c));
        s += v * p[0];
        t += v * p[1];
    }
    s = block_sum(s, red);
    t = block_sum(t, red);
}

__global__ void __launch_bounds__(kThreads) norm_finish(NormGeom g, int chunks, const double *__restrict__ part,
                                                        float *__restrict__ mean, float *__restrict__ rstd)
{
    __shared__ double red[16];
    const int64_t k = blockIdx.x;
    double s, t;
    group_pair(g, chunks, part, k / g.G, int(k % g.G) * g.Cg, [](int) { return 1.0; }, red, s, t);
    if (threadIdx.x == 0) {
        const double n = double(g.Cg) * g.HW, m = s / n;
        const double var = fma(-m, m, t / n);
        mean[k] = float(m);
        rstd[k] = float(1.0 / sqrt((var < 0 ? 0 : var) + double(g.eps)));
    }
}

template <typename T, int N, int NC>
__device__ __forceinline__ void channel_constants(const NormGeom &g, int b, int c, const void *gamma,
                                                  const void *beta, const float *mean, const float *rstd,
                                                  float (&cm)[NC], float (&cr)[NC], float (&cg)[NC], float (&cb)[NC])
{
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        const int64_t k = int64_t(b) * g.G + fdiv(uint32_t(c + j), g.fd_Cg);
        cm[j] = mean[k];
        cr[j] = rstd[k];
    }
    near_params<NC, T>(g, gamma, c, 1.f, cg);
    near_params<NC, T>(g, beta, c, 0.f, cb);
}

template <typename T, int N, bool NHWC, bool PAST>
__global__ void __launch_bounds__(kThreads) norm_apply(NormGeom g, NormSplitPlan q, const T *__restrict__ x,
                                                       const void *__restrict__ gamma,
                                                       const void *__restrict__ beta,
                                                       const float *__restrict__ mean,
                                                       const float *__restrict__ rstd, T *__restrict__ y)
{
    constexpr int NC = NHWC ? N : 1;
    int b;
    const Part<N, NHWC> w = part_of<N, NHWC>(g, q, b);
    if (!w.live) return;
    float cm[NC], cr[NC], cg[NC], cb[NC];
    channel_constants<T, N, NC>(g, b, w.c, gamma, beta, mean, rstd, cm, cr, cg, cb);
    for (int p = w.p; p < w.p1; p += kUnroll * w.step) {
        Vec<T, N> v[kUnroll];
        int64_t o[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int pu = p + u * w.step;
            int skip = 0;
            const int at = NHWC ? pu : pulled_back<N>(pu, w.p1, skip);
            o[u] = w.base + (NHWC ? int64_t(at) * g.C : at);
            if (pu < w.p1) v[u] = load_vec<T, N>(x + o[u]);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (p + u * w.step >= w.p1) break;
            float z[N];
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int k = NC == 1 ? 0 : j;
                z[j] = norm_z(v[u].get(j), cm[k], cr[k], cg[k], cb[k]);
            }
            activate(g.act, z);
            Vec<T, N> out;
            out.put(z);
            put_vec<PAST>(y + o[u], out);
        }
    }
}

// --------------------------------------------------------------- backward --
template <typename T, int N, bool NHWC>
__global__ void __launch_bounds__(kThreads) norm_bwd_sums(NormGeom g, NormSplitPlan q, const T *__restrict__ x,
                                                          const T *__restrict__ dy,
                                                          const void *__restrict__ gamma,
                                                          const void *__restrict__ beta,
                                                          const float *__restrict__ mean,
                                                          const float *__restrict__ rstd, float *__restrict__ part)
{
    constexpr int NC = NHWC ? N : 1;
    int b;
    const Part<N, NHWC> w = part_of<N, NHWC>(g, q, b);
    float s[NC] = {}, t[NC] = {};
    if (w.live) {
        float cm[NC], cr[NC], cg[NC], cb[NC];
        channel_constants<T, N, NC>(g, b, w.c, gamma, beta, mean, rstd, cm, cr, cg, cb);
        for (int p = w.p; p < w.p1; p += w.step) {
            int skip = 0;
            const int at = NHWC ? p : pulled_back<N>(p, w.p1, skip);
            const int64_t o = w.base + (NHWC ? int64_t(at) * g.C : at);
            const Vec<T, N> vx = load_vec<T, N>(x + o), vd = load_vec<T, N>(dy + o);
            float h[N], d[N];
#pragma unroll
            for (int j = 0; j < N; ++j) {
                h[j] = vx.get(j);
                d[j] = vd.get(j);
            }
            act_grad<N, NC>(g.act, h, d, cm, cr, cg, cb);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                if (j < skip) continue;
                s[NC == 1 ? 0 : j] += d[j];
                t[NC == 1 ? 0 : j] = fmaf(d[j], h[j], t[NC == 1 ? 0 : j]);
            }
        }
    }
    write_sums<float, N, NHWC>(g, q, w, b, s, t, part);
}

// c1, c2 per (image, group).
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_bwd_groups(NormGeom g, int chunks, const float *__restrict__ part,
                                                            const void *__restrict__ gamma, float *__restrict__ cc)
{
    __shared__ float red[16];
    const int64_t k = blockIdx.x;
    float s, t;
    group_pair(g, chunks, part, k / g.G, int(k % g.G) * g.Cg, [&](int c) { return param<T>(g, gamma, c, 1.f); }, red, s, t);
    if (threadIdx.x == 0) {
        const float n = 1.f / (float(g.Cg) * float(g.HW));
        cc[2 * k] = s * n;
        cc[2 * k + 1] = t * n;
    }
}

template <typename T, int N, bool NHWC, bool PAST>
__global__ void __launch_bounds__(kThreads) norm_bwd_apply(NormGeom g, NormSplitPlan q, const T *__restrict__ x,
                                                           const T *__restrict__ dy,
                                                           const void *__restrict__ gamma,
                                                           const void *__restrict__ beta,
                                                           const float *__restrict__ mean,
                                                           const float *__restrict__ rstd,
                                                           const float *__restrict__ cc, T *__restrict__ dx)
{
    constexpr int NC = NHWC ? N : 1;
    int b;
    const Part<N, NHWC> w = part_of<N, NHWC>(g, q, b);
    if (!w.live) return;
    float cm[NC], cr[NC], cg[NC], cb[NC], c1[NC], c2[NC];
    channel_constants<T, N, NC>(g, b, w.c, gamma, beta, mean, rstd, cm, cr, cg, cb);
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        const int64_t k = int64_t(b) * g.G + fdiv(uint32_t(w.c + j), g.fd_Cg);
        c1[j] = cc[2 * k];
        c2[j] = cc[2 * k + 1];
    }
    for (int p = w.p; p < w.p1; p += w.step) {
        int skip = 0;
        const int at = NHWC ? p : pulled_back<N>(p, w.p1, skip);
        const int64_t o = w.base + (NHWC ? int64_t(at) * g.C : at);
        const Vec<T, N> vx = load_vec<T, N>(x + o), vd = load_vec<T, N>(dy + o);
        float h[N], d[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            h[j] = vx.get(j);
            d[j] = vd.get(j);
        }
        act_grad<N, NC>(g.act, h, d, cm, cr, cg, cb);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int k = NC == 1 ? 0 : j;
            d[j] = cr[k] * (fmaf(cg[k], d[j], -c1[k]) - h[j] * c2[k]);
        }
        Vec<T, N> out;
        out.put(d);
        put_vec<PAST>(dx + o, out);
    }
}

// dgamma and dbeta from rows partial[row][C][2]: a workgroup takes 4 channels (8
// values, one sector of memory a row), 128 rows at a time, and adds its row lanes
// in order.
constexpr int kParamCols = 8, kParamRows = 128, kParamUnroll = 8;
template <typename T>
__global__ void __launch_bounds__(1024) norm_params(NormGeom g, int64_t rows, const float *__restrict__ part,
                                                    void *__restrict__ dgamma, void *__restrict__ dbeta)
{
    __shared__ float red[kParamRows][kParamCols + 1];
    const int col = threadIdx.x % kParamCols, row = threadIdx.x / kParamCols;
    const int e = blockIdx.x * kParamCols + col;
    float s[kParamUnroll] = {};
    if (e < 2 * g.C) {
        int64_t r = row;
        for (; r + (kParamUnroll - 1) * kParamRows < rows; r += kParamUnroll * kParamRows)
#pragma unroll
            for (int u = 0; u < kParamUnroll; ++u) s[u] += part[(r + u * kParamRows) * 2 * g.C + e];
        for (; r < rows; r += kParamRows) s[0] += part[r * 2 * g.C + e];
    }
    red[row][col] = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
    __syncthreads();
    for (int w = kParamRows / 2; w > 0; w >>= 1) {
        if (row < w) red[row][col] += red[row + w][col];
        __syncthreads();
    }
    if (row == 0 && e < 2 * g.C) set_param<T>(g, e % 2 ? dgamma : dbeta, e / 2, red[0][col]);
}

// ------------------------------------------------------------------- host --
int vec_of(const NormGeom &g, int widest)
{
    int n = widest;
    while (n > 1 && (g.nhwc ? g.C : g.HW) < n) n >>= 1;
    return n;
}

size_t lds_bytes(const NormGeom &g, const NormSplitPlan &q, size_t size)
{
    return g.nhwc ? size_t(q.slots) * q.cols * q.N * 2 * size : 0;
}

}  // namespace

bool plan_norm_split(const NormGeom &g, int dtype, NormSplitPlan &q)
{
    q.N = vec_of(g, dtype == GC_F32 ? 4 : 8);
    // about four workgroups a CU, and no chunk under 8 (NCHW 16) visits a thread
    if (g.nhwc) {
        const int cv = (g.C + q.N - 1) / q.N;
        q.cols = std::min(cv, kThreads);
        q.blocks = (cv + q.cols - 1) / q.cols;
        q.slots = kThreads / q.cols;
        const int64_t units = int64_t(g.B) * q.blocks;
        int64_t chunks = std::max<int64_t>(1, 1024 / std::max<int64_t>(1, units));
        chunks = std::min<int64_t>(chunks, std::max(1, g.HW / (8 * q.slots)));
        q.len = int((g.HW + chunks - 1) / chunks);
        q.chunks = (g.HW + q.len - 1) / q.len;
        q.grid = units * q.chunks;
    } else {
        q.cols = q.blocks = q.slots = 1;
        const int64_t units = int64_t(g.B) * g.C;
        int64_t chunks = std::max<int64_t>(1, 4096 / std::max<int64_t>(1, units));
        chunks = std::min<int64_t>(chunks, std::max(1, g.HW / (16 * 64 * q.N)));
        q.len = int((g.HW + chunks - 1) / chunks);
        if (chunks > 1) q.len = (q.len + q.N - 1) / q.N * q.N;
        q.chunks = (g.HW + q.len - 1) / q.len;
        while (q.chunks > 1 && g.HW - (q.chunks - 1) * q.len < q.N) {
            // the last chunk has to hold a whole vector
            q.len += q.N;
            q.chunks = (g.HW + q.len - 1) / q.len;
        }
        q.grid = (units * q.chunks + kWaves - 1) / kWaves;
    }
    const size_t bytes = size_t(g.B) * g.img * (dtype == GC_F32 ? 4 : 2);
    q.past_fwd = 2 * bytes >= kStreamBytes;
    q.past_bwd = 3 * bytes >= kStreamBytes;
    const size_t pairs = size_t(g.B) * q.chunks * g.C * 2;
    const size_t groups = size_t(g.B) * g.G * 2;
    q.part_bytes_fwd = (pairs * 8 + 255) & ~size_t(255);
    q.part_bytes_bwd = (pairs * 4 + 255) & ~size_t(255);
    q.ws_fwd = q.part_bytes_fwd + groups * 4;   // mean and rstd where the caller wants neither
    q.ws_bwd = q.part_bytes_bwd + groups * 4;
    return launchable(q.grid, kThreads) && launchable(int64_t(g.B) * g.G, kThreads) &&
           int64_t(q.chunks) * g.Cg <= 0x7FFFFFFF;
}

// Launches KERNEL<T, N, layout, ...> over the plan's grid.
#define GC_NORM_LAUNCH(lds, args, KERNEL, ...)                                                           \
    do {                                                                                                 \
        if (g.nhwc)                                                                                      \
            hipLaunchKernelGGL((KERNEL<T, N, true __VA_ARGS__>), dim3(unsigned(q.grid)), dim3(kThreads), \
                               lds, s, GC_NORM_ARGS args);                                               \
        else                                                                                             \
            hipLaunchKernelGGL((KERNEL<T, N, false __VA_ARGS__>), dim3(unsigned(q.grid)), dim3(kThreads), \
                               lds, s, GC_NORM_ARGS args);                                               \
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;                           \
    } while (0)
#define GC_NORM_ARGS(...) g, q, __VA_ARGS__

namespace {
template <typename T, int N>
hipError_t split_fwd(const NormGeom &g, const NormSplitPlan &q, const T *x, const void *gamma, const void *beta,
                     T *y, float *mean, float *rstd, double *part, hipStream_t s)
{
    GC_NORM_LAUNCH(lds_bytes(g, q, 8), (x, part), norm_stats);
    hipLaunchKernelGGL(norm_finish, dim3(unsigned(int64_t(g.B) * g.G)), dim3(kThreads), 0, s,
                       g, q.chunks, part, mean, rstd);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    if (q.past_fwd) GC_NORM_LAUNCH(0, (x, gamma, beta, mean, rstd, y), norm_apply, , true);
    else GC_NORM_LAUNCH(0, (x, gamma, beta, mean, rstd, y), norm_apply, , false);
    return hipSuccess;
}

template <typename T, int N>
hipError_t split_bwd(const NormGeom &g, const NormSplitPlan &q, const T *x, const void *gamma, const void *beta,
                     const T *dy, const float *mean, const float *rstd, T *dx, void *dgamma, void *dbeta,
                     float *part, float *cc, hipStream_t s)
{
    GC_NORM_LAUNCH(lds_bytes(g, q, 4), (x, dy, gamma, beta, mean, rstd, part), norm_bwd_sums);
    hipLaunchKernelGGL(norm_bwd_groups<T>, dim3(unsigned(int64_t(g.B) * g.G)), dim3(kThreads),
                       0, s, g, q.chunks, part, gamma, cc);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    if (q.past_bwd) GC_NORM_LAUNCH(0, (x, dy, gamma, beta, mean, rstd, cc, dx), norm_bwd_apply, , true);
    else GC_NORM_LAUNCH(0, (x, dy, gamma, beta, mean, rstd, cc, dx), norm_bwd_apply, , false);
    return launch_norm_params<T>(g, int64_t(g.B) * q.chunks, part, dgamma, dbeta, s);
}
}  // namespace

template <typename T>
hipError_t launch_norm_params(const NormGeom &g, int64_t rows, const float *part, void *dgamma, void *dbeta,
                              hipStream_t s)
{
    if (!dgamma && !dbeta) return hipSuccess;
    hipLaunchKernelGGL(norm_params<T>, dim3((2 * g.C + kParamCols - 1) / kParamCols), dim3(1024), 0, s, g, rows, part,
                       dgamma, dbeta);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_norm_split_fwd(const NormGeom &g, const NormSplitPlan &q, const void *x, const void *gamma,
                                 const void *beta, void *y, float *mean, float *rstd, void *ws, hipStream_t s)
{
    double *part = static_cast<double *>(ws);
    float *spare = reinterpret_cast<float *>(static_cast<char *>(ws) + q.part_bytes_fwd);
    if (!mean) mean = spare;
    if (!rstd) rstd = spare + size_t(g.B) * g.G;
    switch (q.N) {
    case 8:
        if constexpr (sizeof(T) == 2)
            return split_fwd<T, 8>(g, q, (const T *)x, gamma, beta, (T *)y, mean, rstd, part, s);
        return hipErrorInvalidValue;
    case 4: return split_fwd<T, 4>(g, q, (const T *)x, gamma, beta, (T *)y, mean, rstd, part, s);
    case 2: return split_fwd<T, 2>(g, q, (const T *)x, gamma, beta, (T *)y, mean, rstd, part, s);
    default: return split_fwd<T, 1>(g, q, (const T *)x, gamma, beta, (T *)y, mean, rstd, part, s);
    }
}

template <typename T>
hipError_t launch_norm_split_bwd(const NormGeom &g, const NormSplitPlan &q, const void *x, const void *gamma,
                                 const void *beta, const void *dy, const float *mean, const float *rstd, void *dx,
                                 void *dgamma, void *dbeta, void *ws, hipStream_t s)
{
    float *part = static_cast<float *>(ws);
    float *cc = reinterpret_cast<float *>(static_cast<char *>(ws) + q.part_bytes_bwd);
    const T *xt = (const T *)x, *dyt = (const T *)dy;
    switch (q.N) {
    case 8:
        if constexpr (sizeof(T) == 2)
            return split_bwd<T, 8>(g, q, xt, gamma, beta, dyt, mean, rstd, (T *)dx, dgamma, dbeta, part, cc, s);
        return hipErrorInvalidValue;
    case 4: return split_bwd<T, 4>(g, q, xt, gamma, beta, dyt, mean, rstd, (T *)dx, dgamma, dbeta, part, cc, s);
    case 2: return split_bwd<T, 2>(g, q, xt, gamma, beta, dyt, mean, rstd, (T *)dx, dgamma, dbeta, part, cc, s);
    default: return split_bwd<T, 1>(g, q, xt, gamma, beta, dyt, mean, rstd, (T *)dx, dgamma, dbeta, part, cc, s);
    }
}

#define GC_NORM_INSTANCES(T)                                                                                      \
    template hipError_t launch_norm_params<T>(const NormGeom &, int64_t, const float *, void *, void *, hipStream_t); \
    template hipError_t launch_norm_split_fwd<T>(const NormGeom &, const NormSplitPlan &, const void *, const void *, \
                                                 const void *, void *, float *, float *, void *, hipStream_t);    \
    template hipError_t launch_norm_split_bwd<T>(const NormGeom &, const NormSplitPlan &, const void *, const void *, \
                                                 const void *, const void *, const float *, const float *, void *, \
                                                 void *, void *, void *, hipStream_t);
GC_NORM_INSTANCES(float)
GC_NORM_INSTANCES(bf16_t)

}  // namespace gc
