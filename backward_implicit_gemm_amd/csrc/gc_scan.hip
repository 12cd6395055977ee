// gc_scan.hip -- the gated linear recurrence, forward and backward.
//
//   a = sigmoid(gate),  i = 1 - a,  h_t = h' + i * (value - h')  (coupled),  h_t = h' - i*h' + value  (not),
//   h' = reset ? 0 : h_{t-1};
//   g_t = dout_t + what comes back from step t+1,  dvalue = i*g (g),  dgate = a*i*(h' - value)*g (a*i*h'*g),
//   back to step t-1: reset ? 0 : g - i*g
//
// With i as the small share, a state that keeps for thousands of steps is not worn off by the
// rounding of a next to 1.  Everything is fp32; outputs are rounded once.
//
// Memory bound: three tensors forward, five backward.  A thread walks the steps of N
// neighbouring channels, sixteen steps at a time, whose loads are all in flight together.  The
// backward takes blocks from the last to the first, each from the state that the forward kept
// before it, so h needs no tensor of its own.  Few sequences are cut into chunks: one launch
// folds each chunk into (product of a, state from zero), one carries the states over the
// chunks, and the walk then starts every chunk from its state; that reads the inputs twice.
#include <algorithm>
#include <type_traits>

#include "gc_core.h"

namespace gc {
namespace {

constexpr int kBlock = GC_RECURRENCE_BLOCK;

// Where a thread works: sequence b, channels d .. d+N-1, of which the first `skip` belong to
// the thread before it (the last vector of an odd row is moved back), steps [t0, t1) of chunk c.
template <int N>
struct Lane {
    int b, d, skip, c, t0, t1, valid;
    __device__ __forceinline__ bool find(const ScanGeom &g, const ScanPlan &q, const int32_t *lengths)
    {
        const int64_t lane = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
        if (lane >= q.lanes) return false;
        uint32_t bb, v;
        fdivmod(uint32_t(lane), q.fd_nv, bb, v);
        b = int(bb);
        d = min(int(v) * N, g.D - N);
        skip = int(v) * N - d;
        c = blockIdx.y;
        t0 = min(c * q.len, g.T);
        t1 = min(g.T - t0, q.len) + t0;
        valid = lengths ? min(max(lengths[b], 0), g.T) : g.T;
        return true;
    }
    __device__ __forceinline__ int64_t at(const gc_strides &s, int t) const { return int64_t(b) * s.batch + int64_t(t) * s.step + d; }
    // place among [B][D] fp32, and among [chunks][B][D]
    __device__ __forceinline__ int64_t end(const ScanGeom &g) const { return int64_t(b) * g.D + d; }
    __device__ __forceinline__ int64_t end(const ScanGeom &g, int chunk) const { return (int64_t(chunk) * g.B + b) * g.D + d; }
};

template <typename T, int N>
__device__ __forceinline__ void put_own(T *p, const float (&v)[N], int skip)
{
    if (N == 1 || skip == 0) {
        Vec<T, N> w;
        w.put(v);
        store_vec<T, N>(p, w);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (j >= skip) p[j] = from_f32<T>(v[j]);
    }
}

template <int N>
__device__ __forceinline__ void get_f32(const float *p, float (&v)[N])
{
    const Vec<float, N> w = load_vec<float, N>(p);
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = w.get(j);
}

// a = sigmoid(f) and i = 1 - a, each to fp32 accuracy: e = exp(-f), a = 1/(1+e), i = e*a.  Below -80
// e would overflow; a is then below 2e-35 instead of smaller, NaN stays NaN.
__device__ __forceinline__ void gates(float f, float &a, float &i)
{
    const float e = __expf(-(f < -80.f ? -80.f : f));
    a = __builtin_amdgcn_rcpf(1.f + e);
    i = e * a;
}

// The elements of kBlock steps of a tensor, and the steps' resets as bits.  Steps from
// `n` on are not read.
template <typename T, int N>
struct Steps {
    Vec<T, N> v[kBlock];
    __device__ __forceinline__ void load(const T *p, int64_t step, int n)
    {
#pragma unroll
        for (int u = 0; u < kBlock; ++u)
            if (u < n) v[u] = load_vec<T, N>(p + u * step);
    }
};
__device__ __forceinline__ uint32_t load_resets(const uint8_t *p, int64_t step, int n)
{
    uint32_t bits = 0;
#pragma unroll
    for (int u = 0; u < kBlock; ++u)
        if (u < n) bits |= (p[u * step] ? 1u : 0u) << u;
    return bits;
}

// One step of the state; i is 1 - a.
__device__ __forceinline__ float advance(float before, float i, float v, bool coupled)
{
    return coupled ? fmaf(i, v - before, before) : fmaf(-i, before, before) + v;
}

// ----------------------------------------------------------------- forward --
template <typename T, int N>
__global__ void __launch_bounds__(64) scan_fwd(ScanGeom g, ScanPlan q, const T *__restrict__ gate,
                                               const T *__restrict__ value, const float *start,
                                               const uint8_t *__restrict__ reset, const int32_t *__restrict__ lengths,
                                               T *__restrict__ out, float *last, float *__restrict__ states)
{
    Lane<N> w;
    if (!w.find(g, q, lengths)) return;
    float h[N] = {};
    if (start) get_f32<N>(start + w.end(g, w.c), h);
    const bool coupled = g.coupled;
    for (int t = w.t0; t < w.t1; t += kBlock) {
        const int n = min(kBlock, w.t1 - t), live = min(n, w.valid - t);
        Steps<T, N> f, v;
        f.load(gate + w.at(g.gate, t), g.gate.step, live);
        v.load(value + w.at(g.value, t), g.value.step, live);
        const uint32_t resets = reset ? load_resets(reset + w.b * g.reset.batch + t * g.reset.step, g.reset.step, live) : 0;
        if (states) put_own<float, N>(states + (int64_t(w.b) * ((g.T - 1) / kBlock + 1) + t / kBlock) * g.D + w.d, h, w.skip);
        T *o = out + w.at(g.out, t);
#pragma unroll
        for (int u = 0; u < kBlock; ++u) {
            if (u >= n) break;
            float y[N] = {};
            if (u < live) {
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    float a, i;
                    gates(f.v[u].get(j), a, i);
                    h[j] = advance(resets >> u & 1 ? 0.f : h[j], i, v.v[u].get(j), coupled);
                    y[j] = h[j];
                }
            }
            put_own<T, N>(o + u * g.out.step, y, w.skip);
        }
    }
    if (last && w.c == q.chunks - 1) put_own<float, N>(last + w.end(g), h, w.skip);
}

// A chunk as a step of its own: the product of its a (-1 where a reset cuts the state off), and its
// state from zero.
template <typename T, int N>
__global__ void __launch_bounds__(64) scan_fold_fwd(ScanGeom g, ScanPlan q, const T *__restrict__ gate,
                                                    const T *__restrict__ value, const uint8_t *__restrict__ reset,
                                                    const int32_t *__restrict__ lengths, float *__restrict__ keep,
                                                    float *__restrict__ add)
{
    Lane<N> w;
    if (!w.find(g, q, lengths)) return;
    float h[N] = {}, p[N];
    bool cut = false;
#pragma unroll
    for (int j = 0; j < N; ++j) p[j] = 1.f;
    const bool coupled = g.coupled;
    for (int t = w.t0; t < min(w.t1, w.valid); t += kBlock) {
        const int live = min(kBlock, min(w.t1, w.valid) - t);
        Steps<T, N> f, v;
        f.load(gate + w.at(g.gate, t), g.gate.step, live);
        v.load(value + w.at(g.value, t), g.value.step, live);
        const uint32_t resets = reset ? load_resets(reset + w.b * g.reset.batch + t * g.reset.step, g.reset.step, live) : 0;
        cut |= resets != 0;
#pragma unroll
        for (int u = 0; u < kBlock; ++u) {
            if (u >= live) break;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                float a, i;
                gates(f.v[u].get(j), a, i);
                h[j] = advance(resets >> u & 1 ? 0.f : h[j], i, v.v[u].get(j), coupled);
                p[j] = fmaf(-i, p[j], p[j]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < N; ++j) p[j] = cut ? -1.f : p[j];
    put_own<float, N>(keep + w.end(g, w.c), p, w.skip);
    put_own<float, N>(add + w.end(g, w.c), h, w.skip);
}

// The state before each chunk (BACK: the gradient behind it), written over `keep`: 16 waves fold a
// sixteenth of the chunks each, then walk them again from what the waves before them give.
__device__ __forceinline__ float carry_over(float keep, float add, float h) { return keep < 0.f ? add : fmaf(keep, h, add); }

template <bool BACK>
__global__ void __launch_bounds__(1024) scan_carry(int64_t ends, int chunks, const float *__restrict__ first,
                                                   float *keep, const float *__restrict__ add)
{
    __shared__ float part[2][16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t e = int64_t(blockIdx.x) * 64 + lane;
    const int per = (chunks + 15) / 16, c0 = min(wave * per, chunks), c1 = min(c0 + per, chunks);
    const bool live = e < ends;
    auto place = [&](int c) { return int64_t(BACK ? chunks - 1 - c : c) * ends + e; };
    float p = 1.f, h = 0.f;
    bool cut = false;
    if (live)
        for (int c = c0; c < c1; ++c) {
            const float k = keep[place(c)], a = add[place(c)];
            h = carry_over(k, a, h);
            cut |= k < 0.f;
            p *= k;
        }
    part[0][wave][lane] = cut ? -1.f : p;
    part[1][wave][lane] = h;
    __syncthreads();
    if (!live) return;
    h = first ? first[e] : 0.f;
    for (int w = 0; w < wave; ++w) h = carry_over(part[0][w][lane], part[1][w][lane], h);
    for (int c = c0; c < c1; ++c) {
        const float k = keep[place(c)], a = add[place(c)];
        keep[place(c)] = h;
        h = carry_over(k, a, h);
    }
}

// ---------------------------------------------------------------- backward --
template <typename T, int N>
__global__ void __launch_bounds__(64) scan_bwd(ScanGeom g, ScanPlan q, const T *__restrict__ gate,
                                               const T *__restrict__ value, const float *__restrict__ states,
                                               const uint8_t *__restrict__ reset, const int32_t *__restrict__ lengths,
                                               const T *__restrict__ dout, const float *start, T *__restrict__ dgate,
                                               T *__restrict__ dvalue, float *dh0)
{
    Lane<N> w;
    if (!w.find(g, q, lengths)) return;
    float back[N] = {};
    if (start) get_f32<N>(start + w.end(g, w.c), back);
    const bool coupled = g.coupled;
    for (int t = (w.t1 - 1) / kBlock * kBlock; t >= w.t0 && w.t1 > w.t0; t -= kBlock) {
        const int n = min(kBlock, w.t1 - t), live = min(n, w.valid - t);
        T *df = dgate + w.at(g.dgate, t), *dv = dvalue + w.at(g.dvalue, t);
        Steps<T, N> f, v, d;
        f.load(gate + w.at(g.gate, t), g.gate.step, live);
        v.load(value + w.at(g.value, t), g.value.step, live);
        d.load(dout + w.at(g.out, t), g.out.step, live);
        const uint32_t resets = reset ? load_resets(reset + w.b * g.reset.batch + t * g.reset.step, g.reset.step, live) : 0;
        float h[N] = {}, share[kBlock][N], slope[kBlock][N];
        if (live > 0) get_f32<N>(states + (int64_t(w.b) * ((g.T - 1) / kBlock + 1) + t / kBlock) * g.D + w.d, h);
#pragma unroll
        for (int u = 0; u < kBlock; ++u) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                share[u][j] = slope[u][j] = 0.f;
                if (u < live) {
                    float a, i;
                    gates(f.v[u].get(j), a, i);
                    const float before = resets >> u & 1 ? 0.f : h[j], x = v.v[u].get(j);
                    share[u][j] = i;
                    slope[u][j] = a * i * (coupled ? before - x : before);
                    h[j] = advance(before, i, x, coupled);
                }
            }
        }
#pragma unroll
        for (int u = kBlock - 1; u >= 0; --u) {
            if (u >= n) continue;
            float yf[N] = {}, yv[N] = {};
            if (u < live) {
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const float gr = back[j] + d.v[u].get(j);
                    yf[j] = slope[u][j] * gr;
                    yv[j] = coupled ? share[u][j] * gr : gr;
                    back[j] = resets >> u & 1 ? 0.f : fmaf(-share[u][j], gr, gr);
                }
            }
            put_own<T, N>(df + u * g.dgate.step, yf, w.skip);
            put_own<T, N>(dv + u * g.dvalue.step, yv, w.skip);
        }
    }
    if (dh0 && w.c == 0) put_own<float, N>(dh0 + w.end(g), back, w.skip);
}

template <typename T, int N>
__global__ void __launch_bounds__(64) scan_fold_bwd(ScanGeom g, ScanPlan q, const T *__restrict__ gate,
                                                    const T *__restrict__ dout, const uint8_t *__restrict__ reset,
                                                    const int32_t *__restrict__ lengths, float *__restrict__ keep,
                                                    float *__restrict__ add)
{
    Lane<N> w;
    if (!w.find(g, q, lengths)) return;
    float back[N] = {}, p[N];
    bool cut = false;
#pragma unroll
    for (int j = 0; j < N; ++j) p[j] = 1.f;
    const int t1 = min(w.t1, w.valid);
    for (int t = (w.t1 - 1) / kBlock * kBlock; t >= w.t0 && w.t1 > w.t0; t -= kBlock) {
        const int live = min(kBlock, t1 - t);
        Steps<T, N> f, d;
        f.load(gate + w.at(g.gate, t), g.gate.step, live);
        d.load(dout + w.at(g.out, t), g.out.step, live);
        const uint32_t resets = reset ? load_resets(reset + w.b * g.reset.batch + t * g.reset.step, g.reset.step, live) : 0;
        cut |= resets != 0;
#pragma unroll
        for (int u = kBlock - 1; u >= 0; --u) {
            if (u >= live) continue;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                float a, i;
                gates(f.v[u].get(j), a, i);
                const float gr = back[j] + d.v[u].get(j);
                back[j] = resets >> u & 1 ? 0.f : fmaf(-i, gr, gr);
                p[j] = fmaf(-i, p[j], p[j]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < N; ++j) p[j] = cut ? -1.f : p[j];
    put_own<float, N>(keep + w.end(g, w.c), p, w.skip);
    put_own<float, N>(add + w.end(g, w.c), back, w.skip);
}

template <bool BACK>
hipError_t carry(const ScanGeom &g, const ScanPlan &q, const float *first, float *keep, const float *add, hipStream_t s)
{
    const int64_t ends = int64_t(g.B) * g.D;
    hipLaunchKernelGGL((scan_carry<BACK>), dim3(unsigned((ends + 63) / 64)), dim3(1024), 0, s, ends, q.chunks, first, keep,
                       add);
    return hipGetLastError();
}

template <typename F>
hipError_t with_channels(int n, F f)
{
    return n == 2 ? f(std::integral_constant<int, 2>()) : f(std::integral_constant<int, 1>());
}

}  // namespace

bool plan_scan(const ScanGeom &g, int dtype, bool bwd, ScanPlan &q)
{
    q = ScanPlan{};
    q.N = g.D >= 2 && dtype == GC_BF16 ? 2 : 1;
    q.nv = vectors(g.D, q.N);
    q.lanes = int64_t(g.B) * q.nv;
    if (int64_t(g.B) * g.D >= int64_t(1) << 31) return false;
    const int64_t waves = (q.lanes + 63) / 64;
    const int blocks = g.T ? (g.T - 1) / kBlock + 1 : 1;
    int64_t chunks = 1;
    if (waves && waves < 512) chunks = std::max<int64_t>(1, std::min<int64_t>(2048 / waves, blocks / 4));
    const int per = int((blocks + chunks - 1) / chunks);
    q.len = g.T ? std::min<int64_t>(int64_t(per) * kBlock, 0x7FFFFFF0) : kBlock;
    q.chunks = (blocks + per - 1) / per;
    q.part_bytes = q.chunks > 1 ? (size_t(q.chunks) * g.B * g.D * 4 + 255) & ~size_t(255) : 0;
    q.ws_bytes = 2 * q.part_bytes;
    q.fd_nv = make_fastdiv(uint32_t(q.nv));
    return launchable(waves * q.chunks, 64);
}

template <typename T>
hipError_t launch_scan_fwd(const ScanGeom &g, const ScanPlan &q, const void *gate, const void *value, const float *h0,
                           const uint8_t *reset, const int32_t *lengths, void *out, float *last, float *states,
                           void *ws, hipStream_t s)
{
    if (!q.lanes) return hipSuccess;
    const T *f = static_cast<const T *>(gate), *v = static_cast<const T *>(value);
    float *keep = static_cast<float *>(ws), *add = keep + q.part_bytes / 4;
    const dim3 grid(unsigned((q.lanes + 63) / 64), unsigned(q.chunks));
    return with_channels(q.N, [&](auto nn) {
        constexpr int N = decltype(nn)::value;
        if (q.chunks > 1) {
            hipLaunchKernelGGL((scan_fold_fwd<T, N>), grid, dim3(64), 0, s, g, q, f, v, reset, lengths, keep, add);
            if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
            if (const hipError_t e = carry<false>(g, q, h0, keep, add, s); e != hipSuccess) return e;
        }
        hipLaunchKernelGGL((scan_fwd<T, N>), grid, dim3(64), 0, s, g, q, f, v, q.chunks > 1 ? keep : h0, reset, lengths,
                           static_cast<T *>(out), last, states);
        return hipGetLastError();
    });
}

template <typename T>
hipError_t launch_scan_bwd(const ScanGeom &g, const ScanPlan &q, const void *gate, const void *value,
                           const float *states, const uint8_t *reset, const int32_t *lengths, const void *dout,
                           const float *dlast, void *dgate, void *dvalue, float *dh0, void *ws, hipStream_t s)
{
    if (!q.lanes) return hipSuccess;
    const T *f = static_cast<const T *>(gate), *v = static_cast<const T *>(value), *d = static_cast<const T *>(dout);
    float *keep = static_cast<float *>(ws), *add = keep + q.part_bytes / 4;
    const dim3 grid(unsigned((q.lanes + 63) / 64), unsigned(q.chunks));
    return with_channels(q.N, [&](auto nn) {
        constexpr int N = decltype(nn)::value;
        if (q.chunks > 1) {
            hipLaunchKernelGGL((scan_fold_bwd<T, N>), grid, dim3(64), 0, s, g, q, f, d, reset, lengths, keep, add);
            if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
            if (const hipError_t e = carry<true>(g, q, dlast, keep, add, s); e != hipSuccess) return e;
        }
        hipLaunchKernelGGL((scan_bwd<T, N>), grid, dim3(64), 0, s, g, q, f, v, states, reset, lengths, d,
                           q.chunks > 1 ? keep : dlast, static_cast<T *>(dgate), static_cast<T *>(dvalue), dh0);
        return hipGetLastError();
    });
}

#define GC_SCAN_INSTANCES(T)                                                                                            \
    template hipError_t launch_scan_fwd<T>(const ScanGeom &, const ScanPlan &, const void *, const void *, const float *, \
                                           const uint8_t *, const int32_t *, void *, float *, float *, void *, hipStream_t); \
    template hipError_t launch_scan_bwd<T>(const ScanGeom &, const ScanPlan &, const void *, const void *, const float *, \
                                           const uint8_t *, const int32_t *, const void *, const float *, void *, void *, \
                                           float *, void *, hipStream_t);
GC_SCAN_INSTANCES(float)
GC_SCAN_INSTANCES(bf16_t)

}  // namespace gc
