// grad_clip.hip -- the global norm of a list of tensors, and their clipping:
//     norm = |prescale| * sqrt(sum of g^2 over every element of every tensor)
//     c    = prescale * min(1, max_norm / (norm + eps)),   dst = c * g
//
// The list travels in the kernel arguments (kClipTensors tensors a launch), so
// nothing is kept between calls and a captured graph holds its own copy.  Every
// tensor is cut into chunks of one size; workgroup w of a launch takes chunks
// w, w + grid, ... and finds a chunk's tensor by bisecting the chunk counts
// (wave-uniform scalar loads), then following the list.  (One run of consecutive
// chunks a workgroup was slower, 131 against 120 us for 238 MB: neighbouring
// workgroups then read far apart.)
//
// Pass 1 adds up squares in fp64 (the product of two fp32 values is exact there
// and cannot overflow or vanish; fp64 adds at the vector unit's full rate hide
// behind the loads: fp32 squares time the same) and writes one partial per workgroup.
// Pass 2 sums the partials in the same fixed order in every workgroup, so the norm
// and the result are bit-reproducible, and scales, from the last chunk to the
// first, as the last ones read are still in cache.  Both passes are bound by memory:
// the gradients are read twice and written once (238 MB in 37 us, then 75 us; a copy
// of one 160 MB tensor takes 60 us, its norm and clipping 81).
#include "gc_train.h"
#include "gc_vec.h"

namespace gc {
namespace {

constexpr int kThreads = 256;
// 1024 or 2048 workgroups, chunks of 16 or 32 KB and 2, 4 or 8 vectors in flight
// time within 3 % of each other
constexpr int kMaxGrid = 1024;     // workgroups of a launch: 4 per CU
constexpr int kUnroll = 4;         // vectors a thread has in flight
constexpr int kChunk = 8192;       // fp32 elements of a chunk
constexpr int kFold = 2048;        // more partials than this are folded by a launch of their own

struct ClipArgs {
    const void *src[kClipTensors];
    void *dst[kClipTensors];
    int64_t n[kClipTensors];
    int first[kClipTensors + 1];          // first chunk of each tensor
    uint32_t bf16[kClipTensors / 32];     // bit t: tensor t holds bf16
    int count;
    int chunk;                            // fp32 elements of a chunk; twice as many in bf16
};

// The tensor chunk c lies in: the last t with first[t] <= c (empty tensors
// before it share its first chunk).
__device__ __forceinline__ int tensor_of(const ClipArgs &a, int c)
{
    int lo = 0, hi = a.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.first[mid] <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

template <int K>
__device__ __forceinline__ double sum_of(const double (&s)[K])
{
    double v = s[0];
#pragma unroll
    for (int k = 1; k < K; ++k) v += s[k];
    return v;
}

// A thread takes kUnroll vectors at a time, kThreads vectors apart.
template <typename T>
__device__ __forceinline__ double squares(const T *p, int len)
{
    constexpr int V = kVec<T>;
    const int whole = len / V;
    double s[kUnroll] = {};
    int i = threadIdx.x;
    for (; i + (kUnroll - 1) * kThreads < whole; i += kUnroll * kThreads) {
        Vec<T, V> v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) v[u] = load_vec<T, V>(p + (i + u * kThreads) * V);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
#pragma unroll
            for (int j = 0; j < V; ++j) s[u] = fma(double(v[u].get(j)), double(v[u].get(j)), s[u]);
    }
    for (; i < whole; i += kThreads) {
        const Vec<T, V> v = load_vec<T, V>(p + i * V);
#pragma unroll
        for (int j = 0; j < V; ++j) s[0] = fma(double(v.get(j)), double(v.get(j)), s[0]);
    }
    const int e = whole * V + threadIdx.x;
    if (e < len) s[0] = fma(double(to_f32(p[e])), double(to_f32(p[e])), s[0]);
    return sum_of(s);
}

template <bool PAST, typename T>
__device__ __forceinline__ void scale_vec(T *q, const Vec<T, kVec<T>> &v, float c)
{
    constexpr int V = kVec<T>;
    float f[V];
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = c * v.get(j);
    Vec<T, V> o;
    o.put(f);
    put_vec<PAST>(q, o);
}

template <bool PAST, typename T>
__device__ __forceinline__ void scale(const T *p, T *q, int len, float c)
{
    constexpr int V = kVec<T>;
    const int whole = len / V;
    int i = threadIdx.x;
    for (; i + (kUnroll - 1) * kThreads < whole; i += kUnroll * kThreads) {
        Vec<T, V> v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) v[u] = load_vec<T, V>(p + (i + u * kThreads) * V);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) scale_vec<PAST>(q + (i + u * kThreads) * V, v[u], c);
    }
    for (; i < whole; i += kThreads) scale_vec<PAST>(q + i * V, load_vec<T, V>(p + i * V), c);
    const int e = whole * V + threadIdx.x;
    if (e < len) q[e] = from_f32<T>(c * to_f32(p[e]));
}

__device__ __forceinline__ bool is_bf16(const ClipArgs &a, int t) { return a.bf16[t >> 5] >> (t & 31) & 1; }

// Calls f(t, at, len) for this workgroup's chunks: blockIdx.x, + gridDim.x, ...,
// counted from the last one when BACK.  The tensor is bisected once and then
// followed.
template <bool BACK, typename F>
__device__ __forceinline__ void for_chunks(const ClipArgs &a, F f)
{
    const int chunks = a.first[a.count];
    int t = -1;
    for (int k = blockIdx.x; k < chunks; k += gridDim.x) {
        const int c = BACK ? chunks - 1 - k : k;
        if (t < 0) t = tensor_of(a, c);
        if (BACK)
            while (a.first[t] > c) --t;
        else
            while (a.first[t + 1] <= c) ++t;
        const int chunk = is_bf16(a, t) ? 2 * a.chunk : a.chunk;
        const int64_t at = int64_t(c - a.first[t]) * chunk;
        f(t, at, int(min(int64_t(chunk), a.n[t] - at)));
    }
}

__global__ void __launch_bounds__(kThreads) clip_squares(const ClipArgs a, double *__restrict__ part)
{
    __shared__ double red[16];
    double s = 0;
    for_chunks<false>(a, [&](int t, int64_t at, int len) {
        if (is_bf16(a, t)) s += squares(static_cast<const bf16_t *>(a.src[t]) + at, len);
        else s += squares(static_cast<const float *>(a.src[t]) + at, len);
    });
    s = block_sum(s, red);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__device__ __forceinline__ double sum_partials(const double *part, int np, double *red)
{
    double s = 0;
    for (int i = threadIdx.x; i < np; i += kThreads) s += part[i];
    return block_sum(s, red);
}

__global__ void __launch_bounds__(kThreads) clip_fold(const double *__restrict__ part, int np,
                                                      double *__restrict__ out)
{
    __shared__ double red[16];
    const double s = sum_partials(part, np, red);
    if (threadIdx.x == 0) *out = s;
}

// norm only
__global__ void __launch_bounds__(kThreads) clip_norm(const double *__restrict__ part, int np,
                                                      float prescale, float *__restrict__ norm)
{
    __shared__ double red[16];
    const double s = sum_partials(part, np, red);
    if (threadIdx.x == 0) *norm = float(fabs(double(prescale)) * sqrt(s));
}

template <bool PAST>
__global__ void __launch_bounds__(kThreads) clip_scale(const ClipArgs a, const double *__restrict__ part,
                                                       int np, float max_norm, float prescale, float eps,
                                                       float *__restrict__ norm)
{
    __shared__ double red[16];
    const double total = fabs(double(prescale)) * sqrt(sum_partials(part, np, red));
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = float(total);
    // a NaN norm (or an infinite one against an infinite max_norm) stays NaN
    const double r = double(max_norm) / (total + double(eps));
    const float c = float(double(prescale) * (r >= 1.0 ? 1.0 : r));
    for_chunks<true>(a, [&](int t, int64_t at, int len) {
        if (c == 1.f && a.src[t] == a.dst[t]) return;   // in place, and nothing changes
        if (is_bf16(a, t))
            scale<PAST>(static_cast<const bf16_t *>(a.src[t]) + at, static_cast<bf16_t *>(a.dst[t]) + at, len, c);
        else
            scale<PAST>(static_cast<const float *>(a.src[t]) + at, static_cast<float *>(a.dst[t]) + at, len, c);
    });
}

int launches(int count) { return (count + kClipTensors - 1) / kClipTensors; }

// Chunk size of a list of `total` elements: kChunk, more only where a launch's
// chunk numbers would not stay within 30 bits.
int chunk_of(int64_t total)
{
    int64_t c = kChunk;
    while (total / c > (int64_t(1) << 29)) c *= 2;
    return int(c);
}

// Arguments of launch l (tensors l*kClipTensors ...); returns its grid, 0
// for tensors without elements.
int fill_args(const gc_tensor *list, int count, int l, int chunk, ClipArgs &a)
{
    const int t0 = l * kClipTensors;
    a.count = count - t0 < kClipTensors ? count - t0 : kClipTensors;
    a.chunk = chunk;
    for (uint32_t &b : a.bf16) b = 0;
    int64_t chunks = 0;
    for (int t = 0; t < a.count; ++t) {
        const gc_tensor &x = list[t0 + t];
        a.src[t] = x.src;
        a.dst[t] = x.dst;
        a.n[t] = x.n;
        a.first[t] = int(chunks);
        if (x.dtype == GC_BF16) a.bf16[t >> 5] |= 1u << (t & 31);
        const int64_t each = x.dtype == GC_BF16 ? 2 * chunk : chunk;
        chunks += (x.n + each - 1) / each;
    }
    a.first[a.count] = int(chunks);
    return int(chunks < kMaxGrid ? chunks : kMaxGrid);
}

}  // namespace

size_t grad_clip_ws_bytes(int count)
{
    // one partial a workgroup, and the folded sum
    return (size_t(launches(count)) * kMaxGrid + 1) * sizeof(double);
}

hipError_t launch_grad_clip(const gc_tensor *list, int count, float max_norm, float prescale, float eps,
                            bool scale, float *norm, void *ws, hipStream_t s)
{
    double *part = static_cast<double *>(ws);
    int64_t total = 0, bytes = 0;
    for (int t = 0; t < count; ++t) {
        total += list[t].n;
        bytes += 2 * list[t].n * (list[t].dtype == GC_F32 ? 4 : 2);
    }
    const int chunk = chunk_of(total);
    const int nl = launches(count);
    ClipArgs a;
    const bool past = bytes >= int64_t(kStreamBytes);
    int np = 0;
    for (int l = 0; l < nl; ++l) {
        const int grid = fill_args(list, count, l, chunk, a);
        if (!grid) continue;
        hipLaunchKernelGGL(clip_squares, dim3(grid), dim3(kThreads), 0, s, a, part + np);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
        np += grid;
    }
    if (np > kFold) {
        double *folded = part + np;
        hipLaunchKernelGGL(clip_fold, dim3(1), dim3(kThreads), 0, s, part, np, folded);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
        part = folded;
        np = 1;
    }
    if (!scale || np == 0) {
        hipLaunchKernelGGL(clip_norm, dim3(1), dim3(kThreads), 0, s, part, np, prescale, norm);
        return hipGetLastError();
    }
    for (int l = 0; l < nl; ++l) {
        const int grid = fill_args(list, count, l, chunk, a);
        if (!grid) continue;
        hipLaunchKernelGGL((past ? clip_scale<true> : clip_scale<false>), dim3(grid), dim3(kThreads), 0, s, a,
                           part, np, max_norm, prescale, eps, norm);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace gc
