// gc_scan.hip -- the gated linear recurrence, forward and backward.
//
//   a = sigmoid(gate),  i = 1 - a,  h_t = a*h' + i*value  (coupled),  h_t = a*h' + value  (not),
//   h' = reset ? 0 : h_{t-1};
//   g_t = dout_t + what comes back from step t+1,  dvalue = i*g (g),  dgate = a*i*(h' - value)*g (a*i*h'*g),
//   back to step t-1: reset ? 0 : a*g
//
// Only the smaller of a and i is a factor, s; the larger one is what it leaves: (1 - s)*x = x - s*x.  A state
// that keeps for thousands of steps is not worn off by the rounding of a next to 1, and a gate that closes
// leaves the value, or a share of 1e-9 of the state, right in its own size.  Everything is fp32; outputs
// are rounded once.
//
// Memory bound: three tensors forward, five backward, and the fp32 states (an eighth of a bf16 tensor).
// A thread walks the steps of one channel (backward of bf16: two where there are enough), eight
// or sixteen steps at a time, the loads of the next ones in flight; scalar bases and 32-bit lane offsets
// leave the vector unit to the gates.  A step costs a wave about 60 ns, mostly the exponential, the
// reciprocal and fifteen more instructions, so a walk wants several waves on each of the 1024 SIMDs.  The
// backward takes blocks from the last to the first, each from the state that the forward kept
// before it, so h needs no tensor of its own.
//
// Few sequences are cut into chunks: one launch folds each chunk into (product of a, state from
// zero), one carries the states over the chunks, and the walk then starts every chunk from its
// state; that reads two tensors twice.  512 sequences of 64 x 512 with resets take 25 us forward in bf16
// (107 MB, 4.3 TB/s) and 72 backward in fp32 (342 MB, 4.7 TB/s); one of 32,768 x 1024 bf16 takes 74
// (fold 29 at 4.6 TB/s, carry 5, walk 39), and 2.5 ms if it is walked as a whole.  Times, here and below, are
// of passes whose inputs come from HBM, unless they name the cache.
#include <algorithm>
#include <float.h>
#include <type_traits>

#include "gc_core.h"
#include "gc_norm_res.h"

namespace gc {
namespace {

constexpr int kBlock = GC_RECURRENCE_BLOCK;
constexpr int kHalf = kBlock / 2;
constexpr float kLog2e = 1.44269504088896f;
constexpr float kLeast = 1.4e-45f;     // the smallest number above 0
constexpr int kCarryWaves = 16;
constexpr int kMostChunks = kCarryWaves * 16;

// Where a thread works: sequence b, channels d .. d+N-1, of which the first `skip` belong to
// the thread before it (the last vector of an odd row is moved back), steps [t0, t1) of chunk c.
// b0 is the first thread's sequence, for addresses of a scalar and a 32-bit lane part.
template <int N>
struct Lane {
    int b, b0, d, skip, c, t0, t1, valid;
    __device__ __forceinline__ bool find(const ScanGeom &g, const ScanPlan &q, const int32_t *lengths)
    {
        uint32_t chunk, block;
        fdivmod(die_order(blockIdx.x, gridDim.x), q.fd_blocks, chunk, block);
        const int64_t lane = int64_t(block) * 64 + threadIdx.x;
        if (lane >= q.lanes) return false;
        uint32_t bb, v;
        fdivmod(uint32_t(lane), q.fd_nv, bb, v);
        if (int(v) >= q.nv) return false;
        b = int(bb);
        b0 = __builtin_amdgcn_readfirstlane(b);
        d = min(int(v) * N, g.D - N);
        skip = int(v) * N - d;
        c = int(chunk);
        t0 = min(c * q.len, g.T);
        t1 = min(g.T - t0, q.len) + t0;
        valid = lengths ? min(max(lengths[b], 0), g.T) : g.T;
        return true;
    }
    // place among [B][D] fp32, among [chunks][B][D], and of the state before step t among [B][blocks][D]
    __device__ __forceinline__ int64_t end(const ScanGeom &g) const { return int64_t(b) * g.D + d; }
    __device__ __forceinline__ int64_t end(const ScanGeom &g, int chunk) const { return (int64_t(chunk) * g.B + b) * g.D + d; }
    __device__ __forceinline__ int64_t state(const ScanGeom &g, int t) const
    {
        return (int64_t(b) * ((g.T - 1) / kBlock + 1) + t / kBlock) * g.D + d;
    }
};

// A vector of at most 4 bytes as a word.
struct Words {
    uint32_t w;
};

// Stores the channels that are this thread's own; PAST: past the cache.
template <typename T, int N, bool PAST = false>
__device__ __forceinline__ void put_own(T *p, const float (&v)[N], int skip)
{
    if (N == 1 || skip == 0) {
        Vec<T, N> w;
        w.put(v);
        if constexpr (PAST) {
            typedef std::conditional_t<sizeof(T) * N == 4, uint32_t, uint16_t> bits;
            typedef bits loose __attribute__((aligned(sizeof(T))));
            __builtin_nontemporal_store(bits(__builtin_bit_cast(Words, w).w), reinterpret_cast<loose *>(p));
        } else {
            store_vec<T, N>(p, w);
        }
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

// A tensor along a thread's steps: a scalar base and distance, and the lane's offset from it
// (Off: 32 bits where a wave's sequences lie within 4 GiB of each other).
template <typename T, int N, typename Off>
struct Line {
    typedef std::conditional_t<std::is_const_v<T>, const char, char> byte;
    byte *base;
    int64_t step;  // bytes
    Off off;       // bytes
    __device__ __forceinline__ Line(T *p, const gc_strides &s, const Lane<N> &w)
        : base(reinterpret_cast<byte *>(p + int64_t(w.b0) * s.batch)), step(s.step * int64_t(sizeof(T))),
          off(Off((int64_t(w.b - w.b0) * s.batch + w.d) * int64_t(sizeof(T))))
    {
    }
    // the scalar part of step t's address, which a walk moves on by `step`; and the lane's address
    __device__ __forceinline__ byte *row(int t) const { return base + int64_t(t) * step; }
    __device__ __forceinline__ T *lane(byte *row) const { return reinterpret_cast<T *>(row + off); }
    // `COUNT` steps from t; those from n on are not read
    template <int COUNT, bool FULL>
    __device__ __forceinline__ void load(Vec<std::remove_const_t<T>, N> (&v)[COUNT], int t, int n) const
    {
        byte *p = row(t);
#pragma unroll
        for (int u = 0; u < COUNT; ++u, p += step)
            if (FULL || u < n) v[u] = load_vec<std::remove_const_t<T>, N>(lane(p));
    }
};

// The resets of a thread's steps, as bits.
template <bool SOME>
struct Resets {
    const uint8_t *p;
    int64_t step;
    __device__ __forceinline__ Resets(const uint8_t *reset, const ScanGeom &g, int b)
        : p(SOME ? reset + int64_t(b) * g.reset.batch : nullptr), step(g.reset.step)
    {
    }
    template <int COUNT, bool FULL>
    __device__ __forceinline__ uint32_t load(int t, int n) const
    {
        if (!SOME) return 0;
        uint8_t v[COUNT];
        const uint8_t *at = p + int64_t(t) * step;
#pragma unroll
        for (int u = 0; u < COUNT; ++u, at += step) {
            v[u] = 0;
            if (FULL || u < n) v[u] = *at;
        }
        uint32_t bits = 0;
#pragma unroll
        for (int u = 0; u < COUNT; ++u) bits |= (v[u] ? 1u : 0u) << u;
        return bits;
    }
};

// A step's gate: whether it is open, SCALE (1 or 2) times its smaller share, which is then i and else a, and the
// larger one.  With e = exp(-|f|) nothing overflows.  e is off by up to 1.5|f| + 3 half steps of fp32, as
// exp2 of a rounded product, the smaller share by 5 more, the larger one by 3; shares below 1e-38 may be 0.
template <int SCALE = 1>
struct Gate {
    float small, large;
    bool open;
    __device__ __forceinline__ explicit Gate(float f)
    {
        const float e = __builtin_amdgcn_exp2f(fmaf(fabsf(f), -kLog2e, SCALE - 1.f));
        large = __builtin_amdgcn_rcpf(fmaf(e, 1.f / SCALE, 1.f));
        small = e * large;
        open = f >= 0.f;
    }
};

// (1 - s)*x.  An infinite x meets the largest finite number of its sign, so that it stays and does not become
// NaN.  (NaN becomes a number there, and is NaN in the difference.)
__device__ __forceinline__ float rest(float s, float x)
{
    return fmaf(-s, __builtin_amdgcn_fmed3f(x, -FLT_MAX, FLT_MAX), x);
}

// One step of the state.  In two products, not one with the difference of state and value, which overflows for
// large ones and is NaN for infinite ones.
template <bool COUPLED>
__device__ __forceinline__ float advance(float before, const Gate<> &k, float v)
{
    if (!COUPLED) return (k.open ? rest(k.small, before) : k.small * before) + v;
    return fmaf(k.small, k.open ? v : before, rest(k.small, k.open ? before : v));
}

// ----------------------------------------------------------------- forward --
// Runs step(u, bit u of resets) for COUNT steps.  A second form of the steps, for waves that meet no reset
// meanwhile, costs the registers of both: backward of 512 x 64 x 512 bf16 with resets 54 us so, 41 with one.
template <int COUNT, bool SOME, typename F>
__device__ __forceinline__ void each_step(uint32_t resets, F step)
{
#pragma unroll
    for (int u = 0; u < COUNT; ++u) step(u, SOME && (resets >> u & 1) != 0);
}

// Walks a thread's valid steps: body(t, count, FULL, gates, values, resets) for eight steps at a time while
// every thread of the wave has sixteen more, their loads one half ahead, then for what is left.
template <typename T, int N, bool SOME, typename Off, typename Body>
__device__ __forceinline__ int walk(const Line<const T, N, Off> &x, const Line<const T, N, Off> &y, const Resets<SOME> &r,
                                    int t, int t1, Body body)
{
    Vec<T, N> xa[kHalf], ya[kHalf], xb[kHalf], yb[kHalf];
    if (__all(t + kBlock <= t1)) {
        x.template load<kHalf, true>(xa, t, 0);
        y.template load<kHalf, true>(ya, t, 0);
        uint32_t ra = r.template load<kHalf, true>(t, 0);
        for (;;) {
            x.template load<kHalf, true>(xb, t + kHalf, 0);
            y.template load<kHalf, true>(yb, t + kHalf, 0);
            const uint32_t rb = r.template load<kHalf, true>(t + kHalf, 0);
            body(t, kHalf, std::true_type(), xa, ya, ra);
            const bool more = __all(t + 2 * kBlock <= t1);
            if (more) {
                x.template load<kHalf, true>(xa, t + kBlock, 0);
                y.template load<kHalf, true>(ya, t + kBlock, 0);
                ra = r.template load<kHalf, true>(t + kBlock, 0);
            }
            body(t + kHalf, kHalf, std::true_type(), xb, yb, rb);
            t += kBlock;
            if (!more) break;
        }
    }
    for (; __any(t < t1); t += kHalf) {
        const int n = min(kHalf, t1 - t);
        x.template load<kHalf, false>(xa, t, n);
        y.template load<kHalf, false>(ya, t, n);
        const uint32_t ra = r.template load<kHalf, false>(t, n);
        body(t, n, std::false_type(), xa, ya, ra);
    }
    return t;
}

template <typename T, int N, bool COUPLED, bool SOME, bool PAST, typename Off>
__global__ void __launch_bounds__(64) scan_fwd(ScanGeom g, ScanPlan q, const T *__restrict__ gate,
                                               const T *__restrict__ value, const float *start,
                                               const uint8_t *__restrict__ reset, const int32_t *__restrict__ lengths,
                                               T *__restrict__ out, float *last, float *__restrict__ states)
{
    Lane<N> w;
    if (!w.find(g, q, lengths)) return;
    float h[N] = {};
    if (start) get_f32<N>(start + w.end(g, w.c), h);
    const Line<T, N, Off> o(out, g.out, w);
    // what lies behind the end of a sequence is a state that stands still and zeros
    int t = walk<T, N, SOME, Off>(
        Line<const T, N, Off>(gate, g.gate, w), Line<const T, N, Off>(value, g.value, w), Resets<SOME>(reset, g, w.b), w.t0,
        min(w.t1, w.valid), [&](int t, int n, auto full, const auto &f, const auto &v, uint32_t resets) {
            constexpr bool FULL = decltype(full)::value;
            if (states && t % kBlock == 0 && t < w.t1) put_own<float, N>(states + w.state(g, t), h, w.skip);
            char *to = o.row(t);
            each_step<kHalf, SOME>(resets, [&](int u, bool cut) {
                if (!FULL && t + u >= w.t1) return;
                float y[N] = {};
                if (FULL || u < n) {
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        h[j] = advance<COUPLED>(cut ? 0.f : h[j], Gate<>(f[u].get(j)), v[u].get(j));
                        y[j] = h[j];
                    }
                }
                put_own<T, N, PAST>(o.lane(to), y, w.skip);
                to += o.step;
            });
        });
    const float none[N] = {};
    for (; t < w.t1; ++t) {
        if (states && t % kBlock == 0) put_own<float, N>(states + w.state(g, t), h, w.skip);
        put_own<T, N, PAST>(o.lane(o.row(t)), none, w.skip);
    }
    if (last && w.c == q.chunks - 1) put_own<float, N>(last + w.end(g), h, w.skip);
}

// A chunk as a step of its own: the product of its a (-1 where a reset cuts the state off), and its
// state from zero.  Its steps take a quick form, in which a state behind an infinity, or behind a difference that
// overflows, is not finite until a reset.  Chunks that end so are folded again in the safe form.  Inputs
// that a projection has just left in the cache do not hide the safe form's instructions: forward of 4 x 4000 x 512
// bf16 24.9 us with it for all chunks, 23.4 so (26 both from HBM).
template <typename F>
__device__ __forceinline__ void quick_or_safe(F fold)
{
    if (!__all(fold(std::false_type()))) fold(std::true_type());
}

template <int N>
__device__ __forceinline__ bool all_finite(const float (&v)[N])
{
    bool all = true;
#pragma unroll
    for (int j = 0; j < N; ++j) all &= fabsf(v[j]) < INFINITY;
    return all;
}

// a*x, in the quick form; w is the smaller share, negative where that is a.
__device__ __forceinline__ float through(float w, float x, bool open) { return fmaf(-w, x, open ? x : 0.f); }

// Stores a fold.  A product too small for fp32 stays above 0, so that an infinite state is infinite behind it.
template <int N>
__device__ __forceinline__ void put_fold(const float (&p)[N], const float (&h)[N], bool cut, float *keep, float *add, int skip)
{
    float k[N];
#pragma unroll
    for (int j = 0; j < N; ++j) k[j] = cut ? -1.f : fmaxf(p[j], kLeast);
    put_own<float, N>(keep, k, skip);
    put_own<float, N>(add, h, skip);
}

template <typename T, int N, bool COUPLED, bool SOME, typename Off>
__global__ void __launch_bounds__(64) scan_fold_fwd(ScanGeom g, ScanPlan q, const T *__restrict__ gate,
                                                    const T *__restrict__ value, const uint8_t *__restrict__ reset,
                                                    const int32_t *__restrict__ lengths, float *__restrict__ keep,
                                                    float *__restrict__ add)
{
    Lane<N> w;
    if (!w.find(g, q, lengths)) return;
    const Line<const T, N, Off> fl(gate, g.gate, w), vl(value, g.value, w);
    const Resets<SOME> rl(reset, g, w.b);
    float h[N], p[N];
    bool cut = false;
    quick_or_safe([&](auto safe) {
#pragma unroll
        for (int j = 0; j < N; ++j) h[j] = 0.f, p[j] = 1.f;
        walk<T, N, SOME, Off>(
            fl, vl, rl, w.t0, min(w.t1, w.valid), [&](int, int n, auto full, const auto &f, const auto &v, uint32_t resets) {
                constexpr bool FULL = decltype(full)::value, SAFE = decltype(safe)::value;
                cut |= resets != 0;
                each_step<kHalf, SOME>(resets, [&](int u, bool zero) {
                    if (!FULL && u >= n) return;
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        const Gate<> k(f[u].get(j));
                        const float small = k.open ? k.small : -k.small, before = zero ? 0.f : h[j], x = v[u].get(j);
                        if (SAFE) h[j] = advance<COUPLED>(before, k, x);
                        else if (COUPLED) h[j] = fmaf(small, x - before, k.open ? before : x);
                        else h[j] = through(small, before, k.open) + x;
                        p[j] = through(small, p[j], k.open);
                    }
                });
            });
        return all_finite(h);
    });
    put_fold<N>(p, h, cut, keep + w.end(g, w.c), add + w.end(g, w.c), w.skip);
}

// The state before each chunk (BACK: the gradient behind it), written over `keep`: 16 waves fold a
// sixteenth of the chunks each, then walk them again from what the waves before them give.  A wave's chunks, 16
// at most, are read together: 256 chunks take 4.9 us (9.2 when read one by one).
__device__ __forceinline__ float carry_over(float keep, float add, float h) { return keep < 0.f ? add : fmaf(keep, h, add); }

template <bool BACK>
__global__ void __launch_bounds__(64 * kCarryWaves) scan_carry(int64_t ends, int chunks, const float *__restrict__ first,
                                                   float *keep, const float *__restrict__ add)
{
    __shared__ float part[2][kCarryWaves][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t e = int64_t(blockIdx.x) * 64 + lane;
    const int per = (chunks + kCarryWaves - 1) / kCarryWaves, c0 = min(wave * per, chunks), c1 = min(c0 + per, chunks);
    const bool live = e < ends;
    auto place = [&](int c) { return int64_t(BACK ? chunks - 1 - c : c) * ends + e; };
    float p = 1.f, h = 0.f;
    bool cut = false;
    constexpr int U = kMostChunks / kCarryWaves;
    float k[U], a[U];
    if (live) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c0 + u < c1) {
                k[u] = keep[place(c0 + u)];
                a[u] = add[place(c0 + u)];
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c0 + u < c1) {
                h = carry_over(k[u], a[u], h);
                cut |= k[u] < 0.f;
                p *= k[u];
            }
    }
    part[0][wave][lane] = cut ? -1.f : fmaxf(p, kLeast);
    part[1][wave][lane] = h;
    __syncthreads();
    if (!live) return;
    h = first ? first[e] : 0.f;
    for (int w = 0; w < wave; ++w) h = carry_over(part[0][w][lane], part[1][w][lane], h);
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (c0 + u < c1) {
            keep[place(c0 + u)] = h;
            h = carry_over(k[u], a[u], h);
        }
}

// ---------------------------------------------------------------- backward --
// A block's states are worked out forward from the kept one, leaving two numbers a step: twice the smaller
// share, negative where that is a, and what dgate is of g.  The gates' and values' registers are then
// free for the next block's loads, which fly while the block's gradient is walked back; dout's follow behind it.
template <typename T, int N, bool COUPLED, bool SOME, bool PAST, typename Off>
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
    const Line<const T, N, Off> fl(gate, g.gate, w), vl(value, g.value, w), dl(dout, g.out, w);
    const Line<T, N, Off> dfl(dgate, g.dgate, w), dvl(dvalue, g.dvalue, w);
    const Resets<SOME> rl(reset, g, w.b);
    Vec<T, N> f[kBlock], v[kBlock], d[kBlock];
    float h[N] = {};
    uint32_t resets = 0;
    float share[kBlock][N], slope[kBlock][N];
    auto inputs = [&](auto full, int t, int live) {
        constexpr bool FULL = decltype(full)::value;
        fl.template load<kBlock, FULL>(f, t, live);
        vl.template load<kBlock, FULL>(v, t, live);
        if (FULL || live > 0) get_f32<N>(states + w.state(g, t), h);
    };
    auto gradients = [&](auto full, int t, int live) {
        constexpr bool FULL = decltype(full)::value;
        dl.template load<kBlock, FULL>(d, t, live);
        resets = rl.template load<kBlock, FULL>(t, live);
    };
    auto forward = [&](auto full, int live) {
        constexpr bool FULL = decltype(full)::value;
        each_step<kBlock, SOME>(resets, [&](int u, bool cut) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                // Half the difference does not overflow.  Behind an infinite state h is NaN within a block: dgate is not
                // finite there either way.
                const Gate<2> k(f[u].get(j));
                const float before = cut ? 0.f : h[j], x = v[u].get(j);
                const float half = COUPLED ? fmaf(0.5f, before, -0.5f * x) : 0.5f * before;
                const float two = k.open ? k.small : -k.small;
                float after = fmaf(-two, half, k.open ? before : COUPLED ? x : 0.f);
                if (!COUPLED) after += x;
                // by selections: from stores on two sides of a branch the compiler makes arrays in memory
                const bool valid = FULL || u < live;
                share[u][j] = valid ? two : 0.f;
                slope[u][j] = valid ? k.small * k.large * half : 0.f;
                h[j] = valid ? after : h[j];
            }
        });
    };
    auto backward = [&](auto full, int t, int n, int live) {
        constexpr bool FULL = decltype(full)::value;
        char *to_gate = dfl.row(t + kBlock), *to_value = dvl.row(t + kBlock);
        each_step<kBlock, SOME>(SOME ? __brev(resets) >> (32 - kBlock) : 0, [&](int k, bool cut) {
            const int u = kBlock - 1 - k;
            to_gate -= dfl.step;
            to_value -= dvl.step;
            if (!FULL && u >= n) return;
            float yf[N] = {}, yv[N] = {};
            if (FULL || u < live) {
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const float gr = back[j] + d[u].get(j), s = 0.5f * fabsf(share[u][j]);
                    const bool open = !signbit(share[u][j]);
                    const float less = s * gr, more = rest(s, gr);
                    yf[j] = slope[u][j] * gr;
                    yv[j] = !COUPLED ? gr : open ? less : more;
                    back[j] = cut ? 0.f : open ? more : less;
                }
            }
            put_own<T, N, PAST>(dfl.lane(to_gate), yf, w.skip);
            put_own<T, N, PAST>(dvl.lane(to_value), yv, w.skip);
        });
    };
    // blocks from the last one back: with checks until every step is valid in every thread of the wave
    const int t1 = min(w.t1, w.valid);
    int t = w.t0 + (w.t1 - w.t0 + kBlock - 1) / kBlock * kBlock - kBlock;
    for (; t >= w.t0 && !__all(t + kBlock <= t1); t -= kBlock) {
        const int n = min(kBlock, w.t1 - t), live = min(kBlock, t1 - t);
        inputs(std::false_type(), t, live);
        gradients(std::false_type(), t, live);
        forward(std::false_type(), live);
        backward(std::false_type(), t, n, live);
    }
    if (t >= w.t0) {
        inputs(std::true_type(), t, 0);
        gradients(std::true_type(), t, 0);
        for (;; t -= kBlock) {
            const bool more = t > w.t0;
            forward(std::true_type(), 0);
            if (more) inputs(std::true_type(), t - kBlock, 0);
            backward(std::true_type(), t, 0, 0);
            if (!more) break;
            gradients(std::true_type(), t - kBlock, 0);
        }
    }
    if (dh0 && w.c == 0) put_own<float, N>(dh0 + w.end(g), back, w.skip);
}

template <typename T, int N, bool SOME, typename Off>
__global__ void __launch_bounds__(64) scan_fold_bwd(ScanGeom g, ScanPlan q, const T *__restrict__ gate,
                                                    const T *__restrict__ dout, const uint8_t *__restrict__ reset,
                                                    const int32_t *__restrict__ lengths, float *__restrict__ keep,
                                                    float *__restrict__ add)
{
    Lane<N> w;
    if (!w.find(g, q, lengths)) return;
    const Line<const T, N, Off> fl(gate, g.gate, w), dl(dout, g.out, w);
    const Resets<SOME> rl(reset, g, w.b);
    float back[N], p[N];
    bool cut = false;
    quick_or_safe([&](auto safe) {
#pragma unroll
        for (int j = 0; j < N; ++j) back[j] = 0.f, p[j] = 1.f;
        Vec<T, N> fa[kHalf], da[kHalf], fb[kHalf], db[kHalf];
        const int t1 = min(w.t1, w.valid);
        auto body = [&](int n, auto full, const Vec<T, N>(&f)[kHalf], const Vec<T, N>(&d)[kHalf], uint32_t resets) {
            constexpr bool FULL = decltype(full)::value, SAFE = decltype(safe)::value;
            cut |= resets != 0;
            each_step<kHalf, SOME>(SOME ? __brev(resets) >> (32 - kHalf) : 0, [&](int k, bool zero) {
                const int u = kHalf - 1 - k;
                if (!FULL && u >= n) return;
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const Gate<> gate(f[u].get(j));
                    const float small = gate.open ? gate.small : -gate.small, gr = back[j] + d[u].get(j);
                    if (SAFE) back[j] = zero ? 0.f : gate.open ? rest(gate.small, gr) : gate.small * gr;
                    else back[j] = zero ? 0.f : through(small, gr, gate.open);
                    p[j] = through(small, p[j], gate.open);
                }
            });
        };
        // halves from the last one back; t is the first step of the half behind the next
        int t = w.t0 + (w.t1 - w.t0 + kHalf - 1) / kHalf * kHalf;
        while (t > w.t0 && !__all(t <= t1 && t - w.t0 >= kBlock)) {
            t -= kHalf;
            const int n = min(kHalf, t1 - t);
            fl.template load<kHalf, false>(fa, t, n);
            dl.template load<kHalf, false>(da, t, n);
            body(n, std::false_type(), fa, da, rl.template load<kHalf, false>(t, n));
        }
        if (t > w.t0) {
            // whole halves only; an odd one first, so that pairs are left
            auto fetch = [&](Vec<T, N>(&f)[kHalf], Vec<T, N>(&d)[kHalf], int at) {
                fl.template load<kHalf, true>(f, at, 0);
                dl.template load<kHalf, true>(d, at, 0);
                return rl.template load<kHalf, true>(at, 0);
            };
            if ((t - w.t0) / kHalf % 2) {
                t -= kHalf;
                const uint32_t r = fetch(fa, da, t);
                body(kHalf, std::true_type(), fa, da, r);
            }
            uint32_t ra = fetch(fa, da, t - kHalf);
            while (t > w.t0) {
                const uint32_t rb = fetch(fb, db, t - kBlock);
                body(kHalf, std::true_type(), fa, da, ra);
                t -= kBlock;
                if (t > w.t0) ra = fetch(fa, da, t - kHalf);
                body(kHalf, std::true_type(), fb, db, rb);
            }
        }
        return all_finite(back);
    });
    put_fold<N>(p, back, cut, keep + w.end(g, w.c), add + w.end(g, w.c), w.skip);
}

template <bool BACK>
hipError_t carry(const ScanGeom &g, const ScanPlan &q, const float *first, float *keep, const float *add, hipStream_t s)
{
    const int64_t ends = int64_t(g.B) * g.D;
    hipLaunchKernelGGL((scan_carry<BACK>), dim3(unsigned((ends + 63) / 64)), dim3(64 * kCarryWaves), 0, s, ends, q.chunks,
                       first, keep, add);
    return hipGetLastError();
}

// Calls f(N, COUPLED, SOME, Off) with the plan's channels a thread, the form, whether there are resets,
// and the type of a lane's offset.
template <bool TWO, typename F>
hipError_t with_lanes(const ScanGeom &g, const ScanPlan &q, bool some, F f)
{
    auto with_resets = [&](auto n, auto c, auto off) {
        return some ? f(n, c, std::true_type(), off) : f(n, c, std::false_type(), off);
    };
    auto with_form = [&](auto n, auto off) {
        return g.coupled ? with_resets(n, std::true_type(), off) : with_resets(n, std::false_type(), off);
    };
    if constexpr (TWO)
        if (q.N == 2) return with_form(std::integral_constant<int, 2>(), uint32_t());
    return q.far ? with_form(std::integral_constant<int, 1>(), int64_t())
                 : with_form(std::integral_constant<int, 1>(), uint32_t());
}

// The sequences of a wave lie within 4 GiB of each other, in bytes of the storage type.
bool near(const gc_strides &s, const ScanGeom &g, int nv, int size)
{
    const int64_t others = std::min<int64_t>(g.B - 1, 63 / nv + 1);
    return (__int128)others * s.batch + g.D < (int64_t(1) << 32) / size;
}

}  // namespace

bool plan_scan(const ScanGeom &g, int dtype, bool bwd, bool ragged, ScanPlan &q)
{
    q = ScanPlan{};
    if (int64_t(g.B) * g.D >= int64_t(1) << 31) return false;
    const int blocks = g.T ? (g.T - 1) / kBlock + 1 : 1, size = dtype == GC_F32 ? 4 : 2;
    const int least = vectors(g.D, 2);     // threads of a step's channels, at least
    q.far = !near(g.gate, g, least, size) || !near(g.value, g, least, size) || !near(g.out, g, least, size);
    if (bwd) q.far |= !near(g.dgate, g, least, size) || !near(g.dvalue, g, least, size);
    // Chunks, while a walk leaves most of the chip idle and is long enough to pay for two more launches,
    // so that 2048 waves have two blocks or more each; more than kMostChunks would make the carry longer
    // than it saves.  Walked and in chunks (us): 64 x 128 x 512 bf16 forward 15 and 18; 1 x 200 x 64 15
    // and 12, backward 27 and 15; 1 x 800 x 64 54 and 10; 64 x 512 x 512 (512 waves) fp32 55 and 68.
    // Two channels a thread halve the loads but also the waves: backward of 3 x 12,001 x 776 bf16 97
    // against 116 with one, of 128 x 256 x 512 (512 waves of two) 67 against 52; the forward
    // is never faster with two.
    auto waves_of = [&](int n) { return (int64_t(g.B) * vectors(g.D, n) + 63) / 64; };
    auto chunks_of = [&](int64_t waves) -> int64_t {
        if (!waves || waves >= 512 || blocks < (bwd ? 10 : 15)) return 1;
        return std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(2048 / waves, kMostChunks), blocks / 2));
    };
    q.N = 1;
    if (bwd && dtype == GC_BF16 && g.D >= 2 && !q.far) {
        const int64_t waves = waves_of(2), chunks = chunks_of(waves);
        if (waves * chunks >= (chunks > 1 ? 1536 : 2048)) q.N = 2;
    }
    q.nv = vectors(g.D, q.N);
    // Sequences of their own lengths start with a wave: one that holds two goes step by step, without loads
    // ahead, where either has ended (3 x 12,001 x 777 bf16 of different lengths: 64 us so and 114
    // packed, backward 100 and 112).
    const int wide = ragged && q.nv > 64 && int64_t(g.B) * (q.nv + 63) < int64_t(1) << 31 ? (q.nv + 63) / 64 * 64 : q.nv;
    q.lanes = int64_t(g.B) * wide;
    const int64_t waves = (q.lanes + 63) / 64;
    const int64_t chunks = chunks_of(waves);
    const int per = int((blocks + chunks - 1) / chunks);
    q.len = int(std::min<int64_t>(int64_t(per) * kBlock, 1 << 30));
    q.chunks = (blocks + per - 1) / per;
    auto bytes_of = [&](int64_t n) { return n > 1 ? (size_t(n) * g.B * g.D * 4 + 255) & ~size_t(255) : 0; };
    q.part_bytes = bytes_of(q.chunks);
    // room for the most chunks that any distances lead to
    q.ws_bytes = 2 * bytes_of(std::max(chunks_of(waves_of(1)), bwd && dtype == GC_BF16 ? chunks_of(waves_of(2)) : int64_t(1)));
    // Outputs of large calls go past the cache (512 x 64 x 512 fp32 backward 78 us without, 74 with), but not where
    // rows share words of memory, which would be written in halves (3 x 12,001 x 777 bf16 backward 104 without,
    // 106 with; of different lengths 100 and 106, forward 64 and 70).
    auto words = [&](const gc_strides &s) { return s.step * size % 4 == 0 && (g.B == 1 || s.batch * size % 4 == 0); };
    q.past = size_t(g.B) * g.T * g.D * size * (bwd ? 5 : 3) >= kStreamBytes &&
             (bwd ? words(g.dgate) && words(g.dvalue) : words(g.out));
    q.fd_nv = make_fastdiv(uint32_t(wide));
    q.fd_blocks = make_fastdiv(uint32_t(std::max<int64_t>(1, waves)));
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
    const dim3 grid(unsigned((q.lanes + 63) / 64 * q.chunks));
    return with_lanes<false>(g, q, reset, [&](auto nn, auto form, auto some, auto off) {
        constexpr int N = decltype(nn)::value;
        constexpr bool COUPLED = decltype(form)::value, SOME = decltype(some)::value;
        using Off = decltype(off);
        if (q.chunks > 1) {
            hipLaunchKernelGGL((scan_fold_fwd<T, N, COUPLED, SOME, Off>), grid, dim3(64), 0, s, g, q, f, v, reset, lengths, keep, add);
            if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
            if (const hipError_t e = carry<false>(g, q, h0, keep, add, s); e != hipSuccess) return e;
        }
        return with_past<true>(q.past, [&](auto past) {
            hipLaunchKernelGGL((scan_fwd<T, N, COUPLED, SOME, decltype(past)::value, Off>), grid, dim3(64), 0, s, g, q, f, v,
                               q.chunks > 1 ? keep : h0, reset, lengths, static_cast<T *>(out), last, states);
            return hipGetLastError();
        });
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
    const dim3 grid(unsigned((q.lanes + 63) / 64 * q.chunks));
    return with_lanes<sizeof(T) == 2>(g, q, reset, [&](auto nn, auto form, auto some, auto off) {
        constexpr int N = decltype(nn)::value;
        constexpr bool COUPLED = decltype(form)::value, SOME = decltype(some)::value;
        using Off = decltype(off);
        if (q.chunks > 1) {
            hipLaunchKernelGGL((scan_fold_bwd<T, N, SOME, Off>), grid, dim3(64), 0, s, g, q, f, d, reset, lengths, keep, add);
            if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
            if (const hipError_t e = carry<true>(g, q, dlast, keep, add, s); e != hipSuccess) return e;
        }
        return with_past<true>(q.past, [&](auto past) {
            hipLaunchKernelGGL((scan_bwd<T, N, COUPLED, SOME, decltype(past)::value, Off>), grid, dim3(64), 0, s, g, q, f, v,
                               states, reset, lengths, d, q.chunks > 1 ? keep : dlast, static_cast<T *>(dgate),
                               static_cast<T *>(dvalue), dh0);
            return hipGetLastError();
        });
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
