// gc_distill.hip -- distillation of a head from a teacher's top logits: the loss, its gradient,
// and both at once.
//
//   p = softmax(teacher / t) over a row's entries,  q = softmax(logits / t)
//   loss = t^2 * sum p * (log p - log q[index]),  dlogits = dloss * t * (q - p at the entries)
//
// Memory bound: the logits are read once (the step holds a row in the registers of its
// team between the row's sum and its gradient), the gradient is written once.  A team of
// threads takes a row: lanes of a wave for short rows, a workgroup for long ones.  The teacher's shares
// are worked out by the row's first wave while the others add up the logits; entries are few.  The
// gradient is written as if there were no entries, then the entries' places are written again
// with all that belongs to them.  Many entries are rather looked up, vector by vector, while the
// gradient is written, as each place written again costs a memory line: steps of 4096 rows of 40,960
// bf16 with 256 entries take 375 us the one way and 192 the other, with 64 entries 166 and 159; with
// 8 entries 145, where a look into the lists for every vector takes 156.  Times, here and below, are of
// passes whose inputs come from HBM.
#include <algorithm>
#include <iterator>
#include <math.h>
#include <type_traits>

#include "gc_core.h"
#include "gc_norm_res.h"

namespace gc {
namespace {

constexpr float kLog2e = 1.44269504088896f;

// A row's entries in LDS, in whole fours: place (-1: empty), share, both logits; the place again where the
// entry is the first one there (else -1), and the shares of all there.  More than kScan entries are
// kept in lists too, a vector's in the list of its number modulo their count, a power of two.
struct Entries {
    int *at;
    float *p, *v, *z;
    int *to;
    float *sum;
    int *next, *first;
};
constexpr int kScan = 16;
__host__ __device__ __forceinline__ int fours(int K) { return (K + 3) & ~3; }
__host__ __device__ __forceinline__ int entry_bytes(int K, int lists)
{
    return K > kScan ? 28 * fours(K) + 4 * lists : 24 * fours(K);
}

constexpr int kOwn = 2;   // entries of a lane that stay in registers

// The backward, which meets a row's logits once, walks longer bf16 rows: its few registers leave room for
// more waves (512 x 150,000 69 us, with the row held 73; 4096 x 40,960 with 256 entries 154 and 160;
// 2048 x 40,961 79 and 82).  In fp32 it loses (4096 x 32,000 205 and 192).
template <typename T>
constexpr int kMostBwd = sizeof(T) == 2 ? 8 : 20;   // vectors that a thread of the backward holds

template <typename V, typename F>
__device__ __forceinline__ V lanes_fold(V v, int width, F f)
{
    for (int m = width >> 1; m > 0; m >>= 1) v = f(v, __shfl_xor(v, m, 64));
    return v;
}

// For each entry: the shares of all entries of its place, in their order, and whether it is the first
// one there.  By one wave, whose LDS accesses are in order.
template <int N>
__device__ __forceinline__ void gather_places(const Entries &entry, int K, int lists, int lane, int width)
{
    const int kp = fours(K);
    auto list_of = [&](int at) { return at / N & (lists - 1); };
    if (K > kScan) {
        for (int k = lane; k < lists / 4; k += width) reinterpret_cast<int4 *>(entry.first)[k] = int4{-1, -1, -1, -1};
        team_sync(true);
        for (int k = lane; k < K; k += width)
            if (const int at = entry.at[k]; at >= 0) entry.next[k] = atomicExch(entry.first + list_of(at), k);
    }
    team_sync(true);
    for (int k = lane; k < K; k += width) {
        const int at = entry.at[k];
        float p = at >= 0 ? entry.p[k] : 0.f;
        bool alone = K <= kScan ? false : true, first = at >= 0;
        if (K > kScan && at >= 0)
            for (int o = entry.first[list_of(at)]; o >= 0; o = entry.next[o]) alone &= o == k || entry.at[o] != at;
        if (!alone && at >= 0) {
            p = 0.f;
            for (int o = 0; o < kp; o += 4) {
                const int4 four = *reinterpret_cast<const int4 *>(entry.at + o);
                if (four.x != at && four.y != at && four.z != at && four.w != at) continue;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool same = (j == 0 ? four.x : j == 1 ? four.y : j == 2 ? four.z : four.w) == at;
                    if (same) p += entry.p[o + j];
                    first &= !(same && o + j < k);
                }
            }
        }
        entry.to[k] = first ? at : -1;
        entry.sum[k] = p;
    }
}

// Makes the compiler work out anew what depends on this number: the places of a row's vectors would
// take more registers than the vectors do.
__device__ __forceinline__ int64_t anew(int64_t i)
{
    int v = int(i);
    asm volatile("" : "+v"(v));
    return v;
}

// exp((z - peak) / t), NaN where both are infinite alike
__device__ __forceinline__ float share(float z, float peak, float c) { return __builtin_amdgcn_exp2f((z - peak) * c); }

// OP: GC_OP_FWD writes loss, peak and mass, GC_OP_BWD reads the last two and writes dlogits,
// GC_OP_STEP writes loss and dlogits.  NV vectors of a row stay in registers, 0: the row is walked.
template <typename T, int N, int NV, int OP, bool PAST>
__global__ void __launch_bounds__(1024) distill(DistillGeom g, int L, int lists, const T *logits, const void *__restrict__ index,
                                                const void *__restrict__ teacher, float *__restrict__ peak,
                                                float *__restrict__ mass, const float *__restrict__ dloss,
                                                float *__restrict__ loss, T *dlogits)
{
    __shared__ float red[2][16];
    __shared__ int any[32];      // whether a team's row has entries
    extern __shared__ int4 all[];
    const int tt = threadIdx.x & (L - 1), team = threadIdx.x / L, teams = blockDim.x / L;
    const int64_t row = int64_t(blockIdx.x) * teams + team;
    if (row >= g.rows) return;   // a whole team; a team of several waves is alone in its workgroup
    const int kp = fours(g.K);
    Entries entry;
    entry.at = reinterpret_cast<int *>(reinterpret_cast<char *>(all) + team * entry_bytes(g.K, lists));
    entry.p = reinterpret_cast<float *>(entry.at + kp);
    entry.v = entry.p + kp;
    entry.z = entry.v + kp;
    entry.to = reinterpret_cast<int *>(entry.z + kp);
    entry.sum = reinterpret_cast<float *>(entry.to + kp);
    entry.next = reinterpret_cast<int *>(entry.sum + kp);
    entry.first = entry.next + kp;
    const T *z = logits + row * g.ld;
    const float t = g.temperature, c = kLog2e / t;
    const int nv = vectors(g.V, N);
    const auto most = [](float a, float b) { return fmaxf(a, b); };
    const auto plus = [](float a, float b) { return a + b; };
    constexpr int U = NV ? NV : 4;      // vectors whose loads fly together
    // the step keeps the exponentials of short rows instead of working them out again
    constexpr bool KEEP = OP == GC_OP_STEP && NV > 0 && NV * N <= 48;

    Vec<T, N> held[U];
    float shares[KEEP ? U : 1][N];
    auto fetch = [&](int64_t i) {
#pragma unroll
        for (int u = 0; u < U; ++u) held[u] = load_vec<T, N>(z + Place<N, int64_t>(i + int64_t(u) * L, g.V).at);
    };
    // the teacher's shares, by the team's first wave; a lane's first entries stay in registers
    const int width = L < 64 ? L : 64, lane = tt & (width - 1);
    const bool leads = tt < width;
    auto entry_at = [&](int k, int &at, float &v) {
        const int64_t i = g.i64 ? static_cast<const int64_t *>(index)[row * g.ld_index + k]
                                : static_cast<const int32_t *>(index)[row * g.ld_index + k];
        at = i >= 0 && i < g.V ? int(i) : -1;
        v = g.t32 ? static_cast<const float *>(teacher)[row * g.ld_teacher + k]
                  : to_f32(static_cast<const bf16_t *>(teacher)[row * g.ld_teacher + k]);
        if (at < 0) v = -INFINITY;
    };
    int own_at[kOwn];
    float own_v[kOwn], own_z[kOwn], top = -INFINITY, total = 0.f, inv_total = 0.f;
    // The loss reads the entries' logits, the backward where it writes their places again (2048 x 40,961 bf16 with
    // 64 entries 79 us without the reads, 81 with; 4096 x 40,960 with 256 154 and 153).
    const bool reads = OP != GC_OP_BWD || g.K <= kScan;
    auto logit = [&](int at) { return reads && at >= 0 ? to_f32(z[at]) : 0.f; };
    // f(k, place, teacher's logit, student's logit) for the lane's entries
    auto each_entry = [&](auto f) {
#pragma unroll
        for (int e = 0; e < kOwn; ++e)
            if (lane + e * width < g.K) f(lane + e * width, own_at[e], own_v[e], own_z[e]);
        for (int k = lane + kOwn * width; k < g.K; k += width) {
            int at;
            float v;
            entry_at(k, at, v);
            f(k, at, v, logit(at));
        }
    };
    bool some = false;
    if (leads) {
#pragma unroll
        for (int e = 0; e < kOwn; ++e)
            if (lane + e * width < g.K) entry_at(lane + e * width, own_at[e], own_v[e]);
    }
    // behind the entries, which are waited for first
    fetch(tt);
    float m = 0.f, s = 0.f, scale = 0.f;
    if (OP == GC_OP_BWD) {
        m = peak[row];
        s = mass[row];
    }
    if (OP != GC_OP_FWD) scale = dloss[row];
    if (leads) {
#pragma unroll
        for (int e = 0; e < kOwn; ++e)
            if (lane + e * width < g.K) own_z[e] = logit(own_at[e]);
        each_entry([&](int, int, float v, float) { top = fmaxf(top, v != v ? INFINITY : v); });
        top = lanes_fold(top, width, most);
        some = top > -INFINITY;
        each_entry([&](int, int, float v, float) { total += v == -INFINITY ? 0.f : share(v, top, c); });
        total = lanes_fold(total, width, plus);
        inv_total = 1.f / total;
        if (tt == 0) any[team] = some;
        if (OP != GC_OP_FWD) {
            each_entry([&](int k, int at, float v, float x) {
                entry.at[k] = at;
                entry.p[k] = v == -INFINITY ? 0.f : share(v, top, c) * inv_total;
                entry.v[k] = v;
                entry.z[k] = x;
            });
            if (g.K + lane < kp) entry.at[g.K + lane] = -1;
            gather_places<N>(entry, g.K, lists, lane, width);
        }
    }

    // The student's largest logit and the sum of the exponentials: each thread around its own largest,
    // so that one exchange joins both.
    float mine = -INFINITY, base = 0.f;
    if (OP != GC_OP_BWD) {
        auto add = [&](int64_t i) {
            i = anew(i);
            float high = mine;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const Place<N, int64_t> at(i + int64_t(u) * L, g.V);
#pragma unroll
                for (int j = 0; j < N; ++j) high = fmaxf(high, j >= at.skip ? held[u].get(j) : -INFINITY);
            }
            keep_packed(held);
            i = anew(i);
            base = high == -INFINITY ? 0.f : high;   // nothing yet but masked logits
            if (!NV) s *= share(mine, base, c);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const Place<N, int64_t> at(i + int64_t(u) * L, g.V);
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const float e = j >= at.skip ? share(held[u].get(j), base, c) : 0.f;
                    if (KEEP) shares[u][j] = e;
                    s += e;
                }
            }
            mine = high;
        };
        if (NV) add(tt);
        else
            for (int64_t i = tt; i < nv; i += int64_t(U) * L) {
                if (i != tt) fetch(i);
                add(i);
            }
        // joins two pairs; a thread without a logit above -inf has s == 0
        m = mine;
        auto join = [&](float m2, float s2) {
            const float high = fmaxf(m, m2);
            s = (m == high ? s : s * share(m, high, c)) + (m2 == high ? s2 : s2 * share(m2, high, c));
            m = high;
        };
        for (int w = width >> 1; w > 0; w >>= 1) {
            const float m2 = __shfl_xor(m, w, 64), s2 = __shfl_xor(s, w, 64);
            join(m2, s2);
        }
        if (L > 64) {
            if ((threadIdx.x & 63) == 0) {
                red[0][threadIdx.x >> 6] = m;
                red[1][threadIdx.x >> 6] = s;
            }
            __syncthreads();
            m = red[0][0];
            s = red[1][0];
            for (int w = 1; w < L >> 6; ++w) join(red[0][w], red[1][w]);
        }
    }
    if (OP == GC_OP_FWD && tt == 0) {
        if (peak) peak[row] = m;
        if (mass) mass[row] = s;
    }
    if (OP != GC_OP_BWD && leads) {
        // log q = (z - peak)/t - log(mass), log p = (teacher - top)/t - log(total)
        const float log_s = logf(s), log_total = logf(total);
        float sum = 0.f;
        auto add = [&](float p, float v, float x) {
            // a masked logit's share is 0, but in a row whose sum is NaN
            if (some && p != 0.f)
                sum += x == -INFINITY && s == s ? INFINITY : p * (((v - top) - (x - m)) / t - log_total + log_s);
        };
        if (OP == GC_OP_FWD)
            each_entry([&](int, int, float v, float x) { add(v == -INFINITY ? 0.f : share(v, top, c) * inv_total, v, x); });
        else
            for (int k = lane; k < g.K; k += width) add(entry.p[k], entry.v[k], entry.z[k]);      // this thread's own
        sum = lanes_fold(sum, width, plus);
        if (tt == 0) loss[row] = t * t * sum;
    }
    if (OP == GC_OP_FWD) return;
    if (m == -INFINITY && s == s) {     // of a row of nothing but masked logits every share is 0
        m = 0.f;
        s = INFINITY;
    }

    // the entries are in LDS, and their logits read, should the gradient take their place
    if (OP == GC_OP_BWD || L <= 64) team_sync(L <= 64);
    some = any[team];
    const float by = some ? scale * t : 0.f, inv = by / s;
    // of this thread's exponentials; 0 where all are masked, but in a row whose sum is NaN
    const float own = mine == -INFINITY ? 0.f * inv : share(base, m, c) * inv;
    T *out = dlogits + row * g.ld_grad;
    auto write = [&](int64_t i) {
        if (!KEEP) keep_packed(held);
        i = anew(i);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const Place<N, int64_t> at(i + int64_t(u) * L, g.V);
            if (!at.live) continue;
            float y[N];
#pragma unroll
            for (int j = 0; j < N; ++j) {
                y[j] = KEEP ? shares[u][j] * own : share(held[u].get(j), m, c) * inv;
                if (!some) y[j] = 0.f;
            }
            if (g.K > kScan)
                for (int k = entry.first[(i + int64_t(u) * L) & (lists - 1)]; k >= 0; k = entry.next[k]) {
                    const int place = entry.to[k] - at.at;
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        if (j == place) y[j] -= by * entry.sum[k];
                }
            Vec<T, N> o;
            o.put(y);
            put_own<PAST, T, N>(out + at.at, o, at.skip);
        }
    };
    if (NV) {
        write(tt);
    } else {
        for (int64_t i = tt; i < nv; i += int64_t(U) * L) {
            if (OP == GC_OP_STEP || i != tt) fetch(i);
            write(i);
        }
    }
    if (!some || g.K > kScan) return;
    // the stores above have arrived before any of the entries' begins
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    __builtin_amdgcn_s_waitcnt(0);
    team_sync(L <= 64);
    for (int k = tt; k < g.K; k += L)
        if (const int at = entry.to[k]; at >= 0) out[at] = from_f32<T>(by * (share(entry.z[k], m, c) / s - entry.sum[k]));
}

// Calls f(NV) for the numbers of vectors a thread may hold.
template <typename F>
hipError_t with_held(int nv, F f)
{
    switch (nv) {
    case 0: return f(std::integral_constant<int, 0>());
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 3: return f(std::integral_constant<int, 3>());
    case 4: return f(std::integral_constant<int, 4>());
    case 5: return f(std::integral_constant<int, 5>());
    case 6: return f(std::integral_constant<int, 6>());
    case 8: return f(std::integral_constant<int, 8>());
    case 10: return f(std::integral_constant<int, 10>());
    case 12: return f(std::integral_constant<int, 12>());
    case 16: return f(std::integral_constant<int, 16>());
    case 20: return f(std::integral_constant<int, 20>());
    default: return hipErrorInvalidValue;
    }
}

}  // namespace

void plan_distill(const DistillGeom &g, int dtype, int op, DistillPlan &q)
{
    q = DistillPlan{};
    const int vec = dtype == GC_F32 ? 4 : 8;
    q.N = g.V < vec ? 1 : vec;
    const int64_t nv = vectors(g.V, q.N);
    // The fewest threads whose registers hold the row, so that several rows are at work on a CU and hide each
    // other's waits (bf16 steps of 4096 x 32,000: 256 threads a row 115 us, 512 125; of 2048 x 50,257: 512 threads
    // 115, 1024 134; rows that take all 20 vectors of a thread would rather have twice the threads, 4096 x
    // 40,960 256 threads 158, 512 144, 1024 194), then more while the chip has room for them (512 x 8000
    // bf16: 512 threads 12 us, 64 23).
    const int most = g.V <= 64 * 64 ? 64 / vec : 20;
    q.L = 8;
    while (q.L < 1024 && int64_t(q.L) * most < nv) q.L *= 2;
    while (q.L < 1024 && q.L < nv && g.rows * q.L < kCUs * 1024) q.L *= 2;
    q.threads = std::max(256, q.L);
    q.lists = 4;
    while (q.lists < 4096 && q.lists < nv && q.lists < 64 * g.K) q.lists *= 2;
    while (q.L <= 64 && size_t(q.threads / q.L) * entry_bytes(g.K, q.lists) > 49152) {
        if (q.threads > 64) q.threads /= 2;
        else q.L *= 2;
    }
    if (q.L > 64) q.threads = q.L;
    if (op != GC_OP_FWD) {
        q.NV = int(std::min<int64_t>(21, (nv + q.L - 1) / q.L));
        const int sizes[] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 20};
        const int *next = std::lower_bound(std::begin(sizes), std::end(sizes), q.NV);
        const int held = op != GC_OP_BWD ? 20 : dtype == GC_F32 ? kMostBwd<float> : kMostBwd<bf16_t>;
        q.NV = next == std::end(sizes) || *next > held ? 0 : *next;
    }
    const int teams = q.threads / q.L;
    q.grid = (g.rows + teams - 1) / teams;
    q.lds_bytes = op == GC_OP_FWD ? 0 : size_t(teams) * entry_bytes(g.K, q.lists);
    // Large gradients go past the cache; the backward's do not where rows share 16 bytes of memory, which would be
    // written in parts (4096 x 50,257 bf16 191 us past, 181 not, 4096 x 40,960 154 and 158; a step of 2048 x 40,961
    // fp32 157 past and 166 not).
    const int size = dtype == GC_F32 ? 4 : 2;
    q.past = op != GC_OP_FWD && q.N > 1 && size_t(g.rows) * g.V * 2 * size >= kStreamBytes &&
             (op == GC_OP_STEP || g.ld_grad * size % 16 == 0);
}

template <typename T>
hipError_t launch_distill(const DistillGeom &g, const DistillPlan &q, int op, const void *logits, const void *index,
                          const void *teacher, float *peak, float *mass, const float *dloss, float *loss, void *dlogits,
                          hipStream_t s)
{
    if (!g.rows) return hipSuccess;
    auto go = [&](auto n, auto nv, auto o, auto past) {
        hipLaunchKernelGGL((distill<T, decltype(n)::value, decltype(nv)::value, decltype(o)::value, decltype(past)::value>),
                           dim3(unsigned(q.grid)), dim3(q.threads), q.lds_bytes, s, g, q.L, q.lists,
                           static_cast<const T *>(logits), index, teacher, peak, mass, dloss, loss, static_cast<T *>(dlogits));
        return hipGetLastError();
    };
    using Fwd = std::integral_constant<int, GC_OP_FWD>;
    using Bwd = std::integral_constant<int, GC_OP_BWD>;
    using Step = std::integral_constant<int, GC_OP_STEP>;
    using None = std::integral_constant<int, 0>;
    auto with_op = [&](auto n) {
        constexpr bool WIDE = decltype(n)::value > 1;
        if (op == GC_OP_FWD) return go(n, None(), Fwd(), std::false_type());
        if constexpr (!WIDE) {
            const std::integral_constant<int, 1> one;
            return op == GC_OP_BWD ? go(n, one, Bwd(), std::false_type()) : go(n, one, Step(), std::false_type());
        } else {
            return with_held(q.NV, [&](auto nv) {
                return with_past<true>(q.past, [&](auto past) {
                    if (op != GC_OP_BWD) return go(n, nv, Step(), past);
                    if constexpr (decltype(nv)::value <= kMostBwd<T>) return go(n, nv, Bwd(), past);
                    return hipErrorInvalidValue;
                });
            });
        }
    };
    if (q.N == 1) return with_op(std::integral_constant<int, 1>());
    return with_op(std::integral_constant<int, kVec<T>>());
}

#define GC_DISTILL_INSTANCES(T)                                                                                     \
    template hipError_t launch_distill<T>(const DistillGeom &, const DistillPlan &, int, const void *, const void *, \
                                          const void *, float *, float *, const float *, float *, void *, hipStream_t);
GC_DISTILL_INSTANCES(float)
GC_DISTILL_INSTANCES(bf16_t)

}  // namespace gc
