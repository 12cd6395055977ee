// embed_fwd.hip -- embedding lookup with scaling:
//     out[r][t][:] = scale * table[tok[r][t]][:],   zeros where tok is not in [0, V)
// Rows of out may lie further apart than tokens*D elements (the embedding as a
// part of a wider feature row).
//
// One thread moves 16-byte vectors; a row of D elements takes ceil(D / vector)
// of them, its last moved back to end with the row (the overlap is written
// twice with the same values), so odd D needs no tail.  Rows shorter than a
// vector go element by element.  Each thread keeps kUnroll independent
// token -> row -> store chains in flight (2 chains: 16.3 us for 98 MB of output, 4 chains
// 18.3).  Bound by memory: the output's bytes, 98 MB at 6.2 TB/s, and as many table rows as
// are not in cache.
#include <algorithm>

#include "gc_embed.h"
#include "gc_train.h"
#include "gc_vec.h"

namespace gc {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 2;

template <typename T, int N, bool PAST>
__global__ void __launch_bounds__(kThreads) embed_rows(EmbedGeom g, const void *__restrict__ tok,
                                                       const T *__restrict__ table, T *__restrict__ out,
                                                       float scale, FastDiv fd_vec, int rows_wg)
{
    // this workgroup's tokens and the vectors in them
    const int64_t tok0 = int64_t(blockIdx.x) * rows_wg;
    const int ntok = int(min(int64_t(rows_wg), int64_t(g.n) - tok0));
    const int nvec = ntok * int(fd_vec.d);
    for (int i0 = threadIdx.x; i0 < nvec; i0 += kThreads * kUnroll) {
        Vec<T, N> v[kUnroll];
        int64_t id[kUnroll];
        int at[kUnroll];
        uint32_t k[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = i0 + u * kThreads;
            uint32_t q = 0, r = 0;
            if (i < nvec) fdivmod(uint32_t(i), fd_vec, q, r);
            k[u] = uint32_t(tok0) + q;
            at[u] = min(int(r) * N, g.D - N);
            id[u] = i < nvec ? g.token(tok, k[u]) : -1;
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (id[u] >= 0 && id[u] < g.V) v[u] = load_vec<T, N>(table + size_t(id[u]) * g.D + at[u]);
            else v[u] = Vec<T, N>{};
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = i0 + u * kThreads;
            if (i >= nvec) break;
            float f[N];
#pragma unroll
            for (int j = 0; j < N; ++j) f[j] = scale * v[u].get(j);
            if (!(id[u] >= 0 && id[u] < g.V)) {   // zeros whatever the scale's sign
#pragma unroll
                for (int j = 0; j < N; ++j) f[j] = 0.f;
            }
            Vec<T, N> o;
            o.put(f);
            put_vec<PAST>(out + g.row(k[u]) + at[u], o);
        }
    }
}

template <typename T, int N>
hipError_t launch(const EmbedGeom &g, const void *tok, const void *table, void *out, float scale, hipStream_t s)
{
    const int per_row = vectors_of<N>(g.D);
    // one round of the loop, and more only to keep the launch below 2^32 threads
    const int rows_wg = std::max(std::max(1, kThreads * kUnroll / per_row), int(g.n >> 23));
    const unsigned grid = unsigned((int64_t(g.n) + rows_wg - 1) / rows_wg);
    const bool past = size_t(g.n) * g.D * sizeof(T) >= kStreamBytes;
    hipLaunchKernelGGL((past ? embed_rows<T, N, true> : embed_rows<T, N, false>), dim3(grid), dim3(kThreads), 0, s, g,
                       tok, (const T *)table, (T *)out, scale, make_fastdiv(per_row), rows_wg);
    return hipGetLastError();
}

}  // namespace

template <typename T>
hipError_t launch_embed_fwd(const EmbedGeom &g, const void *tok, const void *table, void *out, float scale,
                            hipStream_t s)
{
    if (g.n == 0) return hipSuccess;
    if (g.D >= kVec<T>) return launch<T, kVec<T>>(g, tok, table, out, scale, s);
    return launch<T, 1>(g, tok, table, out, scale, s);
}

template hipError_t launch_embed_fwd<float>(const EmbedGeom &, const void *, const void *, void *, float, hipStream_t);
template hipError_t launch_embed_fwd<bf16_t>(const EmbedGeom &, const void *, const void *, void *, float, hipStream_t);

}  // namespace gc
