// embed_grad_sort.hip -- the embedding's gradient by sorted tokens:
//     dtable[v][:] = scale * sum over the tokens k with tok[k] == v of dout[k][:]
// in fp32, every sum in an order that the sorted positions alone fix, so the
// result is bit-reproducible; no atomics on values.
//
//   1. A stable radix sort of (token, position), 8 bits a pass: digit counts
//      per tile, (for many tiles a scan of the counts over the tiles,) then
//      each tile ranks its keys and scatters them; up to 4096 tokens are sorted by one
//      workgroup in one launch.  Tokens outside [0, V) carry the key V and end up
//      behind all rows.
//   2. Long runs of one token: every kRun sorted positions that hold one token
//      are summed into a partial row, and likewise every kRun partials of a level into
//      one of the next, all tiles in parallel.  Other tiles cost nothing.  The
//      first launch also notes where each token's run begins and ends.
//   3. Each row of the table adds up its run: positions to the first tile
//      boundary, partials to the first boundary of the next level, and so on up and
//      down again.  Rows without a token are written as zeros; they are known by
//      their noted place not being a run of theirs, so the notes need no clearing.
// Bound by memory: dout is gathered once by rows, dtable written once (32,768 tokens, 40,960
// rows of 1024 bf16: rows 35 us for 146 MB, runs 7 and 5, sort 22); at few tokens by the chain
// of launches.  Bisecting the keys for every row, with rows in order and runs of 64, took
// 222 us for the call instead of 64.
#include <algorithm>

#include "gc_embed.h"
#include "gc_train.h"
#include "gc_vec.h"

namespace gc {
namespace {

constexpr int kThreads = 256;
constexpr int kRun = 32;             // sorted positions of a partial, and partials of one of the next level
constexpr int kLevels = 3;           // partials of 32, 1024 and 32,768 positions
constexpr int kScanTiles = 32;       // more tiles than this are scanned by a launch of their own
constexpr int kInFlight = 8;         // rows a thread has requested at once

// ---------------------------------------------------------------- sorting --
// Key of position i: pass 0 reads the caller's tokens, later passes the
// previous pass's output.
struct SortIn {
    const void *tok;
    const uint32_t *key, *idx;
};
__device__ __forceinline__ uint32_t sort_key(const EmbedGeom &g, const SortIn &in, uint32_t i)
{
    if (in.key) return in.key[i];
    const int64_t t = g.token(in.tok, i);
    return t >= 0 && t < g.V ? uint32_t(t) : uint32_t(g.V);
}

// counts[tile][digit]
template <int ROUNDS>
__global__ void __launch_bounds__(kThreads) sort_count(EmbedGeom g, SortIn in, int shift,
                                                       uint32_t *__restrict__ counts)
{
    __shared__ uint32_t hist[256];
    hist[threadIdx.x] = 0;
    __syncthreads();
    const uint32_t base = blockIdx.x * (kThreads * ROUNDS);
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        const uint32_t i = base + r * kThreads + threadIdx.x;
        if (i < g.n) atomicAdd(&hist[sort_key(g, in, i) >> shift & 255], 1u);
    }
    __syncthreads();
    counts[size_t(blockIdx.x) * 256 + threadIdx.x] = hist[threadIdx.x];
}

// One workgroup a digit: counts become their exclusive prefix over the tiles,
// totals[digit] the sum.
__global__ void __launch_bounds__(kThreads) sort_scan(uint32_t *__restrict__ counts, int tiles,
                                                      uint32_t *__restrict__ totals)
{
    __shared__ uint32_t part[kThreads];
    const int d = blockIdx.x, t = threadIdx.x;
    uint32_t run = 0;
    for (int t0 = 0; t0 < tiles; t0 += kThreads) {
        const int tile = t0 + t;
        const uint32_t c = tile < tiles ? counts[size_t(tile) * 256 + d] : 0;
        part[t] = c;
        __syncthreads();
        for (int w = 1; w < kThreads; w <<= 1) {
            const uint32_t v = t >= w ? part[t - w] : 0;
            __syncthreads();
            part[t] += v;
            __syncthreads();
        }
        if (tile < tiles) counts[size_t(tile) * 256 + d] = run + part[t] - c;
        run += part[kThreads - 1];
        __syncthreads();
    }
    if (t == 0) totals[d] = run;
}

// The rank of a lane's digit among its wave's lanes before it and its wave's
// earlier calls, whose counts `hist` (the wave's own, 256 counters) keeps.  The lanes
// of one digit find each other by ballots over the digit's bits.
__device__ __forceinline__ uint32_t digit_rank(bool valid, uint32_t d, int lane, uint32_t *hist)
{
    uint64_t peers = __ballot(valid);
#pragma unroll
    for (int b = 0; b < 8; ++b) {
        const uint64_t set = __ballot(d >> b & 1);
        peers &= (d >> b & 1) ? set : ~set;
    }
    const uint32_t before = __popcll(peers & ((uint64_t(1) << lane) - 1));
    uint32_t seen = 0;
    if (valid) seen = hist[d];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (valid && before == 0) hist[d] = seen + __popcll(peers);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    return seen + before;
}

// Ranks a tile's keys by their digit (stable) and scatters them; a wave takes 64
// consecutive keys a round.
template <int ROUNDS>
__global__ void __launch_bounds__(kThreads) sort_scatter(EmbedGeom g, SortIn in, int shift,
                                                         const uint32_t *__restrict__ counts,
                                                         const uint32_t *__restrict__ totals, int tiles,
                                                         uint32_t *__restrict__ key_out,
                                                         uint32_t *__restrict__ idx_out)
{
    constexpr int WAVES = kThreads / 64;
    __shared__ uint32_t hist[WAVES][256];
    __shared__ uint32_t scan[256];
    const int t = threadIdx.x, wave = t >> 6, lane = t & 63;
    for (int w = 0; w < WAVES; ++w) hist[w][t] = 0;
    __syncthreads();

    const uint32_t base = blockIdx.x * (kThreads * ROUNDS) + wave * (64 * ROUNDS);
    uint32_t key[ROUNDS], idx[ROUNDS], rank[ROUNDS];
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        const uint32_t i = base + r * 64 + lane;
        key[r] = i < g.n ? sort_key(g, in, i) : 0;
        idx[r] = i < g.n ? (in.key ? in.idx[i] : i) : 0;
    }
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        rank[r] = digit_rank(base + r * 64 + lane < g.n, key[r] >> shift & 255, lane, hist[wave]);
    }

    // thread d: where digit d of this tile starts in the output
    uint32_t total = 0, prefix = 0;
    if (totals) {
        total = totals[t];
        prefix = counts[size_t(blockIdx.x) * 256 + t];
    } else {
#pragma unroll 8
        for (int i = 0; i < tiles; ++i) {
            const uint32_t c = counts[size_t(i) * 256 + t];
            total += c;
            prefix += i < int(blockIdx.x) ? c : 0;
        }
    }
    scan[t] = total;
    __syncthreads();
    for (int w = 1; w < 256; w <<= 1) {
        const uint32_t v = t >= w ? scan[t - w] : 0;
        __syncthreads();
        scan[t] += v;
        __syncthreads();
    }
    uint32_t at = scan[t] - total + prefix;
    for (int w = 0; w < WAVES; ++w) {
        const uint32_t c = hist[w][t];
        hist[w][t] = at;
        at += c;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        if (base + r * 64 + lane >= g.n) continue;
        const uint32_t dst = hist[wave][key[r] >> shift & 255] + rank[r];
        key_out[dst] = key[r];
        idx_out[dst] = idx[r];
    }
}

// All passes for up to kSmall tokens by one workgroup, in LDS, and the runs' ends.
constexpr int kSmall = 4096, kSmallThreads = 1024, kSmallWaves = kSmallThreads / 64;
__global__ void __launch_bounds__(kSmallThreads) sort_small(EmbedGeom g, const void *__restrict__ tok, int passes,
                                                            uint32_t *__restrict__ key_out,
                                                            uint32_t *__restrict__ idx_out,
                                                            uint32_t *__restrict__ first,
                                                            uint32_t *__restrict__ last)
{
    __shared__ uint32_t key[2][kSmall];
    __shared__ uint16_t idx[2][kSmall];
    __shared__ uint32_t hist[kSmallWaves][256];
    __shared__ uint32_t scan[256];
    const int t = threadIdx.x, wave = t >> 6, lane = t & 63, n = int(g.n);
    const SortIn in{tok, nullptr, nullptr};
    for (int i = t; i < n; i += kSmallThreads) {
        key[0][i] = sort_key(g, in, i);
        idx[0][i] = uint16_t(i);
    }
    const int rounds = (n + kSmallThreads - 1) / kSmallThreads;   // of 64 keys a wave, at most 4
    int src = 0;
    for (int pass = 0; pass < passes; ++pass, src ^= 1) {
        const int shift = 8 * pass;
        for (int i = t; i < kSmallWaves * 256; i += kSmallThreads) hist[i / 256][i % 256] = 0;
        __syncthreads();
        uint32_t rank[kSmall / kSmallThreads];
#pragma unroll
        for (int r = 0; r < kSmall / kSmallThreads; ++r) {
            if (r >= rounds) break;
            const int i = (wave * rounds + r) * 64 + lane;
            rank[r] = digit_rank(i < n, i < n ? key[src][i] >> shift & 255 : 0, lane, hist[wave]);
        }
        __syncthreads();
        uint32_t total = 0;
        if (t < 256) {
            for (int w = 0; w < kSmallWaves; ++w) {
                const uint32_t c = hist[w][t];
                hist[w][t] = total;
                total += c;
            }
            scan[t] = total;
        }
        __syncthreads();
        for (int w = 1; w < 256; w <<= 1) {
            const uint32_t v = t < 256 && t >= w ? scan[t - w] : 0;
            __syncthreads();
            if (t < 256) scan[t] += v;
            __syncthreads();
        }
#pragma unroll
        for (int r = 0; r < kSmall / kSmallThreads; ++r) {
            const int i = (wave * rounds + r) * 64 + lane;
            if (r >= rounds || i >= n) break;
            const uint32_t d = key[src][i] >> shift & 255;
            const uint32_t dst = (d ? scan[d - 1] : 0) + hist[wave][d] + rank[r];
            key[src ^ 1][dst] = key[src][i];
            idx[src ^ 1][dst] = idx[src][i];
        }
        __syncthreads();
    }
    for (int i = t; i < n; i += kSmallThreads) {
        const uint32_t k = key[src][i];
        key_out[i] = k;
        idx_out[i] = idx[src][i];
        if (k >= uint32_t(g.V)) continue;
        if (i == 0 || key[src][i - 1] != k) first[k] = i;
        if (i + 1 == n || key[src][i + 1] != k) last[k] = i;
    }
}

// ------------------------------------------------------------------- sums --
// Lanes of a row: `team` (a power of two, at most 256) threads, each owning
// vectors lane, lane + team, ... of the row's D elements.
template <typename T, int N>
__device__ __forceinline__ void add_vec(float (&s)[N], const Vec<T, N> &v)
{
#pragma unroll
    for (int j = 0; j < N; ++j) s[j] += v.get(j);
}

// s += rows idx[a .. b) of dout at column c, in order
template <typename T, int N>
__device__ __forceinline__ void add_positions(const EmbedGeom &g, const T *__restrict__ dout,
                                              const uint32_t *__restrict__ idx, uint32_t a, uint32_t b, int c,
                                              float (&s)[N])
{
    for (; a + kInFlight <= b; a += kInFlight) {
        Vec<T, N> v[kInFlight];
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) v[u] = load_vec<T, N>(dout + g.row(idx[a + u]) + c);
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) add_vec(s, v[u]);
    }
    for (; a < b; ++a) add_vec(s, load_vec<T, N>(dout + g.row(idx[a]) + c));
}

// s += rows a .. b of a partial table at column c
template <int N>
__device__ __forceinline__ void add_partials(const float *__restrict__ part, int D, uint32_t a, uint32_t b, int c,
                                             float (&s)[N])
{
    for (; a + kInFlight <= b; a += kInFlight) {
        Vec<float, N> v[kInFlight];
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) v[u] = load_vec<float, N>(part + size_t(a + u) * D + c);
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) add_vec(s, v[u]);
    }
    for (; a < b; ++a) add_vec(s, load_vec<float, N>(part + size_t(a) * D + c));
}

// The partials of each level: row t of level l sums the kRun^(l+1) sorted positions
// from t * kRun^(l+1) on, and is there if those hold one token of the table.
struct Partials {
    float *part[kLevels];
    uint32_t rows[kLevels];
    int levels;
};

// Level 0, and the runs' ends where `first` is not NULL.
template <typename T, int N>
__global__ void __launch_bounds__(kThreads) run_partials(EmbedGeom g, const T *__restrict__ dout,
                                                         const uint32_t *__restrict__ key,
                                                         const uint32_t *__restrict__ idx, float *__restrict__ part,
                                                         uint32_t *__restrict__ first, uint32_t *__restrict__ last,
                                                         int team)
{
    const uint32_t p = blockIdx.x * (kThreads / team) + threadIdx.x / team;
    const uint32_t a = p * kRun;
    const int lane = threadIdx.x % team;
    for (uint32_t i = a + lane; first && i < min(a + kRun, g.n); i += team) {
        const uint32_t k = key[i];
        if (k >= uint32_t(g.V)) continue;
        if (i == 0 || key[i - 1] != k) first[k] = i;
        if (i + 1 == g.n || key[i + 1] != k) last[k] = i;
    }
    if (a + kRun > g.n) return;
    const uint32_t k = key[a];
    if (k != key[a + kRun - 1] || k >= uint32_t(g.V)) return;
    const int nvec = vectors_of<N>(g.D);
    for (int i = lane; i < nvec; i += team) {
        const int c = min(i * N, g.D - N);
        float s[N] = {};
        add_positions<T, N>(g, dout, idx, a, a + kRun, c, s);
        Vec<float, N> o;
        o.put(s);
        store_vec<float, N>(part + size_t(p) * g.D + c, o);
    }
}

// A level from the one below; `span` positions a row.
template <int N>
__global__ void __launch_bounds__(kThreads) next_partials(int V, int D, const uint32_t *__restrict__ key,
                                                          const float *__restrict__ below,
                                                          float *__restrict__ part, uint32_t rows, uint32_t span,
                                                          int team)
{
    const uint32_t q = blockIdx.x * (kThreads / team) + threadIdx.x / team;
    if (q >= rows) return;
    const uint32_t k = key[q * span];
    if (k != key[q * span + span - 1] || k >= uint32_t(V)) return;
    const int nvec = vectors_of<N>(D);
    for (int i = threadIdx.x % team; i < nvec; i += team) {
        const int c = min(i * N, D - N);
        float s[N] = {};
        add_partials<N>(below, D, q * kRun, (q + 1) * kRun, c, s);
        Vec<float, N> o;
        o.put(s);
        store_vec<float, N>(part + size_t(q) * D + c, o);
    }
}

constexpr int kRowsMax = 256;   // table rows of a workgroup, at most

// Workgroup w takes rows w, w + grid, ...: frequent tokens often are neighbours.
template <typename T, int N, bool PAST>
__global__ void __launch_bounds__(kThreads) table_rows(EmbedGeom g, const T *__restrict__ dout,
                                                       const uint32_t *__restrict__ key,
                                                       const uint32_t *__restrict__ idx, Partials q,
                                                       const uint32_t *__restrict__ first,
                                                       const uint32_t *__restrict__ last, T *__restrict__ dtable,
                                                       float scale, int team, int rows_wg)
{
    __shared__ uint32_t begin[kRowsMax], end[kRowsMax];
    for (int r = threadIdx.x; r < rows_wg; r += kThreads) {
        const int64_t v = blockIdx.x + int64_t(r) * gridDim.x;
        uint32_t a = 0, b = 0;
        if (v < g.V) {
            const uint32_t i = first[v], j = last[v];
            if (i < g.n && key[i] == uint32_t(v) && (i == 0 || key[i - 1] != uint32_t(v))) {
                a = i;
                b = j + 1;
            }
        }
        begin[r] = a;
        end[r] = b;
    }
    __syncthreads();
    const int nvec = vectors_of<N>(g.D);
    const int lane = threadIdx.x % team, teams = kThreads / team;
    for (int r = threadIdx.x / team; r < rows_wg; r += teams) {
        const int64_t v = blockIdx.x + int64_t(r) * gridDim.x;
        if (v >= g.V) break;
        const uint32_t a = begin[r], b = end[r];
        for (int i = lane; i < nvec; i += team) {
            const int c = min(i * N, g.D - N);
            float s[N] = {};
            // up: [at, b) is left in units of level `up`; down: the rest of each level
            uint32_t from[kLevels + 1], to[kLevels + 1];
            uint32_t x = a, y = b;
            int up = 0;
            for (; up < q.levels; ++up) {
                const uint32_t u = (x + kRun - 1) / kRun, w = y / kRun;
                if (u >= w) break;
                if (up == 0) add_positions<T, N>(g, dout, idx, x, u * kRun, c, s);
                else add_partials<N>(q.part[up - 1], g.D, x, u * kRun, c, s);
                from[up] = w * kRun;
                to[up] = y;
                x = u;
                y = w;
            }
            from[up] = x;
            to[up] = y;
            for (; up >= 0; --up) {
                if (up == 0) add_positions<T, N>(g, dout, idx, from[0], to[0], c, s);
                else add_partials<N>(q.part[up - 1], g.D, from[up], to[up], c, s);
            }
#pragma unroll
            for (int j = 0; j < N; ++j) s[j] = a < b ? scale * s[j] : 0.f;
            Vec<T, N> o;
            o.put(s);
            put_vec<PAST>(dtable + v * g.D + c, o);
        }
    }
}

// --------------------------------------------------------------- the plan --
struct SortPlan {
    int rounds;          // 64-key rounds of a wave: the tile is 256 * rounds keys
    int tiles, passes;
    int levels;
    uint32_t rows[kLevels];                                    // partials of each level
    size_t key[2], idx[2], counts, totals, first, last, part[kLevels], bytes;   // byte offsets
};

size_t take(size_t &at, size_t bytes)
{
    const size_t o = at;
    at += (bytes + 255) & ~size_t(255);
    return o;
}

SortPlan plan(const EmbedGeom &g)
{
    SortPlan p{};
    p.rounds = g.n > 131072 ? 16 : 4;
    const uint32_t tile = kThreads * p.rounds;
    p.tiles = int((g.n + tile - 1) / tile);
    int bits = 1;
    while ((uint64_t(1) << bits) <= uint64_t(g.V)) ++bits;   // keys 0 .. V
    p.passes = (bits + 7) / 8;
    // a level pays from a few rows on
    for (uint32_t rows = g.n / kRun; p.levels < kLevels && rows >= 4; rows /= kRun) p.rows[p.levels++] = rows;
    size_t at = 0;
    for (int i = 0; i < 2; ++i) {
        p.key[i] = take(at, size_t(g.n) * 4);
        p.idx[i] = take(at, size_t(g.n) * 4);
    }
    p.counts = take(at, size_t(p.tiles) * 256 * 4);
    p.totals = take(at, 256 * 4);
    p.first = take(at, size_t(g.V) * 4);
    p.last = take(at, size_t(g.V) * 4);
    for (int l = 0; l < p.levels; ++l) p.part[l] = take(at, size_t(p.rows[l]) * g.D * 4);
    p.bytes = at;
    return p;
}

template <int ROUNDS>
hipError_t sort_pass(const EmbedGeom &g, const SortPlan &p, const SortIn &in, int shift, uint32_t *counts,
                     uint32_t *totals, uint32_t *key_out, uint32_t *idx_out, hipStream_t s)
{
    hipLaunchKernelGGL(sort_count<ROUNDS>, dim3(p.tiles), dim3(kThreads), 0, s, g, in, shift, counts);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    const bool scan = p.tiles > kScanTiles;
    if (scan) {
        hipLaunchKernelGGL(sort_scan, dim3(256), dim3(kThreads), 0, s, counts, p.tiles, totals);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(sort_scatter<ROUNDS>, dim3(p.tiles), dim3(kThreads), 0, s, g, in, shift, counts,
                       scan ? totals : nullptr, p.tiles, key_out, idx_out);
    return hipGetLastError();
}

template <typename T, int N>
hipError_t sums(const EmbedGeom &g, const SortPlan &p, const void *dout, const uint32_t *key, const uint32_t *idx,
                char *ws, void *dtable, float scale, hipStream_t s)
{
    const int nvec = vectors_of<N>(g.D);
    int team = 1;
    while (team < nvec && team < kThreads) team <<= 1;
    const int teams = kThreads / team;
    uint32_t *first = reinterpret_cast<uint32_t *>(ws + p.first), *last = reinterpret_cast<uint32_t *>(ws + p.last);
    Partials q{};
    q.levels = p.levels;
    for (int l = 0; l < p.levels; ++l) {
        q.part[l] = reinterpret_cast<float *>(ws + p.part[l]);
        q.rows[l] = p.rows[l];
    }
    const bool noted = g.n <= uint32_t(kSmall);   // the runs' ends, by the sort
    if (p.levels || !noted) {
        const uint32_t tiles = (g.n + kRun - 1) / kRun;
        hipLaunchKernelGGL((run_partials<T, N>), dim3((tiles + teams - 1) / teams), dim3(kThreads), 0, s, g,
                           (const T *)dout, key, idx, q.part[0], noted ? nullptr : first, last, team);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    uint32_t span = kRun;
    for (int l = 1; l < p.levels; ++l) {
        span *= kRun;
        hipLaunchKernelGGL(next_partials<N>, dim3((p.rows[l] + teams - 1) / teams), dim3(kThreads), 0, s, g.V, g.D,
                           key, q.part[l - 1], q.part[l], p.rows[l], span, team);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    const int rows_wg = std::min(kRowsMax, teams * 8);
    const bool past = (size_t(g.n) + g.V) * g.D * sizeof(T) >= kStreamBytes;
    hipLaunchKernelGGL((past ? table_rows<T, N, true> : table_rows<T, N, false>), dim3((uint32_t(g.V) + rows_wg - 1) / rows_wg),
                       dim3(kThreads), 0, s, g, (const T *)dout, key, idx, q, first, last, (T *)dtable, scale, team,
                       rows_wg);
    return hipGetLastError();
}

}  // namespace

size_t embed_grad_sort_ws_bytes(const EmbedGeom &g) { return plan(g).bytes; }

template <typename T>
hipError_t launch_embed_grad_sort(const EmbedGeom &g, const void *tok, const void *dout, void *dtable, float scale,
                                  void *ws, hipStream_t s)
{
    const SortPlan p = plan(g);
    char *base = static_cast<char *>(ws);
    uint32_t *key[2], *idx[2];
    for (int i = 0; i < 2; ++i) {
        key[i] = reinterpret_cast<uint32_t *>(base + p.key[i]);
        idx[i] = reinterpret_cast<uint32_t *>(base + p.idx[i]);
    }
    uint32_t *counts = reinterpret_cast<uint32_t *>(base + p.counts);
    uint32_t *totals = reinterpret_cast<uint32_t *>(base + p.totals);
    SortIn in{tok, nullptr, nullptr};
    const bool small = g.n <= uint32_t(kSmall);
    if (small && g.n) {
        hipLaunchKernelGGL(sort_small, dim3(1), dim3(kSmallThreads), 0, s, g, tok, p.passes, key[0], idx[0],
                           reinterpret_cast<uint32_t *>(base + p.first), reinterpret_cast<uint32_t *>(base + p.last));
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
        in = SortIn{tok, key[0], idx[0]};
    }
    int out = 0;
    for (int pass = 0; pass < p.passes && !small; ++pass) {
        const hipError_t e = p.rounds == 16
            ? sort_pass<16>(g, p, in, 8 * pass, counts, totals, key[out], idx[out], s)
            : sort_pass<4>(g, p, in, 8 * pass, counts, totals, key[out], idx[out], s);
        if (e != hipSuccess) return e;
        in = SortIn{tok, key[out], idx[out]};
        out ^= 1;
    }
    if (g.D >= kVec<T>) return sums<T, kVec<T>>(g, p, dout, in.key, in.idx, base, dtable, scale, s);
    return sums<T, 1>(g, p, dout, in.key, in.idx, base, dtable, scale, s);
}

template hipError_t launch_embed_grad_sort<float>(const EmbedGeom &, const void *, const void *, void *, float,
                                                  void *, hipStream_t);
template hipError_t launch_embed_grad_sort<bf16_t>(const EmbedGeom &, const void *, const void *, void *, float,
                                                   void *, hipStream_t);

}  // namespace gc
