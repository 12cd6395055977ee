// embed_grad_onehot.hip -- the embedding's gradient for small vocabularies, as a
// matrix product:
//     dtable = scale * O * dout,   O[v][k] = 1 where tok[k] == v, else 0
// with O made in registers from the tokens and the product on the matrix cores
// (exact: each product is 1*x or 0*x, the sums are fp32).  No sort, and the time
// does not depend on how often a token occurs.
//
// A workgroup takes 32 columns and kRows rows of the table, and a share of the
// tokens; its four waves take K steps of 32 tokens in turn.  The order of the tokens
// within a step is free as long as both operands share it, so lane (n, q) of a bf16
// step holds tokens 4j + q, j = 0 .. 7: the loads of one j are 4 whole consecutive
// rows, and dout needs no staging and no transposing.  Columns are taken in pairs
// (lane n: 2n and 2n + 1), one load feeding two column blocks.  Token values and row
// offsets are decoded once, into LDS.
//
// 0*Inf and 0*NaN are NaN: a non-finite value of dout would spread over its
// column.  It also leaves a NaN in the sums of rows it does not belong to, so a
// wave that finds a NaN in its sums adds its tokens up again one at a time.
//
// The waves' sums are joined in LDS in order, each workgroup writes one partial, and a
// second launch adds the partials in order: bit-reproducible.  The rollout (1.5 million
// tokens, 128 rows x 32 bf16, 98 MB) takes 31.0 us, of which the sums are 5.  It is not
// bound by memory: with its rows in cache it takes 32.5, without making O and the products
// 25.9, without both 20.0.  So the instructions of a step (12 vector ones for 16 rows of O,
// and two matrix ones) are the loop's time, and what is left is staging the tokens, joining
// the waves and the partials.  In fp32 the minibatch's 6 MB take 13 us and the sums 4.
#include <algorithm>

#include "gc_embed.h"
#include "gc_train.h"
#include "gc_vec.h"

namespace gc {
namespace {

constexpr int kThreads = 256, kWaves = 4;
constexpr int kCols = 32;              // columns of a workgroup
constexpr int kStep = 32;              // tokens of a step
constexpr int kStaged = 3;             // chunks in LDS: read, read by a slower wave, written
constexpr uint16_t kNone = 0xFFFF;

struct OnehotPlan {
    int rows;        // table rows of a workgroup: 32, 64, 128 or 256
    int vblocks, slabs;
    int shares;      // workgroups the tokens are divided among
    int steps;       // steps a wave takes of a staged chunk
    uint32_t chunks;
    size_t bytes;
};

// First column of slab `s`: the last one ends with the row, and shares columns with the one before.
__host__ __device__ __forceinline__ int slab_column(int s, int D) { return D > kCols ? min(s * kCols, D - kCols) : 0; }
// Column of slot i (0 .. 31) of a slab; rows shorter than a slab repeat their last pair.
__device__ __forceinline__ int slot_column(int c0, int i, int D) { return min(c0 + (i & ~1), D - 2) + (i & 1); }

// Where the sum of row v (of a block) and slot i lies: as the matrix instructions
// leave it, [16 rows][half of the column pairs][lane][4 rows].
__device__ __forceinline__ int sum_place(int v, int i)
{
    return ((v / 16 * 2 + i % 2) * 64 + v % 16 / 4 * 16 + i / 2) * 4 + v % 4;
}

// ones (bf16) where the two tokens of t equal v, zeros elsewhere: 1 - x without going
// below 0 is 1 only for x = 0.  In assembly, as the compiler makes two compares, two
// selects and a byte shuffle of it (the rollout's gradient: 42 us that way, 36 this).
__device__ __forceinline__ uint32_t onehot2(uint32_t t, uint32_t v2)
{
    uint32_t a;
    asm("v_pk_sub_u16 %0, 1, %1 op_sel_hi:[0,1] clamp" : "=v"(a) : "v"(t ^ v2));
    asm("v_pk_mul_lo_u16 %0, %1, %2" : "=v"(a) : "v"(a), "v"(0x3F803F80u));
    return a;
}

// A chunk's tokens: STEPS steps for each wave.
template <int STEPS> struct Staged {
    static constexpr int kTokens = kStep * STEPS * kWaves;
    uint16_t key[kTokens];   // [step][q][j]: token 4j + q of the step
    int64_t off[kTokens];    // element offsets of the tokens' rows
};

template <typename T> struct Pair;   // two neighbouring columns of a row
template <> struct Pair<bf16_t> { uint32_t w; };
template <> struct Pair<float> { float x, y; };

template <typename T>
__device__ __forceinline__ Pair<T> load_pair(const T *p)
{
    Pair<T> v;
    __builtin_memcpy(&v, p, sizeof(v));
    return v;
}

// One step: acc[block][half] += O * dout for MB blocks of 16 rows, column pairs' halves.
template <int MB, typename S>
__device__ __forceinline__ void step(const S &s, int st, int q, int m, int v0, const Pair<bf16_t> (&p)[8],
                                     f32x4 (&acc)[MB][2])
{
    uint4 t;
    __builtin_memcpy(&t, &s.key[st * kStep + q * 8], 16);
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        lo[j] = __builtin_amdgcn_perm(p[2 * j + 1].w, p[2 * j].w, 0x05040100);
        hi[j] = __builtin_amdgcn_perm(p[2 * j + 1].w, p[2 * j].w, 0x07060302);
    }
    const bf16x8 b0 = __builtin_bit_cast(bf16x8, lo), b1 = __builtin_bit_cast(bf16x8, hi);
#pragma unroll
    for (int i = 0; i < MB; ++i) {
        const uint32_t v2 = uint32_t(v0 + i * 16 + m) * 0x10001u;
        const uint32_t a[4] = {onehot2(t.x, v2), onehot2(t.y, v2), onehot2(t.z, v2), onehot2(t.w, v2)};
        const bf16x8 av = __builtin_bit_cast(bf16x8, a);
        acc[i][0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, b0, acc[i][0], 0, 0, 0);
        acc[i][1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, b1, acc[i][1], 0, 0, 0);
    }
}

template <int MB, typename S>
__device__ __forceinline__ void step(const S &s, int st, int q, int m, int v0, const Pair<float> (&p)[8],
                                     f32x4 (&acc)[MB][2])
{
    uint16_t t[8];
    __builtin_memcpy(t, &s.key[st * kStep + q * 8], 16);
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            const float a = t[j] == v0 + i * 16 + m ? 1.f : 0.f;
            acc[i][0] = __builtin_amdgcn_mfma_f32_16x16x4f32(a, p[j].x, acc[i][0], 0, 0, 0);
            acc[i][1] = __builtin_amdgcn_mfma_f32_16x16x4f32(a, p[j].y, acc[i][1], 0, 0, 0);
        }
}

template <typename T, int MB, int STEPS>
__global__ void __launch_bounds__(kThreads, MB <= 8 ? 3 : 1) onehot_partials(EmbedGeom g, const void *__restrict__ tok,
                                                            const T *__restrict__ dout, float *__restrict__ part,
                                                            int slabs, int vblocks, int shares, uint32_t chunks)
{
    constexpr int ROWS = MB * 16;
    typedef Staged<STEPS> Stage;
    constexpr int TOKENS = Stage::kTokens, EACH = (TOKENS + kThreads - 1) / kThreads;
    __shared__ union __attribute__((aligned(16))) {
        Stage staged[kStaged];
        float table[ROWS * kCols];
    } lds;
    float *table = lds.table;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n = lane & 15, q = lane >> 4;
    uint32_t id = blockIdx.x;
    const int share = id % shares;
    id /= shares;
    const int c0 = slab_column(id % slabs, g.D);
    const int v0 = int(id / slabs) * ROWS;
    const T *col = dout + min(c0 + 2 * n, g.D - 2);

    f32x4 acc[MB][2];
#pragma unroll
    for (int i = 0; i < MB; ++i) acc[i][0] = acc[i][1] = f32x4{0.f, 0.f, 0.f, 0.f};

    // This thread's tokens of a chunk, read a chunk ahead; past the end an empty
    // token on the last row.
    int64_t ahead[EACH];
    auto read_tokens = [&](uint32_t chunk) {
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            const uint32_t k = chunk * TOKENS + e * kThreads + threadIdx.x;
            ahead[e] = k < g.n ? g.token(tok, k) : -1;
        }
    };
    auto stage_tokens = [&](uint32_t chunk, Stage &s) {
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            const int i = e * kThreads + threadIdx.x;
            if (i >= TOKENS) break;
            const int at = (i & ~31) | (i & 3) << 3 | (i >> 2 & 7);
            s.key[at] = ahead[e] >= 0 && ahead[e] < g.V ? uint16_t(ahead[e]) : kNone;
            s.off[at] = g.row(min(chunk * TOKENS + i, g.n - 1));
        }
    };
    constexpr int RING = STEPS == 1 ? 1 : 4, AHEAD = STEPS == 1 ? 1 : 2;   // steps of rows in registers, and requested early
    Pair<T> p[RING][8];
    auto load = [&](const Stage &s, int st, Pair<T>(&v)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = load_pair(col + s.off[st * kStep + q * 8 + j]);
    };

    // The tokens of the next chunk are staged, and its first rows requested, before
    // the last steps of this one: one barrier a chunk.
    read_tokens(share);
    stage_tokens(share, lds.staged[0]);
    __syncthreads();
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) load(lds.staged[0], u * kWaves + wave, p[u]);
    if (share + shares < chunks) read_tokens(share + shares);
    int b = 0;
    for (uint32_t chunk = share; chunk < chunks; chunk += shares) {
        const int next = b == kStaged - 1 ? 0 : b + 1;
        const bool more = chunk + shares < chunks;
#pragma unroll
        for (int u = 0; u < STEPS; ++u) {
            if (u == STEPS - AHEAD && more) {
                stage_tokens(chunk + shares, lds.staged[next]);
                __syncthreads();
                if (chunk + 2 * shares < chunks) read_tokens(chunk + 2 * shares);
            }
            if (STEPS == 1) {
                step<MB>(lds.staged[b], wave, q, n, v0, p[0], acc);
                if (more) load(lds.staged[next], wave, p[0]);
                continue;
            }
            if (u + AHEAD < STEPS) load(lds.staged[b], (u + AHEAD) * kWaves + wave, p[(u + AHEAD) % RING]);
            else if (more) load(lds.staged[next], (u + AHEAD - STEPS) * kWaves + wave, p[(u + AHEAD) % RING]);
            step<MB>(lds.staged[b], u * kWaves + wave, q, n, v0, p[u], acc);
        }
        b = next;
    }
    __syncthreads();

    // the waves in order, in the accumulators' own layout
    bool nan = false;
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) nan |= acc[i][e / 4][e % 4] != acc[i][e / 4][e % 4];
    nan = __ballot(nan) != 0;
    f32x4 *sums = reinterpret_cast<f32x4 *>(table);
    for (int w = 0; w < kWaves; ++w) {
        if (w) __syncthreads();
        if (w != wave) continue;
        if (!nan) {
#pragma unroll
            for (int i = 0; i < 2 * MB; ++i) {
                f32x4 s = acc[i / 2][i % 2];
                if (w) s += sums[i * 64 + lane];
                sums[i * 64 + lane] = s;
            }
            continue;
        }
        // non-finite values: token by token, lanes 0 .. 31 a column each
        if (w == 0)
            for (int i = lane; i < ROWS * kCols; i += 64) table[i] = 0.f;
        for (uint32_t chunk = share; chunk < chunks; chunk += shares)
            for (int i = 0; i < TOKENS; ++i) {
                const uint32_t k = chunk * TOKENS + i;
                if ((i / kStep) % kWaves != wave || k >= g.n) continue;
                const int64_t t = g.token(tok, k) - v0;
                if (t < 0 || t >= ROWS || t + v0 >= g.V || lane >= kCols) continue;
                table[sum_place(int(t), lane)] += to_f32(dout[g.row(k) + slot_column(c0, lane, g.D)]);
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            }
    }
    __syncthreads();
    f32x4 *o = reinterpret_cast<f32x4 *>(part) + size_t(blockIdx.x) * (ROWS * kCols / 4);
    for (int i = threadIdx.x; i < ROWS * kCols / 4; i += kThreads) o[i] = sums[i];
}

// Sums over the shares, in order; a workgroup takes 32 neighbouring places of a
// block of rows and a slab.
template <typename T>
__global__ void __launch_bounds__(1024) onehot_sum(int V, int D, const float *__restrict__ part,
                                                   T *__restrict__ dtable, float scale, int slabs, int shares,
                                                   int rows)
{
    __shared__ float red[32][33];
    const int i = threadIdx.x % 32, lane = threadIdx.x / 32;
    const int stride = rows * kCols;                  // places of a block
    const int place = int(blockIdx.x % rows) * 32 + i;
    const int block = blockIdx.x / rows;              // (block of rows, slab)
    const float *p = part + size_t(block) * shares * stride + place;
    float s[4] = {};
    int w = lane;
    for (; w + 96 < shares; w += 128)
#pragma unroll
        for (int u = 0; u < 4; ++u) s[u] += p[size_t(w + 32 * u) * stride];
    for (; w < shares; w += 32) s[0] += p[size_t(w) * stride];
    red[lane][i] = (s[0] + s[1]) + (s[2] + s[3]);
    __syncthreads();
    for (int h = 16; h > 0; h >>= 1) {
        if (lane < h) red[lane][i] += red[lane + h][i];
        __syncthreads();
    }
    if (lane == 0) {
        // the inverse of sum_place
        const int frag = place / 256, l = place / 4 % 64;
        const int v = block / slabs * rows + frag / 2 * 16 + l / 16 * 4 + place % 4;
        const int slot = l % 16 * 2 + frag % 2, slab = block % slabs;
        const int c = slot_column(slab_column(slab, D), slot, D);
        // columns of the last slab that the one before holds too are that one's: a non-finite value
        // in either gives the two other sums in another order
        if (v < V && c >= slab * kCols) dtable[size_t(v) * D + c] = from_f32<T>(scale * red[0][i]);
    }
}

int block_rows(int V)
{
    int rows = 32;
    while (rows < 256 && rows < V) rows *= 2;
    return rows;
}

OnehotPlan plan(const EmbedGeom &g)
{
    OnehotPlan p{};
    p.rows = block_rows(g.V);
    p.vblocks = (g.V + p.rows - 1) / p.rows;
    p.slabs = (g.D + kCols - 1) / kCols;
    // three workgroups a CU (what their registers allow); with few tokens, chunks of one
    // step a wave spread them over more workgroups
    const int64_t parts = int64_t(p.vblocks) * p.slabs;
    const int64_t most = std::max<int64_t>(1, 768 / parts);
    p.steps = int64_t(g.n) > most * 2 * 4 * kStep * kWaves ? 4 : 1;
    p.chunks = (g.n + p.steps * kStep * kWaves - 1) / (p.steps * kStep * kWaves);
    p.shares = int(std::min<int64_t>(most, p.chunks));
    p.bytes = size_t(parts) * p.shares * p.rows * kCols * sizeof(float);
    return p;
}

template <typename T, int MB>
hipError_t run(const EmbedGeom &g, const OnehotPlan &p, const void *tok, const void *dout, float *part, hipStream_t s)
{
    const dim3 grid(unsigned(p.vblocks * p.slabs * p.shares));
    if (p.steps == 1)
        hipLaunchKernelGGL((onehot_partials<T, MB, 1>), grid, dim3(kThreads), 0, s, g, tok, (const T *)dout, part,
                           p.slabs, p.vblocks, p.shares, p.chunks);
    else
        hipLaunchKernelGGL((onehot_partials<T, MB, 4>), grid, dim3(kThreads), 0, s, g, tok, (const T *)dout, part,
                           p.slabs, p.vblocks, p.shares, p.chunks);
    return hipGetLastError();
}

}  // namespace

int embed_grad_onehot_rows(int V)
{
    const int rows = block_rows(V);
    return (V + rows - 1) / rows * rows;
}

size_t embed_grad_onehot_ws_bytes(const EmbedGeom &g) { return plan(g).bytes; }

template <typename T>
hipError_t launch_embed_grad_onehot(const EmbedGeom &g, const void *tok, const void *dout, void *dtable, float scale,
                                    void *ws, hipStream_t s)
{
    const OnehotPlan p = plan(g);
    float *part = static_cast<float *>(ws);
    hipError_t e;
    switch (p.rows) {
    case 32: e = run<T, 2>(g, p, tok, dout, part, s); break;
    case 64: e = run<T, 4>(g, p, tok, dout, part, s); break;
    case 128: e = run<T, 8>(g, p, tok, dout, part, s); break;
    default: e = run<T, 16>(g, p, tok, dout, part, s); break;
    }
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(onehot_sum<T>, dim3(unsigned(p.vblocks * p.slabs * p.rows)), dim3(1024), 0, s, g.V, g.D, part, (T *)dtable, scale,
                       p.slabs, p.shares, p.rows);
    return hipGetLastError();
}

template hipError_t launch_embed_grad_onehot<float>(const EmbedGeom &, const void *, const void *, void *, float,
                                                    void *, hipStream_t);
template hipError_t launch_embed_grad_onehot<bf16_t>(const EmbedGeom &, const void *, const void *, void *, float,
                                                     void *, hipStream_t);

}  // namespace gc
