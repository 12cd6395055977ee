// gc_norm_res.h -- pieces of the resident group-norm kernels (norm_res_*.hip):
// groups that stay in the registers of one team of threads between their
// statistics and their output, so every input is read once.
#pragma once

#include <type_traits>

#include "gc_norm.h"
#include "gc_train.h"

namespace gc {

constexpr int kResThreads = 256;   // a workgroup of several teams

// Most threads of a workgroup whose threads hold N*NV elements, by registers: the
// forward holds the packed elements (128 registers a thread at 1024 threads
// do), the backward two fp32 values of each.
constexpr int kHeldMost = 32;   // elements a thread of the backward holds, at most
constexpr int kMixedMost = 8;   // vectors a thread of the forward holds when they mix groups, at most
constexpr int res_threads_fwd(int) { return 1024; }
constexpr int res_threads_bwd(int held) { return held <= 4 ? 1024 : 512; }

// Workgroups are dealt to the chip's 8 dies in turn, each with its own L2.  Neighbouring
// slabs of an image share memory lines: this order gives them to one die, one after
// the other.
__device__ __forceinline__ uint32_t die_order(uint32_t id, uint32_t grid)
{
    const uint32_t per = grid / 8;
    return id < per * 8 ? id % 8 * per + id / 8 : id;
}

// Most vectors of N elements a thread of the small-group kernels holds: with constants
// (and running sums) for each (NCHW), or for all of them (channels last).
constexpr int small_vectors(int N, bool last) { return (last ? 32 : 16) / N; }

// A team is one wave, or the workgroup: LDS traffic within a wave is in order.
__device__ __forceinline__ void team_sync(bool wave)
{
    if (wave) {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    } else {
        __syncthreads();
    }
}

// Makes the compiler forget what it unpacked of bf16 vectors: between two passes over
// them it would rather keep (and spill) the unpacked elements than unpack again.
template <int N, int NV>
__device__ __forceinline__ void keep_packed(Vec<float, N> (&)[NV]) {}
template <int N, int NV>
__device__ __forceinline__ void keep_packed(Vec<bf16_t, N> (&v)[NV])
{
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < (N + 1) / 2; ++j) asm volatile("" : "+v"(v[i].w[j]));
}

// Sum over the L lanes of a team (L <= 64: lanes of a wave; else the
// workgroup is the team, `red` 16 values a call in flight).
template <int K>
__device__ __forceinline__ void team_sum(float (&v)[K], int L, float *red)
{
    const int w = L < 64 ? L : 64;
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = lanes_sum(v[k], w);
    if (L <= 64) return;
    const int nw = L >> 6;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) red[k * 16 + (threadIdx.x >> 6)] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float s = red[k * 16];
        for (int i = 1; i < nw; ++i) s += red[k * 16 + i];
        v[k] = s;
    }
}

// Channels-last teams: per-group sums of K values a thread holds for E entries
// of its row (one when a vector lies in one group, else one a channel).  Every
// thread writes its entries to red[k][slot][width]; P lanes a group add them up in
// a fixed order; stat[k][group] holds the sums for all after the second sync.
template <int K, int E>
__device__ __forceinline__ void team_groups(const NormResPlan &q, bool live, int tt, int slot, int col,
                                            const float (&v)[K][E], float *red, float *stat)
{
    if (live) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int e = 0; e < E; ++e) red[(k * q.slots + slot) * q.width + col * E + e] = v[k][e];
    }
    team_sync(q.wave);
    const int lane = tt & (q.P - 1);
    const int n = q.slots * int(q.fd_Eg.d);
    for (int gg = tt / q.P; gg < q.Gs; gg += q.L / q.P) {
        float s[K] = {};
        for (int i = lane; i < n; i += q.P) {
            uint32_t r, e;
            fdivmod(uint32_t(i), q.fd_Eg, r, e);
#pragma unroll
            for (int k = 0; k < K; ++k) s[k] += red[(k * q.slots + r) * q.width + gg * int(q.fd_Eg.d) + e];
        }
#pragma unroll
        for (int k = 0; k < K; ++k) s[k] = lanes_sum(s[k], q.P);
        if (lane == 0) {
#pragma unroll
            for (int k = 0; k < K; ++k) stat[k * q.Gs + gg] = s[k];
        }
    }
    team_sync(q.wave);
}

// Calls f(NV) with the plan's vectors a thread as a compile-time constant, up to
// `most` of them.
template <int MOST, typename F>
hipError_t with_nv(int nv, F f)
{
    switch (nv) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 3:
        if constexpr (MOST >= 3) return f(std::integral_constant<int, 3>());
        return hipErrorInvalidValue;
    case 4:
        if constexpr (MOST >= 4) return f(std::integral_constant<int, 4>());
        return hipErrorInvalidValue;
    case 8:
        if constexpr (MOST >= 8) return f(std::integral_constant<int, 8>());
        return hipErrorInvalidValue;
    case 16:
        if constexpr (MOST >= 16) return f(std::integral_constant<int, 16>());
        return hipErrorInvalidValue;
    case 32:
        if constexpr (MOST >= 32) return f(std::integral_constant<int, 32>());
        return hipErrorInvalidValue;
    default: return hipErrorInvalidValue;
    }
}

// Calls f(PAST) with whether the output goes past the cache, where a vector is long
// enough for that.
template <bool CAN, typename F>
hipError_t with_past(bool past, F f)
{
    if constexpr (CAN)
        if (past) return f(std::true_type());
    return f(std::false_type());
}

// Calls f(N) with the plan's vector length; 8 elements only in bf16.
template <typename T, typename F>
hipError_t with_n(int n, F f)
{
    switch (n) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 4: return f(std::integral_constant<int, 4>());
    case 8:
        if constexpr (sizeof(T) == 2) return f(std::integral_constant<int, 8>());
        return hipErrorInvalidValue;
    default: return hipErrorInvalidValue;
    }
}

}  // namespace gc
