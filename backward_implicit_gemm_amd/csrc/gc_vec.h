// gc_vec.h -- pieces shared by the memory-bound training-step kernels
// (embedding, group norm, gradient clipping): packed vectors of storage
// elements at any element alignment, and reductions over lanes and
// workgroups in a fixed order.
#pragma once

#include "gc_common.h"

namespace gc {

// N consecutive elements as they lie in memory.  Bf16 stays packed two to a
// register until an element is asked for, so a vector held across a reduction
// costs its bytes.  Copies go through memcpy from element-aligned addresses:
// the compiler emits one wide load or store (the HSA runtime runs gfx9 parts in
// unaligned-access mode).
template <typename T, int N> struct Vec;

template <int N> struct Vec<float, N> {
    float w[N];
    __device__ __forceinline__ float get(int j) const { return w[j]; }
    __device__ __forceinline__ void put(const float (&v)[N])
    {
#pragma unroll
        for (int j = 0; j < N; ++j) w[j] = v[j];
    }
};

template <int N> struct Vec<bf16_t, N> {
    static_assert(N % 2 == 0 || N == 1, "pairs or a single element");
    uint32_t w[(N + 1) / 2];
    __device__ __forceinline__ float get(int j) const
    {
        return __uint_as_float(j % 2 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
    }
    // each value rounded once, to nearest even
    __device__ __forceinline__ void put(const float (&v)[N])
    {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        if (N == 1) {
            w[0] = from_f32<bf16_t>(v[0]);
        } else {
#pragma unroll
            for (int j = 0; j + 1 < N; j += 2) {
                const bf16x2 h = {(__bf16)v[j], (__bf16)v[j + 1]};
                w[j / 2] = __builtin_bit_cast(uint32_t, h);
            }
        }
    }
};

template <typename T, int N>
__device__ __forceinline__ Vec<T, N> load_vec(const T *p)
{
    Vec<T, N> v;
    if (sizeof(T) * N < 4) v.w[0] = 0;
    __builtin_memcpy(v.w, p, sizeof(T) * N);
    return v;
}

template <typename T, int N>
__device__ __forceinline__ void store_vec(T *p, const Vec<T, N> &v)
{
    __builtin_memcpy(p, v.w, sizeof(T) * N);
}

// A store past the cache (PAST), for calls that move kStreamBytes and more: as dirty
// lines their outputs push out what the call still reads and are written back in the way
// of later calls.  The call alone gains: clipping 512 MB of values 122 us past the cache and
// 144 with plain stores, an embedding of 98 MB 16.7 and 19.5.  A reader that follows at once
// pays for it where the 256 MB cache would still have held the output, the two together
// taking, past and plain: norm forward of 32,768 x 128 x 3 x 4 bf16 and a convolution 99.9 and
// 90.5 us, that embedding and an addition 52.8 and 51.7, clipping of 128 MB and the update 65.6
// and 63.9; of 512 MB 271 and 286.  Smaller outputs stay cached for their reader.  A
// compile-time choice: of two stores at the ends of a branch the compiler makes one plain one.
constexpr size_t kStreamBytes = size_t(64) << 20;

template <bool PAST, typename T, int N>
__device__ __forceinline__ void put_vec(T *p, const Vec<T, N> &v)
{
    if constexpr (PAST && sizeof(T) * N >= 8) {
        typedef uint32_t words __attribute__((ext_vector_type(sizeof(T) * N / 4), aligned(sizeof(T))));
        words w;
        __builtin_memcpy(&w, v.w, sizeof(w));
        __builtin_nontemporal_store(w, reinterpret_cast<words *>(p));
    } else {
        store_vec<T, N>(p, v);
    }
}

// elements of a 16-byte vector
template <typename T> constexpr int kVec = 16 / int(sizeof(T));

// Sum over the aligned group of `width` lanes (a power of two, at most 64)
// the lane lies in; every lane gets the same value.
template <typename V>
__device__ __forceinline__ V lanes_sum(V v, int width)
{
    for (int m = width >> 1; m > 0; m >>= 1) v += __shfl_xor(v, m, 64);
    return v;
}

// Sum over a workgroup of up to 16 waves (blockDim.x a multiple of 64); every
// thread gets the same value.  `red` holds 16 values of LDS; the barriers
// make it free for the next call.
template <typename V>
__device__ __forceinline__ V block_sum(V v, V *red)
{
    v = lanes_sum(v, 64);
    if (blockDim.x <= 64) return v;
    const int nw = blockDim.x >> 6;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    V s = red[0];
    for (int i = 1; i < nw; ++i) s += red[i];
    return s;
}

}  // namespace gc
