// gc_embed.h -- the geometry of an embedding call, passed by value to its kernels.
#pragma once

#include "../../include/gc.h"
#include "gc_common.h"

namespace gc {

// Vectors of N elements that a row of D >= 1 takes; D may be the largest int.
template <int N>
__host__ __device__ __forceinline__ int vectors_of(int D) { return (D - 1) / N + 1; }

struct EmbedGeom {
    uint32_t n;        // tokens: rows * tokens of a row, below 2^31
    int V, D;
    int itype;         // GC_I32, GC_I64 or GC_U8
    int64_t ld;        // elements between rows of out / dout
    int64_t ld_tok;    // tokens between rows of tok
    FastDiv fd_T;      // tokens of a row

    // value of token k (row k / T, place k % T)
    __device__ __forceinline__ int64_t token(const void *tok, uint32_t k) const
    {
        uint32_t r, t;
        fdivmod(k, fd_T, r, t);
        const int64_t at = int64_t(r) * ld_tok + t;
        if (itype == GC_I32) return static_cast<const int32_t *>(tok)[at];
        if (itype == GC_I64) return static_cast<const int64_t *>(tok)[at];
        return static_cast<const uint8_t *>(tok)[at];
    }
    // offset of token k's D elements in out / dout
    __device__ __forceinline__ int64_t row(uint32_t k) const
    {
        uint32_t r, t;
        fdivmod(k, fd_T, r, t);
        return int64_t(r) * ld + int64_t(t) * D;
    }
};

}  // namespace gc
