// gc_core.h -- geometry, plans and launchers of the recurrent core's operators (layer norm
// of a residual stream, the gated recurrence, distillation), called by their C ABI layer
// (gc_core_api.hip).
#pragma once

#include "../../include/gc.h"
#include "gc_train.h"
#include "gc_vec.h"

namespace gc {

constexpr int kCUs = 256;   // MI355X

// Vectors of N elements that a row of D >= 1 takes; D may be the largest int.
__host__ __device__ __forceinline__ int vectors(int D, int N) { return (D - 1) / N + 1; }

// ------------------------------------------------------------------ layer norm --
struct RowsGeom {
    int64_t rows;
    int D;
    float eps;
    int pf32;      // gamma, beta and their gradients in fp32 (else the storage type)
    int64_t ld_x, ld_res, ld_total, ld_y;
};
struct RowsPlan {
    int N, NV;      // elements of a vector, vectors a thread holds
    int L;          // threads of a row's team, a power of two
    int threads;    // of a workgroup
    int loop;       // the row does not fit a workgroup's registers
    int past;       // the output goes past the cache
    int64_t grid;
    int64_t parts;  // backward: rows of partial sums
    size_t ws_bytes, lds_bytes;
};
void plan_rows(const RowsGeom &g, int dtype, bool bwd, bool more, RowsPlan &q);
template <typename T>
hipError_t launch_rows_fwd(const RowsGeom &g, const RowsPlan &q, const void *x, const void *res, const void *gamma,
                           const void *beta, void *y, void *total, float *mean, float *rstd, hipStream_t s);
template <typename T>
hipError_t launch_rows_bwd(const RowsGeom &g, const RowsPlan &q, const void *x, const void *gamma, const void *dy,
                           const void *dtotal, const float *mean, const float *rstd, void *dx, void *dgamma,
                           void *dbeta, float *part, hipStream_t s);

// ------------------------------------------------------------------ recurrence --
struct ScanGeom {
    int B, T, D;
    int coupled;
    gc_strides gate, value, out, dgate, dvalue, reset;
};
struct ScanPlan {
    int N;              // channels of a thread
    int nv;             // threads of a step's channels
    int64_t lanes;      // of all sequences
    int past;           // the outputs go past the cache
    int far;            // lanes of a wave may be 4 GiB apart and more
    int chunks, len;    // pieces the steps are cut into, and their length (a multiple of the block)
    size_t part_bytes, ws_bytes;
    FastDiv fd_nv, fd_blocks;
};
bool plan_scan(const ScanGeom &g, int dtype, bool bwd, bool ragged, ScanPlan &q);
template <typename T>
hipError_t launch_scan_fwd(const ScanGeom &g, const ScanPlan &q, const void *gate, const void *value, const float *h0,
                           const uint8_t *reset, const int32_t *lengths, void *out, float *last, float *states,
                           void *ws, hipStream_t s);
template <typename T>
hipError_t launch_scan_bwd(const ScanGeom &g, const ScanPlan &q, const void *gate, const void *value,
                           const float *states, const uint8_t *reset, const int32_t *lengths, const void *dout,
                           const float *dlast, void *dgate, void *dvalue, float *dh0, void *ws, hipStream_t s);

// ---------------------------------------------------------------- distillation --
struct DistillGeom {
    int64_t rows;
    int V, K;
    int i64, t32;       // index type, teacher type
    float temperature;
    int64_t ld, ld_grad, ld_index, ld_teacher;
};
struct DistillPlan {
    int N, NV;      // elements of a vector; vectors a thread holds (0: the row is walked)
    int L;          // threads of a row's team, a power of two
    int threads;    // of a workgroup
    int lists;      // of a row's many entries, a power of two
    int past;       // the output goes past the cache
    int64_t grid;
    size_t lds_bytes;
};
void plan_distill(const DistillGeom &g, int dtype, int op, DistillPlan &q);
template <typename T>
hipError_t launch_distill(const DistillGeom &g, const DistillPlan &q, int op, const void *logits, const void *index,
                          const void *teacher, float *peak, float *mass, const float *dloss, float *loss, void *dlogits,
                          hipStream_t s);

}  // namespace gc
