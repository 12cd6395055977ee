// gc_train.h -- launchers and plans of the operators around the convolutions, called by
// their C ABI layer (gc_train_api.hip).
#pragma once

#include "../../include/gc.h"
#include "gc_common.h"

namespace gc {

// The global gradient norm and clipping (grad_clip.hip).  A launch takes
// kClipTensors tensors in its arguments.
constexpr int kClipTensors = 96;
size_t grad_clip_ws_bytes(int count);
hipError_t launch_grad_clip(const gc_tensor *list, int count, float max_norm, float prescale, float eps,
                            bool scale, float *norm, void *ws, hipStream_t s);

// Embedding lookup (embed_fwd.hip) and its gradient by sorted tokens
// (embed_grad_sort.hip).
struct EmbedGeom;
template <typename T>
hipError_t launch_embed_fwd(const EmbedGeom &g, const void *tok, const void *table, void *out, float scale,
                            hipStream_t s);
size_t embed_grad_sort_ws_bytes(const EmbedGeom &g);
template <typename T>
hipError_t launch_embed_grad_sort(const EmbedGeom &g, const void *tok, const void *dout, void *dtable, float scale,
                                  void *ws, hipStream_t s);

// The gradient as a one-hot matrix product, for small vocabularies
// (embed_grad_onehot.hip); needs D >= 2 and at least one token.
int embed_grad_onehot_rows(int V);   // table rows, padded to its blocks
size_t embed_grad_onehot_ws_bytes(const EmbedGeom &g);
template <typename T>
hipError_t launch_embed_grad_onehot(const EmbedGeom &g, const void *tok, const void *dout, void *dtable, float scale,
                                    void *ws, hipStream_t s);

// Group norm with an activation.  The split kernels (norm_split.hip) take every
// shape; plan_norm_split returns false past the largest grid.
struct NormGeom;
// A launch has to stay below 2^32 threads.
inline bool launchable(int64_t grid, int threads) { return grid * threads < int64_t(1) << 32; }
struct NormSplitPlan {
    int N;                     // elements of a thread's vector
    int cols, blocks, slots;   // channels last: vectors of a workgroup's row, column blocks, rows at a time
    int chunks, len;           // pieces an image's positions are cut into, and their length
    int past_fwd, past_bwd;    // the output goes past the cache
    int64_t grid;
    size_t part_bytes_fwd, part_bytes_bwd, ws_fwd, ws_bwd;
};
bool plan_norm_split(const NormGeom &g, int dtype, NormSplitPlan &q);
template <typename T>
hipError_t launch_norm_split_fwd(const NormGeom &g, const NormSplitPlan &q, const void *x, const void *gamma,
                                 const void *beta, void *y, float *mean, float *rstd, void *ws, hipStream_t s);
template <typename T>
hipError_t launch_norm_split_bwd(const NormGeom &g, const NormSplitPlan &q, const void *x, const void *gamma,
                                 const void *beta, const void *dy, const float *mean, const float *rstd, void *dx,
                                 void *dgamma, void *dbeta, void *ws, hipStream_t s);
// Groups that stay in registers (norm_res_nchw.hip, norm_res_nhwc.hip; planned in
// norm_plan.hip): plan_norm_res returns false where a group is too large.
struct NormResPlan {
    int N, NV;             // elements of a vector, vectors a thread holds
    int L, teams, threads; // threads of a team, teams of a workgroup, threads of a workgroup
    int small;             // the small-group kernels (norm_res_small.hip)
    int join;              // their backward writes one row of partials a workgroup
    int two;               // NCHW: vectors may straddle two channels
    int wave;              // channels last: a team is one wave
    int mix;               // channels last: 0 vectors mix groups, 1 lie in one, 2 do and the last of a row is moved back
    int past;              // the output goes past the cache
    int P;                 // lanes that add up one group (channels last) or channel (NCHW)
    int slots, CW, slabs, Gs;   // channels last: rows at a time; channels, number and groups of a slab
    int width, team_lds;   // channels last: LDS entries of a row, LDS words of a team
    int images;            // backward: image slots walking the batch
    int rows;              // backward: rows of per-channel partials
    FastDiv fd_cols, fd_Eg;
    int64_t grid;
    size_t lds_bytes, ws_bytes;
};
bool plan_norm_res(const NormGeom &g, int dtype, bool bwd, NormResPlan &q);
template <typename T>
hipError_t launch_norm_res_nchw_fwd(const NormGeom &g, const NormResPlan &q, const void *x, const void *gamma,
                                    const void *beta, void *y, float *mean, float *rstd, hipStream_t s);
template <typename T>
hipError_t launch_norm_res_nchw_bwd(const NormGeom &g, const NormResPlan &q, const void *x, const void *gamma,
                                    const void *beta, const void *dy, const float *mean, const float *rstd, void *dx,
                                    float *part, hipStream_t s);
template <typename T>
hipError_t launch_norm_res_nhwc_fwd(const NormGeom &g, const NormResPlan &q, const void *x, const void *gamma,
                                    const void *beta, void *y, float *mean, float *rstd, hipStream_t s);
template <typename T>
hipError_t launch_norm_res_nhwc_bwd(const NormGeom &g, const NormResPlan &q, const void *x, const void *gamma,
                                    const void *beta, const void *dy, const float *mean, const float *rstd, void *dx,
                                    float *part, hipStream_t s);
template <typename T>
hipError_t launch_norm_res_small_fwd(const NormGeom &g, const NormResPlan &q, const void *x, const void *gamma,
                                     const void *beta, void *y, float *mean, float *rstd, hipStream_t s);
template <typename T>
hipError_t launch_norm_res_small_bwd(const NormGeom &g, const NormResPlan &q, const void *x, const void *gamma,
                                     const void *beta, const void *dy, const float *mean, const float *rstd, void *dx,
                                     float *part, hipStream_t s);
// dgamma and dbeta from `rows` rows of per-channel pairs (dbeta's, dgamma's)
template <typename T>
hipError_t launch_norm_params(const NormGeom &g, int64_t rows, const float *part, void *dgamma, void *dbeta,
                              hipStream_t s);

}  // namespace gc
