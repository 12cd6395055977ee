// gc_kernels.h -- launchers of the gfx950 kernels, called by the C ABI layer.
#pragma once

#include "../../include/gc.h"
#include "gc_common.h"

namespace gc {

// Shape-generic implicit GEMM (igemm_generic.hip).
template <typename T>
hipError_t launch_fwd_generic(const Geom &g, const void *x, const void *w, const void *bias,
                              void *y, int relu, hipStream_t s);
template <typename T>
hipError_t launch_dgrad_generic(const Geom &g, const void *dy, const void *w, const void *ym,
                                void *dx, int relu, hipStream_t s);
template <typename T>
hipError_t launch_wgrad_generic(const Geom &g, const void *x, const void *dy, const void *ym,
                                float *part, int splits, int relu, hipStream_t s);
int wgrad_generic_splits(const Geom &g);

// Image-group kernels on fp32 MFMA for shapes the kernels below do not plan
// (dgrad_ig_f32.hip, wgrad_ig_f32.hip).  plan_* returns false when a shape
// does not fit them.
struct DgradIgPlan;
struct WgradIgPlan;
struct DgradBfPlan;
struct WgradBfPlan;
struct WgradRfPlan;
struct BwdFusedBfPlan;
struct BwdFusedF32Plan;
// d_input and wgrad run on fp32 MFMA for both storage types (T = float or
// bf16_t; bf16 is widened exactly while staging).
bool plan_dgrad_ig_f32(const Geom &g, DgradIgPlan &p);
template <typename T>
hipError_t launch_dgrad_ig(const Geom &g, const DgradIgPlan &p, const void *dy, const void *w,
                           const void *ym, void *dx, int relu, hipStream_t s);
bool plan_wgrad_ig_f32(const Geom &g, WgradIgPlan &p);
template <typename T>
hipError_t launch_wgrad_ig(const Geom &g, const WgradIgPlan &p, const void *x, const void *dy,
                           const void *ym, float *part, int relu, hipStream_t s);

// Forward kernels with loader and MFMA waves.
struct FwdWsPlan;
// packs w into the B-fragment order of the bf16 forward for `nblocks`
// 16-channel blocks (fwd_pack.hip)
hipError_t launch_pack_w_fwd_bf16(const Geom &g, int NCG, int TS, int nblocks, const void *w,
                                  void *wf, size_t ws_bytes, hipStream_t s);
// bf16 forward with loader and MFMA waves; plan_* returns false when a shape
// does not fit it
bool plan_fwd_ws_bf16(const Geom &g, FwdWsPlan &p);
hipError_t launch_fwd_ws_bf16(const Geom &g, const FwdWsPlan &p, const void *x, const void *w,
                              const void *bias, void *y, void *ws, int relu, hipStream_t s);
// Bias gradient db[oc] = sum over (b, oh, ow) of dz (bias_grad.hip): fp32
// partials per image chunk in `part`, then the fixed-order reduction.
size_t bias_grad_ws_bytes(const Geom &g);
template <typename T>
hipError_t launch_bias_grad(const Geom &g, const void *dy, const void *ym, void *db, float *part,
                            int relu, hipStream_t s);
// packs w into the B-fragment order of the fp32 forward's MFMA steps (see
// FwdF32Steps) for `nblocks` 16-channel blocks (fwd_pack.hip)
hipError_t launch_pack_w_fwd_f32(const Geom &g, int NCG, int CPP, int TS, int lo, int nblocks,
                                 const void *w, void *wf, size_t ws_bytes, hipStream_t s);
// fp32 forward with loader and MFMA waves
bool plan_fwd_ws_f32(const Geom &g, FwdWsPlan &p);
hipError_t launch_fwd_ws_f32(const Geom &g, const FwdWsPlan &p, const void *x, const void *w,
                             const void *bias, void *y, void *ws, int relu, hipStream_t s);
// LDS pitch of the forwards' channels-innermost x tile (fwd_pack.hip)
void pick_lds_pitch(const Geom &g, int G, int MB, int TS, int &WP_out, int &IS_out);
bool plan_dgrad_ig_bf16(const Geom &g, DgradBfPlan &p);
// fp32 d_input on fp32 MFMA, weights read in place (dgrad_rf_f32.hip); the
// plan struct is shared with the bf16 kernel, KS holding the 16-channel
// blocks, and needs no workspace.
bool plan_dgrad_rf_f32(const Geom &g, DgradBfPlan &p);
hipError_t launch_dgrad_rf_f32(const Geom &g, const DgradBfPlan &p, const void *dy, const void *w,
                               const void *ym, void *dx, int relu, hipStream_t s);
// fp32 wgrad with image-quad staging: partial tiles then the fixed-order
// reduction into dw (fp32 storage only)
bool plan_wgrad_rf_f32(const Geom &g, WgradRfPlan &p);
// the same with the bias gradient as one more column (x = 1) of the tiles
bool plan_wgrad_rf_f32_bias(const Geom &g, WgradRfPlan &p);
// db (the bias gradient) is written when the plan has the bias column
hipError_t launch_wgrad_rf_f32(const Geom &g, const WgradRfPlan &p, const void *x, const void *dy,
                               const void *ym, void *dw, void *db, void *ws, int relu,
                               hipStream_t s);
// bf16 backward (d_input + wgrad) in three or four launches: pre-passes, both
// main kernels in one grid (or one after the other), reduction.  Same results
// as the separate calls.
bool plan_bwd_fused_bf16(const Geom &g, BwdFusedBfPlan &p);
hipError_t launch_bwd_fused_bf16(const Geom &g, const BwdFusedBfPlan &p, const void *x,
                                 const void *w, const void *dy, const void *ym, void *dx, void *dw,
                                 void *ws, int relu, hipStream_t s);
// fp32 backward in two launches: the d_input and wgrad workgroups in one
// grid, then the reduction.  Same results as the separate calls.
bool plan_bwd_fused_f32(const Geom &g, BwdFusedF32Plan &p);
hipError_t launch_bwd_fused_f32(const Geom &g, const BwdFusedF32Plan &p, const void *x,
                                const void *w, const void *dy, const void *ym, void *dx, void *dw,
                                void *ws, int relu, hipStream_t s);
bool plan_wgrad_ig_bf16(const Geom &g, WgradBfPlan &p);
// the same with the bias gradient as one more column (x = 1) of the tiles
bool plan_wgrad_ig_bf16_bias(const Geom &g, WgradBfPlan &p);
// the same for one given tile width (64*JW columns)
bool plan_wgrad_bf16_tiles(const Geom &g, int JW, WgradBfPlan &p, int bias = 0);
// dz regrouping, the partial-tile kernel and the fixed-order reduction into dw
hipError_t launch_wgrad_ig_bf16(const Geom &g, const WgradBfPlan &p, const void *x, const void *dy,
                                const void *ym, void *dw, void *db, void *ws, int relu,
                                hipStream_t s);
hipError_t launch_dgrad_ig_bf16(const Geom &g, const DgradBfPlan &p, const void *dy, const void *w,
                                const void *ym, void *dx, void *ws, int relu, hipStream_t s);

// Fixed-order sum of split partials, then the store in the output type
// (wgrad_reduce.hip).
template <typename T>
hipError_t launch_wgrad_reduce(const float *part, void *dw, int splits, int n, hipStream_t s);
// The same over partial rows of NP columns: columns 0..N-1 of row oc go to
// dw[oc][...], column N to db[oc], the rest (padding) nowhere.
template <typename T>
hipError_t launch_wgrad_reduce_bias(const float *part, void *dw, void *db, int splits, int OC, int N,
                                    int NP, hipStream_t s);

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
