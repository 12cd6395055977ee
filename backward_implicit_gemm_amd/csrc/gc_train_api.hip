// gc_train_api.hip -- the C ABI of the operators around the convolutions
// (embedding, group norm, gradient clipping), declared in include/gc.h:
// argument checks, workspace sizes and the choice of kernels.  All checks
// come before the first HIP call.
#include <limits.h>
#include <math.h>
#include <stdio.h>

#include "gc_embed.h"
#include "gc_norm.h"
#include "gc_train.h"

using namespace gc;

namespace {

bool valid_dtype(int dtype) { return dtype == GC_F32 || dtype == GC_BF16; }

bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool aligned_to(const void *p, int dtype) { return aligned(p, dtype == GC_F32 ? 4 : 2); }

int hip_status(hipError_t e) { return e == hipSuccess ? GC_OK : GC_ERR_HIP; }

int check_workspace(const void *ws, size_t have, size_t need)
{
    if (!need) return GC_OK;
    if (!ws || have < need || !aligned(ws, 256)) return GC_ERR_WORKSPACE;
    return GC_OK;
}

// ---------------------------------------------------------------- embedding --
int check_embed(const gc_embed_desc *d, EmbedGeom *g)
{
    if (!d || d->rows < 0 || d->tokens < 0 || d->V < 1 || d->D < 1) return GC_ERR_INVALID_ARG;
    if (d->itype != GC_I32 && d->itype != GC_I64 && d->itype != GC_U8) return GC_ERR_INVALID_ARG;
    const __int128 n = (__int128)d->rows * d->tokens;
    if (n > INT_MAX || (__int128)d->tokens * d->D > INT_MAX) return GC_ERR_INVALID_ARG;
    if (d->ld < (int64_t)d->tokens * d->D || d->ld_tok < d->tokens) return GC_ERR_INVALID_ARG;
    const __int128 most = (__int128)1 << 60;   // byte offsets stay within 64 bits
    if ((__int128)d->rows * d->ld > most || (__int128)d->rows * d->ld_tok > most) return GC_ERR_INVALID_ARG;
    if (g) {
        g->n = uint32_t(n);
        g->V = d->V;
        g->D = d->D;
        g->itype = d->itype;
        g->ld = d->ld;
        g->ld_tok = d->ld_tok;
        g->fd_T = make_fastdiv(d->tokens > 0 ? uint32_t(d->tokens) : 1u);
    }
    return GC_OK;
}

// The gradient's kernels.  The one-hot product costs rows * slabs (of 32 columns) *
// tokens, sorting hardly depends on the number of rows.  Measured (us, one-hot and
// sort, bf16): 20,000 tokens, 32 columns, 1024 rows 36 and 65, 4096 rows 57 and 52;
// 256 columns, 512 rows 55 and 79, 1024 rows 79 and 63; 400,000 tokens, 32 columns,
// 1024 rows 79 and 147, 4096 rows 224 and 156; 500 tokens, 256 columns, 512 rows 21 and
// 27, 1024 rows 32 and 24.  In fp32 the matrix cores take longer: 400,000 tokens, 32
// columns, 256 rows 102 and 222, 1024 rows 284 and 196; 20,000 tokens, 256 columns, 256
// rows 66 and 74, 512 rows 98 and 64.
bool embed_onehot(const EmbedGeom &g, int dtype)
{
    if (g.D < 2 || g.n == 0 || g.V > 4096) return false;
    const int64_t cells = int64_t(embed_grad_onehot_rows(g.V)) * ((int64_t(g.D) + 31) / 32);
    return dtype == GC_BF16 ? cells <= 4096 && cells * g.n <= 800000000
                            : cells <= 2048 && cells * g.n <= 150000000;
}

size_t embed_grad_ws_bytes(const EmbedGeom &g, int dtype)
{
    return embed_onehot(g, dtype) ? embed_grad_onehot_ws_bytes(g) : embed_grad_sort_ws_bytes(g);
}

template <typename T>
hipError_t embed_grad(const EmbedGeom &g, const void *tok, const void *dout, void *dtable, float scale, void *ws,
                      hipStream_t s)
{
    return embed_onehot(g, sizeof(T) == 4 ? GC_F32 : GC_BF16) ? launch_embed_grad_onehot<T>(g, tok, dout, dtable, scale, ws, s)
                           : launch_embed_grad_sort<T>(g, tok, dout, dtable, scale, ws, s);
}

uintptr_t token_size(int itype) { return itype == GC_I32 ? 4 : itype == GC_I64 ? 8 : 1; }

// ---------------------------------------------------------------- group norm --
constexpr int kNormMost = 1 << 30, kNormChannels = 1 << 23;

int check_norm(const gc_norm_desc *d, NormGeom *g)
{
    if (!d || d->B < 1 || d->C < 1 || d->H < 1 || d->W < 1 || d->groups < 1) return GC_ERR_INVALID_ARG;
    if (d->C % d->groups) return GC_ERR_INVALID_ARG;
    if (d->layout != GC_NCHW && d->layout != GC_NHWC) return GC_ERR_INVALID_ARG;
    if (d->act < GC_ACT_NONE || d->act > GC_ACT_GELU) return GC_ERR_INVALID_ARG;
    if (!(d->eps >= 0.f) || isinf(d->eps)) return GC_ERR_INVALID_ARG;
    const int64_t hw = (int64_t)d->H * d->W;
    // so that the kernels' counters, a stride past the end, stay within 31 bits and no
    // launch over the channels reaches 2^32 threads
    if (d->B > kNormMost || d->C > kNormChannels || hw > kNormMost || hw * d->C > kNormMost) return GC_ERR_INVALID_ARG;
    if (g) {
        g->B = d->B;
        g->C = d->C;
        g->HW = int(hw);
        g->G = d->groups;
        g->Cg = d->C / d->groups;
        // with one position or one channel both layouts are the same memory
        g->nhwc = d->layout == GC_NHWC && hw > 1 && d->C > 1;
        g->act = d->act;
        g->eps = d->eps;
        g->img = hw * d->C;
        g->fd_HW = make_fastdiv(uint32_t(hw));
        g->fd_Cg = make_fastdiv(uint32_t(g->Cg));
    }
    return GC_OK;
}

int check_norm_types(int dtype, int param_dtype, NormGeom &g)
{
    if (!valid_dtype(dtype) || !valid_dtype(param_dtype)) return GC_ERR_INVALID_ARG;
    if (param_dtype != GC_F32 && param_dtype != dtype) return GC_ERR_INVALID_ARG;
    g.pf32 = param_dtype == GC_F32;
    return GC_OK;
}

// The kernels of a group norm: resident where a group fits, else split.
enum class NormKind { Resident, Split, None };
struct NormSel {
    NormKind k;
    NormResPlan r;
    NormSplitPlan q;
    size_t ws_bytes;
};
NormSel select_norm(const NormGeom &g, int dtype, bool bwd)
{
    NormSel s{};
    if (plan_norm_res(g, dtype, bwd, s.r)) {
        s.k = NormKind::Resident;
        s.ws_bytes = s.r.ws_bytes;
    } else if (plan_norm_split(g, dtype, s.q)) {
        s.k = NormKind::Split;
        s.ws_bytes = bwd ? s.q.ws_bwd : s.q.ws_fwd;
    } else {
        s.k = NormKind::None;
    }
    return s;
}

template <typename T>
hipError_t norm_fwd(const NormGeom &g, const NormSel &s, const void *x, const void *gamma, const void *beta, void *y,
                    float *mean, float *rstd, void *ws, hipStream_t st)
{
    if (s.k == NormKind::Split) return launch_norm_split_fwd<T>(g, s.q, x, gamma, beta, y, mean, rstd, ws, st);
    if (s.r.small) return launch_norm_res_small_fwd<T>(g, s.r, x, gamma, beta, y, mean, rstd, st);
    return g.nhwc ? launch_norm_res_nhwc_fwd<T>(g, s.r, x, gamma, beta, y, mean, rstd, st)
                  : launch_norm_res_nchw_fwd<T>(g, s.r, x, gamma, beta, y, mean, rstd, st);
}

template <typename T>
hipError_t norm_bwd(const NormGeom &g, const NormSel &s, const void *x, const void *gamma, const void *beta,
                    const void *dy, const float *mean, const float *rstd, void *dx, void *dgamma, void *dbeta,
                    void *ws, hipStream_t st)
{
    if (s.k == NormKind::Split)
        return launch_norm_split_bwd<T>(g, s.q, x, gamma, beta, dy, mean, rstd, dx, dgamma, dbeta, ws, st);
    float *part = dgamma || dbeta ? static_cast<float *>(ws) : nullptr;
    const hipError_t e = s.r.small ? launch_norm_res_small_bwd<T>(g, s.r, x, gamma, beta, dy, mean, rstd, dx, part, st)
                         : g.nhwc  ? launch_norm_res_nhwc_bwd<T>(g, s.r, x, gamma, beta, dy, mean, rstd, dx, part, st)
                                   : launch_norm_res_nchw_bwd<T>(g, s.r, x, gamma, beta, dy, mean, rstd, dx, part, st);
    return e == hipSuccess && part ? launch_norm_params<T>(g, s.r.rows, part, dgamma, dbeta, st) : e;
}

int check_list(const gc_tensor *list, int count, bool dst)
{
    if (count < 0 || (count > 0 && !list)) return GC_ERR_INVALID_ARG;
    __int128 total = 0;
    for (int i = 0; i < count; ++i) {
        const gc_tensor &t = list[i];
        if (t.n < 0 || !valid_dtype(t.dtype)) return GC_ERR_INVALID_ARG;
        if (t.n && (!t.src || !aligned_to(t.src, t.dtype))) return GC_ERR_INVALID_ARG;
        if (dst && t.n && (!t.dst || !aligned_to(t.dst, t.dtype))) return GC_ERR_INVALID_ARG;
        total += t.n;
    }
    // the chunk numbers of a launch stay within 31 bits
    return total <= ((__int128)1 << 42) ? GC_OK : GC_ERR_INVALID_ARG;
}

}  // namespace

extern "C" {

int gc_embed_fwd(const void *tokens, const void *table, void *out, const gc_embed_desc *d, float scale, int dtype,
                 void *stream)
{
    EmbedGeom g;
    const int st = check_embed(d, &g);
    if (st != GC_OK) return st;
    if (!valid_dtype(dtype) || !table || !aligned_to(table, dtype) || !isfinite(scale)) return GC_ERR_INVALID_ARG;
    if (g.n == 0) return GC_OK;
    if (!tokens || !out || !aligned(tokens, token_size(d->itype)) || !aligned_to(out, dtype))
        return GC_ERR_INVALID_ARG;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return hip_status(dtype == GC_F32 ? launch_embed_fwd<float>(g, tokens, table, out, scale, s)
                                      : launch_embed_fwd<bf16_t>(g, tokens, table, out, scale, s));
}

size_t gc_embed_workspace_bytes(const gc_embed_desc *d, int dtype)
{
    EmbedGeom g;
    if (check_embed(d, &g) != GC_OK || !valid_dtype(dtype)) return 0;
    return embed_grad_ws_bytes(g, dtype);
}

int gc_embed_bwd(const void *tokens, const void *dout, void *dtable, void *workspace, size_t ws_bytes,
                 const gc_embed_desc *d, float scale, int dtype, void *stream)
{
    EmbedGeom g;
    int st = check_embed(d, &g);
    if (st != GC_OK) return st;
    if (!valid_dtype(dtype) || !dtable || !aligned_to(dtable, dtype) || !isfinite(scale)) return GC_ERR_INVALID_ARG;
    if (g.n && (!tokens || !dout || !aligned(tokens, token_size(d->itype)) || !aligned_to(dout, dtype)))
        return GC_ERR_INVALID_ARG;
    st = check_workspace(workspace, ws_bytes, embed_grad_ws_bytes(g, dtype));
    if (st != GC_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return hip_status(dtype == GC_F32 ? embed_grad<float>(g, tokens, dout, dtable, scale, workspace, s)
                                      : embed_grad<bf16_t>(g, tokens, dout, dtable, scale, workspace, s));
}

size_t gc_group_norm_workspace_bytes(int op, const gc_norm_desc *d, int dtype)
{
    NormGeom g;
    if (check_norm(d, &g) != GC_OK || !valid_dtype(dtype) || (op != GC_OP_FWD && op != GC_OP_BWD)) return 0;
    return select_norm(g, dtype, op == GC_OP_BWD).ws_bytes;
}

int gc_group_norm_fwd(const void *x, const void *gamma, const void *beta, void *y, float *mean, float *rstd,
                      void *workspace, size_t ws_bytes, const gc_norm_desc *d, int dtype, int param_dtype,
                      void *stream)
{
    NormGeom g;
    int st = check_norm(d, &g);
    if (st == GC_OK) st = check_norm_types(dtype, param_dtype, g);
    if (st != GC_OK) return st;
    if (!x || !y || !aligned_to(x, dtype) || !aligned_to(y, dtype)) return GC_ERR_INVALID_ARG;
    if ((gamma && !aligned_to(gamma, param_dtype)) || (beta && !aligned_to(beta, param_dtype)))
        return GC_ERR_INVALID_ARG;
    if (!aligned(mean, 4) || !aligned(rstd, 4)) return GC_ERR_INVALID_ARG;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const NormSel sel = select_norm(g, dtype, false);
    if (sel.k == NormKind::None) return GC_ERR_UNSUPPORTED;
    st = check_workspace(workspace, ws_bytes, sel.ws_bytes);
    if (st != GC_OK) return st;
    return hip_status(dtype == GC_F32 ? norm_fwd<float>(g, sel, x, gamma, beta, y, mean, rstd, workspace, s)
                                      : norm_fwd<bf16_t>(g, sel, x, gamma, beta, y, mean, rstd, workspace, s));
}

int gc_group_norm_bwd(const void *x, const void *gamma, const void *beta, const void *dy, const float *mean,
                      const float *rstd, void *dx, void *dgamma, void *dbeta, void *workspace, size_t ws_bytes,
                      const gc_norm_desc *d, int dtype, int param_dtype, void *stream)
{
    NormGeom g;
    int st = check_norm(d, &g);
    if (st == GC_OK) st = check_norm_types(dtype, param_dtype, g);
    if (st != GC_OK) return st;
    if (!x || !dy || !mean || !rstd || !dx) return GC_ERR_INVALID_ARG;
    if (!aligned_to(x, dtype) || !aligned_to(dy, dtype) || !aligned_to(dx, dtype) || !aligned(mean, 4) ||
        !aligned(rstd, 4))
        return GC_ERR_INVALID_ARG;
    const void *params[] = {gamma, beta, dgamma, dbeta};
    for (const void *p : params)
        if (p && !aligned_to(p, param_dtype)) return GC_ERR_INVALID_ARG;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const NormSel sel = select_norm(g, dtype, true);
    if (sel.k == NormKind::None) return GC_ERR_UNSUPPORTED;
    st = check_workspace(workspace, ws_bytes, sel.ws_bytes);
    if (st != GC_OK) return st;
    return hip_status(dtype == GC_F32 ? norm_bwd<float>(g, sel, x, gamma, beta, dy, mean, rstd, dx, dgamma, dbeta,
                                                        workspace, s)
                                      : norm_bwd<bf16_t>(g, sel, x, gamma, beta, dy, mean, rstd, dx, dgamma, dbeta,
                                                         workspace, s));
}

int gc_group_norm_plan_name(int op, const gc_norm_desc *d, int dtype, char *buf, size_t buf_bytes)
{
    NormGeom g;
    const int st = check_norm(d, &g);
    if (st != GC_OK) return st;
    if (!valid_dtype(dtype) || (op != GC_OP_FWD && op != GC_OP_BWD) || !buf || !buf_bytes) return GC_ERR_INVALID_ARG;
    const bool bwd = op == GC_OP_BWD;
    const NormSel s = select_norm(g, dtype, bwd);
    const char *dir = bwd ? "bwd" : "fwd";
    // past: the output goes past the cache
    if (s.k == NormKind::Split)
        snprintf(buf, buf_bytes, "norm_split_%s<N=%d,NHWC=%d> chunks=%d grid=%lld past=%d", dir, s.q.N, g.nhwc,
                 s.q.chunks, (long long)s.q.grid, bwd ? s.q.past_bwd : s.q.past_fwd);
    else if (s.k == NormKind::None)
        snprintf(buf, buf_bytes, "none");
    else if (s.r.small)
        snprintf(buf, buf_bytes, "res_small_%s<N=%d,NV=%d,LAST=%d> threads=%d teams=%d grid=%lld past=%d", dir, s.r.N,
                 s.r.NV, g.nhwc, s.r.L, s.r.teams, (long long)s.r.grid, s.r.past);
    else if (g.nhwc)
        snprintf(buf, buf_bytes, "res_nhwc_%s<N=%d,NV=%d,MIX=%d> threads=%d teams=%d slab=%d grid=%lld past=%d", dir,
                 s.r.N, s.r.NV, s.r.mix, s.r.L, s.r.teams, s.r.CW, (long long)s.r.grid, s.r.past);
    else
        snprintf(buf, buf_bytes, "res_nchw_%s<N=%d,NV=%d,TWO=%d> threads=%d teams=%d grid=%lld past=%d", dir, s.r.N,
                 s.r.NV, s.r.two, s.r.L, s.r.teams, (long long)s.r.grid, s.r.past);
    return GC_OK;
}

int gc_embed_plan_name(const gc_embed_desc *d, int dtype, char *buf, size_t buf_bytes)
{
    EmbedGeom g;
    const int st = check_embed(d, &g);
    if (st != GC_OK) return st;
    if (!valid_dtype(dtype) || !buf || !buf_bytes) return GC_ERR_INVALID_ARG;
    snprintf(buf, buf_bytes, "%s", embed_onehot(g, dtype) ? "embed_grad_onehot" : "embed_grad_sort");
    return GC_OK;
}

size_t gc_grad_clip_workspace_bytes(int count) { return count < 0 ? 0 : grad_clip_ws_bytes(count); }

int gc_grad_norm(const gc_tensor *list, int count, float prescale, float *norm, void *workspace, size_t ws_bytes,
                 void *stream)
{
    int st = check_list(list, count, false);
    if (st != GC_OK) return st;
    if (!norm || !aligned(norm, 4) || !isfinite(prescale)) return GC_ERR_INVALID_ARG;
    st = check_workspace(workspace, ws_bytes, grad_clip_ws_bytes(count));
    if (st != GC_OK) return st;
    return hip_status(launch_grad_clip(list, count, 0.f, prescale, 0.f, false, norm, workspace,
                                       static_cast<hipStream_t>(stream)));
}

int gc_grad_clip(const gc_tensor *list, int count, float max_norm, float prescale, float eps, float *norm,
                 void *workspace, size_t ws_bytes, void *stream)
{
    int st = check_list(list, count, true);
    if (st != GC_OK) return st;
    if (!norm || !aligned(norm, 4) || !isfinite(prescale) || !isfinite(eps)) return GC_ERR_INVALID_ARG;
    if (!(max_norm >= 0.f) || eps < 0.f) return GC_ERR_INVALID_ARG;
    st = check_workspace(workspace, ws_bytes, grad_clip_ws_bytes(count));
    if (st != GC_OK) return st;
    return hip_status(launch_grad_clip(list, count, max_norm, prescale, eps, true, norm, workspace,
                                       static_cast<hipStream_t>(stream)));
}

}  // extern "C"
