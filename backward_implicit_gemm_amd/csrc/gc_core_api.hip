// gc_core_api.hip -- the C ABI of the recurrent core's operators (layer norm of a residual
// stream, the gated recurrence, distillation), declared in include/gc.h: argument checks,
// workspace sizes and the choice of kernels.  All checks come before the first HIP call.
#include <limits.h>
#include <math.h>
#include <stdio.h>
#include <utility>

#include "gc_core.h"

using namespace gc;

namespace {

bool valid_dtype(int dtype) { return dtype == GC_F32 || dtype == GC_BF16; }
bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
uintptr_t size_of(int dtype) { return dtype == GC_F32 ? 4 : 2; }
// a pointer that has to be there, and one that may be NULL
bool given(const void *p, uintptr_t a) { return p && aligned(p, a); }

int hip_status(hipError_t e) { return e == hipSuccess ? GC_OK : GC_ERR_HIP; }

int check_workspace(const void *ws, size_t have, size_t need)
{
    if (!need) return GC_OK;
    return ws && have >= need && aligned(ws, 256) ? GC_OK : GC_ERR_WORKSPACE;
}

// n steps of distance d stay within 2^60 elements, so byte offsets within 64 bits
bool in_reach(int64_t n, int64_t d) { return (__int128)n * d <= (__int128)1 << 60; }

// ------------------------------------------------------------------ layer norm --
int check_rows(const gc_layer_norm_desc *d, RowsGeom &g)
{
    if (!d || d->rows < 0 || d->rows > INT_MAX || d->D < 1 || d->D > 1 << 23) return GC_ERR_INVALID_ARG;
    if (!(d->eps >= 0.f) || isinf(d->eps)) return GC_ERR_INVALID_ARG;
    for (const int64_t ld : {d->ld_x, d->ld_residual, d->ld_total, d->ld_y})
        if (ld < d->D || !in_reach(d->rows, ld)) return GC_ERR_INVALID_ARG;
    g = RowsGeom{d->rows, d->D, d->eps, 1, d->ld_x, d->ld_residual, d->ld_total, d->ld_y};
    return GC_OK;
}

int check_types(int dtype, int param_dtype, RowsGeom &g)
{
    if (!valid_dtype(dtype) || (param_dtype != GC_F32 && param_dtype != dtype)) return GC_ERR_INVALID_ARG;
    g.pf32 = param_dtype == GC_F32;
    return GC_OK;
}

// ------------------------------------------------------------------ recurrence --
// B sequences of T steps of D elements do not run into each other
bool apart(const gc_strides &s, int B, int T, int D)
{
    if (B < 1 || T < 1) return true;
    std::pair<int64_t, int64_t> inner(s.step, T), outer(s.batch, B);
    if (T == 1) inner = {D, 1};
    if (B == 1) outer = {INT64_MAX, 1};
    if (inner.first > outer.first) std::swap(inner, outer);
    if (inner.first < D) return false;
    return outer.second == 1 || (__int128)inner.first * (inner.second - 1) + D <= outer.first;
}

bool reachable(const gc_strides &s, int B, int T)
{
    return s.batch >= 0 && s.step >= 0 && in_reach(B, s.batch) && in_reach(T, s.step);
}

int check_scan(const gc_recurrence_desc *d, bool bwd, ScanGeom &g)
{
    if (!d || d->B < 0 || d->T < 0 || d->T > 1 << 30 || d->D < 1) return GC_ERR_INVALID_ARG;
    if (d->coupled != 0 && d->coupled != 1) return GC_ERR_INVALID_ARG;
    for (const gc_strides &s : {d->gate, d->value, d->out, d->reset})
        if (!reachable(s, d->B, d->T)) return GC_ERR_INVALID_ARG;
    if (bwd) {
        for (const gc_strides &s : {d->dgate, d->dvalue})
            if (!reachable(s, d->B, d->T) || !apart(s, d->B, d->T, d->D)) return GC_ERR_INVALID_ARG;
    } else if (!apart(d->out, d->B, d->T, d->D)) {
        return GC_ERR_INVALID_ARG;
    }
    g = ScanGeom{d->B, d->T, d->D, d->coupled, d->gate, d->value, d->out, d->dgate, d->dvalue, d->reset};
    return GC_OK;
}

// ---------------------------------------------------------------- distillation --
constexpr int kMostTop = 1024;

int check_distill(const gc_distill_desc *d, DistillGeom &g)
{
    if (!d || d->rows < 0 || d->rows > INT_MAX || d->V < 1 || d->K < 1 || d->K > kMostTop) return GC_ERR_INVALID_ARG;
    if ((d->itype != GC_I32 && d->itype != GC_I64) || !valid_dtype(d->teacher_dtype)) return GC_ERR_INVALID_ARG;
    // its square and the reciprocal stay normal numbers
    if (!(d->temperature >= 1e-18f && d->temperature <= 1e18f)) return GC_ERR_INVALID_ARG;
    if (d->ld < d->V || d->ld_grad < d->V || d->ld_index < d->K || d->ld_teacher < d->K) return GC_ERR_INVALID_ARG;
    for (const int64_t ld : {d->ld, d->ld_grad, d->ld_index, d->ld_teacher})
        if (!in_reach(d->rows, ld)) return GC_ERR_INVALID_ARG;
    g = DistillGeom{d->rows, d->V, d->K, d->itype == GC_I64, d->teacher_dtype == GC_F32, d->temperature,
                    d->ld, d->ld_grad, d->ld_index, d->ld_teacher};
    return GC_OK;
}

bool entries_given(const gc_distill_desc *d, const void *logits, const void *index, const void *teacher, int dtype)
{
    return given(logits, size_of(dtype)) && given(index, d->itype == GC_I64 ? 8 : 4) &&
           given(teacher, size_of(d->teacher_dtype));
}

int distill_call(const DistillGeom &g, int op, const void *logits, const void *index, const void *teacher, float *peak,
                 float *mass, const float *dloss, float *loss, void *dlogits, int dtype, void *stream)
{
    DistillPlan q;
    plan_distill(g, dtype, op, q);
    if (!launchable(q.grid, q.threads)) return GC_ERR_UNSUPPORTED;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return hip_status(dtype == GC_F32
                          ? launch_distill<float>(g, q, op, logits, index, teacher, peak, mass, dloss, loss, dlogits, s)
                          : launch_distill<bf16_t>(g, q, op, logits, index, teacher, peak, mass, dloss, loss, dlogits, s));
}

}  // namespace

extern "C" {

int gc_layer_norm_fwd(const void *x, const void *residual, const void *gamma, const void *beta, void *y, void *total,
                      float *mean, float *rstd, const gc_layer_norm_desc *d, int dtype, int param_dtype, void *stream)
{
    RowsGeom g;
    int st = check_rows(d, g);
    if (st == GC_OK) st = check_types(dtype, param_dtype, g);
    if (st != GC_OK) return st;
    for (const void *p : {gamma, beta})
        if (!aligned(p, size_of(param_dtype))) return GC_ERR_INVALID_ARG;
    if (!aligned(mean, 4) || !aligned(rstd, 4)) return GC_ERR_INVALID_ARG;
    if (g.rows == 0) return GC_OK;
    if (!given(x, size_of(dtype)) || !given(y, size_of(dtype))) return GC_ERR_INVALID_ARG;
    if (!aligned(residual, size_of(dtype)) || !aligned(total, size_of(dtype))) return GC_ERR_INVALID_ARG;
    RowsPlan q;
    plan_rows(g, dtype, false, residual, q);
    hipStream_t s = static_cast<hipStream_t>(stream);
    return hip_status(dtype == GC_F32 ? launch_rows_fwd<float>(g, q, x, residual, gamma, beta, y, total, mean, rstd, s)
                                      : launch_rows_fwd<bf16_t>(g, q, x, residual, gamma, beta, y, total, mean, rstd, s));
}

size_t gc_layer_norm_workspace_bytes(const gc_layer_norm_desc *d, int dtype)
{
    RowsGeom g;
    if (check_rows(d, g) != GC_OK || !valid_dtype(dtype)) return 0;
    RowsPlan q;
    plan_rows(g, dtype, true, true, q);
    return g.rows ? q.ws_bytes : 0;
}

int gc_layer_norm_bwd(const void *x, const void *gamma, const void *dy, const void *dtotal, const float *mean,
                      const float *rstd, void *dx, void *dgamma, void *dbeta, void *workspace, size_t ws_bytes,
                      const gc_layer_norm_desc *d, int dtype, int param_dtype, void *stream)
{
    RowsGeom g;
    int st = check_rows(d, g);
    if (st == GC_OK) st = check_types(dtype, param_dtype, g);
    if (st != GC_OK) return st;
    for (const void *p : {gamma, static_cast<const void *>(dgamma), static_cast<const void *>(dbeta)})
        if (!aligned(p, size_of(param_dtype))) return GC_ERR_INVALID_ARG;
    if (g.rows) {
        const uintptr_t a = size_of(dtype);
        if (!given(x, a) || !given(dy, a) || !given(dx, a) || !aligned(dtotal, a)) return GC_ERR_INVALID_ARG;
        if (!given(mean, 4) || !given(rstd, 4)) return GC_ERR_INVALID_ARG;
    }
    RowsPlan q;
    plan_rows(g, dtype, true, dtotal, q);
    st = check_workspace(workspace, ws_bytes, g.rows && (dgamma || dbeta) ? q.ws_bytes : 0);
    if (st != GC_OK) return st;
    float *part = static_cast<float *>(workspace);
    hipStream_t s = static_cast<hipStream_t>(stream);
    return hip_status(dtype == GC_F32
                          ? launch_rows_bwd<float>(g, q, x, gamma, dy, dtotal, mean, rstd, dx, dgamma, dbeta, part, s)
                          : launch_rows_bwd<bf16_t>(g, q, x, gamma, dy, dtotal, mean, rstd, dx, dgamma, dbeta, part, s));
}

int gc_layer_norm_plan_name(int op, const gc_layer_norm_desc *d, int dtype, char *buf, size_t buf_bytes)
{
    RowsGeom g;
    const int st = check_rows(d, g);
    if (st != GC_OK) return st;
    if (!valid_dtype(dtype) || (op != GC_OP_FWD && op != GC_OP_BWD) || !buf || !buf_bytes) return GC_ERR_INVALID_ARG;
    RowsPlan q;
    plan_rows(g, dtype, op == GC_OP_BWD, false, q);
    const char *dir = op == GC_OP_BWD ? "bwd" : "fwd";
    if (q.loop)
        snprintf(buf, buf_bytes, "rows_%s_loop<N=%d> grid=%lld", dir, q.N, (long long)q.grid);
    else
        snprintf(buf, buf_bytes, "rows_%s<N=%d,NV=%d> team=%d threads=%d grid=%lld past=%d", dir, q.N, q.NV, q.L,
                 q.threads, (long long)q.grid, q.past);
    return GC_OK;
}

size_t gc_recurrence_workspace_bytes(int op, const gc_recurrence_desc *d, int dtype)
{
    ScanGeom g;
    ScanPlan q;
    if ((op != GC_OP_FWD && op != GC_OP_BWD) || !valid_dtype(dtype)) return 0;
    return check_scan(d, op == GC_OP_BWD, g) == GC_OK && plan_scan(g, dtype, op == GC_OP_BWD, false, q) ? q.ws_bytes : 0;
}

int gc_recurrence_fwd(const void *gate, const void *value, const float *h0, const uint8_t *reset, const int32_t *lengths,
                      void *out, float *last, float *states, void *workspace, size_t ws_bytes,
                      const gc_recurrence_desc *d, int dtype, void *stream)
{
    ScanGeom g;
    int st = check_scan(d, false, g);
    if (st != GC_OK) return st;
    if (!valid_dtype(dtype)) return GC_ERR_INVALID_ARG;
    if (!aligned(h0, 4) || !aligned(last, 4) || !aligned(states, 4) || !aligned(lengths, 4)) return GC_ERR_INVALID_ARG;
    if (g.B && g.T)
        for (const void *p : {gate, value, static_cast<const void *>(out)})
            if (!given(p, size_of(dtype))) return GC_ERR_INVALID_ARG;
    ScanPlan q;
    if (!plan_scan(g, dtype, false, lengths, q)) return GC_ERR_UNSUPPORTED;
    st = check_workspace(workspace, ws_bytes, q.ws_bytes);
    if (st != GC_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return hip_status(dtype == GC_F32
                          ? launch_scan_fwd<float>(g, q, gate, value, h0, reset, lengths, out, last, states, workspace, s)
                          : launch_scan_fwd<bf16_t>(g, q, gate, value, h0, reset, lengths, out, last, states, workspace, s));
}

int gc_recurrence_bwd(const void *gate, const void *value, const float *states, const uint8_t *reset,
                      const int32_t *lengths, const void *dout, const float *dlast, void *dgate, void *dvalue, float *dh0,
                      void *workspace, size_t ws_bytes, const gc_recurrence_desc *d, int dtype, void *stream)
{
    ScanGeom g;
    int st = check_scan(d, true, g);
    if (st != GC_OK) return st;
    if (!valid_dtype(dtype)) return GC_ERR_INVALID_ARG;
    if (!aligned(dlast, 4) || !aligned(dh0, 4) || !aligned(lengths, 4)) return GC_ERR_INVALID_ARG;
    if (g.B && g.T) {
        for (const void *p : {gate, value, dout, static_cast<const void *>(dgate), static_cast<const void *>(dvalue)})
            if (!given(p, size_of(dtype))) return GC_ERR_INVALID_ARG;
        if (!given(states, 4)) return GC_ERR_INVALID_ARG;
    }
    ScanPlan q;
    if (!plan_scan(g, dtype, true, lengths, q)) return GC_ERR_UNSUPPORTED;
    st = check_workspace(workspace, ws_bytes, q.ws_bytes);
    if (st != GC_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    return hip_status(dtype == GC_F32 ? launch_scan_bwd<float>(g, q, gate, value, states, reset, lengths, dout, dlast, dgate,
                                                               dvalue, dh0, workspace, s)
                                      : launch_scan_bwd<bf16_t>(g, q, gate, value, states, reset, lengths, dout, dlast,
                                                                dgate, dvalue, dh0, workspace, s));
}

int gc_recurrence_plan_name(int op, const gc_recurrence_desc *d, int dtype, char *buf, size_t buf_bytes)
{
    if ((op != GC_OP_FWD && op != GC_OP_BWD) || !valid_dtype(dtype) || !buf || !buf_bytes) return GC_ERR_INVALID_ARG;
    ScanGeom g;
    const int st = check_scan(d, op == GC_OP_BWD, g);
    if (st != GC_OK) return st;
    ScanPlan q;
    if (!plan_scan(g, dtype, op == GC_OP_BWD, false, q)) snprintf(buf, buf_bytes, "none");
    else
        snprintf(buf, buf_bytes, "scan_%s<N=%d> chunks=%d steps=%d lanes=%lld past=%d far=%d",
                 op == GC_OP_BWD ? "bwd" : "fwd", q.N, q.chunks, q.len, (long long)q.lanes, q.past, q.far);
    return GC_OK;
}

int gc_distill_fwd(const void *logits, const void *index, const void *teacher, float *loss, float *peak, float *mass,
                   const gc_distill_desc *d, int dtype, void *stream)
{
    DistillGeom g;
    const int st = check_distill(d, g);
    if (st != GC_OK) return st;
    if (!valid_dtype(dtype)) return GC_ERR_INVALID_ARG;
    if (g.rows == 0) return GC_OK;
    if (!entries_given(d, logits, index, teacher, dtype) || !given(loss, 4) || !aligned(peak, 4) || !aligned(mass, 4))
        return GC_ERR_INVALID_ARG;
    return distill_call(g, GC_OP_FWD, logits, index, teacher, peak, mass, nullptr, loss, nullptr, dtype, stream);
}

int gc_distill_bwd(const void *logits, const void *index, const void *teacher, const float *peak, const float *mass,
                   const float *dloss, void *dlogits, const gc_distill_desc *d, int dtype, void *stream)
{
    DistillGeom g;
    const int st = check_distill(d, g);
    if (st != GC_OK) return st;
    if (!valid_dtype(dtype)) return GC_ERR_INVALID_ARG;
    if (g.rows == 0) return GC_OK;
    if (!entries_given(d, logits, index, teacher, dtype) || !given(peak, 4) || !given(mass, 4) || !given(dloss, 4) ||
        !given(dlogits, size_of(dtype)))
        return GC_ERR_INVALID_ARG;
    return distill_call(g, GC_OP_BWD, logits, index, teacher, const_cast<float *>(peak), const_cast<float *>(mass), dloss,
                        nullptr, dlogits, dtype, stream);
}

int gc_distill_step(const void *logits, const void *index, const void *teacher, const float *dloss, float *loss,
                    void *dlogits, const gc_distill_desc *d, int dtype, void *stream)
{
    DistillGeom g;
    const int st = check_distill(d, g);
    if (st != GC_OK) return st;
    if (!valid_dtype(dtype)) return GC_ERR_INVALID_ARG;
    if (g.rows == 0) return GC_OK;
    if (!entries_given(d, logits, index, teacher, dtype) || !given(dloss, 4) || !given(loss, 4) ||
        !given(dlogits, size_of(dtype)))
        return GC_ERR_INVALID_ARG;
    return distill_call(g, GC_OP_STEP, logits, index, teacher, nullptr, nullptr, dloss, loss, dlogits, dtype, stream);
}

int gc_distill_plan_name(int op, const gc_distill_desc *d, int dtype, char *buf, size_t buf_bytes)
{
    DistillGeom g;
    const int st = check_distill(d, g);
    if (st != GC_OK) return st;
    if (!valid_dtype(dtype) || (op != GC_OP_FWD && op != GC_OP_BWD && op != GC_OP_STEP) || !buf || !buf_bytes)
        return GC_ERR_INVALID_ARG;
    DistillPlan q;
    plan_distill(g, dtype, op, q);
    const char *name = op == GC_OP_FWD ? "fwd" : op == GC_OP_BWD ? "bwd" : "step";
    if (!launchable(q.grid, q.threads)) snprintf(buf, buf_bytes, "none");
    else
        snprintf(buf, buf_bytes, "distill_%s<N=%d,NV=%d> team=%d threads=%d grid=%lld past=%d", name, q.N, q.NV, q.L,
                 q.threads, (long long)q.grid, q.past);
    return GC_OK;
}

}  // extern "C"
