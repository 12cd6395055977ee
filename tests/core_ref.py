"""Definitions in 64 bits of the recurrent core's operators (layer norm of a residual
stream, the gated recurrence, distillation), and bounds on how far a kernel may be
from them.

U = 2^-24 is half a step of fp32, half(t) that of the storage type t.  exp of an fp32
argument x, as exp2 of x times a rounded log2(e), is off by 3|x|U + 2U relative, a reciprocal
and each other step by at most 2U.
"""
import math

import torch

from train_ref import U, half, over  # noqa: F401

MORE = 1.01      # second-order terms
TINY = 1e-37


# -------------------------------------------------------------- layer norm --
def wide(p, D, none, like):
    return torch.full((D,), none, dtype=torch.float64, device=like.device) if p is None else p.double()


def chain(D):
    """Additions that a value of a row goes through: a thread adds at most 32 in a row (a workgroup's
    1024 threads take a longer row in turns, 8 values each), then lanes and waves."""
    return max(32, 8 * (D // 8192 + 1)) + 24


def rows_fwd(x, residual, gamma, beta, eps, t):
    """y, mean, rstd and total, each with its bound."""
    D = x.shape[1]
    s = x.double() if residual is None else x.double() + residual.double()
    g, b, k = wide(gamma, D, 1.0, x), wide(beta, D, 0.0, x), chain(D)
    mean = s.mean(1, keepdim=True)
    off = s - mean
    var = off.square().mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    y = off * rstd * g + b
    d_s = 0 * s if residual is None else U * s.abs()
    d_mean = (k + 3) * U * s.abs().mean(1, keepdim=True) + d_s.mean(1, keepdim=True)
    d_off = (d_s + d_mean + U * off.abs()) * MORE
    d_var = (2 * off.abs() * d_off + d_off.square()).mean(1, keepdim=True) + (k + 6) * U * var
    r_rstd = (d_var / (var + eps) / 2 + 5 * U) * MORE
    d_y = (g.abs() * rstd * (d_off + off.abs() * (r_rstd + 3 * U)) + U * (y.abs() + b.abs())) * MORE
    return ((y, d_y + half(t) * (y.abs() + d_y) + TINY), (mean[:, 0], d_mean[:, 0] * MORE + TINY),
            (rstd[:, 0], (r_rstd * rstd)[:, 0] + TINY), (s, d_s + half(t) * (s.abs() + d_s) + TINY))


def rows_bwd(x, gamma, dy, mean, rstd, dtotal, t, pt):
    """dx, dgamma and dbeta, each with its bound."""
    rows, D = x.shape
    g, k = wide(gamma, D, 1.0, x), chain(D)
    r = rstd.double()[:, None]
    hat = (x.double() - mean.double()[:, None]) * r
    d = dy.double()
    w = g * d
    wh = w * hat
    c1, c2 = w.mean(1, keepdim=True), wh.mean(1, keepdim=True)
    a1, a2 = w.abs().mean(1, keepdim=True), wh.abs().mean(1, keepdim=True)
    dx = r * (w - c1 - hat * c2)
    d_c1, d_c2 = (k + 4) * U * a1, (k + 8) * U * a2
    d_dx = r * (2 * U * w.abs() + d_c1 + 2 * U * (hat * c2).abs() + hat.abs() * d_c2
                + 5 * U * (w.abs() + c1.abs() + (hat * c2).abs())) + U * dx.abs()
    if dtotal is not None:
        dx = dx + dtotal.double()
        d_dx = d_dx + U * dx.abs()
    d_dx = d_dx * MORE
    # a team adds its rows, its workgroup's teams and the workgroups' rows of partials are added in turn
    kp = rows // 64 + 64
    dgamma, dbeta = (d * hat).sum(0), d.sum(0)
    d_gamma, d_beta = (kp + 4) * U * (d * hat).abs().sum(0) * MORE, kp * U * d.abs().sum(0) * MORE
    return ((dx, d_dx + half(t) * (dx.abs() + d_dx) + TINY), (dgamma, d_gamma + half(pt) * (dgamma.abs() + d_gamma) + TINY),
            (dbeta, d_beta + half(pt) * (dbeta.abs() + d_beta) + TINY))


# -------------------------------------------------------------- recurrence --
def gates(f):
    """a, i = 1 - a, and the relative errors of both."""
    a, i = torch.sigmoid(f), torch.sigmoid(-f)
    r_e = (3 * f.abs() + 2) * U
    # a stays at 1.8e-35 below -80, which counts as an absolute error of the state
    return a, i, (i * r_e + 4 * U) * MORE, (a * r_e + 6 * U) * MORE


def _masks(gate, reset, lengths):
    B, T, _ = gate.shape
    dev = gate.device
    cut = torch.zeros((B, T), dtype=torch.bool, device=dev) if reset is None else reset.bool()
    n = torch.full((B,), T, device=dev) if lengths is None else lengths.long().clamp(0, T)
    return cut[..., None], (torch.arange(T, device=dev) < n[:, None])[..., None]


class Scan:
    """The recurrence step by step: out, last and every state before a step, with bounds.

    The kernels may cut the steps into chunks and carry states over them, which adds the
    shares of a state in another order: a state is a sum of positive shares of the values and
    of h0, and each rounding counts for the sum of their absolute values (`size`), twice for
    the two ways a share goes (through its chunk and over the others)."""

    def __init__(self, gate, value, h0, reset, lengths, coupled):
        B, T, D = gate.shape
        f, v = gate.double(), value.double()
        self.a, self.i, self.r_a, self.r_i = gates(f)
        self.cut, self.ok = _masks(gate, reset, lengths)
        self.v, self.coupled = v, coupled
        h = torch.zeros((B, D), dtype=torch.float64, device=gate.device) if h0 is None else h0.double()
        size, err = h.abs(), torch.zeros_like(h)
        shape = (B, T, D)
        self.out, self.d_out, self.before, self.d_before = (torch.zeros(shape, dtype=torch.float64, device=gate.device)
                                                            for _ in range(4))
        for t in range(T):
            a, i = self.a[:, t], self.i[:, t]
            b, sb, eb = (torch.where(self.cut[:, t], 0.0, q) for q in (h, size, err))
            self.before[:, t], self.d_before[:, t] = b, eb
            take = i if coupled else torch.ones_like(i)
            new = a * b + take * v[:, t]
            s = a * sb + take * v[:, t].abs()
            local = i * (self.r_i[:, t] + 2 * U) * (sb + (v[:, t].abs() if coupled else 0.0)) + 3 * U * s + 2e-35 * sb
            e = (a * eb + 2 * local) * (1 + 4 * U)
            ok = self.ok[:, t]
            self.out[:, t], self.d_out[:, t] = new * ok, e * ok
            h, size, err = (torch.where(ok, p, q) for p, q in ((new, h), (s, size), (e, err)))
        self.last, self.d_last = h, err * MORE + TINY

    def stored(self, t):
        e = self.d_out * MORE
        return self.out, e + half(t) * (self.out.abs() + e) + TINY * self.ok

    def backward(self, dout, dlast, t):
        """dgate, dvalue and dh0, each with its bound."""
        B, T, D = self.out.shape
        back = torch.zeros((B, D), dtype=torch.float64, device=dout.device) if dlast is None else dlast.double()
        size, err = back.abs(), torch.zeros_like(back)
        res = [torch.zeros((B, T, D), dtype=torch.float64, device=dout.device) for _ in range(4)]
        dg, e_g, dv, e_v = res
        for s in range(T - 1, -1, -1):
            a, i, ra, ri = (q[:, s] for q in (self.a, self.i, self.r_a, self.r_i))
            d, ok, cut = dout[:, s].double(), self.ok[:, s], self.cut[:, s]
            g, gs, ge = back + d, size + d.abs(), err + U * (size + d.abs())
            v = self.v[:, s] if self.coupled else 0.0
            off = self.before[:, s] - v
            d_off = self.d_before[:, s] + U * off.abs()
            slope = a * i * off
            dg[:, s] = slope * g * ok
            e_g[:, s] = ok * (slope.abs() * ((ra + ri + 5 * U) * gs + ge) + a * i * d_off * (gs + ge))
            dv[:, s] = (i * g if self.coupled else g) * ok
            e_v[:, s] = ok * (i * ((ri + U) * gs + ge) if self.coupled else ge)
            through = [torch.where(cut, 0.0, q) for q in (a * g, a * gs, a * ge + 2 * (i * ri + 3 * U) * gs + 2e-35 * gs)]
            back, size, err = (torch.where(ok, p, q) for p, q in zip(through, (back, size, err)))
        out = []
        for val, e in ((dg, e_g), (dv, e_v)):
            e = e * MORE
            out.append((val, e + half(t) * (val.abs() + e) + TINY * self.ok))
        return (*out, (back, err * MORE + TINY))


# ------------------------------------------------------------ distillation --
def distill(logits, index, teacher, tau, dloss, t):
    """(loss, bound), (peak, mass and its bound), (dlogits, bound).  Logits without NaN or
    +inf, teacher's shares where a logit is -inf allowed."""
    rows, V = logits.shape
    K = index.shape[1]
    z, idx = logits.double(), index.long()
    ok = (idx >= 0) & (idx < V)
    at = torch.where(ok, idx, 0)
    peak = z.amax(1, keepdim=True)
    x = (z - peak) / tau
    e = torch.exp(x)
    mass = e.sum(1, keepdim=True)
    q = e / mass
    finite = torch.where(torch.isfinite(x), x.abs(), 0.0)
    k = max(64, V // 1024 + 8) + 24
    r_s = (q * 3 * U * finite).sum(1, keepdim=True) + (2 + 4 * k) * U
    tt = torch.where(ok, teacher.double() / tau, -math.inf)
    top = tt.amax(1, keepdim=True)
    some = top > -math.inf
    y = torch.where(some, tt - top, -math.inf)
    total = torch.exp(y).sum(1, keepdim=True)
    p = torch.where(some, torch.exp(y) / total, 0.0)
    fy = torch.where(torch.isfinite(y), y.abs(), 0.0)
    r_t = (p * 3 * U * fy).sum(1, keepdim=True) + (K // 8 + 12) * U
    r_p = 3 * U * fy + r_t + 5 * U
    zk = torch.where(ok, x.gather(1, at), 0.0)
    logs, logt = torch.log(mass), torch.log(torch.where(some, total, 1.0))
    term = torch.where(p > 0, y - logt - zk + logs, 0.0)
    fz = torch.where(torch.isfinite(zk), zk.abs(), 0.0)
    d_term = 5 * U * (fy + fz) + 4 * U * (logs.abs() + logt.abs()) + r_s + r_t + 2 * U
    each = torch.where(p > 0, p * term, 0.0)
    loss = tau * tau * each.sum(1)
    d_loss = tau * tau * (p * d_term + torch.where(torch.isfinite(each), each.abs(), 0.0) * (r_p + (K // 8 + 12) * U)).sum(1)
    at_p, d_p = (torch.zeros_like(z).scatter_add_(1, at, torch.where(ok, v, 0.0)) for v in (p, p * (r_p + K * U)))
    by = torch.where(some, dloss.double()[:, None] * tau, 0.0)
    dz = by * (torch.where(some, q, 0.0) - at_p)
    d_dz = by.abs() * (q * (3 * U * finite + r_s + 6 * U) + d_p + 2 * U * (q + at_p)) * MORE
    return ((loss, d_loss * MORE + TINY), (peak[:, 0], mass[:, 0], r_s[:, 0] * mass[:, 0] * MORE),
            (dz, d_dz + half(t) * (dz.abs() + d_dz) + TINY))
