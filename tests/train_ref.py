"""Definitions in 64 bits of the operators around the convolutions, and bounds
on how far a kernel may be from them.

u = 2^-24 is half a step of fp32, half(t) that of the storage type t.  A sum
whose longest chain of additions is k values is off by at most k*u times
the sum of the absolute values.
"""
import math

import torch

U = 2.0 ** -24
DEV = "cuda"


def half(t):
    return torch.finfo(t).eps / 2


def over(got, ref, bound):
    """The largest |got - ref| / bound (0/0 counts as 0)."""
    err = (got.double() - ref).abs()
    assert bool(torch.isfinite(err).all()), "not finite"
    return float(torch.where(err == 0, 0.0, err / bound).max()) if err.numel() else 0.0


# --------------------------------------------------------------- embedding --
def embed_fwd(tok, table, scale):
    ok = (tok >= 0) & (tok < table.shape[0])
    rows = table.double()[torch.where(ok, tok, 0).long()] * scale
    return torch.where(ok[..., None], rows, 0.0)


def embed_bwd(tok, dout, V, scale):
    """The gradient, the sum of absolute values behind it and each row's number of tokens."""
    D = dout.shape[-1]
    ok = ((tok >= 0) & (tok < V)).reshape(-1)
    # by sorted tokens: 64-bit atomics on one row take minutes where all tokens are equal
    t, order = tok.reshape(-1)[ok].long().sort(stable=True)
    rows = (dout.reshape(-1, D)[ok].double() * scale)[order]
    counts = torch.searchsorted(t, torch.arange(V + 1, device=t.device)).diff()

    def total(v):
        return torch.segment_reduce(v, "sum", lengths=counts, axis=0, unsafe=True, initial=0.0)

    return total(rows), total(rows.abs()), counts


# -------------------------------------------------------------- group norm --
def act(z, name):
    if name == "relu":
        return z.clamp(min=0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * torch.special.ndtr(z)
    return z


def act_grad(z, name):
    if name == "relu":
        return (z > 0).double()
    if name == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def act_error(z, name):
    """Bound on the kernels' error in act(z) and in act'(z), beyond that of z itself: exp's argument
    is off by u relative (|z| u, and as much again for the factor log2 e), each further step by u;
    gelu's Phi by 0.75e-7 (Abramowitz and Stegun 7.1.26)."""
    a = z.abs()
    if name == "silu":
        return a * (2 * a + 12) * U, (1 + a) * (2 * a + 16) * U
    if name == "gelu":
        phi = 0.75e-7 + (2 * a * a * torch.exp(-a * a / 2) + 12) * U
        return a * phi, phi + a * torch.exp(-a * a / 2) * (2 * a * a + 12) * U
    return torch.zeros_like(a), torch.zeros_like(a)


def per_image(m, C):
    """(B, groups) as (B, C, 1, 1)."""
    return m.double().repeat_interleave(C // m.shape[1], 1)[:, :, None, None]


def channels(p, C, none, like):
    return torch.full((1, C, 1, 1), none, dtype=torch.float64, device=like.device) if p is None \
        else p.double().reshape(1, C, 1, 1)


def norm_stats(x, G, eps):
    v = x.double().reshape(x.shape[0], G, -1)
    mean = v.mean(2)
    var = (v - mean[:, :, None]).square().mean(2)
    return mean, 1 / torch.sqrt(var + eps), var


def norm_fwd(x, gamma, beta, G, name, eps):
    C = x.shape[1]
    mean, rstd, _ = norm_stats(x, G, eps)
    z = (x.double() - per_image(mean, C)) * per_image(rstd, C) * channels(gamma, C, 1.0, x) + channels(beta, C, 0.0, x)
    return act(z, name), mean, rstd


def chain(M):
    """Additions one value goes through in a group's sum: a thread adds up to 128 values in a row,
    then lanes and waves (16 + 10)."""
    return min(M, 128) + 26


def norm_fwd_bounds(x, gamma, beta, G, name, eps):
    """Bounds for y, mean and rstd."""
    B, C = x.shape[:2]
    t = x.dtype
    mean, rstd, var = norm_stats(x, G, eps)
    v = x.double().reshape(B, G, -1)
    k = chain(v.shape[2])
    d_mean = k * U * v.abs().mean(2) + U * mean.abs()
    # two passes: each square is off by 4u, the sum by k u, and the mean's error adds its own square
    r_rstd = ((k + 6) * U + d_mean.square() / (var + eps)) / 2 + 4 * U
    g, b = channels(gamma, C, 1.0, x).abs(), channels(beta, C, 0.0, x).abs()
    off = x.double() - per_image(mean, C)
    term = off.abs() * per_image(rstd, C) * g
    z = off * per_image(rstd, C) * channels(gamma, C, 1.0, x) + channels(beta, C, 0.0, x)
    d_z = g * per_image(rstd, C) * (per_image(d_mean, C) + U * off.abs()) + term * (per_image(r_rstd, C) + 3 * U) \
        + U * (z.abs() + b * U)
    y = act(z, name)
    d_y = 1.13 * d_z + act_error(z, name)[0]      # silu' and gelu' stay below 1.13
    return d_y * 1.01 + half(t) * (y.abs() + d_y) + 1e-37, d_mean + 1e-37, r_rstd * rstd + 1e-37


def norm_bwd(x, gamma, beta, dy, mean, rstd, G, name):
    B, C = x.shape[:2]
    r = per_image(rstd, C)
    hat = (x.double() - per_image(mean, C)) * r
    gm = channels(gamma, C, 1.0, x)
    g = dy.double() * act_grad(hat * gm + channels(beta, C, 0.0, x), name)
    w = g * gm
    c1 = per_image(w.reshape(B, G, -1).mean(2), C)
    c2 = per_image((w * hat).reshape(B, G, -1).mean(2), C)
    return r * (w - c1 - hat * c2), (g * hat).sum((0, 2, 3)), g.sum((0, 2, 3))


def norm_bwd_bounds(x, gamma, beta, dy, mean, rstd, G, name):
    """Bounds for dx, dgamma and dbeta."""
    B, C, H, W = x.shape
    r = per_image(rstd, C)
    hat = (x.double() - per_image(mean, C)) * r
    gm, bt = channels(gamma, C, 1.0, x), channels(beta, C, 0.0, x)
    z = hat * gm + bt
    d_hat = 2 * U * hat.abs() * 1.01
    d_z = d_hat * gm.abs() + U * z.abs() * 1.01
    # |silu''| and |gelu''| stay below 1
    d_der = act_error(z, name)[1] + (d_z if name in ("silu", "gelu") else 0 * d_z)
    a_dy = dy.double().abs()
    g = a_dy * act_grad(z, name).abs()
    d_g = (a_dy * d_der + U * g) * 1.01
    k = chain(C // G * H * W)

    def mean_of(v):
        return per_image(v.reshape(B, G, -1).mean(2), C)

    w, d_w = g * gm.abs(), (d_g + 2 * U * g) * gm.abs()
    wh, d_wh = w * hat.abs(), d_w * hat.abs() + w * d_hat + 2 * U * w * hat.abs()
    c1, c2 = mean_of(w), mean_of(wh)
    d_c1, d_c2 = mean_of(d_w) + (k + 4) * U * c1, mean_of(d_wh) + (k + 4) * U * c2
    d_dx = r * (d_w + d_c1 + d_hat * c2 + hat.abs() * d_c2 + 6 * U * (w + c1 + hat.abs() * c2)) * 1.01
    dx = r * (w + c1 + hat.abs() * c2)
    # parameters: a chain within an image, up to 1024 images of a workgroup in a row, then rows of partials
    kp = min(H * W, 128) + 26 + min(B, 1024) + B // 32 + 64
    over_all = (0, 2, 3)
    d_beta = d_g.sum(over_all) + kp * U * g.sum(over_all)
    gh = g * hat.abs()
    d_gamma = (d_g * hat.abs() + g * d_hat + U * gh).sum(over_all) + kp * U * gh.sum(over_all)
    t = x.dtype
    return (d_dx + half(t) * (dx + d_dx) + 1e-37, d_gamma + 1e-37, d_beta + 1e-37)
