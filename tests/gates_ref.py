"""The gated recurrence in 64 bits, with bounds that count every rounding for what the gate lets of it through.

U = 2^-24 is half a step of fp32.  A gate f has a smaller share s and a larger one, 1 - s: open (f >= 0) it
takes s of the value and keeps the rest of the state, closed it keeps s of the state.  e = exp(-|f|) as
exp2 of a product with a rounded log2(e): the product and the addition to it are off by
(1.3|f| + 0.7)U in the exponent, exp2 by 2U, so e by r_e = (1.5|f| + 3)U relative; 1/(1 + e) by 3U + s*r_e;
s = e/(1 + e) by r_s = r_e + 5U.  Below 2^-126 both may be 0: FLOOR, absolute.

A step is s*q + (p - s*p) or p + s*(q - p), p the one it has the larger share of: r_s of s*(|p| + |q|) and U of
each product and sum.  Where steps are cut into chunks, what came from before a chunk and what began in it
are worked out apart and added, so sizes are sums of absolute shares (`size`), and each rounding
counts twice.
"""
import torch

from train_ref import U, half

FLOOR = 2.0 ** -126
MORE = 1.01
TINY = 1e-37


class Shares:
    """Outputs and gradients with a bound each; neither resets nor lengths."""

    def __init__(self, gate, value, h0, coupled):
        B, T, D = gate.shape
        self.T, self.v, self.coupled = T, value.double(), coupled
        f = gate.double()
        self.a, self.i = torch.sigmoid(f), torch.sigmoid(-f)
        self.s = torch.minimum(self.a, self.i)
        r_e = (1.5 * f.abs() + 3) * U
        # absolute errors of s, and of 1 - s
        self.d_s = self.s * (r_e + 5 * U) + FLOOR
        self.r_large = 3 * U + self.s * r_e
        h = torch.zeros((B, D), dtype=torch.float64, device=gate.device) if h0 is None else h0.double()
        size, err = h.abs(), torch.zeros_like(h)
        self.out, self.d_out, self.before, self.d_before = (torch.empty_like(f) for _ in range(4))
        for t in range(T):
            a, v, s, d_s = self.a[:, t], self.v[:, t], self.s[:, t], self.d_s[:, t]
            self.before[:, t], self.d_before[:, t] = h, err
            take = self.i[:, t] if coupled else 1.0
            both = size + (v.abs() if coupled else 0.0)
            new = a * size + take * v.abs()
            local = (d_s + 2 * U * s) * both + 2 * U * new
            h, size, err = a * h + take * v, new, a * err + 2 * local
            self.out[:, t], self.d_out[:, t] = h, err
        self.last, self.d_last = h, err * MORE + TINY

    def stored(self, t):
        e = self.d_out * MORE
        return self.out, e + half(t) * (self.out.abs() + e) + TINY

    def backward(self, dout, dlast, t):
        """dgate, dvalue and dh0, each with its bound."""
        back = dlast.double()
        size, err = back.abs(), torch.zeros_like(back)
        dg, e_g, dv, e_v = (torch.empty_like(self.out) for _ in range(4))
        for k in range(self.T - 1, -1, -1):
            a, i, s, d_s = (q[:, k] for q in (self.a, self.i, self.s, self.d_s))
            d = dout[:, k].double()
            g, gs, ge = back + d, size + d.abs(), err + U * (size + d.abs())
            v = self.v[:, k] if self.coupled else torch.zeros_like(d)
            off, slope = self.before[:, k] - v, a * i * (self.before[:, k] - v)
            d_off = self.d_before[:, k] + U * off.abs()
            r_slope = self.r_large[:, k] + 5 * U
            dg[:, k] = slope * g
            e_g[:, k] = slope.abs() * (r_slope * gs + ge) + (1 - s) * (d_s * off.abs() + s * d_off) * (gs + ge)
            dv[:, k] = i * g if self.coupled else g
            e_v[:, k] = (d_s + 2 * U * i) * gs + i * ge if self.coupled else ge
            back, size, err = a * g, a * gs, a * ge + 2 * (d_s + 2 * U * a) * gs
        out = []
        for val, e in ((dg, e_g), (dv, e_v)):
            e = e * MORE
            out.append((val, e + half(t) * (val.abs() + e) + TINY))
        return (*out, (back, err * MORE + TINY))
