"""Plain 64-bit forms of the calls of include/gdn_stack.h (test infrastructure), written from their
definitions, with what bounds their rounding errors.

Error bounds count roundings of E32 = 2^-24 (half a step of fp32, relative):

norm     a sum of d squares by 8 terms in a lane and 4 or 3 levels of lanes is off by at most 12 E32 relative, plus the
         mean's and eps' one each; the reciprocal root by half of that and 2 of its own: 9.  x r, w, the scale: 3.  The
         rotation: an angle in 64 bits, rounded as a fraction of a turn (pi E32 of the radius), sine and cosine within 4,
         product and sum 2: 10.  In all 22 of the magnitudes that the rotation adds; 32 are allowed.
backward 32 for w dz and for n alike, twice that for their products' sum, whose magnitude is the sum of magnitudes, 12 for
         its own additions, 3 for the last step: 32 of |w dz| r and 80 of |n| c sum |w dz n| r; 96 are allowed of both.
         A weight's gradient: 64 for each term and one for each addition, of which there are at most as many as terms.
scan     a decay is off by 2 (the exponential) + 1.5 |g| (its argument, rounded twice); a state's product and sum 2 more,
         and a product of decays over the tokens of a run, with the run's step, 2 more.  A term that a state took in m
         tokens ago is off by at most m (6 + 1.5 |g|) of its magnitude, so the bound is a recurrence of its own beside that of magnitudes.
         A term itself: 1 - e^g within 10, its product 1.
"""

import numpy as np
import torch

E32, E16 = 2.0 ** -24, 2.0 ** -8


def half_step(dtype):
    return E16 if dtype == torch.bfloat16 else E32


# ---------------------------------------------------------------- norm


def _pairs(d, rotary, interleaved):
    """Channels u and w of the pairs."""
    i = torch.arange(rotary // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)


def turned(x, positions, freq, interleaved, back=False):
    """x [T, heads, d] rotated, and the magnitudes that were added."""
    y, mag = x.clone(), x.abs()
    if freq is None:
        return y, mag
    u, w = _pairs(x.shape[-1], 2 * freq.numel(), interleaved)
    a = positions.double()[:, None, None] * freq.double()[None, None, :]
    c, s = torch.cos(a), torch.sin(a) * (-1 if back else 1)
    y[..., u], y[..., w] = x[..., u] * c - x[..., w] * s, x[..., u] * s + x[..., w] * c
    both = x[..., u].abs() + x[..., w].abs()
    mag[..., u], mag[..., w] = both, both
    return y, mag


def _norm(x, norm, eps):
    """r and c."""
    d = x.shape[-1]
    c = 1.0 / d if norm == 2 else 1.0
    return (torch.ones_like(x[..., :1]) if norm == 0 else (x.square().sum(-1, keepdim=True) * c + eps).rsqrt()), c


def qk_norm(x, norm, eps, weight, positions, freq, interleaved, scale):
    """x [T, heads, d] in float64; returns y and the bound of its fp32 arithmetic."""
    r, _ = _norm(x, norm, eps)
    z = x * r * (1.0 if weight is None else weight)
    y, mag = turned(z, positions, freq, interleaved)
    return y * scale, 32 * E32 * mag * abs(scale)


def qk_norm_backward(x, dy, norm, eps, weight, positions, freq, interleaved, scale):
    """Returns (dx, its bound, dw, its bound)."""
    r, c = _norm(x, norm, eps)
    n = x * r
    dz, mag = turned(dy * scale, positions, freq, interleaved, back=True)
    dw, big = (dz * n).sum((0, 1)), (mag * n.abs()).sum((0, 1))
    terms = x.shape[0] * x.shape[1]
    w = 1.0 if weight is None else weight
    dn, mn = dz * w, mag * (w if weight is None else weight.abs())
    if norm == 0:
        return dn, 96 * E32 * mn, dw, (64 + terms) * E32 * big
    dx = r * (dn - n * c * (dn * n).sum(-1, keepdim=True))
    bound = 96 * E32 * r * (mn + n.abs() * c * (mn * n.abs()).sum(-1, keepdim=True))
    return dx, bound, dw, (64 + terms) * E32 * big


# ---------------------------------------------------------------- scan


def scan(x, g, cu, mix, init):
    """float64 tensors; returns dict(h, final and their bounds dh_, dfinal_, and h_{t-1} with magnitude and bound)."""
    T, C = x.shape
    a, n = torch.exp(g), len(cu) - 1
    b = (1 - a) * x if mix else x
    off = 6 + 1.5 * g.abs()
    out = {k: torch.zeros((T, C), dtype=torch.float64) for k in ("h", "bound", "before", "big", "off")}
    final = torch.zeros((n, C), dtype=torch.float64) if init is None else init.clone()
    final_bound = torch.zeros((n, C), dtype=torch.float64)
    for m in range(n):
        s = final[m].clone()
        mag, err = s.abs(), torch.zeros(C, dtype=torch.float64)
        for t in range(cu[m], cu[m + 1]):
            out["before"][t], out["big"][t], out["off"][t] = s, mag, err
            err = torch.where(mag > 0, a[t] * (err + off[t] * mag), 0.0) + 12 * b[t].abs()
            s = a[t] * s + b[t]
            mag = a[t] * mag + b[t].abs()
            out["h"][t], out["bound"][t] = s, err * E32
        final[m], final_bound[m] = s, err * E32
    return dict(out, final=final, final_bound=final_bound)


def scan_backward(x, g, cu, mix, init, dh, d_final):
    """Returns dx, dg, d_init, each with its bound."""
    T, C = x.shape
    f = scan(x, g, cu, mix, init)
    a, n = torch.exp(g), len(cu) - 1
    off = 6 + 1.5 * g.abs()
    lam, big, err = (torch.zeros((T, C), dtype=torch.float64) for _ in range(3))
    d_init = torch.zeros((n, C), dtype=torch.float64) if d_final is None else d_final.clone()
    d_init_bound = torch.zeros((n, C), dtype=torch.float64)
    for m in range(n):
        c, mag, e = d_init[m].clone(), d_init[m].abs(), torch.zeros(C, dtype=torch.float64)
        for t in reversed(range(cu[m], cu[m + 1])):
            lam[t], big[t] = dh[t] + c, dh[t].abs() + mag
            err[t] = e + big[t]
            c, mag, e = a[t] * lam[t], a[t] * big[t], a[t] * (err[t] + off[t] * big[t])
        d_init[m], d_init_bound[m] = c, e * E32
    om = 1 - a if mix else torch.ones_like(a)
    past = f["before"] - x if mix else f["before"]
    past_mag, past_err = f["big"] + (x.abs() if mix else 0), f["off"] + (f["big"] + x.abs() if mix else 0)
    c_err = a * (err + off * big)
    dg = a * lam * past
    return dict(dx=om * lam, dx_bound=E32 * om * (err + 12 * big), dg=dg,
                dg_bound=E32 * (c_err * past_mag + a * big * past_err + 2 * a * big * past_mag), d_init=d_init,
                d_init_bound=d_init_bound)


def scan_pool(x, g, states, slots, cu, commit, mix):
    """Returns h (NaN where nothing is written), states, and bounds."""
    h, bound = torch.full_like(x, np.nan), torch.zeros_like(x)
    out, out_bound = states.clone(), torch.zeros_like(states)
    for n, slot in enumerate(slots):
        if not 0 <= slot < states.shape[0]:
            continue
        lo, hi = cu[n], cu[n + 1]
        if hi <= lo:
            continue
        f = scan(x[lo:hi], g[lo:hi], [0, hi - lo], mix, states[slot][None])
        h[lo:hi], bound[lo:hi] = f["h"], f["bound"]
        keep = hi - lo if commit is None else min(commit[n], hi - lo)
        if keep > 0:
            out[slot], out_bound[slot] = f["h"][keep - 1], f["bound"][keep - 1]
    return h, bound, out, out_bound
