"""Plain 64-bit forms of the 8-bit operators and of the layer for a few
tokens, on the CPU, with the bounds their kernels are held to."""
import math

import torch

from tests.ops_ref import U, half_step, smallest


def swiglu(x):
    """silu(gate) * up in 64 bits."""
    gate, up = x.double().chunk(2, dim=1)
    return gate / (1.0 + torch.exp(-gate)) * up


def quant(v):
    """(q, s) of rows v in 64 bits: q rounded as the exact quotient is.  The
    numerators of 24-bit values times 127 are exact, and two different
    quotients of such numbers, or one and a tie, are further apart than 64 bits
    round."""
    v = v.double()
    most = v.abs().amax(1)
    fine = torch.isfinite(most) & (most > 0)
    q = torch.round(127.0 * v / torch.where(fine, most, torch.ones_like(most))[:, None])
    q = torch.where(fine[:, None], q, torch.zeros_like(q))
    s = torch.where(torch.isfinite(most), most / 127.0, torch.full_like(most, math.nan))
    return q.to(torch.int8), s


def product_i8(first, count, x, xs, w, ws, out):
    """Exact sums times the scales, written over `out` (64 bits); rows of no
    group stay."""
    rows = x.shape[0]
    for g, (f, c) in enumerate(zip(first, count)):
        lo, hi = max(0, f), min(rows, f + c)
        if hi > lo:
            y = x[lo:hi].double() @ w[g].double().t()  # integers below 2^53: exact
            out[lo:hi] = y * xs[lo:hi].double()[:, None] * ws[g].double()
    return out


def product_i8_bound(ref, dtype):
    """The sum's rounding to fp32, the two products' and the output's."""
    return ref.abs() * (3.0 * U * (1 + 3 * U) + half_step(dtype)) * (1 + 2 ** -10) + smallest(dtype)


def layer(x, idx, w, w13, w2, s13, s2):
    """(out, bound part): out [T, H] in 64 bits, and the sum of the errors of
    the 32-bit sums before the last rounding.

    gate, up: (2 H + 8) U of their absolute sums (matrix sums may truncate: 2 U
    a term).  silu has a slope of at most 1.1 and the product rule gives
    dh <= |up| 1.1 dgate + |silu| dup, plus 2^-20 of |h| for the exponential,
    the reciprocal and the products (the exponential's argument is rounded to
    2^-24 of at most ~88 before it counts), plus 2^-17 of |h| for the two parts
    (2^-9 * 2^-9 and their rounding).  The down sums: (2 terms + 8) U of their
    absolute sums over all pairs, the shares' products included; fp16 weights
    leave out 2^-8 * 2^-8 of each term (both low parts)."""
    T, H = x.shape
    I = w2.shape[2]
    out = torch.zeros(T, H, dtype=torch.float64)
    err = torch.zeros(T, H, dtype=torch.float64)
    total = torch.zeros(T, H, dtype=torch.float64)
    E = w2.shape[0]
    terms = 0
    for t in range(T):
        for j in range(idx.shape[1]):
            e = int(idx[t, j])
            if not 0 <= e < E:
                continue
            a, b = w13[e].double(), w2[e].double()
            if s13 is not None:
                a, b = a * s13[e].double()[:, None], b * s2[e].double()[:, None]
            xt = x[t].double()
            gu, ga = a @ xt, a.abs() @ xt.abs()
            dg = (2 * H + 8) * U * ga + 2 * U * gu.abs()
            g, u = gu[:I], gu[I:]
            silu = g / (1.0 + torch.exp(-g))
            h = silu * u
            dh = u.abs() * 1.1 * dg[:I] + (silu.abs() + 1.1 * dg[:I]) * dg[I:] + \
                (2.0 ** -20 + 2.0 ** -17) * h.abs()
            wt = float(w[t, j])
            out[t] += wt * (b @ h)
            err[t] += abs(wt) * (b.abs() @ dh)
            total[t] += abs(wt) * (b.abs() @ h.abs())
            terms += I
    n = max(1, terms // max(1, T))
    lost = 2.0 ** -15 if w2.dtype == torch.float16 else 0.0
    return out, err + ((2 * n + 64) * U + lost) * total


def layer_bound(ref, err, dtype):
    return half_step(dtype) * (ref.abs() + err) + err + smallest(dtype)
