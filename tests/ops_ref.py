"""Plain 64-bit forms of the operators around the MoE path, for their tests,
with the bounds their kernels' 32-bit arithmetic is held to.

A bound is a tensor of absolute errors: half a step of the output's type
times the value (the one final rounding), plus the error of the 32-bit sums
before it, each at most (terms + a few) * 2^-24 times the sum of the
absolute terms.  U is that unit; sums inside the matrix instructions may
truncate instead of rounding, which costs up to 2 U per term.
"""
import math

import torch

U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def smallest(dtype):
    """Half the distance of the numbers next to zero."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def assert_within(got, ref, bound, what):
    got = got.detach().double().cpu()
    ref, bound = ref.double().cpu(), bound.double().cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    if got.numel() == 0:
        return
    err = (got - ref).abs()
    bad = ~(err <= bound)
    if bool(bad.any()):
        i = int((err / bound.clamp_min(1e-300)).nan_to_num(nan=math.inf).argmax())
        raise AssertionError("%s: %d of %d off; worst got %r want %r bound %.3e" % (
            what, int(bad.sum()), bad.numel(), float(got.flatten()[i]), float(ref.flatten()[i]),
            float(bound.flatten()[i])))


# ------------------------------------------------------ products by group --
def rows_of(first, count, rows):
    """[(lo, hi)] of the groups' rows inside [0, rows)."""
    out = []
    for f, c in zip(first, count):
        lo, hi = max(0, f), min(rows, f + c)
        out.append((lo, max(lo, hi)))
    return out


def product(a, b):
    """a @ b with its bound's sum of absolute terms, in 64 bits on the CPU."""
    a, b = a.double(), b.double()
    return a @ b, a.abs() @ b.abs()


def product_bound(ref, absum, terms, dtype):
    return half_step(dtype) * ref.abs() + (2 * terms + 8) * U * absum + smallest(dtype)


# ------------------------------------------------------------- the router --
def choose(logits, topk, score, bias, groups, kept):
    """ids [T, K] (list of lists), from 64-bit values."""
    T, E = logits.shape
    per = E // groups
    ids = []
    for t in range(T):
        l = [float(v) for v in logits[t].double()]
        ok = [v == v and v != -math.inf for v in l]
        if bias is None and groups == 1:
            c = [v if o else -math.inf for v, o in zip(l, ok)]
        else:
            if score == "softmax":
                m = max([v for v, o in zip(l, ok) if o], default=0.0)
                p = [(1.0 if v == m else math.exp(v - m)) if o else 0.0 for v, o in zip(l, ok)]
                s = sum(p)
                c = [v / s if s else 0.0 for v in p]
            else:
                c = [(1.0 / (1.0 + math.exp(-v)) if v > -700 else math.exp(v)) if o else 0.0
                     for v, o in zip(l, ok)]
            if bias is not None:
                c = [v + float(b) for v, b in zip(c, bias.double())]
            c = [v if o and v == v else -math.inf for v, o in zip(c, ok)]
        keep = set(range(groups))
        if groups > 1:
            gs = []
            for g in range(groups):
                best = sorted((v for v in c[g * per:(g + 1) * per] if v > -math.inf),
                              reverse=True)[:2]
                gs.append(sum(best) if best else -math.inf)
            keep = set(sorted(range(groups), key=lambda g: (-gs[g], g))[:kept])
        order = sorted((e for e in range(E) if e // per in keep), key=lambda e: (-c[e], e))
        ids.append(order[:topk])
    return ids


def weights(logits, ids, score, renorm, scale):
    """Weights [T, K] in 64 bits (differentiable in logits); ids a tensor."""
    lc = logits.gather(1, ids)
    if score == "sigmoid":
        s = torch.sigmoid(lc)
        if renorm:
            # logits far below zero keep their proportions
            down = lc.detach().amax(1, keepdim=True).clamp_max(0.0)
            down = torch.where(torch.isinf(down), torch.zeros_like(down), down)
            s = torch.exp(lc - down) / (1.0 + torch.exp(lc))
            big = lc > 0
            s = torch.where(big, 1.0 / (1.0 + torch.exp(-lc.abs())), s)  # down is 0 then
    else:
        over = lc if renorm else logits
        m = over.detach().amax(1, keepdim=True)
        m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
        s = torch.exp(lc - m)
        if not renorm:
            total = torch.exp(logits - m).sum(1, keepdim=True)
            s = torch.where(total > 0, s / total.clamp_min(1e-300), torch.zeros_like(s))
    if renorm:
        total = s.sum(1, keepdim=True)
        s = torch.where(total > 0, s / total.clamp_min(1e-300), torch.zeros_like(s))
    return scale * s


# --------------------------------------------------- norms around a block --
def block(x, y, post, gate, pre, scale, eps):
    """(out, u) in 64 bits; gate [H] or [T, 1]."""
    out = x
    if y is not None:
        z = y
        if post is not None:
            z = y / torch.sqrt(y.square().mean(1, keepdim=True) + eps) * post
        out = x + scale * (z if gate is None else gate * z)
    u = None
    if pre is not None:
        u = out / torch.sqrt(out.square().mean(1, keepdim=True) + eps) * pre
    return out, u
