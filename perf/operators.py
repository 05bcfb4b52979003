"""The operators around the MoE path, case by case: what a case's inputs are,
its plain form in elementary torch operations, and the call a user makes.

    group_product   y = x W^T, dx = dy W, dW = dy^T x over rows grouped by expert
    route           choice of experts and their weights, with the gradient
    block_norm      norm after a block, gate, residual, norm before the next,
                    with the gradient

`own` False: the plain forms (32 bits, rounded once at the end); True: the
library's kernels.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # a training batch through the experts' gate and up weights
        # (DeepSeek-V3-shaped: 8192 tokens, top-8 of 256 experts)
        dict(name="product_train", op="product", dtype="bf16", groups=256, rows=65536, n=4096,
             k=7168, skew=0.1),
        # one decoding step of 256 tokens through the down weights: about
        # 8 rows per expert, every expert's weights are read
        dict(name="product_decode", op="product", dtype="bf16", groups=256, rows=2048, n=7168,
             k=2048, skew=0.1),
        # the small parity layer, half precision: latency
        dict(name="product_small", op="product", dtype="fp16", groups=8, rows=256, n=1024, k=256,
             skew=0.5),
        # gradient of the down product's rows, the same training batch
        dict(name="dx_train", op="dx", dtype="bf16", groups=256, rows=65536, n=7168, k=2048,
             skew=0.1),
        # gradient of the down weights, few large experts (Mixtral-shaped),
        # kept in 32 bits as an optimizer wants it
        dict(name="dw_train", op="dw", dtype="bf16", groups=8, rows=8192, n=4096, k=14336,
             skew=0.1, out="fp32"),
        # weight gradient of fine-grained experts with uneven popularity
        # (some get no rows), sizes that fill no tile
        dict(name="dw_uneven", op="dw", dtype="bf16", groups=37, rows=5003, n=1000, k=1416,
             skew=2.0, out="bf16"),
        # routing of one decoding step: sigmoid scores, balancing bias,
        # choice limited to 4 of 8 groups of experts
        dict(name="route_decode", op="route", dtype="fp32", tokens=256, experts=256, topk=8,
             score="sigmoid", bias=True, renorm=True, scale=2.5, groups=8, kept=4),
        # routing of a training batch with its gradient: softmax scores
        dict(name="route_train", op="route_train", dtype="fp32", tokens=16384, experts=256, topk=8,
             score="softmax", bias=False, renorm=False, scale=1.0, groups=1, kept=1),
        # the norms around a block while decoding
        dict(name="norm_decode", op="norm", dtype="bf16", tokens=16, hidden=7168, post=True,
             pre=True, gate="none", wdtype="bf16"),
        # ... of a training batch, gated per channel
        dict(name="norm_train", op="norm", dtype="bf16", tokens=8192, hidden=7168, post=True,
             pre=True, gate="channel", wdtype="fp32"),
        # ... and their gradient
        dict(name="norm_grad_train", op="norm_grad", dtype="bf16", tokens=8192, hidden=7168,
             post=True, pre=True, gate="channel", wdtype="fp32"),
        # a width that fills no vector group, gated per token, without the
        # norm after the block
        dict(name="norm_grad_uneven", op="norm_grad", dtype="fp16", tokens=1237, hidden=4999,
             post=False, pre=True, gate="token", wdtype="fp32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["product", "dx", "dw", "product", "dx", "dw", "route", "route_train", "norm",
                     "norm_grad"])
    if op in ("product", "dx", "dw"):
        c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp16"]))
        while True:
            c["groups"] = _log(rng, 1, 256)
            c["rows"] = _log(rng, 1, 65536)
            c["n"], c["k"] = _log(rng, 64, 14336), _log(rng, 64, 14336)
            if rng.random() < 0.75:  # rows of whole 16 bytes are the usual case
                c["n"], c["k"] = max(8, c["n"] // 8 * 8), max(8, c["k"] // 8 * 8)
            w = c["groups"] * c["n"] * c["k"]
            if w <= 2 ** 30 and 2.0 * c["rows"] * c["n"] * c["k"] <= 2e12:
                break
        c["skew"] = rng.choice([0.1, 0.5, 1.0, 2.0])
        if op == "dw":
            c["out"] = rng.choice(["fp32", "same"])
            if c["out"] == "same":
                c["out"] = c["dtype"]
        return c
    if op in ("route", "route_train"):
        groups = rng.choice([1, 1, 2, 4, 8])
        if groups == 1:
            experts = rng.randint(2, 512)
        else:
            experts = groups * rng.randint(2, 512 // groups)
        kept = rng.randint(1, groups)
        topk = rng.randint(1, min(16, kept * (experts // groups)))
        score = rng.choice(["softmax", "sigmoid"])
        return dict(op=op, dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]),
                    tokens=_log(rng, 1, 16384), experts=experts, topk=topk, score=score,
                    bias=rng.random() < 0.5, renorm=rng.random() < 0.6,
                    scale=rng.choice([1.0, 2.5]), groups=groups, kept=kept)
    post, pre = rng.choice([(True, True), (True, True), (False, True), (True, False)])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    hidden = _log(rng, 32, 8192)
    if rng.random() < 0.6:
        hidden = max(32, hidden // 8 * 8)
    return dict(op=op, dtype=dtype, tokens=_log(rng, 1, 8192 if dtype != "fp32" else 4096),
                hidden=hidden, post=post, pre=pre, gate=rng.choice(["none", "channel", "token"]),
                wdtype=rng.choice(["fp32", dtype]))


# ----------------------------------------------------------------- inputs --
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1_000_003 + 17)
    return g


def _randn(shape, dtype, g, std=1.0):
    t = torch.empty(shape, dtype=_DT[dtype], device="cuda")
    # large tensors in pieces, so that no 32-bit copy of the whole is made
    flat = t.view(-1)
    step = 1 << 28
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=g, device="cuda") * std
    return t


def _group_sizes(case, seed):
    """Rows per group: popularity exp(skew * N(0, 1)), each row's group drawn
    from it; the groups follow one another and cover every row."""
    g = torch.Generator()
    g.manual_seed(seed * 7919 + 5)
    p = torch.exp(case["skew"] * torch.randn(case["groups"], generator=g, dtype=torch.float64))
    pick = torch.multinomial(p, case["rows"], replacement=True, generator=g)
    return torch.bincount(pick, minlength=case["groups"])


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case=case)
    op = case["op"]
    if op in ("product", "dx", "dw"):
        count = _group_sizes(case, seed)
        first = torch.cumsum(count, 0) - count
        st["sizes"] = [int(c) for c in count]
        st["first"] = first.to(torch.int32).cuda()
        st["count"] = count.to(torch.int32).cuda()
        r, n, k, e, dt = case["rows"], case["n"], case["k"], case["groups"], case["dtype"]
        if op != "dx":
            st["x"] = _randn((r, k), dt, g)
        if op != "product":
            st["dy"] = _randn((r, n), dt, g)
        if op != "dw":
            st["w"] = _randn((e, n, k), dt, g, 0.02)
        shape = dict(product=(r, n), dx=(r, k), dw=(e, n, k))[op]
        st["out"] = torch.empty(shape, dtype=_DT[case.get("out", dt)], device="cuda")
    elif op in ("route", "route_train"):
        t, e, kk = case["tokens"], case["experts"], case["topk"]
        st["logits"] = _randn((t, e), case["dtype"], g)
        st["bias"] = torch.randn(e, generator=g, device="cuda") * 0.1 if case["bias"] else None
        if op == "route_train":
            st["dw"] = torch.randn((t, kk), generator=g, device="cuda")
    else:
        t, h, dt = case["tokens"], case["hidden"], case["dtype"]
        st["x"] = _randn((t, h), dt, g, 2.0)
        st["y"] = _randn((t, h), dt, g, 0.5)

        def weight():
            return (1.0 + 0.1 * torch.randn(h, generator=g, device="cuda")).to(_DT[case["wdtype"]])

        st["post"] = weight() if case["post"] else None
        st["pre"] = weight() if case["pre"] else None
        st["gate"] = None
        if case["gate"] == "channel":
            st["gate"] = (0.5 + 0.1 * torch.randn(h, generator=g, device="cuda")
                          ).to(_DT[case["wdtype"]])
        elif case["gate"] == "token":
            st["gate"] = torch.rand(t, generator=g, device="cuda")
        if op == "norm_grad":
            st["dout"] = _randn((t, h), dt, g)
            st["du"] = _randn((t, h), dt, g) if case["pre"] else None
    return st


_EPS, _SCALE = 1e-6, 0.7


# ------------------------------------------------------------- the passes --
def run(st):
    case = st["case"]
    return (_run_own if own else _run_plain)(case["op"], case, st)


def _run_own(op, case, st):
    import combine_symmetric_memory_amd as cco
    if op == "product":
        return cco.group_product(st["first"], st["count"], st["x"], st["w"], out=st["out"])
    if op == "dx":
        return cco.group_product_dx(st["first"], st["count"], st["dy"], st["w"], out=st["out"])
    if op == "dw":
        return cco.group_product_dw(st["first"], st["count"], st["dy"], st["x"], out=st["out"])
    if op in ("route", "route_train"):
        kw = dict(score=case["score"], renorm=case["renorm"], scale=case["scale"])
        idx, w = cco.route(st["logits"], case["topk"], bias=st["bias"], groups=case["groups"],
                           kept=case["kept"], **kw)
        if op == "route":
            return idx, w
        return idx, w, cco.route_grad(st["logits"], idx, st["dw"], **kw)
    kw = dict(post=st["post"], pre=st["pre"], scale=_SCALE, eps=_EPS)
    if case["gate"] != "none":
        kw["gate" if case["gate"] == "channel" else "token_gate"] = st["gate"]
    if op == "norm":
        out, u = cco.block_norm(st["x"], st["y"], **kw)
        return [t for t in (out, u) if t is not None]
    d = cco.block_norm_grad(st["x"], st["y"], st["dout"], st["du"], **kw)
    return [t for t in d if t is not None]


def _run_plain(op, case, st):
    if op in ("product", "dx", "dw"):
        out = torch.empty_like(st["out"])
        lo = 0
        for e, c in enumerate(st["sizes"]):
            hi = lo + c
            if op == "dw":
                out[e] = torch.mm(st["dy"][lo:hi].float().t(), st["x"][lo:hi].float())
            elif c:
                w = st["w"][e].float()
                a = (st["x"] if op == "product" else st["dy"])[lo:hi].float()
                out[lo:hi] = torch.mm(a, w.t() if op == "product" else w)
            lo = hi
        return out
    if op in ("route", "route_train"):
        idx = _plain_choice(case, st)
        lc = torch.gather(st["logits"].float(), 1, idx.long())
        s, total = _plain_scores(case, st["logits"].float(), lc)
        w = case["scale"] * (s / total if case["renorm"] else s)
        if op == "route":
            return idx, w
        return idx, w, _plain_route_grad(case, st, idx, s, total)
    if op == "norm":
        f = _plain_norm(case, st)
        dt = _DT[case["dtype"]]
        return [f["out"].to(dt)] + ([f["u"].to(dt)] if case["pre"] else [])
    return _plain_norm_grad(case, st)


def _plain_choice(case, st):
    """The K ids in descending order of choice, ties to the lower id."""
    l = st["logits"].float()
    t, e = l.shape
    if case["bias"] or case["groups"] > 1:
        l = l.double()  # values next to a border
        if case["score"] == "softmax":
            s = torch.exp(l - l.amax(1, keepdim=True))
            c = s / s.sum(1, keepdim=True)
        else:
            c = 1.0 / (1.0 + torch.exp(-l))
        if case["bias"]:
            c = c + st["bias"].double()
    else:
        c = l
    ids = torch.arange(e, device=l.device)
    low = torch.full((), -math.inf, dtype=c.dtype, device=c.device)

    def best(v, n):  # position of the first largest value
        at = torch.arange(n, device=v.device)
        return torch.where(v == v.amax(-1, keepdim=True), at, n).amin(-1)

    if case["groups"] > 1:
        ng, per = case["groups"], e // case["groups"]
        v = c.view(t, ng, per)
        one = v.amax(-1)
        two = torch.where(torch.arange(per, device=v.device) == best(v, per).unsqueeze(-1), low, v)
        score = one + two.amax(-1) if per > 1 else one
        keep = torch.zeros((t, ng), dtype=torch.bool, device=v.device)
        for _ in range(case["kept"]):
            j = best(score, ng)
            hit = torch.arange(ng, device=v.device) == j.unsqueeze(1)
            keep |= hit
            score = torch.where(hit, low, score)
        c = torch.where(keep.unsqueeze(2), v, low).reshape(t, e)
    idx = torch.empty((t, case["topk"]), dtype=torch.int32, device=l.device)
    for j in range(case["topk"]):
        b = best(c, e)
        idx[:, j] = b
        c = torch.where(ids == b.unsqueeze(1), low, c)
    return idx


def _plain_scores(case, l, lc):
    if case["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-lc))
        return s, s.sum(1, keepdim=True)
    m = lc.amax(1, keepdim=True) if case["renorm"] else l.amax(1, keepdim=True)
    s = torch.exp(lc - m)
    if case["renorm"]:
        return s, s.sum(1, keepdim=True)
    return s / torch.exp(l - m).sum(1, keepdim=True), None


def _plain_route_grad(case, st, idx, s, total):
    l, dw = st["logits"].float(), st["dw"]
    if case["renorm"]:
        q = s / total
        ds = case["scale"] * (dw - (dw * q).sum(1, keepdim=True)) / total  # to the scores s
    else:
        ds = case["scale"] * dw
    if case["score"] == "sigmoid":
        lc = torch.gather(l, 1, idx.long())
        part = ds * s * (1.0 / (1.0 + torch.exp(lc)))  # 1 - s without its cancellation
        return torch.zeros_like(l).scatter_(1, idx.long(), part).to(st["logits"].dtype)
    part = ds * s
    grad = torch.zeros_like(l).scatter_(1, idx.long(), part)
    if not case["renorm"]:
        p = torch.exp(l - l.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
        grad = grad - p * part.sum(1, keepdim=True)
    return grad.to(st["logits"].dtype)


def _plain_norm(case, st):
    x, y = st["x"].float(), st["y"].float()
    f = dict(x=x, y=y)
    z = y
    if case["post"]:
        f["ry"] = 1.0 / torch.sqrt((y * y).mean(1, keepdim=True) + _EPS)
        z = y * f["ry"] * st["post"].float()
    f["z"] = z
    gate = 1.0
    if case["gate"] == "channel":
        gate = st["gate"].float()
    elif case["gate"] == "token":
        gate = st["gate"].unsqueeze(1)
    f["gate"] = gate
    out = x + _SCALE * gate * z
    f["out"] = out
    if case["pre"]:
        f["ro"] = 1.0 / torch.sqrt((out * out).mean(1, keepdim=True) + _EPS)
        f["u"] = out * f["ro"] * st["pre"].float()
    return f


def _plain_norm_grad(case, st):
    """[dx, dy, dpost, dgate, dpre] (those that exist)."""
    f = _plain_norm(case, st)
    d = st["dout"].float()
    dpre = None
    if case["pre"]:
        du, o, r = st["du"].float(), f["out"], f["ro"]
        dpre = (du * o * r).sum(0)
        a = du * st["pre"].float()
        d = d + r * a - o * r ** 3 * (a * o).mean(1, keepdim=True)
    dgate = None
    if case["gate"] == "channel":
        dgate = (_SCALE * f["z"] * d).sum(0)
    elif case["gate"] == "token":
        dgate = (_SCALE * f["z"] * d).sum(1)
    dz = _SCALE * f["gate"] * d
    dy, dpost = dz, None
    if case["post"]:
        y, r = f["y"], f["ry"]
        dpost = (dz * y * r).sum(0)
        a = dz * st["post"].float()
        dy = r * a - y * r ** 3 * (a * y).mean(1, keepdim=True)
    dt = _DT[case["dtype"]]
    return [v for v in (d.to(dt), dy.to(dt), dpost, dgate, dpre) if v is not None]


# --------------------------------------------------------- in 64 bits -------
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("product", "dx", "dw"):
        return _exact_group(op, st)
    if op in ("route", "route_train"):
        return _exact_route(op, case, st)
    return _exact_norm(op, case, st)


def _exact_group(op, st):
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    ends = torch.cumsum(torch.tensor(st["sizes"]), 0).tolist()
    for e, end in enumerate(ends):
        rows = slice(end - st["sizes"][e], end)
        if st["sizes"][e] == 0:
            continue
        if op == "product":
            out[rows] = st["x"][rows].double() @ st["w"][e].double().transpose(0, 1).contiguous()
        elif op == "dx":
            out[rows] = st["dy"][rows].double() @ st["w"][e].double()
        else:
            out[e] = st["dy"][rows].double().transpose(0, 1).contiguous() @ st["x"][rows].double()
    return out


def _exact_route(op, case, st):
    l = st["logits"].double().requires_grad_(op == "route_train")
    t, e = l.shape
    score = torch.softmax(l, 1) if case["score"] == "softmax" else torch.sigmoid(l)
    with torch.no_grad():
        c = l.detach() if not (case["bias"] or case["groups"] > 1) else score.detach()
        if case["bias"]:
            c = c + st["bias"].double()
        if case["groups"] > 1:
            v = c.view(t, case["groups"], -1)
            gs = v.sort(dim=-1, descending=True).values[..., :2].sum(-1)
            order = gs.sort(dim=1, descending=True, stable=True).indices[:, :case["kept"]]
            keep = torch.zeros_like(gs).scatter_(1, order, 1.0) > 0
            c = v.masked_fill(~keep.unsqueeze(2), -math.inf).reshape(t, e)
        idx = c.sort(dim=1, descending=True, stable=True).indices[:, :case["topk"]]
    w = score.gather(1, idx)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = w * case["scale"]
    if op == "route":
        return idx.to(torch.int32), w
    grad, = torch.autograd.grad(w, l, st["dw"].double())
    return idx.to(torch.int32), w.detach(), grad


def _exact_norm(op, case, st):
    grad = op == "norm_grad"
    v = {n: st[n].double().requires_grad_(grad) for n in ("x", "y", "post", "gate", "pre")
         if st[n] is not None}

    def rms(t, weight):
        return t / torch.sqrt(t.square().mean(1, keepdim=True) + _EPS) * weight

    z = rms(v["y"], v["post"]) if case["post"] else v["y"]
    if case["gate"] == "channel":
        z = z * v["gate"]
    elif case["gate"] == "token":
        z = z * v["gate"][:, None]
    out = v["x"] + _SCALE * z
    u = rms(out, v["pre"]) if case["pre"] else None
    if not grad:
        return [out] + ([u] if u is not None else [])
    outs, ds = [out], [st["dout"].double()]
    if u is not None:
        outs.append(u)
        ds.append(st["du"].double())
    names = [n for n in ("x", "y", "post", "gate", "pre") if n in v]
    return list(torch.autograd.grad(outs, [v[n] for n in names], ds))


# ------------------------------------------------------------- the floors --
def work(case):
    op = case["op"]
    if op in ("product", "dx", "dw"):
        r, n, k, e = case["rows"], case["n"], case["k"], case["groups"]
        flops = 2 * r * n * k
        if op == "dw":
            size = 4 if case["out"] == "fp32" else 2
            return dict(bytes=r * (n + k) * 2 + e * n * k * size, flops=flops)
        return dict(bytes=r * (n + k) * 2 + min(e, r) * n * k * 2, flops=flops)
    size = 4 if case["dtype"] == "fp32" else 2
    if op in ("route", "route_train"):
        t, e, kk = case["tokens"], case["experts"], case["topk"]
        b, f = t * e * size + t * kk * 8, 4 * t * e
        if op == "route_train":
            b, f = b + t * e * size + t * kk * 4, 2 * f
        return dict(bytes=b, flops=f)
    t, h = case["tokens"], case["hidden"]
    if op == "norm":
        return dict(bytes=t * h * size * (4 if case["pre"] else 3), flops=10 * t * h)
    return dict(bytes=t * h * size * (6 if case["pre"] else 5), flops=30 * t * h)
