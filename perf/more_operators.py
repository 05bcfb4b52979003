"""Experts in 8-bit integers and the layer for a few tokens, case by case: what
a case's inputs are, its plain form in elementary torch operations, and the
calls a user makes.

    product   y = xs ws (xq wq^T) of 8-bit rows grouped by expert
    rows      16-bit rows to 8 bits, then that product
    act       silu(gate) * up to 8 bits, then the down product
    few       the whole layer (SwiGLU experts, weighted sum) for a few tokens

`own` False: the plain forms (32 bits, rounded once at the end); True: the
library's kernels.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "int8": 1}


def listed():
    return [
        # one decoding step of 256 tokens through 8-bit down weights
        # (DeepSeek-V3-shaped): about 8 rows an expert, every weight is read
        dict(name="product_decode", op="product", out="bf16", groups=256, rows=2048, n=7168, k=2048,
             skew=0.1),
        # a prompt's rows through few large experts (Mixtral-shaped)
        dict(name="product_prompt", op="product", out="bf16", groups=8, rows=8192, n=4096, k=14336,
             skew=0.1),
        # uneven popularity, sizes that fill no tile and rows that are not
        # whole 16 bytes, results in 32 bits
        dict(name="product_uneven", op="product", out="fp32", groups=37, rows=5003, n=1000, k=1416,
             skew=1.0),
        # a dense projection of a prompt (one group): rows quantised first
        dict(name="rows_dense", op="rows", dtype="bf16", out="bf16", groups=1, rows=8192, n=4096,
             k=7168, skew=0.1),
        # the small parity layer's gate and up product: latency
        dict(name="rows_small", op="rows", dtype="fp16", out="fp16", groups=8, rows=128, n=1024,
             k=256, skew=0.5),
        # the down product of a prompt of 8192 tokens, top-8 of 256 experts,
        # from the gate and up product's rows
        dict(name="act_prompt", op="act", dtype="bf16", out="bf16", groups=256, rows=65536, n=7168,
             k=2048, skew=0.1),
        # ... of 16 tokens, top-2 of 8 experts (Mixtral-shaped)
        dict(name="act_decode", op="act", dtype="bf16", out="bf16", groups=8, rows=32, n=4096,
             k=14336, skew=0.1),
        # the layer for one token: 8 experts' weights out of 256
        dict(name="few_one", op="few", dtype="bf16", wdtype="bf16", tokens=1, hidden=7168,
             inter=2048, experts=256, topk=8, masked=0.0),
        # ... for a small batch of streams, weights in 8 bits
        dict(name="few_batch", op="few", dtype="bf16", wdtype="int8", tokens=16, hidden=7168,
             inter=2048, experts=256, topk=8, masked=0.0),
        # few large experts, the most tokens: every weight is read
        dict(name="few_large", op="few", dtype="bf16", wdtype="bf16", tokens=64, hidden=4096,
             inter=14336, experts=8, topk=2, masked=0.0),
        # the small parity layer: latency
        dict(name="few_small", op="few", dtype="fp16", wdtype="fp16", tokens=4, hidden=256,
             inter=512, experts=8, topk=2, masked=0.0),
        # sizes that fill no vector, a padded batch (pairs without an expert)
        dict(name="few_uneven", op="few", dtype="bf16", wdtype="int8", tokens=33, hidden=1001,
             inter=1419, experts=37, topk=3, masked=0.2),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["product", "product", "rows", "act", "few", "few", "few"])
    if op == "few":
        dtype = rng.choice(["bf16", "bf16", "fp16"])
        c = dict(op=op, dtype=dtype, wdtype=rng.choice([dtype, "int8"]), tokens=_log(rng, 1, 64))
        while True:
            c["experts"] = _log(rng, 1, 256)
            c["hidden"], c["inter"] = _log(rng, 64, 7168), _log(rng, 64, 14336)
            if rng.random() < 0.75:  # rows of whole 16 bytes are the usual case
                c["hidden"], c["inter"] = (max(64, v // 16 * 16) for v in (c["hidden"], c["inter"]))
            if c["experts"] * c["hidden"] * c["inter"] <= 2 ** 30:
                break
        c["topk"] = rng.randint(1, min(8, c["experts"]))
        c["masked"] = rng.choice([0.0, 0.0, 0.2])
        return c
    c = dict(op=op, out=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    if op != "product":
        c["dtype"] = rng.choice(["bf16", "bf16", "fp16"])
        if op == "act":
            c["out"] = c["dtype"]
    while True:
        c["groups"], c["rows"] = _log(rng, 1, 256), _log(rng, 1, 65536)
        c["n"], c["k"] = _log(rng, 64, 14336), _log(rng, 64, 14336)
        if rng.random() < 0.75:
            c["n"], c["k"] = max(64, c["n"] // 16 * 16), max(64, c["k"] // 16 * 16)
        c["skew"] = rng.choice([0.1, 0.5, 1.0])
        if c["groups"] * c["n"] * c["k"] <= 2 ** 30 and \
           2.0 * c["rows"] * c["n"] * c["k"] <= 1e12 and \
           c["rows"] * (c["n"] + 3 * c["k"]) * math.exp(3 * c["skew"]) <= 2e9:
            return c


# ----------------------------------------------------------------- inputs --
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1_000_003 + 29)
    return g


def _pieces(t, fill):
    """fill(n) for the whole of t, in pieces, so that no 32-bit copy of it is
    made."""
    flat, step = t.view(-1), 1 << 28
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = fill(n)
    return t


def _randn(shape, dtype, g, std=1.0):
    t = torch.empty(shape, dtype=_DT[dtype], device="cuda")
    return _pieces(t, lambda n: torch.randn(n, generator=g, device="cuda").mul_(std))


def _codes(shape, g):
    """8-bit values as a quantised normal distribution has them: the largest
    of a row at 127 is about four standard deviations."""
    t = torch.empty(shape, dtype=torch.int8, device="cuda")
    return _pieces(t, lambda n: torch.randn(n, generator=g, device="cuda").mul_(32.0).round_()
                   .clamp_(-127, 127))


def _scales(shape, g, std):
    """Scales of such values for a standard deviation of about `std`."""
    return (0.75 + 0.5 * torch.rand(shape, generator=g, device="cuda")) * (std / 32.0)


def _group_sizes(case, seed):
    """Rows per group: popularity exp(skew * N(0, 1)), each row's group drawn
    from it; the groups follow one another and cover every row."""
    g = torch.Generator()
    g.manual_seed(seed * 7919 + 11)
    p = torch.exp(case["skew"] * torch.randn(case["groups"], generator=g, dtype=torch.float64))
    pick = torch.multinomial(p, case["rows"], replacement=True, generator=g)
    return torch.bincount(pick, minlength=case["groups"])


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case=case)
    if case["op"] == "few":
        t, h, i, e, k = (case[n] for n in ("tokens", "hidden", "inter", "experts", "topk"))
        st["x"] = _randn((t, h), case["dtype"], g)
        # distinct experts a token, uneven popularity; weights sum to one
        logits = torch.randn((t, e), generator=g, device="cuda") + \
            0.5 * torch.randn(e, generator=g, device="cuda")
        top, idx = logits.topk(k, dim=1)
        w = torch.sigmoid(top)
        w = w / w.sum(1, keepdim=True)
        gone = torch.rand((t, k), generator=g, device="cuda") < case["masked"]
        st["idx"] = idx.masked_fill(gone, -1).to(torch.int32)
        st["w"] = w.masked_fill(gone, 0.0)
        st["s13"] = st["s2"] = None
        if case["wdtype"] == "int8":
            st["w13"], st["w2"] = _codes((e, 2 * i, h), g), _codes((e, h, i), g)
            st["s13"], st["s2"] = _scales((e, 2 * i), g, 0.02), _scales((e, h), g, 0.02)
        else:
            st["w13"] = _randn((e, 2 * i, h), case["wdtype"], g, 0.02)
            st["w2"] = _randn((e, h, i), case["wdtype"], g, 0.02)
        return st
    count = _group_sizes(case, seed)
    st["most"] = int(count.max())
    st["first"] = (torch.cumsum(count, 0) - count).to(torch.int32).cuda()
    st["count"] = count.to(torch.int32).cuda()
    r, n, k, e = case["rows"], case["n"], case["k"], case["groups"]
    st["wq"], st["ws"] = _codes((e, n, k), g), _scales((e, n), g, 0.02)
    if case["op"] == "product":
        st["xq"], st["xs"] = _codes((r, k), g), _scales((r,), g, 1.0)
    else:
        st["x"] = _randn((r, k if case["op"] == "rows" else 2 * k), case["dtype"], g)
    st["out"] = torch.empty((r, n), dtype=_DT[case["out"]], device="cuda")
    return st


# ------------------------------------------------------------- the passes --
def run(st):
    return _run_own(st["case"], st) if own else _run_plain(st["case"], st)


def _run_own(case, st):
    import combine_symmetric_memory_amd as cco
    if case["op"] == "few":
        return cco.moe_few(st["x"], st["idx"], st["w"], st["w13"], st["w2"], s13=st["s13"],
                           s2=st["s2"])
    if case["op"] == "product":
        xq, xs = st["xq"], st["xs"]
    elif case["op"] == "rows":
        xq, xs = cco.quant_rows(st["x"])
    else:
        xq, xs = cco.quant_swiglu(st["x"])
    return cco.group_product_i8(st["first"], st["count"], xq, xs, st["wq"], st["ws"],
                                out=st["out"])


def _swiglu(v):
    gate, up = v.chunk(2, dim=-1)
    return gate / (1.0 + torch.exp(-gate)) * up


def _run_plain(case, st):
    if case["op"] == "few":
        return _plain_few(case, st)
    if case["op"] == "product":
        q, xs = st["xq"].float(), st["xs"]
    else:
        v = st["x"].float()
        if case["op"] == "act":
            v = _swiglu(v)
        most = v.abs().amax(1, keepdim=True)
        q = torch.round(127.0 * v / most.clamp_min(1e-30))
        xs = most[:, 0] / 127.0
    # the rows of every group side by side, padded to the longest group's
    at = torch.arange(case["rows"], device="cuda")
    gid = torch.searchsorted(st["first"] + st["count"], at.to(torch.int32), right=True)
    pos = at - st["first"][gid]
    a = torch.zeros((case["groups"], st["most"], case["k"]), device="cuda")
    a[gid, pos] = q
    y = torch.bmm(st["wq"].float(), a.transpose(1, 2).contiguous())
    st["out"].copy_(y[gid, :, pos] * xs[:, None] * st["ws"][gid])
    return st["out"]


def _plain_few(case, st):
    x, idx = st["x"].float(), st["idx"].long()
    here = idx >= 0
    t, k, e, h = case["tokens"], case["topk"], case["experts"], case["hidden"]
    weights = [(st["w13"], st["s13"]), (st["w2"], st["s2"])]

    def product(a, which, ids):
        """a [b, rows, columns] by the experts' matrices, all or those of ids"""
        m, s = weights[which]
        m = m if ids is None else m[ids]
        y = torch.bmm(m.float(), a.transpose(1, 2).contiguous()).transpose(1, 2)
        return y if s is None else y * (s if ids is None else s[ids])[:, None, :]

    if t * k <= e:
        # every pair's matrices
        ids = idx.clamp_min(0).flatten()
        a = x[:, None, :].expand(t, k, h).reshape(t * k, 1, h)
        y = product(_swiglu(product(a, 0, ids)), 1, ids).view(t, k, h)
        y = torch.where(here[:, :, None], y * st["w"][:, :, None], torch.zeros_like(y))
        return y.sum(1).to(st["x"].dtype)
    # every token by every expert, weighted by what the token gives it
    share = torch.zeros((t, e), device="cuda")
    share.scatter_add_(1, idx.clamp_min(0), torch.where(here, st["w"], torch.zeros_like(st["w"])))
    y = product(_swiglu(product(x.expand(e, t, h), 0, None)), 1, None)
    return (y * share.t()[:, :, None]).sum(0).to(st["x"].dtype)


# --------------------------------------------------------- in 64 bits -------
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "few":
        return _exact_few(case, st)
    if case["op"] == "product":
        q, xs = st["xq"].double(), st["xs"].double()
    else:
        v = st["x"].double()
        if case["op"] == "act":
            v = torch.nn.functional.silu(v[:, :case["k"]]) * v[:, case["k"]:]
        most = v.abs().max(dim=1).values
        q = torch.round(v * 127 / torch.where(most > 0, most, torch.ones_like(most))[:, None])
        xs = most / 127
    y = torch.empty((case["rows"], case["n"]), dtype=torch.float64, device="cuda")
    lo = 0
    for e, c in enumerate(st["count"].tolist()):
        rows = slice(lo, lo + c)
        if c:
            y[rows] = (q[rows] @ st["wq"][e].double().t().contiguous()) * st["ws"][e].double()
        lo += c
    return y * xs[:, None]


def _exact_few(case, st):
    out = torch.zeros((case["tokens"], case["hidden"]), dtype=torch.float64, device="cuda")
    for e in torch.unique(st["idx"][st["idx"] >= 0]).tolist():
        rows, cols = (st["idx"] == e).nonzero(as_tuple=True)
        w13, w2 = st["w13"][e].double(), st["w2"][e].double()
        if st["s13"] is not None:
            w13, w2 = w13 * st["s13"][e].double()[:, None], w2 * st["s2"][e].double()[:, None]
        gu = st["x"][rows].double() @ w13.t().contiguous()
        i = case["inter"]
        y = (torch.nn.functional.silu(gu[:, :i]) * gu[:, i:]) @ w2.t().contiguous()
        out.index_add_(0, rows, y * st["w"][rows, cols].double()[:, None])
    return out


# ------------------------------------------------------------- the floors --
def work(case):
    if case["op"] == "few":
        t, h, i, e, k = (case[n] for n in ("tokens", "hidden", "inter", "experts", "topk"))
        pairs = t * k * (1.0 - case["masked"])
        # experts that some pair has, as if all were as likely
        live = e * (1.0 - (1.0 - 1.0 / e) ** pairs) if t > 1 else min(e, pairs)
        b = live * (3 * h * i * _SIZE[case["wdtype"]] +
                    (4 * (2 * i + h) if case["wdtype"] == "int8" else 0))
        return dict(bytes=int(b + t * (4 * h + 8 * k)), flops=int(6 * pairs * h * i))
    r, n, k, e = case["rows"], case["n"], case["k"], case["groups"]
    b = min(e, r) * n * (k + 4) + r * n * _SIZE[case["out"]]
    b += r * (k + 4 if case["op"] == "product" else (2 if case["op"] == "rows" else 4) * k)
    return dict(bytes=b, flops=2 * r * n * k)
