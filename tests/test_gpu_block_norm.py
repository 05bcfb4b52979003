"""The norms around a block (cco_block_norm and its gradient) and the fused
combine (cco_moe_combine_norm): against 64-bit forms with derived bounds,
every presence of post, gate and pre, widths that fill no vector, in place,
streams and graphs."""
import math

import pytest
import torch

from tests import ops_ref as ref
from tests.gpu_util import make_case, make_moe, say

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-5


@pytest.fixture(scope="module")
def cco():
    import combine_symmetric_memory_amd as m
    assert torch.cuda.is_available()
    return m


def _inputs(T, H, dtype, wdtype, post, gate, pre, y=True, seed=0):
    g = torch.Generator().manual_seed(seed)

    def r(shape, std, dt):
        return (torch.randn(shape, generator=g) * std).to(dt)

    d = dict(x=r((T, H), 2.0, dtype), y=r((T, H), 0.5, dtype) if y else None)
    d["post"] = (1 + r(H, 0.2, F32)).to(wdtype) if post else None
    d["pre"] = (1 + r(H, 0.2, F32)).to(wdtype) if pre else None
    d["gate"] = r(H, 1.0, wdtype) if gate == "channel" else None
    d["token_gate"] = r(T, 1.0, F32) if gate == "token" else None
    d["dout"] = r((T, H), 1.0, dtype)
    d["du"] = r((T, H), 1.0, dtype) if pre else None
    return d


def _kw(d, dev=True):
    names = ("post", "gate", "token_gate", "pre")
    return {n: (d[n].cuda() if dev else d[n]) for n in names if d[n] is not None}


def _c(t):
    return None if t is None else t.cuda()


def _ref(d, scale, grad):
    v = {n: d[n].double().requires_grad_(grad) for n in
         ("x", "y", "post", "gate", "token_gate", "pre") if d[n] is not None}
    gate = v.get("gate")
    if "token_gate" in v:
        gate = v["token_gate"][:, None]
    out, u = ref.block(v["x"], v.get("y"), v.get("post"), gate, v.get("pre"), scale, EPS)
    return v, out, u


# A row's sum of squares: at most 16 terms per thread in a chain, 6 + 16
# additions over the lanes and wavefronts: 40 U, and half of that for its
# root; the products around it a few U each.
ROW = 48 * ref.U


def _check(cco, T, H, dtype, wdtype=F32, post=True, gate="none", pre=True, y=True, scale=0.7,
           seed=0, use_dout=True):
    say("case: block_norm T=%d H=%d %s/%s post=%s gate=%s pre=%s y=%s" % (
        T, H, dtype, wdtype, post, gate, pre, y))
    d = _inputs(T, H, dtype, wdtype, post, gate, pre, y, seed)
    v, out, u = _ref(d, scale, True)
    kw = dict(_kw(d), scale=scale, eps=EPS)
    x, yy = d["x"].cuda(), _c(d["y"])
    o, uu = cco.block_norm(x, yy, **kw)
    o64 = out.detach()
    size = d["x"].double().abs() + (o64 - d["x"].double()).abs()  # |x| + |scale gate z|
    hs, sm = ref.half_step(dtype), ref.smallest(dtype)
    eo = ROW * size  # error of the unrounded out
    if y:
        ref.assert_within(o, o64, hs * o64.abs() + eo + sm, "out")
    else:
        assert o is None
    if pre:
        p = d["pre"].double().abs()
        r = 1 / torch.sqrt(o64.square().mean(1, keepdim=True) + EPS)
        # u = out r pre: out's error, and r's from the whole row's
        er = (o64.abs() * eo).mean(1, keepdim=True) * r ** 2
        bu = p * r * (eo + o64.abs() * (er + ROW))
        ref.assert_within(uu, u.detach(), hs * u.detach().abs() + bu + sm, "u")
    else:
        assert uu is None
    # gradient
    dout = d["dout"] if use_dout or not pre else None
    got = cco.block_norm_grad(x, yy, _c(dout), _c(d["du"]), **kw)
    outs = [out] if dout is not None else []
    gs = [dout.double()] if dout is not None else []
    if pre:
        outs.append(u)
        gs.append(d["du"].double())
    names = [n for n in ("x", "y", "post", "gate", "token_gate", "pre") if n in v]
    want = dict(zip(names, torch.autograd.grad(outs, [v[n] for n in names], gs)))
    # sizes of the terms, everything in absolute values
    ad = torch.zeros_like(o64) if dout is None else dout.double().abs()
    a_o = size
    if pre:
        q = (d["du"].double() * d["pre"].double()).abs()
        ad = ad + r * q + r ** 3 * a_o * (q * a_o).mean(1, keepdim=True)
    ge = torch.ones_like(o64)
    if gate == "channel":
        ge = d["gate"].double().abs().expand_as(o64)
    elif gate == "token":
        ge = d["token_gate"].double().abs()[:, None].expand_as(o64)
    E = 4 * ROW  # out twice, r, q, the sums
    ref.assert_within(got[0], want["x"], hs * want["x"].abs() + E * ad + sm, "dx")
    if not y:
        assert got[1] is None
    else:
        ay = d["y"].double().abs()
        adz = abs(scale) * ge * ad
        ady, z, bz = adz, ay, adz
        if post:
            ry = 1 / torch.sqrt(d["y"].double().square().mean(1, keepdim=True) + EPS)
            bz = adz * d["post"].double().abs()
            ady = ry * bz + ay * ry ** 3 * (bz * ay).mean(1, keepdim=True)
            z = ay * ry * d["post"].double().abs()
            chain = (T / 64 + 40) * ref.U
            ref.assert_within(got[2], want["post"],
                              (2 * E + chain) * (adz * ay * ry).sum(0), "dpost")
        ref.assert_within(got[1], want["y"], hs * want["y"].abs() + 2 * E * ady + sm, "dy")
        if gate == "channel":
            chain = (T / 64 + 40) * ref.U
            ref.assert_within(got[3], want["gate"], (2 * E + chain) * (abs(scale) * z * ad).sum(0),
                              "dgate")
        elif gate == "token":
            ref.assert_within(got[3], want["token_gate"], 2 * E * (abs(scale) * z * ad).sum(1),
                              "dgate")
    if pre:
        chain = (T / 64 + 40) * ref.U
        ref.assert_within(got[4], want["pre"],
                          (2 * E + chain) * (d["du"].double().abs() * a_o * r).sum(0), "dpre")


FORMS = [(True, "none", True), (True, "channel", True), (True, "token", True),
         (False, "none", True), (False, "channel", False), (False, "token", True),
         (True, "channel", False), (False, "none", False), (True, "token", False)]


@pytest.mark.parametrize("post,gate,pre", FORMS)
@pytest.mark.parametrize("dtype,wdtype", [(BF, F32), (BF, BF), (HF, HF), (F32, F32)])
def test_forms(cco, post, gate, pre, dtype, wdtype):
    _check(cco, 19, 520, dtype, wdtype, post, gate, pre)
    _check(cco, 5, 77, dtype, wdtype, post, gate, pre)


@pytest.mark.parametrize("H", [1, 2, 7, 8, 64, 72, 511, 512, 513, 1024, 1025, 2048, 4095, 4096,
                               4104, 7168, 8191, 8192, 8200, 9999, 16383, 16384])
def test_widths(cco, H):
    _check(cco, 3, H, BF, F32, True, "channel", True)
    _check(cco, 2, H, HF, F32, False, "token", True)
    _check(cco, 2, H, F32, F32, True, "token", True)


@pytest.mark.parametrize("T", [1, 2, 255, 256, 257, 700, 2049, 5000])
def test_lengths(cco, T):
    _check(cco, T, 264, BF, F32, True, "channel", True)
    _check(cco, T, 33, BF, F32, True, "token", True)


def test_pre_norm_alone(cco):
    for H in (256, 4999, 7168):
        _check(cco, 9, H, BF, BF, False, "none", True, y=False)
        _check(cco, 300, H, BF, F32, False, "none", True, y=False, use_dout=False)


def test_du_alone_and_scale_signs(cco):
    _check(cco, 40, 512, BF, F32, True, "channel", True, use_dout=False)
    _check(cco, 40, 512, BF, F32, True, "channel", True, scale=-1.5)
    _check(cco, 40, 512, BF, F32, True, "channel", True, scale=0.0)


def test_no_tokens(cco):
    z = torch.empty((0, 64), dtype=BF, device="cuda")
    w = torch.ones(64, device="cuda")
    out, u = cco.block_norm(z, z, post=w, pre=w, gate=w)
    assert out.shape == (0, 64) and u.shape == (0, 64)
    dx, dy, dp, dg, dq = cco.block_norm_grad(z, z, z, z, post=w, pre=w, gate=w)
    assert not dp.any() and not dg.any() and not dq.any()
    tg = torch.empty(0, device="cuda")
    assert cco.block_norm_grad(z, z, z, z, post=w, pre=w, token_gate=tg)[3].shape == (0,)


def test_out_alone_is_optional(cco):
    # through the C entry: u without out
    from combine_symmetric_memory_amd import _capi
    import ctypes
    d = _inputs(6, 264, BF, F32, True, "none", True)
    x, y, post, pre = (d[n].cuda() for n in ("x", "y", "post", "pre"))
    o, u = cco.block_norm(x, y, post=post, pre=pre, eps=EPS)
    desc = _capi.cco_block_norm_desc(264, _capi.CCO_BF16, _capi.CCO_F32, 0, 1.0, EPS,
                                     post.data_ptr(), None, pre.data_ptr())
    u2 = torch.empty_like(u)
    assert _capi.lib.cco_block_norm(ctypes.byref(desc), x.data_ptr(), y.data_ptr(), 6, None,
                                    u2.data_ptr(), None) == 0
    torch.cuda.synchronize()
    assert torch.equal(u, u2)


@pytest.mark.parametrize("H", [520, 77, 8200])
def test_in_place(cco, H):
    d = _inputs(30, H, BF, F32, True, "channel", True)
    kw = dict(_kw(d), scale=0.7, eps=EPS)
    x, y, dout, du = (d[n].cuda() for n in ("x", "y", "dout", "du"))
    o, u = cco.block_norm(x, y, **kw)
    want = cco.block_norm_grad(x, y, dout, du, **kw)
    x2, y2 = x.clone(), y.clone()
    cco.block_norm(x2, y2, out=x2, u=y2, **kw)
    assert torch.equal(x2, o) and torch.equal(y2, u)
    for a, b in ((dout.clone(), du.clone()),):
        got = cco.block_norm_grad(x, y, a, b, dx=a, dy=b, **kw)
        for g, w in zip(got, want):
            assert torch.equal(g, w)
    x2, y2 = x.clone(), y.clone()
    got = cco.block_norm_grad(x2, y2, dout, du, dx=x2, dy=y2, **kw)
    for g, w in zip(got, want):
        assert torch.equal(g, w)


def test_unaligned_rows_and_vectors(cco):
    # pointers aligned to an element only
    d = _inputs(12, 264, BF, BF, True, "channel", True)

    def odd(t):
        b = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        b[1:] = t.flatten()
        return b[1:].view(t.shape)

    kw = dict(scale=0.7, eps=EPS)
    base = cco.block_norm(d["x"].cuda(), d["y"].cuda(), **_kw(d), **kw)
    bg = cco.block_norm_grad(d["x"].cuda(), d["y"].cuda(), d["dout"].cuda(), d["du"].cuda(),
                             **_kw(d), **kw)
    po = {n: odd(t.cuda()) for n, t in _kw(d).items()}
    # only the vectors: the same kernel, the same bits
    got = cco.block_norm(d["x"].cuda(), d["y"].cuda(), **po, **kw)
    for a, b in zip(got, base):
        assert torch.equal(a, b)
    got = cco.block_norm(odd(d["x"].cuda()), odd(d["y"].cuda()), **po, **kw)
    for a, b in zip(got, base):  # another order of addition: one step of bf16
        assert bool(((a.float() - b.float()).abs() <= 2.0 ** -7 * b.float().abs() + 1e-6).all())
    gg = cco.block_norm_grad(odd(d["x"].cuda()), odd(d["y"].cuda()), odd(d["dout"].cuda()),
                             odd(d["du"].cuda()), **po, **kw)
    for a, b in zip(gg, bg):
        assert bool(((a.float() - b.float()).abs() <=
                     2.0 ** -7 * b.float().abs() + 1e-4).all())


def test_bad_rows_stay_alone(cco):
    d = _inputs(8, 520, BF, F32, True, "token", True)
    x, y = d["x"].cuda(), d["y"].cuda()
    x[2, 5] = math.inf
    y[4, 7] = math.nan
    y[5] = 0
    x[6] = 0
    y[6] = 0
    kw = dict(_kw(d), scale=0.7, eps=EPS)
    out, u = cco.block_norm(x, y, **kw)
    dx, dy = cco.block_norm_grad(x, y, d["dout"].cuda(), d["du"].cuda(), **kw)[:2]
    good = [0, 1, 3, 5, 6, 7]
    for t in (out, u, dx, dy):
        assert torch.isfinite(t[good]).all()
    assert not out[6].any() and not u[6].any()
    assert torch.isnan(out[4]).all() and torch.isnan(u[2]).any()


def test_gradient_against_differences(cco):
    d = _inputs(3, 24, F32, F32, True, "channel", True)
    kw = dict(_kw(d), scale=0.7, eps=EPS)
    got = cco.block_norm_grad(d["x"].cuda(), d["y"].cuda(), d["dout"].cuda(), d["du"].cuda(), **kw)

    def loss(v):
        out, u = ref.block(v["x"], v["y"], v["post"], v["gate"], v["pre"], 0.7, EPS)
        return float((out * d["dout"].double()).sum() + (u * d["du"].double()).sum())

    base = {n: d[n].double() for n in ("x", "y", "post", "gate", "pre")}
    h = 1e-5
    for n, g in zip(("x", "y", "post", "gate", "pre"), got):
        flat = g.cpu().double().flatten()
        for i in range(0, flat.numel(), 5):
            up, dn = dict(base), dict(base)
            for v, s in ((up, h), (dn, -h)):
                v[n] = base[n].clone()
                v[n].view(-1)[i] += s
            diff = (loss(up) - loss(dn)) / (2 * h)
            # h^2 of a third derivative of some hundreds, 1e-16 * |loss| / h,
            # and the kernel's own bound of about 400 U times terms below 50
            assert abs(float(flat[i]) - diff) <= 2e-3, (n, i, float(flat[i]), diff)


def test_streams_and_graph(cco):
    d = _inputs(300, 264, BF, F32, True, "channel", True)
    kw = dict(_kw(d), scale=0.7, eps=EPS)
    x, y, dout, du = (d[n].cuda() for n in ("x", "y", "dout", "du"))
    base = cco.block_norm(x, y, **kw) + cco.block_norm_grad(x, y, dout, du, **kw)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = [cco.block_norm(x, y, stream=s, **kw) +
           cco.block_norm_grad(x, y, dout, du, stream=s, **kw) for s in (s1, s2, s1, s2)]
    torch.cuda.synchronize()
    for r in got:
        for a, b in zip(r, base):
            assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, u = cco.block_norm(x, y, **kw)
        g = cco.block_norm_grad(x, y, dout, du, **kw)
    for i in range(3):
        x.mul_(1.25)
        du.mul_(-0.5)
        graph.replay()
        torch.cuda.synchronize()
        want = cco.block_norm(x, y, **kw) + cco.block_norm_grad(x, y, dout, du, **kw)
        for a, b in zip((o, u) + tuple(g), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("config,T", [("tiny", 128), ("tiny", 1), ("dsv3", 37), ("zipf", 50)])
@pytest.mark.parametrize("post,gate,pre", [(True, "channel", True), (False, "none", False),
                                           (True, "token", True), (False, "none", True)])
def test_fused_combine_is_the_two_calls(cco, config, T, post, gate, pre):
    from synth import get_config
    cfg = get_config(config).with_(I=0)  # identity experts: the rows are what counts
    c = make_case(cfg, T)
    heap, moe = make_moe(cfg, T)
    with heap:
        moe.plan(c.idx)
        moe.dispatch(c.x, c.w)
        y, _ = moe.combine(c.w)
        d = _inputs(T, cfg.H, BF, F32, post, gate, pre)
        kw = dict(_kw(d), scale=0.7, eps=EPS)
        x = d["x"].cuda()
        want = cco.block_norm(x, y, **kw)
        out, u, yy = cco.combine_norm(moe, x, c.w, keep_y=True, **kw)
        assert torch.equal(yy, y) and torch.equal(out, want[0])
        assert (u is None and want[1] is None) or torch.equal(u, want[1])
        out2, u2, none = cco.combine_norm(moe, x, c.w, **kw)
        assert none is None and torch.equal(out2, out)
        with pytest.raises(cco.CcoError):
            cco.combine_norm(moe, x[:0], c.w[:0], **dict(kw, token_gate=None, gate=None))


def test_fused_combine_with_dropped_pairs_and_many_choices(cco):
    import numpy as np
    from synth import get_config
    cfg = get_config("tiny").with_(I=0, K=19, E=32, S=4, H=520)
    T = 40
    rng = np.random.default_rng(1)
    idx = np.stack([rng.choice(32, 19, replace=False) for _ in range(T)]).astype(np.int32)
    idx[3, 2] = 99  # invalid: contributes nothing
    idx[5, 0] = -1
    w = rng.random((T, 19)).astype(np.float32)
    c = make_case(cfg, T, (idx, w))
    heap, moe = make_moe(cfg, T)
    with heap:
        moe.plan(c.idx)
        moe.dispatch(c.x, c.w)
        y, _ = moe.combine(c.w)
        pre = torch.ones(cfg.H, device="cuda")
        want = cco.block_norm(c.x, y, pre=pre)
        out, u, _ = cco.combine_norm(moe, c.x, c.w, pre=pre)
        assert torch.equal(out, want[0]) and torch.equal(u, want[1])


def test_rows_past_32_bits(cco):
    # more than 2^31 elements: the last rows lie behind 4 GiB
    T, H = 300_000, 7168
    x = torch.zeros((T, H), dtype=BF, device="cuda")
    y = torch.zeros((T, H), dtype=BF, device="cuda")
    d = _inputs(3, H, BF, F32, True, "channel", True)
    x[-3:], y[-3:] = d["x"].cuda(), d["y"].cuda()
    kw = dict(_kw(d), scale=0.7, eps=EPS)
    out, u = cco.block_norm(x, y, **kw)
    want = cco.block_norm(x[-3:].contiguous(), y[-3:].contiguous(), **kw)
    assert torch.equal(out[-3:], want[0]) and torch.equal(u[-3:], want[1])
    assert not out[:-3].any()
    dout, du = out.zero_(), u.zero_()
    dout[-3:], du[-3:] = d["dout"].cuda(), d["du"].cuda()
    got = cco.block_norm_grad(x, y, dout, du, dx=dout, dy=du, **kw)
    wg = cco.block_norm_grad(d["x"].cuda(), d["y"].cuda(), d["dout"].cuda(), d["du"].cuda(), **kw)
    for i in (0, 1):
        assert torch.equal(got[i][-3:], wg[i]) and not got[i][:-3].any()
    for i in (2, 3, 4):  # three rows' terms, at most in another order
        assert bool(((got[i] - wg[i]).abs() <= 8 * ref.U * 60 * (1 + wg[i].abs())).all())
