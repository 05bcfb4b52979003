"""The norms around a block where they go wrong most easily: infinite and NaN
rows that the gradient's formula does not read, rows far from one, and
launches whose workgroups take several rows in every kernel form."""
import math

import pytest
import torch

from tests import test_gpu_block_norm as base
from tests.gpu_util import make_case, make_moe, say

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-5


@pytest.fixture(scope="module")
def cco():
    import combine_symmetric_memory_amd as m
    assert torch.cuda.is_available()
    return m


def _equal(a, b):
    return (a is None and b is None) or torch.equal(a, b)


@pytest.mark.parametrize("H", [520, 77, 5, 8200])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("post,gate", [(True, "none"), (True, "channel"), (True, "token"),
                                       (False, "none"), (False, "channel"), (False, "token")])
def test_without_pre_the_gradient_does_not_read_x(cco, H, dtype, post, gate):
    # out = x + scale gate z: no derivative of out depends on x
    say("case: x outside the gradient H=%d %s post=%s gate=%s" % (H, dtype, post, gate))
    d = base._inputs(6, H, dtype, F32, post, gate, False)
    kw = dict(base._kw(d), scale=0.7, eps=EPS)
    y, dout = d["y"].cuda(), d["dout"].cuda()
    x = torch.zeros((6, H), dtype=dtype, device="cuda")
    want = cco.block_norm_grad(x, y, dout, **kw)
    for t in want:
        assert t is None or bool(torch.isfinite(t).all())
    x[0, 0] = math.inf
    x[1, H - 1] = -math.inf
    x[2, H // 2] = math.nan
    x[3] = torch.finfo(dtype).max
    x[4] = math.inf
    got = cco.block_norm_grad(x, y, dout, **kw)
    assert torch.equal(got[0], dout)
    for g, w in zip(got, want):
        assert _equal(g, w)


@pytest.mark.parametrize("H", [520, 77, 5, 8200])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
def test_without_norms_dy_does_not_read_y(cco, H, gate):
    # z = y: dx = dout and dy = scale gate dout whatever y holds, and a gate's
    # gradient meets only the columns or tokens that hold the infinities
    d = base._inputs(6, H, BF, F32, False, gate, False)
    kw = dict(base._kw(d), scale=0.7, eps=EPS)
    x, y, dout = d["x"].cuda(), d["y"].cuda(), d["dout"].cuda()
    want = cco.block_norm_grad(x, y, dout, **kw)
    bad = y.clone()
    bad[1, 0] = math.inf
    bad[2, H - 1] = math.nan
    bad[4] = torch.finfo(BF).max
    got = cco.block_norm_grad(x, bad, dout, **kw)
    assert torch.equal(got[0], dout) and torch.equal(got[1], want[1])
    assert bool(torch.isfinite(got[1]).all())
    if gate == "token":
        good = [0, 3, 5]
        assert torch.equal(got[3][good], want[3][good])
        assert not bool(torch.isfinite(got[3][[1, 2]]).any())
    if gate == "channel":
        bad[4] = y[4]
        got = cco.block_norm_grad(x, bad, dout, **kw)
        assert torch.equal(got[3][1:H - 1], want[3][1:H - 1])
        assert not bool(torch.isfinite(got[3][[0, H - 1]]).any())


@pytest.mark.parametrize("factor", [1e15, 3e16, 1e-14, 1e-17])
@pytest.mark.parametrize("post,gate,pre", [f for f in base.FORMS if f[0] or f[2]])
def test_rows_far_from_one(cco, monkeypatch, factor, post, gate, pre):
    # x and y scaled by `factor` and dout by its inverse, eps 0: every term
    # of the gradient keeps its share
    plain = base._inputs

    def scaled(T, H, dtype, *a, **kw):
        d = plain(T, H, dtype, *a, **kw)
        d["x"] = (d["x"].double() * factor).to(dtype)
        if d["y"] is not None:
            d["y"] = (d["y"].double() * factor).to(dtype)
        d["dout"] = (d["dout"].double() / factor).to(dtype)
        return d

    monkeypatch.setattr(base, "_inputs", scaled)
    monkeypatch.setattr(base, "EPS", 0.0)
    # z is normalised with post and takes its size from scale, from y without
    scale = 0.7 * (factor if post else 1.0)
    for dtype, H in ((BF, 256), (F32, 77), (BF, 8200)):
        base._check(cco, 5, H, dtype, F32, post, gate, pre, scale=scale)
        if pre:
            base._check(cco, 3, H, dtype, F32, post, gate, pre, scale=scale, use_dout=False)


# -------------------------------------- several rows a workgroup, every form
@pytest.mark.parametrize("H,dtype", [(8200, BF), (9999, HF), (16384, BF), (12001, F32)])
@pytest.mark.parametrize("post,gate", [(True, "channel"), (True, "token"), (False, "none")])
def test_widest_rows_several_a_workgroup(cco, H, dtype, post, gate):
    base._check(cco, 600, H, dtype, F32, post, gate, True)


@pytest.mark.parametrize("config,over,T", [("dsv3", dict(), 1300), ("tiny", dict(H=256), 9000),
                                           ("tiny", dict(H=8448), 700)])
@pytest.mark.parametrize("post,gate,pre", [(True, "channel", True), (True, "token", True),
                                           (False, "token", False), (False, "none", True)])
def test_fused_combine_several_rows_a_workgroup(cco, config, over, T, post, gate, pre):
    from synth import get_config
    cfg = get_config(config).with_(I=0, **over)
    say("case: combine_norm %s H=%d T=%d" % (config, cfg.H, T))
    c = make_case(cfg, T)
    heap, moe = make_moe(cfg, T)
    with heap:
        moe.plan(c.idx)
        moe.dispatch(c.x, c.w)
        y, _ = moe.combine(c.w)
        d = base._inputs(T, cfg.H, BF, F32, post, gate, pre)
        kw = dict(base._kw(d), scale=0.7, eps=EPS)
        x = d["x"].cuda()
        want = cco.block_norm(x, y, **kw)
        for _ in range(3):
            out, u, yy = cco.combine_norm(moe, x, c.w, keep_y=True, **kw)
            assert torch.equal(yy, y) and torch.equal(out, want[0]) and _equal(u, want[1])
            out, u, _ = cco.combine_norm(moe, x, c.w, **kw)
            assert torch.equal(out, want[0]) and _equal(u, want[1])
