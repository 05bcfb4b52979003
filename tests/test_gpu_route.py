"""The router (cco_route, cco_route_grad): ids equal to a 64-bit choice,
weights and gradients within derived bounds, masked, equal, infinite and NaN
logits, invalid and repeated ids."""
import math

import pytest
import torch

from tests import ops_ref as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
INF = math.inf


@pytest.fixture(scope="module")
def cco():
    import combine_symmetric_memory_amd as m
    assert torch.cuda.is_available()
    return m


def _weights_bound(logits, ids, want, scale):
    """exp's argument is off by |l - m| U, exp itself and the quotient by a
    few U, a sum of n terms by (n / 64 + 8) U."""
    l = logits.double()
    l = torch.where(torch.isinf(l), torch.zeros_like(l), l)
    spread = (l.amax(1) - l.amin(1)).unsqueeze(1)
    n = logits.shape[1]
    return want.abs() * (2 * spread + 48 + n / 32) * ref.U + abs(scale) * 2.0 ** -126


def _check(cco, logits, topk, score, renorm, scale=1.0, bias=None, groups=1, kept=1, seed=0):
    say("case: route %s K=%d %s renorm=%s bias=%s groups=%d/%d" % (
        tuple(logits.shape), topk, score, renorm, bias is not None, kept, groups))
    T, E = logits.shape
    ld = logits.cuda()
    bd = None if bias is None else bias.cuda()
    idx, w = cco.route(ld, topk, score=score, renorm=renorm, scale=scale, bias=bd, groups=groups,
                       kept=kept)
    want = ref.choose(logits, topk, score, bias, groups, kept)
    assert idx.cpu().tolist() == want
    ids = torch.tensor(want, dtype=torch.int64).reshape(T, topk)
    l64 = logits.double().requires_grad_(True)
    ww = ref.weights(l64, ids, score, renorm, scale)
    ref.assert_within(w, ww.detach(), _weights_bound(logits, ids, ww.detach(), scale), "weights")
    g = torch.Generator().manual_seed(seed)
    dw = torch.randn((T, topk), generator=g)
    got = cco.route_grad(ld, idx, dw.cuda(), score=score, renorm=renorm, scale=scale)
    assert got.dtype == logits.dtype
    want_g, = torch.autograd.grad(ww, l64, dw.double())
    # every part of a logit's gradient is a product of the factors above
    # with dw; the largest of them bounds the cancelling ones
    l = logits.double()
    l = torch.where(torch.isinf(l), torch.zeros_like(l), l)
    spread = (l.amax(1) - l.amin(1)).unsqueeze(1)
    size = (ww.detach().abs() * dw.double().abs()).sum(1, keepdim=True) + \
        ww.detach().abs().amax(1, keepdim=True) * dw.double().abs().amax(1, keepdim=True)
    bound = ref.half_step(logits.dtype) * want_g.abs() + ref.smallest(logits.dtype) + \
        size * (4 * spread + 96 + E / 16) * ref.U
    ref.assert_within(got, want_g, bound, "gradient")
    return idx, w


MODES = [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)]


@pytest.mark.parametrize("score,renorm", MODES)
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (3, 2, 2), (5, 8, 2), (70, 63, 7), (9, 64, 32),
                                   (33, 65, 5), (40, 256, 8), (6, 300, 6), (7, 512, 16),
                                   (5, 1024, 32)])
def test_sizes(cco, T, E, K, score, renorm):
    g = torch.Generator().manual_seed(T * E)
    logits = torch.randn((T, E), generator=g) * 2
    _check(cco, logits, K, score, renorm, scale=2.5)
    _check(cco, logits, K, score, renorm, bias=torch.randn(E, generator=g) * 0.2)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("score,renorm", MODES)
def test_half_types_and_equal_values(cco, dtype, score, renorm):
    # few distinct values: many ties, which go to the lower id
    g = torch.Generator().manual_seed(3)
    logits = (torch.randint(-3, 4, (50, 130), generator=g) * 0.5).to(dtype)
    _check(cco, logits, 9, score, renorm)
    _check(cco, logits, 9, score, renorm, bias=torch.zeros(130))
    _check(cco, torch.zeros((4, 100), dtype=dtype), 5, score, renorm)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,kept,K", [(16, 8, 1, 2), (16, 8, 8, 4), (64, 4, 2, 8),
                                             (256, 8, 4, 8), (192, 64, 5, 6), (35, 5, 2, 3),
                                             (1024, 2, 1, 32), (63, 63, 10, 10)])
def test_groups(cco, score, E, groups, kept, K):
    g = torch.Generator().manual_seed(E + groups)
    logits = torch.randn((40, E), generator=g)
    _check(cco, logits, K, score, True, groups=groups, kept=kept)
    _check(cco, logits, K, score, True, scale=2.5, bias=torch.randn(E, generator=g) * 0.1,
           groups=groups, kept=kept)
    # equal groups
    _check(cco, torch.zeros((2, E)), K, score, True, groups=groups, kept=kept)


@pytest.mark.parametrize("score,renorm", MODES)
def test_masked_experts(cco, score, renorm):
    g = torch.Generator().manual_seed(5)
    logits = torch.randn((60, 96), generator=g)
    logits[torch.rand((60, 96), generator=g) < 0.7] = -INF
    logits[7] = -INF            # a row of nothing
    logits[8, 1:] = -INF        # at most one expert left, fewer than K
    logits[9] = torch.finfo(F32).min
    bias = torch.rand(96, generator=g) * 3
    for kw in (dict(), dict(bias=bias), dict(groups=8, kept=3),
               dict(bias=bias, groups=8, kept=3)):
        idx, w = _check(cco, logits, 6, score, renorm, **kw)
        assert not w[7].any()
        ids = idx[7].cpu().tolist()
        assert ids == list(range(6))
        assert torch.isfinite(w).all()
        left = torch.isfinite(logits[8]).sum()
        assert int((w[8] > 0).sum()) == int(left)


@pytest.mark.parametrize("score,renorm", MODES)
def test_one_expert_left(cco, score, renorm):
    logits = torch.full((3, 70), -INF)
    logits[0, 69] = 0.5
    logits[1, 0] = -3.0
    logits[2, 33] = 20.0
    _, w = _check(cco, logits, 4, score, renorm)
    assert bool((w[:, 0] > 0).all()) and not w[:, 1:].any()


def test_low_logits_keep_their_proportions(cco):
    logits = torch.tensor([[-200.0, -201.0, -199.0, -300.0], [-95.0, -94.0, -96.0, -97.0],
                           [90.0, 95.0, 100.0, -100.0]])
    for score in ("softmax", "sigmoid"):
        _check(cco, logits, 3, score, True)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kw", [dict(), dict(bias=1), dict(groups=4, kept=2)])
def test_nan_and_infinity_give_valid_ids(cco, score, kw):
    g = torch.Generator().manual_seed(8)
    logits = torch.randn((8, 40), generator=g)
    logits[1, 3] = math.nan
    logits[2] = math.nan
    logits[3, 5] = INF
    logits[4, 5] = INF
    logits[4, 39] = INF
    logits[5, 0] = -INF
    logits[5, 1] = math.nan
    if "bias" in kw:
        kw = dict(bias=torch.randn(40, generator=g) * 0.1)
    idx, w = cco.route(logits.cuda(), 6, score=score, bias=kw["bias"].cuda() if "bias" in kw
                       else None, groups=kw.get("groups", 1), kept=kw.get("kept", 1))
    want = ref.choose(logits, 6, score, kw.get("bias"), kw.get("groups", 1), kw.get("kept", 1))
    assert idx.cpu().tolist() == want
    good = [0, 6, 7] + ([1, 3, 4, 5] if score == "sigmoid" else [])
    assert torch.isfinite(w[good]).all()
    if score == "softmax":
        assert torch.isnan(w[[1, 2, 3, 4, 5]]).all()


@pytest.mark.parametrize("score,renorm", MODES)
def test_gradient_of_any_ids(cco, score, renorm):
    # outside ids take no part, repeated ones count twice
    g = torch.Generator().manual_seed(2)
    logits = torch.randn((6, 70), generator=g)
    dw = torch.randn((6, 4), generator=g)
    idx = torch.tensor([[1, 1, 5, 69], [-1, 3, 70, 4], [-1, -5, 2 ** 31 - 1, 99], [7, 7, 7, 7],
                        [0, 64, 1, 65], [2, -1, 2, -1]], dtype=torch.int32)
    got = cco.route_grad(logits.cuda(), idx.cuda(), dw.cuda(), score=score, renorm=renorm,
                         scale=1.5)
    for t in range(6):
        on = [j for j in range(4) if 0 <= int(idx[t, j]) < 70]
        if not on:
            assert not got[t].any()
            continue
        l = logits[t:t + 1].double().requires_grad_(True)
        w = ref.weights(l, idx[t:t + 1, on].long(), score, renorm, 1.5)
        want, = torch.autograd.grad(w, l, dw[t:t + 1, on].double())
        bound = torch.full_like(want, 400 * ref.U * 1.5 * float(dw[t].abs().sum()))
        ref.assert_within(got[t:t + 1], want, bound, "row %d" % t)


@pytest.mark.parametrize("score,renorm", MODES)
def test_gradient_against_differences(cco, score, renorm):
    g = torch.Generator().manual_seed(4)
    logits = torch.randn((5, 24), generator=g)
    dw = torch.randn((5, 6), generator=g)
    idx, _ = cco.route(logits.cuda(), 6, score=score, renorm=renorm)
    got = cco.route_grad(logits.cuda(), idx, dw.cuda(), score=score, renorm=renorm).cpu().double()
    ids = idx.cpu().long()
    h = 1e-6
    for e in range(24):
        up, dn = logits.double().clone(), logits.double().clone()
        up[:, e] += h
        dn[:, e] -= h
        d = ((ref.weights(up, ids, score, renorm, 1.0) - ref.weights(dn, ids, score, renorm, 1.0))
             * dw.double()).sum(1) / (2 * h)
        # differences: h^2 / 6 of a third derivative below 8, and 1e-16 / h
        assert bool(((got[:, e] - d).abs() <= 1e-8 + 400 * ref.U * dw.double().abs().sum(1)).all())


def test_row_distances_streams_and_graph(cco):
    g = torch.Generator().manual_seed(1)
    buf = torch.full((30, 140), math.nan)
    buf[:, 4:133] = torch.randn((30, 129), generator=g)
    logits = buf[:, 4:133].contiguous()
    view = buf.cuda()[:, 4:133]
    dw = torch.randn((30, 8), generator=g).cuda()
    idx, w = cco.route(view, 8, score="sigmoid", renorm=True)
    i2, w2 = cco.route(logits.cuda(), 8, score="sigmoid", renorm=True)
    assert torch.equal(idx, i2) and torch.equal(w, w2)
    out = torch.full((30, 131), 5.0, device="cuda")
    cco.route_grad(view, idx, dw, score="sigmoid", renorm=True, out=out[:, :129])
    d2 = cco.route_grad(logits.cuda(), idx, dw, score="sigmoid", renorm=True)
    assert torch.equal(out[:, :129], d2) and bool((out[:, 129:] == 5).all())
    s = torch.cuda.Stream()
    i3, w3 = cco.route(view, 8, score="sigmoid", renorm=True, stream=s)
    s.synchronize()
    assert torch.equal(idx, i3) and torch.equal(w, w3)
    gi, gw = torch.zeros_like(idx), torch.zeros_like(w)
    graph = torch.cuda.CUDAGraph()
    src = logits.cuda()
    with torch.cuda.graph(graph):
        cco.route(src, 8, score="sigmoid", renorm=True, idx=gi, w=gw)
        cco.route_grad(src, gi, dw, score="sigmoid", renorm=True, out=d2)
    for i in range(3):
        src.copy_(torch.randn((30, 129), generator=g))
        graph.replay()
        torch.cuda.synchronize()
        a, b = cco.route(src, 8, score="sigmoid", renorm=True)
        assert torch.equal(a, gi) and torch.equal(b, gw)
        assert torch.equal(cco.route_grad(src, a, dw, score="sigmoid", renorm=True), d2)


def test_no_tokens(cco):
    idx, w = cco.route(torch.empty((0, 8), device="cuda"), 2)
    assert idx.shape == (0, 2) and w.shape == (0, 2)
    assert cco.route_grad(torch.empty((0, 8), device="cuda"), idx, w).shape == (0, 8)


def test_tokens_past_32_bits(cco):
    T, E = 8_400_000, 256
    logits = torch.zeros((T, E), dtype=BF, device="cuda")
    g = torch.Generator().manual_seed(6)
    tail = torch.randn((5, E), generator=g).to(BF)
    logits[-5:] = tail.cuda()
    idx, w = cco.route(logits, 4, score="sigmoid", renorm=True)
    i2, w2 = cco.route(tail.cuda(), 4, score="sigmoid", renorm=True)
    assert torch.equal(idx[-5:], i2) and torch.equal(w[-5:], w2)
    assert idx[0].tolist() == [0, 1, 2, 3]
    dw = torch.ones((T, 4), device="cuda")
    dw[-5:, 1] = -2
    got = cco.route_grad(logits, idx, dw, score="sigmoid", renorm=True, out=logits)
    want = cco.route_grad(tail.cuda(), i2, dw[-5:].contiguous(), score="sigmoid", renorm=True)
    assert torch.equal(got[-5:], want) and not got[:-5].any()
