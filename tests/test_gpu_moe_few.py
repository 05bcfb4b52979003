"""The layer for a few tokens against the 64-bit layer, at every weight type,
at sizes that end inside steps, pieces and tiles, with pairs that take no part."""
import math

import pytest
import torch

from tests import ops_ref, serve_ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
TYPES = [(BF, BF), (FP, FP), (BF, torch.int8), (FP, torch.int8)]


@pytest.fixture(scope="module")
def cco():
    import combine_symmetric_memory_amd as m
    assert torch.cuda.is_available()
    return m


def _case(T, H, I, E, K, dtype, wdtype, seed=0, std=0.08):
    g = torch.Generator().manual_seed(seed)

    def r(shape, s):
        return torch.randn(shape, generator=g) * s

    c = dict(x=r((T, H), 1.0).to(dtype), s13=None, s2=None)
    c["idx"] = torch.rand((T, E), generator=g).argsort(1)[:, :K].to(torch.int32)
    if K > E:
        c["idx"] = torch.randint(0, E, (T, K), generator=g, dtype=torch.int32)
    c["w"] = torch.rand((T, K), generator=g) - 0.2
    if wdtype == torch.int8:
        c["w13"], c["w2"] = (torch.randint(-128, 128, s, generator=g, dtype=torch.int32)
                             .to(torch.int8) for s in ((E, 2 * I, H), (E, H, I)))
        c["s13"] = (0.5 + torch.rand((E, 2 * I), generator=g)) * std / 64
        c["s2"] = (0.5 + torch.rand((E, H), generator=g)) * std / 64
    else:
        c["w13"], c["w2"] = r((E, 2 * I, H), std).to(wdtype), r((E, H, I), std).to(wdtype)
    return c


def _call(cco, c, **kw):
    d = {k: v.cuda() if v is not None else None for k, v in c.items()}
    return cco.moe_few(d["x"], d["idx"], d["w"], d["w13"], d["w2"], s13=d["s13"], s2=d["s2"], **kw)


def _check(cco, c):
    got = _call(cco, c)
    want, err = serve_ref.layer(**c)
    ops_ref.assert_within(got, want, serve_ref.layer_bound(want, err, c["x"].dtype), "out")
    return got


@pytest.mark.parametrize("dtype,wdtype", TYPES)
@pytest.mark.parametrize("T,H,I,E,K", [(1, 256, 512, 8, 2), (1, 64, 64, 1, 1), (2, 96, 40, 3, 3),
                                       (4, 256, 512, 8, 2), (17, 128, 96, 5, 2),
                                       (33, 160, 80, 2, 2), (64, 256, 128, 1, 1),
                                       (64, 128, 144, 9, 4), (7, 2048, 272, 40, 8)])
def test_sizes(cco, dtype, wdtype, T, H, I, E, K):
    say("case: few %s %s T=%d H=%d I=%d E=%d K=%d" % (dtype, wdtype, T, H, I, E, K))
    _check(cco, _case(T, H, I, E, K, dtype, wdtype, T + H))


@pytest.mark.parametrize("dtype,wdtype", TYPES)
@pytest.mark.parametrize("H,I", [(1, 1), (1, 70), (65, 1), (15, 17), (31, 33), (257, 129),
                                 (1001, 419), (130, 1003)])
def test_odd_sizes(cco, dtype, wdtype, H, I):
    say("case: few odd %s %s H=%d I=%d" % (dtype, wdtype, H, I))
    for T in (1, 5):
        _check(cco, _case(T, H, I, 6, 3, dtype, wdtype, H))


@pytest.mark.parametrize("dtype,wdtype", TYPES)
@pytest.mark.parametrize("T,H,I,E,K", [(20, 200, 1003, 3, 2), (40, 130, 2048, 2, 1),
                                       (9, 16, 8, 2, 2), (3, 4100, 700, 1, 1),
                                       (1, 4112, 300, 2, 1), (64, 80, 257, 4, 4),
                                       (64, 72, 520, 64, 2), (64, 4200, 40, 200, 1)])
def test_both_forms_of_the_down_product(cco, dtype, wdtype, T, H, I, E, K):
    # several parts of the reduction, ends of rows and of column blocks
    say("case: few down %s %s T=%d H=%d I=%d E=%d K=%d" % (dtype, wdtype, T, H, I, E, K))
    _check(cco, _case(T, H, I, E, K, dtype, wdtype, T + I))


@pytest.mark.parametrize("wdtype", [BF, torch.int8])
def test_pairs_that_take_no_part(cco, wdtype):
    c = _case(12, 128, 96, 7, 3, BF, wdtype, 1)
    c["idx"][0] = -1
    c["idx"][1, 1] = 7
    c["idx"][2] = torch.tensor([2 ** 31 - 1, -2 ** 31, 3])
    c["idx"][5] = 1 << 20
    # what stands beside such an id does not count
    c["w"][0, 0], c["w"][1, 1], c["w"][5] = math.nan, math.inf, math.nan
    got = _call(cco, c)
    assert not bool(got[0].any()) and not bool(got[5].any())
    c["w"][0, 0] = c["w"][1, 1] = 0.0
    c["w"][5] = 0.0
    want, err = serve_ref.layer(**c)
    ops_ref.assert_within(got, want, serve_ref.layer_bound(want, err, BF), "out")


def test_nobody_has_an_expert(cco):
    c = _case(5, 64, 32, 3, 2, BF, BF, 2)
    c["idx"].fill_(-1)
    out = torch.full((5, 64), 9.0, dtype=BF, device="cuda")
    assert _call(cco, c, out=out) is out
    assert not bool(out.any())


@pytest.mark.parametrize("dtype,wdtype", TYPES)
def test_an_expert_several_times_in_a_token(cco, dtype, wdtype):
    c = _case(6, 128, 64, 4, 5, dtype, wdtype, 3)
    c["idx"][0] = 2
    c["idx"][1] = torch.tensor([1, 3, 1, -1, 3])
    _check(cco, c)


def test_all_tokens_at_one_expert(cco):
    c = _case(64, 256, 160, 300, 2, BF, BF, 4)
    c["idx"][:, 0] = 299
    c["idx"][:, 1] = torch.arange(64, dtype=torch.int32)
    _check(cco, c)


@pytest.mark.parametrize("dtype,wdtype", TYPES)
@pytest.mark.parametrize("T", [17, 33, 64])
def test_an_expert_with_more_tokens_than_the_others(cco, dtype, wdtype, T):
    # several rounds of 16 tokens for one expert, none for some
    c = _case(T, 192, 600, 8, 1, dtype, wdtype, 14)
    c["idx"][:] = 3
    c["idx"][5] = 6
    _check(cco, c)


def test_many_experts_and_pairs(cco):
    c = _case(64, 64, 32, 1024, 32, BF, torch.int8, 5)
    _check(cco, c)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("where", ["x", "w13", "w2", "w"])
def test_what_is_not_a_number_stays_with_its_tokens(cco, where, bad):
    # token 3 has it; every other token's result is that of the clean call,
    # bit for bit, although they share the tiles
    c = _case(9, 128, 64, 6, 2, BF, BF, 6)
    c["idx"][:] = torch.tensor([0, 1], dtype=torch.int32)
    c["idx"][3] = torch.tensor([4, 1], dtype=torch.int32)
    clean = _call(cco, c)
    if where == "x":
        c["x"][3, 77] = bad
    elif where == "w13":
        c["w13"][4, 5] = bad
    elif where == "w2":
        c["w2"][4] = bad
    else:
        c["w"][3, 0] = bad
    got = _call(cco, c)
    others = [t for t in range(9) if t != 3]
    assert torch.equal(got[others], clean[others])
    assert not bool(torch.isfinite(got[3].float()).all())


def test_fp16_intermediate_rows_past_fp16(cco):
    # h far beyond 65504, and far below 2^-24: out is an ordinary number
    H, I = 64, 64
    for big in (2.0 ** 10, 2.0 ** -9):
        c = _case(3, H, I, 2, 1, FP, FP, 7, 1.0)
        c["x"] = (c["x"].float() * big).to(FP)
        c["w2"] = (c["w2"].float() * (2.0 ** -10 if big > 1 else 2.0 ** 4)).to(FP)
        c["w"].fill_(2.0 ** -10 if big > 1 else 1.0)
        want, err = serve_ref.layer(**c)
        assert bool((want.abs() < 65504).all())
        ops_ref.assert_within(_call(cco, c), want, serve_ref.layer_bound(want, err, FP), "out")


def test_an_unused_expert_is_not_read(cco):
    c = _case(3, 128, 64, 6, 2, BF, BF, 8)
    c["idx"] = torch.tensor([[0, 2], [2, 5], [5, 0]], dtype=torch.int32)
    for e in (1, 3, 4):
        c["w13"][e] = math.nan
        c["w2"][e] = math.nan
    _check(cco, c)


@pytest.mark.parametrize("wdtype", [BF, torch.int8])
def test_unaligned_weights(cco, wdtype):
    c = _case(3, 96, 64, 4, 2, BF, wdtype, 9)
    want = _call(cco, c)
    d = {k: v.cuda() if v is not None else None for k, v in c.items()}
    for k in ("x", "w13", "w2"):
        flat = torch.empty(d[k].numel() + 1, dtype=d[k].dtype, device="cuda")
        moved = flat[1:].view(d[k].shape)
        moved.copy_(d[k])
        d[k] = moved
    got = cco.moe_few(d["x"], d["idx"], d["w"], d["w13"], d["w2"], s13=d["s13"], s2=d["s2"])
    assert torch.equal(got, want)


def test_repeats_streams_and_a_graph(cco):
    c = _case(8, 512, 384, 12, 3, BF, torch.int8, 10)
    d = {k: v.cuda() for k, v in c.items()}

    def call(**kw):
        return cco.moe_few(d["x"], d["idx"], d["w"], d["w13"], d["w2"], s13=d["s13"], s2=d["s2"],
                           **kw)

    want = call()
    for _ in range(5):
        assert torch.equal(call(), want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = call(stream=side)
    other = call()  # at the same time: nothing is shared
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(other, want)
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = call()
    for seed in range(3):
        n = _case(8, 512, 384, 12, 3, BF, torch.int8, 20 + seed)
        for k in ("x", "idx", "w"):
            d[k].copy_(n[k])
        eager = call()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager)


def test_too_many_tokens_are_refused(cco):
    c = _case(65, 32, 32, 2, 1, BF, BF, 11)
    with pytest.raises(cco.CcoError) as e:
        _call(cco, c)
    assert e.value.code == cco.CCO_ERR_TOO_LARGE
    c = _case(1, 32, 32, 2, 1, BF, BF, 12)
    for k in ("x", "idx", "w"):
        c[k] = c[k][:0]
    assert _call(cco, c).shape == (0, 32)
