"""The layer for a few tokens: both forms of one token's down product, and what
a token gets in batches of other tokens, against the 64-bit layer."""
import math

import pytest
import torch

from tests import few_cases, ops_ref, serve_ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def cco():
    import combine_symmetric_memory_amd as m
    assert torch.cuda.is_available()
    return m


def _weights(H, I, E, wdtype, g, std):
    if wdtype == torch.int8:
        w13, w2 = (torch.randint(-128, 128, s, generator=g, dtype=torch.int32).to(torch.int8)
                   for s in ((E, 2 * I, H), (E, H, I)))
        return w13, w2, (0.5 + torch.rand((E, 2 * I), generator=g)) * std / 64, \
            (0.5 + torch.rand((E, H), generator=g)) * std / 64
    return (torch.randn((E, 2 * I, H), generator=g) * std).to(wdtype), \
        (torch.randn((E, H, I), generator=g) * std).to(wdtype), None, None


def _layer(x, idx, w, weights):
    """The 64-bit layer of one token, of the experts it has."""
    w13, w2, s13, s2 = weights
    es = sorted({int(e) for e in idx.flatten() if 0 <= int(e) < w2.shape[0]})
    at = torch.tensor([[es.index(int(e)) if int(e) in es else -1 for e in idx.flatten()]])
    return serve_ref.layer(x, at, w, w13[es], w2[es], None if s13 is None else s13[es],
                           None if s2 is None else s2[es])


@pytest.mark.parametrize("dtype,wdtype", few_cases.TYPES)
@pytest.mark.parametrize("case", range(5))
def test_one_token(cco, dtype, wdtype, case):
    T, H, I, E, K, _ = few_cases.one_token(wdtype)[case]
    say("case: few one token %s %s H=%d I=%d E=%d K=%d" % (dtype, wdtype, H, I, E, K))
    g = torch.Generator().manual_seed(case)
    x = torch.randn((T, H), generator=g).to(dtype)
    idx = torch.randint(0, E, (T, K), generator=g, dtype=torch.int32)
    w = torch.rand((T, K), generator=g) - 0.2
    weights = _weights(H, I, E, wdtype, g, 0.03)
    dev = [t if t is None else t.cuda() for t in weights]
    got = cco.moe_few(x.cuda(), idx.cuda(), w.cuda(), dev[0], dev[1], s13=dev[2], s2=dev[3])
    want, err = _layer(x, idx, w, weights)
    ops_ref.assert_within(got, want, serve_ref.layer_bound(want, err, dtype), "out")


@pytest.mark.parametrize("dtype,wdtype", few_cases.TYPES)
@pytest.mark.parametrize("H,I,E,K", [(256, 1024, 64, 8), (512, 600, 8, 2)])
def test_a_token_among_others(cco, dtype, wdtype, H, I, E, K):
    # The order of a token's sums may depend on the others, nothing else of its
    # result: it stays within the bound of its own 64-bit layer in every batch,
    # whatever they hold, and the same batch gives the same bits.
    g = torch.Generator().manual_seed(H)
    x1 = torch.randn((1, H), generator=g).to(dtype)
    idx1 = torch.randperm(E, generator=g)[:K].to(torch.int32)[None]
    w1 = torch.rand((1, K), generator=g) - 0.2
    weights = _weights(H, I, E, wdtype, g, 0.08)
    dev = [t if t is None else t.cuda() for t in weights]
    want, err = _layer(x1, idx1, w1, weights)
    bound = serve_ref.layer_bound(want, err, dtype)
    for T, at, bad in [(1, 0, 0.0), (2, 1, math.inf), (5, 0, math.nan), (9, 4, 0.0),
                       (17, 16, -math.inf), (33, 7, 0.0), (64, 63, math.nan), (64, 20, 0.0)]:
        say("case: few among others %s %s H=%d I=%d T=%d at %d" % (dtype, wdtype, H, I, T, at))
        x = torch.randn((T, H), generator=g).to(dtype)
        w = torch.rand((T, K), generator=g)
        if bad:
            x[:, 3] = bad
            w[::2, 0] = bad
        idx = torch.randint(-1, E + 1, (T, K), generator=g, dtype=torch.int32)
        if T == 5:
            idx[:] = idx1  # the same experts for all
        x[at], idx[at], w[at] = x1[0], idx1[0], w1[0]
        args = (x.cuda(), idx.cuda(), w.cuda(), dev[0], dev[1])
        got = cco.moe_few(*args, s13=dev[2], s2=dev[3])
        ops_ref.assert_within(got[at:at + 1], want, bound, "token %d of %d" % (at, T))
        again = cco.moe_few(*args, s13=dev[2], s2=dev[3])
        assert torch.equal(got.view(torch.int16), again.view(torch.int16))
