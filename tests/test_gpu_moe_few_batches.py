"""The layer for a few tokens: both forms of one token's down product, against
the 64-bit layer."""
import pytest
import torch

from tests import few_cases, ops_ref, serve_ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


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
