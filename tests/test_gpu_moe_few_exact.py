"""The layer for a few tokens where its 64-bit result is known term by term:
what its splits into two bf16 values may lose, and the ends of their range.

silu(32) is 32 in 32 bits (e^-32 is below half a step of one), so h = 32 u is
what the test puts there, exactly."""
import pytest
import torch

from tests import ops_ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def cco():
    import combine_symmetric_memory_amd as m
    assert torch.cuda.is_available()
    return m


def _tokens(T, K):
    return (torch.zeros(T, K, dtype=torch.int32, device="cuda"),
            torch.full((T, K), 1.0 / K, device="cuda"))


@pytest.mark.parametrize("T,K", [(1, 1), (2, 2), (20, 2)])
def test_fp16_weights_by_h(cco, T, K):
    # One column of weights over every significand of fp16, times an h whose
    # low part is half a bf16 step, the largest there is; a second column takes
    # the product with the high part away again, so that the result, w times
    # that low part, shows what the products of the parts leave out.  Allowed:
    # the product of both low parts, 2^-8 of w by 2^-8 of h; h itself, its
    # difference and the sums are exact or to a few 2^-24, and the result is
    # rounded to fp16.
    say("case: few fp16 significands T=%d K=%d" % (T, K))
    H, I = 1024, 8
    sig = 1.0 + torch.arange(1024, dtype=torch.float64) / 1024
    h0 = 32.0 * (1.0 + 2.0 ** -8)
    x = torch.zeros(T, H, dtype=FP)
    x[:, 0] = 1.0
    w13 = torch.zeros(1, 2 * I, H, dtype=FP)
    w13[0, :2, 0] = 32.0                        # gates
    w13[0, I, 0], w13[0, I + 1, 0] = 1.0 + 2.0 ** -8, 1.0
    w2 = torch.zeros(1, H, I, dtype=FP)
    w2[0, :, 0], w2[0, :, 1] = sig.to(FP), -sig.to(FP)
    assert torch.equal(w2[0, :, 0].double(), sig)
    idx, w = _tokens(T, K)
    got = cco.moe_few(x.cuda(), idx, w, w13.cuda(), w2.cuda())
    want = (sig * (h0 - 32.0)).expand(T, H)
    total = sig * (h0 + 32.0)
    bound = 2.0 ** -16 * sig * h0 + 16 * ops_ref.U * total + ops_ref.half_step(FP) * want
    ops_ref.assert_within(got, want, bound, "out")
