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


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("wdtype", [BF, torch.int8])
@pytest.mark.parametrize("T,K", [(1, 1), (2, 2), (20, 2)])
def test_h_next_to_the_largest_float(cco, T, K, wdtype, sign):
    # h = (1 - 2^-n) 2^128 lies above bf16's largest value, below infinity: a
    # gate of 2^64 and an up value of n terms 2^63, 2^62, ..
    say("case: few h next to the largest float T=%d K=%d %s" % (T, K, wdtype))
    H, I = 48, 16
    n = [9, 10, 11, 14]
    x = torch.zeros(T, H, dtype=BF)
    x[:, 0] = 2.0 ** 60
    x[:, 1:17] = (2.0 ** (64 - torch.arange(1, 17, dtype=torch.float64))).to(BF)
    w13, w2 = torch.zeros(1, 2 * I, H), torch.zeros(1, H, I)
    for i, k in enumerate(n):
        w13[0, i, 0] = 16.0
        w13[0, I + i, 1:1 + k] = sign
        w2[0, i::len(n), i] = 1.0
    s13 = s2 = None
    if wdtype == torch.int8:
        s13 = torch.ones(1, 2 * I, device="cuda")
        s2 = torch.full((1, H), 2.0 ** -100, device="cuda")
    else:
        w2 *= 2.0 ** -100
    idx, w = _tokens(T, K)
    got = cco.moe_few(x.cuda(), idx, w, w13.to(wdtype).cuda(), w2.to(wdtype).cuda(), s13=s13,
                      s2=s2)
    want = torch.tensor([sign * (1.0 - 2.0 ** -k) * 2.0 ** 28 for k in n],
                        dtype=torch.float64).repeat(H // len(n)).expand(T, H)
    # h is held to 2^-17; the sums and the products with scales and shares take
    # a few steps of 2^-24
    bound = (2.0 ** -17 + 16 * ops_ref.U + ops_ref.half_step(BF)) * want.abs()
    ops_ref.assert_within(got, want, bound, "out")
