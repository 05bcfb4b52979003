"""Rows to 8-bit integers: every code as the exact quotient rounds, at sizes of
every form of the kernel, and the rows where it can go wrong."""
import math

import pytest
import torch

from tests import ops_ref, serve_ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module")
def cco():
    import combine_symmetric_memory_amd as m
    assert torch.cuda.is_available()
    return m


def _x(rows, cols, dtype, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, cols, generator=g) * std).to(dtype)


def _scale_bound(s):
    return s.abs() * ops_ref.U * (1 + 2 ** -10) + 2.0 ** -150


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [1, 2, 7, 8, 9, 15, 64, 513, 1000, 1024, 2047, 2048, 4096, 5003,
                                  8192, 14336, 16384, 16391, 40000])
def test_codes_and_scales(cco, dtype, cols):
    say("case: quant %s cols=%d" % (dtype, cols))
    for rows in (1, 5):
        x = _x(rows, cols, dtype, cols)
        q, s = cco.quant_rows(x.cuda())
        want, ws = serve_ref.quant(x)
        assert torch.equal(q.cpu(), want)
        ops_ref.assert_within(s, ws, _scale_bound(ws), "scales")


@pytest.mark.parametrize("dtype", DTYPES)
def test_ties_go_to_the_even_code(cco, dtype):
    # with a largest value of 254 the quotient is v / 2: odd v are ties
    v = torch.arange(-254, 255, dtype=torch.float32)
    x = v.to(dtype)
    assert torch.equal(x.float(), v)
    q, s = cco.quant_rows(x.cuda()[None])
    assert float(s[0]) == 2.0
    assert torch.equal(q[0].cpu().float(), torch.round(v / 2))
    # ... and half the largest value is one whatever that is
    for top in (1.0, 3.0, 1.0078125, 77.5):
        q, _ = cco.quant_rows(torch.tensor([[top, top / 2, -top / 2, 0.0] * 4], dtype=dtype,
                                           device="cuda"))
        assert q[0, :4].tolist() == [127, 64, -64, 0]


def test_values_next_to_a_tie(cco):
    # fp32 values one step from a tie, on either side of it
    top = torch.tensor(1.0 + 2.0 ** -23)
    rows = []
    for k in range(0, 127, 9):
        tie = (k + 0.5) * float(top) / 127
        t = torch.tensor(tie, dtype=torch.float32)
        near = [float(t)]
        up = down = t
        for _ in range(3):
            up = torch.nextafter(up, torch.tensor(2.0))
            down = torch.nextafter(down, torch.tensor(-2.0))
            near += [float(up), float(down)]
        rows.append(near + [float(top)])
    x = torch.tensor(rows, dtype=torch.float32)
    q, _ = cco.quant_rows(x.cuda())
    # the exact quotient's rounding, in integers
    from fractions import Fraction
    for r, row in enumerate(x.tolist()):
        m = Fraction(max(abs(v) for v in row))
        assert q[r].tolist() == [round(Fraction(v) * 127 / m) for v in row]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [5, 40, 3000, 20000])
def test_rows_of_zeros_infinities_and_nan(cco, dtype, cols):
    x = _x(6, cols, dtype, 3)
    x[0] = 0
    x[1] = -0.0
    x[2, cols // 2] = math.inf
    x[3, cols - 1] = -math.inf
    x[4, 0] = math.nan
    q, s = cco.quant_rows(x.cuda())
    assert not bool(q[:5].any())
    assert s[:2].tolist() == [0.0, 0.0] and bool(torch.isnan(s[2:5]).all())
    want, ws = serve_ref.quant(x[5:])
    assert torch.equal(q[5:].cpu(), want)


@pytest.mark.parametrize("top", [2.0 ** -149, 2.0 ** -140, 2.0 ** -126, 1e-30, 3e38])
def test_the_ends_of_the_range(cco, top):
    x = _x(3, 700, torch.float32, 5)
    x = (x.double() / x.double().abs().max() * top).float()
    x[:, 17] = top
    q, s = cco.quant_rows(x.cuda())
    want, ws = serve_ref.quant(x)
    assert torch.equal(q.cpu(), want)
    ops_ref.assert_within(s, ws, _scale_bound(ws), "scales")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("inter", [1, 3, 8, 33, 512, 1419, 2048, 14336, 20001])
def test_swiglu(cco, dtype, inter):
    say("case: swiglu %s inter=%d" % (dtype, inter))
    x = _x(5, 2 * inter, dtype, inter)
    q, s = cco.quant_swiglu(x.cuda())
    h = serve_ref.swiglu(x)
    want, ws = serve_ref.quant(h)
    # h is in 32 bits: 2^-20 of it (exponential, reciprocal, products)
    ops_ref.assert_within(s, ws, 2.0 ** -20 * ws + 2.0 ** -149, "scales")
    # a code may differ where the quotient is that close to a tie
    quotient = 127.0 * h / h.abs().amax(1, keepdim=True)
    assert bool(((q.cpu().double() - quotient).abs() <= 0.5 + 127 * 2.0 ** -19).all())


def test_swiglu_far_from_zero(cco):
    gate = torch.tensor([[-1e4, -200.0, -88.0, 0.0, 88.0, 200.0, 1e4, 1.0]] * 2)
    up = torch.ones(2, 8)
    up[1, 0] = math.inf  # times a silu of zero: NaN
    q, s = cco.quant_swiglu(torch.cat((gate, up), 1).cuda())
    assert float(s[0]) == pytest.approx(1e4 / 127, rel=1e-6)
    assert q[0].tolist() == [0, 0, 0, 0, 1, 3, 127, 0]
    assert math.isnan(float(s[1])) and not bool(q[1].any())


def test_strided_rows_and_scales(cco):
    x = _x(9, 300, torch.bfloat16, 1)
    wide = torch.zeros(9, 401, dtype=torch.bfloat16)
    wide[:, 3:303] = x
    out = torch.full((9, 333), 77, dtype=torch.int8, device="cuda")
    sc = torch.full((9, 5), -1.0, device="cuda")
    q, s = cco.quant_rows(wide.cuda()[:, 3:303], out=out[:, 1:301], scales=sc[:, 2])
    want, ws = serve_ref.quant(x)
    assert torch.equal(q.cpu(), want) and q.data_ptr() == out.data_ptr() + 1
    ops_ref.assert_within(sc[:, 2], ws, _scale_bound(ws), "scales")
    # what is not theirs stays
    assert bool((out[:, 0] == 77).all()) and bool((out[:, 301:] == 77).all())
    assert bool((sc[:, [0, 1, 3, 4]] == -1).all())


def test_no_rows_and_streams(cco):
    q, s = cco.quant_rows(torch.empty(0, 64, device="cuda"))
    assert q.shape == (0, 64) and s.shape == (0,)
    x = _x(300, 256, torch.float16, 2).cuda()
    want = cco.quant_rows(x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = cco.quant_rows(x, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_more_rows_than_one_grid(cco):
    # four rows a workgroup and 2^20 workgroups: the last rows come from the loop
    rows = (1 << 22) + 5
    x = torch.zeros(rows, 8, dtype=torch.float16, device="cuda")
    x[:, 0] = 1
    x[-5:, 3] = -2
    q, s = cco.quant_rows(x)
    assert bool((q[:-5, 0] == 127).all()) and bool((q[-5:, 3] == -127).all())
    assert bool((q[-5:, 0] == 64).all())
